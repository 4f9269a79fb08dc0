"""Attention over the paged 8-bit KV cache where values lie many binades apart,
against the plain 64-bit form: what a row does not see, or gives no weight,
must not cost it any bits."""
import numpy as np
import pytest

import kv8_model as M
from test_gpu_kv8 import build, lib, normal, starts, tree_words  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [0, 1])          # many and few query vectors' kernel: max_rows never changes the result
@pytest.mark.parametrize("size", [1e9, 1e12, 1e30, 3e38])
@pytest.mark.parametrize("rows,hd,tree,what", [(40, 128, True, "v"), (40, 128, False, "k"), (121, 128, True, "k"), (121, 64, False, "v"),
                                               (300, 64, False, "k"), (300, 128, False, "v"), (40, 64, True, "kv")])
def test_unseen_rows_of_any_size_do_not_leak(lib, rows, hd, tree, what, size, hint):
    """A huge finite K or V, in a row that most rows do not see, changes nothing in those."""
    import torch
    cache = build(lib, [70, 0, 260], hd, 64, 2)
    counts = [rows, 3, 5]
    n = sum(counts)
    q, k, v = normal((n, 4, hd), 1), normal((n, 2, hd), 2), normal((n, 2, hd), 3)
    big = [2, rows // 2] if tree else [rows - 2]
    for b in big:
        for x, name in ((k, "k"), (v, "v")):
            if name in what:
                x[b, 0, 5] = size
                x[b, 1] = torch.where(x[b, 1] > 0, size, -size)
    see = [[j for j in range(r + 1) if j < 256 and (j not in big or j == r)] for r in range(rows)] if tree else [list(range(r + 1)) for r in range(rows)]
    see += [list(range(r + 1)) for c in counts[1:] for r in range(c)]
    first = np.concatenate([[0], np.cumsum(counts)])
    vis = torch.from_numpy(tree_words(see)).cuda() if tree else None
    out = cache.attention(q, k, v, row_start=starts(counts), vis=vis, max_rows=hint)
    cache.status()
    blind = [r for r in range(n) if r >= rows or not set(see[r]) & set(big)]
    assert len(blind) >= n - len(big) - 2
    want, tol = M.attention(cache, q, k, v, counts, see=lambda s, r: see[first[s] + r])
    got = out.cpu().double().numpy()
    err = np.abs(got - want)[blind] / tol[blind]
    assert np.all(err <= 1), f"worst {np.nanmax(err):.3g} of the tolerance, {np.isnan(err).sum()} NaN"
