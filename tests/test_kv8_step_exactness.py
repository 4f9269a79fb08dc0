"""How far a lookahead step over the paged 8-bit cache is from the same tokens
fed one at a time, in 64 bits: in a step a candidate attends to the candidates
before it as they are (bf16), one at a time they meet as stored e4m3 bytes.
Greedy decoding over that cache therefore follows a step's own logits, which are
close to those of single steps, not equal to them."""
import types

import numpy as np
import pytest
import torch

import kv8_model as M
import synth
from helpers import ensure_built
from oracle import decoder, lookahead as la

# Logits here are of order one (largest about 4); the decoder's contract with the oracle is 2e-2.
# An e4m3 rounding (2^-4) of up to N - 1 of some tens of keys: three times that at
# most.  The sequences below come to 0.030 and 0.040.
PIN = 6e-2


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


@pytest.fixture(autouse=True)
def rounded_attention(monkeypatch):
    plain = decoder.attention
    monkeypatch.setattr(decoder, "attention", lambda q, k, v, visible: bf16(plain(bf16(q), bf16(k), bf16(v), visible)))


class Slot:
    """One sequence's cache, from the definitions of kv8_model."""

    def __init__(self, dims, page, room):
        pool, n = (dims.n_layers, -(-room // page), dims.n_kv_heads), -(-room // page)
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
        self.m = M.Model(types.SimpleNamespace(
            page=page, k=z(*pool, page, dims.head_dim, dtype=torch.uint8), v=z(*pool, dims.head_dim, page, dtype=torch.uint8),
            k_scale=z(*pool, dtype=torch.float32), v_scale=z(*pool, dtype=torch.float32), table=z(1, n) - 1, lens=z(1), refs=z(n)))

    def append(self, kv):
        k, v = (bf16(np.stack([x[i] for x in kv])) for i in (0, 1))
        assert self.m.append(k, v, [k.shape[1]]) == [k.shape[1]]

    def read(self):
        m, n = self.m, int(self.m.lens[0])
        ids = m.table[0, :-(-n // m.page)]
        out = []
        for l in range(m.k.shape[0]):
            k = (M.E4M3[m.k[l, ids]] * m.k_scale[l, ids][..., None, None].astype(np.float64)).transpose(0, 2, 1, 3)
            v = (M.E4M3[m.v[l, ids]] * m.v_scale[l, ids][..., None, None].astype(np.float64)).transpose(0, 3, 1, 2)
            out.append(tuple(x.reshape(-1, *x.shape[2:])[:n] for x in (k, v)))
        return out


def one_by_one(w, slot, token, n):
    """Logits of `token` and of the n - 1 greedy tokens behind it, each fed alone and then stored."""
    out, tokens = [], []
    for _ in range(n):
        past = slot.read()
        P = len(past[0][0])
        logits, kv = decoder.forward(w, [token], np.array([P]), np.ones((1, P + 1), bool), cache=past)
        slot.append(kv)
        token = la.argmax_lowest(logits[0])
        out.append(logits[0])
        tokens.append(token)
    return out, tokens


@pytest.mark.parametrize("dims,page,n", [(synth.ModelDims(2, 512, 8, 2, 128, 1024, 2048, dtype="bf16"), 64, 60),
                                         (synth.ModelDims(2, 256, 4, 4, 64, 688, 1024, dtype="bf16"), 32, 31)])
def test_a_step_is_close_to_single_steps(dims, page, n):
    w = synth.model_weights(dims, 3, lm_head_std=1.28 / np.sqrt(dims.d_model))
    rows, worst, differs = 5, 0.0, False
    for seed in range(4):
        p = [int(t) for t in synth.uniform_tokens(n, dims.vocab, seed=20 + seed)]
        logits, kv = decoder.forward(w, p, np.arange(n), decoder.causal_mask(0, n), logit_rows=[n - 1])
        slot = Slot(dims, page, n + rows + 1)
        slot.append(kv)
        past, token = slot.read(), la.argmax_lowest(logits[0])
        single, tokens = one_by_one(w, slot, token, rows)
        step, _ = decoder.forward(w, [token] + tokens[:-1], np.arange(n, n + rows), decoder.causal_mask(n, rows), cache=past)
        assert np.abs(step[0] - single[0]).max() <= 1e-9      # the last committed token: the same keys
        err = [np.abs(a - b).max() for a, b in zip(step[1:], single[1:])]
        worst, differs = max(worst, *err), differs or max(err) > 1e-4
    print(f"worst {worst:.4f}")
    assert differs and worst <= PIN
