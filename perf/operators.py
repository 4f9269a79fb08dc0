"""Cases that measure the operators of the paged 8-bit KV cache: attention of
new rows over it, appending new tokens to it, and the bookkeeping of its pages
(forking, freeing, compacting).

The cache of one model: K as e4m3 bytes [layer][page][KV head][token][dim], V
transposed [layer][page][KV head][dim][token], one power-of-two scale for each
(layer, page, KV head) of K and of V, and per sequence slot a row of page
numbers and a length.  A page may belong to several sequences; refs counts how
many rows of the table name it, and a page that none names is free.

`own` False: the operators in elementary torch operations.  True: the calls of
exact_decoding_gb300.Kv8Cache.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60      # exponents that a page's scale may take


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token early in a chat, heads of a 7B decoder: the smallest call, latency is all
        dict(name="attend token short", op="attend", seqs=1, rows=1, len=117, heads=32, kv_heads=32, hd=128, page=64,
             mask="causal", ragged=False, N=0, W=0, G=0),
        # one user's next token deep in a long document, grouped heads (64 over 8): the long axis has to be split
        dict(name="attend token long", op="attend", seqs=1, rows=1, len=65413, heads=64, kv_heads=8, hd=128, page=128,
             mask="causal", ragged=False, N=0, W=0, G=0),
        # a serving batch of single tokens with lengths from a few tokens to 8192
        dict(name="attend batch", op="attend", seqs=64, rows=1, len=8192, heads=64, kv_heads=8, hd=128, page=64,
             mask="causal", ragged=True, N=0, W=0, G=0),
        # a batch of a small model: head_dim 64, small pages, short lengths
        dict(name="attend batch narrow", op="attend", seqs=48, rows=1, len=1500, heads=12, kv_heads=4, hd=64, page=32,
             mask="causal", ragged=True, N=0, W=0, G=0),
        # one lookahead step (N=5, W=15, G=15: 121 rows under the tree mask) over a 2048-token context, 32 heads
        dict(name="attend step", op="attend", seqs=1, rows=121, len=2171, heads=32, kv_heads=32, hd=128, page=64,
             mask="tree", ragged=False, N=5, W=15, G=15),
        # the last pass of a long prompt: 256 causal rows behind 16 thousand cached tokens
        dict(name="attend prompt", op="attend", seqs=1, rows=256, len=16127, heads=32, kv_heads=8, hd=128, page=64,
             mask="causal", ragged=False, N=0, W=0, G=0),
        # the tokens of one decoding step of a batch, all layers
        dict(name="append tokens", op="append", seqs=64, rows=1, len=1000, layers=32, kv_heads=8, hd=128, page=64),
        # a prompt's rows committed after its forward pass, all layers
        dict(name="append prompt", op="append", seqs=1, rows=2048, len=333, layers=40, kv_heads=8, hd=128, page=64),
        # a small model's prompt branches into a few samples, each of which then adds one token
        dict(name="branch few", op="branch", parents=1, fan=3, len=200, layers=4, kv_heads=4, hd=64, page=32),
        # a batch of prompts, each continued by several samples
        dict(name="branch batch", op="branch", parents=8, fan=7, len=2000, layers=32, kv_heads=8, hd=128, page=64),
        # a small pool after a few sequences ended
        dict(name="compact small", op="compact", pages=96, live=48, layers=4, kv_heads=4, hd=64, page=32, seqs=6),
        # a large pool, fragmented by many sequences that ended, before its upper half is given back
        dict(name="compact large", op="compact", pages=1024, live=500, layers=32, kv_heads=8, hd=128, page=64, seqs=40),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "branch", "compact"])
    hd, page = rng.choice([64, 128, 128]), rng.choice([32, 64, 128])
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 6, 8])
        kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        kv = max(1, min(kv, 64 // group))
        mask = rng.choice(["causal", "causal", "tree"])
        if mask == "tree":
            N, W, G = rng.randint(2, 6), rng.randint(1, 16), rng.randint(0, 16)
            while 1 + (W + G) * (N - 1) > 128:
                W, G = max(1, W - 1), max(0, G - 1)
            rows, seqs, ragged = 1 + (W + G) * (N - 1), 1, False
        else:
            N = W = G = 0
            rows = rng.choice([1, 1, _log(rng, 1, 256)])
            seqs, ragged = _log(rng, 1, 64), rng.random() < 0.7
        # at most about the work of the largest listed cases
        most = min(65536, (1 << 29) // (seqs * kv * hd * 2), (1 << 27) // (rows * kv * group) * 4 // seqs)
        return dict(op=op, seqs=seqs, rows=rows, len=_log(rng, 1, max(2, most)), heads=kv * group, kv_heads=kv, hd=hd, page=page,
                    mask=mask, ragged=ragged, N=N, W=W, G=G)
    if op == "append":
        layers, kv, seqs = _log(rng, 1, 40), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, 2048 // seqs))
        return dict(op=op, seqs=seqs, rows=rows, len=_log(rng, 1, 1000), layers=layers, kv_heads=kv, hd=hd, page=page)
    if op == "branch":
        return dict(op=op, parents=rng.randint(1, 8), fan=rng.randint(1, 7), len=_log(rng, 1, 2000), layers=_log(rng, 1, 32),
                    kv_heads=rng.choice([1, 2, 4, 8]), hd=hd, page=min(page, 64))
    pages = _log(rng, 24, 1024)
    return dict(op=op, pages=pages, live=rng.randint(8, max(9, pages // 2)), layers=_log(rng, 1, 32),
                kv_heads=rng.choice([1, 2, 4, 8]), hd=hd, page=min(page, 64), seqs=rng.randint(2, 8))


def _spread(most, n, ragged):
    """n lengths up to `most`: all `most`, or spread from short to long in a mixed order."""
    if not ragged:
        return [most] * n
    return [max(1, most * (1 + (i * 37 + 11) % n) // n) for i in range(n)]


def _lens(case):
    return _spread(case["len"], case["seqs"], case.get("ragged", True))


def _rows(case):
    if case["op"] == "append":
        return _spread(case["rows"], case["seqs"], case["seqs"] > 1 and case["rows"] > 1)
    return _spread(case["rows"], case["seqs"], case["ragged"])


def _parents(N, W, G):
    """Parent of each row of a lookahead step (row 0: the last token; W columns of N-1 levels; G candidates)."""
    L, par = N - 1, [-1]
    for k in range(L):
        par += [(0 if j == 0 else len(par) + j - 1) if k == 0 else len(par) + j - W for j in range(W)]
    for _ in range(G):
        base = len(par)
        par += [0 if m == 0 else base + m - 1 for m in range(L)]
    return par


def _tree(case):
    """Visible rows of each row, as truth values [rows][rows]."""
    par = _parents(case["N"], case["W"], case["G"])
    see = torch.zeros(len(par), len(par), dtype=torch.bool)
    for r in range(len(par)):
        x = r
        while x >= 0:
            see[r, x] = True
            x = par[x]
    return see


def work(case):
    op = case["op"]
    if op == "attend":
        lens, rows = _lens(case), _rows(case)
        nh, kv, hd = case["heads"], case["kv_heads"], case["hd"]
        pages = sum(-(-n // case["page"]) for n in lens)
        seen = _tree(case).sum().item() if case["mask"] == "tree" else sum(r * (r + 1) // 2 for r in rows)
        pairs = sum(n * r for n, r in zip(lens, rows)) + seen
        return {"bytes": sum(lens) * kv * hd * 2 + pages * kv * 8 + sum(rows) * (nh * 2 + kv * 2) * hd * 2, "flops": 4 * pairs * nh * hd}
    width = case["layers"] * case["kv_heads"] * case["hd"] * 2      # bytes of one stored token
    if op == "append":
        return {"bytes": 3 * sum(_rows(case)) * width, "flops": 2 * sum(_rows(case)) * width}
    if op == "branch":
        kids = case["parents"] * case["fan"]
        # each child copies the stored tokens of its last page and adds one of its own
        return {"bytes": kids * (2 * (case["len"] % case["page"]) + 3) * width, "flops": kids * width}
    holes = sum(1 for p in _live_pages(case) if p >= case["live"])
    return {"bytes": 2 * holes * case["page"] * width + 8 * case["pages"], "flops": 0}


def _live_pages(case):
    """Which pages of a fragmented pool are in use: spread over all of it."""
    return sorted(i * case["pages"] // case["live"] for i in range(case["live"]))


# ------------------------------------------------------------------ inputs
def _exponent(amax):
    """Exponent of the smallest power-of-two scale that brings `amax` to 448 or less."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _power(e):
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float32, device=e.device), e)


def _byte(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(b):
    return b.view(torch.float8_e4m3fn).float()


def _filled(layers, pages, kv, page, hd, g):
    """A pool of quantised K and V as a model's activations look: a few strong K channels, pages of different size."""
    shape = (layers, pages, kv)
    strong = 1 + 3 * (torch.rand(layers, 1, kv, 1, hd, generator=g, device="cuda") < 0.03)
    size = torch.exp(0.5 * torch.randn(*shape, generator=g, device="cuda"))[..., None, None]
    pool = {}
    for name in ("k", "v"):
        b = torch.empty(*shape, *((page, hd) if name == "k" else (hd, page)), dtype=torch.uint8, device="cuda")
        s = torch.empty(shape, dtype=torch.float32, device="cuda")
        for layer in range(layers):
            x = torch.randn(*b.shape[1:], generator=g, device="cuda")
            x = x * strong[layer] if name == "k" else x * size[layer]
            e = _exponent(x.abs().amax((-1, -2)))
            s[layer] = _power(e)
            b[layer] = _byte(x * _power(-e)[..., None, None])
        pool[name], pool[name + "_scale"] = b, s
    return pool


def _numbers(rows_of, total, max_pages, g):
    """Table and reference counts where sequence s holds rows_of[s] pages, dealt out in a random order of `total`."""
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(rows_of), max_pages), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(total, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(rows_of):
        table[s, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    return table, refs


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, kv, hd, page = case["op"], case["kv_heads"], case["hd"], case["page"]
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = {"case": dict(case)}
    if op == "attend":
        lens, rows = _lens(case), _rows(case)
        held = [-(-n // page) for n in lens]
        st["table"], st["refs"] = _numbers(held, sum(held) + 3, max(held), g)
        st.update(_filled(1, sum(held) + 3, kv, page, hd, g))
        st["lens"], st["row_start"] = _ints(lens), _starts(rows)
        for s, n in enumerate(lens):                       # what lies behind a sequence's last token is stale: NaN here
            if n % page:
                last = int(st["table"][s, held[s] - 1])
                st["k"][0, last, :, n % page:] = 0x7F
                st["v"][0, last, :, :, n % page:] = 0x7F
        # q, k and v of the new rows as one projection writes them: columns of one buffer
        qkv = bf(sum(rows), (case["heads"] + 2 * kv) * hd)
        nh = case["heads"]
        qkv[:, :nh * hd] *= 1.5
        st["q"] = qkv[:, :nh * hd].unflatten(1, (nh, hd))
        st["k_new"] = qkv[:, nh * hd:(nh + kv) * hd].unflatten(1, (kv, hd))
        st["v_new"] = qkv[:, (nh + kv) * hd:].unflatten(1, (kv, hd))
        st["vis"], st["see"] = None, None
        if case["mask"] == "tree":
            see = _tree(case)
            words = torch.zeros(see.shape[0], 256, dtype=torch.int64)
            words[:, :see.shape[0]] = see
            words = (words.view(-1, 8, 32) << torch.arange(32)).sum(-1)
            st["vis"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()
            st["see"] = see.cuda()
        st["out"] = torch.empty(sum(rows), nh, hd, dtype=torch.bfloat16, device="cuda")
        st["max_rows"], st["max_len"] = max(rows), max(lens)
    elif op == "append":
        lens, rows = _spread(case["len"], case["seqs"], case["seqs"] > 1), _rows(case)
        held, most = [-(-n // page) for n in lens], max(-(-(n + r) // page) for n, r in zip(lens, rows))
        total = sum(-(-(n + r) // page) for n, r in zip(lens, rows)) + 5
        st["table"], st["refs"] = _numbers(held, total, most, g)
        st.update(_filled(case["layers"], total, kv, page, hd, g))
        st["lens"], st["keep"], st["row_start"] = _ints(lens), _ints(lens), _starts(rows)
        st["slots"] = torch.arange(len(lens), dtype=torch.int32, device="cuda")
        st["k_new"], st["v_new"] = bf(case["layers"], sum(rows), kv, hd), bf(case["layers"], sum(rows), kv, hd)
        st["max_rows"] = max(rows)
    elif op == "branch":
        # slots: the parents, then `fan` children of each; the children hold last round's branches
        n, fan, P = case["len"], case["fan"], case["parents"]
        lens = [max(1, n - 3 * p) for p in range(P)]
        held = [-(-x // page) for x in lens]
        total, most = sum(held) + 2 * P * fan + 3, -(-(n + 1) // page)
        table, refs = _numbers(held + [0] * (P * fan), total, most, g)
        st.update(_filled(case["layers"], total, kv, page, hd, g))
        st["src"] = torch.arange(P, dtype=torch.int32, device="cuda").repeat_interleave(fan)
        st["dst"] = torch.arange(P, P + P * fan, dtype=torch.int32, device="cuda")
        st["table"], st["refs"] = table, refs
        st["lens"] = _ints(lens + [0] * (P * fan))
        st["slots"] = st["dst"]
        st["row_start"] = _starts([0] * P + [1] * (P * fan))
        st["k_new"], st["v_new"] = bf(case["layers"], P * fan, kv, hd), bf(case["layers"], P * fan, kv, hd)
        st["max_rows"] = 1
    else:
        live, S = _live_pages(case), case["seqs"]
        pages = torch.tensor(live, device="cuda")[torch.randperm(len(live), generator=g, device="cuda")].to(torch.int32)
        share = pages[:2]                                   # a prefix that every sequence shares
        per = -(-(len(live) - len(share)) // S)
        st["table"] = torch.full((S, per + 2), -1, dtype=torch.int32, device="cuda")
        st["table"][:, :2] = share
        rest = pages[2:]
        for s in range(S):
            own_pages = rest[s * per:(s + 1) * per]
            st["table"][s, 2:2 + len(own_pages)] = own_pages
        named = st["table"][st["table"] >= 0].long()
        st["refs"] = torch.bincount(named, minlength=case["pages"]).to(torch.int32)
        st["lens"] = ((st["table"] >= 0).sum(1) * page - 1).to(torch.int32)
        st.update(_filled(case["layers"], case["pages"], kv, page, hd, g))
        st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
    if own:
        import exact_decoding_gb300 as la
        names = ("k", "v", "k_scale", "v_scale", "table", "lens", "refs")
        st["cache"] = la.Kv8Cache(st["k"].shape[0], st["k"].shape[1], page, kv, hd, st["table"].shape[0], st["table"].shape[1],
                                  tensors={n: st[n] for n in names})
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return {"attend": _attend, "append": _append, "branch": _branch, "compact": _compact}[st["case"]["op"]](st)


def _attend(st):
    if own:
        return st["cache"].attention(st["q"], st["k_new"], st["v_new"], row_start=st["row_start"], vis=st["vis"], out=st["out"],
                                     max_rows=st["max_rows"], max_len=st["max_len"])
    return _plain_attend(st)


def _append(st):
    if own:
        st["cache"].free(st["slots"], keep=st["keep"])
        st["cache"].append(st["k_new"], st["v_new"], row_start=st["row_start"], max_rows=st["max_rows"])
    else:
        _plain_free(st, st["slots"], st["keep"])
        _plain_append(st, st["slots"])
    return _cache_of(st)


def _branch(st):
    if own:
        st["cache"].free(st["dst"])
        st["cache"].fork(st["src"], st["dst"])
        st["cache"].append(st["k_new"], st["v_new"], row_start=st["row_start"], max_rows=st["max_rows"])
    else:
        _plain_free(st, st["dst"], torch.zeros_like(st["dst"]))
        _plain_fork(st)
        _plain_append(st, st["slots"])
    return _cache_of(st)


def _compact(st):
    if own:
        live = st["cache"].compact(table_out=st["table_out"], refs_out=st["refs_out"])
    else:
        live = _plain_compact(st)
    return {"live": live, "table": st["table_out"], "refs": st["refs_out"], **_pool_of(st)}


def _pool_of(st):
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn), "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _cache_of(st):
    return {"table": st["table"], "lens": st["lens"], "refs": st["refs"], **_pool_of(st)}


# ------------------------------------------------------------------ plain forms
def _plain_attend(st):
    """Softmax over a sequence's cached tokens and its visible new rows, in 32 bits."""
    q, kn, vn, lens, start = st["q"], st["k_new"], st["v_new"], st["lens"], st["row_start"].long()
    nh, kv, hd, page = q.shape[1], kn.shape[1], q.shape[2], st["k"].shape[3]
    S, R = lens.shape[0], st["max_rows"]
    group = nh // kv
    at = st["table"].clamp(min=0).long()
    k = _value(st["k"][0][at]) * st["k_scale"][0][at][..., None, None]                # [S, pages, kv, page, hd]
    v = _value(st["v"][0][at]) * st["v_scale"][0][at][..., None, None]                # [S, pages, kv, hd, page]
    k = k.permute(0, 2, 1, 3, 4).reshape(S, kv, -1, hd)
    v = v.permute(0, 2, 1, 4, 3).reshape(S, kv, -1, hd)
    live = torch.arange(k.shape[2], device=q.device) < lens[:, None]                  # [S, keys]
    k = torch.where(live[:, None, :, None], k, 0.0)
    v = torch.where(live[:, None, :, None], v, 0.0)
    # the new rows of every sequence, padded to R
    i = torch.arange(R, device=q.device)
    row = start[:-1, None] + i
    there = row < start[1:, None]                                                     # [S, R]
    row = row.clamp(max=q.shape[0] - 1)
    qs = q[row].float().view(S, R, kv, group, hd).permute(0, 2, 1, 3, 4).reshape(S, kv, R * group, hd)
    ks, vs = (x[row].float().permute(0, 2, 1, 3) for x in (kn, vn))
    see = i[:, None] >= i if st["see"] is None else st["see"]
    see = see & there[:, None, :] & there[:, :, None]                                 # [S, R, R]
    see = see[:, :, None].expand(S, R, group, R).reshape(S, 1, R * group, R)
    scores = torch.cat([torch.where(live[:, None, None], qs @ k.transpose(2, 3), -math.inf),
                        torch.where(see, qs @ ks.transpose(2, 3), -math.inf)], -1) / math.sqrt(hd)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m > -math.inf, m, 0.0))
    o = (p[..., :k.shape[2]] @ v + p[..., k.shape[2]:] @ vs) / p.sum(-1, keepdim=True)
    o = o.view(S, kv, R, group, hd).permute(0, 2, 1, 3, 4).reshape(S, R, nh, hd)
    back = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(start[1:], back, right=True)
    return o[seq, back - start[seq]].to(torch.bfloat16)


def _plain_free(st, slots, keep):
    """The sequences keep their first `keep` tokens; pages behind them lose a reference."""
    table, page, s = st["table"], st["k"].shape[3], slots.long()
    keep = torch.minimum(keep, st["lens"][s])
    rows = table[s]
    gone = (rows >= 0) & (torch.arange(table.shape[1], device=table.device) >= ((keep + page - 1) // page)[:, None])
    st["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    table[s] = torch.where(gone, -1, rows)
    st["lens"][s] = keep


def _plain_fork(st):
    """The children name their parents' pages."""
    rows = st["table"][st["src"].long()]
    st["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    st["table"][st["dst"].long()] = rows
    st["lens"][st["dst"].long()] = st["lens"][st["src"].long()]


def _plain_append(st, slots):
    """New tokens behind the sequences `slots`, each of which gets at least one row."""
    table, refs, start, s = st["table"], st["refs"], st["row_start"].long(), slots.long()
    page, kn, vn = st["k"].shape[3], st["k_new"], st["v_new"]
    layers, total, kv, hd = kn.shape
    lens, n = st["lens"][s].long(), start[s + 1] - start[s]
    # pages: the lowest free ones, in the order of the sequences; a shared last page is replaced by a copy
    first, held, want = lens // page, (lens + page - 1) // page, (lens + n + page - 1) // page
    old = table[s, first.clamp(max=table.shape[1] - 1)].clamp(min=0).long()
    part = lens % page > 0
    copy = part & (refs[old] > 1)
    take = want - held + copy.long()
    free = torch.argsort((refs > 0).to(torch.int32), stable=True)
    begin, base = torch.where(copy, first, held), torch.cumsum(take, 0) - take
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= begin[:, None]) & (col < want[:, None])
    ids = free[(base[:, None] + col - begin[:, None]).clamp(0, refs.shape[0] - 1)]
    rows = torch.where(fresh, ids, table[s].long())
    refs.index_add_(0, ids.flatten(), fresh.flatten().to(torch.int32))
    refs.index_add_(0, old, -copy.to(torch.int32))
    table[s] = rows.to(torch.int32)
    st["lens"][s] = (lens + n).to(torch.int32)
    # where every row goes
    every = torch.arange(total, device=table.device)
    which = torch.searchsorted(start[s + 1], every, right=True)
    pos = lens[which] + every - start[s][which]
    touched = -(-st["max_rows"] // page) + 1
    group = which * touched + pos // page - first[which]
    to, off = rows[which, pos // page], pos % page
    fresh_first = rows.gather(1, first[:, None])[:, 0]
    kept = (torch.arange(page, device=table.device) < (lens % page)[:, None])         # [S, page]
    for name, new in (("k", kn), ("v", vn)):
        pool, scale = st[name], st[name + "_scale"]
        x = new.float()
        most = torch.zeros(layers, kv, len(s) * touched, device=x.device)
        most.scatter_reduce_(2, group.expand(layers, kv, total), x.abs().amax(-1).transpose(1, 2), "amax")
        e = _exponent(most)
        was = torch.frexp(scale[:, old])[1] - 1                                      # [layers, S, kv]
        lead = e.view(layers, kv, len(s), touched)
        lead[..., 0] = torch.maximum(lead[..., 0], torch.where(part[:, None], was, MIN_EXP).transpose(1, 2))
        # the stored tokens of the first page, at the new scale and in its new place
        shrink = _power(was - lead[..., 0].transpose(1, 2))[..., None, None]
        keep = kept[:, None, :, None] if name == "k" else kept[:, None, None, :]
        moved = _byte(_value(pool[:, old]) * shrink)
        pool[:, fresh_first] = torch.where(keep, moved, pool[:, fresh_first])
        scale[:, to] = _power(e[:, :, group]).transpose(1, 2)
        b = _byte(x * _power(-e[:, :, group]).transpose(1, 2)[..., None])            # [layers, rows, kv, hd]
        if name == "k":
            pool[:, to, :, off] = b.transpose(0, 1)
        else:
            pool[:, to, :, :, off] = b.transpose(0, 1)


def _plain_compact(st):
    """Pages in use above the number of them move into the free ones below it, lowest to lowest."""
    used = st["refs"] > 0
    live = used.sum()
    number = torch.arange(used.shape[0], device=used.device)
    src, dst = (used & (number >= live)).nonzero()[:, 0], (~used & (number < live)).nonzero()[:, 0]
    to = number.to(torch.int32)
    to[src] = dst.to(torch.int32)
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name][:, dst] = st[name][:, src]
    st["table_out"].copy_(torch.where(st["table"] >= 0, to[st["table"].clamp(min=0).long()], -1))
    st["refs_out"].copy_(st["refs"])
    st["refs_out"][dst] = st["refs"][src]
    st["refs_out"][src] = 0
    return live.to(torch.int32).view(1)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_scale(amax):
    """2^e with the least e in [-60, 60] for which amax <= 448 * 2^e."""
    s = torch.full_like(amax, 2.0 ** MIN_EXP)
    for e in range(MIN_EXP + 1, MAX_EXP + 1):
        s = torch.where(amax > E4M3_MAX * 2.0 ** (e - 1), 2.0 ** e, s)
    return s


def _exact_e4m3(x):
    """Nearest e4m3 value (3 fraction bits, least exponent -6), ties to even, magnitudes up to 448."""
    step = torch.full_like(x, 2.0 ** -9)
    for e in range(-5, 9):
        step = torch.where(x.abs() >= 2.0 ** e, 2.0 ** (e - 3), step)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    if case["op"] == "compact":
        return None                                        # nothing is computed: numbers and bytes move
    global own
    asked, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = asked
    page, lens, start = case["page"], st["lens"].tolist(), st["row_start"].tolist()
    if case["op"] == "attend":
        group = case["heads"] // case["kv_heads"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for s, n in enumerate(lens):
            mine = st["table"][s, :-(-n // page)].long()
            ks, vs = (st[x + "_scale"][0, mine].double()[..., None, None] for x in "kv")
            k = (st["k"][0, mine].view(torch.float8_e4m3fn).double() * ks).transpose(0, 1).flatten(1, 2)[:, :n]
            v = (st["v"][0, mine].view(torch.float8_e4m3fn).double() * vs).permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
            r = slice(start[s], start[s + 1])
            k = torch.cat([k, st["k_new"][r].double().transpose(0, 1)], 1)
            v = torch.cat([v, st["v_new"][r].double().transpose(0, 1)], 1)
            R = start[s + 1] - start[s]
            tail = torch.ones(R, R, dtype=torch.bool, device="cuda").tril() if st["see"] is None else st["see"]
            see = torch.cat([torch.ones(R, n, dtype=torch.bool, device="cuda"), tail], 1)
            for h in range(case["heads"]):
                z = st["q"][r, h].double() @ k[h // group].T / math.sqrt(case["hd"])
                out[r, h] = torch.softmax(z.masked_fill(~see, -math.inf), -1) @ v[h // group]
        return out
    # append and branch: the pool after one pass; table, lens and refs are whole numbers
    names = ("k", "v", "k_scale", "v_scale")
    got = {x: (st[x].view(torch.float8_e4m3fn) if x in "kv" else st[x]).double() for x in names}
    table, refs = st["table"].tolist(), st["refs"].tolist()
    if case["op"] == "branch":
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            table[b], lens[b] = list(table[a]), lens[a]
            for p in table[a]:
                if p >= 0:
                    refs[p] += 1
    shared = [c > 1 for c in refs]
    unused = iter([p for p, c in enumerate(refs) if c == 0])
    for s in range(len(lens)):
        r, done = start[s], 0
        while r + done < start[s + 1]:
            pos = lens[s] + done
            j, o = divmod(pos, page)
            n = min(page - o, start[s + 1] - r - done)
            was = table[s][j] if o else -1
            to = was if o and not shared[was] else next(unused)
            table[s][j] = to
            rows = slice(r + done, r + done + n)
            for x, new in (("k", st["k_new"]), ("v", st["v_new"])):
                y = new[:, rows].double().transpose(1, 2)                            # [layers, kv, n, hd]
                scale = _exact_scale(y.abs().amax((2, 3)))
                if o:
                    prev = got[x + "_scale"][:, was]
                    scale = torch.maximum(scale, prev)
                    oldv = got[x][:, was] * (prev / scale)[..., None, None]
                    if x == "k":
                        got[x][:, to, :, :o] = _exact_e4m3(oldv[:, :, :o])
                    else:
                        got[x][:, to, :, :, :o] = _exact_e4m3(oldv[..., :o])
                b = _exact_e4m3(y / scale[..., None, None])
                if x == "k":
                    got[x][:, to, :, o:o + n] = b
                else:
                    got[x][:, to, :, :, o:o + n] = b.transpose(2, 3)
                got[x + "_scale"][:, to] = scale
            done += n
    return {"table": None, "lens": None, "refs": None, **got}
