"""Cases that measure what a model outside this library runs around the paged
8-bit KV cache in one decoding step: projections with 4-bit weights, norms of
queries and keys with the position rotation, attention with a sliding window
and a few first tokens that stay visible, and log probabilities of the tokens.

`own` False: the operators in elementary torch operations.  True: the calls of
exact_decoding_gb300 (W4Matrix.matvec, Kv8Cache.norm_rope, Kv8Cache.attention
with window and sinks, logprobs).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # projections of one user's next token: the attention's output matrix of a 7B decoder, the smallest call
        dict(name="w4 token", op="w4", rows=1, out=4096, k=4096, group=128),
        # five users at once, the up projection of a 13B decoder: sizes that no power of two divides, finer groups
        dict(name="w4 few", op="w4", rows=5, out=13824, k=5120, group=64),
        # a full batch through the down projection of a 70B decoder: the largest matrix
        dict(name="w4 batch", op="w4", rows=16, out=8192, k=28672, group=128),
        # one user's next token late in a conversation: q, k and v of a projection in 32 bits
        dict(name="rotate token", op="rotate", seqs=1, rows=1, heads=32, kv_heads=32, hd=128, type="f32", norm=True, values=True, len=65413),
        # prompts of several users in one pass, grouped heads, a projection in 16 bits
        dict(name="rotate prompt", op="rotate", seqs=3, rows=2048, heads=64, kv_heads=8, hd=128, type="bf16", norm=True, values=False, len=5000),
        # one user's next token in an endless stream: 4 first tokens and a window of the last 4096
        dict(name="window token", op="window", seqs=1, rows=1, len=65413, heads=64, kv_heads=8, hd=128, page=128, mask="causal", ragged=False,
             N=0, W=0, G=0, window=4096, sinks=4),
        # a serving batch of single tokens, short sequences and long ones, a window of 1024
        dict(name="window batch", op="window", seqs=64, rows=1, len=8192, heads=64, kv_heads=8, hd=128, page=64, mask="causal", ragged=True,
             N=0, W=0, G=0, window=1024, sinks=4),
        # one lookahead step (N=5, W=15, G=15: 121 rows under the tree mask) that keeps 512 tokens of 2171, and none of the first
        dict(name="window step", op="window", seqs=1, rows=121, len=2171, heads=32, kv_heads=32, hd=128, page=64, mask="tree", ragged=False,
             N=5, W=15, G=15, window=512, sinks=0),
        # the last pass of a long prompt, a first page of instructions kept besides a window of 4096
        dict(name="window prompt", op="window", seqs=1, rows=256, len=16127, heads=32, kv_heads=8, hd=128, page=64, mask="causal", ragged=False,
             N=0, W=0, G=0, window=4096, sinks=64),
        # the token that was just chosen, with the alternatives that an interface shows
        dict(name="score token", op="score", rows=1, vocab=32000, pad=0, type="f32", given=1, top=5, masked=0.0),
        # the rows of a lookahead step's candidates under a grammar that forbids most tokens; 16-bit logits tie often
        dict(name="score step", op="score", rows=76, vocab=32016, pad=0, type="bf16", given=4, top=20, masked=0.7),
        # every token of a prompt (perplexity, distillation)
        dict(name="score prompt", op="score", rows=2048, vocab=32000, pad=0, type="f32", given=1, top=20, masked=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w4", "rotate", "window", "window", "score"])
    hd, page = rng.choice([64, 128, 128]), rng.choice([32, 64, 128])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        k = group * max(1, _log(rng, 256, 28672) // group)
        return dict(op=op, rows=rng.choice([1, _log(rng, 1, 16)]), out=_log(rng, 64, min(32016, (8192 * 28672) // k)), k=k, group=group)
    group = rng.choice([1, 2, 3, 4, 6, 8])
    kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    kv = max(1, min(kv, 64 // group))
    if op == "rotate":
        seqs = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, (3 * 2048 * 72) // (seqs * (group + 2) * kv * 2)))
        return dict(op=op, seqs=seqs, rows=min(rows, 8192), heads=kv * group, kv_heads=kv, hd=hd, type=rng.choice(["f32", "bf16"]),
                    norm=rng.random() < 0.8, values=rng.random() < 0.5, len=_log(rng, 1, 131072))
    if op == "window":
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
        most = min(65536, (1 << 29) // (seqs * kv * hd * 2), (1 << 27) // (rows * kv * group) * 4 // seqs)
        return dict(op=op, seqs=seqs, rows=rows, len=_log(rng, 1, max(2, most)), heads=kv * group, kv_heads=kv, hd=hd, page=page, mask=mask,
                    ragged=ragged, N=N, W=W, G=G, window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, _log(rng, 1, 256)]))
    vocab = _log(rng, 100, 150000)
    return dict(op=op, rows=_log(rng, 1, max(1, min(4096, (2048 * 32000) // vocab))), vocab=vocab, pad=rng.choice([0, 0, 5, 64]),
                type=rng.choice(["f32", "bf16"]), given=rng.choice([1, 1, 3]), top=rng.choice([0, 1, 5, 20, 32]),
                masked=rng.choice([0.0, 0.0, 0.5, 0.95]))


def _spread(most, n, ragged):
    """n lengths up to `most`: all `most`, or spread from short to long in a mixed order."""
    if not ragged:
        return [most] * n
    return [max(1, most * (1 + (i * 37 + 11) % n) // n) for i in range(n)]


def _lens(case):
    return _spread(case["len"], case["seqs"], case.get("ragged", True))


def _rows(case):
    return _spread(case["rows"], case["seqs"], case.get("ragged", True))


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
    if op == "w4":
        n = case["out"] * case["k"]
        return {"bytes": n // 2 + n // case["group"] * 2 + case["rows"] * (case["k"] * 2 + case["out"] * 4), "flops": 2 * n * case["rows"]}
    if op == "rotate":
        total, kv = sum(_rows(case)), case["kv_heads"]
        width = (case["heads"] + kv * (2 if case["values"] else 1)) * case["hd"]
        turned = (case["heads"] + kv) * case["hd"]
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": total * width * (size + 2) + (case["seqs"] + 1) * 8 + case["hd"] * 8, "flops": total * turned * 7}
    if op == "score":
        size = 4 if case["type"] == "f32" else 2
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * (case["given"] * 8 + 4 + case["top"] * 8), "flops": n * 5}
    lens, rows, nh, kv, hd = _lens(case), _rows(case), case["heads"], case["kv_heads"], case["hd"]
    w, a = case["window"], case["sinks"]
    held = pages = pairs = 0
    for n, r in zip(lens, rows):
        depth = _tree(case).sum(1).tolist() if case["mask"] == "tree" else range(1, r + 1)
        first = max(0, n + min(depth) - w)                   # the oldest cached token in any row's window
        toks = n if first <= a else min(a, n) + max(0, n - first)
        held += toks
        pages += min(-(-n // case["page"]), -(-toks // case["page"]) + 1)
        pairs += sum(min(n + d, w + a) for d in depth)
    return {"bytes": held * kv * hd * 2 + pages * kv * 8 + sum(rows) * (nh * 2 + kv * 2) * hd * 2, "flops": 4 * pairs * nh * hd}


# ------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def _pool(pages, kv, page, hd, g):
    """One layer of quantised K and V as a model's activations look: a few strong K channels, pages of different size."""
    strong = 1 + 3 * (torch.rand(1, 1, kv, 1, hd, generator=g, device="cuda") < 0.03)
    size = torch.exp(0.5 * torch.randn(1, pages, kv, generator=g, device="cuda"))[..., None, None]
    pool = {}
    for name in ("k", "v"):
        x = torch.randn(1, pages, kv, *((page, hd) if name == "k" else (hd, page)), generator=g, device="cuda")
        x = x * strong if name == "k" else x * size
        m, e = torch.frexp(x.abs().amax((-1, -2)))           # the least power of two that brings the page to 448 or less
        e = torch.where(m <= 0.875, e - 9, e - 8)
        one = torch.ones(e.shape, dtype=torch.float32, device="cuda")
        pool[name + "_scale"] = torch.ldexp(one, e)
        pool[name] = (x * torch.ldexp(one, -e)[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, st = case["op"], {"case": dict(case)}
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if own:
        import exact_decoding_gb300 as la
    if op == "w4":
        out, k, group = case["out"], case["k"], case["group"]
        # weights near 0 are the frequent ones; two to a byte, the even one in the low half
        w = torch.empty(out, k // 2, dtype=torch.uint8, device="cuda")
        for i in range(0, out, 4096):
            q = (torch.randn(min(4096, out - i), k, generator=g, device="cuda") * 2.7).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
            w[i:i + 4096] = q[:, ::2] | q[:, 1::2] << 4
        st["w"] = w
        st["scales"] = (torch.exp(0.4 * torch.randn(out, k // group, generator=g, device="cuda")) * 0.007).to(torch.bfloat16)
        # activations behind a norm, with a few strong channels
        st["x"] = (torch.randn(case["rows"], k, generator=g, device="cuda") *
                   (1 + 15 * (torch.rand(1, k, generator=g, device="cuda") < 0.01))).to(torch.bfloat16)
        st["y"] = torch.empty(case["rows"], out, dtype=torch.float32, device="cuda")
        if own:
            st["matrix"] = la.W4Matrix(w, st["scales"])
        return st
    if op == "score":
        rows, vocab = case["rows"], case["vocab"]
        # logits of a language model: a few tokens stand out, in some rows one takes nearly all
        z = torch.randn(rows, vocab + case["pad"], generator=g, device="cuda") * 2.0
        peak = torch.randint(0, vocab, (rows, 8), generator=g, device="cuda")
        z.scatter_add_(1, peak, torch.rand(rows, 8, generator=g, device="cuda") * 12 + 6 * torch.rand(rows, 1, generator=g, device="cuda"))
        if case["masked"]:
            allowed = torch.rand(rows, vocab + case["pad"], generator=g, device="cuda") >= case["masked"]
            allowed.scatter_(1, peak, True)
            allowed[:, :64] = True
            z = torch.where(allowed, z, -math.inf)
            del allowed
        st["logits"] = z.to(TYPES[case["type"]])[:, :vocab]
        pick = torch.randint(0, 8, (rows, case["given"]), generator=g, device="cuda")
        st["tokens"] = peak.gather(1, pick).to(torch.int32)
        st["out"] = (torch.empty(rows, case["given"], device="cuda"), torch.empty(rows, device="cuda"),
                     torch.empty(rows, case["top"], dtype=torch.int32, device="cuda"), torch.empty(rows, case["top"], device="cuda"))
        return st
    lens, rows, nh, kv, hd = _lens(case), _rows(case), case["heads"], case["kv_heads"], case["hd"]
    page = case.get("page", 64)
    held = [-(-n // page) for n in lens]
    st["lens"], st["row_start"] = _ints(lens), _starts(rows)
    if op == "rotate":
        # q, k and v as one projection writes them: columns of one buffer
        qkv = torch.randn(sum(rows), (nh + 2 * kv) * hd, generator=g, device="cuda").to(TYPES[case["type"]])
        gain = lambda: 1 + 0.3 * torch.randn(hd, generator=g, device="cuda")  # noqa: E731
        st["q_weight"], st["k_weight"] = (gain().to(torch.bfloat16), gain().to(torch.bfloat16)) if case["norm"] else (None, None)
        new = lambda h: torch.empty(sum(rows), h, hd, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        st["out"] = (new(nh), new(kv), new(kv)) if case["values"] else (new(nh), new(kv))
        pages, held = 1, [0] * len(lens)
        table = torch.full((len(lens), max(-(-(n + r) // page) for n, r in zip(lens, rows))), -1, dtype=torch.int32, device="cuda")
    else:
        pages = sum(held) + 3
        order, at = torch.randperm(pages, generator=g, device="cuda").to(torch.int32), 0
        table = torch.full((len(lens), max(held)), -1, dtype=torch.int32, device="cuda")
        for s, n in enumerate(held):
            table[s, :n] = order[at:at + n]
            at += n
        qkv = bf(sum(rows), (nh + 2 * kv) * hd)
        qkv[:, :nh * hd] *= 1.5
    st["table"] = table
    st["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    st.update(_pool(pages, kv, page, hd, g))
    st["q"] = qkv[:, :nh * hd].unflatten(1, (nh, hd))
    st["k_new"] = qkv[:, nh * hd:(nh + kv) * hd].unflatten(1, (kv, hd))
    st["v_new"] = qkv[:, (nh + kv) * hd:].unflatten(1, (kv, hd)) if case.get("values", True) else None
    if op == "window":
        for s, n in enumerate(lens):                       # what lies behind a sequence's last token is stale: NaN here
            if n % page:
                last = int(table[s, held[s] - 1])
                st["k"][0, last, :, n % page:] = 0x7F
                st["v"][0, last, :, :, n % page:] = 0x7F
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
    if own:
        names = ("k", "v", "k_scale", "v_scale", "table", "lens", "refs")
        st["cache"] = la.Kv8Cache(1, pages, page, kv, hd, len(lens), table.shape[1], tensors={n: st[n] for n in names})
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return {"w4": _w4, "rotate": _rotate, "window": _window, "score": _score}[st["case"]["op"]](st)


def _w4(st):
    if own:
        return st["matrix"].matvec(st["x"], out=st["y"])
    return _plain_w4(st)


def _rotate(st):
    if own:
        return st["cache"].norm_rope(st["q"], st["k_new"], st["v_new"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-5,
                                     rope_base=10000.0, row_start=st["row_start"], out=st["out"])
    return _plain_rotate(st)


def _window(st):
    if own:
        return st["cache"].attention(st["q"], st["k_new"], st["v_new"], row_start=st["row_start"], vis=st["vis"], out=st["out"],
                                     max_rows=st["max_rows"], max_len=st["max_len"], window=st["case"]["window"], sinks=st["case"]["sinks"])
    return _plain_window(st)


def _score(st):
    if own:
        import exact_decoding_gb300 as la
        return la.logprobs(st["logits"], st["tokens"], top=st["case"]["top"], out=st["out"])
    return _plain_score(st)


# ------------------------------------------------------------------ plain forms
def _plain_w4(st):
    """y = x W^T with W = (q - 8) scale, in 32 bits."""
    w, group = st["w"], st["case"]["group"]
    q = torch.stack([w & 15, w >> 4], -1).flatten(1).float() - 8
    m = (q.view(w.shape[0], -1, group) * st["scales"].float()[..., None]).flatten(1)
    return st["x"].float() @ m.T


def _plain_rotate(st):
    """Norm of each head, gain, rotation by the position (angles in 64 bits); values are only rounded."""
    hd, lens, start = st["q"].shape[2], st["lens"], st["row_start"].long()
    row = torch.arange(st["q"].shape[0], device=lens.device)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = lens[seq] + row - start[seq]
    freq = 10000.0 ** (-torch.arange(0, hd, 2, dtype=torch.float64, device=lens.device) / hd)
    angle = pos.double()[:, None] * freq
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    outs = []
    for x, gain in ((st["q"], st["q_weight"]), (st["k_new"], st["k_weight"])):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * gain.float()
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        outs.append(torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16))
    return (*outs, st["v_new"].to(torch.bfloat16)) if st["case"]["values"] else tuple(outs)


def _plain_window(st):
    """Softmax over the first `sinks` and the last `window` of a row's keys (cached tokens, then visible new rows), in 32 bits."""
    q, kn, vn, lens, start = st["q"], st["k_new"], st["v_new"], st["lens"], st["row_start"].long()
    nh, kv, hd = q.shape[1], kn.shape[1], q.shape[2]
    S, R, w, a = lens.shape[0], st["max_rows"], st["case"]["window"], st["case"]["sinks"]
    group = nh // kv
    at = st["table"].clamp(min=0).long()
    value = lambda name: st[name][0][at].view(torch.float8_e4m3fn).float() * st[name + "_scale"][0][at][..., None, None]  # noqa: E731
    k = value("k").permute(0, 2, 1, 3, 4).reshape(S, kv, -1, hd)
    v = value("v").permute(0, 2, 1, 4, 3).reshape(S, kv, -1, hd)
    j = torch.arange(k.shape[2], device=q.device)
    live = j < lens[:, None]                                                          # [S, keys]
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
    # places in a row's list of keys: cached tokens 0 .. len - 1, then its visible new rows in order
    count = see.sum(-1)                                                               # [S, R]
    first = (lens[:, None] + count - w)[..., None]                                    # the window's first place
    place = lens[:, None, None] + see.cumsum(-1) - 1
    see = see & ((place < a) | (place >= first))
    old = live[:, None, :] & ((j < a) | (j >= first))                                 # [S, R, keys]
    see, old = (x[:, :, None].expand(S, R, group, x.shape[-1]).reshape(S, 1, R * group, x.shape[-1]) for x in (see, old))
    scores = torch.cat([torch.where(old, qs @ k.transpose(2, 3), -math.inf),
                        torch.where(see, qs @ ks.transpose(2, 3), -math.inf)], -1) / math.sqrt(hd)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m > -math.inf, m, 0.0))
    o = (p[..., :k.shape[2]] @ v + p[..., k.shape[2]:] @ vs) / p.sum(-1, keepdim=True)
    o = o.view(S, kv, R, group, hd).permute(0, 2, 1, 3, 4).reshape(S, R, nh, hd)
    back = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(start[1:], back, right=True)
    return o[seq, back - start[seq]].to(torch.bfloat16)


def _plain_score(st):
    """Log softmax at the given tokens, its entropy, and the largest ones, lowest index first among equals."""
    z = st["logits"].float()
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    s = e.sum(-1, dtype=torch.float64)                       # a sum of many, and 1 and little more where one token has it all
    log_s = torch.log(s)
    entropy = log_s - torch.where(e > 0, e * d, 0.0).sum(-1, dtype=torch.float64) / s
    given = d.gather(1, st["tokens"].long()).double() - log_s[:, None]
    n = st["case"]["top"]
    ids = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :n] if n else torch.empty(z.shape[0], 0, dtype=torch.int64, device=z.device)
    best = d.gather(1, ids).double() - log_s[:, None]
    return given.float(), entropy.float(), ids.to(torch.int32), best.float()


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    global own
    asked, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = asked
    op = case["op"]
    if op == "w4":
        out, k, group = case["out"], case["k"], case["group"]
        y = torch.empty(case["rows"], out, dtype=torch.float64, device="cuda")
        x = st["x"].double()
        for i in range(0, out, 1024):                        # some rows of the matrix at a time
            b = st["w"][i:i + 1024].long()
            m = torch.empty(b.shape[0], k, dtype=torch.float64, device="cuda")
            m[:, 0::2], m[:, 1::2] = (b % 16 - 8).double(), (b // 16 - 8).double()
            m *= st["scales"][i:i + 1024].double().repeat_interleave(group, 1)
            y[:, i:i + 1024] = x @ m.T
        return y
    if op == "score":
        z = st["logits"].double()
        lp = torch.log_softmax(z, -1)
        p = lp.exp()
        entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1)
        # the n-th best: the largest logit of those left, and of its places the first
        ids = []
        left = z.clone()
        place = torch.arange(case["vocab"], device="cuda")
        for _ in range(case["top"]):
            best = left.amax(-1, keepdim=True)
            ids.append(torch.where(left == best, place, case["vocab"]).amin(-1, keepdim=True))
            left.scatter_(1, ids[-1], -math.inf)
        ids = torch.cat(ids, 1) if ids else torch.empty(case["rows"], 0, dtype=torch.int64, device="cuda")
        return lp.gather(1, st["tokens"].long()), entropy, ids.to(torch.int32), lp.gather(1, ids)
    lens, start = st["lens"].tolist(), st["row_start"].tolist()
    nh, hd = case["heads"], case["hd"]
    if op == "rotate":
        pos = torch.cat([torch.arange(n, n + b - a) for n, a, b in zip(lens, start, start[1:])]).double().cuda()
        outs = []
        for x, gain in ((st["q"], st["q_weight"]), (st["k_new"], st["k_weight"])):
            x = x.double()
            if gain is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / hd + 1e-5) * gain.double()
            y = torch.empty_like(x)
            for i in range(hd // 2):                         # the plane of dims i and i + hd / 2 turns by pos base^(-2 i / hd)
                t = pos * math.exp(-2 * i / hd * math.log(10000.0))
                turn = torch.polar(torch.ones_like(t), t)[:, None] * torch.complex(x[..., i], x[..., i + hd // 2])
                y[..., i], y[..., i + hd // 2] = turn.real, turn.imag
            outs.append(y)
        return (*outs, st["v_new"].double()) if case["values"] else tuple(outs)
    page, group, w, a = case["page"], case["heads"] // case["kv_heads"], case["window"], case["sinks"]
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
        tail = torch.ones(R, R, dtype=torch.bool).tril() if st["see"] is None else st["see"].cpu()
        see = torch.zeros(R, n + R, dtype=torch.bool)
        for i in range(R):
            keys = torch.cat([torch.arange(n), n + tail[i].nonzero()[:, 0]])          # the row's list of keys
            see[i, keys[:a]] = True
            see[i, keys[-w:]] = True
        see = see.cuda()
        for h in range(nh):
            z = st["q"][r, h].double() @ k[h // group].T / math.sqrt(hd)
            out[r, h] = torch.softmax(z.masked_fill(~see, -math.inf), -1) @ v[h // group]
    return out
