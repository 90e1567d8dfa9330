"""The training side of the block-sparse attention as it is measured: cases, inputs, plain forms, 64-bit values.

  tables  rotary_tables         cosines and sines of the positions, frequencies stretched for
                                long contexts
  rotate  rotary_embed          queries and keys turned by their positions, or gradients turned
                                back
  grad    blocksparse_attn_bwd  gradients of attention over SparseMask block bounds

Where ``own`` is false ``run`` computes the operator with elementary torch operations in 32
bits (angles in 64); where it is true it makes the library's calls.  The documents of a row
follow from the case, all values from the seed.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
QB = 128  # query block of the bounds


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the tables of a short context: latency only
        dict(name="tables 2k", op="tables", n=2048, rot=64, factor=1.0, original=0, amplitude=1.0),
        # a long context, low frequencies stretched and high ones kept, heads wholly rotated
        dict(name="tables 128k", op="tables", n=131072, rot=128, factor=8.0, original=16384, amplitude=1.2),
        # one short 32-bit row: latency only
        dict(name="rotate tiny", op="rotate", B=1, T=256, Hq=4, Hkv=1, D=64, rot=64, pairs=False,
             inverse=False, f32=True, sliced=False, doc=0, pad=0),
        # packed documents of an odd number of tokens, parts of one projection's output, half
        # of each head turned in neighbouring pairs
        dict(name="rotate packed", op="rotate", B=1, T=3001, Hq=16, Hkv=4, D=64, rot=32, pairs=True,
             inverse=False, f32=False, sliced=True, doc=400, pad=9),
        # a training batch ahead of the attention
        dict(name="rotate batch", op="rotate", B=4, T=16384, Hq=32, Hkv=8, D=128, rot=128, pairs=False,
             inverse=False, f32=False, sliced=True, doc=2048, pad=300),
        # gradients of a long batch on their way back to the projection
        dict(name="rotate gradients", op="rotate", B=2, T=8192, Hq=64, Hkv=4, D=128, rot=128, pairs=True,
             inverse=True, f32=False, sliced=False, doc=0, pad=0),
        # a short row of small documents: latency only
        dict(name="grad tiny", op="grad", B=1, T=256, Hq=4, Hkv=2, D=64, kb=64, doc=90, pad=11,
             causal=True, left=-1, right=-1),
        # a few documents behind a window
        dict(name="grad small", op="grad", B=2, T=1024, Hq=4, Hkv=2, D=128, kb=64, doc=300, pad=70,
             causal=True, left=256, right=0),
        # heads of 64, an odd number of them for each KV head, both sides of a token in view
        dict(name="grad both sides", op="grad", B=2, T=4096, Hq=12, Hkv=4, D=64, kb=128, doc=900, pad=0,
             causal=False, left=500, right=300),
        # one long document, all of the past in view
        dict(name="grad long", op="grad", B=1, T=8192, Hq=16, Hkv=4, D=128, kb=128, doc=0, pad=77,
             causal=True, left=-1, right=-1),
        # a training batch of packed documents behind a window of 1024
        dict(name="grad batch", op="grad", B=4, T=16384, Hq=32, Hkv=8, D=128, kb=128, doc=2048, pad=300,
             causal=True, left=1024, right=0),
    ]


def draw(rng):
    op = rng.choice(["tables", "rotate", "rotate", "grad", "grad", "grad"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    if op == "tables":
        n = log(1, 131072)
        factor = rng.choice([1.0, 1.0, 2.0, 8.0, 31.5])
        return dict(op=op, n=n, rot=16 * rng.randint(1, 8), factor=factor,
                    original=rng.choice([0, 2048, 16384]) if factor > 1 else 0,
                    amplitude=rng.choice([1.0, 1.0, 1.0 + 0.1 * math.log(factor)]))
    if op == "rotate":
        D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
        T = log(1, 16384)
        f32 = rng.random() < 0.3
        Hq = Hkv * rng.choice([1, 3, 4, 8])
        most = (4 if not f32 else 2) * 16384 * 40 * 128 // (T * (Hq + Hkv) * D)
        return dict(op=op, B=log(1, max(1, min(16, most))), T=T, Hq=Hq, Hkv=Hkv, D=D, rot=16 * rng.randint(1, D // 16),
                    pairs=rng.random() < 0.5, inverse=rng.random() < 0.4, f32=f32, sliced=rng.random() < 0.5,
                    doc=rng.choice([0, 50, 700]), pad=rng.choice([0, 0, min(T // 2, 13)]))
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, B=1, T=QB * log(1, 128), Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv, D=D,
             kb=rng.choice([64, 128]), causal=rng.random() < 0.7)
    c["doc"] = rng.choice([0, 40, log(20, 4000)])
    c["pad"] = rng.choice([0, rng.randint(1, min(500, c["T"] // 2))])
    c["left"] = rng.choice([-1, log(1, 3000), 1024])
    c["right"] = rng.choice([-1, 0, log(1, 500)])
    cost = lambda: c["B"] * c["Hq"] * c["T"] * _width(c)  # noqa: E731
    while cost() > 1.2e9 and c["left"] != 512:
        c.update(left=512, right=min(c["right"], 512) if c["right"] >= 0 else 0)
    while cost() > 1.2e9 and c["T"] > QB:
        c["T"] = max(QB, c["T"] // 2 // QB * QB)
        c["pad"] = min(c["pad"], c["T"] // 2)
    most = int(1.2e9 // max(1, cost()))
    c["B"] = log(1, max(1, min(8, most)))
    return c


# ------------------------------------------------------------------ structure of a case
def _segments(case):
    """Documents of the rows: ids [B, T], -1 for the padded end.  Lengths from a hundredth of
    the mean to four times it."""
    B, T, real = case["B"], case["T"], case["T"] - case["pad"]
    seg = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        seg[b, :real] = 0
        if case["doc"]:
            u = np.modf(0.37 * (b + 1) + 0.6180339887 * np.arange(1, 100 * real // case["doc"] + 2))[0]
            ends = np.cumsum(np.ceil(-np.log1p(-u * 0.98) * case["doc"] + 0.01 * case["doc"]).astype(np.int64))
            seg[b, :real] = np.searchsorted(ends, np.arange(real), side="right")
    return seg


def _sides(case):
    """(tokens in view before, after) a token; None for all."""
    left = case["left"] if case["left"] >= 0 else None
    right = case["right"] if case["right"] >= 0 else None
    if case["causal"]:
        right = 0
    return left, right


def _views(case):
    """First and last key of each token's view [B, T] (last < first: none)."""
    seg = _segments(case)
    B, T = seg.shape
    left, right = _sides(case)
    t = np.arange(T)
    first, last = np.zeros((B, T), dtype=np.int64), np.full((B, T), -1, dtype=np.int64)
    for b in range(B):
        cut = np.flatnonzero(np.diff(seg[b])) + 1
        begin, end = np.r_[0, cut], np.r_[cut, T] - 1
        of = np.searchsorted(begin, t, side="right") - 1
        first[b] = begin[of] if left is None else np.maximum(begin[of], t - left)
        last[b] = end[of] if right is None else np.minimum(end[of], t + right)
        first[b, seg[b] < 0], last[b, seg[b] < 0] = 0, -1
    return first, last


def _bounds(case):
    """Block bounds [B, NB]: key blocks in view of some token, and those in view of all."""
    first, last = _views(case)
    B, T = first.shape
    kb = case["kb"]
    f, z = first.reshape(B, -1, QB), last.reshape(B, -1, QB)
    some = z >= f
    lo = np.where(some, f, T).min(-1) // kb
    up = np.where(some, z, -1).max(-1) // kb + 1
    lo, up = np.where(some.any(-1), lo, 0), np.where(some.any(-1), up, 0)
    full_lo = -(-f.max(-1) // kb)
    full_up = (z.min(-1) + 1) // kb
    none = ~some.all(-1) | (full_up <= full_lo)
    return lo, up, np.where(none, T // kb, full_lo), np.where(none, 0, full_up)


def _width(case):
    """Keys that the widest query block goes over."""
    lo, up, _, _ = _bounds(case)
    return max(1, int((up - lo).max())) * case["kb"]


def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + what) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, seed, what, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, what), device=DEV, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    c = case
    if c["op"] == "tables":
        # the base that a model was trained with, or was moved to
        return dict(case=c, base=1e4 * (1 + 99 * float(torch.rand((), generator=torch.Generator().manual_seed(int(seed) & 0xFFFFFFFF)))))
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    seg = _segments(c)
    if c["op"] == "rotate":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        parts = _randn((B, T, (Hq + 2 * Hkv) * D), seed, 1, dtype)  # one projection's output
        q, k = parts[..., :Hq * D].unflatten(-1, (Hq, D)), parts[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        pos = np.arange(T) - np.stack([np.r_[0, np.flatnonzero(np.diff(s)) + 1][np.r_[0, np.cumsum(np.diff(s) != 0)]] for s in seg])
        pos[seg < 0] = -1                                           # padding stays as it is
        n = max(1, int(pos.max()) + 1)
        turn = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        whole = not c["doc"] and not c["pad"]
        return dict(case=c, q=q if c["sliced"] else q.contiguous(), k=k if c["sliced"] else k.contiguous(),
                    cos=turn.cos().float(), sin=turn.sin().float(),
                    pos=None if whole else torch.from_numpy(pos.astype(np.int32)).to(DEV))
    st = dict(case=c, width=_width(c))
    for i, (name, heads) in enumerate((("q", Hq), ("k", Hkv), ("v", Hkv), ("do", Hq))):
        st[name] = _randn((B, T, heads, D), seed, 10 + i, torch.bfloat16)
    at = np.broadcast_to(np.arange(T, dtype=np.int32), (B, T)).copy()
    st["pos"], st["seg"] = torch.from_numpy(at).to(DEV), torch.from_numpy(seg).to(DEV)
    st["bounds"] = [torch.from_numpy(x.astype(np.int32)[:, None]).to(DEV) for x in _bounds(c)]
    # what the forward pass left
    q, k, v, key, see = _blocks(st)
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).masked_fill_(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = s.sub_(torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None]).exp_()
    st["out"], st["lse"] = _tokens(p @ v, c).to(torch.bfloat16), _tokens(lse[..., None], c)[..., 0].contiguous()
    return st


# ------------------------------------------------------------------ plain forms
def _tokens(x, c):
    """[B, NB, Hkv, G * 128, n] -> [B, T, Hq, n]."""
    B, NB, Hkv, _, n = x.shape
    return x.reshape(B, NB, Hkv, c["Hq"] // Hkv, QB, n).permute(0, 1, 4, 2, 3, 5).reshape(B, NB * QB, c["Hq"], n)


def _rows(x, c):
    """[B, T, Hq, n] -> [B, NB, Hkv, G * 128, n] in 32 bits."""
    B, T, Hq, n = x.shape
    G = Hq // c["Hkv"]
    return x.float().view(B, T // QB, QB, c["Hkv"], G, n).permute(0, 1, 3, 4, 2, 5).reshape(B, T // QB, c["Hkv"], G * QB, n)


def _blocks(st):
    """Rows of each query block, the keys and values that it goes over, their indices, and
    which of them a row sees."""
    c = st["case"]
    lower, upper = (b[:, 0].long() for b in st["bounds"][:2])
    key = lower[..., None] * c["kb"] + torch.arange(st["width"], device=DEV)          # [B, NB, W]
    inside = key < upper[..., None] * c["kb"]
    key = torch.where(inside, key, torch.zeros_like(key))
    row = torch.arange(c["B"], device=DEV)[:, None, None]
    k, v = (st[n][row, key].float().transpose(2, 3) for n in ("k", "v"))              # [B, NB, Hkv, W, D]
    sq, pq = (st[n].view(c["B"], -1, QB, 1) for n in ("seg", "pos"))
    sk, pk = (st[n][row, key][:, :, None] for n in ("seg", "pos"))
    see = inside[:, :, None] & (sq == sk) & (sq >= 0)
    left, right = _sides(c)
    if left is not None:
        see &= pk >= pq - left
    if right is not None:
        see &= pk <= pq + right
    see = see[:, :, None].expand(-1, -1, c["Hq"] // c["Hkv"], -1, -1).flatten(2, 3)[:, :, None]
    return _rows(st["q"], c), k, v, key, see


def _grad_plain(st):
    c = st["case"]
    q, k, v, key, see = _blocks(st)
    scale = 1.0 / math.sqrt(c["D"])
    do = _rows(st["do"], c)
    delta = (do * _rows(st["out"], c)).sum(-1, keepdim=True)
    p = (q @ k.transpose(-1, -2)).mul_(scale).sub_(_rows(st["lse"][..., None], c)).exp_().masked_fill_(~see, 0.0)
    ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = _tokens((ds @ k).mul_(scale), c)
    at = (key + c["T"] * torch.arange(c["B"], device=DEV)[:, None, None]).flatten()

    def keys(x):
        y = torch.zeros((c["B"] * c["T"], c["Hkv"], c["D"]), device=DEV)
        return y.index_add_(0, at, x.transpose(2, 3).flatten(0, 2)).view(st["k"].shape).to(torch.bfloat16)

    return dict(dq=dq.to(torch.bfloat16), dk=keys((ds.transpose(-1, -2) @ q).mul_(scale)), dv=keys(p.transpose(-1, -2) @ do))


def _frequencies(c, base):
    """Radians a position of each pair, in 64 bits: a pair that makes more than 32 turns over the
    original length keeps its frequency, one of less than 1 has it divided by the factor."""
    f = base ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    keep = torch.zeros_like(f)
    if c["original"]:
        keep = ((c["original"] * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / c["factor"])


def _tables_plain(st):
    c = st["case"]
    turn = torch.arange(c["n"], device=DEV, dtype=torch.float64)[:, None] * _frequencies(c, st["base"])
    return dict(cos=(c["amplitude"] * turn.cos()).float(), sin=(c["amplitude"] * turn.sin()).float())


def _rotate_plain(st):
    c = st["case"]
    rot = c["rot"]
    pos = st["pos"].long() if st["pos"] is not None else torch.arange(c["T"], device=DEV).expand(c["B"], -1)
    cos, sin = (st[n][pos.clamp(min=0)][:, :, None] for n in ("cos", "sin"))
    if c["inverse"]:
        sin = -sin

    def turned(x):
        y = x.float().clone()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["pairs"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        a.copy_(lo), b.copy_(hi)
        return torch.where((pos >= 0)[..., None, None], y.to(x.dtype), x)

    return dict(q=turned(st["q"]), k=turned(st["k"]))


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        import selected_block_attention_gb300 as sba
        if c["op"] == "tables":
            cos, sin = sba.rotary_tables(c["n"], c["rot"], base=st["base"], factor=c["factor"], original_length=c["original"],
                                         slow=1.0, fast=32.0, amplitude=c["amplitude"], device=DEV)
            return dict(cos=cos, sin=sin)
        if c["op"] == "rotate":
            q, k = sba.rotary_embed(st["q"], st["k"], st["cos"], st["sin"], positions=st["pos"], interleaved=c["pairs"], inverse=c["inverse"])
            return dict(q=q, k=k)
        # as the forward leaves it: for rows of one query block the state's may be a view in another order
        out = st["out"].contiguous()
        dq, dk, dv = sba.blocksparse_attn_bwd(st["q"], st["k"], st["v"], out, st["lse"], st["do"], st["pos"], st["seg"], st["pos"], st["seg"],
                                              *st["bounds"], QB, c["kb"], causal=c["causal"], window_left=c["left"], window_right=c["right"])
        return dict(dq=dq, dk=dk, dv=dv)
    return {"tables": _tables_plain, "rotate": _rotate_plain, "grad": _grad_plain}[c["op"]](st)


def work(case):
    c = case
    if c["op"] == "tables":
        return dict(bytes=c["n"] * c["rot"] * 4, flops=c["n"] * c["rot"] * 4)
    N, D = c["B"] * c["T"], c["D"]
    if c["op"] == "rotate":
        seg = _segments(c)
        n = max(int(np.bincount(s[s >= 0]).max()) if (s >= 0).any() else 0 for s in seg)
        heads = c["Hq"] + c["Hkv"]
        return dict(bytes=N * heads * D * 2 * (4 if c["f32"] else 2) + n * c["rot"] * 4 + (4 * N if c["doc"] or c["pad"] else 0),
                    flops=N * heads * 3 * c["rot"])
    first, last = _views(c)
    pairs = int((last - first + 1).sum())
    return dict(bytes=N * D * 2 * (4 * c["Hq"] + 4 * c["Hkv"]) + N * (4 * c["Hq"] + 16) + 16 * c["B"] * c["T"] // QB,
                flops=10 * D * c["Hq"] * pairs)


# ------------------------------------------------------------------ values in 64 bits
def _exact_tables(case, seed):
    base = prepare(case, seed)["base"]
    cols = []
    for i in range(case["rot"] // 2):
        f = math.exp(-2.0 * i / case["rot"] * math.log(base))
        turns = case["original"] * f / (2.0 * math.pi)
        share = min(1.0, max(0.0, (turns - 1.0) / 31.0)) if case["original"] else 0.0
        cols.append(share * f + (1.0 - share) * f / case["factor"])
    z = torch.arange(case["n"], dtype=torch.float64, device=DEV)[:, None] * torch.tensor(cols, dtype=torch.float64, device=DEV)[None]
    return dict(cos=case["amplitude"] * torch.cos(z), sin=case["amplitude"] * torch.sin(z))


def _exact_rotate(case, seed):
    st = prepare(case, seed)
    rot, T = case["rot"], case["T"]
    pos = st["pos"] if st["pos"] is not None else torch.arange(T, dtype=torch.int32, device=DEV).repeat(case["B"], 1)
    still = pos < 0
    at = torch.where(still, torch.zeros_like(pos), pos).long()
    wheel = torch.complex(st["cos"].double(), st["sin"].double() * (-1.0 if case["inverse"] else 1.0))[at]
    wheel[still] = 1.0
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        part = x[..., :rot]
        pair = part.unflatten(-1, (rot // 2, 2)) if case["pairs"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * wheel[:, :, None])
        out[name] = torch.cat(((z if case["pairs"] else z.transpose(-1, -2)).flatten(-2), x[..., rot:]), -1)
    return out


def _exact_grad(case, seed):
    c = case
    first, last = _views(c)
    B, T = first.shape
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    some = last >= first
    spans = [[(int(first[b, t:t + QB][some[b, t:t + QB]].min()), int(last[b, t:t + QB].max()) + 1) if some[b, t:t + QB].any() else None
              for t in range(0, T, QB)] for b in range(B)]
    if sum(s[1] - s[0] for r in spans for s in r if s) * QB * Hq * D * 10.0 > 8e12:
        return None
    st = prepare(case, seed)
    f, z = (torch.from_numpy(x).to(DEV) for x in (first, last))
    dq = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
    dk, dv = (torch.zeros((B, T, Hkv, D), dtype=torch.float64, device=DEV) for _ in range(2))
    root = math.sqrt(D)
    for b in range(B):
        for n, span in enumerate(spans[b]):
            if span is None:
                continue
            a, e = span
            t = slice(n * QB, (n + 1) * QB)
            heads = lambda x: x[b, t].double().view(QB, Hkv, G, D).permute(1, 2, 0, 3)       # noqa: E731
            q, do = heads(st["q"]), heads(st["do"])                                          # [Hkv, G, 128, D]
            k, v = (st[x][b, a:e].double().transpose(0, 1)[:, None] for x in "kv")           # [Hkv, 1, keys, D]
            j = torch.arange(a, e, device=DEV)
            dark = (j < f[b, t, None]) | (j > z[b, t, None])
            logit = (torch.matmul(q, k.mT) / root).masked_fill(dark, -math.inf)
            w = torch.softmax(logit, -1).masked_fill(dark, 0.0)
            back = torch.matmul(do, v.mT)
            g = w * (back - (w * back).sum(-1, keepdim=True)) / root
            dq[b, t] = torch.matmul(g, k).permute(2, 0, 1, 3).reshape(QB, Hq, D)
            dk[b, a:e] += torch.matmul(g.flatten(1, 2).mT, q.flatten(1, 2)).transpose(0, 1)
            dv[b, a:e] += torch.matmul(w.flatten(1, 2).mT, do.flatten(1, 2)).transpose(0, 1)
    return dict(dq=dq, dk=dk, dv=dv)


def exact(case, seed):
    return {"tables": _exact_tables, "rotate": _exact_rotate, "grad": _exact_grad}[case["op"]](case, seed)
