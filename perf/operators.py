"""The paged-cache operators as they are measured: cases, inputs, plain forms, 64-bit values.

  append  paged_kv_append       new keys and values into a paged cache (8 bits with a scale
                                per page and head, or bfloat16), keys and queries rotated by
                                their positions on the way
  attend  paged_attention_fwd   attention of one or several query tokens per row over the
                                pages of that row
  select  nsa_select_paged_fwd  selected-block attention of decode tokens over the pages

Where ``own`` is false ``run`` computes the operator with elementary torch operations in 32
bits; where it is true it makes the library's calls.  A row's length and its number of new
tokens follow from the case, all values from the seed.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: latency only
        dict(name="append decode b8", op="append", B=8, lo=100, hi=4000, new=1, ragged=False,
             Hq=32, Hkv=8, D=128, P=64, f8=True, rot=128, pairs=False),
        # one decode step of a large serving batch
        dict(name="append decode b256", op="append", B=256, lo=1, hi=8192, new=1, ragged=False,
             Hq=32, Hkv=8, D=128, P=64, f8=True, rot=128, pairs=False),
        # prompts of different lengths packed into one call
        dict(name="append prompts", op="append", B=12, lo=0, hi=700, new=2600, ragged=True,
             Hq=32, Hkv=8, D=128, P=64, f8=True, rot=128, pairs=False),
        # the same into a bfloat16 cache of small pages, part of each head rotated in
        # neighbouring pairs
        dict(name="append prompts bf16", op="append", B=7, lo=0, hi=333, new=3001, ragged=True,
             Hq=16, Hkv=4, D=64, P=16, f8=False, rot=32, pairs=True),
        # one row, one token: latency only
        dict(name="attend decode b1", op="attend", B=1, lo=2011, hi=2011, new=1, ragged=False,
             Hq=32, Hkv=8, D=128, P=64, f8=True, left=-1, right=-1, cap=0.0, sinks=0),
        # a serving batch with a sliding window, capped scores and biased first keys
        dict(name="attend decode window", op="attend", B=64, lo=1, hi=32768, new=1, ragged=False,
             Hq=32, Hkv=8, D=128, P=64, f8=True, left=4096, right=0, cap=50.0, sinks=4),
        # few rows, long contexts
        dict(name="attend decode long", op="attend", B=4, lo=60000, hi=131072, new=1,
             ragged=False, Hq=64, Hkv=4, D=128, P=128, f8=True, left=-1, right=-1, cap=0.0,
             sinks=0),
        # a batch of decode rows and short drafts being verified, bfloat16 cache, some rows
        # without tokens
        dict(name="attend drafts bf16", op="attend", B=48, lo=0, hi=6000, new=8, ragged=True,
             Hq=16, Hkv=4, D=64, P=16, f8=False, left=-1, right=0, cap=0.0, sinks=0),
        # prompts processed in chunks of 512 tokens over their cached prefix
        dict(name="attend chunks", op="attend", B=4, lo=512, hi=16384, new=512, ragged=False,
             Hq=32, Hkv=8, D=128, P=64, f8=True, left=-1, right=0, cap=0.0, sinks=0),
        # two rows: latency only
        dict(name="select decode b2", op="select", B=2, lo=700, hi=3000, new=1, Hq=16, Hkv=2,
             D=64, P=32, f8=False, S=8, block=32, gate=False),
        # a serving batch of selected-block decode over long contexts
        dict(name="select decode b64", op="select", B=64, lo=1000, hi=65536, new=1, Hq=64,
             Hkv=4, D=128, P=64, f8=True, S=16, block=64, gate=True),
    ]


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "select"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    c = dict(op=op, Hkv=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128]),
             P=rng.choice([16, 32, 64, 128]), f8=rng.random() < 0.7)
    if op == "append":
        c.update(B=log(1, 200), ragged=rng.random() < 0.5, rot=rng.choice([0, 16, c["D"] // 2, c["D"]]),
                 pairs=rng.random() < 0.4, Hq=c["Hkv"] * rng.choice([1, 4, 5, 8]))
        c["new"] = log(1, max(2, 8000 // c["B"]))
        c["lo"] = rng.randrange(0, 100)
        c["hi"] = c["lo"] + log(1, 3000)
    elif op == "attend":
        c.update(Hq=c["Hkv"] * rng.choice([1, 3, 4, 8, 16]), ragged=rng.random() < 0.5,
                 cap=rng.choice([0.0, 0.0, 20.0, 50.0]), sinks=rng.choice([0, 0, 1, 4, 16]))
        if rng.random() < 0.2:  # a chunk of a prompt
            c.update(B=log(1, 4), new=log(40, 300), lo=0, hi=log(50, 9000), left=-1, right=0)
        else:
            c.update(B=log(1, 100), new=rng.choice([1, 1, 1, 2, 5, 8]), lo=rng.randrange(0, 40))
            c.update(hi=log(50, 60000 if c["B"] < 12 else 12000), left=rng.choice([-1, -1, 0, 100, 1500]),
                     right=rng.choice([-1, 0, 0, 3]))
    else:
        c.update(B=log(1, 100), new=rng.choice([1, 1, 2, 3]), Hq=c["Hkv"] * rng.choice([1, 4, 8, 16]),
                 lo=rng.randrange(1, 200), hi=log(300, 50000), S=rng.choice([1, 5, 8, 16, 32]),
                 block=rng.choice([32, 64, 128]), gate=rng.random() < 0.5)
        c["hi"] = min(c["hi"], 3000000 // c["B"])
    return c


# ------------------------------------------------------------------ structure of a case
def _spread(n, step, start):
    return np.modf(start + step * np.arange(n))[0]


def _tokens(case):
    """(lengths with the new tokens, number of new tokens) of the rows, and the padded table width."""
    B = case["B"]
    lens = case["lo"] + np.floor((case["hi"] - case["lo"] + 1) * _spread(B, 0.6180339887, 0.37)).astype(np.int64)
    if case.get("ragged"):
        n = np.floor((case["new"] + 1) * _spread(B, 0.7548776662, 0.58)).astype(np.int64)
    else:
        n = np.full(B, case["new"], dtype=np.int64)
    if case["op"] == "append":
        lens = lens + n          # lo..hi tokens are there already
    else:
        lens = np.maximum(lens, n)
        if case.get("ragged"):
            lens[5::11] = 0      # slots of the batch without a sequence
            n[5::11] = 1
    return lens, n


def _width(case):
    lens, _ = _tokens(case)
    return max(1, -(-int(lens.max()) // case["P"]))


def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + what) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, seed, what, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, what), device=DEV, dtype=torch.float32).to(dtype)


def _pow2_scale(amax):
    """Smallest power of two s >= 2^-126 with 448 s >= amax (amax in 32 bits)."""
    m, e = torch.frexp(amax)                 # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)      # 448 = 0.875 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), e)


def _pool(case, pages, seed, what):
    """A pool of pages: values of about unit size, a little different from page to page."""
    shape = (pages, case["Hkv"], case["P"], case["D"])
    if not case["f8"]:
        return _randn(shape, seed, what, torch.bfloat16), None
    codes = torch.empty(shape, dtype=F8, device=DEV)
    scales = torch.empty(shape[:2], dtype=torch.float32, device=DEV)
    g = _gen(seed, what)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i),) + shape[1:], generator=g, device=DEV)
        x *= torch.exp2(0.7 * torch.randn(x.shape[:2], generator=g, device=DEV))[..., None, None]
        s = _pow2_scale(x.abs().amax((2, 3)))
        scales[i:i + step] = s
        codes[i:i + step] = (x / s[..., None, None]).to(F8)
    return codes, scales


def prepare(case, seed):
    c = case
    lens, n = _tokens(c)
    B, W = c["B"], _width(c)
    used = -(-lens // c["P"])
    pages = int(used.sum()) + 3
    order = torch.randperm(pages, generator=_gen(seed, 1), device=DEV).cpu().numpy()
    table = np.full((B, W), -1, dtype=np.int32)   # entries past a row's length belong to nobody
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += int(used[b])
    st = dict(case=c, table=torch.from_numpy(table).to(DEV),
              lens=torch.from_numpy(lens.astype(np.int32)).to(DEV))
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N = int(cu[-1])
    st["cu"] = torch.from_numpy(cu).to(DEV) if c.get("ragged") else None
    st["k_pages"], st["k_scales"] = _pool(c, pages, seed, 2)
    st["v_pages"], st["v_scales"] = _pool(c, pages, seed, 3)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "append":
        # the three parts of one projection's output
        qkv = _randn((N, (Hq + 2 * Hkv) * D), seed, 4, torch.bfloat16)
        st["q"] = qkv[:, :Hq * D].view(N, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(N, Hkv, D)
        if not c["ragged"]:
            for name in ("q", "k", "v"):
                st[name] = st[name].unflatten(0, (B, c["new"]))
        st["cos"] = st["sin"] = None
        if c["rot"]:
            pos = torch.arange(max(1, int(lens.max())), device=DEV, dtype=torch.float64)
            freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
            st["cos"] = (pos[:, None] * freq).cos().float()
            st["sin"] = (pos[:, None] * freq).sin().float()
        return st
    q = _randn((N, Hq, D), seed, 4, torch.bfloat16)
    st["q"] = q if c.get("ragged") else q.view(B, c["new"], Hq, D)
    if c["op"] == "attend":
        st["bias"] = 0.1 * _randn((Hq, c["sinks"]), seed, 5) if c["sinks"] else None
        return st
    # selected blocks: the token's own block and earlier ones, shuffled, padded with -1
    Q, S, bs = c["new"], c["S"], c["block"]
    pos = (torch.from_numpy(lens).to(DEV)[:, None] - Q + torch.arange(Q, device=DEV)).view(B, Q, 1, 1)
    nb = pos // bs + 1
    NB = -(-int(lens.max()) // bs)
    blocks = torch.arange(NB, device=DEV)
    key = torch.rand((B, Q, Hkv, NB), generator=_gen(seed, 6), device=DEV)
    key = torch.where(blocks < nb, key, torch.full_like(key, 2.0))
    key = torch.where(blocks == nb - 1, torch.full_like(key, -1.0), key)
    take = min(S, NB)
    first = key.argsort(-1)[..., :take]
    idx = torch.full((B, Q, Hkv, S), -1, device=DEV, dtype=torch.int64)
    idx[..., :take] = torch.where(first < nb, first, torch.full_like(first, -1))
    mix = torch.rand(idx.shape, generator=_gen(seed, 7), device=DEV).argsort(-1)
    st["idx"] = idx.gather(-1, mix).to(torch.int32)
    st["gate"] = torch.sigmoid(_randn((B, Q, Hq), seed, 8)).to(torch.bfloat16) if c["gate"] else None
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rot, pairs):
    """x [..., heads, D] in 32 bits, cos / sin [..., 1, rot / 2]."""
    if not rot:
        return x
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = lo, hi
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = lo, hi
    return y


def _row_of(st):
    """(row, position) of each new token."""
    c = st["case"]
    B = c["B"]
    lens = st["lens"].long()
    if st["cu"] is None:
        row = torch.arange(B, device=DEV).repeat_interleave(c["new"])
        i = torch.arange(c["new"], device=DEV).repeat(B)
        return row, lens[row] - c["new"] + i
    N = st["q"].shape[0]
    cu = st["cu"].long()
    t = torch.arange(N, device=DEV)
    row = torch.searchsorted(cu, t, right=True) - 1
    return row, lens[row] - cu[row + 1] + t


def _to_f8(x, scale):
    return (x * (1.0 / scale)).clamp(-F8_MAX, F8_MAX).to(F8)


def _store(pages, scales, x, page, off, first_page, first_off, P):
    """x [N, Hkv, D] in 32 bits into pages[page, :, off]."""
    if scales is None:
        pages[page, :, off] = x.to(pages.dtype)
        return
    mag = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
    amax = torch.zeros_like(scales).index_reduce_(0, page, mag, "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=DEV)
    touched[page] = True
    start = torch.full((scales.shape[0],), P, dtype=off.dtype, device=DEV).index_reduce_(0, page, off, "amin")
    old = torch.where((start > 0)[:, None], scales, torch.zeros_like(scales))
    new = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(amax)), scales)
    # tokens that a row's first page holds already, in the page's new scale
    was = pages[first_page].float() * scales[first_page][..., None, None]
    kept = torch.arange(P, device=DEV) < first_off[:, None]
    raw = pages.view(torch.uint8)
    again = _to_f8(was, new[first_page][..., None, None]).view(torch.uint8)
    raw[first_page] = torch.where(kept[:, None, :, None], again, raw[first_page])
    raw[page, :, off] = _to_f8(x, new[page][..., None]).view(torch.uint8)
    scales.copy_(new)


def _append_plain(st):
    c = st["case"]
    P, rot, pairs = c["P"], c["rot"], c["pairs"]
    row, pos = _row_of(st)
    N = row.numel()
    q, k, v = (st[n].reshape(N, -1, c["D"]).float() for n in ("q", "k", "v"))
    if rot:
        cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
        q, k = _rotate(q, cos, sin, rot, pairs), _rotate(k, cos, sin, rot, pairs)
    page, off = st["table"][row, pos // P].long(), pos % P
    lens = st["lens"].long()
    n = st["cu"].diff().long() if st["cu"] is not None else torch.full_like(lens, c["new"])
    start = lens - n
    slot = (start // P).clamp(max=st["table"].shape[1] - 1)
    first_page = st["table"].gather(1, slot[:, None])[:, 0].long()
    spare = st["k_pages"].shape[0] - 1
    first_off = torch.where((first_page >= 0) & (n > 0), start % P, torch.zeros_like(start))
    first_page = torch.where(first_off > 0, first_page, torch.full_like(first_page, spare))
    _store(st["k_pages"], st["k_scales"], k, page, off, first_page, first_off, P)
    _store(st["v_pages"], st["v_scales"], v, page, off, first_page, first_off, P)
    out = dict(q=q.to(torch.bfloat16).view(st["q"].shape), k=st["k_pages"], v=st["v_pages"])
    if c["f8"]:
        out.update(ks=st["k_scales"], vs=st["v_scales"])
    return out


def _values(pages, scales, table):
    """[B, Hkv, keys, D] in 32 bits of the pages in table [B, W]."""
    at = table.long().clamp(min=0)
    x = pages.view(torch.uint8)[at].view(pages.dtype).float() if pages.dtype == F8 else pages[at].float()
    if scales is not None:
        x = x * scales[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend_plain(st):
    c = st["case"]
    B, Hq, Hkv, D, Q = c["B"], c["Hq"], c["Hkv"], c["D"], c["new"]
    G = Hq // Hkv
    lens = st["lens"].long()
    k = _values(st["k_pages"], st["k_scales"], st["table"])
    v = _values(st["v_pages"], st["v_scales"], st["table"])
    key = torch.arange(k.shape[2], device=DEV)
    if st["cu"] is None:
        q, i = st["q"], torch.arange(Q, device=DEV).expand(B, Q)
        n = torch.full_like(lens, Q)
    else:
        cu = st["cu"].long()
        n = cu.diff()
        i = torch.arange(Q, device=DEV).expand(B, Q)
        q = st["q"][(cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)]
    pos = (lens - n)[:, None] + i                                             # [B, Q]
    qf = q.float().view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    s = (qf @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))                     # [B, Hkv, G Q, keys]
    if c["cap"] > 0:
        s = c["cap"] * torch.tanh(s / c["cap"])
    see = torch.ones((B, Q, key.numel()), dtype=torch.bool, device=DEV)
    if c["left"] >= 0:
        see &= key >= (pos - c["left"])[..., None]
    if c["right"] >= 0:
        see &= key <= (pos + c["right"])[..., None]
    s = s.view(B, Hkv, G, Q, -1)
    if c["sinks"]:
        see |= key < c["sinks"]
        m = min(c["sinks"], key.numel())
        s[..., :m] += st["bias"][:, :m].view(1, Hkv, G, 1, m)
    see &= key < lens[:, None, None]
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    v = torch.where((key < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = (e.view(B, Hkv, G * Q, -1) @ v).view(B, Hkv, G, Q, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, Q, Hq)
    if st["cu"] is not None:
        row, _ = _row_of(st)
        at = torch.arange(row.numel(), device=DEV) - cu[row]
        o, lse = o[row, at], lse[row, at]
    return dict(out=o.to(torch.bfloat16), lse=lse.contiguous())


def _select_plain(st):
    c = st["case"]
    B, Q, Hq, Hkv, D, S, bs, P = c["B"], c["new"], c["Hq"], c["Hkv"], c["D"], c["S"], c["block"], c["P"]
    G = Hq // Hkv
    lens = st["lens"].long()
    pos = ((lens - Q)[:, None] + torch.arange(Q, device=DEV)).view(B, Q, 1, 1)
    idx = st["idx"].long()
    again = ((idx[..., :, None] == idx[..., None, :]) & torch.ones((S, S), dtype=torch.bool, device=DEV).tril(-1)).any(-1)
    ok = (idx >= 0) & (idx * bs <= pos) & ~again
    key = (idx[..., None] * bs + torch.arange(bs, device=DEV)).flatten(-2)   # [B, Q, Hkv, S bs]
    see = ok.repeat_interleave(bs, -1) & (key <= pos)
    key = torch.where(see, key, torch.zeros_like(key))
    row = torch.arange(B, device=DEV).view(B, 1, 1, 1)
    page = st["table"][row, key // P].long()
    head = torch.arange(Hkv, device=DEV).view(1, 1, Hkv, 1)

    def rows(pages, scales):
        raw = pages.view(torch.uint8)[page, head, key % P].view(pages.dtype) if pages.dtype == F8 else pages[page, head, key % P]
        return raw.float() if scales is None else raw.float() * scales[page, head][..., None]

    q = st["q"].float().view(B, Q, Hkv, G, D)
    s = (q @ rows(st["k_pages"], st["k_scales"]).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    s.masked_fill_(~see[..., None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    o = ((e @ rows(st["v_pages"], st["v_scales"])) / total).reshape(B, Q, Hq, D)
    if st["gate"] is not None:
        o = o * st["gate"].float()[..., None]
    return dict(out=o.to(torch.bfloat16), lse=(top + total.log()).reshape(B, Q, Hq))


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        import selected_block_attention_gb300 as sba
        pool = (st["k_pages"], st["v_pages"], st["table"], st["lens"])
        scales = dict(k_scales=st["k_scales"], v_scales=st["v_scales"])
        if c["op"] == "append":
            q = sba.paged_kv_append(st["k"], st["v"], *pool, **scales, cu_seqlens=st["cu"], q=st["q"],
                                    cos=st["cos"], sin=st["sin"], interleaved=c["pairs"])
            out = dict(q=q, k=st["k_pages"], v=st["v_pages"])
            if c["f8"]:
                out.update(ks=st["k_scales"], vs=st["v_scales"])
            return out
        if c["op"] == "attend":
            out, lse = sba.paged_attention_fwd(st["q"], *pool, **scales, cu_seqlens=st["cu"], window_left=c["left"],
                                               window_right=c["right"], logits_soft_cap=c["cap"], sink_bias=st["bias"])
        else:
            out, lse = sba.nsa_select_paged_fwd(st["q"], *pool, st["idx"], c["S"], c["block"], **scales, g_slc=st["gate"])
        return dict(out=out, lse=lse)
    return {"append": _append_plain, "attend": _attend_plain, "select": _select_plain}[c["op"]](st)


def work(case):
    c = case
    lens, n = _tokens(c)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    item = 1 if c["f8"] else 2
    N = int(n.sum())
    W = _width(c)
    if c["op"] == "append":
        pages = sum(-(-int(e) // c["P"]) - int(e - m) // c["P"] for e, m in zip(lens, n) if m)
        b = N * (2 * Hq + 2 * Hkv) * D * 2 + N * 2 * Hkv * D * item + pages * (4 + (16 * Hkv if c["f8"] else 0))
        if c["rot"]:
            b += min(N, int(lens.max())) * c["rot"] * 4
        return dict(bytes=b, flops=N * ((Hq + Hkv) * 3 * c["rot"] + (6 * Hkv * D if c["f8"] else 0)))
    keys = pairs = 0     # cache rows read (per head), (query, key) pairs
    if c["op"] == "attend":
        for e, m in zip(lens, n):
            e, m = int(e), int(m)
            if not e or not m:
                continue
            pos = e - m + np.arange(m)
            lo = np.clip(pos - c["left"] if c["left"] >= 0 else np.zeros(m, int), 0, e)
            hi = np.clip(pos + c["right"] + 1 if c["right"] >= 0 else np.full(m, e), 0, e)
            sink = np.minimum(c["sinks"], e)
            extra = np.clip(np.minimum(sink, lo), 0, None) + np.clip(sink - np.maximum(hi, 0), 0, None)
            pairs += int((np.clip(hi - lo, 0, None) + extra).sum())
            keys += int(hi.max() - lo.min()) + int(min(sink, lo.min()))
        extra_bytes = 4 * Hq * c["sinks"]
    else:
        for e in lens:
            for p in int(e) - c["new"] + np.arange(c["new"]):
                nb = int(p) // c["block"] + 1
                pairs += (min(c["S"], nb) - 1) * c["block"] + int(p) % c["block"] + 1
        keys = pairs
        extra_bytes = N * Hkv * c["S"] * 4 + (N * Hq * 2 if c["gate"] else 0)
    b = keys * Hkv * D * 2 * item + N * Hq * (4 * D + 4) + extra_bytes
    b += 4 * (keys // c["P"]) * (1 + (2 * Hkv if c["f8"] else 0)) + 8 * c["B"]
    return dict(bytes=b, flops=4 * D * Hq * pairs)


# ------------------------------------------------------------------ values in 64 bits
def _nearest_e4m3(y):
    """The e4m3 value next to y (ties to even), y in 64 bits, |y| limited to 448."""
    y = y.clamp(-F8_MAX, F8_MAX)
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exact_append(case, seed):
    st = prepare(case, seed)
    lens, n = _tokens(case)
    N, D, P, rot = int(n.sum()), case["D"], case["P"], case["rot"]
    x = {m: st[m].reshape(N, -1, D).double() for m in ("q", "k", "v")}
    ends = np.cumsum(n)
    table = st["table"].cpu().numpy()
    pool = {m: (st[m + "_pages"].double(), None if st[m + "_scales"] is None else st[m + "_scales"].double()) for m in "kv"}
    if rot:
        cs, sn = st["cos"].double(), st["sin"].double()
    for b in range(case["B"]):
        if not n[b]:
            continue
        t0, t1 = int(ends[b] - n[b]), int(ends[b])
        p0 = int(lens[b] - n[b])
        if rot:
            co, si = cs[p0:int(lens[b]), None], sn[p0:int(lens[b]), None]
            for m in ("q", "k"):
                z = x[m][t0:t1]
                w = z[..., :rot].unflatten(-1, (rot // 2, 2)) if case["pairs"] else z[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                w = torch.stack((w[..., 0] * co - w[..., 1] * si, w[..., 1] * co + w[..., 0] * si), -1)
                w = w.flatten(-2) if case["pairs"] else w.transpose(-1, -2).flatten(-2)
                x[m][t0:t1] = torch.cat((w, z[..., rot:]), -1)
        for j in range(p0 // P, -(-int(lens[b]) // P)):
            pg = int(table[b, j])
            a, e = max(p0, j * P), min(int(lens[b]), (j + 1) * P)
            for m in "kv":
                pages, scales = pool[m]
                fresh = x[m][t0 + a - p0:t0 + e - p0].transpose(0, 1)        # [Hkv, tokens, D]
                if scales is None:
                    pages[pg, :, a - j * P:e - j * P] = fresh
                    continue
                peak = fresh.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2((peak / F8_MAX).clamp(min=2.0 ** -126))))
                if a > j * P:
                    was = scales[pg].clone()
                    need = torch.maximum(was, need)
                    held = pages[pg, :, :a - j * P] * (was / need)[:, None, None]
                    pages[pg, :, :a - j * P] = _nearest_e4m3(held)
                scales[pg] = need
                pages[pg, :, a - j * P:e - j * P] = _nearest_e4m3(fresh / need[:, None, None])
    out = dict(q=x["q"].view(st["q"].shape), k=pool["k"][0], v=pool["v"][0])
    if case["f8"]:
        out.update(ks=pool["k"][1], vs=pool["v"][1])
    return out


def _softmax_rows(logit, v):
    """logit [G, keys], v [keys, D] -> output, log of the sum; 64 bits."""
    if logit.shape[1] == 0:
        return logit.new_zeros(logit.shape[0], v.shape[1]), logit.new_full((logit.shape[0],), -math.inf)
    lse = torch.logsumexp(logit, -1)
    safe = torch.where(lse.isinf(), torch.zeros_like(lse), lse)
    return torch.exp(logit - safe[:, None]) @ v, lse


def _exact_attend(case, seed):
    st = prepare(case, seed)
    lens, n = _tokens(case)
    if float(np.dot(lens, n)) * case["Hq"] * case["D"] > 4e12:
        return None
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["P"]
    G = Hq // Hkv
    q = st["q"].reshape(-1, Hq, D).double()
    out = q.new_zeros(q.shape)
    lse = q.new_full(q.shape[:2], -math.inf)
    t = 0
    for b in range(case["B"]):
        e, m = int(lens[b]), int(n[b])
        if e and m:
            pg = st["table"][b, :-(-e // P)].long()
            key = torch.arange(e, device=DEV)
            at = (e - m + torch.arange(m, device=DEV))[:, None]
            off = torch.zeros((m, e), dtype=torch.bool, device=DEV)
            if case["left"] >= 0:
                off |= key < at - case["left"]
            if case["right"] >= 0:
                off |= key > at + case["right"]
            off &= ~(key < case["sinks"])
            for h in range(Hkv):
                kv = []
                for x in "kv":
                    y = st[x + "_pages"][pg, h].double()
                    if case["f8"]:
                        y = y * st[x + "_scales"][pg, h].double()[:, None, None]
                    kv.append(y.flatten(0, 1)[:e])
                z = q[t:t + m, h * G:(h + 1) * G].reshape(m * G, D) @ kv[0].T / math.sqrt(D)
                if case["cap"] > 0:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                z = z.view(m, G, e)
                if case["sinks"]:
                    w = min(e, case["sinks"])
                    z[..., :w] += st["bias"][h * G:(h + 1) * G, :w].double()
                z = z.masked_fill(off[:, None], -math.inf).view(m * G, e)
                o, ls = _softmax_rows(z, kv[1])
                out[t:t + m, h * G:(h + 1) * G] = o.view(m, G, D)
                lse[t:t + m, h * G:(h + 1) * G] = ls.view(m, G)
        t += m
    return dict(out=out.view(st["q"].shape), lse=lse.view(st["q"].shape[:-1]))


def _exact_select(case, seed):
    st = prepare(case, seed)
    lens, _ = _tokens(case)
    B, Q, Hq, Hkv, D, P, bs = case["B"], case["new"], case["Hq"], case["Hkv"], case["D"], case["P"], case["block"]
    G = Hq // Hkv
    out = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Q, Hq), dtype=torch.float64, device=DEV)
    chosen = st["idx"].cpu().numpy()
    for b in range(B):
        for i in range(Q):
            p = int(lens[b]) - Q + i
            for h in range(Hkv):
                keys = [np.arange(j * bs, min((j + 1) * bs, p + 1)) for j in sorted(set(int(j) for j in chosen[b, i, h])) if 0 <= j <= p // bs]
                keys = torch.from_numpy(np.concatenate(keys)).to(DEV)
                pg = st["table"][b][keys // P].long()
                kv = []
                for x in "kv":
                    y = st[x + "_pages"].view(torch.uint8)[pg, h, keys % P].view(F8).double() if case["f8"] else st[x + "_pages"][pg, h, keys % P].double()
                    kv.append(y * st[x + "_scales"][pg, h].double()[:, None] if case["f8"] else y)
                hs = slice(h * G, (h + 1) * G)
                o, ls = _softmax_rows(st["q"][b, i, hs].double() @ kv[0].T / math.sqrt(D), kv[1])
                if st["gate"] is not None:
                    o = o * st["gate"][b, i, hs].double()[:, None]
                out[b, i, hs], lse[b, i, hs] = o, ls
    return dict(out=out, lse=lse)


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "select": _exact_select}[case["op"]](case, seed)
