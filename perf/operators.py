"""Timing cases of the 8-bit paged KV cache: the append with position rotation and the attention over it.

A page of the pool holds the rows of one block of tokens for one KV head, keys or values, as
8-bit codes [block_tokens][head_dim] with one power-of-two scale per page (its exponent in an
int8 array indexed by page): value = code * 2**exponent.  The block table of a sequence lists,
per block and KV head, the page of the keys and the page of the values; pages are scattered.

  append  rotates the keys (and queries) of the batch's new tokens by their positions and writes
          keys and values to the cache, growing a block's exponent where a new token needs it
  attend  softmax(scale * q k^T) v of every new token over its sequence's cache

With ``own`` false ``run`` computes both in elementary torch operations in fp32; with ``own``
true it makes the library's calls.
"""
import math
import random

import torch

own = False

#: Largest magnitude of a code, and the exponent a block of zeros gets.
E4M3_MAX, INT8_MAX, MIN_EXPONENT = 448.0, 127.0, -40


# ---- cases --------------------------------------------------------------------------------
def _case(name, op, **more):
    c = dict(name=name, op=op, hidden=4096, hq=32, hkv=32, d=128, fmt="e4m3", n_dec=0, n_multi=0, q_lo=1, q_hi=1,
             ctx_lo=0, ctx_hi=0, window=0, rot=128, interleaved=False, shape_seed=1)
    c.update(more)
    return c


def listed():
    return [
        # one user's next token, grouped-query model: latency counts
        _case("append_one_token", "append", hkv=8, n_dec=1, ctx_lo=700, ctx_hi=700),
        # the 13B-shaped decode batch: 512 tokens, every sequence at its own length
        _case("append_decode_13b", "append", hidden=5120, hq=40, hkv=40, n_dec=512, ctx_lo=30, ctx_hi=1000),
        # the mixed iteration: 8 prompts of 256-1024 tokens beside 384 decode tokens; adjacent pairs, half the row
        # rotated
        _case("append_mixed_7b", "append", n_dec=384, n_multi=8, q_lo=256, q_hi=1024, ctx_hi=900, rot=64,
              interleaved=True),
        # one long prompt of an odd length, int8, 64-wide heads
        _case("append_long_prompt", "append", hkv=8, d=64, rot=64, fmt="int8", n_multi=1, q_lo=16381, q_hi=16381,
              ctx_lo=3, ctx_hi=3),
        # one user's next token over a short context: latency counts
        _case("attend_one_token", "attend", hkv=8, n_dec=1, ctx_lo=700, ctx_hi=700),
        # the 13B-shaped decode batch
        _case("attend_decode_13b", "attend", hidden=5120, hq=40, hkv=40, n_dec=512, ctx_lo=30, ctx_hi=1000),
        # a few users deep into long documents: few rows, a long axis
        _case("attend_decode_long", "attend", hkv=8, fmt="int8", n_dec=4, ctx_lo=60000, ctx_hi=131000),
        # sliding-window layers of a model with 64-wide heads
        _case("attend_window", "attend", hkv=4, d=64, rot=64, fmt="int8", n_dec=48, ctx_lo=300, ctx_hi=20000,
              window=1000),
        # checking drafted tokens: a few new tokens per sequence
        _case("attend_draft_check", "attend", hkv=8, n_multi=24, q_lo=3, q_hi=8, ctx_lo=500, ctx_hi=8000),
        # the prefill batch: 16 prompts of 512 tokens
        _case("attend_prefill_7b", "attend", n_multi=16, q_lo=512, q_hi=512),
        # the mixed iteration: 8 prompts of 256-1024 tokens beside 384 decode tokens
        _case("attend_mixed_7b", "attend", n_dec=384, n_multi=8, q_lo=256, q_hi=1024, ctx_hi=900),
        # the next chunk of a long prompt
        _case("attend_chunk", "attend", hkv=8, fmt="int8", n_multi=1, q_lo=2048, q_hi=2048, ctx_lo=30001,
              ctx_hi=30001),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    kind = rng.choice(["decode", "decode", "few", "prompt", "mixed"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 16, 32, 40])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * hkv <= 64])
    c = _case("", op, hidden=rng.choice([2048, 4096, 4096, 5120]), d=d, hkv=hkv, hq=hkv * group,
              fmt=rng.choice(["e4m3", "int8"]), rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
              shape_seed=rng.randrange(1 << 20))
    del c["name"]
    if kind in ("decode", "mixed"):
        c["n_dec"] = _log_int(rng, 1, 512)
        c["ctx_hi"] = _log_int(rng, 16, 131000)
        c["ctx_lo"] = c["ctx_hi"] // rng.choice([1, 2, 20])
    if kind == "few":
        c["n_multi"], c["q_hi"] = _log_int(rng, 1, 64), rng.randrange(2, 17)
        c["q_lo"] = rng.randrange(1, c["q_hi"] + 1)
        c["ctx_hi"] = _log_int(rng, 16, 16000)
        c["ctx_lo"] = c["ctx_hi"] // rng.choice([1, 4])
    if kind in ("prompt", "mixed"):
        c["n_multi"], c["q_hi"] = _log_int(rng, 1, 16), _log_int(rng, 17, 2048)
        c["q_lo"] = rng.randrange(c["q_hi"] // 2 + 1, c["q_hi"] + 1)
        if kind == "prompt":
            c["ctx_hi"] = rng.choice([0, 0, _log_int(rng, 16, 16000)])
            c["ctx_lo"] = c["ctx_hi"] // 2
    if op == "attend" and rng.random() < 0.25:
        c["window"] = _log_int(rng, 64, 4096)
    # no costlier than the largest listed case: fewer sequences, then shorter ones
    while _cost(c) > 0.6:
        if c["n_dec"] > 1 or c["n_multi"] > 1:
            c["n_dec"], c["n_multi"] = (c["n_dec"] + 1) // 2, (c["n_multi"] + 1) // 2
        else:
            c["ctx_lo"], c["ctx_hi"] = c["ctx_lo"] * 2 // 3, c["ctx_hi"] * 2 // 3
            c["q_hi"] = max(1, c["q_hi"] * 3 // 4)
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
    return c


def _lengths(c):
    """(new tokens, cache length with them) per sequence: the single-token sequences first."""
    r = random.Random(c["shape_seed"])
    n = [1] * c["n_dec"] + [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["n_multi"])]
    return [(q, q + r.randint(c["ctx_lo"], c["ctx_hi"])) for q in n]


def _block(c):
    return c["hidden"] * 2 // c["d"] // 8 * 8


def _pairs(q, length, window):
    """Sum over the q last positions of the keys each sees."""
    if not window:
        return q * length - q * (q - 1) // 2
    return sum(min(p + 1, window) for p in range(length - q, length))


def _cost(c):
    """Share of the largest listed case in memory or arithmetic, whichever is more (the plain form pads)."""
    L = _lengths(c)
    pad = 0
    for sel in (L[:c["n_dec"]], L[c["n_dec"]:]):
        if sel:
            keys, rows = max(x for _, x in sel), max(q for q, _ in sel)
            pad += len(sel) * keys * (2 * c["hkv"] * c["d"] + (rows * c["hq"] if c["op"] == "attend" else 0))
    w = work(c)
    return max(pad / 5.0e9, w["bytes"] / 2.6e9, w["flops"] / 1.0e12)


def work(c):
    L = _lengths(c)
    T, d, hq, hkv = sum(q for q, _ in L), c["d"], c["hq"], c["hkv"]
    if c["op"] == "append":
        kv = 2 * T * hkv * d
        return {"bytes": kv * 2 + kv + 2 * T * hq * d * 2 + T * c["rot"] * 4,
                "flops": 3 * T * (hkv + hq) * c["rot"] + 2 * kv}
    seen = sum(min(n, c["window"] + q - 1) if c["window"] else n for q, n in L)
    pairs = sum(_pairs(q, n, c["window"]) for q, n in L)
    return {"bytes": 2 * seen * hkv * d + 2 * T * hq * d * 2 + 4 * T * hq, "flops": 4 * d * hq * pairs}


# ---- inputs -------------------------------------------------------------------------------
def _limit(fmt):
    return E4M3_MAX if fmt == "e4m3" else INT8_MAX


def _exponent(amax, fmt):
    """Smallest exponent e with amax <= limit * 2**e."""
    m, x = torch.frexp(amax)
    top, shift = (0.875, 9) if fmt == "e4m3" else (127 / 128, 7)
    e = x - shift + (m > top)
    return torch.where(amax > 0, e, MIN_EXPONENT).clamp(min=MIN_EXPONENT)


def _encode(x, fmt):
    """fp32 values in units of their scale -> codes, as bytes."""
    if fmt == "e4m3":
        return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nan_to_num(x, nan=0.0).round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8).view(torch.uint8)


def _code_type(fmt):
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.int8


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    L, BT, d, hq, hkv, fmt = _lengths(c), _block(c), c["d"], c["hq"], c["hkv"], c["fmt"]
    S, T = len(L), sum(q for q, _ in L)
    blocks = [-(-n // BT) for _, n in L]
    max_blocks = max(blocks) + 1
    num_pages = 2 * hkv * sum(blocks)

    # block table: the pages in a random order; blocks that a sequence does not have stay -1
    order = torch.randperm(num_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    width = torch.tensor(blocks, device=dev)
    table = torch.full((S, max_blocks, hkv, 2), -1, dtype=torch.int32, device=dev)
    table[torch.arange(max_blocks, device=dev)[None] < width[:, None]] = order.view(-1, hkv, 2)
    n_new = torch.tensor([q for q, _ in L], dtype=torch.int32, device=dev)
    indptr = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), n_new.cumsum(0).to(torch.int32)])
    kv_len = torch.tensor([n for _, n in L], dtype=torch.int32, device=dev)
    s = dict(case=c, T=T, S=S, BT=BT, max_blocks=max_blocks, max_q=max(q for q, _ in L), max_len=max(n for _, n in L),
             indptr=indptr, kv_len=kv_len, table=table, scale=1.0 / math.sqrt(d))

    # the cache: normal values, some channels larger, every page with a spread of its own
    page_bytes = c["hidden"] * 2
    if own:
        from rank_delta_paged_gb300.harness import KVSession
        s["kv"] = KVSession(c["hidden"], num_pages, hkv, d, fmt)
        s["pages"], s["exponents"] = s["kv"].pages, s["kv"].exponents
    else:
        s["pages"] = torch.empty((num_pages, page_bytes), dtype=torch.uint8, device=dev)
        s["exponents"] = torch.empty(num_pages, dtype=torch.int8, device=dev)
    channel = torch.exp(0.5 * torch.randn(d, generator=g, device=dev))
    step = max(1, (1 << 27) // page_bytes)
    for a in range(0, num_pages, step):
        n = min(step, num_pages - a)
        x = torch.randn((n, BT, d), generator=g, device=dev) * channel
        x *= torch.exp(0.7 * torch.randn((n, 1, 1), generator=g, device=dev))
        e = _exponent(x.abs().amax(dim=(1, 2)), fmt)
        s["pages"][a:a + n] = 0
        s["pages"][a:a + n, :BT * d] = _encode(x * torch.exp2(-e.float())[:, None, None], fmt).view(n, BT * d)
        s["exponents"][a:a + n] = e.to(torch.int8)

    # the new tokens' queries, keys and values stand in rows of one buffer, as a fused projection leaves them
    qkv = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=dev).half()
    s["q"] = qkv[:, :hq * d].view(T, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    s["out"] = torch.empty((T, hq, d), dtype=torch.float16, device=dev)
    if c["op"] == "append":
        s["q_out"] = torch.empty((T, hq, d), dtype=torch.float16, device=dev)
        seq = torch.repeat_interleave(torch.arange(S, device=dev), n_new.long())
        s["positions"] = (kv_len[seq] - indptr[seq + 1] + torch.arange(T, device=dev)).to(torch.int32)
        angle = torch.arange(s["max_len"], dtype=torch.float64, device=dev)[:, None] * (
            10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"]))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["lse"] = torch.empty((T, hq), dtype=torch.float32, device=dev)
    if own:
        import rank_delta_paged_gb300 as rdp
        s["batch"] = rdp.KVBatch(T, S, s["max_q"], max_blocks, indptr, kv_len, table)
        if c["op"] == "append":
            s["rope"] = rdp.KVRope(c["rot"], c["interleaved"], s["max_len"], s["cos"], s["sin"], s["positions"])
    return s


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import rank_delta_paged_gb300 as rdp
        row = s["q"].stride(0)
        if c["op"] == "append":
            rdp.slora_kv_append(s["kv"].kv, s["batch"], s["k"], row, s["v"], row, s["q"], row, s["q_out"],
                                s["q_out"].stride(0), c["hq"], s["rope"])
            return _cache(s)
        rdp.slora_kv_attend(s["kv"].kv, s["batch"], s["q"], row, c["hq"], s["out"], s["out"].stride(0), s["lse"],
                            s["scale"], True, c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    return _plain_append(s) if c["op"] == "append" else _plain_attend(s)


def _cache(s):
    return {"codes": s["pages"].view(_code_type(s["case"]["fmt"])), "exponents": s["exponents"], "q": s["q_out"]}


def _rotate(x, cos, sin, interleaved):
    """x [T][heads][d] fp32, cos and sin [T][rot/2]: the pairs of the first rot channels turned by their angles."""
    h = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    c, BT, d, fmt = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"]
    dev = s["kv_len"].device
    t = torch.arange(s["T"], device=dev)
    seq = torch.searchsorted(s["indptr"][1:].long(), t, right=True)
    pos = s["kv_len"][seq].long() - s["indptr"][seq + 1] + t
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c["interleaved"]))
    x = torch.stack([_rotate(s["k"].float(), cos, sin, c["interleaved"]), s["v"].float()], dim=2)   # [T][hkv][2][d]
    page = s["table"][seq, pos // BT].long()   # [T][hkv][2]

    # what each touched page needs for its new tokens
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=-1)
    top = torch.zeros(s["exponents"].shape[0], device=dev).scatter_reduce_(0, page.flatten(), size.flatten(), "amax")
    need = _exponent(top, fmt)

    # a block that already holds tokens keeps its exponent or grows it, and its codes with it
    first = s["kv_len"].long() - (s["indptr"][1:] - s["indptr"][:-1])
    held = (first % BT)[:, None, None].expand(-1, c["hkv"], 2)
    page0 = s["table"][torch.arange(s["S"], device=dev), first // BT].long()
    old = s["exponents"][page0].int()
    grown = torch.where(held > 0, torch.maximum(old, need[page0]), need[page0])
    s["exponents"].scatter_(0, page.flatten(), need[page].flatten().to(torch.int8))
    s["exponents"].scatter_(0, page0.flatten(), grown.flatten().to(torch.int8))
    rows = s["pages"][:, :BT * d].unflatten(1, (BT, d))
    codes = rows[page0]   # [S][hkv][2][BT][d]
    moved = _encode(codes.view(_code_type(fmt)).float() * torch.exp2((old - grown).float())[..., None, None], fmt)
    keep = torch.arange(BT, device=dev) < held[..., None]
    rows[page0] = torch.where(keep[..., None], moved, codes)

    unit = torch.exp2(-s["exponents"][page].float())
    rows[page, (pos % BT)[:, None, None].expand_as(page)] = _encode(x * unit[..., None], fmt)
    return _cache(s)


def _values(s, some, which, nb):
    """The cached keys (0) or values (1) of some sequences as fp32 [s][hkv][nb * BT][d]."""
    c = s["case"]
    page = s["table"][some, :nb, :, which].clamp(min=0).long()
    x = s["pages"][:, :s["BT"] * c["d"]][page].view(_code_type(c["fmt"])).float()
    x *= torch.exp2(s["exponents"][page].float())[..., None]
    return x.unflatten(-1, (s["BT"], c["d"])).transpose(1, 2).flatten(2, 3)


def _attend_some(s, some, most_q):
    """The sequences `some` (a slice), padded to the longest: at most most_q new tokens each."""
    c, dev = s["case"], s["kv_len"].device
    hq, hkv, d, w = c["hq"], c["hkv"], c["d"], c["window"]
    length, start = s["kv_len"][some].long(), s["indptr"][:-1][some].long()
    n_new = s["indptr"][1:][some].long() - start
    nb = -(-s["max_len"] // s["BT"])
    n = length.shape[0]
    i = torch.arange(most_q, device=dev)
    row = torch.where(i < n_new[:, None], start[:, None] + i, s["T"])                    # [n][most_q], T: none
    pos = (length - n_new)[:, None] + i
    j = torch.arange(nb * s["BT"], device=dev)
    seen = (j <= pos[..., None]) & (j < length[:, None, None])
    if w:
        seen &= j > pos[..., None] - w
    q = s["q"].float()[row.clamp(max=s["T"] - 1)].unflatten(2, (hkv, hq // hkv))          # [n][most_q][hkv][g][d]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                                            # [n][hkv][g * most_q][d]
    sc = (q @ _values(s, some, 0, nb).transpose(2, 3)).mul_(s["scale"]).unflatten(2, (hq // hkv, most_q))
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = sc.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    v = _values(s, some, 1, nb)
    v.masked_fill_((j >= length[:, None])[:, None, :, None], 0.0)
    o = (p.flatten(2, 3) @ v).unflatten(2, (hq // hkv, most_q)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4), lse.permute(0, 3, 1, 2)
    return row.flatten(), o.reshape(n * most_q, hq, d), lse.reshape(n * most_q, hq)


def _plain_attend(s):
    c, dev = s["case"], s["kv_len"].device
    out = torch.empty((s["T"] + 1, c["hq"], c["d"]), dtype=torch.float16, device=dev)
    lse = torch.empty((s["T"] + 1, c["hq"]), dtype=torch.float32, device=dev)
    if c["n_dec"]:
        row, o, l = _attend_some(s, slice(0, c["n_dec"]), 1)
        out[row], lse[row] = o.half(), l
    if c["n_multi"]:
        row, o, l = _attend_some(s, slice(c["n_dec"], s["S"]), s["max_q"])
        out[row], lse[row] = o.half(), l
    return {"out": out[:s["T"]], "lse": lse[:s["T"]]}


# ---- the definition in 64 bits --------------------------------------------------------------
def _f64(codes, fmt):
    """Bytes -> the numbers that the codes stand for."""
    b = codes.long()
    if fmt == "int8":
        return torch.where(b > 127, b - 256, b).double()
    sign, ex, man = 1.0 - 2.0 * (b >> 7).double(), (b >> 3) & 15, (b & 7).double()
    big = (1.0 + man / 8.0) * torch.exp2(ex.double() - 7.0)
    return sign * torch.where(ex > 0, big, man * 2.0 ** -9)


def _nearest(x, fmt):
    """The nearest code's number, ties to even, within the format's range; x in fp64."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return ((x / ulp).round() * ulp).clamp(-448, 448)


def _exact_exponent(amax, fmt):
    if amax == 0:
        return MIN_EXPONENT
    e = math.frexp(amax / (448.0 if fmt == "e4m3" else 127.0))
    return max(MIN_EXPONENT, e[1] - 1 if e[0] == 0.5 else e[1])


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    c, BT, d, fmt = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"]
    L = _lengths(c)
    if sum(-(-q // BT) + 1 for q, _ in L) > 6000:
        return None
    cos, sin = s["cos"].double(), s["sin"].double()
    dev, h = cos.device, c["rot"] // 2
    pair = [(2 * i, 2 * i + 1) if c["interleaved"] else (i, h + i) for i in range(h)]
    a, b = torch.tensor([p for p, _ in pair], device=dev), torch.tensor([p for _, p in pair], device=dev)

    def turn(x):
        x = x.double()
        y, at = x.clone(), s["positions"].long()
        for k in range(0, x.shape[1], 8):
            u, w = x[:, k:k + 8][..., a], x[:, k:k + 8][..., b]
            co, si = cos[at][:, None], sin[at][:, None]
            y[:, k:k + 8][..., a] = u * co - w * si
            y[:, k:k + 8][..., b] = w * co + u * si
        return y

    new = (turn(s["k"]), s["v"].double())
    pages, exps, table = s["pages"].clone(), s["exponents"].clone(), s["table"].tolist()
    exps_host = exps.tolist()
    at = 0
    for sq, (q, n) in enumerate(L):
        for blk in range((n - q) // BT, (n - 1) // BT + 1):
            lo, hi = max(n - q, blk * BT), min(n, (blk + 1) * BT)
            for w in (0, 1):
                rows = new[w][at + lo - (n - q):at + hi - (n - q)]                     # [tokens][hkv][d]
                fit = rows.abs().amax(dim=(0, 2)).tolist()
                held = lo - blk * BT
                ids = [table[sq][blk][hd][w] for hd in range(c["hkv"])]
                e = [_exact_exponent(v, fmt) for v in fit]
                if held:
                    e = [max(x, exps_host[p]) for x, p in zip(e, ids)]
                pid = torch.tensor(ids, device=dev)
                ev = torch.tensor(e, dtype=torch.float64, device=dev)
                cells = pages[pid][:, :BT * d].view(c["hkv"], BT, d)
                val = _f64(cells, fmt)
                if held:
                    oldv = torch.tensor([exps_host[p] for p in ids], dtype=torch.float64, device=dev)
                    val[:, :held] = _nearest(val[:, :held] * torch.exp2(oldv - ev)[:, None, None], fmt)
                val[:, held:held + hi - lo] = _nearest(rows.transpose(0, 1) * torch.exp2(-ev)[:, None, None], fmt)
                pages[pid, :BT * d] = val.float().to(_code_type(fmt)).view(torch.uint8).view(c["hkv"], BT * d)
                exps[pid] = ev.to(torch.int8)
        at += q
    return {"codes": pages.view(_code_type(fmt)), "exponents": exps, "q": turn(s["q"])}


def _exact_attend(s):
    c, BT, d, fmt, hq, hkv = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"], s["case"]["hq"], s["case"]["hkv"]
    L = _lengths(c)
    if work(c)["flops"] > 3.0e12:
        return None
    dev, g = s["pages"].device, hq // hkv
    out = torch.zeros((s["T"], hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for sq, (q, n) in enumerate(L):
        lo = max(0, n - q - c["window"] + 1) // BT if c["window"] else 0
        hi = -(-n // BT)
        key = torch.arange(lo * BT, hi * BT, device=dev)
        pos = torch.arange(n - q, n, device=dev)
        ok = key[None] <= pos[:, None]
        if c["window"]:
            ok &= pos[:, None] - key[None] < c["window"]
        per = max(1, int(2.0e8 // (max(q, 2 * d) * key.numel())))                          # KV heads at a time
        for k0 in range(0, hkv, per):
            k1 = min(hkv, k0 + per)
            k, v = ((_f64(s["pages"][p][..., :BT * d], fmt) * 2.0 ** s["exponents"][p].double()[..., None])
                    .view(hi - lo, k1 - k0, BT, d).transpose(0, 1).reshape(k1 - k0, (hi - lo) * BT, d)
                    for p in (s["table"][sq, lo:hi, k0:k1, 0].long(), s["table"][sq, lo:hi, k0:k1, 1].long()))
            for r in range(g):
                heads = torch.arange(k0, k1, device=dev) * g + r
                qq = s["q"][at:at + q][:, heads].double().transpose(0, 1)
                z = torch.einsum("hqd,hkd->hqk", qq, k) / math.sqrt(d)
                z = torch.where(ok, z, -math.inf)
                l = torch.logsumexp(z, dim=-1)
                lse[at:at + q, heads] = l.transpose(0, 1)
                out[at:at + q, heads] = torch.einsum("hqk,hkd->hqd", torch.exp(z - l[..., None]), v).transpose(0, 1)
        at += q
    return {"out": out, "lse": lse}
