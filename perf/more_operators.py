"""Timing cases of the 8-bit paged KV cache beyond append and attention: normed appends, attention with a window
and sinks, copies of pages, and the compaction of sequences.

A page of the pool holds the rows of one block of tokens for one KV head, keys or values, as
8-bit codes [block_tokens][head_dim] with one power-of-two scale per page (its exponent in an
int8 array indexed by page): value = code * 2**exponent.  The block table of a sequence lists,
per block and KV head, the page of the keys and the page of the values; pages are scattered.

  norm     normalises queries and keys per head, rotates them by their positions and writes keys and
           values to the cache: y = (x - mean) * w / sqrt(var + eps), or without the mean
  sinks    softmax(scale * q k^T) v of every new token over the last `window` tokens and the first
           `sinks` of its sequence; the blocks in between are gone from the table
  copy     rows of pages, and their exponents, to other pages
  compact  moves the kept tokens of each sequence to the front, in place or into other pages, a block's
           exponent being the smallest that its rows fit

With ``own`` false ``run`` computes them in elementary torch operations in fp32; with ``own``
true it makes the library's calls.
"""
import math
import random

import torch

own = False

#: Largest magnitude of a code, and the exponent a block of zeros gets.
E4M3_MAX, INT8_MAX, MIN_EXPONENT = 448.0, 127.0, -40


# ---- cases --------------------------------------------------------------------------------
_BATCH = dict(hidden=4096, hq=32, hkv=8, d=128, fmt="e4m3", n_dec=0, n_multi=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0,
              shape_seed=1)
_DEFAULTS = {
    "norm": dict(_BATCH, rot=128, interleaved=False, centered=False, per_head=False, eps=1e-6),
    "sinks": dict(_BATCH, window=1024, sinks=4),
    "copy": dict(hidden=4096, d=128, fmt="e4m3", n=1, partial=False, shape_seed=1),
    "compact": dict(hidden=4096, hkv=8, d=128, fmt="e4m3", n_seqs=1, ctx_lo=1, ctx_hi=1, kept_lo=1, kept_hi=1, tail=0,
                    per_head=False, in_place=False, shape_seed=1),
}


def _case(name, op, **more):
    return dict(_DEFAULTS[op], name=name, op=op, **more)


def listed():
    return [
        # one user's next token, grouped-query model: latency counts
        _case("norm_one_token", "norm", n_dec=1, ctx_lo=700, ctx_hi=700),
        # the 13B-shaped decode batch: 512 tokens, every sequence at its own length
        _case("norm_decode_13b", "norm", hidden=5120, hq=40, hkv=40, n_dec=512, ctx_lo=30, ctx_hi=1000),
        # the mixed iteration: 8 prompts of 256-1024 tokens beside 384 decode tokens; the mean taken out, a weight
        # for each head, adjacent pairs, half the row rotated, int8
        _case("norm_mixed_7b", "norm", hkv=32, fmt="int8", n_dec=384, n_multi=8, q_lo=256, q_hi=1024, ctx_hi=900,
              rot=64, interleaved=True, centered=True, per_head=True),
        # one user far into a stream: latency counts
        _case("sinks_one_token", "sinks", n_dec=1, ctx_lo=30000, ctx_hi=30000, window=1020, sinks=4),
        # many users at their own places in long streams
        _case("sinks_decode", "sinks", n_dec=256, ctx_lo=500, ctx_hi=60000, window=4096, sinks=64),
        # checking drafted tokens: a few new tokens per sequence, 64-wide heads, int8
        _case("sinks_draft_check", "sinks", d=64, fmt="int8", n_multi=48, q_lo=3, q_hi=8, ctx_lo=500, ctx_hi=20000,
              window=1000, sinks=4),
        # the next chunks of long prompts
        _case("sinks_chunks", "sinks", n_multi=8, q_lo=1500, q_hi=2048, ctx_lo=0, ctx_hi=30000, window=2048, sinks=128),
        # a request forks: its last block, of 8 KV heads, to pages of the fork's own
        _case("copy_fork", "copy", n=16, partial=True),
        # pages of many sequences to other places of the pool, at odd sizes
        _case("copy_many", "copy", hidden=5120, fmt="int8", n=30011),
        # the accepted tokens of drafted trees move up behind the sequence, in place
        _case("compact_drafts", "compact", n_seqs=24, ctx_lo=500, ctx_hi=8000, kept_lo=1, kept_hi=6, tail=24, in_place=True),
        # long sequences are cut to the tokens that counted, in pages of their own
        _case("compact_evict", "compact", n_seqs=6, ctx_lo=16000, ctx_hi=60000, kept_lo=2000, kept_hi=8000),
        # the same with a choice for each head, 64-wide heads, int8
        _case("compact_evict_heads", "compact", d=64, fmt="int8", n_seqs=16, ctx_lo=3000, ctx_hi=20000, kept_lo=1000,
              kept_hi=2500, per_head=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "sinks", "sinks", "sinks", "copy", "compact", "compact"])
    c = dict(_DEFAULTS[op], op=op, hidden=rng.choice([2048, 4096, 4096, 5120]), d=rng.choice([64, 128, 128]),
             fmt=rng.choice(["e4m3", "int8"]), shape_seed=rng.randrange(1 << 20))
    if op == "copy":
        c.update(n=_log_int(rng, 1, 30000), partial=rng.random() < 0.5)
        return c
    c["hkv"] = rng.choice([1, 2, 4, 8, 8, 16, 32, 40])
    if op == "compact":
        c.update(n_seqs=_log_int(rng, 1, 64), per_head=rng.random() < 0.4, in_place=rng.random() < 0.4)
        c["kept_hi"] = _log_int(rng, 1, 8000)
        c["kept_lo"] = c["kept_hi"] // rng.choice([1, 2, 10])
        c["ctx_hi"] = min(60000, c["kept_hi"] * rng.choice([1, 2, 8, 40]) + rng.randrange(0, 200))
        c["ctx_lo"] = max(1, c["ctx_hi"] // rng.choice([1, 2]))
        if rng.random() < 0.5:
            c["tail"] = rng.randrange(c["kept_hi"], 4 * c["kept_hi"] + 1)
        while _cost(c) > 0.9:
            if c["n_seqs"] > 1:
                c["n_seqs"] = (c["n_seqs"] + 1) // 2
            else:
                c["hkv"] = (c["hkv"] + 1) // 2
        return c
    c["hq"] = c["hkv"] * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * c["hkv"] <= 64])
    kind = rng.choice(["decode", "decode", "few", "prompt", "mixed"])
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
    if op == "norm":
        c.update(rot=rng.choice([c["d"], c["d"], c["d"] // 2, 0]), interleaved=rng.random() < 0.3,
                 centered=rng.random() < 0.3, per_head=rng.random() < 0.3, eps=rng.choice([1e-6, 1e-5]))
    else:
        c.update(window=_log_int(rng, 64, 8192), sinks=_log_int(rng, 1, 256))
    # no costlier than the largest listed case: fewer sequences, then shorter ones
    while _cost(c) > 0.9:
        if c["n_dec"] > 1 or c["n_multi"] > 1:
            c["n_dec"], c["n_multi"] = (c["n_dec"] + 1) // 2, (c["n_multi"] + 1) // 2
        else:
            c["ctx_lo"], c["ctx_hi"] = c["ctx_lo"] * 2 // 3, c["ctx_hi"] * 2 // 3
            c["q_hi"] = max(1, c["q_hi"] * 3 // 4)
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
    return c


def _block(c):
    return c["hidden"] * 2 // c["d"] // 8 * 8


def _lengths(c):
    """(new tokens, cache length with them) per sequence: the single-token sequences first."""
    r = random.Random(c["shape_seed"])
    n = [1] * c["n_dec"] + [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["n_multi"])]
    return [(q, q + r.randint(c["ctx_lo"], c["ctx_hi"])) for q in n]


def _moves(c):
    """(length, first destination, kept tokens) per sequence; a sequence's own length without a tail is its context."""
    r = random.Random(c["shape_seed"])
    out = []
    for _ in range(c["n_seqs"]):
        ctx, kept = r.randint(c["ctx_lo"], c["ctx_hi"]), r.randint(c["kept_lo"], c["kept_hi"])
        first, n = (ctx, ctx + c["tail"]) if c["tail"] else (0, ctx)
        out.append((n, first, min(kept, n - first)))
    return out


def _rows(c):
    """Rows of each page to copy."""
    r = random.Random(c["shape_seed"])
    BT = _block(c)
    return [r.randint(1, BT) for _ in range(c["n"])] if c["partial"] else [BT] * c["n"]


def _seen(q, n, c):
    """Keys that any of a sequence's new tokens sees, and the pairs of a new token and a key."""
    w, k = c["window"], c["sinks"]
    lo = max(0, n - q - w + 1)
    keys = n - lo + min(k, lo)
    pairs = sum(min(p + 1, w) + min(k, max(0, p + 1 - w)) for p in range(n - q, n))
    return keys, pairs


def _cost(c):
    """Share of the largest listed case in memory or arithmetic, whichever is more (the plain form pads)."""
    w = work(c)
    if c["op"] == "compact":
        kept = sum(k for _, _, k in _moves(c))
        return max(w["bytes"] / 1.2e8, sum(n for n, _, _ in _moves(c)) * c["hkv"] * c["d"] / 4.0e8, kept * c["hkv"] * c["d"] / 5.0e7)
    if c["op"] == "norm":
        pages = sum(-(-n // _block(c)) for _, n in _lengths(c)) * 2 * c["hkv"] * c["hidden"] * 2
        return max(w["bytes"] / 2.6e8, pages / 4.0e9)
    L = _lengths(c)
    pad = 0
    for sel in (L[:c["n_dec"]], L[c["n_dec"]:]):
        if sel:
            rows = max(q for q, _ in sel)
            pad += len(sel) * (c["sinks"] + c["window"] + rows) * (2 * c["hkv"] * c["d"] + rows * c["hq"])
    return max(pad / 3.5e9, w["bytes"] / 2.4e9, w["flops"] / 4.5e11)


def work(c):
    if c["op"] == "copy":
        return {"bytes": sum(_rows(c)) * c["d"] * 2 + c["n"] * (10 if not c["partial"] else 14), "flops": 0}
    if c["op"] == "compact":
        kept = sum(k for _, _, k in _moves(c))
        return {"bytes": kept * (4 * c["hkv"] * c["d"] + 4 * (c["hkv"] if c["per_head"] else 1)), "flops": 0}
    L = _lengths(c)
    T, d, hq, hkv = sum(q for q, _ in L), c["d"], c["hq"], c["hkv"]
    if c["op"] == "norm":
        kv = 2 * T * hkv * d
        return {"bytes": kv * 2 + kv + 2 * T * hq * d * 2 + T * c["rot"] * 4,
                "flops": T * (hkv + hq) * (3 * c["rot"] + 4 * d) + 2 * kv}
    keys, pairs = (sum(x) for x in zip(*(_seen(q, n, c) for q, n in L)))
    return {"bytes": 2 * keys * hkv * d + 2 * T * hq * d * 2 + 4 * T * hq, "flops": 4 * d * hq * pairs}


# ---- inputs -------------------------------------------------------------------------------
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


def _cache(s):
    return {"codes": s["pages"].view(_code_type(s["case"]["fmt"])), "exponents": s["exponents"]}


def _make_pages(s, g, num_pages, hkv):
    """The pool: normal values, some channels larger, every page with a spread of its own."""
    c, dev, BT, d = s["case"], s["dev"], s["BT"], s["case"]["d"]
    page_bytes = c["hidden"] * 2
    if own:
        from rank_delta_paged_gb300.harness import KVSession
        s["kv"] = KVSession(c["hidden"], num_pages, hkv, d, c["fmt"])
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
        e = _exponent(x.abs().amax(dim=(1, 2)), c["fmt"])
        s["pages"][a:a + n] = 0
        s["pages"][a:a + n, :BT * d] = _encode(x * torch.exp2(-e.float())[:, None, None], c["fmt"]).view(n, BT * d)
        s["exponents"][a:a + n] = e.to(torch.int8)


def _ints(dev, values):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _table(order, there, hkv):
    """The block table [S][blocks][hkv][2]: the next pages of `order` where a block is `there`, else -1."""
    table = torch.full((*there.shape, hkv, 2), -1, dtype=torch.int32, device=order.device)
    table[there] = order.view(-1, hkv, 2)
    return table


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=c, dev=dev, BT=_block(c))
    {"copy": _prepare_copy, "compact": _prepare_compact}.get(c["op"], _prepare_batch)(s, g)
    return s


def _prepare_copy(s, g):
    c, dev, n = s["case"], s["dev"], s["case"]["n"]
    order = torch.randperm(2 * n + 3, generator=g, device=dev)[:2 * n].to(torch.int32)
    s["src"], s["dst"] = order[:n].contiguous(), order[n:].contiguous()
    s["rows"] = _ints(dev, _rows(c)) if c["partial"] else None
    _make_pages(s, g, 2 * n + 3, 1)


def _prepare_compact(s, g):
    c, dev, BT, hkv = s["case"], s["dev"], s["BT"], s["case"]["hkv"]
    M = _moves(c)
    S, heads = len(M), hkv if c["per_head"] else 1
    blocks = -(-_ints(dev, [n for n, _, _ in M]) // BT)
    wide = max(-(-n // BT) for n, _, _ in M)
    there = torch.arange(wide, device=dev)[None] < blocks[:, None]
    begin, end = _ints(dev, [f // BT for _, f, _ in M]), -(-_ints(dev, [f + k for _, f, k in M]) // BT)
    dst_wide = max(-(-(f + k) // BT) for _, f, k in M)
    b = torch.arange(dst_wide, device=dev)[None]
    fresh = (b >= begin[:, None]) & (b < end[:, None])
    n_src = int(there.sum()) * 2 * hkv
    num_pages = n_src + (0 if c["in_place"] else int(fresh.sum()) * 2 * hkv)
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    s["table"] = _table(order[:n_src], there, hkv)
    s["dst_table"] = None if c["in_place"] else _table(order[n_src:], fresh, hkv)
    s["first"], s["kv_len"] = _ints(dev, [f for _, f, _ in M]), _ints(dev, [n for n, _, _ in M])
    s["indptr"], s["max_kept"] = _ints(dev, _sums([k for _, _, k in M])), max(k for _, _, k in M)
    # the kept tokens: any of those from the first destination on, in order
    kept = [torch.sort(f + torch.rand((heads, n - f), generator=g, device=dev).topk(k, dim=1).indices, dim=1).values
            for n, f, k in M]
    s["kept"] = torch.cat(kept, dim=1).to(torch.int32).contiguous()
    s["new_len"] = torch.zeros(S, dtype=torch.int32, device=dev)
    _make_pages(s, g, num_pages, hkv)
    if own:
        import rank_delta_paged_gb300 as rdp
        K = s["kept"].shape[1]
        s["keep"] = rdp.KVKeep(S, K, s["max_kept"], wide, s["indptr"], s["kept"], s["first"], s["kv_len"], s["table"],
                               dst_blocks=dst_wide, dst_table=s["dst_table"], head_stride=K if c["per_head"] else 0,
                               new_len=s["new_len"])


def _prepare_batch(s, g):
    c, dev, BT = s["case"], s["dev"], s["BT"]
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    L = _lengths(c)
    S, T = len(L), sum(q for q, _ in L)
    wide = max(-(-n // BT) for _, n in L) + 1
    s["indptr"], s["kv_len"] = _ints(dev, _sums([q for q, _ in L])), _ints(dev, [n for _, n in L])
    s.update(T=T, S=S, max_blocks=wide, max_q=max(q for q, _ in L), max_len=max(n for _, n in L), scale=1.0 / math.sqrt(d))
    at = torch.arange(wide, device=dev)[None] * BT
    n_new = s["indptr"][1:] - s["indptr"][:-1]
    there = at < s["kv_len"][:, None]
    if c["op"] == "sinks":      # blocks that no token sees any more have been given back
        there &= (at + BT > (s["kv_len"] - n_new - c["window"] + 1)[:, None]) | (at < c["sinks"])
    num_pages = int(there.sum()) * 2 * hkv
    s["table"] = _table(torch.randperm(num_pages, generator=g, device=dev).to(torch.int32), there, hkv)
    _make_pages(s, g, num_pages, hkv)

    # the new tokens' queries, keys and values stand in rows of one buffer, as a fused projection leaves them
    qkv = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=dev).half()
    s["q"] = qkv[:, :hq * d].view(T, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    if c["op"] == "norm":
        s["q_out"] = torch.empty((T, hq, d), dtype=torch.float16, device=dev)
        s["qw"], s["kw"] = (1.0 + 0.3 * torch.randn((h if c["per_head"] else 1, d), generator=g, device=dev) for h in (hq, hkv))
        if c["rot"]:
            angle = torch.arange(s["max_len"], dtype=torch.float64, device=dev)[:, None] * (
                10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"]))
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["out"] = torch.empty((T, hq, d), dtype=torch.float16, device=dev)
        s["lse"] = torch.empty((T, hq), dtype=torch.float32, device=dev)
    if own:
        import rank_delta_paged_gb300 as rdp
        s["batch"] = rdp.KVBatch(T, S, s["max_q"], wide, s["indptr"], s["kv_len"], s["table"])
        if c["op"] == "norm":
            each = d if c["per_head"] else 0
            s["norm"] = rdp.KVNorm(c["eps"], c["centered"], s["qw"], each, s["kw"], each)
            s["rope"] = rdp.KVRope(c["rot"], c["interleaved"], s["max_len"], s["cos"], s["sin"]) if c["rot"] else None


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "sinks": _plain_sinks, "copy": _plain_copy, "compact": _plain_compact}[s["case"]["op"]](s)


def _own(s):
    import rank_delta_paged_gb300 as rdp
    c = s["case"]
    if c["op"] == "copy":
        rdp.slora_kv_copy(s["kv"].kv, c["n"], s["src"], s["dst"], s["rows"])
        return _cache(s)
    if c["op"] == "compact":
        rdp.slora_kv_compact(s["kv"].kv, s["keep"])
        return dict(_cache(s), new_len=s["new_len"])
    row = s["q"].stride(0)
    if c["op"] == "norm":
        rdp.slora_kv_append_norm(s["kv"].kv, s["batch"], s["k"], row, s["v"], row, s["q"], row, s["q_out"],
                                 s["q_out"].stride(0), c["hq"], s["norm"], s["rope"])
        return dict(_cache(s), q=s["q_out"])
    rdp.slora_kv_attend_sinks(s["kv"].kv, s["batch"], s["q"], row, c["hq"], s["out"], s["out"].stride(0), s["lse"],
                              s["scale"], c["window"], c["sinks"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_copy(s):
    """Rows behind a page's last copied one stay as they were."""
    c, BT, d = s["case"], s["BT"], s["case"]["d"]
    src, dst = s["src"].long(), s["dst"].long()
    rows = s["pages"][:, :BT * d].unflatten(1, (BT, d))
    new = rows[src]
    if c["partial"]:
        new = torch.where((torch.arange(BT, device=s["dev"]) < s["rows"][:, None])[..., None], new, rows[dst])
    rows[dst] = new
    s["exponents"][dst] = s["exponents"][src]
    return _cache(s)


def _plain_compact(s):
    c, BT, d, dev, fmt = s["case"], s["BT"], s["case"]["d"], s["dev"], s["case"]["fmt"]
    hkv = c["hkv"]
    n = s["indptr"][1:] - s["indptr"][:-1]
    # rows to write: the kept ones, and those before the first of them in its block
    held = s["first"] % BT * (n > 0)
    count = (held + n).long()
    seq = torch.repeat_interleave(torch.arange(len(count), device=dev), count)
    i = torch.arange(seq.shape[0], device=dev) - (count.cumsum(0) - count)[seq] - held[seq]     # < 0: held
    to = s["first"][seq] + i
    at = (s["indptr"][seq] + i).clamp(min=0)
    origin = torch.where(i < 0, to, s["kept"][:, at].long())                                    # [heads or 1][rows]
    origin = origin.expand(hkv, -1).t()
    head = torch.arange(hkv, device=dev)
    page = s["table"][seq[:, None], origin // BT, head].long()                                  # [rows][hkv][2]
    dst_table = s["table"] if s["dst_table"] is None else s["dst_table"]
    dst = dst_table[seq, to // BT].long()
    rows = s["pages"][:, :BT * d].unflatten(1, (BT, d))
    x = rows[page, (origin % BT)[..., None].expand_as(page)].view(_code_type(fmt)).float()      # [rows][hkv][2][d]
    x *= torch.exp2(s["exponents"][page].float())[..., None]
    size = x.abs().amax(dim=-1)
    top = torch.zeros(s["exponents"].shape[0], device=dev).scatter_reduce_(0, dst.flatten(), size.flatten(), "amax")
    e = _exponent(top, fmt)[dst]
    s["exponents"].scatter_(0, dst.flatten(), e.flatten().to(torch.int8))
    rows[dst, (to % BT)[:, None, None].expand_as(dst)] = _encode(x * torch.exp2(-e.float())[..., None], fmt)
    s["new_len"].copy_(s["first"] + n)
    return dict(_cache(s), new_len=s["new_len"])


def _mean(x):
    """The mean over the last axis, of 64 or 128 channels, summed in an order that is the same for everybody: the even
    and the odd channels of each 8, one after another, then neighbours by twos."""
    y = x.unflatten(-1, (-1, 4, 2))
    y = (y[..., 0, :] + y[..., 1, :] + y[..., 2, :] + y[..., 3, :]).sum(-1)
    y = y.unflatten(-1, (-1, 2)).sum(-1).unflatten(-1, (-1, 2)).sum(-1).unflatten(-1, (-1, 2)).sum(-1)
    return (y.sum(-1) if x.shape[-1] == 128 else y[..., 0])[..., None] * (1.0 / x.shape[-1])


def _norm(x, w, c):
    x = x.float()
    if c["centered"]:
        x = x - _mean(x)
    return x * torch.rsqrt(_mean(x * x) + c["eps"]) * w


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


def _plain_norm(s):
    c, BT, d, fmt, dev = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"], s["dev"]
    t = torch.arange(s["T"], device=dev)
    seq = torch.searchsorted(s["indptr"][1:].long(), t, right=True)
    pos = s["kv_len"][seq].long() - s["indptr"][seq + 1] + t
    q, k = _norm(s["q"], s["qw"], c), _norm(s["k"], s["kw"], c)
    if c["rot"]:
        cos, sin = s["cos"][pos], s["sin"][pos]
        q, k = _rotate(q, cos, sin, c["interleaved"]), _rotate(k, cos, sin, c["interleaved"])
    s["q_out"].copy_(q)
    x = torch.stack([k, s["v"].float()], dim=2)                                                  # [T][hkv][2][d]
    page = s["table"][seq, pos // BT].long()                                                     # [T][hkv][2]

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
    codes = rows[page0]                                                                          # [S][hkv][2][BT][d]
    moved = _encode(codes.view(_code_type(fmt)).float() * torch.exp2((old - grown).float())[..., None, None], fmt)
    keep = torch.arange(BT, device=dev) < held[..., None]
    rows[page0] = torch.where(keep[..., None], moved, codes)

    unit = torch.exp2(-s["exponents"][page].float())
    rows[page, (pos % BT)[:, None, None].expand_as(page)] = _encode(x * unit[..., None], fmt)
    return dict(_cache(s), q=s["q_out"])


def _sinks_some(s, some, most_q):
    """The sequences `some` (a slice), padded to the longest: at most most_q new tokens each."""
    c, dev, BT = s["case"], s["dev"], s["BT"]
    hq, hkv, w, k = c["hq"], c["hkv"], c["window"], c["sinks"]
    length, start = s["kv_len"][some].long(), s["indptr"][:-1][some].long()
    n_new = s["indptr"][1:][some].long() - start
    n = length.shape[0]
    i = torch.arange(most_q, device=dev)
    row = torch.where(i < n_new[:, None], start[:, None] + i, s["T"])                    # [n][most_q], T: none
    pos = (length - n_new)[:, None] + i
    # the keys that any of them sees: the window's, and the first k where they lie before it
    lo = (length - n_new - w + 1).clamp(min=0)
    j = torch.cat([torch.arange(k, device=dev).expand(n, k), lo[:, None] + torch.arange(w + most_q - 1, device=dev)], dim=1)
    there = j < length[:, None]
    there[:, :k] &= j[:, :k] < lo[:, None]
    seen = there[:, None] & (j[:, None] <= pos[..., None]) & ((j[:, None] > pos[..., None] - w) | (j[:, None] < k))
    at = torch.where(there, j, (length - 1)[:, None])
    page = torch.where(there[..., None, None], s["table"][some][torch.arange(n, device=dev)[:, None], at // BT], 0).long()
    rows = s["pages"][:, :BT * c["d"]].unflatten(1, (BT, c["d"]))

    def values(which):
        p = page[..., which]                                                              # [n][keys][hkv]
        x = rows[p, (at % BT)[..., None].expand_as(p)].view(_code_type(c["fmt"])).float()
        x *= torch.exp2(s["exponents"][p].float())[..., None]
        return x.masked_fill_(~there[..., None, None], 0.0).transpose(1, 2)               # [n][hkv][keys][d]

    q = s["q"].float()[row.clamp(max=s["T"] - 1)].unflatten(2, (hkv, hq // hkv))          # [n][most_q][hkv][g][d]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                                            # [n][hkv][g * most_q][d]
    sc = (q @ values(0).transpose(2, 3)).mul_(s["scale"]).unflatten(2, (hq // hkv, most_q))
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = sc.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.flatten(2, 3) @ values(1)).unflatten(2, (hq // hkv, most_q)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4), lse.permute(0, 3, 1, 2)
    return row.flatten(), o.reshape(n * most_q, hq, c["d"]), lse.reshape(n * most_q, hq)


def _plain_sinks(s):
    c, dev = s["case"], s["dev"]
    out = torch.empty((s["T"] + 1, c["hq"], c["d"]), dtype=torch.float16, device=dev)
    lse = torch.empty((s["T"] + 1, c["hq"]), dtype=torch.float32, device=dev)
    if c["n_dec"]:
        row, o, l = _sinks_some(s, slice(0, c["n_dec"]), 1)
        out[row], lse[row] = o.half(), l
    if c["n_multi"]:
        row, o, l = _sinks_some(s, slice(c["n_dec"], s["S"]), s["max_q"])
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


def _bytes_of(values, fmt):
    return values.float().to(_code_type(fmt)).view(torch.uint8)


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return {"norm": _exact_norm, "sinks": _exact_sinks, "copy": _exact_copy, "compact": _exact_compact}[case["op"]](s)


def _exact_copy(s):
    c, d, dev = s["case"], s["case"]["d"], s["dev"]
    pages, exps = s["pages"].clone(), s["exponents"].clone()
    byte = torch.arange(pages.shape[1], device=dev)
    size = _ints(dev, _rows(c)) * d
    for a in range(0, c["n"], 4096):
        src, dst = s["src"][a:a + 4096].long(), s["dst"][a:a + 4096].long()
        pages[dst] = torch.where(byte < size[a:a + 4096, None], s["pages"][src], s["pages"][dst])
        exps[dst] = s["exponents"][src]
    return {"codes": pages.view(_code_type(c["fmt"])), "exponents": exps}


def _exact_compact(s):
    c, BT, d, fmt, hkv, dev = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"], s["case"]["hkv"], s["dev"]
    M = _moves(c)
    if sum(-(-(f + k) // BT) - f // BT for _, f, k in M) > 4000:
        return None
    pages, exps = s["pages"].clone(), s["exponents"].clone()
    to_table = s["table"] if s["dst_table"] is None else s["dst_table"]
    at, heads = 0, torch.arange(hkv, device=dev)
    for sq, (n, f, k) in enumerate(M):
        for blk in range(f // BT, -(-(f + k) // BT) if k else f // BT):
            lo, hi = max(f, blk * BT), min(f + k, (blk + 1) * BT)
            origin = s["kept"][:, at + lo - f:at + hi - f].long().expand(hkv, -1)
            if lo > blk * BT:
                origin = torch.cat([torch.arange(blk * BT, lo, device=dev).expand(hkv, -1), origin], dim=1)
            for w in (0, 1):
                page = s["table"][sq, origin // BT, heads[:, None], w].long()                    # [hkv][rows]
                val = _f64(s["pages"][:, :BT * d].unflatten(1, (BT, d))[page, origin % BT], fmt)
                val = val * torch.exp2(s["exponents"][page].double())[..., None]
                e = [_exact_exponent(v, fmt) for v in val.abs().amax(dim=(1, 2)).tolist()]
                ev = torch.tensor(e, dtype=torch.float64, device=dev)
                dst = to_table[sq, blk, :, w].long()
                pages[dst, :origin.shape[1] * d] = _bytes_of(_nearest(val * torch.exp2(-ev)[:, None, None], fmt), fmt).flatten(1)
                exps[dst] = ev.to(torch.int8)
        at += k
    return {"codes": pages.view(_code_type(fmt)), "exponents": exps, "new_len": _ints(dev, [f + k for _, f, k in M])}


def _exact_norm(s):
    c, BT, d, fmt, dev = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"], s["dev"]
    L = _lengths(c)
    if sum(-(-q // BT) + 1 for q, _ in L) > 6000:
        return None
    h = c["rot"] // 2
    pair = [(2 * i, 2 * i + 1) if c["interleaved"] else (i, h + i) for i in range(h)]
    a, b = (torch.tensor([p[i] for p in pair], dtype=torch.long, device=dev) for i in (0, 1))
    at = torch.cat([torch.arange(n - q, n, device=dev) for q, n in L])

    def turn(x, w):
        x = x.double()
        if c["centered"]:
            x = x - x.mean(dim=-1, keepdim=True)
        y = x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + c["eps"]) * w.double()
        if h:
            co, si = s["cos"].double()[at][:, None], s["sin"].double()[at][:, None]
            u, v = y[..., a], y[..., b]
            y[..., a], y[..., b] = u * co - v * si, v * co + u * si
        return y

    new = (turn(s["k"], s["kw"]), s["v"].double())
    pages, exps, table = s["pages"].clone(), s["exponents"].clone(), s["table"].tolist()
    exps_host = exps.tolist()
    t = 0
    for sq, (q, n) in enumerate(L):
        for blk in range((n - q) // BT, (n - 1) // BT + 1):
            lo, hi = max(n - q, blk * BT), min(n, (blk + 1) * BT)
            for w in (0, 1):
                rows = new[w][t + lo - (n - q):t + hi - (n - q)]                       # [tokens][hkv][d]
                fit = rows.abs().amax(dim=(0, 2)).tolist()
                held = lo - blk * BT
                ids = [table[sq][blk][hd][w] for hd in range(c["hkv"])]
                e = [_exact_exponent(v, fmt) for v in fit]
                if held:
                    e = [max(x, exps_host[p]) for x, p in zip(e, ids)]
                pid = torch.tensor(ids, device=dev)
                ev = torch.tensor(e, dtype=torch.float64, device=dev)
                val = _f64(pages[pid][:, :BT * d].view(c["hkv"], BT, d), fmt)
                if held:
                    oldv = torch.tensor([exps_host[p] for p in ids], dtype=torch.float64, device=dev)
                    val[:, :held] = _nearest(val[:, :held] * torch.exp2(oldv - ev)[:, None, None], fmt)
                val[:, held:held + hi - lo] = _nearest(rows.transpose(0, 1) * torch.exp2(-ev)[:, None, None], fmt)
                pages[pid, :BT * d] = _bytes_of(val, fmt).view(c["hkv"], BT * d)
                exps[pid] = ev.to(torch.int8)
        t += q
    return {"codes": pages.view(_code_type(fmt)), "exponents": exps, "q": turn(s["q"], s["qw"])}


def _exact_sinks(s):
    c, BT, d, fmt, hq, hkv = s["case"], s["BT"], s["case"]["d"], s["case"]["fmt"], s["case"]["hq"], s["case"]["hkv"]
    L = _lengths(c)
    if work(c)["flops"] > 1.0e12 or len(L) * hkv > 6000:
        return None
    dev, g = s["dev"], hq // hkv
    out = torch.zeros((s["T"], hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], hq), -math.inf, dtype=torch.float64, device=dev)
    rows = s["pages"][:, :BT * d].unflatten(1, (BT, d))
    t = 0
    for sq, (q, n) in enumerate(L):
        lo = max(0, n - q - c["window"] + 1)
        key = torch.cat([torch.arange(0, min(c["sinks"], lo), device=dev), torch.arange(lo, n, device=dev)])
        pos = torch.arange(n - q, n, device=dev)[:, None]
        ok = (key <= pos) & ((pos - key < c["window"]) | (key < c["sinks"]))
        per = max(1, int(2.0e8 // (max(q, 2 * d) * key.numel() * g)))                          # KV heads at a time
        for k0 in range(0, hkv, per):
            k1 = min(hkv, k0 + per)
            page = s["table"][sq, key // BT, k0:k1].long()                                     # [keys][heads][2]
            x = _f64(rows[page, (key % BT)[:, None, None].expand_as(page)], fmt) * torch.exp2(s["exponents"][page].double())[..., None]
            qq = s["q"][t:t + q, k0 * g:k1 * g].double().unflatten(1, (k1 - k0, g))
            z = torch.einsum("qhgd,khd->hgqk", qq, x[:, :, 0]) / math.sqrt(d)
            z = torch.where(ok, z, -math.inf)
            l = torch.logsumexp(z, dim=-1)
            lse[t:t + q, k0 * g:k1 * g] = l.permute(2, 0, 1).flatten(1)
            out[t:t + q, k0 * g:k1 * g] = torch.einsum("hgqk,khd->qhgd", torch.exp(z - l[..., None]), x[:, :, 1]).flatten(1, 2)
        t += q
    return {"out": out, "lse": lse}
