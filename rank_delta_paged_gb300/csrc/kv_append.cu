// Append to the 8-bit paged KV cache: the new tokens' keys, rotated by their positions, and
// values become codes with one power-of-two scale per page; queries are rotated beside them.
//
//     (a, b) -> (a cos - b sin, b cos + a sin)      per pair of channels
//     e = max(e of the block if it holds tokens, smallest e with max |x| <= limit 2^e)
//     code = round(x 2^-e)
//
// What bounds it: reading the fp16 keys, values and queries once and writing the codes and the
// rotated queries once; for a few tokens, the chain of dependent reads (offsets, page ids and rows,
// angles and exponents).  The scale of a block needs the largest value of all its new tokens
// before the first code can be written, so a block's tokens stay in registers between the two.
//
// Sequences with one new token (append_one_kernel): a CTA takes a share of the token's rows, keys,
// values and queries alike; a row is a group of head_dim / 8 lanes, which holds two of them at a
// time, and all of its reads that do not depend on others go first.
// Other sequences (append_kernel): the pages of all blocks that they touch form one list, of which
// every CTA takes an equal run, page after page by the whole CTA with the next page's rows under
// way.  Their queries are a kernel of their own (rotate_kernel).
//
// Measured: 512 single tokens of 40 heads 15 us; 5046 tokens, of which 384 are single, of 32 heads 65 us
// (3.2 TB/s); 16381 tokens of 8 heads of 64 51 us (3.7 TB/s).  The instructions between the reads and
// the writes (some 180 per warp and 16 bytes a lane) and the waits for a page's reads take the time.
// With two CTAs' worth of pages per block and CTAs found by a search of the token offsets, the
// 5046 tokens took 93 us: half the SMs had twice the work of the others.
// These times are of tokens that no block's exponent grows for.  Where it does, the group of lanes that has the
// page's token rescales the rows before it one after another: the 512 single tokens, from a cold cache
// and with the launch, take 23 us without, 58 with 681 of their 40960 pages growing and 136 with 9841 (INT8 66
// and 160); the 5046 tokens 71, then 91 with 4379 pages growing.
// Pages above 8192 bytes have more rows per lane: 4096 tokens in prompts, cold, 57 us at 8192 bytes and 32
// heads (3.0 TB/s), 98 at 10240 and 40 (2.2 TB/s: the registers for 3 rows at two CTAs per SM spill), 111
// at 16384 and 64 (3.0 TB/s).
#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"

namespace slora {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kBlockThreads = 512;  // append_kernel: two rows of 64 per group of 16 lanes
constexpr int kMaxUnits = 128;     // pages of a block at a time, at most
constexpr int kSeqChunks = 64;
// append_kernel's CTAs per SM: those that fit with 2 or 3 rows per lane (with 4 one fits, and the other half of
// the grid follows it).  4 and 8 cost 1 to 8 us more for their starts.
constexpr int kBlockCtas = 2;
constexpr int kQHeads = 4;         // query heads per group and step

struct Params {
    AppendArgs a;
    // append_one_kernel:
    int32_t splits;      // CTAs per sequence
    int32_t units;       // rows per CTA
    int32_t q_rows;      // query heads that go with the keys and values
};

// append_kernel's place in its run: what is left, and the part at hand.
struct Walk {
    int64_t left;                       // pages
    int32_t s, skip, unit;              // sequence, block from its first, page of the block
    int32_t u0, u1;                     // pages of the part at hand
    int32_t held, nt, row0, from;       // rows already there, new rows, first of them, its position
};

// threadIdx.x, read anew: what is made from it is not kept across a loop around its use.
__device__ __forceinline__ int fresh_tid()
{
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}

struct Rot {
    float c[8], s[8];
    bool on;
};

// The angles of the 8 channels that this lane holds (chunk ch of the row).
__device__ __forceinline__ void load_rot(const AppendArgs &a, int32_t pos, int ch, Rot &r)
{
    r.on = a.rot != 0 && ch * 8 < a.rot;
    if (r.on && (pos < 0 || pos >= a.n_pos)) {
        set_status(a.c.status, SLORA_DEV_BAD_POSITION);
        r.on = false;
    }
    if (!r.on) return;
    const int half = a.rot / 2;
    const int64_t row = (int64_t)pos * half;
    if (a.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(a.cos + row) + ch);
        const float4 s = __ldg(reinterpret_cast<const float4 *>(a.sin + row) + ch);
        r.c[0] = c.x, r.c[1] = c.y, r.c[2] = c.z, r.c[3] = c.w;
        r.s[0] = s.x, r.s[1] = s.y, r.s[2] = s.z, r.s[3] = s.w;
    } else {
        const int k = ch * 8 < half ? ch : ch - half / 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 c = __ldg(reinterpret_cast<const float4 *>(a.cos + row) + 2 * k + i);
            const float4 s = __ldg(reinterpret_cast<const float4 *>(a.sin + row) + 2 * k + i);
            r.c[4 * i] = c.x, r.c[4 * i + 1] = c.y, r.c[4 * i + 2] = c.z, r.c[4 * i + 3] = c.w;
            r.s[4 * i] = s.x, r.s[4 * i + 1] = s.y, r.s[4 * i + 2] = s.z, r.s[4 * i + 3] = s.w;
        }
        if (ch * 8 < half)      // a cos + b (-sin)
#pragma unroll
            for (int i = 0; i < 8; ++i) r.s[i] = -r.s[i];
    }
}

// Rotates the 8 channels of chunk ch; every lane of the row's group (LPR lanes) calls it.  Products and sums are
// rounded one by one, so the codes do not depend on contraction.
template <int LPR>
__device__ __forceinline__ void rotate(const AppendArgs &a, const Rot &r, int ch, float (&x)[8])
{
    if (a.rot == 0) return;
    if (a.interleaved) {
        if (r.on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], w = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(u, r.c[i]), __fmul_rn(w, r.s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(w, r.c[i]), __fmul_rn(u, r.s[i]));
            }
        }
        return;
    }
    const int m = a.rot / 16;            // chunks of half the rotated channels
    const int from = ch < m ? ch + m : (ch < 2 * m ? ch - m : ch);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(~0u, x[i], from, LPR);
        if (r.on) x[i] = __fadd_rn(__fmul_rn(x[i], r.c[i]), __fmul_rn(y, r.s[i]));
    }
}

__device__ __forceinline__ void unpack(uint4 v, float (&x)[8])
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The largest finite magnitude.
__device__ __forceinline__ float size_of(const float (&x)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));      // passes over NaN
    if (__builtin_expect(m == INFINITY, 0)) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(x[i]) < INFINITY) m = fmaxf(m, fabsf(x[i]));
    }
    return m;
}

// The largest of the lanes' values, none negative: their bit patterns are in the same order.
__device__ __forceinline__ float max_of(unsigned lanes, float m)
{
    return __uint_as_float(__reduce_max_sync(lanes, __float_as_uint(m)));
}

template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float unit)
{
    uint2 r;
    r.x = encode2<FMT>(x[0] * unit, x[1] * unit) | encode2<FMT>(x[2] * unit, x[3] * unit) << 16;
    r.y = encode2<FMT>(x[4] * unit, x[5] * unit) | encode2<FMT>(x[6] * unit, x[7] * unit) << 16;
    return r;
}

// Eight codes divided by a power of two (unit < 1).
template <int FMT>
__device__ __forceinline__ uint2 rescale8(uint2 v, float unit)
{
    float x[8];
    uint32_t h[4];
    decode4<FMT>(v.x, h[0], h[1]);
    decode4<FMT>(v.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    return encode8<FMT>(x, unit);
}

__device__ __forceinline__ int32_t position(const AppendArgs &a, int32_t t, int32_t in_cache)
{
    return a.positions ? a.positions[t] : in_cache;
}

// Single tokens.  Row u of a token: keys, then values, of the KV heads, then query heads, so that most warps
// have rows of one kind and those of values do not rotate.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) append_one_kernel(const __grid_constant__ Params p)
{
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR, ILP = 2;
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    const unsigned row_lanes = ((1u << LPR) - 1u) << (tid & 31 & -LPR);
    griddep_wait();
    griddep_launch_dependents();
    const int32_t s = (int32_t)(blockIdx.x / (unsigned)p.splits), part = (int32_t)(blockIdx.x - (unsigned)s * p.splits);
    const int32_t t0 = a.b.indptr[s], t1 = a.b.indptr[s + 1], len = a.b.kv_len[s];
    int32_t bad = 0;
    if (t0 < 0 || t1 < t0 || t1 > a.b.T || t1 - t0 > a.b.max_q)
        bad = SLORA_DEV_BAD_SEGMENT;
    else if (t1 > t0 && (len < t1 - t0 || too_long(a.c, a.b, len)))
        bad = SLORA_DEV_BAD_LENGTH;
    if (bad) {
        if (tid == 0) set_status(a.c.status, bad);
        return;
    }
    if (t1 - t0 != 1) return;
    const int32_t kv = 2 * a.c.n_kv, all = kv + p.q_rows;
    const int32_t u0 = part * p.units, u1 = u0 + p.units < all ? u0 + p.units : all;
    const int32_t blk = (len - 1) / a.c.bt, held = len - 1 - blk * a.c.bt;
    const int32_t *table = a.b.table + ((int64_t)s * a.b.max_blocks + blk) * kv;
    const int32_t pos = a.rot ? (a.positions ? a.positions[t0] : len - 1) : 0;
    Rot rot;
    rot.on = false;
#pragma unroll 1
    for (int32_t ub = u0; ub < u1; ub += ILP * GROUPS) {
        uint4 raw[ILP];
        int32_t page[ILP], old[ILP];
#pragma unroll
        for (int i = 0; i < ILP; ++i) {
            const int32_t u = ub + i * GROUPS + grp;
            raw[i] = make_uint4(0, 0, 0, 0);
            page[i] = -1;
            old[i] = kMinExponent;
            if (u < u1) {
                const bool val = u >= a.c.n_kv;
                const int32_t h = val ? u - a.c.n_kv : u;
                const __half *src = u >= kv ? a.q + t0 * a.q_stride + (int64_t)(u - kv) * D
                                   : val    ? a.v + t0 * a.v_stride + (int64_t)h * D
                                            : a.k + t0 * a.k_stride + (int64_t)h * D;
                raw[i] = *reinterpret_cast<const uint4 *>(src + ch * 8);
                if (u < kv) page[i] = table[2 * h + val];
            }
        }
        if (ub == u0) load_rot(a, pos, ch, rot);
#pragma unroll
        for (int i = 0; i < ILP; ++i) {
            const int32_t u = ub + i * GROUPS + grp;
            if (u < u1 && u < kv) {
                if (page[i] < 0 || page[i] >= a.c.num_pages) {
                    if (ch == 0) set_status(a.c.status, SLORA_DEV_BAD_PAGE);
                    page[i] = -1;
                } else if (held && ch == 0) {
                    old[i] = clamp_exponent(a.c.exps[page[i]]);    // by the lane that writes it
                }
            }
        }
#pragma unroll
        for (int i = 0; i < ILP; ++i) {
            const int32_t u = ub + i * GROUPS + grp;
            float x[8];
            unpack(raw[i], x);
            const bool turns = u < a.c.n_kv || u >= kv;
            if (__any_sync(~0u, turns)) {
                Rot r = rot;
                r.on = rot.on && turns;
                rotate<LPR>(a, r, ch, x);
            }
            float m = size_of(x);
            m = max_of(row_lanes, m);
            const int was = __shfl_sync(~0u, old[i], 0, LPR);
            if (u >= kv && u < u1) {
                uint4 w;
                __half2 *h = reinterpret_cast<__half2 *>(&w);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                *reinterpret_cast<uint4 *>(a.q_out + t0 * a.q_out_stride + (int64_t)(u - kv) * D + ch * 8) = w;
            }
            if (page[i] < 0) continue;
            const int fit = fit_exponent<FMT>(m), e = held && was > fit ? was : fit;
            uint8_t *dst = a.c.pool + page[i] * a.c.page_bytes + ch * 8;
            if (held && was < e) {
                const float unit = pow2(was - e);
#pragma unroll 1
                for (int k = 0; k < held; ++k) {
                    uint2 *w = reinterpret_cast<uint2 *>(dst + k * D);
                    *w = rescale8<FMT>(*w, unit);
                }
            }
            if (ch == 0) a.c.exps[page[i]] = (int8_t)e;
            *reinterpret_cast<uint2 *>(dst + held * D) = encode8<FMT>(x, pow2(-e));
        }
    }
}

// The queries of a batch: kQHeads heads of one token per group of lanes and step.
template <int D>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ Params p)
{
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    const unsigned row_lanes = ((1u << LPR) - 1u) << (tid & 31 & -LPR);
    // as append_kernel
    griddep_launch_dependents();
    const int32_t per = (a.n_q + kQHeads - 1) / kQHeads;
    const int64_t total = (int64_t)a.b.T * per;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
#pragma unroll 1
    for (int64_t i0 = (int64_t)blockIdx.x * GROUPS; i0 < total; i0 += step) {
        const int64_t i = i0 + grp;
        const bool live = i < total;
        const int32_t t = live ? (int32_t)(i / per) : 0, h0 = live ? (int32_t)(i - (int64_t)t * per) * kQHeads : 0;
        uint4 v[kQHeads];
#pragma unroll
        for (int k = 0; k < kQHeads; ++k)
            if (live && h0 + k < a.n_q)
                v[k] = *reinterpret_cast<const uint4 *>(a.q + t * a.q_stride + (int64_t)(h0 + k) * D + ch * 8);
        int32_t pos = a.positions && live ? a.positions[t] : 0;
        // rows outside every sequence, and those of a sequence that is skipped, are left alone
        int32_t lo = 0, n = a.b.S;               // the last of n from lo that starts at or before t, a lane per part of them
#pragma unroll 1
        while (__any_sync(~0u, n > 1)) {
            const int32_t step = (n + LPR - 1) / LPR;
            const bool before = ch * step < n && a.b.indptr[lo + ch * step] <= t;
            const int k = __popc(__ballot_sync(~0u, before) & row_lanes);
            if (k > 1) lo += (k - 1) * step, n -= (k - 1) * step;
            if (n > step) n = step;
        }
        const int32_t begin = a.b.indptr[lo], end = a.b.indptr[lo + 1], len = a.b.kv_len[lo];
        const bool mine = live && begin >= 0 && begin <= t && t < end && end <= a.b.T && end - begin <= a.b.max_q &&
                          len >= end - begin && !too_long(a.c, a.b, len);
        if (mine && !a.positions) pos = len - end + t;
        Rot r;
        r.on = false;
        if (mine) load_rot(a, pos, ch, r);
#pragma unroll
        for (int k = 0; k < kQHeads; ++k) {
            float x[8];
            if (!(mine && h0 + k < a.n_q)) v[k] = make_uint4(0, 0, 0, 0);
            unpack(v[k], x);
            rotate<LPR>(a, r, ch, x);
            uint4 w;
            __half2 *h = reinterpret_cast<__half2 *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
            if (mine && h0 + k < a.n_q)
                *reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + (int64_t)(h0 + k) * D + ch * 8) = w;
        }
    }
    griddep_wait();
}

// A block's nt new rows of the pages [u0, u1), page after page by the whole CTA.
template <int D, int FMT, int PASSES>
__device__ __forceinline__ void full_rows(const AppendArgs &a, int32_t u0, int32_t u1, int32_t nt, int32_t held,
                                          int32_t row0, int32_t from, const int32_t *s_page, const int8_t *s_exp,
                                          uint32_t *s_max, int &turn)
{
    constexpr int LPR = D / 8, GROUPS = kBlockThreads / LPR;
    const int tid = fresh_tid(), ch = tid % LPR, grp = tid / LPR;
    uint4 raw[PASSES];
    auto read = [&](int32_t u) {
        const __half *src = (u & 1 ? a.v : a.k) + (int64_t)(u >> 1) * D + ch * 8;
        const int64_t stride = u & 1 ? a.v_stride : a.k_stride;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = i * GROUPS + grp;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (r < nt) raw[i] = *reinterpret_cast<const uint4 *>(src + (int64_t)(row0 + r) * stride);
        }
    };
    read(u0);
#pragma unroll 1
    for (int32_t u = u0; u < u1; ++u) {
        const bool val = u & 1;
        const int32_t page = s_page[u - u0];
        const int old = s_exp[u - u0];
        float x[PASSES][8];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (i * GROUPS >= nt) break;
            unpack(raw[i], x[i]);
        }
        if (u + 1 < u1) read(u + 1);
        if (page < 0) continue;             // the whole CTA
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (i * GROUPS >= nt) break;
            const int r = i * GROUPS + grp;
            if (!val) {
                Rot rt;
                rt.on = false;
                if (r < nt) load_rot(a, position(a, row0 + r, from + r), ch, rt);
                rotate<LPR>(a, rt, ch, x[i]);
            }
            m = fmaxf(m, size_of(x[i]));
        }
        // the page's maximum, by turns in three words: one is added to, one read, one cleared
        m = max_of(~0u, m);
        if ((tid & 31) == 0) atomicMax(&s_max[turn], __float_as_uint(m));
        if (tid == 0) s_max[turn == 2 ? 0 : turn + 1] = 0;
        __syncthreads();
        m = __uint_as_float(s_max[turn]);
        turn = turn == 2 ? 0 : turn + 1;
        int e = fit_exponent<FMT>(m);
        uint8_t *dst = a.c.pool + page * a.c.page_bytes;
        if (held) {
            if (old >= e) {
                e = old;
            } else {
                const float unit = pow2(old - e);
#pragma unroll 1
                for (int r = grp; r < held; r += GROUPS) {
                    uint2 *w = reinterpret_cast<uint2 *>(dst + r * D + ch * 8);
                    *w = rescale8<FMT>(*w, unit);
                }
            }
        }
        if (tid == 0) a.c.exps[page] = (int8_t)e;
        const float unit = pow2(-e);
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = i * GROUPS + grp;
            if (r < nt) *reinterpret_cast<uint2 *>(dst + (held + r) * D + ch * 8) = encode8<FMT>(x[i], unit);
        }
    }
}

// The blocks that sequence s writes in append_kernel: none if it is skipped or has one new token or
// none (append_one_kernel's, which reports what is wrong).
__device__ __forceinline__ int32_t blocks_of(const AppendArgs &a, int64_t s)
{
    if (s >= a.b.S) return 0;
    const int32_t t0 = a.b.indptr[s], t1 = a.b.indptr[s + 1], len = a.b.kv_len[s], n = t1 - t0, bt = a.c.bt;
    if (t0 < 0 || t1 < t0 || t1 > a.b.T || n > a.b.max_q || n <= 1 || len < n || too_long(a.c, a.b, len))
        return 0;
    return (len - 1) / bt - (len - n) / bt + 1;
}

// The next part of a CTA's run, by one warp: pages of one block.  A function of its own, so that what it
// knows takes no registers while rows are in them.
__device__ __noinline__ void next_part(const Params &p, Walk &w, int32_t *s_page, int8_t *s_exp)
{
    const AppendArgs &a = p.a;
    const int32_t lane = threadIdx.x & 31, bt = a.c.bt, all = 2 * a.c.n_kv, S = a.b.S;
    int64_t left = w.left;
    int32_t q = w.s, skip = w.skip;
    // the first sequence at or behind q that has block `skip`, counted from q
    bool found = false;
#pragma unroll 1
    while (left > 0 && !found && q < S) {
        const int32_t nb = blocks_of(a, (int64_t)q + lane);
        int32_t sum = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned beyond = __ballot_sync(~0u, sum > skip);
        found = beyond != 0;
        const int l = found ? __ffs(beyond) - 1 : 31;
        skip -= __shfl_sync(~0u, found ? sum - nb : sum, l);
        q += found ? l : 32;
    }
    int32_t u0 = 0, u1 = 0;
    if (found) {
        const int32_t t0 = a.b.indptr[q], n = a.b.indptr[q + 1] - t0, len = a.b.kv_len[q];
        const int32_t p0 = len - n;                                   // position of the first new token
        const int32_t blk = p0 / bt + skip;
        const int32_t from = blk * bt > p0 ? blk * bt : p0, to = (blk + 1) * bt < len ? (blk + 1) * bt : len;
        const int32_t held = from - blk * bt;
        u0 = w.unit;
        u1 = left < all - u0 ? u0 + (int32_t)left : all;
        if (u1 > u0 + kMaxUnits) u1 = u0 + kMaxUnits;
        // the block's pages of this CTA and, if it holds tokens, their exponents
#pragma unroll 1
        for (int32_t u = u0 + lane; u < u1; u += 32) {
            int32_t page = a.b.table[((int64_t)q * a.b.max_blocks + blk) * all + u];
            if (page < 0 || page >= a.c.num_pages) {
                set_status(a.c.status, SLORA_DEV_BAD_PAGE);
                page = -1;
            }
            s_page[u - u0] = page;
            s_exp[u - u0] = (int8_t)(held && page >= 0 ? clamp_exponent(a.c.exps[page]) : 0);
        }
        __syncwarp();                       // w.unit has been read
        if (lane == 0) {
            w.held = held;
            w.nt = to - from;
            w.row0 = t0 + from - p0;
            w.from = from;
            w.left = left - (u1 - u0);
            w.s = q;
            w.skip = u1 == all ? skip + 1 : skip;
            w.unit = u1 == all ? 0 : u1;
        }
    }
    if (lane == 0) {
        w.u0 = u0;
        w.u1 = u1;
    }
}

template <int D, int FMT, int PASSES>
__device__ __forceinline__ void append_blocks(const Params &p)
{
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x;
    __shared__ uint32_t s_max[3];
    __shared__ int32_t s_page[kMaxUnits];
    __shared__ int8_t s_exp[kMaxUnits];
    __shared__ int64_t s_sum[kSeqChunks];
    __shared__ Walk s_walk;
    const int lane = tid & 31;
    const int32_t all = 2 * a.c.n_kv, S = a.b.S;
    // ---- the list of blocks; every CTA sums it for itself ------------------------------------
    const int32_t per = ((S + kSeqChunks - 1) / kSeqChunks + 31) / 32 * 32, chunks = (S + per - 1) / per;
    if (tid == 0) s_max[0] = 0;
    if (tid >= chunks && tid < kSeqChunks) s_sum[tid] = 0;
#pragma unroll 1
    for (int c = tid >> 5; c < chunks; c += kBlockThreads / 32) {
        int64_t t = 0;
#pragma unroll 1
        for (int64_t q = (int64_t)c * per + lane; q < (int64_t)(c + 1) * per; q += 32) t += blocks_of(a, q);
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) s_sum[c] = t;
    }
    __syncthreads();
    // Warp 0 walks the list; what it knows stands in shared memory between its steps, since the rows
    // of a page take all the registers there are.
    if (tid < 32) {
        const int64_t v0 = s_sum[2 * lane], v1 = s_sum[2 * lane + 1];
        int64_t W = v0 + v1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(~0u, W, o);
            if (lane >= o) W += x;
        }
        const int64_t before = W - v0 - v1;
        W = __shfl_sync(~0u, W, 31) * all;
        // an equal run of pages per CTA
        const int64_t run = (W + gridDim.x - 1) / gridDim.x, w0 = blockIdx.x * run;
        int64_t skip = w0 / all;                   // blocks before this CTA's first
        const int32_t unit = (int32_t)(w0 - skip * all);
        const int at = 31 - __clz(__ballot_sync(~0u, before <= skip));
        skip -= __shfl_sync(~0u, before, at);
        const int64_t first = __shfl_sync(~0u, v0, at);
        if (lane == 0) {
            s_walk.left = w0 + run < W ? run : W - w0;
            s_walk.s = 2 * at * per + (skip >= first ? per : 0);
            s_walk.skip = (int32_t)(skip >= first ? skip - first : skip);
            s_walk.unit = unit;
        }
        __syncwarp();
    }
    int turn = 0;
#pragma unroll 1
    for (;;) {
        if (tid < 32) next_part(p, s_walk, s_page, s_exp);
        __syncthreads();
        const int32_t u0 = s_walk.u0, u1 = s_walk.u1, nt = s_walk.nt, held = s_walk.held, row0 = s_walk.row0,
                      from = s_walk.from;
        if (u1 == 0) return;
        // unit: KV head * 2 + (0 keys, 1 values)
        full_rows<D, FMT, PASSES>(a, u0, u1, nt, held, row0, from, s_page, s_exp, s_max, turn);
        __syncthreads();                           // s_walk, s_page and s_exp have been read
    }
}

template <int D, int FMT, int PASSES>
__global__ void __launch_bounds__(kBlockThreads, PASSES <= 3 ? 2 : 1) append_kernel(const __grid_constant__ Params p)
{
    // append_one_kernel, the one before, has waited for what came before it, and nothing here depends on
    // its results; the kernel after this one waits for what this one has waited for
    griddep_launch_dependents();
    append_blocks<D, FMT, PASSES>(p);
    griddep_wait();
}

template <class... Args>
cudaError_t start(void (*kernel)(Args...), const Params &p, int64_t ctas, cudaStream_t stream, int threads = kThreads)
{
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_d(Params &p, int fmt, int num_sms, cudaStream_t stream, int *launches)
{
    constexpr int groups = kThreads / (D / 8);
    const AppendArgs &a = p.a;
    const bool e4m3 = fmt == SLORA_KV_E4M3;
    cudaError_t e;
    {
        // two rows per group of lanes and CTA
        p.q_rows = a.b.max_q == 1 ? a.n_q : 0;
        const int32_t all = 2 * a.c.n_kv + p.q_rows;
        p.splits = (all + 2 * groups - 1) / (2 * groups);
        p.units = (all + p.splits - 1) / p.splits;
        e = start(e4m3 ? append_one_kernel<D, SLORA_KV_E4M3> : append_one_kernel<D, SLORA_KV_INT8>, p,
                  (int64_t)a.b.S * p.splits, stream);
        *launches += e == cudaSuccess;
        if (e != cudaSuccess || a.b.max_q == 1) return e;
    }
    const int64_t ctas = (int64_t)kBlockCtas * num_sms;
    // rows of a block over the CTA's groups: the registers for 2, 3 or 4 of them per lane (a
    // page of up to 8192, 12288 or 16384 bytes)
    constexpr int block_groups = kBlockThreads / (D / 8);
    const int passes = (a.c.bt + block_groups - 1) / block_groups;
    if (passes <= 2)
        e = start(e4m3 ? append_kernel<D, SLORA_KV_E4M3, 2> : append_kernel<D, SLORA_KV_INT8, 2>, p, ctas, stream, kBlockThreads);
    else if (passes <= 3)
        e = start(e4m3 ? append_kernel<D, SLORA_KV_E4M3, 3> : append_kernel<D, SLORA_KV_INT8, 3>, p, ctas, stream, kBlockThreads);
    else
        e = start(e4m3 ? append_kernel<D, SLORA_KV_E4M3, 4> : append_kernel<D, SLORA_KV_INT8, 4>, p, ctas, stream, kBlockThreads);
    *launches += e == cudaSuccess;
    if (e != cudaSuccess || !a.q) return e;
    const int64_t items = (int64_t)a.b.T * ((a.n_q + kQHeads - 1) / kQHeads);
    int64_t q_ctas = (items + groups - 1) / groups;
    if (q_ctas > 32ll * num_sms) q_ctas = 32ll * num_sms;
    e = start(rotate_kernel<D>, p, q_ctas, stream);
    *launches += e == cudaSuccess;
    return e;
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int head_dim, int fmt, int num_sms, cudaStream_t stream, int *launches)
{
    Params p = {};
    p.a = a;
    return head_dim == 128 ? launch_d<128>(p, fmt, num_sms, stream, launches)
                           : launch_d<64>(p, fmt, num_sms, stream, launches);
}

}  // namespace kv
}  // namespace slora
