// Append to the 8-bit paged KV cache: the new tokens' keys, rotated by their positions, and
// values become codes with one power-of-two scale per page; queries are rotated beside them.  With
// NORM, queries and keys are normalised per head before that.
//
//     y = (x - m) / sqrt(mean((x - m)^2) + eps) w        m = 0 or the mean of x (NORM)
//     (a, b) -> (a cos - b sin, b cos + a sin)      per pair of channels
//     e = max(e of the block if it holds tokens, smallest e with max |x| <= limit 2^e)
//     code = round(x 2^-e)
//
// What bounds it: reading the fp16 keys, values and queries once and writing the codes and the
// rotated queries once; for a few tokens, the chain of dependent reads (offsets, page ids and rows,
// angles and exponents).  The scale of a block needs the largest value of all its new tokens
// before the first code can be written, so a block's tokens stay in registers between the two.
//
// A lane holds 16 channels of a row, two chunks of 8.  Where rows turn in halves, whole or in part, they are
// partners (Own), with one set of angles; and what a row costs besides its channels (page ids,
// exponents, addresses) is shared by twice as many of them as with 8 a lane.  With 8 channels a lane and shuffles between partners
// 512 single tokens of 40 heads took 15.3 us instead of 10.5, 5046 tokens 65 instead of 54 (their queries two heads at a time).
//
// Sequences with one new token (append_one_kernel): a CTA takes a share of the token's rows, keys,
// values and queries alike; a row is a group of head_dim / 16 lanes, and all of its reads that do not
// depend on others go first.  (A CTA that goes on to other tokens with their offsets read ahead: no gain without
// norms, 21.9 us instead of 16.4 with them, for its registers.)
// Other sequences (append_kernel): the pages of all blocks that they touch form one list, of which
// every CTA takes an equal run, page after page by the whole CTA.  Shared memory, of which every thread
// reads what it has written itself, holds the rows of the page and the next two (asynchronous copies) and
// the rows' angles, which are the same for all heads of the block.  Their queries are a kernel of their own (rotate_kernel).
//
// Measured: 512 single tokens of 40 heads 10.6 us, with norms 14; 5046 tokens, of which 384 are single, of 32
// heads 47 us (4.4 TB/s), with the mean taken out and a weight for each head 71; 16381 tokens of 8 heads of 64 42 us
// (4.5 TB/s).  The instructions between the reads and the writes, the barrier of a page's maximum and the waits for
// exponents take the time.
// With two CTAs' worth of pages per block and CTAs found by a search of the token offsets, the
// 5046 tokens took 93 us: half the SMs had twice the work of the others.
// These times are of tokens that no block's exponent grows for.  Where it does, the group of lanes that has the
// page's token rescales the rows before it, eight at a time: the 512 single tokens, from a cold cache
// and with the call, take 26 us without, 45 with 215 of their 40960 pages growing and 55 with 9632 (INT8 25, 51 with
// 246, 87 with 11157); row by row before the new codes were written it was 71 and 100.  The 5046 tokens some 60, then 80 with
// 10720 pages growing.  Four rows per group of lanes, all their reads first: 9.3 us for the 512 tokens, 14.1 with norms, and 5.4 us
// instead of 2.9 for one token; for 2048 tokens 32.7 instead of 38.9 and 42.9 instead of 53.9 (not built: where it
// starts to win is not known).
// Pages above 8192 bytes have two rows per lane and one CTA per SM: 4096 tokens in prompts, cold, 52 us at 8192 bytes and
// 32 heads (3.3 TB/s), 70 at 10240 and 40 (3.1 TB/s), 91 at 16384 and 64 (3.7 TB/s).
#include <mutex>

#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"

namespace slora {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kBlockThreads = 512;  // append_kernel: 64 rows of 128 channels, or 128 of 64
constexpr int kMaxUnits = 128;     // pages of a block at a time, at most
constexpr int kSeqChunks = 64;
// append_kernel's CTAs per SM: those that fit with a row per lane (with 2 one fits, and the other half of
// the grid follows it).  4 and 8 cost 1 to 8 us more for their starts.
constexpr int kBlockCtas = 2;
constexpr int kStages = 3;         // append_kernel: a page's rows and those of the next two
constexpr int kQHeads = 2;         // rotate_kernel: query heads at a time, and CTAs per SM.  1 and 4: 3 to 6 % slower
constexpr int kQCtas = 3;

struct Params {
    AppendArgs a;
    // append_one_kernel:
    int32_t splits;      // CTAs per sequence
    int32_t units;       // rows per CTA
    int32_t q_rows;      // query heads that go with the keys and values
    int32_t q_run;       // rotate_kernel: heads per group of lanes
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

// The two chunks of 8 channels that lane ch of a row holds.  With the first 2 m chunks turning in halves, lanes below m hold
// a chunk and its partner, which turn by the same angles, and the others two chunks that do not turn; else chunk ch of
// either half of the row (m is half the row's chunks: AppendArgs::pairs).  With chunk ch of either half for every rotation, partners
// by shuffles and, where more than half the row turned, angles by channel, 96 of 128 channels took 95 us
// instead of 50 on the 5046 tokens.
struct Own {
    int lo, hi;
};
template <int D>
__device__ __forceinline__ Own own_chunks(const AppendArgs &a, int ch)
{
    const bool pair = ch < a.pairs;
    return {pair ? ch : ch + a.pairs, ch + (pair ? a.pairs : D / 16)};
}

// The angles of this lane's channels.
struct Rot {
    float c[8], s[8];
    bool on;            // whether its pair of chunks turns; adjacent pairs: whether the token does
};

// The angles of chunks ch and its partner where rows turn in halves, or (the first four, then the last four) of the lane's
// adjacent pairs.
template <int D>
__device__ __forceinline__ void load_rot(const AppendArgs &a, int32_t pos, int ch, Rot &r)
{
    r.on = a.rot != 0;
    if (r.on && (pos < 0 || pos >= a.n_pos)) {
        set_status(a.c.status, SLORA_DEV_BAD_POSITION);
        r.on = false;
    }
    const bool halves = !a.interleaved;
    if (halves && ch >= a.pairs) r.on = false;
    if (!r.on) return;
    const int64_t row = (int64_t)pos * (a.rot / 2);
    const float4 *cos = reinterpret_cast<const float4 *>(a.cos + row), *sin = reinterpret_cast<const float4 *>(a.sin + row);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = halves ? 2 * ch + i : ch + i * (D / 16);
        const bool turns = halves || ch * 8 + i * (D / 2) < a.rot;
        const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), none = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 c = turns ? __ldg(cos + k) : one, s = turns ? __ldg(sin + k) : none;
        r.c[4 * i] = c.x, r.c[4 * i + 1] = c.y, r.c[4 * i + 2] = c.z, r.c[4 * i + 3] = c.w;
        r.s[4 * i] = s.x, r.s[4 * i + 1] = s.y, r.s[4 * i + 2] = s.z, r.s[4 * i + 3] = s.w;
    }
}

// Rotates this lane's channels.  Products and sums are rounded one by one, so the codes do not depend on contraction.
template <int D>
__device__ __forceinline__ void rotate(const AppendArgs &a, const Rot &r, int ch, float (&x)[16])
{
    if (!r.on) return;
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            if (ch * 8 + (i >> 2) * (D / 2) < a.rot) {
                x[2 * i] = __fsub_rn(__fmul_rn(u, r.c[i]), __fmul_rn(w, r.s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(w, r.c[i]), __fmul_rn(u, r.s[i]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[i], w = x[8 + i];
            x[i] = __fsub_rn(__fmul_rn(u, r.c[i]), __fmul_rn(w, r.s[i]));
            x[8 + i] = __fadd_rn(__fmul_rn(w, r.c[i]), __fmul_rn(u, r.s[i]));
        }
    }
}

// Two fp32 numbers at a time, each rounded as by itself.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The sum over a row's channels in an order that depends on D alone: the even and the odd channels of each 8, one after
// another, then the eights of either half by twos.  No product is contracted into it.
template <int D>
__device__ __forceinline__ float row_sum(const AppendArgs &p, int ch, const uint64_t (&x)[8])
{
    constexpr int LPR = D / 16;
    const float2 t = unpair(add2(add2(add2(x[0], x[1]), x[2]), x[3])), u = unpair(add2(add2(add2(x[4], x[5]), x[6]), x[7]));
    float a = __fadd_rn(t.x, t.y), b = __fadd_rn(u.x, u.y);
    if (p.pairs != LPR) {
        // chunks ch and ch + LPR, from the lanes that hold them (Own)
        const int m = p.pairs, from_a = ch < m ? ch : ch - m, from_b = ch < m ? ch + LPR - m : ch;
        const float a0 = __shfl_sync(~0u, a, from_a, LPR), a1 = __shfl_sync(~0u, b, from_a, LPR);
        const float b0 = __shfl_sync(~0u, a, from_b, LPR), b1 = __shfl_sync(~0u, b, from_b, LPR);
        a = ch >= m && ch < 2 * m ? a1 : a0;
        b = ch < m && ch + LPR >= 2 * m ? b0 : b1;
    }
#pragma unroll
    for (int k = 1; k < LPR; k *= 2) {
        a = __fadd_rn(a, __shfl_xor_sync(~0u, a, k));
        b = __fadd_rn(b, __shfl_xor_sync(~0u, b, k));
    }
    return __fadd_rn(a, b);
}

// The norm of a row: x <- (x - mean) / sqrt(mean of squares + eps) * w, the mean taken out if `centered`, the head's weights
// from w on (nullptr: ones).  Every lane of the warp calls it; with SOME, rows that are not `on` keep their values.
// The mean is the sum times a power of two.
template <int D, bool SOME>
__device__ __forceinline__ void normalise(const AppendArgs &a, bool on, const float *w, int ch, float (&x)[16])
{
    uint64_t y[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = pair(x[2 * i], x[2 * i + 1]);
    if (a.centered) {
        const float m = -(row_sum<D>(a, ch, y) * (1.f / D));
        const uint64_t mm = pair(m, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = add2(y[i], mm);
    }
    // (the squares one by one: the compiler makes one rounding of a packed product and its sum)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = unpair(y[i]);
        z[i] = pair(__fmul_rn(t.x, t.x), __fmul_rn(t.y, t.y));
    }
    const float r = rsqrtf(__fadd_rn(row_sum<D>(a, ch, z) * (1.f / D), a.eps));
    const uint64_t rr = pair(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], rr);
    if (w != nullptr) {
        const Own own = own_chunks<D>(a, ch);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(w) + 2 * (i >> 1 ? own.hi : own.lo) + (i & 1));
            y[2 * i] = mul2(y[2 * i], pair(v.x, v.y));
            y[2 * i + 1] = mul2(y[2 * i + 1], pair(v.z, v.w));
        }
    }
    if (!SOME || on)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = unpair(y[i]);
            x[2 * i] = t.x;
            x[2 * i + 1] = t.y;
        }
}

// A row's two pieces of this lane.
struct Raw {
    uint4 a, b;
};
template <int D>
__device__ __forceinline__ Raw read_row(const __half *row, Own own)
{
    return {*reinterpret_cast<const uint4 *>(row + own.lo * 8), *reinterpret_cast<const uint4 *>(row + own.hi * 8)};
}

__device__ __forceinline__ void unpack(const Raw &v, float (&x)[16])
{
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The rotated query of this lane in fp16.
template <int D>
__device__ __forceinline__ void write_query(__half *row, Own own, const float (&x)[16])
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(row + own.lo * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(row + own.hi * 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The largest finite magnitude.
__device__ __forceinline__ float size_of(const float (&x)[16])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));      // passes over NaN
    if (__builtin_expect(m == INFINITY, 0)) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (fabsf(x[i]) < INFINITY) m = fmaxf(m, fabsf(x[i]));
    }
    return m;
}

// The largest of the lanes' values, none negative: their bit patterns are in the same order.
__device__ __forceinline__ float max_of(unsigned lanes, float m)
{
    return __uint_as_float(__reduce_max_sync(lanes, __float_as_uint(m)));
}

// INT8 codes with an infinity or a NaN among them: out of line, for its registers.
static __device__ __noinline__ uint32_t encode4_odd(float a, float b, float c, float d)
{
    return encode2<SLORA_KV_INT8>(a, b) | encode2<SLORA_KV_INT8>(c, d) << 16;
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float unit)
{
    if (FMT == SLORA_KV_INT8) {
        // The last bit of 1.5 2^23 + 128 is 1, so the sum's low byte is the code + 128, rounded to nearest even; the
        // bytes above are the same for -128 .. 127, which leaves infinities and NaN to the conversions, whose
        // pipe takes a quarter of the numbers per cycle.  Their -128 is no code, and no value is below -127 units but where
        // the exponent is held at its limit (new_exponent): there all codes are the conversions'.
        const float magic = 12583040.f;
        const uint32_t u = __float_as_uint(__fmaf_rn(a, unit, magic)), v = __float_as_uint(__fmaf_rn(b, unit, magic));
        const uint32_t w = __float_as_uint(__fmaf_rn(c, unit, magic)), x = __float_as_uint(__fmaf_rn(d, unit, magic));
        const uint32_t k = 0x4B400000u;
        if (__builtin_expect(((u ^ k) | (v ^ k) | (w ^ k) | (x ^ k)) < 256u && unit > pow2(-kExpLimit), 1))
            return __byte_perm(__byte_perm(u, v, 0x0040), __byte_perm(w, x, 0x0040), 0x5410) ^ 0x80808080u;
        return encode4_odd(a * unit, b * unit, c * unit, d * unit);
    }
    return encode2<FMT>(a * unit, b * unit) | encode2<FMT>(c * unit, d * unit) << 16;
}
// The exponent of new values: with weights it may be any, and what is read back ends at kExpLimit.
template <int FMT, bool NORM>
__device__ __forceinline__ int new_exponent(float m)
{
    const int e = fit_exponent<FMT>(m);
    return NORM && e > kExpLimit ? kExpLimit : e;
}

// This lane's codes to a row.
template <int D, int FMT>
__device__ __forceinline__ void write_codes(uint8_t *row, Own own, const float (&x)[16], float unit)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint2 *>(row + (h ? own.hi : own.lo) * 8) =
            make_uint2(encode4<FMT>(x[8 * h], x[8 * h + 1], x[8 * h + 2], x[8 * h + 3], unit),
                       encode4<FMT>(x[8 * h + 4], x[8 * h + 5], x[8 * h + 6], x[8 * h + 7], unit));
}

// This lane's sixteen codes of the rows r0, r0 + step, .. below `held` of a page divided by a power of two (unit < 1),
// N rows' reads at a time.
template <int D, int FMT, int N>
__device__ __forceinline__ void rescale_rows(uint8_t *page, int ch, int r0, int step, int held, float unit)
{
    uint4 *at = reinterpret_cast<uint4 *>(page + ch * 16);
#pragma unroll 1
    for (int k = r0; k < held; k += N * step) {
        uint4 v[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (k + j * step < held) v[j] = at[(k + j * step) * (D / 16)];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (k + j * step >= held) break;
            uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;
                decode4<FMT>(w[i], lo, hi);
                const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
                w[i] = encode4<FMT>(a.x, a.y, b.x, b.y, unit);
            }
            at[(k + j * step) * (D / 16)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__device__ __forceinline__ int32_t position(const AppendArgs &a, int32_t t, int32_t in_cache)
{
    return a.positions ? a.positions[t] : in_cache;
}

// Single tokens.  Row u of a token: keys, then values, of the KV heads, then query heads, so that most warps
// have rows of one kind and those of values do not rotate.
// CTAs per SM: with norms by 3, 4 (a few spills) 15.2 and 13.8 us for the 512 tokens; without, 5 fit.
template <int D, int FMT, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 4 : 5) append_one_kernel(const __grid_constant__ Params p)
{
    constexpr int LPR = D / 16;
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    const unsigned row_lanes = ((1u << LPR) - 1u) << (tid & 31 & -LPR);
    const Own own = own_chunks<D>(a, ch);
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
    const int32_t n_kv = a.c.n_kv, kv = 2 * n_kv, all = kv + p.q_rows;
    const int32_t u = part * p.units + grp;         // this group's row
    const bool live = grp < p.units && u < all, query = u >= kv, val = u >= n_kv && !query;
    const int32_t h = query ? u - kv : val ? u - n_kv : u;
    const int32_t blk = (len - 1) / a.c.bt, held = len - 1 - blk * a.c.bt;
    Raw raw = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    int32_t page = -1, old = kMinExponent;
    if (live) {
        const __half *src = query ? a.q + t0 * a.q_stride : val ? a.v + t0 * a.v_stride : a.k + t0 * a.k_stride;
        raw = read_row<D>(src + (int64_t)h * D, own);
        if (!query) page = a.b.table[((int64_t)s * a.b.max_blocks + blk) * kv + 2 * h + val];
    }
    const bool turns = live && !val;
    Rot rot;
    rot.on = false;
    if (turns) load_rot<D>(a, a.rot ? (a.positions ? a.positions[t0] : len - 1) : 0, ch, rot);
    if (live && !query) {
        if (page < 0 || page >= a.c.num_pages) {
            if (ch == 0) set_status(a.c.status, SLORA_DEV_BAD_PAGE);
            page = -1;
        } else if (held && ch == 0) {
            old = clamp_exponent(a.c.exps[page]);   // by the lane that writes it
        }
    }
    float x[16];
    unpack(raw, x);
    if (__any_sync(~0u, turns)) {
        if (NORM) {
            const float *w = query ? a.q_weight : a.k_weight;
            if (w != nullptr) w = turns ? w + h * (query ? a.q_weight_stride : a.k_weight_stride) : nullptr;
            normalise<D, true>(a, turns, w, ch, x);
        }
        rotate<D>(a, rot, ch, x);
    }
    const float m = max_of(row_lanes, size_of(x));
    const int was = __shfl_sync(~0u, old, 0, LPR);
    if (live && query) write_query<D>(a.q_out + t0 * a.q_out_stride + (int64_t)h * D, own, x);
    if (page < 0) return;
    const int fit = new_exponent<FMT, NORM>(m), e = held && was > fit ? was : fit;
    uint8_t *dst = a.c.pool + page * a.c.page_bytes;
    if (ch == 0) a.c.exps[page] = (int8_t)e;
    write_codes<D, FMT>(dst + held * D, own, x, pow2(-e));
    if (held && was < e) rescale_rows<D, FMT, 8>(dst, ch, 0, 1, held, pow2(was - e));
}

// The queries of a batch: q_run heads of one token per group of lanes, kQHeads at a time with the next ones on their way.
template <int D, bool NORM>
__global__ void __launch_bounds__(kThreads, kQCtas) rotate_kernel(const __grid_constant__ Params p)
{
    constexpr int LPR = D / 16, GROUPS = kThreads / LPR;
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    const unsigned row_lanes = ((1u << LPR) - 1u) << (tid & 31 & -LPR);
    const Own own = own_chunks<D>(a, ch);
    // as append_kernel
    griddep_launch_dependents();
    const int32_t per = (a.n_q + p.q_run - 1) / p.q_run;
    const int64_t total = (int64_t)a.b.T * per;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
#pragma unroll 1
    for (int64_t i0 = (int64_t)blockIdx.x * GROUPS; i0 < total; i0 += step) {
        const int64_t i = i0 + grp;
        const bool live = i < total;
        // (at most 2^20 tokens and 2^12 runs of heads)
        const int32_t t = live ? (int32_t)((uint32_t)i / (uint32_t)per) : 0, h0 = live ? (int32_t)(i - (int64_t)t * per) * p.q_run : a.n_q;
        const int32_t hend = h0 + p.q_run < a.n_q ? h0 + p.q_run : a.n_q;
        const __half *src = a.q + t * a.q_stride;
        Raw v[kQHeads];
        auto read = [&](int32_t h) {
#pragma unroll
            for (int k = 0; k < kQHeads; ++k) {
                v[k] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (h + k < hend) v[k] = read_row<D>(src + (int64_t)(h + k) * D, own);
            }
        };
        read(h0);
        int32_t pos = a.positions && live ? a.positions[t] : 0;
        // rows outside every sequence, and those of a sequence that is skipped, are left alone
        // the last of n from lo that starts at or before t, a lane for every other of 2 LPR parts of them.  (64 sequences of
        // a few tokens with 64 channels, whose rows have four lanes: one round more, and 0.6 us, with LPR parts.)
        int32_t lo = 0, n = a.b.S;
#pragma unroll 1
        while (__any_sync(~0u, n > 1)) {
            const int32_t step = (n + 2 * LPR - 1) / (2 * LPR), x = ch * step, y = x + LPR * step;
            const bool at_x = x < n && a.b.indptr[lo + x] <= t, at_y = y < n && a.b.indptr[lo + y] <= t;
            const int k = __popc(__ballot_sync(~0u, at_x) & row_lanes) + __popc(__ballot_sync(~0u, at_y) & row_lanes);
            if (k > 1) lo += (k - 1) * step, n -= (k - 1) * step;
            if (n > step) n = step;
        }
        const int32_t begin = a.b.indptr[lo], end = a.b.indptr[lo + 1], len = a.b.kv_len[lo];
        const bool mine = live && begin >= 0 && begin <= t && t < end && end <= a.b.T && end - begin <= a.b.max_q &&
                          len >= end - begin && !too_long(a.c, a.b, len);
        if (mine && !a.positions) pos = len - end + t;
        Rot r;
        r.on = false;
        if (mine) load_rot<D>(a, pos, ch, r);
        __half *dst = a.q_out + t * a.q_out_stride;
#pragma unroll 1
        for (int32_t h = 0; h < p.q_run; h += kQHeads) {
            Raw w[kQHeads];
#pragma unroll
            for (int k = 0; k < kQHeads; ++k) w[k] = v[k];
            if (h + kQHeads < p.q_run) read(h0 + h + kQHeads);
#pragma unroll
            for (int k = 0; k < kQHeads; ++k) {
                const int32_t head = h0 + h + k;
                const bool some = mine && head < hend;
                float x[16];
                unpack(w[k], x);
                if (NORM) normalise<D, false>(a, true, some && a.q_weight ? a.q_weight + head * a.q_weight_stride : nullptr, ch, x);
                rotate<D>(a, r, ch, x);
                if (some) write_query<D>(dst + (int64_t)head * D, own, x);
            }
        }
    }
    griddep_wait();
}

// A block's nt new rows of the pages [u0, u1), page after page by the whole CTA.
template <int D, int FMT, int PASSES, bool NORM>
__device__ __forceinline__ void full_rows(const AppendArgs &a, int32_t u0, int32_t u1, int32_t nt, int32_t held,
                                          int32_t row0, int32_t from, const int32_t *s_page, const int8_t *s_exp,
                                          uint32_t *s_max, int &turn)
{
    constexpr int LPR = D / 16, GROUPS = kBlockThreads / LPR;
    const int tid = fresh_tid(), ch = tid % LPR, grp = tid / LPR;
    const Own own = own_chunks<D>(a, ch);
    // Shared memory of which every thread has pieces of its own: the rows of this page and the next ones, and the angles.
    extern __shared__ uint4 s_own[];
    uint4 *ring = s_own + tid;
    float4 *s_rot = reinterpret_cast<float4 *>(s_own + kStages * PASSES * 2 * kBlockThreads) + tid;
    auto piece = [&](int slot, int i, int h) { return ring + ((slot * PASSES + i) * 2 + h) * kBlockThreads; };
    auto read = [&](int32_t u, int slot) {
        if (u < u1) {
            const __half *src = (u & 1 ? a.v : a.k) + (int64_t)(u >> 1) * D;
            const int64_t stride = u & 1 ? a.v_stride : a.k_stride;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = i * GROUPS + grp;
                if (r >= nt) break;
                const __half *row = src + (int64_t)(row0 + r) * stride;
                cp_async16(piece(slot, i, 0), row + own.lo * 8, 16);
                cp_async16(piece(slot, i, 1), row + own.hi * 8, 16);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) read(u0 + k, k);
    // a row's angles are those of all heads: a thread keeps its own in shared memory
    bool turns[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = i * GROUPS + grp;
        turns[i] = false;
        if (a.rot == 0 || r >= nt) continue;
        Rot rt;
        load_rot<D>(a, position(a, row0 + r, from + r), ch, rt);
        if (!rt.on) continue;
        turns[i] = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float *v = j < 2 ? rt.c + 4 * j : rt.s + 4 * (j - 2);
            s_rot[(4 * i + j) * kBlockThreads] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    int slot = 0;
#pragma unroll 1
    for (int32_t u = u0; u < u1; ++u, slot = slot == kStages - 1 ? 0 : slot + 1) {
        const bool val = u & 1;
        const int32_t page = s_page[u - u0];
        const int old = s_exp[u - u0];
        float x[PASSES][16];
        float m = 0.f;
        read(u + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
        cp_async_wait<kStages - 1>();
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            Raw raw = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (i * GROUPS + grp < nt) raw = {*piece(slot, i, 0), *piece(slot, i, 1)};
            unpack(raw, x[i]);
        }
        if (page < 0) continue;             // the whole CTA
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = i * GROUPS + grp;
            if (__all_sync(~0u, r >= nt)) break;
            if (!val) {
                if (NORM) normalise<D, false>(a, true, a.k_weight ? a.k_weight + (u >> 1) * a.k_weight_stride : nullptr, ch, x[i]);
                Rot rt;
                rt.on = turns[i];
                if (rt.on)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = s_rot[(4 * i + j) * kBlockThreads];
                        float *w = j < 2 ? rt.c + 4 * j : rt.s + 4 * (j - 2);
                        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                    }
                rotate<D>(a, rt, ch, x[i]);
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
        int e = new_exponent<FMT, NORM>(m);
        uint8_t *dst = a.c.pool + page * a.c.page_bytes;
        if (held && old > e) e = old;
        if (tid == 0) a.c.exps[page] = (int8_t)e;
        const float unit = pow2(-e);
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = i * GROUPS + grp;
            if (r < nt) write_codes<D, FMT>(dst + (held + r) * D, own, x[i], unit);
        }
        if (held && old < e) rescale_rows<D, FMT, 1>(dst, ch, grp, GROUPS, held, pow2(old - e));
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

template <int D, int FMT, int PASSES, bool NORM>
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
        full_rows<D, FMT, PASSES, NORM>(a, u0, u1, nt, held, row0, from, s_page, s_exp, s_max, turn);
        __syncthreads();                           // s_walk, s_page and s_exp have been read
    }
}

template <int D, int FMT, int PASSES, bool NORM>
__global__ void __launch_bounds__(kBlockThreads, PASSES == 1 ? 2 : 1) append_kernel(const __grid_constant__ Params p)
{
    // append_one_kernel, the one before, has waited for what came before it, and nothing here depends on
    // its results; the kernel after this one waits for what this one has waited for
    griddep_launch_dependents();
    append_blocks<D, FMT, PASSES, NORM>(p);
    griddep_wait();
}

template <class... Args>
cudaError_t start(void (*kernel)(Args...), const Params &p, int64_t ctas, cudaStream_t stream, int threads = kThreads,
                  size_t smem = 0)
{
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int FMT, int PASSES, bool NORM>
cudaError_t start_blocks(const Params &p, int64_t ctas, cudaStream_t stream)
{
    constexpr size_t smem = (size_t)PASSES * (2 * kStages + 4) * kBlockThreads * 16;
    {
        static std::mutex mu;
        static bool set[64] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 64 || !set[dev]) {
            e = cudaFuncSetAttribute(append_kernel<D, FMT, PASSES, NORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            if (dev < 64) set[dev] = true;
        }
    }
    return start(append_kernel<D, FMT, PASSES, NORM>, p, ctas, stream, kBlockThreads, smem);
}

template <int D, bool NORM>
cudaError_t launch_d(Params &p, int fmt, int num_sms, cudaStream_t stream, int *launches)
{
    constexpr int groups = kThreads / (D / 16);
    const AppendArgs &a = p.a;
    const bool e4m3 = fmt == SLORA_KV_E4M3;
    p.a.pairs = a.rot == 0 || a.interleaved ? D / 16 : a.rot / 16;
    cudaError_t e;
    {
        // a row per group of lanes
        p.q_rows = a.b.max_q == 1 ? a.n_q : 0;
        const int32_t all = 2 * a.c.n_kv + p.q_rows;
        p.splits = (all + groups - 1) / groups;
        p.units = (all + p.splits - 1) / p.splits;
        e = start(e4m3 ? append_one_kernel<D, SLORA_KV_E4M3, NORM> : append_one_kernel<D, SLORA_KV_INT8, NORM>, p,
                  (int64_t)a.b.S * p.splits, stream);
        *launches += e == cudaSuccess;
        if (e != cudaSuccess || a.b.max_q == 1) return e;
    }
    const int64_t ctas = (int64_t)kBlockCtas * num_sms;
    // rows of a block over the CTA's groups: one or two per lane (a page of up to 8192 or 16384 bytes)
    constexpr int block_groups = kBlockThreads / (D / 16);
    if (a.c.bt <= block_groups)
        e = e4m3 ? start_blocks<D, SLORA_KV_E4M3, 1, NORM>(p, ctas, stream) : start_blocks<D, SLORA_KV_INT8, 1, NORM>(p, ctas, stream);
    else
        e = e4m3 ? start_blocks<D, SLORA_KV_E4M3, 2, NORM>(p, ctas, stream) : start_blocks<D, SLORA_KV_INT8, 2, NORM>(p, ctas, stream);
    *launches += e == cudaSuccess;
    if (e != cudaSuccess || !a.q) return e;
    // Heads per group of lanes: a run of them shares the search for its token's sequence and the angles, and the next
    // ones' reads are under way; as long as the runs fill the SMs.  By 2, 4, 8 and 16: 5046 tokens of 32 heads 55.7, 50.1,
    // 47.7 and 46.3 us, with norms 79, 73, 71 and 74; 16381 of 32 heads of 64 channels 52.1, 44.7, 42.2 and 43.2.
    for (p.q_run = 8; p.q_run > 2; p.q_run /= 2)
        if ((int64_t)a.b.T * ((a.n_q + p.q_run - 1) / p.q_run) >= (int64_t)kQCtas * num_sms * groups) break;
    const int64_t items = (int64_t)a.b.T * ((a.n_q + p.q_run - 1) / p.q_run);
    int64_t q_ctas = (items + groups - 1) / groups;
    if (q_ctas > 32ll * num_sms) q_ctas = 32ll * num_sms;
    e = start(rotate_kernel<D, NORM>, p, q_ctas, stream);
    *launches += e == cudaSuccess;
    return e;
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, bool norm, int head_dim, int fmt, int num_sms, cudaStream_t stream,
                          int *launches)
{
    Params p = {};
    p.a = a;
    if (head_dim == 128)
        return norm ? launch_d<128, true>(p, fmt, num_sms, stream, launches)
                    : launch_d<128, false>(p, fmt, num_sms, stream, launches);
    return norm ? launch_d<64, true>(p, fmt, num_sms, stream, launches)
                : launch_d<64, false>(p, fmt, num_sms, stream, launches);
}

}  // namespace kv
}  // namespace slora
