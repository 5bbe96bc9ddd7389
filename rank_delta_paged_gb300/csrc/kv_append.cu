// Append to the 8-bit paged KV cache: the new tokens' keys, rotated by their positions, and
// values become codes with one power-of-two scale per page; queries are rotated beside them.
//
//     (a, b) -> (a cos - b sin, b cos + a sin)      per pair of channels
//     e = max(e of the block if it holds tokens, smallest e with max |x| <= limit 2^e)
//     code = round(x 2^-e)
//
// What bounds it: reading the fp16 keys, values and queries once and writing the codes and the
// rotated queries once.  The scale of a block needs the largest value of all its new tokens
// before the first code can be written, so a block's tokens stay in registers between the
// two.  The work is cut by (block of the cache, run of its pages): a CTA finds its block by a binary
// search of the token offsets, in which block `slot` of the batch is
// counted as if every sequence before it had touched floor(tokens / block) + 2 blocks
// (at least as many as it can), so no prefix sum over the sequences has to be made first.
// Blocks with at most kFew new tokens (every decode token) go to groups of head_dim / 8 lanes,
// one page each, with no barrier; fuller blocks to the whole CTA, page after page.
#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"

namespace slora {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kFew = 4;
constexpr int kMaxUnits = 128;     // pages per CTA at most
constexpr int kQHeads = 4;         // query heads per group and step

struct Params {
    AppendArgs a;
    int32_t slots;       // blocks of the cache, counted as above
    int32_t per_seq;     // slots per sequence besides its tokens / block: 2, or 1 and no search if max_q is 1
    int32_t splits;      // CTAs per slot
    int32_t units;       // pages per CTA
    int64_t kv_ctas;     // slots * splits; later CTAs rotate queries
};

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
    const bool low = ch < m;
    const int from = low ? ch + m : (ch < 2 * m ? ch - m : ch);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(~0u, x[i], from, LPR);
        if (r.on) {
            const float p = __fmul_rn(x[i], r.c[i]), q = __fmul_rn(y, r.s[i]);
            x[i] = low ? __fsub_rn(p, q) : __fadd_rn(p, q);
        }
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

__device__ __forceinline__ float size_of(const float (&x)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        if (u < 0x7F800000u) m = fmaxf(m, __uint_as_float(u));
    }
    return m;
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

// A block's nt <= kFew new rows of the pages [u0, u1): one page per group of lanes and step.
// The rows' loads do not need the pages and go first; for a single token the next step's are
// under way while one is written.
template <int D, int FMT>
__device__ __forceinline__ void few_rows(const AppendArgs &a, int32_t u0, int32_t u1, int32_t nt, int32_t held,
                                         int32_t row0, int32_t from, const int32_t *s_page, const int8_t *s_exp)
{
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    auto row_of = [&](int32_t u, int i) {
        const __half *src = u & 1 ? a.v : a.k;
        const int64_t stride = u & 1 ? a.v_stride : a.k_stride;
        return *reinterpret_cast<const uint4 *>(src + (int64_t)(row0 + i) * stride + (int64_t)(u >> 1) * D + ch * 8);
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 next = u0 + grp < u1 ? row_of(u0 + grp, 0) : zero;
    Rot rot0;
    rot0.on = false;
    load_rot(a, position(a, row0, from), ch, rot0);
    __syncthreads();
    for (int32_t ub = u0; ub < u1; ub += GROUPS) {
        const int32_t u = ub + grp;
        const bool val = u & 1;
        const int32_t page = u < u1 ? s_page[u - u0] : -1;
        uint4 raw[kFew];
        raw[0] = next;
#pragma unroll
        for (int i = 1; i < kFew; ++i) raw[i] = i < nt && page >= 0 ? row_of(u, i) : zero;
        next = u + GROUPS < u1 ? row_of(u + GROUPS, 0) : zero;
        float x[kFew][8];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            if (i >= nt) break;
            unpack(raw[i], x[i]);
            Rot r = rot0;
            if (i > 0 && !val && page >= 0) load_rot(a, position(a, row0 + i, from + i), ch, r);
            r.on = r.on && !val;
            rotate<LPR>(a, r, ch, x[i]);
            m = fmaxf(m, size_of(x[i]));
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (page < 0) continue;
        int e = fit_exponent<FMT>(m);
        uint8_t *dst = a.c.pool + page * a.c.page_bytes;
        if (held) {
            const int old = s_exp[u - u0];
            if (old >= e) {
                e = old;
            } else {
                const float unit = pow2(old - e);
#pragma unroll 1
                for (int r = 0; r < held; ++r) {
                    uint2 *w = reinterpret_cast<uint2 *>(dst + r * D + ch * 8);
                    *w = rescale8<FMT>(*w, unit);
                }
            }
        }
        if (ch == 0) a.c.exps[page] = (int8_t)e;
        const float unit = pow2(-e);
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            if (i >= nt) break;
            *reinterpret_cast<uint2 *>(dst + (held + i) * D + ch * 8) = encode8<FMT>(x[i], unit);
        }
    }
}

template <int D, int FMT, int PASSES>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Params p)
{
    constexpr int LPR = D / 8;                 // lanes per row
    constexpr int GROUPS = kThreads / LPR;
    const AppendArgs &a = p.a;
    const int tid = threadIdx.x, ch = tid % LPR, grp = tid / LPR;
    __shared__ float s_max[2][kThreads / 32];
    __shared__ int32_t s_page[kMaxUnits];
    __shared__ int8_t s_exp[kMaxUnits];

    griddep_wait();
    griddep_launch_dependents();

    if (blockIdx.x >= p.kv_ctas) {
        // ---- queries: kQHeads heads of one token per group --------------------------------
        const int32_t per = (a.n_q + kQHeads - 1) / kQHeads;
        const int64_t total = (int64_t)a.b.T * per;
        const int64_t step = (int64_t)(gridDim.x - p.kv_ctas) * GROUPS;
        for (int64_t i0 = (blockIdx.x - p.kv_ctas) * GROUPS; i0 < total; i0 += step) {
            const int64_t i = i0 + grp;
            const bool live = i < total;
            const int32_t t = live ? (int32_t)(i / per) : 0, h0 = live ? (int32_t)(i - (int64_t)t * per) * kQHeads : 0;
            bool mine = live;
            int32_t pos = 0;
            if (a.positions) {
                if (live) pos = a.positions[t];
            } else {
                int32_t lo = 0, hi = a.b.S - 1;      // last sequence that starts at or before t
                while (lo < hi) {
                    const int32_t mid = (lo + hi + 1) / 2;
                    if (a.b.indptr[mid] <= t) lo = mid; else hi = mid - 1;
                }
                const int32_t end = a.b.indptr[lo + 1];
                mine = live && a.b.indptr[lo] <= t && t < end;
                if (mine) pos = a.b.kv_len[lo] - end + t;
            }
            uint4 v[kQHeads];
#pragma unroll
            for (int k = 0; k < kQHeads; ++k)
                if (mine && h0 + k < a.n_q)
                    v[k] = *reinterpret_cast<const uint4 *>(a.q + t * a.q_stride + (int64_t)(h0 + k) * D + ch * 8);
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
        return;
    }

    // ---- keys and values of one block of the cache ------------------------------------------
    const int32_t slot = (int32_t)(blockIdx.x / p.splits), part = (int32_t)(blockIdx.x - (int64_t)slot * p.splits);
    const int32_t bt = a.c.bt;
    int32_t lo = slot;
    if (p.per_seq == 2) {
        // last sequence whose slots start at or before this one, 32 at a time; every warp for itself
        lo = 0;
        for (int32_t n = a.b.S; n > 1;) {
            const int32_t step = (n + 31) / 32, at = lo + (tid & 31) * step;
            const bool le = at < lo + n && (int64_t)(a.b.indptr[at] / bt) + 2ll * at <= slot;
            const int k = 31 - __clz(__ballot_sync(~0u, le) | 1u);
            n = n - k * step < step ? n - k * step : step;
            lo += k * step;
        }
    }
    const int32_t s = lo, t0 = a.b.indptr[s], t1 = a.b.indptr[s + 1], len = a.b.kv_len[s];
    const int32_t n = t1 - t0;
    int32_t bad = 0;
    if (t0 < 0 || t1 < t0 || t1 > a.b.T || n > a.b.max_q)
        bad = SLORA_DEV_BAD_SEGMENT;
    else if (len < n || (int64_t)len > (int64_t)a.b.max_blocks * bt)
        bad = SLORA_DEV_BAD_LENGTH;
    if (bad) {
        if (tid == 0) set_status(a.c.status, bad);
        return;
    }
    if (n == 0) return;
    const int32_t p0 = len - n;                                   // position of the first new token
    const int64_t nth = p.per_seq == 2 ? slot - ((int64_t)(t0 / bt) + 2ll * s) : 0;    // nth touched block of the sequence
    if (nth < 0 || p0 / bt + nth > (len - 1) / bt) return;
    const int32_t blk = p0 / bt + (int32_t)nth;
    const int32_t from = blk * bt > p0 ? blk * bt : p0, to = (blk + 1) * bt < len ? (blk + 1) * bt : len;
    const int32_t held = from - blk * bt, nt = to - from;         // rows already there, new rows
    const int32_t row0 = t0 + from - p0;                          // first of the new tokens' rows
    const int32_t all = 2 * a.c.n_kv;
    const int32_t u0 = part * p.units, u1 = u0 + p.units < all ? u0 + p.units : all;
    // the CTA's pages and, for a block that holds tokens, their exponents
    if (tid < u1 - u0) {
        int32_t page = a.b.table[((int64_t)s * a.b.max_blocks + blk) * all + u0 + tid];
        if (page < 0 || page >= a.c.num_pages) {
            set_status(a.c.status, SLORA_DEV_BAD_PAGE);
            page = -1;
        }
        s_page[tid] = page;
        s_exp[tid] = (int8_t)(held && page >= 0 ? clamp_exponent(a.c.exps[page]) : 0);
    }

    if (nt <= kFew) {
        // one page per group and step; unit: KV head * 2 + (0 keys, 1 values)
        few_rows<D, FMT>(a, u0, u1, nt, held, row0, from, s_page, s_exp);
        return;
    }
    __syncthreads();

    int turn = 0;        // s_max alternates, so one barrier per page is enough
    for (int32_t u = u0; u < u1; ++u) {
        const int32_t head = u >> 1;
        const bool val = u & 1;
        const int32_t page = s_page[u - u0];
        if (page < 0) continue;             // the whole CTA
        const __half *src = (val ? a.v : a.k) + (int64_t)head * D + ch * 8;
        const int64_t stride = val ? a.v_stride : a.k_stride;
        const int old = s_exp[u - u0];
        uint4 raw[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = i * GROUPS + grp;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (r < nt) raw[i] = *reinterpret_cast<const uint4 *>(src + (int64_t)(row0 + r) * stride);
        }
        float x[PASSES][8];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (i * GROUPS >= nt) break;
            const int r = i * GROUPS + grp;
            unpack(raw[i], x[i]);
            if (!val) {
                Rot rt;
                rt.on = false;
                if (r < nt) load_rot(a, position(a, row0 + r, from + r), ch, rt);
                rotate<LPR>(a, rt, ch, x[i]);
            }
            m = fmaxf(m, size_of(x[i]));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        float *sm = s_max[turn ^= 1];
        if ((tid & 31) == 0) sm[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, sm[i]);
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

template <int D>
cudaError_t launch_d(const Params &p, int fmt, unsigned grid, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // rows of a block over the CTA's groups: the registers for 4, 5 or 8 of them per lane (a
    // page of up to 8192, 10240 or 16384 bytes)
    const int passes = (p.a.c.bt + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
    auto go = [&](auto e4m3, auto int8) {
        return cudaLaunchKernelEx(&cfg, fmt == SLORA_KV_E4M3 ? e4m3 : int8, p);
    };
    if (passes <= 4) return go(append_kernel<D, SLORA_KV_E4M3, 4>, append_kernel<D, SLORA_KV_INT8, 4>);
    if (passes <= 5) return go(append_kernel<D, SLORA_KV_E4M3, 5>, append_kernel<D, SLORA_KV_INT8, 5>);
    return go(append_kernel<D, SLORA_KV_E4M3, 8>, append_kernel<D, SLORA_KV_INT8, 8>);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int head_dim, int fmt, int num_sms, cudaStream_t stream, int *launches)
{
    Params p;
    p.a = a;
    const int groups = kThreads / (head_dim / 8);
    const int32_t all = 2 * a.c.n_kv;
    p.per_seq = a.b.max_q == 1 ? 1 : 2;
    p.slots = p.per_seq == 1 ? a.b.S : a.b.T / a.c.bt + 2 * a.b.S;
    // Pages of one slot over several CTAs where the batch has few slots; a CTA's groups need
    // a page each when the blocks gain a token or so each.
    const int64_t want = 8ll * num_sms;
    int64_t splits = (want + p.slots - 1) / p.slots;
    const int64_t most = a.b.max_q <= kFew ? (all + groups - 1) / groups : all;
    if (splits > most) splits = most;
    if (splits * kMaxUnits < all) splits = (all + kMaxUnits - 1) / kMaxUnits;
    p.units = (int32_t)((all + splits - 1) / splits);
    p.splits = (all + p.units - 1) / p.units;
    p.kv_ctas = (int64_t)p.slots * p.splits;
    int64_t q_ctas = 0;
    if (a.q) {
        const int64_t items = (int64_t)a.b.T * ((a.n_q + kQHeads - 1) / kQHeads);
        q_ctas = (items + groups - 1) / groups;
        if (q_ctas > 16ll * num_sms) q_ctas = 16ll * num_sms;
    }
    if (p.kv_ctas + q_ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)(p.kv_ctas + q_ctas);
    cudaError_t e = head_dim == 128 ? launch_d<128>(p, fmt, grid, stream) : launch_d<64>(p, fmt, grid, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace kv
}  // namespace slora
