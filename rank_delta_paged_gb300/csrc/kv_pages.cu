// Pages of the 8-bit KV cache moved about: copies of pages, and the compaction of sequences to their kept tokens.
//
// What bounds a copy: its rows are read and written once.
#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"

namespace slora {
namespace kv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 8;       // per SM

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int32_t s = a.src[i], d = a.dst[i], rows = a.rows ? a.rows[i] : a.c.bt;
        if (s < 0 || s >= a.c.num_pages || d < 0 || d >= a.c.num_pages || rows < 0 || rows > a.c.bt) {
            if (tid == 0)
                set_status(a.c.status, rows < 0 || rows > a.c.bt ? SLORA_DEV_BAD_LENGTH : SLORA_DEV_BAD_PAGE);
            continue;
        }
        if (s == d || rows == 0) continue;
        const uint4 *from = reinterpret_cast<const uint4 *>(a.c.pool + s * a.c.page_bytes);
        uint4 *to = reinterpret_cast<uint4 *>(a.c.pool + d * a.c.page_bytes);
        const int32_t chunks = rows * a.row_bytes / 16;
#pragma unroll 1
        for (int32_t k = tid; k < chunks; k += 4 * kCopyThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j * kCopyThreads < chunks) v[j] = from[k + j * kCopyThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j * kCopyThreads < chunks) to[k + j * kCopyThreads] = v[j];
        }
        if (tid == 0) a.c.exps[d] = a.c.exps[s];
    }
}

// ---- compaction -------------------------------------------------------------------------
// A block's rows come from pages with scales of their own:
//     e = the smallest exponent that max |code 2^e_row| fits        code <- round(code 2^(e_row - e))
// What bounds it: the kept rows are read and written once; for few of them the chain of dependent reads (offsets,
// kept positions, pages, exponents, rows).
constexpr int kCompactThreads = 128;
constexpr int kMaxBlock = 256;     // rows of the largest page
constexpr int kCompactCtas = 12;   // per SM

// The largest finite magnitude of 16 codes, as a code without its sign.
template <int FMT>
__device__ __forceinline__ uint32_t top_code(uint4 v)
{
    auto one = [](uint32_t w) {
        if (FMT == SLORA_KV_INT8) return __vabsss4(w);
        w &= 0x7F7F7F7Fu;
        return w & ~__vcmpeq4(w, 0x7F7F7F7Fu);
    };
    uint32_t m = __vmaxu4(__vmaxu4(one(v.x), one(v.y)), __vmaxu4(one(v.z), one(v.w)));
    m = __vmaxu4(m, m >> 16);
    return __vmaxu4(m, m >> 8) & 0xFFu;
}

// Four codes times a power of two.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float unit)
{
    uint32_t lo, hi;
    decode4<FMT>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    return encode2<FMT>(a.x * unit, a.y * unit) | encode2<FMT>(b.x * unit, b.y * unit) << 16;
}

struct Span {
    int32_t t0, n, first, len;   // entries of the list, how many, where they go, the sequence's length
};

// Sequence s; 0, or the status of one that cannot be used.
__device__ __forceinline__ int32_t load_span(const CompactArgs &a, int32_t s, Span &q)
{
    const int32_t t0 = a.indptr[s], t1 = a.indptr[s + 1];
    q.t0 = t0;
    q.n = t1 - t0;
    q.len = a.kv_len[s];
    q.first = a.first ? a.first[s] : 0;
    if (t0 < 0 || t1 < t0 || t1 > a.n_kept || q.n > a.max_kept) return SLORA_DEV_BAD_SEGMENT;
    if (q.len < 0 || q.len > 1 << 30 || (int64_t)q.len > (int64_t)a.max_blocks * a.c.bt || q.first < 0 || q.first > q.len ||
        q.n > q.len - q.first)
        return SLORA_DEV_BAD_LENGTH;
    return 0;
}

// PASSES: 16-byte pieces of a page per thread.
template <int D, int FMT, int PASSES>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactArgs a, int32_t nb, int64_t items)
{
    constexpr int LPR = D / 16;
    __shared__ int64_t s_from[kMaxBlock];
    __shared__ int8_t s_exp[kMaxBlock];
    __shared__ uint32_t s_max[kCompactThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int32_t units = 2 * a.c.n_kv, bt = a.c.bt;
    const bool in_place = a.dst_table == nullptr;
#pragma unroll 1
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        // (sequence, block, page of the block), or in place (sequence, page of its blocks)
        const int64_t at = it / units;
        const int32_t u = (int32_t)(it - at * units), s = (int32_t)(in_place ? at : at / nb);
        const int32_t b = in_place ? 0 : (int32_t)(at - (int64_t)s * nb);
        Span q;
        const int32_t bad = load_span(a, s, q);
        if (bad) {
            if (tid == 0 && u == 0 && b == 0) set_status(a.c.status, bad);
            continue;
        }
        if (tid == 0 && u == 0 && b == 0 && a.new_len) a.new_len[s] = q.first + q.n;
        if (q.n == 0) continue;
        const int32_t *kept = a.kept + (u >> 1) * a.head_stride + q.t0;
        const int32_t *table = a.table + (int64_t)s * a.max_blocks * units + u;
        const int32_t *dst_table = in_place ? table : a.dst_table + (int64_t)s * a.dst_blocks * units + u;
        const int32_t end = q.first + q.n, last = (end - 1) / bt;
        const int32_t b0 = q.first / bt + b, b1 = in_place ? last : (b0 < last ? b0 : last);
#pragma unroll 1
        for (int32_t blk = b0; blk <= b1; ++blk) {
            const int32_t to0 = blk * bt, rows = end - to0 < bt ? end - to0 : bt;
            int32_t wrong = 0;
#pragma unroll 1
            for (int32_t r = tid; r < rows; r += kCompactThreads) {
                const int32_t to = to0 + r, i = to - q.first;
                int32_t p = to;
                if (i >= 0) {
                    p = kept[i];
                    if (p < to || p >= q.len || (i > 0 && kept[i - 1] >= p)) {
                        wrong = SLORA_DEV_BAD_POSITION;
                        continue;
                    }
                }
                const int32_t sb = p / bt, page = table[(int64_t)sb * units];
                if (page < 0 || page >= a.c.num_pages) {
                    wrong = SLORA_DEV_BAD_PAGE;
                    continue;
                }
                s_from[r] = page * a.c.page_bytes + (p - sb * bt) * D;
                s_exp[r] = (int8_t)clamp_exponent(a.c.exps[page]);
            }
            int32_t dst = -1;
            if (blk >= a.dst_blocks) {
                wrong = SLORA_DEV_BAD_LENGTH;
            } else {
                dst = dst_table[(int64_t)blk * units];
                if (dst < 0 || dst >= a.c.num_pages) wrong = SLORA_DEV_BAD_PAGE;
            }
            if (wrong) set_status(a.c.status, wrong);
            if (__syncthreads_or(wrong)) continue;      // (nothing of shared memory has been read)
            uint4 v[PASSES];
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                const int32_t x = k * kCompactThreads + tid, r = x / LPR;
                v[k] = make_uint4(0, 0, 0, 0);
                if (r < rows) v[k] = *reinterpret_cast<const uint4 *>(a.c.pool + s_from[r] + x % LPR * 16);
            }
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                const int32_t r = (k * kCompactThreads + tid) / LPR;
                if (r >= rows) continue;
                uint32_t lo, hi;
                decode4<FMT>(top_code<FMT>(v[k]), lo, hi);
                m = fmaxf(m, __low2float(*reinterpret_cast<__half2 *>(&lo)) * pow2(s_exp[r]));
            }
            const uint32_t w = __reduce_max_sync(~0u, __float_as_uint(m));
            if ((tid & 31) == 0) s_max[tid >> 5] = w;
            __syncthreads();
            uint32_t top = s_max[0];
#pragma unroll
            for (int k = 1; k < kCompactThreads / 32; ++k) top = top > s_max[k] ? top : s_max[k];
            const int e = fit_exponent<FMT>(__uint_as_float(top));
            uint8_t *page = a.c.pool + dst * a.c.page_bytes;
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                const int32_t x = k * kCompactThreads + tid, r = x / LPR;
                if (r >= rows) continue;
                const int shift = s_exp[r] - e;
                if (shift != 0) {
                    const float unit = pow2(shift);
                    v[k] = make_uint4(rescale4<FMT>(v[k].x, unit), rescale4<FMT>(v[k].y, unit), rescale4<FMT>(v[k].z, unit),
                                      rescale4<FMT>(v[k].w, unit));
                }
                *reinterpret_cast<uint4 *>(page + x * 16) = v[k];
            }
            if (tid == 0) a.c.exps[dst] = (int8_t)e;
            __syncthreads();
        }
    }
}

template <int D, int FMT>
cudaError_t launch_compact_d(const CompactArgs &a, int num_sms, cudaStream_t stream)
{
    // the blocks that a sequence's kept tokens touch, at most
    const int32_t nb = a.dst_table ? (a.max_kept + a.c.bt - 1) / a.c.bt + 1 : 1;
    const int64_t items = (int64_t)a.S * nb * 2 * a.c.n_kv, ctas = (int64_t)num_sms * kCompactCtas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items < ctas ? items : ctas));
    cfg.blockDim = dim3(kCompactThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // pages of up to 8192 and up to 16384 bytes
    return a.c.bt * D <= 4 * 16 * kCompactThreads ? cudaLaunchKernelEx(&cfg, compact_kernel<D, FMT, 4>, a, nb, items)
                                                  : cudaLaunchKernelEx(&cfg, compact_kernel<D, FMT, 8>, a, nb, items);
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, int head_dim, int fmt, int num_sms, cudaStream_t stream, int *launches)
{
    cudaError_t e;
    if (head_dim == 128)
        e = fmt == SLORA_KV_E4M3 ? launch_compact_d<128, SLORA_KV_E4M3>(a, num_sms, stream)
                                 : launch_compact_d<128, SLORA_KV_INT8>(a, num_sms, stream);
    else
        e = fmt == SLORA_KV_E4M3 ? launch_compact_d<64, SLORA_KV_E4M3>(a, num_sms, stream)
                                 : launch_compact_d<64, SLORA_KV_INT8>(a, num_sms, stream);
    *launches += e == cudaSuccess;
    return e;
}

cudaError_t launch_copy(const CopyArgs &a, int num_sms, cudaStream_t stream, int *launches)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t ctas = (int64_t)num_sms * kCopyCtas;
    cfg.gridDim = dim3((unsigned)(a.n < ctas ? a.n : ctas));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_kernel, a);
    *launches += e == cudaSuccess;
    return e;
}

}  // namespace kv
}  // namespace slora
