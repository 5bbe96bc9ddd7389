// Pages of the 8-bit KV cache moved about: copies of pages, and the compaction of sequences to their kept tokens.
//
// What bounds a copy: its rows are read and written once.  A CTA takes a page at a time, 16 bytes a lane and up to
// four pieces a lane under way, with the next page's entries read meanwhile.
// Measured: 30011 pages of 10 KB 98 us, 6.3 TB/s, 93 % of a plain copy's rate (106 without the reads ahead; by 512 threads and 4
// CTAs per SM 125, by 128 and 16 98); 16 pages 1.8 us on the GPU.
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
    int32_t i = (int32_t)blockIdx.x;
    auto rows_of = [&](int32_t k) { return a.rows ? __ldg(a.rows + k) : a.c.bt; };
    int32_t s = __ldg(a.src + i), d = __ldg(a.dst + i), rows = rows_of(i);
#pragma unroll 1
    for (;;) {
        // the next page's entries, while this one's rows are on their way
        const int32_t next = a.n - i > (int32_t)gridDim.x ? i + (int32_t)gridDim.x : -1;
        int32_t ns = 0, nd = 0, nrows = 0;
        if (next >= 0) ns = __ldg(a.src + next), nd = __ldg(a.dst + next), nrows = rows_of(next);
        if (s < 0 || s >= a.c.num_pages || d < 0 || d >= a.c.num_pages || rows < 0 || rows > a.c.bt) {
            if (tid == 0)
                set_status(a.c.status, rows < 0 || rows > a.c.bt ? SLORA_DEV_BAD_LENGTH : SLORA_DEV_BAD_PAGE);
        } else if (s != d && rows > 0) {
            const uint4 *from = reinterpret_cast<const uint4 *>(a.c.pool + s * a.c.page_bytes);
            uint4 *to = reinterpret_cast<uint4 *>(a.c.pool + d * a.c.page_bytes);
            const int32_t chunks = rows * a.row_bytes / 16;
            const int8_t e = tid == 0 ? a.c.exps[s] : 0;
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
            if (tid == 0) a.c.exps[d] = e;
        }
        if (next < 0) return;
        i = next, s = ns, d = nd, rows = nrows;
    }
}

// ---- compaction -------------------------------------------------------------------------
// A block's rows come from pages with scales of their own:
//     e = the smallest exponent that max |code 2^e_row| fits        code <- round(code 2^(e_row - e))
// What bounds it: the kept rows are read and written once; for few of them the chain of dependent reads (offsets,
// kept positions, pages, exponents, rows).
// Measured: 30 thousand kept tokens of six sequences, 8 heads, into pages of their own 29 us, 4.3 TB/s of rows of 128 bytes;
// 29 thousand of a choice for each head, rows of 64 bytes, 24 us (2.6 TB/s; memory moves 1.7 times as much for such rows);
// 24 drafted branches in place 5 us on the GPU.  At 68 % issue the instructions are the bound, some 180 per lane and 16
// bytes.  With the rows in registers instead of shared memory 36 us (the decoded codes of the maximum were kept, and
// spilled), with codes rescaled in fp32 51; the maximum over the codes as integers 30.
constexpr int kMaxCluster = 8;
constexpr int kFill = 1280;      // threads per SM that the registers are to allow (1024 and 1536: within 3 %)
constexpr int64_t kCompactCtas = 1 << 20;     // of a grid, at most: the hardware deals them out as SMs become free

// The largest finite magnitude of 16 codes.
template <int FMT>
__device__ __forceinline__ float top_code(uint4 v)
{
    __half2 m = __float2half2_rn(0.f);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        decode4<FMT>(w[i], lo, hi);
        m = __hmax2(m, __habs2(*reinterpret_cast<__half2 *>(&lo)));     // passes over NaN
        m = __hmax2(m, __habs2(*reinterpret_cast<__half2 *>(&hi)));
    }
    return fmaxf(__low2float(m), __high2float(m));
}

// Four codes times a power of two, -infinity < shift <= 15, rounded to nearest even.  fp16 loses nothing that counts: an
// E4M3 product of 2^-11 or more has its last bit at 2^-14 or above, a smaller one is 0 as a code; an INT8
// product and 1536, whose sum has its last bit at 1, are rounded together, and its low byte is the code.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, __half2 unit)
{
    uint32_t lo, hi;
    decode4<FMT>(w, lo, hi);
    const __half2 a = *reinterpret_cast<__half2 *>(&lo), b = *reinterpret_cast<__half2 *>(&hi);
    if (FMT == SLORA_KV_E4M3) {
        const __half2 x = __hmul2(a, unit), y = __hmul2(b, unit);
        uint32_t r;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "r"(*reinterpret_cast<const uint32_t *>(&x)), "r"(*reinterpret_cast<const uint32_t *>(&y)));
        return r;
    }
    const __half2 off = __float2half2_rn(1536.f);
    const __half2 x = __hfma2(a, unit, off), y = __hfma2(b, unit, off);
    return __byte_perm(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y), 0x6420);
}
template <int FMT>
__device__ __forceinline__ uint4 rescale16(uint4 v, int shift)
{
    const __half2 unit = __float2half2_rn(pow2(shift < 15 ? shift : 15));
    return make_uint4(rescale4<FMT>(v.x, unit), rescale4<FMT>(v.y, unit), rescale4<FMT>(v.z, unit), rescale4<FMT>(v.w, unit));
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

// A CTA takes one block of one head, keys and values: two pages, each by half of its threads, with its rows in shared
// memory between the reads and the writes, where a thread finds what it has copied itself.  PT threads per page: 64,
// or 128 for pages above 8192 bytes.
// A page that cannot be used, as a source or to write to, keeps its half from writing, not the other: as everywhere
// in the cache, work is skipped by the page.
// In place a cluster of CTAs goes through a sequence's blocks from the first, a block each at a time: a block takes rows
// from itself and later ones only, so what a round writes no later one reads, and within a round all have read
// before one writes.  Where the next round's rows come from is looked up under this one's reads.
template <int D, int FMT, int PT>
__global__ void __launch_bounds__(2 * PT, kFill / (2 * PT)) compact_kernel(const __grid_constant__ CompactArgs a, int32_t nb, int64_t items)
{
    constexpr int LPR = D / 16, kRows = 8 * PT / LPR;
    constexpr uint32_t kBad = ~0u;
    __shared__ uint4 s_code[2][kRows * LPR];
    __shared__ int32_t s_page[2][2][kRows], s_row[2][kRows];
    __shared__ float s_unit[2][kRows];              // 2^exponent of the rows' pages
    __shared__ uint32_t s_max[2 * PT / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, w = tid / PT, pt = tid % PT;
    const int32_t n_kv = a.c.n_kv, bt = a.c.bt;
    const bool in_place = a.dst_table == nullptr;
    const int32_t ctas = (int32_t)cluster_nctarank();    // more than one in place only, and then one item per cluster
    uint4 *codes = s_code[w];
#pragma unroll 1
    for (int64_t it = blockIdx.x / (unsigned)ctas; it < items; it += gridDim.x) {
        // (sequence, block, head), or in place (sequence, head)
        const int64_t at = it / n_kv;
        const int32_t h = (int32_t)(it - at * n_kv), s = (int32_t)(in_place ? at : at / nb);
        const int32_t b = in_place ? (int32_t)(blockIdx.x % (unsigned)ctas) : (int32_t)(at - (int64_t)s * nb);
        Span q;
        const int32_t unfit = load_span(a, s, q);
        const bool tells = tid == 0 && h == 0 && b == 0;
        if (unfit) {
            if (tells) set_status(a.c.status, unfit);
            continue;
        }
        if (tells && a.new_len) a.new_len[s] = q.first + q.n;
        if (q.n == 0) continue;
        const int32_t *kept = a.kept + h * a.head_stride + q.t0;
        const int32_t *table = a.table + ((int64_t)s * a.max_blocks * n_kv + h) * 2 + w;
        const int32_t *dst_table = in_place ? table : a.dst_table + ((int64_t)s * a.dst_blocks * n_kv + h) * 2 + w;
        const int32_t end = q.first + q.n, last = (end - 1) / bt;
        const int32_t b0 = q.first / bt + b, b1 = in_place || b0 > last ? last : b0;
        // the pages and rows of a block's kept tokens; false if this thread found one that cannot be used
        auto look_up = [&](int32_t blk, int buf) {
            const int32_t to0 = blk * bt, rows = end - to0 < bt ? end - to0 : bt;
            bool good = true;
#pragma unroll 1
            for (int32_t r = pt; r < rows; r += PT) {
                const int32_t to = to0 + r, i = to - q.first;
                int32_t p = to, page = -1;
                bool fine = true;
                if (i >= 0) {
                    p = __ldg(kept + i);
                    fine = p >= to && p < q.len && (i == 0 || __ldg(kept + i - 1) < p);
                    if (!fine) set_status(a.c.status, SLORA_DEV_BAD_POSITION);
                }
                if (fine) {
                    const int32_t sb = p / bt;
                    page = __ldg(table + (int64_t)sb * n_kv * 2);
                    if (page < 0 || page >= a.c.num_pages) {
                        set_status(a.c.status, SLORA_DEV_BAD_PAGE);
                        page = -1;
                    }
                    s_row[buf][r] = p - sb * bt;    // (the same by either half)
                }
                s_page[buf][w][r] = page;
                good &= page >= 0;
            }
            return good;
        };
        auto to_page = [&](int32_t blk) { return blk < a.dst_blocks ? __ldg(dst_table + (int64_t)blk * n_kv * 2) : -1; };
        int buf = 0;
        bool next_good = b0 > b1 || look_up(b0, 0);
        int32_t next_dst = b0 > b1 ? 0 : to_page(b0);
        // (a cluster's CTAs go through as many rounds as its first one)
#pragma unroll 1
        for (int32_t blk = b0; blk - b <= b1 - (in_place ? 0 : b); blk += ctas, buf ^= 1) {
            const int32_t rows = blk > b1 ? 0 : end - blk * bt < bt ? end - blk * bt : bt;
            bool bad = !next_good;
            const int32_t dst = next_dst;
            __syncthreads();
            const int32_t pieces = rows * LPR;
#pragma unroll 4
            for (int32_t x = pt; x < pieces; x += PT) {
                const int32_t r = x / LPR, page = s_page[buf][w][r];
                if (page >= 0)
                    cp_async16(&codes[x], a.c.pool + page * a.c.page_bytes + (s_row[buf][r] * D + x % LPR * 16), 16);
            }
            cp_async_commit();
            // the exponents, while the rows are on their way
#pragma unroll 1
            for (int32_t r = pt; r < rows; r += PT) {
                const int32_t page = s_page[buf][w][r];
                s_unit[w][r] = page >= 0 ? pow2(clamp_exponent(a.c.exps[page])) : 0.f;
            }
            if (dst < 0 || dst >= a.c.num_pages) {
                if (pt == 0) set_status(a.c.status, blk < a.dst_blocks ? SLORA_DEV_BAD_PAGE : SLORA_DEV_BAD_LENGTH);
                bad = true;
            }
            if (b1 - blk >= ctas) {
                next_good = look_up(blk + ctas, buf ^ 1);
                next_dst = to_page(blk + ctas);
            }
            cp_async_wait<0>();
            if (ctas > 1) {
                __syncwarp();
                cluster_sync_all();
            } else {
                __syncthreads();
            }
            if (rows == 0) break;                   // the cluster's last round
            float m = 0.f;
#pragma unroll 2
            for (int32_t x = pt; x < pieces; x += PT)
                if (s_page[buf][w][x / LPR] >= 0) m = fmaxf(m, top_code<FMT>(codes[x]) * s_unit[w][x / LPR]);
            const uint32_t mine = __reduce_max_sync(~0u, bad ? kBad : __float_as_uint(m));
            if ((tid & 31) == 0) s_max[tid >> 5] = mine;
            __syncthreads();
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < PT / 32; ++k) {
                const uint32_t y = s_max[w * (PT / 32) + k];
                top = top > y ? top : y;
            }
            if (top != kBad) {
                // (no higher than is read: a -128 of the caller's stays as it is there)
                const int e = min(fit_exponent<FMT>(__uint_as_float(top)), kExpLimit);
                uint4 *page = reinterpret_cast<uint4 *>(a.c.pool + dst * a.c.page_bytes);
#pragma unroll 2
                for (int32_t x = pt; x < pieces; x += PT) {
                    const int shift = (int)(__float_as_uint(s_unit[w][x / LPR]) >> 23) - 127 - e;
                    uint4 v = codes[x];
                    if (shift != 0) v = rescale16<FMT>(v, shift);
                    if (FMT == SLORA_KV_E4M3 && shift > 15) v = rescale16<FMT>(v, shift - 15);
                    page[x] = v;
                }
                if (pt == 0) a.c.exps[dst] = (int8_t)e;
            }
        }
        if (it + gridDim.x < items) __syncthreads();
    }
}

template <int D, int FMT>
cudaError_t launch_compact_d(const CompactArgs &a, int num_sms, cudaStream_t stream)
{
    const int pt = a.c.bt * D <= 8192 ? 64 : 128;
    // the blocks that a sequence's kept tokens touch, at most
    const int32_t nb = a.dst_table ? (a.max_kept + a.c.bt - 1) / a.c.bt + 1 : 1;
    const int64_t items = (int64_t)a.S * nb * a.c.n_kv;
    // In place, the most CTAs per cluster that find blocks and room.  By 1, 2, 4 and 8, in us:
    // a sequence of 8 heads that keeps 8000 tokens 364, 223, 115, 60 (10 into pages of their own); 8 sequences that
    // keep 2000 to 8000 each 370, 216, 119, 72 (36); 64 that keep 500 40, 34, 34, 34 (31).
    int cluster = 1;
    if (!a.dst_table)
        while (cluster < kMaxCluster && cluster * 2 <= (a.max_kept + a.c.bt - 1) / a.c.bt && items * cluster * 2 <= 8ll * num_sms) cluster *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items < kCompactCtas ? items : kCompactCtas) * cluster);
    cfg.blockDim = dim3(2 * pt);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return pt == 64 ? cudaLaunchKernelEx(&cfg, compact_kernel<D, FMT, 64>, a, nb, items)
                    : cudaLaunchKernelEx(&cfg, compact_kernel<D, FMT, 128>, a, nb, items);
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
