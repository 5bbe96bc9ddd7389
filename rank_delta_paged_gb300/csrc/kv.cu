// Host side of the 8-bit paged KV cache: the cache's handle, the checks of arguments and the
// choice of kernels.
#include <atomic>
#include <cmath>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "slora.h"

using namespace slora;

struct slora_kv {
    int device = 0;
    int num_sms = 0;
    int head_dim = 0;
    int format = 0;
    kv::Cache c = {};
    int64_t *launches = nullptr;
    uint8_t *ws = nullptr;     // the attention's partial results and counters (the pool's)
    kv::PageMaps maps;
};

namespace {

// Rows per KV head (new tokens x query heads of the group) up to which a sequence is the streaming
// kernel's, 16 rows at a time; the rest is the tensor cores' kernel's, 256 at a time.  Sequences of 500
// to 8000 tokens, 8 KV heads, streaming and the other in us:
//     rows    4 sequences    24 sequences    96 sequences
//      16      50     65      91     132      224     379
//      32      54     65     138     136      420     389
//      64      69     66     245     140      809     398
constexpr int32_t kSmallRows = 32;

std::atomic<int32_t> g_give_up{-1};     // slora_debug_kv_give_up

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Boxes of whole rows, swizzled by the row's length.
bool encode_maps(slora_kv *k)
{
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return false;
    const cuuint64_t d = (cuuint64_t)k->head_dim, pb = (cuuint64_t)k->c.page_bytes;
    const cuuint64_t dims[3] = {d, pb / d, (cuuint64_t)k->c.num_pages};
    const cuuint64_t strides[2] = {d, pb};
    const cuuint32_t es[3] = {1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        const cuuint32_t box[3] = {(cuuint32_t)d, (k->c.bt % 16 == 0 ? 16u : 8u) << i, 1};
        if (reinterpret_cast<EncodeTiledFn>(fn)(&k->maps.m[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, k->c.pool, dims, strides,
                                                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                                d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

// The checks that append and attend share.
slora_status check_batch(const char *fn, slora_kv_t k, const slora_kv_batch *b, kv::Batch *out)
{
    if (!k || !b)
        return fail(SLORA_ERR_INVALID_ARG, "%s: null cache or batch", fn);
    if (b->n_tokens < 0 || b->n_tokens > (1 << 20) || b->n_seqs < 0 || b->n_seqs > (1 << 20) || b->max_q < 1 ||
        b->max_blocks < 1)
        return fail(SLORA_ERR_INVALID_ARG, "%s: n_tokens=%d n_seqs=%d max_q=%d max_blocks=%d", fn, b->n_tokens,
                    b->n_seqs, b->max_q, b->max_blocks);
    if (b->n_tokens > 0 && b->n_seqs > 0 && (!b->tok_indptr || !b->kv_len || !b->block_table))
        return fail(SLORA_ERR_INVALID_ARG, "%s: null tok_indptr, kv_len or block_table", fn);
    if (!aligned4(b->tok_indptr) || !aligned4(b->kv_len) || !aligned4(b->block_table))
        return fail(SLORA_ERR_INVALID_ARG, "%s: misaligned tok_indptr, kv_len or block_table", fn);
    *out = kv::Batch{b->n_tokens, b->n_seqs, b->max_q < b->n_tokens ? b->max_q : b->n_tokens, b->max_blocks,
                     b->tok_indptr, b->kv_len, b->block_table};
    return SLORA_OK;
}

// `none`: the call has no rows, and the pointer (that of an empty tensor is null) is not looked at.
slora_status check_rows(const char *fn, const char *what, const void *p, int64_t stride, int64_t row, bool none)
{
    if ((!none && (!p || !aligned16(p))) || stride % 8 != 0 || stride < row)
        return fail(SLORA_ERR_INVALID_ARG, "%s: %s is null or misaligned, or its stride %lld is below %lld or no multiple of 8",
                    fn, what, (long long)stride, (long long)row);
    return SLORA_OK;
}

}  // namespace

extern "C" slora_status slora_kv_create(slora_pool_t pool, int32_t n_kv_heads, int32_t head_dim, int32_t format,
                                        slora_kv_t *out)
{
    if (!out)
        return fail(SLORA_ERR_INVALID_ARG, "kv_create: null out");
    *out = nullptr;
    PoolHotPath hp;
    slora_status st = pool_hot_path(pool, &hp);
    if (st != SLORA_OK)
        return st;
    if (n_kv_heads < 1 || n_kv_heads > 1024 || (format != SLORA_KV_E4M3 && format != SLORA_KV_INT8))
        return fail(SLORA_ERR_INVALID_ARG, "kv_create: n_kv_heads=%d format=%d", n_kv_heads, format);
    if (head_dim != 64 && head_dim != 128)
        return fail(SLORA_ERR_UNSUPPORTED, "kv_create: head_dim=%d (64 or 128)", head_dim);
    const int64_t page_bytes = (int64_t)hp.pv.hidden * 2;
    const int32_t bt = (int32_t)(page_bytes / head_dim / 8 * 8);
    if (bt < 8)
        return fail(SLORA_ERR_UNSUPPORTED, "kv_create: a page of %lld bytes holds no 8 rows of %d",
                    (long long)page_bytes, head_dim);
    DeviceScope dev_scope(hp.device);
    cudaError_t e = dev_scope.error();
    if (e != cudaSuccess)
        return fail(SLORA_ERR_CUDA, "kv_create: cudaSetDevice: %s", cudaGetErrorString(e));
    slora_kv *k = new (std::nothrow) slora_kv();
    if (!k)
        return fail(SLORA_ERR_HOST_ALLOC, "kv_create");
    k->device = hp.device;
    k->num_sms = hp.num_sms > 0 ? hp.num_sms : 1;
    k->head_dim = head_dim;
    k->format = format;
    k->launches = hp.launches;
    k->c.pool = reinterpret_cast<uint8_t *>(const_cast<uint16_t *>(hp.pv.pool));
    k->c.num_pages = hp.pv.num_pages;
    k->c.page_bytes = page_bytes;
    k->c.n_kv = n_kv_heads;
    k->c.bt = bt;
    k->c.status = hp.pv.status;
    void *ws = nullptr;
    st = pool_kv_scratch(pool, kv::decode_workspace_bytes(k->num_sms) + kv::prefill_workspace_bytes(k->num_sms), &ws);
    if (st != SLORA_OK) {
        delete k;
        return st;
    }
    k->ws = static_cast<uint8_t *>(ws);
    if ((e = cudaMalloc(&k->c.exps, (size_t)hp.pv.num_pages)) == cudaSuccess &&
        (e = cudaMemset(k->c.exps, 0, (size_t)hp.pv.num_pages)) == cudaSuccess)
        e = cudaDeviceSynchronize();
    st = e == cudaSuccess ? SLORA_OK : fail(SLORA_ERR_CUDA, "kv_create: %s", cudaGetErrorString(e));
    if (st == SLORA_OK && !encode_maps(k))
        st = fail(SLORA_ERR_CUDA, "kv_create: no tensor map of the pool");
    if (st != SLORA_OK) {
        cudaFree(k->c.exps);
        delete k;
        return st;
    }
    *out = k;
    return SLORA_OK;
}

extern "C" slora_status slora_kv_destroy(slora_kv_t k)
{
    if (!k)
        return SLORA_OK;
    DeviceScope dev_scope(k->device);
    cudaDeviceSynchronize();
    cudaFree(k->c.exps);
    delete k;
    return SLORA_OK;
}

extern "C" slora_status slora_kv_block_tokens(slora_kv_t k, int32_t *out)
{
    if (!k || !out)
        return fail(SLORA_ERR_INVALID_ARG, "kv_block_tokens: null");
    *out = k->c.bt;
    return SLORA_OK;
}

extern "C" slora_status slora_kv_exponents(slora_kv_t k, int8_t **out)
{
    if (!k || !out)
        return fail(SLORA_ERR_INVALID_ARG, "kv_exponents: null");
    *out = k->c.exps;
    return SLORA_OK;
}

namespace {

// Append, with the norm of keys and queries if there is one.
slora_status append(const char *fn, slora_kv_t k, const slora_kv_batch *batch, const void *kk, int64_t k_stride,
                    const void *v, int64_t v_stride, const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                    int32_t n_q_heads, const slora_kv_norm *norm, const slora_kv_rope *rope, slora_stream_t stream)
{
    kv::AppendArgs a = {};
    slora_status st = check_batch(fn, k, batch, &a.b);
    if (st != SLORA_OK)
        return st;
    const bool none = a.b.T == 0 || a.b.S == 0;
    const int64_t row = (int64_t)k->c.n_kv * k->head_dim;
    if ((st = check_rows(fn, "k", kk, k_stride, row, none)) != SLORA_OK ||
        (st = check_rows(fn, "v", v, v_stride, row, none)) != SLORA_OK)
        return st;
    if ((!none && (q == nullptr) != (q_out == nullptr)) || (q && !rope && !norm))
        return fail(SLORA_ERR_INVALID_ARG, "%s: q needs q_out, and rope or a norm", fn);
    if (q) {
        if (n_q_heads < 1 || n_q_heads > 8192)
            return fail(SLORA_ERR_INVALID_ARG, "%s: n_q_heads=%d", fn, n_q_heads);
        const int64_t qrow = (int64_t)n_q_heads * k->head_dim;
        if ((st = check_rows(fn, "q", q, q_stride, qrow, none)) != SLORA_OK ||
            (st = check_rows(fn, "q_out", q_out, q_out_stride, qrow, none)) != SLORA_OK)
            return st;
        a.q = static_cast<const __half *>(q);
        a.q_out = static_cast<__half *>(q_out);
        a.q_stride = q_stride;
        a.q_out_stride = q_out_stride;
        a.n_q = n_q_heads;
    }
    if (rope) {
        if (rope->rot_dim < 16 || rope->rot_dim > k->head_dim || rope->rot_dim % 16 != 0 ||
            (rope->interleaved != 0 && rope->interleaved != 1) || rope->n_positions < 1 || !rope->cos || !rope->sin ||
            !aligned16(rope->cos) || !aligned16(rope->sin) || !aligned4(rope->positions))
            return fail(SLORA_ERR_INVALID_ARG, "%s: rope with rot_dim=%d interleaved=%d n_positions=%d, or its tables", fn,
                        rope->rot_dim, rope->interleaved, rope->n_positions);
        a.rot = rope->rot_dim;
        a.interleaved = rope->interleaved;
        a.n_pos = rope->n_positions;
        a.cos = rope->cos;
        a.sin = rope->sin;
        a.positions = rope->positions;
    }
    if (norm) {
        auto weight = [&](const float *w, int64_t stride) {
            return aligned16(w) && (stride == 0 || (stride >= k->head_dim && stride % 4 == 0));
        };
        if ((norm->centered != 0 && norm->centered != 1) || !(norm->eps >= 0.f) || !std::isfinite(norm->eps) ||
            !weight(norm->q_weight, norm->q_weight_stride) || !weight(norm->k_weight, norm->k_weight_stride))
            return fail(SLORA_ERR_INVALID_ARG, "%s: norm with centered=%d eps=%g, or its weights", fn, norm->centered,
                        (double)norm->eps);
        a.q_weight = norm->q_weight;
        a.k_weight = norm->k_weight;
        a.q_weight_stride = norm->q_weight_stride;
        a.k_weight_stride = norm->k_weight_stride;
        a.eps = norm->eps;
        a.centered = norm->centered;
    }
    if (none)
        return SLORA_OK;
    a.c = k->c;
    a.k = static_cast<const __half *>(kk);
    a.v = static_cast<const __half *>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    DeviceScope dev_scope(k->device);
    cudaError_t e = dev_scope.error();
    int launches = 0;
    if (e == cudaSuccess)
        e = kv::launch_append(a, norm != nullptr, k->head_dim, k->format, k->num_sms, (cudaStream_t)stream, &launches);
    *k->launches += launches;
    return e == cudaSuccess ? SLORA_OK : fail(SLORA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

}  // namespace

extern "C" slora_status slora_kv_append(slora_kv_t k, const slora_kv_batch *batch, const void *kk, int64_t k_stride,
                                        const void *v, int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                        int64_t q_out_stride, int32_t n_q_heads, const slora_kv_rope *rope,
                                        slora_stream_t stream)
{
    return append("kv_append", k, batch, kk, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride, n_q_heads, nullptr,
                  rope, stream);
}

extern "C" slora_status slora_kv_append_norm(slora_kv_t k, const slora_kv_batch *batch, const void *kk, int64_t k_stride,
                                             const void *v, int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                             int64_t q_out_stride, int32_t n_q_heads, const slora_kv_norm *norm,
                                             const slora_kv_rope *rope, slora_stream_t stream)
{
    const char *fn = "kv_append_norm";
    if (!norm)
        return fail(SLORA_ERR_INVALID_ARG, "%s: null norm", fn);
    return append(fn, k, batch, kk, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride, n_q_heads, norm, rope, stream);
}

namespace {

slora_status attend(const char *fn, slora_kv_t k, const slora_kv_batch *batch, const void *q, int64_t q_stride,
                    int32_t n_q_heads, void *out, int64_t out_stride, float *lse, float softmax_scale, int32_t causal,
                    int32_t window, int32_t sinks, slora_stream_t stream)
{
    kv::AttendArgs a = {};
    slora_status st = check_batch(fn, k, batch, &a.b);
    if (st != SLORA_OK)
        return st;
    if (n_q_heads < 1 || n_q_heads > 8192 || n_q_heads % k->c.n_kv != 0)
        return fail(SLORA_ERR_INVALID_ARG, "%s: n_q_heads=%d is no multiple of the cache's %d", fn, n_q_heads, k->c.n_kv);
    const bool none = a.b.T == 0 || a.b.S == 0;
    const int64_t row = (int64_t)n_q_heads * k->head_dim;
    if ((st = check_rows(fn, "q", q, q_stride, row, none)) != SLORA_OK ||
        (st = check_rows(fn, "out", out, out_stride, row, none)) != SLORA_OK)
        return st;
    const int32_t group = n_q_heads / k->c.n_kv;
    if ((int64_t)a.b.max_q * group > 1 << 30)
        return fail(SLORA_ERR_UNSUPPORTED, "%s: %d new tokens of %d query heads per KV head", fn, a.b.max_q, group);
    if (!none && out == q)
        return fail(SLORA_ERR_INVALID_ARG, "%s: out is q", fn);
    if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) || !std::isfinite(softmax_scale))
        return fail(SLORA_ERR_INVALID_ARG, "%s: causal=%d window=%d softmax_scale=%g", fn, causal, window,
                    (double)softmax_scale);
    if (!aligned4(lse))
        return fail(SLORA_ERR_INVALID_ARG, "%s: lse is misaligned", fn);
    if (none)
        return SLORA_OK;
    a.c = k->c;
    a.q = static_cast<const __half *>(q);
    a.out = static_cast<__half *>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_q = n_q_heads;
    a.group = group;
    a.group_inverse = group == 1 ? 0u : (uint32_t)(((1ull << 32) + group - 1) / group);
    a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
    a.causal = causal;
    a.window = window;
    a.sinks = sinks;
    a.give_up = g_give_up.load();
    DeviceScope dev_scope(k->device);
    cudaError_t e = dev_scope.error();
    int launches = 0;
    // A batch whose sequences may be of both kinds runs both kernels.  One takes them all where the mean
    // is near max_q, or where the sequences that may have few rows (all but those that T needs, at max_q
    // new tokens each) add at most a unit per SM: the second launch costs 2 to 8 us (16 prompts 120 us
    // by one, 123 by two), and few rows gain little by it (24 sequences of 8 to 24 drafted tokens, 4 rows
    // each: 138 us by one, 163 by two; of 2 to 60: 150 and 172).  Single tokens in number are
    // dear beside prompts: 8 prompts and 64 of them take 346 us by one, 228 by two.
    const int64_t most = (int64_t)a.b.max_q * a.group;
    const bool big = most > kSmallRows;
    const int64_t others = a.b.max_q > 1 ? a.b.S - ((int64_t)a.b.T - a.b.S) / (a.b.max_q - 1) : 0;
    const bool alike = (int64_t)a.b.T * 4 >= (int64_t)a.b.S * a.b.max_q * 3 || others * k->c.n_kv <= k->num_sms;
    if (e == cudaSuccess && big)
        e = kv::launch_attend_prefill(a, k->head_dim, k->format, alike ? 0 : kSmallRows,
                                      k->ws + kv::decode_workspace_bytes(k->num_sms), k->num_sms, (cudaStream_t)stream,
                                      &launches);
    if (e == cudaSuccess && !(big && alike))
        e = kv::launch_attend_decode(a, k->maps, k->head_dim, k->format, kSmallRows, k->ws, k->num_sms,
                                     (cudaStream_t)stream, &launches);
    *k->launches += launches;
    return e == cudaSuccess ? SLORA_OK : fail(SLORA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

}  // namespace

extern "C" slora_status slora_kv_attend(slora_kv_t k, const slora_kv_batch *batch, const void *q, int64_t q_stride,
                                        int32_t n_q_heads, void *out, int64_t out_stride, float *lse,
                                        float softmax_scale, int32_t causal, int32_t window, slora_stream_t stream)
{
    return attend("kv_attend", k, batch, q, q_stride, n_q_heads, out, out_stride, lse, softmax_scale, causal, window, 0, stream);
}

extern "C" slora_status slora_kv_attend_sinks(slora_kv_t k, const slora_kv_batch *batch, const void *q, int64_t q_stride,
                                              int32_t n_q_heads, void *out, int64_t out_stride, float *lse,
                                              float softmax_scale, int32_t window, int32_t n_sinks, slora_stream_t stream)
{
    const char *fn = "kv_attend_sinks";
    if (n_sinks < 0 || n_sinks > (1 << 30) || window < 1)
        return fail(SLORA_ERR_INVALID_ARG, "%s: window=%d n_sinks=%d", fn, window, n_sinks);
    return attend(fn, k, batch, q, q_stride, n_q_heads, out, out_stride, lse, softmax_scale, 1, window, n_sinks, stream);
}

extern "C" slora_status slora_kv_copy(slora_kv_t k, int64_t n, const int32_t *src, const int32_t *dst, const int32_t *rows,
                                      slora_stream_t stream)
{
    if (!k)
        return fail(SLORA_ERR_INVALID_ARG, "kv_copy: null cache");
    if (n < 0 || n > INT32_MAX || (n > 0 && (!src || !dst)) || !aligned4(src) || !aligned4(dst) || !aligned4(rows))
        return fail(SLORA_ERR_INVALID_ARG, "kv_copy: n=%lld, or a list is null or misaligned", (long long)n);
    if (n == 0)
        return SLORA_OK;
    const kv::CopyArgs a = {k->c, (int32_t)n, src, dst, rows, k->head_dim};
    DeviceScope dev_scope(k->device);
    cudaError_t e = dev_scope.error();
    int launches = 0;
    if (e == cudaSuccess)
        e = kv::launch_copy(a, k->num_sms, (cudaStream_t)stream, &launches);
    *k->launches += launches;
    return e == cudaSuccess ? SLORA_OK : fail(SLORA_ERR_CUDA, "kv_copy: %s", cudaGetErrorString(e));
}

extern "C" slora_status slora_kv_compact(slora_kv_t k, const slora_kv_keep *keep, slora_stream_t stream)
{
    const char *fn = "kv_compact";
    if (!k || !keep)
        return fail(SLORA_ERR_INVALID_ARG, "%s: null cache or lists", fn);
    const int32_t *dst_table = keep->dst_table == keep->block_table ? nullptr : keep->dst_table;
    if (keep->n_seqs < 0 || keep->n_seqs > (1 << 20) || keep->n_kept < 0 || keep->n_kept > (1 << 30) || keep->max_kept < 0 ||
        keep->max_kept > (1 << 30) || keep->max_blocks < 1 || (dst_table && keep->dst_blocks < 1) ||
        (keep->kept_head_stride != 0 && keep->kept_head_stride < keep->n_kept))
        return fail(SLORA_ERR_INVALID_ARG, "%s: n_seqs=%d n_kept=%d max_kept=%d max_blocks=%d dst_blocks=%d kept_head_stride=%lld", fn,
                    keep->n_seqs, keep->n_kept, keep->max_kept, keep->max_blocks, keep->dst_blocks,
                    (long long)keep->kept_head_stride);
    if (keep->n_seqs > 0 && (!keep->kept_indptr || !keep->kv_len || !keep->block_table || (keep->n_kept > 0 && !keep->kept)))
        return fail(SLORA_ERR_INVALID_ARG, "%s: null kept_indptr, kept, kv_len or block_table", fn);
    for (const void *p : {(const void *)keep->kept_indptr, (const void *)keep->kept, (const void *)keep->first,
                          (const void *)keep->kv_len, (const void *)keep->block_table, (const void *)keep->dst_table,
                          (const void *)keep->new_len})
        if (!aligned4(p))
            return fail(SLORA_ERR_INVALID_ARG, "%s: a misaligned array", fn);
    // a sequence's arrays are read by CTAs that start after another has written its new length
    auto apart = [&](const int32_t *p, int64_t n) {
        const uintptr_t x = (uintptr_t)keep->new_len, y = (uintptr_t)p;
        return !p || !keep->new_len || x + 4 * (uintptr_t)keep->n_seqs <= y || y + 4 * (uintptr_t)n <= x;
    };
    if (!apart(keep->kept_indptr, (int64_t)keep->n_seqs + 1) || !apart(keep->first, keep->n_seqs) ||
        !apart(keep->kv_len, keep->n_seqs))
        return fail(SLORA_ERR_INVALID_ARG, "%s: new_len overlaps kept_indptr, first or kv_len", fn);
    if (keep->n_seqs == 0)
        return SLORA_OK;
    kv::CompactArgs a = {};
    a.c = k->c;
    a.S = keep->n_seqs;
    a.n_kept = keep->n_kept;
    a.max_kept = keep->max_kept < keep->n_kept ? keep->max_kept : keep->n_kept;
    a.max_blocks = keep->max_blocks;
    a.dst_blocks = dst_table ? keep->dst_blocks : keep->max_blocks;
    a.indptr = keep->kept_indptr;
    a.kept = keep->kept;
    a.first = keep->first;
    a.kv_len = keep->kv_len;
    a.table = keep->block_table;
    a.dst_table = dst_table;
    a.head_stride = keep->kept_head_stride;
    a.new_len = keep->new_len;
    DeviceScope dev_scope(k->device);
    cudaError_t e = dev_scope.error();
    int launches = 0;
    if (e == cudaSuccess)
        e = kv::launch_compact(a, k->head_dim, k->format, k->num_sms, (cudaStream_t)stream, &launches);
    *k->launches += launches;
    return e == cudaSuccess ? SLORA_OK : fail(SLORA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

extern "C" slora_status slora_debug_kv_give_up(int32_t cta)
{
    if (cta < -1)
        return fail(SLORA_ERR_INVALID_ARG, "debug_kv_give_up: cta=%d", cta);
    g_give_up.store(cta);
    return SLORA_OK;
}
