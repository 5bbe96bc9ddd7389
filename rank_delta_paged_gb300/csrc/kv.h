// The 8-bit KV cache in the pool's pages: what its kernels read about the cache and a batch,
// the conversions between fp32 / fp16 and the 8-bit codes, and the kernel launchers.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ptx.h"
#include "slora.h"

namespace slora {
namespace kv {

// Smallest exponent of a block's scale: 2^-40 is below the smallest fp16 subnormal over
// the largest code (2^-24 / 448), rotated values included, so it never costs precision, and
// a block of zeros starts there and can grow.
constexpr int kMinExponent = -40;

// Exponents beyond this are read as this; append writes -40 .. 11.  The softmax's sum carries
// 2^-exponent of the value blocks, which must stay a normal fp32 number, and so must the
// ratio of two scales.
constexpr int kExpLimit = 60;

// The softmax's weights are rounded to fp16 for the product with the values, so they stand high in its range: a
// reference m is taken kHeadRoom below the largest score, and kept until weights would pass
// 2^kMaxWeight (fp16 ends at 2^16).  A weight keeps its 11 bits down to 2^-21 of the largest and is lost below
// 2^-32 of it; with m at the largest score itself those were 2^-14 and 2^-25, and a key that held
// most of the softmax made the rest's weights coarse (errors of 1 part in 100 in their sum).
constexpr float kHeadRoom = 7.f;
constexpr float kMaxWeight = 15.f;

struct Cache {
    uint8_t *pool;          // page p starts at pool + p * page_bytes
    int8_t *exps;           // [num_pages]
    int64_t num_pages;
    int64_t page_bytes;
    int32_t n_kv;           // KV heads
    int32_t bt;             // tokens per block (page)
    int32_t *status;        // the pool's device status word
};

struct Batch {
    int32_t T, S, max_q, max_blocks;
    const int32_t *indptr;
    const int32_t *kv_len;
    const int32_t *table;   // [S][max_blocks][n_kv][2]
};

struct AppendArgs {
    Cache c;
    Batch b;
    const __half *k, *v, *q;
    __half *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int32_t n_q;
    int32_t rot, interleaved, n_pos;    // rot 0: no rotation
    const float *cos, *sin;
    const int32_t *positions;           // nullptr: positions in the cache
};

struct AttendArgs {
    Cache c;
    Batch b;
    const __half *q;
    __half *out;
    float *lse;
    int64_t q_stride, out_stride;
    int32_t n_q, group;
    uint32_t group_inverse;             // ceil(2^32 / group), 0 for 1
    float scale_log2;                   // softmax scale * log2(e)
    int32_t causal, window;
    int32_t give_up;                    // test hook: this CTA gives up at its start; -1: none
};

// The pages as a tensor [num_pages][rows][head_dim] of bytes, in boxes of R, 2R and 4R rows of a
// page (R = 16 if blocks are multiples of 16 tokens, else 8).
struct PageMaps {
    CUtensorMap m[3];
};

// Lengths beyond the block table; and above 2^30 tokens positions would leave 32 bits at the end of a tile.
__device__ __forceinline__ bool too_long(const Cache &c, const Batch &b, int32_t len)
{
    return len > 1 << 30 || (int64_t)len > (int64_t)b.max_blocks * c.bt;
}

// One sequence of a batch as the attention kernels see it: its new rows, its keys, and
// whether its sizes can be used.
struct Seq {
    int32_t row0;   // first row of q / out
    int32_t n;      // new tokens (0: skip)
    int32_t len;    // keys
};

__device__ __forceinline__ Seq load_seq(const AttendArgs &a, int32_t s, int32_t *bad)
{
    Seq q;
    const int32_t t0 = a.b.indptr[s], t1 = a.b.indptr[s + 1];
    q.row0 = t0;
    q.n = t1 - t0;
    q.len = a.b.kv_len[s];
    if (t0 < 0 || t1 < t0 || t1 > a.b.T || q.n > a.b.max_q) {
        *bad = SLORA_DEV_BAD_SEGMENT;
        q.n = 0;
    } else if (q.n > 0 && (q.len < 0 || too_long(a.c, a.b, q.len))) {
        *bad = SLORA_DEV_BAD_LENGTH;
        q.n = 0;
    }
    return q;
}

// r / group, 0 <= r < 2^31: the product with the inverse is the quotient or one more.
__device__ __forceinline__ int32_t div_group(const AttendArgs &a, int32_t r)
{
    if (a.group_inverse == 0) return r;
    const int32_t q = (int32_t)__umulhi((uint32_t)r, a.group_inverse);
    return q * a.group > r ? q - 1 : q;
}

// The same lane of the warp every time, and one that the compiler knows to be one.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// 64-bit quotients are long code; none is on a path that matters.
static __device__ __noinline__ int32_t div_list(int64_t x, int64_t y)
{
    if (((uint64_t)x | (uint64_t)y) >> 32 == 0) return (int32_t)((uint32_t)x / (uint32_t)y);
    return (int32_t)(x / y);
}

// First key that any of the rows [r0, r1) of new tokens sees, and one past the last; tokens
// counted from the sequence's first new one.
__device__ __forceinline__ int32_t first_key(const AttendArgs &a, const Seq &q, int32_t tok)
{
    if (a.window == 0) return 0;
    const int64_t p = (int64_t)q.len - q.n + tok - a.window + 1;
    return p > 0 ? (int32_t)p : 0;
}
__device__ __forceinline__ int32_t end_key(const AttendArgs &a, const Seq &q, int32_t tok)
{
    if (!a.causal) return q.len;
    const int32_t p = q.len - q.n + tok + 1;
    return p > 0 ? p : 0;
}

// Milliseconds or so, to be compared by differences.
__device__ __forceinline__ int32_t work_clock(uint64_t ns) { return (int32_t)(uint32_t)(ns >> 20); }

// Bounded wait on an mbarrier phase, as wait_phase of ptx.h: true once the phase has completed;
// false after the first timeout in the CTA (*abort, SLORA_DEV_TIMEOUT), from when on every wait that
// would have to wait gives up soon.  One try, which the hardware holds for up to 20 us, stands
// in line and the rest in a function: these kernels have some thirty waits, and with whole
// loops at each the code is fetched from L2 again and again.  The limit also counts from the work_clock() in
// abort[1], which is that of the start until a warp at long work renews it.
static __device__ __noinline__ bool wait_more(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 63u) != 0) continue;
        if (*abort) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        // (the other warp's clock may have been read after this one's)
        if (now - t0 > kWaitLimitNs && (int32_t)((uint32_t)work_clock(now) - (uint32_t)abort[1]) > work_clock(kWaitLimitNs)) {
            set_status(status, SLORA_DEV_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status)
{
    return mbar_try_wait(bar, parity) || wait_more(bar, parity, abort, status);
}

// ---- joins ---------------------------------------------------------------------------
// A unit that is cut between CTAs is joined by the last of them to arrive.  The words that count the arrivals
// outlive a call, and a CTA that gave up never arrives; so a count belongs to its launch, and whatever
// an earlier one left is below it.  The launches are numbered on the device, for a graph that is
// replayed passes the same arguments each time: n threads of a launch add to `started` when they start, all
// but one of them 1 and that one what makes 2^16, so the number stands above 16 bits of it, for arrivals.
struct Joins {
    unsigned long long *started;
    unsigned long long *word;
};
__device__ __forceinline__ uint64_t start_launch(const Joins &j, bool first, uint32_t n)
{
    return atomicAdd(j.started, first ? 0x10000ull - (n - 1) : 1ull);
}
// Whether this is the last of a unit's n arrivals in the launch.
__device__ __forceinline__ bool arrive_last(unsigned long long *word, uint64_t started, int32_t n)
{
    const unsigned long long none = started & ~0xFFFFull;
    atomicMax(word, none);              // without a result, and before the addition at the same address
    return atomicAdd(word, 1ull) == none + (unsigned)(n - 1);
}

// ---- codes ---------------------------------------------------------------------------
template <int FMT>
__device__ __forceinline__ constexpr float code_limit()
{
    return FMT == SLORA_KV_E4M3 ? 448.f : 127.f;
}

// Smallest e >= kMinExponent with amax <= limit * 2^e, amax finite and >= 0: compares the
// significands, limit = 1.75 * 2^8 (E4M3) or 1.984375 * 2^6 (INT8).
template <int FMT>
__device__ __forceinline__ int fit_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;
    const uint32_t top = FMT == SLORA_KV_E4M3 ? 0x600000u : 0x7E0000u;
    const int e = x - (FMT == SLORA_KV_E4M3 ? 8 : 6) + ((u & 0x7FFFFFu) > top);
    return e < kMinExponent ? kMinExponent : e;
}

// An exponent as read from memory that the caller may have written.
__device__ __forceinline__ int clamp_exponent(int e)
{
    return e < -kExpLimit ? -kExpLimit : e > kExpLimit ? kExpLimit : e;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e)
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two values in units of the scale -> two codes (x in the low byte).
template <int FMT>
__device__ __forceinline__ uint32_t encode2(float x, float y)
{
    if (FMT == SLORA_KV_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
        return r;
    }
    // the conversion saturates to -128 .. 127 and takes NaN to 0
    int32_t a, b;
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(fmaxf(x, -127.f)));
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(fmaxf(y, -127.f)));
    return __byte_perm((uint32_t)(x != x ? 0 : a), (uint32_t)(y != y ? 0 : b), 0x7740) & 0xFFFFu;
}

// Four codes -> fp16 pairs (bytes 0, 1) and (bytes 2, 3); exact in both formats.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if (FMT == SLORA_KV_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // byte b + 128 in the low bits of the fp16 number 1024 is 1024 + 128 + b
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __float2half2_rn(1152.f);
        uint32_t p = __byte_perm(u, 0x64646464u, 0x4140), q = __byte_perm(u, 0x64646464u, 0x4342);
        __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&p), off);
        __half2 b = __hsub2(*reinterpret_cast<__half2 *>(&q), off);
        lo = *reinterpret_cast<uint32_t *>(&a);
        hi = *reinterpret_cast<uint32_t *>(&b);
    }
}

// The bytes of four codes that are NaN, as their top bits (E4M3 without the sign: 127; INT8 has none).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// ---- launchers -------------------------------------------------------------------------
cudaError_t launch_append(const AppendArgs &a, int head_dim, int fmt, int num_sms, cudaStream_t stream,
                          int *launches);

// The attention's workspace: partial results of rows whose keys are split over several CTAs, and
// the words of their joins (zero at first).
size_t decode_workspace_bytes(int num_sms);
// The rows of sequences with at most small_rows (new tokens * group) rows per KV head; INT32_MAX: all.
cudaError_t launch_attend_decode(const AttendArgs &a, const PageMaps &maps, int head_dim, int fmt,
                                 int32_t small_rows, void *ws, int num_sms, cudaStream_t stream, int *launches);

// The rows of sequences with more than small_rows rows per KV head.
size_t prefill_workspace_bytes(int num_sms);
cudaError_t launch_attend_prefill(const AttendArgs &a, int head_dim, int fmt, int32_t small_rows, void *ws, int num_sms,
                                  cudaStream_t stream, int *launches);

}  // namespace kv
}  // namespace slora
