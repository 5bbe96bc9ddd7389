// Attention over the 8-bit paged KV cache for many rows per KV head (prompts and their chunks)
// on the 5th-generation tensor cores.
//
// The mathematics is that of kv_decode.cu: scores in units of log2, the value pages'
// exponents in the weights, one pass with a running maximum and sum.  A unit is 256 rows (new
// token * group + query head of the group) of one sequence and KV head, as two tiles of 128:
//     S_t = Q_t K^T      128 x 128 keys, fp32 in tensor memory
//     P_t = 2^(S_t f + g - m)  in fp16, over S_t's own columns of tensor memory
//     O_t += P_t V       fp32 in tensor memory
// What bounds it: 4 D flops per row and key on the tensor cores; the codes are read once per 256
// rows.  The tensor cores take fp16 from shared memory, so the codes of 128 keys and values are
// converted once per unit and tile for both row tiles (a sixteenth of the exponentials' work).
//
// Per CTA (one per SM): warps 0-3 and 4-7 are the softmax of row tile 0 and 1, a row per
// thread, so a row's maximum and sum need no exchange; warp 13 walks the work list and looks up
// pages and exponents some tiles ahead; warps 8-11 read the codes, a tile ahead in registers,
// and convert them into the swizzled operand tiles (K by rows, V as it stands: its channels run
// along N; tensor-map copies into a ring of raw pieces cost these warps more in waits than the
// loads do); warps 12 and 14 issue the products of row tile 0 and 1,
// O_t += P_t V and S_t = Q_t K' by turns, so that one row tile's softmax runs under the other's
// products (one warp for both was the bound: an issue costs it some 60 cycles, of 64 that a product takes).
// The roles' inner loops are kept short: with 15 warps in four programs, straight-line code is
// fetched again for every tile, and the warps wait for that.
//
// The key tiles of all units form one list, of which every CTA takes an equal run; a unit that
// is cut between CTAs is joined by the last of them to finish, in the order of the list.
//
// Measured: 2048 tokens x 32 heads over 30001 keys of 8 KV heads: 0.93 ms, 1.12 PFLOP/s, 58% of what a library
// product reaches; 16 prompts of 512, 32 heads: 108 us (E4M3; 105 without the look for NaN outputs).  A tile takes 2.3 us where its products need
// 1.3: the warps' instruction fetch and the softmax's waits for tensor memory.  Prompts this
// short are held up by a unit's start and end, about three tiles' time for two to four tiles.
#include <cstddef>
#include <mutex>

#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"
#include "tcgen05.h"

namespace slora {
namespace kv {
namespace {

constexpr int kTile = 128;                // keys per tile
constexpr int kRows = 256;                // rows per unit
constexpr int kThreads = 480;
constexpr int kConvWarp = 8, kMmaWarp = 12, kPlanWarp = 13, kMmaWarp1 = 14;
// What a unit costs besides its tiles, in tiles: its rows' loads, the first tile's maxima, the outputs.
// 24 prompts of 16 to 1500 tokens beside what they have cached: 512 us by 3, 547 by 0; 96 sequences
// of 2 to 60 drafted tokens 493 and 507; 16 equal prompts the same by either.
constexpr int kUnitCost = 3;
constexpr int kSeqChunks = 64;
constexpr int kDescs = 8;                 // tile descriptors: 3 being prepared, the others in use

enum : uint32_t {
    kFirst = 1, kLast = 2, kWhole = 4, kPlain = 8,
    kAct = 16,          // << t: row tile t sees keys of this tile
    kFirstAct = 64,     // << t: the first such tile of the unit in this CTA
    kLastAct = 256,     // << t: the last
    kEnd = 1024         // the CTA's last tile
};

struct Desc {
    int64_t off[2][16];     // keys and values: bytes from the pool's start to the first row of 8 tokens
    float ks[16];           // 2^exponent of the key pages, per 8 tokens
    float lv[16];           // exponent of the value pages
    float li[16];           // 2^-exponent of the value pages
    uint32_t flags;
    int32_t j0;             // first key
    int32_t lo, hi;         // keys that any of the unit's rows sees
    int32_t row0, n, len, head;
    int32_t r0, nrows;      // first row of the unit, and rows
    int32_t c0, c1;         // first and last CTA of the unit
    uint32_t ok;            // bit g: tokens 8g .. 8g+7 are there
    int32_t pad[3];
};
static_assert(sizeof(Desc) % 16 == 0 && offsetof(Desc, flags) % 16 == 0, "Desc");

template <int D>
struct Shape {
    static constexpr int kBlocks = D / 64;                   // 64-channel blocks of 128-byte rows
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kKVTile = kTile * D * 2;
    static constexpr int kStage = 32 * 64;                   // a warp's 32 rows of 32 channels on their way out
    static constexpr size_t kSmem =
        1024 + 2 * (size_t)kQTile + 4 * (size_t)kKVTile + 8 * (size_t)kStage + kDescs * sizeof(Desc);
    static constexpr int kPart = 2 * 128 + 128 * D;          // floats of a row tile's partial result: m, l, O
};

struct PrefillParams {
    AttendArgs a;
    int32_t small_rows;    // sequences with at most this many rows are another kernel's
    int32_t box_rows;      // 16 if blocks are multiples of 16 tokens, else 8
    int32_t min_tiles;
    uint32_t bt_inverse;
    float scale;           // softmax scale * log2(e), not zero
    uint32_t unseen;       // what a product must be for a score of -infinity
    float *part;           // [CTAs][2][2] partial results
    Joins joins;           // a word per CTA and row tile
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two fp32 numbers at a time.
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint4 ld_codes(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t ad)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(ad));
    return v;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t src_bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t ad, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(ad), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The product takes a NaN value to every row of the unit, as 0 times NaN to those that do not see its key. A warp
// goes through its rows: where an output is NaN in a channel in which one of the unit's keys that
// the row does not see is NaN, it sums the channel again over the keys that it sees, by the reference and the sum that the
// softmax has found (inv < 0: not this row).  (Channels that are NaN by a key which every row sees are right as they are.)  Rare, and
// slow: abort[1] tells the waits of the CTA's other warps that it goes on.
template <int D, int FMT>
static __device__ __noinline__ void sum_again(const PrefillParams &p, int32_t row0, int32_t head, int32_t r, int32_t rend, float base,
                                              float inv, volatile int *abort)
{
    const AttendArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    constexpr int CL = D / 32;                           // channels of a lane
    int32_t s = 0;
    for (int32_t hi = a.b.S - 1; s < hi;) {              // the last sequence that starts at or before row0
        const int32_t mid = (s + hi + 1) / 2;
        if (a.b.indptr[mid] <= row0) s = mid; else hi = mid - 1;
    }
    if (a.b.indptr[s] != row0)                           // offsets that decrease elsewhere
        for (s = 0; s < a.b.S - 1 && !(a.b.indptr[s] == row0 && a.b.indptr[s + 1] > row0);) ++s;
    int32_t bad = 0;
    const Seq q = load_seq(a, s, &bad);
    if ((int64_t)q.n * a.group < rend) return;           // offsets changed under the call
    const int32_t first = first_key(a, q, div_group(a, r & -kRows)), end = end_key(a, q, div_group(a, rend - 1));
    const int32_t *table = a.b.table + ((int64_t)s * a.b.max_blocks * a.c.n_kv + head) * 2;
    // the pages' rows of key k; false if it is not seen by any row
    auto place = [&](int32_t k, int32_t &kp, int32_t &vp, int32_t &row) {
        const int32_t blk = k / a.c.bt;
        row = (k - blk * a.c.bt) * D;
        kp = table[(int64_t)blk * a.c.n_kv * 2];
        vp = table[(int64_t)blk * a.c.n_kv * 2 + 1];
        return kp >= 0 && kp < a.c.num_pages && vp >= 0 && vp < a.c.num_pages;
    };
    // this lane's channels of a row of codes, the first in the low byte
    auto codes = [&](int64_t at) -> uint32_t {
        const uint8_t *c = a.c.pool + at + CL * lane;
        return CL == 4 ? *reinterpret_cast<const uint32_t *>(c) : *reinterpret_cast<const uint16_t *>(c);
    };
#pragma unroll 1
    for (unsigned rows = __ballot_sync(~0u, inv >= 0.f); rows; rows &= rows - 1) {
        const int l = __ffs(rows) - 1;
        const int32_t rr = __shfl_sync(~0u, r, l);
        const float m = __shfl_sync(~0u, base, l), iv = __shfl_sync(~0u, inv, l);
        const int32_t tok = div_group(a, rr), qh = head * a.group + (rr - tok * a.group);
        const int32_t k0 = first_key(a, q, tok), k1 = end_key(a, q, tok);
        __half *out = a.out + (int64_t)(q.row0 + tok) * a.out_stride + (int64_t)qh * D + CL * lane;
        uint32_t odd = 0;                                // channels: bit 8 c + 7, as nan_bytes has them
#pragma unroll
        for (int c = 0; c < CL; ++c)
            if ((__ldcg(reinterpret_cast<const unsigned short *>(out) + c) & 0x7FFFu) > 0x7C00u) odd |= 0x80u << (8 * c);
        if (!__any_sync(~0u, odd != 0)) continue;
        uint32_t unseen = 0;
#pragma unroll 1
        for (int32_t k = first; k < end; ++k) {
            if (k >= k0 && k < k1) {
                k = k1 - 1;
                continue;
            }
            int32_t kp, vp, row;
            if (place(k, kp, vp, row)) unseen |= nan_bytes(codes(vp * a.c.page_bytes + row));
        }
        odd &= unseen;
        if (!__any_sync(~0u, odd != 0)) continue;
        const uint4 *query = reinterpret_cast<const uint4 *>(a.q + (int64_t)(q.row0 + tok) * a.q_stride + (int64_t)qh * D);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int32_t kb = k0; kb < k1; kb += 32) {
            if (lane == 0) abort[1] = work_clock(global_timer_ns());
            // a key per lane, then a channel per lane
            int32_t kp, vp, row;
            float e = 0.f;
            int64_t at = -1;
            if (kb + lane < k1 && place(kb + lane, kp, vp, row)) {
                at = vp * a.c.page_bytes + row;
                const uint4 *key = reinterpret_cast<const uint4 *>(a.c.pool + kp * a.c.page_bytes + row);
                float dot = 0.f;
#pragma unroll 1
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 w = key[i], q0 = query[2 * i], q1 = query[2 * i + 1];
                    const uint32_t kw[4] = {w.x, w.y, w.z, w.w}, qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t h[2];
                        decode4<FMT>(kw[j], h[0], h[1]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&h[x]));
                            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&qw[2 * j + x]));
                            dot = fmaf(u.x, v.x, dot);
                            dot = fmaf(u.y, v.y, dot);
                        }
                    }
                }
                const float kx = pow2(clamp_exponent(a.c.exps[kp])) * p.scale;
                e = ex2(fmaf(dot, kx, (float)clamp_exponent(a.c.exps[vp])) - m);
            }
            __syncwarp();
#pragma unroll 4
            for (int j = 0; j < 32; ++j) {
                const float ej = __shfl_sync(~0u, e, j);
                const int64_t aj = __shfl_sync(~0u, at, j);
                uint32_t h[2] = {0u, 0u};
                if (aj >= 0) decode4<FMT>(codes(aj), h[0], h[1]);
#pragma unroll
                for (int x = 0; x < CL / 2; ++x) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[x]));
                    o[2 * x] = fmaf(ej, v.x, o[2 * x]);
                    o[2 * x + 1] = fmaf(ej, v.y, o[2 * x + 1]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CL; ++c)
            if (odd >> (8 * c + 7) & 1u) out[c] = __float2half_rn(o[c] * iv);
    }
}

struct Tiles {
    int32_t lo, hi;        // key tiles [lo, hi) of a unit, one at least
    int32_t k0, k1;        // keys
    int32_t b[2], e[2];    // key tiles that row tile t sees
};
__device__ __forceinline__ void unit_tiles(const AttendArgs &a, const Seq &q, int32_t r0, int32_t r1, Tiles &t)
{
    t.k0 = first_key(a, q, div_group(a, r0));
    t.k1 = end_key(a, q, div_group(a, r1 - 1));
    t.lo = t.k0 / kTile;
    t.hi = (t.k1 + kTile - 1) / kTile;
    if (t.hi <= t.lo) t.hi = t.lo + 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t x0 = r0 + 128 * i, x1 = r1 < x0 + 128 ? r1 : x0 + 128;
        t.b[i] = t.e[i] = 0;
        if (x0 < x1) {
            const int32_t k0 = first_key(a, q, div_group(a, x0)), k1 = end_key(a, q, div_group(a, x1 - 1));
            if (k1 > k0) {
                t.b[i] = k0 / kTile;
                t.e[i] = (k1 + kTile - 1) / kTile;
            }
        }
    }
}
// Its places in the list: the tiles, then kUnitCost empty ones.
__device__ __forceinline__ int32_t unit_count(const AttendArgs &a, const Seq &q, int32_t rows, int32_t rt)
{
    const int32_t r0 = rt * kRows, r1 = rows < r0 + kRows ? rows : r0 + kRows;
    const int32_t lo = first_key(a, q, div_group(a, r0)) / kTile, hi = (end_key(a, q, div_group(a, r1 - 1)) + kTile - 1) / kTile;
    return (hi > lo ? hi - lo : 1) + kUnitCost;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) attend_prefill_kernel(const __grid_constant__ PrefillParams p)
{
    using Sh = Shape<D>;
    constexpr int NB = Sh::kBlocks;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t q_sm = (smem_u32(smem_raw) + 1023) & ~1023u;      // two row tiles
    const uint32_t k_sm = q_sm + 2 * Sh::kQTile, v_sm = k_sm + 2 * Sh::kKVTile;
    const uint32_t stage_sm = v_sm + 2 * Sh::kKVTile;
    Desc *desc = reinterpret_cast<Desc *>(smem_raw + (stage_sm + 8 * Sh::kStage - smem_u32(smem_raw)));
    __shared__ uint64_t s_tfull[kDescs], s_tempty[kDescs], s_kfull[2], s_kempty[2], s_vfull[2], s_vempty[2];
    __shared__ uint64_t s_qfull, s_qempty, s_sfull[2], s_pfull[2], s_odone[2], s_ofree[2], s_join[2], s_said[2], s_turn[2], s_fin, s_unit;
    __shared__ int64_t s_sum[kSeqChunks];
    __shared__ uint32_t s_tmem;
    __shared__ uint64_t s_launch;
    __shared__ int s_abort[2], s_last[2];

    const AttendArgs &a = p.a;
    int32_t *status = a.c.status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(&s_tfull[i], 1);
            mbar_init(&s_tempty[i], 14);         // 4 converting, 8 softmax and 2 issuing warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_kfull[i], 4);
            mbar_init(&s_kempty[i], 2);
            mbar_init(&s_vfull[i], 4);
            mbar_init(&s_vempty[i], 2);
            mbar_init(&s_sfull[i], 1);
            mbar_init(&s_pfull[i], 4);
            mbar_init(&s_odone[i], 1);
            mbar_init(&s_ofree[i], 4);
            mbar_init(&s_join[i], 4);
            mbar_init(&s_said[i], 1);
            mbar_init(&s_turn[i], 1);
        }
        mbar_init(&s_qfull, 4);
        mbar_init(&s_qempty, 2);
        mbar_init(&s_fin, 2);
        mbar_init(&s_unit, 1);
        fence_mbar_init();
        s_abort[0] = 0;
        s_abort[1] = work_clock(global_timer_ns());
    }
    griddep_wait();
    griddep_launch_dependents();
    uint64_t started = 0;
    if (tid == 32 * kPlanWarp) started = start_launch(p.joins, blockIdx.x == 0, gridDim.x);
    if (tid == 0 && (int32_t)blockIdx.x == a.give_up) {
        set_status(status, SLORA_DEV_TIMEOUT);
        s_abort[0] = 1;
    }

    // Tiles of each run of `per` sequences; every CTA sums them for itself.
    const int S = a.b.S;
    const int per = ((S + kSeqChunks - 1) / kSeqChunks + 31) / 32 * 32;
    const int chunks = (S + per - 1) / per;
    if (tid >= chunks && tid < kSeqChunks) s_sum[tid] = 0;
    int32_t bad = 0;
#pragma unroll 1
    for (int c = warp; c < chunks; c += kThreads / 32) {
        int64_t t = 0;
#pragma unroll 1
        for (int64_t s = (int64_t)c * per; s < S && s < (int64_t)(c + 1) * per; s += 32) {
            Seq q = {0, 0, 0};
            if (s + lane < S) q = load_seq(a, (int32_t)s + lane, &bad);
            const int64_t rows64 = (int64_t)q.n * a.group;
            unsigned big = __ballot_sync(~0u, rows64 > p.small_rows && q.n > 0);
#pragma unroll 1
            while (big) {
                const int l = __ffs(big) - 1;
                big &= big - 1;
                Seq u;
                u.row0 = __shfl_sync(~0u, q.row0, l);
                u.n = __shfl_sync(~0u, q.n, l);
                u.len = __shfl_sync(~0u, q.len, l);
                const int32_t rows = u.n * a.group;
#pragma unroll 1
                for (int32_t rt = lane; rt * kRows < rows; rt += 32) t += unit_count(a, u, rows, rt);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) s_sum[c] = t * a.c.n_kv;
    }
    if (bad && blockIdx.x == 0) set_status(status, bad);
    __syncthreads();
    int64_t v0 = s_sum[2 * lane], v1 = s_sum[2 * lane + 1], W = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(~0u, W, o);
        if (lane >= o) W += u;
    }
    const int64_t before = W - v0 - v1;
    W = __shfl_sync(~0u, W, 31);
    int64_t run = div_list(W + gridDim.x - 1, gridDim.x);
    if (run < p.min_tiles) run = p.min_tiles;
    const int64_t w0 = (int64_t)blockIdx.x * run, w1 = w0 + run < W ? w0 + run : W;
    if (w0 >= W - kUnitCost) return;
    volatile int *abort = s_abort;

    if (warp == kMmaWarp) tc::tmem_alloc(&s_tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    // columns: S_0, S_1 (P over them), O_0, O_1
    const uint32_t tm_s = tmem, tm_o = tmem + 256;

    if (warp == kPlanWarp) {
        // ---- the work list -----------------------------------------------------------------
        const unsigned hit = __ballot_sync(~0u, before <= w0);
        const int at = 31 - __clz(hit);
        int chunk = 2 * at;
        int64_t base = __shfl_sync(~0u, before, at);
        const int64_t half = __shfl_sync(~0u, v0, at);
        if (base + half <= w0) {
            base += half;
            ++chunk;
        }
        // the 32 sequences that the lanes hold, and those of them with work
        int32_t s32 = chunk * per, at_lane = -1;
        Seq q, u = {0, 0, 0};
        unsigned big = 0;
        s32 -= 32;
        int32_t rows = 0, head = 0, rt = 0;
        // the next sequence with work; false if there is none
        auto next_seq = [&]() {
#pragma unroll 1
            while (big == 0) {
                s32 += 32;
                if (s32 >= S) return false;
                q = Seq{0, 0, 0};
                int32_t ignore;
                if (s32 + lane < S) q = load_seq(a, s32 + lane, &ignore);
                big = __ballot_sync(~0u, q.n > 0 && (int64_t)q.n * a.group > p.small_rows);
            }
            at_lane = __ffs(big) - 1;
            big &= big - 1;
            u.row0 = __shfl_sync(~0u, q.row0, at_lane);
            u.n = __shfl_sync(~0u, q.n, at_lane);
            u.len = __shfl_sync(~0u, q.len, at_lane);
            rows = u.n * a.group;
            head = rt = 0;
            return true;
        };
        bool found = false;
#pragma unroll 1
        while (next_seq()) {
            int64_t t = 0;
#pragma unroll 1
            for (int32_t i = lane; i * kRows < rows; i += 32) t += unit_count(a, u, rows, i);
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
            if (base + t * a.c.n_kv > w0) {
                head = div_list(w0 - base, t);
                base += head * t;
                found = true;
                break;
            }
            base += t * a.c.n_kv;
        }
        // the row tile of the head that holds w0
#pragma unroll 1
        while (found) {
            const int32_t i = rt + lane;
            const int32_t mine = (int64_t)i * kRows < rows ? unit_count(a, u, rows, i) : 0;
            int32_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned past = __ballot_sync(~0u, base + sum > w0);
            if (past) {
                const int l = __ffs(past) - 1;
                rt += l;
                base += __shfl_sync(~0u, sum - mine, l);
                break;
            }
            base += __shfl_sync(~0u, sum, 31);
            rt += 32;
            if ((int64_t)rt * kRows >= rows) found = false;
        }
        if (!found && lane == 0) {        // the lengths changed under the call
            set_status(status, SLORA_DEV_BAD_LENGTH);
            s_abort[0] = 1;
        }
        Tiles ut = {};
        int32_t r0 = 0, r1 = 0, tile = 0, c0 = 0, c1 = 0;
        bool whole = false;
        int32_t ta = 0, tb = 0;                    // the unit's key tiles in this CTA
        int32_t plain_lo = 0, plain_hi = 0;        // keys that all of its rows see
        const int32_t *table = nullptr;
        auto enter = [&](int64_t u0) {             // the unit starts at u0 of the list
            r0 = rt * kRows;
            r1 = rows < r0 + kRows ? rows : r0 + kRows;
            unit_tiles(a, u, r0, r1, ut);
            const int64_t u1 = u0 + ut.hi - ut.lo;
            whole = u0 >= w0 && u1 <= w1;
            c0 = c1 = 0;
            if (!whole) {
                c0 = div_list(u0, run);
                c1 = div_list(u1 - 1, run);
            }
            ta = u0 >= w0 ? ut.lo : w0 - u0 < ut.hi - ut.lo ? ut.lo + (int32_t)(w0 - u0) : ut.hi;
            tb = u1 <= w1 ? ut.hi : ut.hi - (int32_t)(u1 - w1);
            tile = ta;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (ut.b[t] < ta) ut.b[t] = ta;
                if (ut.e[t] > tb) ut.e[t] = tb;
            }
            plain_lo = first_key(a, u, div_group(a, r1 - 1));
            plain_hi = end_key(a, u, div_group(a, r0));
            table = a.b.table + ((int64_t)(s32 + at_lane) * a.b.max_blocks * a.c.n_kv + head) * 2;
        };
        int64_t u0 = base;
        bool more = found;
        bool fresh = true;                              // the unit has yet to be entered
        const int gl = lane & 15, kvl = lane >> 4;      // this lane's 8 tokens of a tile, and keys or values
        const int R = p.box_rows;                       // tokens that share a page: 16, or 8
        struct Box {
            bool want;
            int32_t page, row;
        };
        int slot = 0;
        uint32_t slot_parity = 1;
        // The next tile: everything but pages and scales goes to its descriptor at once.
        auto describe = [&](Box &x) {
            x.want = false;
            x.page = x.row = 0;
            while (more && (fresh || tile >= tb)) {
                if (!fresh) {
                    u0 += ut.hi - ut.lo + kUnitCost;
                    if (u0 >= w1) {
                        more = false;
                        break;
                    }
                    if ((int64_t)(++rt) * kRows >= rows) {
                        rt = 0;
                        if (++head == a.c.n_kv && !next_seq()) {      // the lengths changed under the call
                            if (lane == 0) set_status(status, SLORA_DEV_BAD_LENGTH);
                            more = false;
                            break;
                        }
                    }
                }
                enter(u0);          // (nothing of it is left if w0 is among its empty places)
                fresh = false;
            }
            if (!more) return false;
            if (!wait_bar(&s_tempty[slot], slot_parity, abort, status)) return false;
            Desc &d = desc[slot];
            if (++slot == kDescs) {
                slot = 0;
                slot_parity ^= 1;
            }
            const int32_t j0 = tile * kTile, j = j0 + (8 * gl & -R);      // first token of the box
            x.want = j < ut.k1 && j + R > ut.k0;
            if (x.want) {
                int32_t blk = (int32_t)__umulhi((uint32_t)j, p.bt_inverse);
                x.row = j - blk * a.c.bt;
                if (x.row < 0) {
                    --blk;
                    x.row += a.c.bt;
                }
                x.page = __ldg(table + (int64_t)blk * a.c.n_kv * 2 + kvl);
            }
            if (lane == 0) {
                uint32_t f = (tile == ta ? kFirst : 0) | (tile == tb - 1 ? kLast : 0) | (whole ? kWhole : 0);
                if (tile == tb - 1 && (tb < ut.hi || u0 + ut.hi - ut.lo + kUnitCost >= w1)) f |= kEnd;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (tile >= ut.b[t] && tile < ut.e[t])
                        f |= (kAct << t) | (tile == ut.b[t] ? kFirstAct << t : 0) | (tile == ut.e[t] - 1 ? kLastAct << t : 0);
                }
                if (j0 >= plain_lo && j0 + kTile <= plain_hi) f |= kPlain;
                int4 *di = reinterpret_cast<int4 *>(&d.flags);
                di[0] = make_int4((int)f, j0, ut.k0, ut.k1);
                di[1] = make_int4(u.row0, u.n, u.len, head);
                di[2] = make_int4(r0, r1 - r0, c0, c1);
            }
            ++tile;
            return true;
        };
        auto exponent_of = [&](Box &x) {
            if (x.want && (x.page < 0 || x.page >= a.c.num_pages)) {
                set_status(status, SLORA_DEV_BAD_PAGE);
                x.want = false;
            }
            return x.want ? (int32_t)a.c.exps[x.page] : 0;
        };
        // A tile lies between the reading of a tile's page ids and of its exponents, and one more between
        // those and their use; but the first tile goes out as soon as it can.
        const Box none = {false, 0, 0};
        Box b0 = none, b1 = none, b2;
        bool n0 = false, n1 = false, n2;
        int32_t e0 = 0, e1;
#pragma unroll 1
        for (int32_t i = -2;; ++i, b0 = b1, b1 = b2, n0 = n1, n1 = n2, e0 = e1) {
            e1 = exponent_of(b1);
            n2 = describe(b2);
            if (i == -2) {
                __syncwarp();
                if (lane == 0 && n2) mbar_arrive(&s_unit);       // the first unit is known
                e0 = exponent_of(b2);                            // checks its pages, before anything is made of them
                b0 = b2;
                n0 = n2;
            } else if (i < 0) {
                continue;
            }
            if (!n0 || *abort) break;
            if (i == 0) continue;
            Desc &d = desc[i < 0 ? 0 : i % kDescs];
            // a group needs both its keys and its values
            const unsigned have = __ballot_sync(~0u, b0.want), ok = have & have >> 16 & 0xFFFFu;
            const bool both = ok >> gl & 1u;
            const int e = both ? clamp_exponent(e0) : 0;
            d.off[kvl][gl] = both ? (int64_t)b0.page * a.c.page_bytes + (b0.row + (8 * gl & (R - 1))) * D : 0;
            if (kvl == 0) {
                d.ks[gl] = pow2(e);
            } else {
                d.lv[gl] = (float)e;
                d.li[gl] = pow2(-e);
            }
            if (lane == 0) {
                d.ok = ok;
                if (ok != 0xFFFFu) d.flags &= ~kPlain;
            }
            __syncwarp();
            if (lane == 0) {
                if (i < 0) s_launch = started;          // with the first tile
                mbar_arrive(&s_tfull[i < 0 ? 0 : i % kDescs]);
            }
        }
    } else if (warp == kMmaWarp || warp == kMmaWarp1) {
        // ---- products of one row tile -------------------------------------------------------
        // The whole warp walks the tiles, by values that are the same in every lane, so that
        // the descriptors stay in uniform registers; one lane issues.
        constexpr uint32_t id_s = tc::idesc_f16_f32(128, kTile, 0, 0), id_o = tc::idesc_f16_f32(128, D, 0, 1);
        const uint32_t t = __shfl_sync(~0u, warp == kMmaWarp1 ? 1u : 0u, 0);
        // Descriptors: 16 channels are 32 bytes of a swizzled row of Q and K, 64 a block of 128
        // rows; 16 keys are 16 rows of V.  Only the low words differ.
        const uint64_t dq = tc::smem_desc_sw128(q_sm + t * Sh::kQTile, 16, 1024), dk = tc::smem_desc_sw128(k_sm, 16, 1024);
        const uint64_t dv = tc::smem_desc_sw128(v_sm, 128 * 128, 1024);
        const uint32_t ut = __shfl_sync(~0u, tmem, 0), o = ut + 256 + D * t, w = ut + 128 * t;
        const bool leader = elect_one();
        uint32_t q_par = 0, p_par = 0, of_par = 1, turn = t ^ 1u, f = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(~0u, wait_bar(bar, parity, abort, status)) != 0; };
        auto scores = [&](int32_t j) {
            const uint64_t y = dk + (uint32_t)((j & 1) * (Sh::kKVTile >> 4));
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t step = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
                    tc::mma_f16(w, dq + step, y + step, id_s, kk != 0);
                }
                tc::commit(&s_sfull[t]);
            }
        };
        // Tile i's weights times its values, then tile i + 1's scores, in turn with the other row tile's
        // warp: products of both at once would end together, and the two softmaxes would run
        // side by side instead of each under the other's products.
#pragma unroll 1
        for (int32_t i = -1;; ++i) {
            const int32_t j = i + 1;
            const bool more = (f & kEnd) == 0;
            uint32_t g = 0;
            if (more) {
                if (!wait(&s_tfull[j % kDescs], (uint32_t)(j / kDescs) & 1u)) break;
                g = __shfl_sync(~0u, desc[j % kDescs].flags, 0);
                if (!wait(&s_kfull[j & 1], (uint32_t)(j >> 1) & 1u)) break;
            }
            const bool fresh = g & kFirst;           // tile j is another unit's: its rows are still to come
            if (i >= 0) {
                const bool act = f & (kAct << t), first = f & (kFirstAct << t);
                if (!wait(&s_vfull[i & 1], (uint32_t)(i >> 1) & 1u)) break;
                if (act) {
                    if (!wait(&s_pfull[t], p_par)) break;
                    p_par ^= 1u;
                    if (first) {
                        if (!wait(&s_ofree[t], of_par)) break;
                        of_par ^= 1u;
                    }
                }
                if (!wait(&s_turn[t], turn)) break;
                turn ^= 1u;
                tc::fence_after_sync();
                if (act && leader) {
                    const uint64_t d = dv + (uint32_t)((i & 1) * (Sh::kKVTile >> 4));
                    tc::mma_f16_ts(o, w, d, id_o, !first);
#pragma unroll 1
                    for (int kk = 1; kk < kTile / 16; ++kk) tc::mma_f16_ts(o, w + kk * 8, d + kk * (2048 >> 4), id_o, 1);
                    if (f & (kLastAct << t)) tc::commit(&s_odone[t]);
                }
                if (more && !fresh && (g & (kAct << t))) scores(j);
                if (leader) {
                    mbar_arrive(&s_turn[t ^ 1u]);
                    tc::commit(&s_vempty[i & 1]);
                    mbar_arrive(&s_tempty[i % kDescs]);
                }
            }
            if (!more) break;
            if (fresh) {
                if (!wait(&s_qfull, q_par)) break;
                q_par ^= 1;
                tc::fence_after_sync();
                if (g & (kAct << t)) scores(j);
            }
            if (leader) {
                tc::commit(&s_kempty[j & 1]);
                if (g & kLast) tc::commit(&s_qempty);
            }
            f = g;
        }
        // every product issued has completed before tensor memory is released
        if (leader) tc::commit(&s_fin);
        volatile int gone[2] = {0, abort[1]};
        wait_bar(&s_fin, 0, gone, status);
        __syncwarp();
    } else if (warp >= kConvWarp && warp < kMmaWarp) {
        // ---- codes to fp16 operand tiles -----------------------------------------------------
        const int ct = tid - kConvWarp * 32;                   // 0 .. 127
        // Warp w of the four has rows 32 w .. + 31: a lane loads chunks ch (and ch + 4 if D = 128) of rows rw,
        // rw + 8, rw + 16, rw + 24, so that eight lanes store to all banks.
        constexpr int NC = D / 64, NL = 4 * NC;
        const int ch = lane & 3, r0 = (warp - kConvWarp) * 32, rw = lane >> 2;
        const uint8_t *codes = a.c.pool + rw * D + ch * 16;
        const uint32_t put = (r0 + rw) * 128 + (((2 * ch) ^ rw) << 4);
        auto load = [&](const Desc &d, int kvl, uint4 (&r)[NL]) {
            const longlong2 *o = reinterpret_cast<const longlong2 *>(&d.off[kvl][r0 / 8]);
            const longlong2 o0 = o[0], o1 = o[1];
            const int64_t at[4] = {o0.x, o0.y, o1.x, o1.y};
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int c = 0; c < NC; ++c) r[x * NC + c] = ld_codes(codes + at[x] + 64 * c);
        };
        auto store = [&](const Desc &d, uint32_t dst, uint4 (&r)[NL]) {
            // the conversions stay behind the waits before this call: moved up to the loads, they
            // would wait for them there
#pragma unroll
            for (int x = 0; x < NL; ++x) asm volatile("" : "+r"(r[x].x), "+r"(r[x].y), "+r"(r[x].z), "+r"(r[x].w));
            if (__builtin_expect(!(d.ok == 0xFFFFu && d.j0 >= d.lo && d.j0 + kTile <= d.hi), 0)) {
                // rows that are not seen may hold anything: zeros
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = r0 + rw + 8 * x;
                    const int32_t j = d.j0 + row;
                    if (!((d.ok >> (row >> 3) & 1u) && j >= d.lo && j < d.hi))
#pragma unroll
                        for (int c = 0; c < NC; ++c) r[x * NC + c] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint4 v = r[x * NC + c];
                    const uint32_t at = dst + put + x * 8 * 128 + c * (128 * 128);
                    uint32_t h[8];
                    decode4<FMT>(v.x, h[0], h[1]);
                    decode4<FMT>(v.y, h[2], h[3]);
                    decode4<FMT>(v.z, h[4], h[5]);
                    decode4<FMT>(v.w, h[6], h[7]);
                    sts128(at, h[0], h[1], h[2], h[3]);
                    sts128(at ^ 16u, h[4], h[5], h[6], h[7]);
                }
        };
        auto done = [&](uint64_t *bar) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // The rows of a unit by asynchronous copies of 16 bytes, zeros past the last: chunk ct & 7 of row
        // (ct >> 3) + 16 s of each 64-channel block.
        auto load_rows = [&](const Desc &e) {
            const int qc = ct & 7;
            const int32_t nrows = e.nrows, steps = nrows > 128 ? 16 : 8;
            const __half *src0 = a.q + (int64_t)e.row0 * a.q_stride + (int64_t)e.head * a.group * D + qc * 8;
#pragma unroll 2
            for (int s = 0; s < steps; ++s) {
                const int row = (ct >> 3) + 16 * s;
                const int32_t r = e.r0 + (row < nrows ? row : 0);
                const int32_t tok = div_group(a, r);
                const __half *src = src0 + (int64_t)tok * a.q_stride + (r - tok * a.group) * D;
                const uint32_t at = q_sm + (row >> 7) * Sh::kQTile + (row & 127) * 128 + ((qc ^ (row & 7)) << 4);
#pragma unroll
                for (int b = 0; b < NB; ++b) copy16(at + b * (128 * 128), src + b * 64, row < nrows ? 16u : 0u);
            }
            cp_async_commit();
        };
        // Keys run a tile ahead of values: K_0, K_1, V_0, K_2, V_1, ..  One loop for both, with the next half
        // tile's codes on their way in rb, keeps the code short; the moves at its end cost less than a second copy.
        uint4 ra[NL], rb[NL];
        uint32_t qe_par = 0;
        bool rows_under_way = true;
        int32_t i = 0, last = 0x7FFFFFFF;                      // the tile, and the last of the run once known
        int kv = 0;
        // the first unit's rows, under way while its pages are looked up
        if (wait_bar(&s_unit, 0, abort, status)) load_rows(desc[0]);
        if (wait_bar(&s_tfull[0], 0, abort, status)) {
            load(desc[0], 0, ra);
#pragma unroll 1
            for (;;) {
                const Desc &d = desc[i % kDescs];
                if (kv == 0 && (d.flags & kEnd)) last = i;
                // the half tile after this one
                int nk = 1;
                int32_t ni = i - 1;
                if (kv == 1) {
                    nk = i + 2 <= last ? 0 : 1;
                    ni = i + 2 <= last ? i + 2 : i + 1;
                } else if (i == 0) {
                    nk = last > 0 ? 0 : 1;
                    ni = last > 0 ? 1 : 0;
                }
                const bool more = ni <= last;
                if (more) {
                    if (nk == 0 && !wait_bar(&s_tfull[ni % kDescs], (uint32_t)(ni / kDescs) & 1u, abort, status)) break;
                    load(desc[ni % kDescs], nk, rb);
                }
                if (!wait_bar(kv ? &s_vempty[i & 1] : &s_kempty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, abort, status)) break;
                store(d, (kv ? v_sm : k_sm) + (i & 1) * Sh::kKVTile, ra);
                done(kv ? &s_vfull[i & 1] : &s_kfull[i & 1]);
                if (__builtin_expect(rows_under_way, 0)) {
                    cp_async_wait<0>();
                    done(&s_qfull);
                    rows_under_way = false;
                }
                if (kv && lane == 0) mbar_arrive(&s_tempty[i % kDescs]);
                // the rows of a unit that starts with the next tile
                if (kv && i < last && __builtin_expect(desc[(i + 1) % kDescs].flags & kFirst, 0)) {
                    if (!wait_bar(&s_qempty, qe_par, abort, status)) break;
                    qe_par ^= 1;
                    load_rows(desc[(i + 1) % kDescs]);
                    rows_under_way = true;
                }
                if (!more) break;
#pragma unroll
                for (int x = 0; x < NL; ++x) ra[x] = rb[x];
                kv = nk;
                i = ni;
            }
        }
        cp_async_wait<0>();
    } else if (warp < kConvWarp) {
        // ---- softmax: one row per thread -------------------------------------------------------
        const int t = warp >> 2;                               // row tile
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21; // lane 32 (warp & 3) of tensor memory
        const uint32_t ts = tm_s + 128 * t + lane_base, to = tm_o + D * t + lane_base;
        const int row = tid & 127;
        uint32_t s_par = 0, od_par = 0, j_par = 0;
        float mx = -INFINITY, sum = 0.f;
        bool any = false;
        // The largest score of 32 keys.
        auto top_of = [&](const Desc &d, const uint32_t (&x)[32], int h) {
            float top = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float kx = d.ks[4 * h + g] * p.scale, lv = d.lv[4 * h + g];
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaf(__uint_as_float(x[8 * g + k]), kx, lv));
            }
            return top;
        };
        int32_t klo = 0, khi = 0;                              // keys that the row sees
        uint32_t f = 0;
        for (int32_t i = 0; (f & kEnd) == 0; ++i) {
            if (!wait_bar(&s_tfull[i % kDescs], (uint32_t)(i / kDescs) & 1u, abort, status)) break;
            const Desc &d = desc[i % kDescs];
            f = d.flags;
            if (f & kFirst) {
                mx = -INFINITY;
                sum = 0.f;
                any = false;
                const Seq q = {d.row0, d.n, d.len};
                const int32_t r = d.r0 + 128 * t + row, last = d.r0 + d.nrows - 1;
                const int32_t tok = div_group(a, r < last ? r : last);
                klo = first_key(a, q, tok);
                khi = end_key(a, q, tok);
            }
            if (f & (kAct << t)) {
                if (!wait_bar(&s_sfull[t], s_par, abort, status)) break;
                s_par ^= 1;
                tc::fence_after_sync();
                const bool plain = f & kPlain;
                const int32_t m0 = klo - d.j0;
                const uint32_t mn = khi > klo ? (uint32_t)(khi - klo) : 0u;
                const uint32_t ok = d.ok;
                // The loops over a tile's columns stay rolled and what is rare stays out of them: the
                // roles' code has to fit the instruction caches.
                uint32_t x[32];
                int hn = 4;                                    // some row of the warp sees keys 32 (hn - 1) .. + 31, none later ones
                if (__builtin_expect(!plain, 0)) {
                    // the scores of unseen keys, in place, where some rows see some of 32 keys
                    const int32_t v0 = m0 < 0 ? 0 : m0, v1 = m0 + (int32_t)mn;
                    const int32_t a1 = __reduce_max_sync(~0u, v0);
                    const int32_t z0 = __reduce_min_sync(~0u, v1), z1 = __reduce_max_sync(~0u, v1);
                    while (hn > 0 && (z1 <= 32 * hn - 32 || (ok >> (4 * hn - 4) & 15u) == 0)) --hn;
#pragma unroll 1
                    for (int h = 0; h < hn; ++h) {
                        const uint32_t okh = ok >> (4 * h) & 15u;
                        if (a1 <= 32 * h && z0 >= 32 * h + 32 && okh == 15u) continue;
                        tc::ld_32x32b_x32(ts + 32 * h, x);
                        tc::ld_wait(x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const bool see = (uint32_t)(32 * h + k - m0) < mn && (okh >> (k / 8) & 1u);
                            if (!see) x[k] = p.unseen;
                        }
                        tc::st_32x32b_x32(ts + 32 * h, x);
                    }
                    tc::st_wait();
                }
                if (__builtin_expect(__any_sync(~0u, mx == -INFINITY), 0)) {
                    // rows that have seen nothing yet start from this tile's maximum
                    float top = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < hn; ++h) {
                        tc::ld_32x32b_x32(ts + 32 * h, x);
                        tc::ld_wait(x);
                        top = fmaxf(top, top_of(d, x, h));
                    }
                    if (mx == -INFINITY) mx = top - kHeadRoom;
                }
                // The weights, 32 keys at a time, by the running maximum as it stands.  It follows only when the
                // 32 weights' sum passes 2^kMaxWeight, to kHeadRoom below the largest score itself: a key
                // that outweighs all others then has the weight 2^7, which fp16 holds exactly (an integer above
                // its score made the outputs' error 2.9e-4 of their norm instead of 2.3e-4).  What this tile's
                // earlier keys made with the old one is rounded a second time.
                uint32_t xa[16], xb[16], pk[16];
                float raw, add, base = mx == -INFINITY ? 0.f : mx;
                // 16 scores into pk[at ..], their sums plain and without the value pages' scales
                auto weigh = [&](const uint32_t (&v)[16], int c, int at) {
                    const float2 ks = *reinterpret_cast<const float2 *>(&d.ks[2 * c]);
                    const float2 lv = *reinterpret_cast<const float2 *>(&d.lv[2 * c]);
                    const float2 li = *reinterpret_cast<const float2 *>(&d.li[2 * c]);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float kx = (g ? ks.y : ks.x) * p.scale, lx = (g ? lv.y : lv.x) - base;
                        const uint64_t k2 = pair(kx, kx), l2 = pair(lx, lx);
                        uint64_t s2 = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 z = unpair(fma2(pair(__uint_as_float(v[8 * g + 2 * k]),
                                                              __uint_as_float(v[8 * g + 2 * k + 1])), k2, l2));
                            const float e0 = ex2(z.x), e1 = ex2(z.y);
                            s2 = add2(s2, pair(e0, e1));
                            const __half2 hh = __floats2half2_rn(e0, e1);
                            pk[at + 4 * g + k] = *reinterpret_cast<const uint32_t *>(&hh);
                        }
                        const float2 sg = unpair(s2);
                        raw += sg.x + sg.y;
                        add = fmaf(sg.x + sg.y, g ? li.y : li.x, add);
                    }
                };
                tc::ld_32x32b_x16(ts, xa);
#pragma unroll 1
                for (int h = 0; h < hn; ++h) {
                    raw = add = 0.f;
                    tc::ld_wait(xa);
                    tc::ld_32x32b_x16(ts + 32 * h + 16, xb);
                    weigh(xa, 2 * h, 0);
                    tc::ld_wait(xb);
                    tc::ld_32x32b_x16(ts + (32 * (h + 1) & 127), xa);      // (not used after the last)
                    weigh(xb, 2 * h + 1, 8);
                    const bool up = raw > 32768.f;
                    if (__builtin_expect(__any_sync(~0u, up), 0)) {
                        tc::ld_32x32b_x32(ts + 32 * h, x);
                        tc::ld_wait(x);
                        const float nm = up ? top_of(d, x, h) - kHeadRoom : mx;
                        const float k = mx == nm ? 1.f : ex2(mx - nm);
                        mx = nm;
                        base = mx == -INFINITY ? 0.f : mx;
                        sum *= k;
                        uint32_t y[16];
                        if (any)
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                tc::ld_32x32b_x16(to + 16 * c, y);
                                tc::ld_wait(y);
#pragma unroll
                                for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * k);
                                tc::st_32x32b_x16(to + 16 * c, y);
                            }
                        // in two steps where k is so small that fp16 has few bits of it
                        float part = fmaxf(k, 0x1p-13f);
#pragma unroll 1
                        for (int e = 0; e < 2; ++e) {
                            const __half2 kh = __float2half2_rn(part);
#pragma unroll 1
                            for (int c = 0; c < h; ++c) {
                                tc::ld_32x32b_x16(ts + 16 * c, y);
                                tc::ld_wait(y);
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    __half2 w = __hmul2(*reinterpret_cast<__half2 *>(&y[j]), kh);
                                    y[j] = *reinterpret_cast<uint32_t *>(&w);
                                }
                                tc::st_32x32b_x16(ts + 16 * c, y);
                            }
                            tc::st_wait();
                            if (__all_sync(~0u, k >= 0x1p-13f)) break;
                            part = fminf(k * 0x1p13f, 1.f);
                        }
                        // these 32 again, from scores rounded as the maximum was, so that no weight
                        // is above 2^8 however large they are
                        add = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float kv = d.ks[4 * h + j / 8] * p.scale, l = d.lv[4 * h + j / 8];
                            const float e0 = ex2(fmaf(__uint_as_float(x[j]), kv, l) - base);
                            const float e1 = ex2(fmaf(__uint_as_float(x[j + 1]), kv, l) - base);
                            add = fmaf(e0 + e1, d.li[4 * h + j / 8], add);
                            const __half2 hh = __floats2half2_rn(e0, e1);
                            pk[j / 2] = *reinterpret_cast<const uint32_t *>(&hh);
                        }
                    }
                    sum += add;
                    // columns already read: 32 keys' weights take 16 of the 32 that their scores took
                    tc::st_32x32b_x16(ts + 16 * h, pk);
                }
                tc::ld_wait(xa);
                if (__builtin_expect(hn < 4, 0)) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = 0;
                    for (int h = hn; h < 4; ++h) tc::st_32x32b_x16(ts + 16 * h, pk);
                }
                any = true;
                tc::st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_pfull[t]);
            }
            const int32_t row0 = d.row0, head = d.head, r = d.r0 + 128 * t + row, rend = d.r0 + d.nrows, c0 = d.c0, c1 = d.c1;
            const bool live = 128 * t + row < d.nrows;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_tempty[i % kDescs]);
            if (!(f & kLast)) continue;

            // ---- the unit's end in this CTA ---------------------------------------------------
            if (any) {
                if (!wait_bar(&s_odone[t], od_par, abort, status)) break;
                od_par ^= 1;
                tc::fence_after_sync();
            }
            const bool whole = f & kWhole;
            float M = mx, L = sum, B = 0.f, o[32];
            // a part of a unit: m and l of each row, and O by fours of channels, rows side by side
            auto slot = [&](int32_t k) { return p.part + ((size_t)(2 * k + (k == c0 ? 1 : 0)) * 2 + t) * Sh::kPart; };
            auto own = [&](int h) {
                uint32_t y[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = 0;
                if (any) {                                     // uniform over the warp
                    tc::ld_32x32b_x32(to + 32 * h, y);
                    tc::ld_wait(y);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(y[j]);
            };
            auto release = [&]() {
                if (any) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_ofree[t]);
                }
            };
            if (!whole) {
                float *mine = slot((int32_t)blockIdx.x);
                __stcg(mine + row, mx);
                __stcg(mine + 128 + row, sum);
                if (any) {
#pragma unroll 1
                    for (int h = 0; h < D / 32; ++h) {
                        own(h);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            __stcg(reinterpret_cast<float4 *>(mine + 256) + (8 * h + j) * 128 + row,
                                   make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                    }
                }
                release();
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_join[t]);
                if (!wait_bar(&s_join[t], j_par, abort, status)) break;
                if (row == 0) {
                    __threadfence();
                    s_last[t] = arrive_last(p.joins.word + 2 * c0 + t, s_launch, c1 - c0 + 1);
                    __threadfence();
                    mbar_arrive(&s_said[t]);
                }
                if (!wait_bar(&s_said[t], j_par, abort, status)) break;
                j_par ^= 1;
                if (!s_last[t]) continue;
                M = -INFINITY;
                L = 0.f;
#pragma unroll 1
                for (int32_t k = c0; k <= c1; ++k) M = fmaxf(M, __ldcg(slot(k) + row));
                B = M == -INFINITY ? 0.f : M;
#pragma unroll 1
                for (int32_t k = c0; k <= c1; ++k) L += __ldcg(slot(k) + 128 + row) * ex2(__ldcg(slot(k) + row) - B);
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            // The rows' outputs, turned in shared memory 32 channels at a time so that four lanes
            // write 64 bytes of a row: this lane's rows, then, are (lane >> 2) + 8 j of the warp's.
            const uint32_t turn = stage_sm + warp * Sh::kStage;
            auto place = [&](int32_t rr) {
                const int32_t tk = div_group(a, rr);
                return (int64_t)(row0 + tk) * a.out_stride + ((int64_t)head * a.group + (rr - tk * a.group)) * D;
            };
            const int32_t rw = r - lane + (lane >> 2);
            int64_t at[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) at[j] = place(rw + 8 * j);
            __half2 probe = __float2half2_rn(0.f);             // the largest output that this lane writes, NaN if one is
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
                if (whole) {
                    own(h);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.f;
#pragma unroll 1
                    for (int32_t k = c0; k <= c1; ++k) {
                        const float *s = slot(k);
                        const float m = __ldcg(s + row);
                        if (m == -INFINITY) continue;          // nothing seen there: its O was not written
                        const float e = ex2(m - B);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + 256) + (8 * h + j) * 128 + row);
                            o[4 * j] = fmaf(v.x, e, o[4 * j]);
                            o[4 * j + 1] = fmaf(v.y, e, o[4 * j + 1]);
                            o[4 * j + 2] = fmaf(v.z, e, o[4 * j + 2]);
                            o[4 * j + 3] = fmaf(v.w, e, o[4 * j + 3]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2 hh = __floats2half2_rn(o[8 * j + 2 * k] * inv, o[8 * j + 2 * k + 1] * inv);
                        w[k] = *reinterpret_cast<const uint32_t *>(&hh);
                    }
                    sts128(turn + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4), w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int y = (lane >> 2) + 8 * j, c = lane & 3;
                    const uint4 v = lds128(turn + y * 64 + ((c ^ (y >> 1 & 3)) << 4));
                    if (FMT == SLORA_KV_E4M3) {
                        const __half2 *x = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
                        for (int k = 0; k < 4; ++k) probe = __hmax2_nan(probe, __habs2(x[k]));
                    }
                    if (rw + 8 * j < rend) *reinterpret_cast<uint4 *>(a.out + at[j] + 32 * h + 8 * c) = v;
                }
                __syncwarp();
            }
            if (whole) release();
            if (FMT == SLORA_KV_E4M3) {
                const float2 x = __half22float2(probe);
                if (__builtin_expect(__any_sync(~0u, !(x.x == x.x && x.y == x.y)), 0)) {
                    // (the row's outputs were written by other lanes, behind the loop's __syncwarp)
                    sum_again<D, FMT>(p, row0, head, r, rend, M == -INFINITY ? 0.f : M, live && M < INFINITY && L < INFINITY ? inv : -1.f, abort);
                    __syncwarp();
                }
            }
            if (live && a.lse) {
                const int32_t tok = div_group(a, r);
                a.lse[(int64_t)(row0 + tok) * a.n_q + (int64_t)head * a.group + (r - tok * a.group)] =
                    L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, int FMT>
cudaError_t launch(const PrefillParams &p, int num_sms, cudaStream_t stream)
{
    static std::mutex mu;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 64 || !set[dev]) {
            e = cudaFuncSetAttribute(attend_prefill_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)Shape<D>::kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) set[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<D>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_prefill_kernel<D, FMT>, p);
}

}  // namespace

size_t prefill_workspace_bytes(int num_sms)
{
    return (size_t)num_sms * 4 * Shape<128>::kPart * 4 + ((size_t)num_sms * 2 + 1) * 8;
}

cudaError_t launch_attend_prefill(const AttendArgs &a, int head_dim, int fmt, int32_t small_rows, void *ws, int num_sms,
                                  cudaStream_t stream, int *launches)
{
    PrefillParams p;
    p.a = a;
    p.small_rows = small_rows;
    p.box_rows = a.c.bt % 16 == 0 ? 16 : 8;
    p.min_tiles = 1 + kUnitCost;
    p.bt_inverse = (uint32_t)(((1ull << 32) + a.c.bt - 1) / a.c.bt);
    // unseen products are an infinity times this, so it may not be zero: at 2^-60 no score of fp16
    // queries and 8-bit codes differs from zero
    p.scale = a.scale_log2;
    if (p.scale < 0x1p-60f && p.scale > -0x1p-60f) p.scale = 0x1p-60f;
    p.unseen = p.scale < 0.f ? 0x7F800000u : 0xFF800000u;
    p.part = static_cast<float *>(ws);
    p.joins.started = reinterpret_cast<unsigned long long *>(p.part + (size_t)num_sms * 4 * Shape<128>::kPart);
    p.joins.word = p.joins.started + 1;
    cudaError_t e;
    if (head_dim == 128)
        e = fmt == SLORA_KV_E4M3 ? launch<128, SLORA_KV_E4M3>(p, num_sms, stream) : launch<128, SLORA_KV_INT8>(p, num_sms, stream);
    else
        e = fmt == SLORA_KV_E4M3 ? launch<64, SLORA_KV_E4M3>(p, num_sms, stream) : launch<64, SLORA_KV_INT8>(p, num_sms, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace kv
}  // namespace slora
