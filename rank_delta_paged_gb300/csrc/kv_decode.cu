// Attention over the 8-bit paged KV cache for few rows per KV head: single tokens, drafted
// tokens, and every row that has no larger tile to fill.
//
// For a row (new token t, query head j) with keys k_i = c_i 2^e, values v_i = d_i 2^f (codes
// c, d; exponents e, f of the key's pages):
//     s_i = q . c_i * 2^e * scale * log2(e)        m = max_i (s_i + f) - 7, or up to 8 less
//     w_i = 2^(s_i + f - m)                        out = sum_i w_i d_i / sum_i w_i 2^-f
// The exponent of the value page goes into the weight, so that values enter the product as
// plain codes, exact in fp16, and the weights of all pages share one scale; the sum of the
// softmax takes it out again in fp32.
//
// What bounds it: the codes of the keys and values, each read once per KV head for all of its
// group * n rows: 2 * head_dim bytes per token and head against a few hundred flops.  So the
// work is cut into tiles of 64 tokens of one (sequence, KV head, group of 8 or 16 rows), all
// tiles of the batch form one list, and every CTA takes an equal run of it: the memory system
// sees the same load from every SM whatever the lengths.  A unit whose tiles fall into several
// CTAs is joined by the last of them to finish, in the order of the list.
//
// Per CTA: one producer warp walks the list, writes a descriptor per tile (its unit, pages
// and scales) into shared memory some tiles ahead, since a page id and then the exponent of its
// page are two reads of a microsecond or two each under load, and copies the tiles into a ring by tensor
// maps, in boxes of 64 rows down to 16 (8), so a sequence's last page is not read past its last 16
// tokens; the copy engine's swizzle spreads the rows over the banks.  Four consumer warps take 16
// tokens of each tile.  Copies by the consumers' lanes (cp.async) reached 4.4 TB/s on long
// sequences, with the load path full.
// S^T = K Q^T and O^T = V^T P^T run on mma.sync m16n8k16, the tokens or the channels as the
// 16 rows and the query rows as the 8 columns: a single row wastes 7 columns of a product that
// is far from being the bound, and not 15 rows of registers.  The codes go to fp16 in registers,
// half an instruction (e4m3) to one and a quarter (int8) per code.
//
// With SINKS the keys between a sequence's first tokens and its window are left out of the numbering of its tiles
// (kv.h, key_shift), box by box of 16 (8) rows, so the sinks share the window's first tile.  256 single tokens over windows of
// 4096 and 64 sinks: 341 us, 6.1 TB/s, 90 % of a plain copy's rate (322 without the sinks); one over 1020 and 4: 12.9; 48
// sequences of 3 to 8 drafted tokens, 64 channels, over 1000 and 4: 42.5 us by three CTAs per SM, 45.6 by two (without the
// sinks, by two, 43).
//
// Measured: 512 single tokens over 30 to 1000 keys, 40 KV heads: 476 us, 5.7 TB/s; 4 over 60000 to 131000
// keys: 116 us, 5.5 TB/s; one over 700: 11.7 us, of which the launch and the chain of dependent reads (lengths,
// page id, exponent, codes, parts) is nearly all.  Short sequences are held up by their last tiles, which
// cost the consumers as much as full ones, by the join of a unit's four warps, and by SMs that memory
// serves a tenth slower than others; long ones by the start and the join of the parts.  The producer
// is as busy as the consumers: a copy issued by one lane of a branch cost 340 cycles, by an elected
// lane from values that are uniform over the warp half of that (520 to 485 us).
#include <cstddef>
#include <mutex>

#include "host_common.h"
#include "internal.h"
#include "kv.h"
#include "ptx.h"

namespace slora {
namespace kv {
namespace {

constexpr int kTile = 64;                       // tokens per tile
constexpr int kConsumers = 4;                   // warps, 16 tokens of a tile each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kMaxCtas = 3;                      // per SM, of any shape
// What a unit costs besides its tiles, in tiles: starting and joining its four warps' results.  By 0, 1,
// 2 and 3, in us with a cold cache: 512 single tokens over 30 to 1000 keys 549, 501, 502, 508; 24 sequences
// of 3 to 8 drafted tokens 131, 121, 111, 111; 384 single tokens beside 8 prompts 458, 423, 417, 423.
constexpr int kUnitCost = 2;
constexpr int kSeqChunks = 64;                  // partial sums of the tile counts
constexpr int kMaxRows = 16;
constexpr int kDescs = 32;                      // descriptors: 4 batches of 4 being prepared, 4 in use
constexpr int kPartStride = 2 * kMaxRows + kMaxRows * 128;   // floats of one partial result: m, l, O

template <class T>
__device__ __forceinline__ T uniform(T x)
{
    return __shfl_sync(~0u, x, 0);
}
__device__ __forceinline__ int4 uniform(int4 v)
{
    return make_int4(uniform(v.x), uniform(v.y), uniform(v.z), uniform(v.w));
}

struct Meta {
    float ks[8];       // 2^exponent of the key pages, per 8 tokens of the tile
    float lv[8];       // exponent of the value pages
    float li[8];       // 2^-exponent of the value pages
    int32_t plain;     // every token of the tile is seen by every row
    int32_t first, last;   // first / last tile of the unit within this CTA
    int32_t whole;     // the unit lies within this CTA
    int32_t j0;        // first token
    int32_t row0, n, len;  // the sequence
    int32_t head;      // KV head
    int32_t r0;        // first row (token * group + head within the group)
    int32_t c0, c1;    // first and last CTA of the unit
    uint32_t ok;       // bit g: tokens 8g .. 8g+7 of the tile are loaded
    int32_t pad[3];
    int32_t page[2][8];    // keys' and values' page of each box of 16 (8) rows
    int32_t row[8];        // and its first row there
};
static_assert(sizeof(Meta) % 16 == 0 && offsetof(Meta, plain) % 16 == 0, "Meta");

// CTAs per SM and stages of the ring.  Two groups of 8 rows of 64 channels by three CTAs and 5 stages instead of two and 7:
// 48 sequences of 3 to 8 drafted tokens over windows of 1000 with sinks 42.6 us instead of 45.6 (the parts of the plain kernel's
// results stay as they are).
template <int D, int NT, bool SINKS>
struct Shape {
    static constexpr bool kThree = NT == 1 || (SINKS && D == 64);
    static constexpr int kCtas = kThree ? 3 : 2;
    static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 4) : (NT == 1 ? 6 : kThree ? 5 : 7);
    static constexpr int kHalf = kTile * D;                  // bytes of a tile's keys
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kMergeFloats = kConsumers * 8 * NT * (D + 2);
    static constexpr size_t kSmem =
        1024 + (size_t)kStages * kStage + kDescs * sizeof(Meta) + kMergeFloats * 4;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int32_t c1, int32_t c2, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                 "%3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void lds128(uint32_t ad, uint32_t (&w)[4])
{
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(ad));
}

// Which token (of 8) is row m of an S^T tile.  The copy engine's swizzle moves 16-byte chunk
// c of row t to chunk c ^ (t & 7) (128-byte rows) or c ^ (t >> 1 & 3) (64-byte rows).  Both the
// reads of the keys (lanes 4m .. 4m+3 read chunks 0..3 of row m) and of the values (lane 4g + c
// reads chunk g of rows 2c and 2c+1) touch every bank once if rows 2i and 2i+1 differ in the
// half of the 128 bytes that their chunks 0..3 fall into and rows 0, 2, 4, 6 (1, 3, 5, 7)
// have four different pairs of chunks.
template <int D>
__device__ __forceinline__ int token_of_row(int m)
{
    if (D == 128) return m ^ ((m & 1) << 2);
    const int i = m >> 1;
    return ((i & 1) | (i & 2) << 1) ^ (m & 1 ? 3 : 0);
}

struct DecodeParams {
    AttendArgs a;
    int32_t box_rows;      // 16 if blocks are multiples of 16 tokens, else 8
    int32_t small_rows;
    int32_t rows;          // rows per unit: 8 * NT
    int32_t min_tiles;     // a CTA's run is at least this long: more than kUnitCost, or a run would have no tile and its warps wait
    uint32_t bt_inverse;   // ceil(2^32 / block tokens): a token's block, or one more
    float *part;           // [CTAs][2] partial results
    Joins joins;           // a word per CTA: the unit that starts there and goes on in others
};

// Tiles of sequence s: tiles per unit, units per KV head.  With sinks its length becomes one of the numbers that
// key_shift gives its keys.
template <bool SINKS>
__device__ __forceinline__ void seq_tiles(const DecodeParams &p, Seq &q, int32_t *tiles, int32_t *groups,
                                          int32_t *first, int32_t *shift)
{
    *tiles = 0;
    *groups = 0;
    *first = 0;
    *shift = 0;
    const int64_t rows = (int64_t)q.n * p.a.group;
    if (q.n == 0 || rows > p.small_rows) return;
    if (SINKS) {
        *shift = key_shift(p.a, first_key(p.a, q, 0), p.box_rows);
        q.len -= *shift;
    }
    const int32_t lo = SINKS ? 0 : first_key(p.a, q, 0) / kTile, hi = (end_key(p.a, q, q.n - 1) + kTile - 1) / kTile;
    *tiles = hi > lo ? hi - lo : 1;     // a row that sees nothing still writes zeros
    *groups = (int32_t)((rows + p.rows - 1) >> (p.rows == 8 ? 3 : 4));
    *first = lo;
}

template <int D, int NT, int FMT, bool SINKS>
__global__ void __launch_bounds__(kThreads, Shape<D, NT, SINKS>::kCtas)
attend_decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ PageMaps maps)
{
    using Sh = Shape<D, NT, SINKS>;
    constexpr int NS = Sh::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    Meta *meta = reinterpret_cast<Meta *>(ring + (size_t)NS * Sh::kStage);
    float *merge = reinterpret_cast<float *>(meta + kDescs);
    __shared__ uint64_t s_full[NS], s_empty[NS], s_merge[3];
    __shared__ int64_t s_sum[kSeqChunks];
    __shared__ int s_abort[2], s_last;
    __shared__ uint64_t s_launch;               // tid 0's
    __shared__ float s_row[2][kMaxRows];

    const AttendArgs &a = p.a;
    int32_t *status = a.c.status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kConsumers);
        }
        mbar_init(&s_merge[0], kConsumers);
        mbar_init(&s_merge[1], kConsumers);
        mbar_init(&s_merge[2], 1);
        fence_mbar_init();
        s_abort[0] = 0;
        s_abort[1] = work_clock(global_timer_ns());
    }
    griddep_wait();
    griddep_launch_dependents();
    uint64_t started = 0;
    if (tid == 0) {
        started = start_launch(p.joins, blockIdx.x == 0, gridDim.x);
        if ((int32_t)blockIdx.x == a.give_up) {
            set_status(status, SLORA_DEV_TIMEOUT);
            s_abort[0] = 1;
        }
    }

    // Tiles of each run of `per` sequences; every CTA sums them for itself, which costs less
    // than a launch.
    const int S = a.b.S;
    const int per = ((S + kSeqChunks - 1) / kSeqChunks + 31) / 32 * 32;
    const int chunks = (S + per - 1) / per;
    if (tid >= chunks && tid < kSeqChunks) s_sum[tid] = 0;
    int32_t bad = 0;
#pragma unroll 1
    for (int c = warp; c < chunks; c += kThreads / 32) {
        int64_t t = 0;
#pragma unroll 1
        for (int64_t s = (int64_t)c * per + lane; s < S && s < (int64_t)(c + 1) * per; s += 32) {
            int32_t tiles, groups, first, shift;
            Seq q = load_seq(a, (int32_t)s, &bad);
            seq_tiles<SINKS>(p, q, &tiles, &groups, &first, &shift);
            t += (int64_t)(tiles + kUnitCost) * groups;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
        if (lane == 0) s_sum[c] = t * a.c.n_kv;
    }
    if (bad && blockIdx.x == 0) set_status(status, bad);
    __syncthreads();
    // This CTA's run [w0, w1) of the list's W places: a unit's tiles, then kUnitCost empty ones.
    int64_t v0 = s_sum[2 * lane], v1 = s_sum[2 * lane + 1], W = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(~0u, W, o);
        if (lane >= o) W += u;
    }
    const int64_t before = W - v0 - v1;          // tiles before chunk 2 * lane
    W = __shfl_sync(~0u, W, 31);
    int64_t run = div_list(W + gridDim.x - 1, gridDim.x);
    if (run < p.min_tiles) run = p.min_tiles;
    const int64_t w0 = (int64_t)blockIdx.x * run, w1 = w0 + run < W ? w0 + run : W;
    if (w0 >= W - kUnitCost) return;
    volatile int *abort = s_abort;
    const int R = p.box_rows;                  // rows of a tile that share a page
    const int batch_log = R == 16 ? 2 : 1;     // tiles per batch of descriptors
    const int n_batches = kDescs >> batch_log;

    if (warp == kConsumers) {
        // ---- producer ------------------------------------------------------------------
        // the sequence that holds tile w0: its chunk, then 32 sequences at a time
        const bool leader = elect_one();
        const unsigned hit = __ballot_sync(~0u, before <= w0);
        const int at = 31 - __clz(hit);
        int chunk = 2 * at;
        int64_t base = __shfl_sync(~0u, before, at);
        const int64_t half = __shfl_sync(~0u, v0, at);
        if (base + half <= w0) {
            base += half;
            ++chunk;
        }
        int32_t s32 = chunk * per;               // first of the 32 sequences that the lanes hold
        Seq q;
        int32_t tiles, groups, first, shift;
        auto hold = [&](int32_t s) {
            q.n = 0;
            tiles = groups = first = shift = 0;
            int32_t ignore;
            if (s + lane < S) {
                q = load_seq(a, s + lane, &ignore);
                seq_tiles<SINKS>(p, q, &tiles, &groups, &first, &shift);
            }
        };
        int at_lane = 0;
#pragma unroll 1
        for (;; s32 += 32) {
            hold(s32);
            if (s32 >= S) {       // the lengths changed under the call: nothing to copy
                if (lane == 0) {
                    set_status(status, SLORA_DEV_BAD_LENGTH);
                    s_abort[0] = 1;
                }
                return;
            }
            int64_t mine = (int64_t)(tiles + kUnitCost) * groups * a.c.n_kv, sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += u;
            }
            const unsigned past = __ballot_sync(~0u, base + sum > w0);
            if (past) {
                at_lane = __ffs(past) - 1;
                base += __shfl_sync(~0u, sum - mine, at_lane);
                break;
            }
            base += __shfl_sync(~0u, sum, 31);
        }
        // position in the list: sequence, KV head, row group, tile
        int32_t u_tiles = __shfl_sync(~0u, tiles, at_lane), u_groups = __shfl_sync(~0u, groups, at_lane);
        int32_t u_first = __shfl_sync(~0u, first, at_lane), u_shift = SINKS ? __shfl_sync(~0u, shift, at_lane) : 0;
        int64_t in_seq = w0 - base;
        int32_t head = div_list(in_seq, (int64_t)(u_tiles + kUnitCost) * u_groups);
        in_seq -= (int64_t)head * (u_tiles + kUnitCost) * u_groups;
        int32_t grp = div_list(in_seq, u_tiles + kUnitCost), tile = (int32_t)(in_seq - (int64_t)grp * (u_tiles + kUnitCost));
        Seq u;
        u.row0 = __shfl_sync(~0u, q.row0, at_lane);
        u.n = __shfl_sync(~0u, q.n, at_lane);
        u.len = __shfl_sync(~0u, q.len, at_lane);

        // What the tiles of a unit share, worked out when the list enters it.
        struct Unit {
            int32_t r0, whole, c0, c1;
            int32_t lo, hi;                    // keys that any of its sequence's rows sees
            int32_t plain_lo, plain_hi;        // keys that all of its rows see
            const int32_t *table;              // entry (block 0, its head, keys)
        } un;
        auto enter = [&](int64_t w) {          // w: the unit's tile `tile` in the list
            const int64_t u0 = w - tile, u1 = u0 + u_tiles;
            un.whole = u0 >= w0 && u1 <= w1;
            un.c0 = un.c1 = 0;
            if (!un.whole) {
                un.c0 = div_list(u0, run);
                un.c1 = div_list(u1 - 1, run);
            }
            un.r0 = grp * p.rows;
            const int32_t rows = u.n * a.group, r1 = un.r0 + p.rows < rows ? un.r0 + p.rows : rows;
            un.lo = first_key(a, u, 0);
            un.hi = end_key(a, u, u.n - 1);
            un.plain_lo = un.lo;
            un.plain_hi = un.hi;
            if (u.n > 1) {
                un.plain_lo = first_key(a, u, div_group(a, r1 - 1));
                un.plain_hi = end_key(a, u, div_group(a, un.r0));
            }
            if (SINKS && un.plain_lo <= a.sinks) un.plain_lo = 0;
            un.table = a.b.table + ((int64_t)(s32 + at_lane) * a.b.max_blocks * a.c.n_kv + head) * 2;
        };
        bool fresh = true;              // the unit has yet to be entered

        // A batch of tiles at a time, `lanes` lanes each, one lane per box (R rows of keys or
        // values): their page ids and their exponents are read together, one batch ahead.
        const int boxes = kTile / R, lanes = 2 * boxes, per_batch = 32 / lanes;
        const int my_tile = lane / lanes, gl = (lane % lanes) >> 1, kvl = lane & 1;
        const int32_t table_step = a.c.n_kv * 2;
        struct Box {
            bool want;                  // whether any row of the sequence needs it
            int32_t page, row;          // its page and first row there
            int32_t e;                  // and its exponent
        };
        int64_t ahead = w0;             // place of `tile` in the list, the first not yet described
        bool begun = false;
        // Batch of descriptors that the next call fills.  It was last used by the batch 8 (16 for
        // R = 8) earlier, 4 (12) batches before the last one copied, whose tiles the consumers
        // have left: the last copy waited for the tile NS before it.
        int slot = 0;
        // The tiles of the next batch: everything but pages and scales goes to the ring at once.
        auto describe = [&](Box &m) {
            m.want = false;
            m.page = 0;
            m.row = 0;
            Meta *ms = &meta[(slot << batch_log) + my_tile];
            // this lane's tile is t of the unit, at `at` in the list
            auto fill = [&](int32_t t, int64_t at, bool first) {
                const int32_t j0 = (u_first + t) * kTile, j = j0 + gl * R;
                m.want = j < un.hi && (j + R > un.lo || (SINKS && j < a.sinks));
                if (m.want) {
                    const int32_t key = SINKS && j >= sinks_end(a, R) ? j + u_shift : j;
                    int32_t blk = (int32_t)__umulhi((uint32_t)key, p.bt_inverse);
                    m.row = key - blk * a.c.bt;
                    if (m.row < 0) {
                        --blk;
                        m.row += a.c.bt;
                    }
                    m.page = __ldg(un.table + (int64_t)blk * table_step + kvl);
                }
                if (lane % lanes == 0) {
                    int4 *mi = reinterpret_cast<int4 *>(&ms->plain);
                    const bool end = t == u_tiles - 1, last = end || at == w1 - 1;
                    const bool run_end = at + 1 + (end ? kUnitCost : 0) >= w1;
                    mi[0] = make_int4((j0 >= un.plain_lo || (SINKS && j0 + kTile <= a.sinks)) && j0 + kTile <= un.plain_hi,
                                      first || t == 0,
                                      (last ? 1 : 0) | (run_end ? 2 : 0), un.whole);
                    mi[1] = make_int4(j0, u.row0, u.n, u.len);
                    mi[2] = make_int4(head, un.r0, un.c0, un.c1);
                }
            };
            int count = 0;
            do {                        // the part of the batch that lies in one unit
                if (tile >= u_tiles) {
                    // the next unit
                    ahead += u_tiles + kUnitCost - tile;
                    if (ahead >= w1) break;
                    if (++grp == u_groups) {
                        grp = 0;
                        if (++head == a.c.n_kv) {
                            head = 0;
                            unsigned next;
#pragma unroll 1
                            while ((next = __ballot_sync(~0u, tiles > 0 && lane > at_lane)) == 0 && s32 + 32 < S) {
                                s32 += 32;
                                at_lane = -1;
                                hold(s32);
                            }
                            if (next == 0) {      // the lengths changed under the call
                                if (lane == 0) set_status(status, SLORA_DEV_BAD_LENGTH);
                                ahead = w1;
                                break;
                            }
                            at_lane = __ffs(next) - 1;
                            u_tiles = __shfl_sync(~0u, tiles, at_lane);
                            u_groups = __shfl_sync(~0u, groups, at_lane);
                            u_first = __shfl_sync(~0u, first, at_lane);
                            if (SINKS) u_shift = __shfl_sync(~0u, shift, at_lane);
                            u.row0 = __shfl_sync(~0u, q.row0, at_lane);
                            u.n = __shfl_sync(~0u, q.n, at_lane);
                            u.len = __shfl_sync(~0u, q.len, at_lane);
                        }
                    }
                    tile = 0;
                    fresh = true;
                }
                if (ahead >= w1) break;
                if (fresh) {
                    enter(ahead);
                    fresh = false;
                }
                int32_t n = per_batch - count < u_tiles - tile ? per_batch - count : u_tiles - tile;
                if (w1 - ahead < n) n = (int32_t)(w1 - ahead);
                const int32_t t = my_tile - count;
                if (t >= 0 && t < n) fill(tile + t, ahead + t, !begun && my_tile == 0);
                tile += n;
                ahead += n;
                count += n;
            } while (count < per_batch);
            if (count == 0) return 0;
            begun = true;
            if (++slot == n_batches) slot = 0;
            return count;
        };
        // The batch's page ids are there: into the descriptors with them, and on to the exponents.
        auto settle = [&](Box &m, int n, int at) {
            if (m.want && (m.page < 0 || m.page >= a.c.num_pages)) {
                set_status(status, SLORA_DEV_BAD_PAGE);
                m.want = false;
            }
            // a box needs both its keys and its values: bits 2 gl of `have`
            unsigned have = __ballot_sync(~0u, m.want);
            have &= have >> 1 & 0x55555555u;
            if (lanes < 32) have = have >> (my_tile * lanes) & ((1u << lanes) - 1u);
            m.want = have >> (2 * gl) & 1u;
            m.e = m.want ? (int32_t)a.c.exps[m.page] : 0;
            // bits 2 g spread over the 8-token groups of Meta.ok
            uint32_t ok;
            if (R == 16)
                ok = (have & 1u) * 3u | (have >> 2 & 1u) * 12u | (have >> 4 & 1u) * 48u | (have >> 6 & 1u) * 192u;
            else
                ok = (have & 1u) | (have >> 1 & 2u) | (have >> 2 & 4u) | (have >> 3 & 8u) | (have >> 4 & 16u) |
                     (have >> 5 & 32u) | (have >> 6 & 64u) | (have >> 7 & 128u);
            if (my_tile < n) {
                Meta *ms = &meta[(at << batch_log) + my_tile];
                ms->page[kvl][gl] = m.page;
                if (kvl == 0) ms->row[gl] = m.row;
                if (lane % lanes == 0) {
                    ms->ok = ok;
                    if (ok != 0xFFu) ms->plain = 0;
                }
            }
            __syncwarp();
        };
        // The copies of a tile.  The whole warp goes through it by values that are the same in every lane, and one
        // elected lane issues: a lane's own values would be turned into uniform ones for every copy.
        auto copy_tile = [&](const Meta &m, int st, bool arrive, bool issue) {
            const uint32_t ok = uniform(m.ok), dst = uniform(smem_u32(ring) + st * Sh::kStage);
            uint64_t *bar = &s_full[st];
            if (arrive && leader) mbar_arrive_expect_tx(bar, (uint32_t)__popc(ok) * 16u * D);
            if (!issue) return;
            auto copy = [&](int box, int level, int32_t row, int32_t kp, int32_t vp) {    // R << level rows
                if (leader) {
                    tma_load_3d(dst + box * R * D, &maps.m[level], row, kp, bar);
                    tma_load_3d(dst + box * R * D + Sh::kHalf, &maps.m[level], row, vp, bar);
                }
            };
            if (R == 16) {
                // the tile's four boxes as one, as two halves, or one by one: a box can be
                // joined to the one before unless it starts a page
                const int4 row = uniform(*reinterpret_cast<const int4 *>(m.row));
                const int4 kp = uniform(*reinterpret_cast<const int4 *>(m.page[0]));
                const int4 vp = uniform(*reinterpret_cast<const int4 *>(m.page[1]));
                // (with sinks: unless it does not follow it there)
                auto joined = [&](int32_t r0, int32_t r1, int32_t k0, int32_t k1, int32_t v0, int32_t v1) {
                    return SINKS ? r1 == r0 + 16 && k1 == k0 && v1 == v0 : r1 != 0;
                };
                const bool xy = joined(row.x, row.y, kp.x, kp.y, vp.x, vp.y), zw = joined(row.z, row.w, kp.z, kp.w, vp.z, vp.w);
                if (ok == 0xFFu && xy && zw && joined(row.y, row.z, kp.y, kp.z, vp.y, vp.z)) {
                    copy(0, 2, row.x, kp.x, vp.x);
                } else {
                    if ((ok & 15u) == 15u && xy) {
                        copy(0, 1, row.x, kp.x, vp.x);
                    } else {
                        if (ok & 1u) copy(0, 0, row.x, kp.x, vp.x);
                        if (ok & 4u) copy(1, 0, row.y, kp.y, vp.y);
                    }
                    if ((ok & 0xF0u) == 0xF0u && zw) {
                        copy(2, 1, row.z, kp.z, vp.z);
                    } else {
                        if (ok & 16u) copy(2, 0, row.z, kp.z, vp.z);
                        if (ok & 64u) copy(3, 0, row.w, kp.w, vp.w);
                    }
                }
            } else {
#pragma unroll 1
                for (int x = 0; x < 8; ++x)
                    if (ok >> x & 1u) copy(x, 0, uniform(m.row[x]), uniform(m.page[0][x]), uniform(m.page[1][x]));
            }
        };
        // Two batches lie between the reading of a batch's page ids and of its exponents, and one more
        // between those and their use: under load either read takes a microsecond or two.  The first
        // tiles' copies start as soon as their pages are known, and the first batch waits for nothing else.
        const Box none = {false, 0, 0, 0};
        Box b0 = none, b1 = none, b2 = none, b3;
        int n0 = 0, n1 = 0, n2 = 0, n3;
        int batch = 0, stage = 0;
        uint32_t parity = 1;
        int32_t issued = 0;
        int early = 0;
#pragma unroll 1
        for (int step = 0;; ++step, b0 = b1, b1 = b2, b2 = b3, n0 = n1, n1 = n2, n2 = n3) {
            n3 = describe(b3);
            if (step == 0) {
                settle(b3, n3, 0);
                early = n3 < NS ? n3 : NS;
#pragma unroll 1
                for (int t = 0; t < early; ++t) copy_tile(meta[t], t, false, true);
            }
            if (step < 3) continue;
            if (n0 == 0 || *abort) break;
            if (step > 3) settle(b1, n1, (step - 2) % n_batches);
            if (my_tile < n0) {
                const int e = b0.want ? clamp_exponent(b0.e) : 0;
                const float ef = (float)e, up = pow2(e), down = pow2(-e);
                Meta *ms = &meta[(batch << batch_log) + my_tile];
                if (R == 16) {
                    if (kvl == 0) {
                        *reinterpret_cast<float2 *>(&ms->ks[2 * gl]) = make_float2(up, up);
                    } else {
                        *reinterpret_cast<float2 *>(&ms->lv[2 * gl]) = make_float2(ef, ef);
                        *reinterpret_cast<float2 *>(&ms->li[2 * gl]) = make_float2(down, down);
                    }
                } else {
                    if (kvl == 0) {
                        ms->ks[gl] = up;
                    } else {
                        ms->lv[gl] = ef;
                        ms->li[gl] = down;
                    }
                }
            }
            __syncwarp();
#pragma unroll 1
            for (int t = 0; t < n0; ++t, ++issued) {
                if (!wait_bar(&s_empty[stage], parity, abort, status)) break;
                copy_tile(meta[(batch << batch_log) + t], stage, true, issued >= early);
                if (++stage == NS) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if (++batch == n_batches) batch = 0;
            if (step == 3) settle(b1, n1, 1);
        }
        // No copy outlives the CTA: wait for the last ones, whatever the consumers do.  If the CTA gave up,
        // some of the early ones may not have been handed on yet, and their barriers know nothing of them.
#pragma unroll 1
        for (int t = issued; t < early; ++t)
            if (leader) mbar_arrive_expect_tx(&s_full[t], (uint32_t)__popc(meta[t].ok) * 16u * D);
        const int32_t copied = issued > early ? issued : early;
        volatile int gone[2] = {0, abort[1]};
#pragma unroll 1
        for (int i = 0; i < NS && i < copied && !gone[0]; ++i) {
            const int t = copied - 1 - i;
            wait_bar(&s_full[t % NS], (uint32_t)(t / NS & 1), gone, status);
        }
        return;
    }

    // ---- consumers ---------------------------------------------------------------------
    if (tid == 0) s_launch = started;
    const int g = lane >> 2, c = lane & 3;
    const int krow[2] = {token_of_row<D>(g), token_of_row<D>(g) + 8};
    // the tokens of this lane's two rows of V^T P^T's inner index, in both halves of the 16
    const int vrow[4] = {token_of_row<D>(2 * c), token_of_row<D>(2 * c + 1), token_of_row<D>(2 * c) + 8,
                         token_of_row<D>(2 * c + 1) + 8};
    constexpr int KS = D / 16;          // k steps of S^T, and 16-row tiles of O^T
    float o[NT][KS][4], mx[NT][2], sum[NT][2];
    uint32_t qf[NT][KS][2];
    const uint32_t my_ring = smem_u32(ring) + warp * 16 * D;
    int stage = 0;
    uint32_t parity = 0, mparity[2] = {0, 0}, jparity = 0, toggle = 0;
    bool pending = false;      // the last unit's reads of the merge buffer may still be under way
    auto meet = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_merge[k]);
        const bool fine = wait_bar(&s_merge[k], mparity[k], abort, status);
        mparity[k] ^= 1;
        return fine;
    };

    // This lane's share of the rows of m's unit: k step i holds channels 4 (i & 3) .. + 3 of
    // chunk c + 4 (i >> 2).
    auto load_q = [&](const Meta &m) {
        const int32_t nrows = m.n * a.group - m.r0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = 8 * t + g;
            const bool live = r < nrows;
            const int tok = div_group(a, m.r0 + r), hd = (m.r0 + r) - tok * a.group;
            const __half *src = a.q + (int64_t)(m.row0 + tok) * a.q_stride + ((int64_t)m.head * a.group + hd) * D;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                uint2 v = make_uint2(0, 0);
                if (live) v = __ldg(reinterpret_cast<const uint2 *>(src + (c + 4 * (i >> 2)) * 16 + 4 * (i & 3)));
                qf[t][i][0] = v.x;
                qf[t][i][1] = v.y;
            }
        }
    };
    bool more = true;
    for (int32_t it = 0; more; ++it) {
        if (!wait_bar(&s_full[stage], parity, abort, status)) break;
        const Meta &m = meta[it % kDescs];
        const int4 flags = *reinterpret_cast<const int4 *>(&m.plain);
        const bool plain = flags.x != 0, last = flags.z & 1, whole = flags.w != 0;
        more = (flags.z & 2) == 0;
        const uint32_t kbase = my_ring + stage * Sh::kStage;
        const uint32_t vbase = kbase + Sh::kHalf;
        const int32_t nrows = m.n * a.group - m.r0;       // rows of this unit
        if (flags.y) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mx[t][0] = mx[t][1] = -INFINITY;
                sum[t][0] = sum[t][1] = 0.f;
#pragma unroll
                for (int i = 0; i < KS; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
            }
            if (it == 0) load_q(m);
        }
        // S^T: this warp's 16 tokens x the rows
        float sc[NT][4], sd[NT][4];       // two chains of products, so that one hides the other's latency
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[t][x] = sd[t][x] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            uint32_t kw[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int tok = krow[x];
                lds128(kbase + tok * D + (D == 128 ? (c + 4 * h) ^ (tok & 7) : c ^ (tok >> 1 & 3)) * 16, kw[x]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a0, a1, a2, a3;
                decode4<FMT>(kw[0][j], a0, a2);
                decode4<FMT>(kw[1][j], a1, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    mma16816(j & 1 ? sd[t] : sc[t], a0, a1, a2, a3, qf[t][4 * h + j][0], qf[t][4 * h + j][1]);
            }
        }
        // the values' codes, while the scores are worked on
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int tok = vrow[x];
            if constexpr (D == 128) {
                lds128(vbase + tok * D + (g ^ (tok & 7)) * 16, vw[x]);
            } else {
                const uint32_t ad = vbase + tok * D + ((g >> 1) ^ (tok >> 1 & 3)) * 16 + (g & 1) * 8;
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(vw[x][0]), "=r"(vw[x][1]) : "r"(ad));
            }
        }
        // the next unit's rows, while this one's last tile is finished
        if (last && more) {
            const bool wrap = stage + 1 == NS;
            if (!wait_bar(&s_full[wrap ? 0 : stage + 1], parity ^ (wrap ? 1u : 0u), abort, status)) break;
            load_q(meta[(it + 1) % kDescs]);
        }
        const float f0 = m.ks[2 * warp] * a.scale_log2, f1 = m.ks[2 * warp + 1] * a.scale_log2;
        const float lv0 = m.lv[2 * warp], lv1 = m.lv[2 * warp + 1];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sc[t][0] = fmaf(sc[t][0] + sd[t][0], f0, lv0);
            sc[t][1] = fmaf(sc[t][1] + sd[t][1], f0, lv0);
            sc[t][2] = fmaf(sc[t][2] + sd[t][2], f1, lv1);
            sc[t][3] = fmaf(sc[t][3] + sd[t][3], f1, lv1);
        }
        if (!plain) {
            Seq q;
            q.row0 = m.row0;
            q.n = m.n;
            q.len = m.len;
            const bool ok0 = m.ok >> (2 * warp) & 1, ok1 = m.ok >> (2 * warp + 1) & 1;
            const int j0 = m.j0 + warp * 16 + krow[0], j1 = j0 + 8;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 8 * t + 2 * c + x;
                    const int tok = div_group(a, m.r0 + (r < nrows ? r : 0));
                    const int lo = first_key(a, q, tok), hi = end_key(a, q, tok);
                    if (!(ok0 && (j0 >= lo || (SINKS && j0 < a.sinks)) && j0 < hi)) sc[t][x] = -INFINITY;
                    if (!(ok1 && (j1 >= lo || (SINKS && j1 < a.sinks)) && j1 < hi)) sc[t][2 + x] = -INFINITY;
                }
        }
        // A row's reference is taken up only when a score passes it by kMaxWeight (the first one always
        // does), so the rescaling of O is rare.  The difference of the two is exact where it decides.
        bool up = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                up |= fmaxf(sc[t][x], sc[t][2 + x]) - mx[t][x] > kMaxWeight;
        if (__any_sync(~0u, up)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = fmaxf(sc[t][x], sc[t][2 + x]);
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
                    v = fmaxf(v - kHeadRoom, mx[t][x]);
                    const float k = mx[t][x] == -INFINITY ? 0.f : ex2(mx[t][x] - v);
                    mx[t][x] = v;
                    sum[t][x] *= k;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[t][i][x] *= k;
                        o[t][i][2 + x] *= k;
                    }
                }
        }
        uint32_t pf[NT][2];
        const float li0 = m.li[2 * warp], li1 = m.li[2 * warp + 1];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float b0 = mx[t][0] == -INFINITY ? 0.f : mx[t][0], b1 = mx[t][1] == -INFINITY ? 0.f : mx[t][1];
            const float p0 = ex2(sc[t][0] - b0), p1 = ex2(sc[t][1] - b1);
            const float p2 = ex2(sc[t][2] - b0), p3 = ex2(sc[t][3] - b1);
            sum[t][0] += p0 * li0 + p2 * li1;
            sum[t][1] += p1 * li0 + p3 * li1;
            __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
            pf[t][0] = transpose8x8(*reinterpret_cast<uint32_t *>(&h0));
            pf[t][1] = transpose8x8(*reinterpret_cast<uint32_t *>(&h1));
        }
        // O^T += V^T P^T
        if (!plain) {
            // weights of unseen tokens are zero, but what lies in their place may be NaN
            const Seq q = {m.row0, m.n, m.len};
            const int lo = first_key(a, q, 0), hi = end_key(a, q, m.n - 1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = m.j0 + warp * 16 + vrow[x];
                const bool ok = (m.ok >> (2 * warp + (x >> 1)) & 1) && (j >= lo || (SINKS && j < a.sinks)) && j < hi;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) vw[x][i] = ok ? vw[x][i] : 0u;
            }
            if (FMT == SLORA_KV_E4M3 && m.n > 1) {
                // A NaN reaches the rows that see its token, and by the product, as 0 times NaN, the others too:
                // it is taken out of that and put into those rows' sums.
                uint32_t odd = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) odd |= nan_bytes(vw[x][i]);
                if (__builtin_expect(__any_sync(~0u, odd != 0), 0)) {
                    uint64_t mine = 0;       // 16 bits per token x: its channels of this lane's D / 8
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            const uint32_t b = nan_bytes(vw[x][i]) >> 7;
                            vw[x][i] &= ~(b * 0xFFu);
                            mine |= (uint64_t)((b * 0x10204080u) >> 28) << (16 * x + 4 * i);
                        }
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {
                        const uint32_t set = (uint32_t)(__shfl_sync(~0u, mine, (lane & ~3) + (k >> 2)) >> (16 * (k & 3))) & 0xFFFFu;
                        const int j = m.j0 + warp * 16 + token_of_row<D>(2 * (k >> 2) + (k & 1)) + 8 * (k >> 1 & 1);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int r = 8 * t + 2 * c + x;
                                const int tok = div_group(a, m.r0 + (r < nrows ? r : 0));
                                const uint32_t see = (j >= first_key(a, q, tok) || (SINKS && j < a.sinks)) && j < end_key(a, q, tok) ? set : 0u;
#pragma unroll
                                for (int h = 0; h < D / 8; ++h)
                                    if (see >> h & 1u) o[t][h >> 1][x + 2 * (h & 1)] = __int_as_float(0x7FFFFFFF);
                            }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint32_t a0[2], a1[2], a2[2], a3[2];
            // channels 4i, 4i+1 then 4i+2, 4i+3 of this lane's run, token pairs in one register
            decode4<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x5140), a0[0], a1[0]);
            decode4<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x7362), a0[1], a1[1]);
            decode4<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x5140), a2[0], a3[0]);
            decode4<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x7362), a2[1], a3[1]);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    mma16816(o[t][2 * i + y], a0[y], a1[y], a2[y], a3[y], pf[t][0], pf[t][1]);
        }
        const int32_t row0 = m.row0, head = m.head, r0 = m.r0, c0 = m.c0, c1 = m.c1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[stage]);
        if (++stage == NS) {
            stage = 0;
            parity ^= 1;
        }
        if (!last) continue;

        // ---- the unit's end: the four warps' results become one --------------------------
        const int live = nrows < 8 * NT ? nrows : 8 * NT;
        // with few rows the units take turns at the buffer's halves, and a unit's writes need not
        // wait for the reads of the one before
        const bool halves = live <= 4 * NT;
        toggle ^= 1;
        if (!halves && pending && !meet(1)) break;
        pending = whole && halves;
        const int mr = halves ? 4 * NT : 8 * NT;        // rows per warp
        float *mm = merge + (halves && toggle ? kConsumers * 4 * NT * (D + 2) : 0);
        float *ml = mm + kConsumers * mr, *mo = ml + kConsumers * mr;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = sum[t][x];
                l += __shfl_xor_sync(~0u, l, 4);
                l += __shfl_xor_sync(~0u, l, 8);
                l += __shfl_xor_sync(~0u, l, 16);
                const int r = 8 * t + 2 * c + x;
                if (r < live) {
                    if (g == 0) {
                        mm[warp * mr + r] = mx[t][x];
                        ml[warp * mr + r] = l;
                    }
                    // accumulators x, 2 + x: channels 2i, 2i + 1 of this lane's D / 8
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        *reinterpret_cast<float2 *>(&mo[(warp * mr + r) * D + g * (D / 8) + 2 * i]) =
                            make_float2(o[t][i][x], o[t][i][2 + x]);
                }
            }
        if (!meet(0)) break;
        float *part = p.part + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == c0 ? 1 : 0)) * kPartStride;
        auto emit = [&](int r, int d, float2 v, float M, float L) {
            const int tok = div_group(a, r0 + r), hd = (r0 + r) - tok * a.group;
            const int64_t qh = (int64_t)head * a.group + hd;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            __half2 h = __floats2half2_rn(v.x * inv, v.y * inv);
            *reinterpret_cast<__half2 *>(a.out + (int64_t)(row0 + tok) * a.out_stride + qh * D + d) = h;
            if (a.lse && d == 0)
                a.lse[(int64_t)(row0 + tok) * a.n_q + qh] =
                    L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        };
#pragma unroll 1
        for (int i = tid; i < live * (D / 2); i += 32 * kConsumers) {
            const int r = i / (D / 2), d = (i - r * (D / 2)) * 2;
            float M = -INFINITY;
#pragma unroll
            for (int k = 0; k < kConsumers; ++k) M = fmaxf(M, mm[k * mr + r]);
            const float B = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kConsumers; ++k) {
                const float e = ex2(mm[k * mr + r] - B);
                const float2 x = *reinterpret_cast<const float2 *>(&mo[(k * mr + r) * D + d]);
                L += ml[k * mr + r] * e;
                v.x = fmaf(x.x, e, v.x);
                v.y = fmaf(x.y, e, v.y);
            }
            if (whole) {
                emit(r, d, v, M, L);
            } else {
                __stcg(reinterpret_cast<float2 *>(part + 2 * kMaxRows + r * D + d), v);
                if (d == 0) {
                    __stcg(part + r, M);
                    __stcg(part + kMaxRows + r, L);
                }
            }
        }
        if (pending) continue;
        if (!whole) {
            // the last CTA of the unit to arrive joins the parts in the order of the list
            __threadfence();
            if (!meet(1)) break;
            if (tid == 0) {
                __threadfence();
                s_last = arrive_last(p.joins.word + c0, s_launch, c1 - c0 + 1);
                __threadfence();
                mbar_arrive(&s_merge[2]);
            }
            if (!wait_bar(&s_merge[2], jparity, abort, status)) break;
            jparity ^= 1;
            if (s_last) {
                auto slot = [&](int k) { return p.part + (size_t)(2 * k + (k == c0 ? 1 : 0)) * kPartStride; };
                // each row's maximum and sum by eight lanes
                const int r8 = tid >> 3, j8 = tid & 7;
                float M = -INFINITY, L = 0.f;
                if (r8 < live)
#pragma unroll 4
                    for (int k = c0 + j8; k <= c1; k += 8) M = fmaxf(M, __ldcg(slot(k) + r8));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
                const float B = M == -INFINITY ? 0.f : M;
                if (r8 < live)
#pragma unroll 4
                    for (int k = c0 + j8; k <= c1; k += 8)
                        L = fmaf(__ldcg(slot(k) + kMaxRows + r8), ex2(__ldcg(slot(k) + r8) - B), L);
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) L += __shfl_xor_sync(~0u, L, o);
                if (j8 == 0) {
                    s_row[0][r8] = M;
                    s_row[1][r8] = L;
                }
                if (!meet(1)) break;
#pragma unroll 1
                for (int i = tid; i < live * (D / 4); i += 32 * kConsumers) {
                    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
                    const float Mr = s_row[0][r], Lr = s_row[1][r], Br = Mr == -INFINITY ? 0.f : Mr;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) {
                        const float *sl = slot(k);
                        const float e = ex2(__ldcg(sl + r) - Br);
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(sl + 2 * kMaxRows + r * D + d));
                        v.x = fmaf(x.x, e, v.x);
                        v.y = fmaf(x.y, e, v.y);
                        v.z = fmaf(x.z, e, v.z);
                        v.w = fmaf(x.w, e, v.w);
                    }
                    emit(r, d, make_float2(v.x, v.y), Mr, Lr);
                    emit(r, d + 2, make_float2(v.z, v.w), Mr, Lr);
                }
            }
        } else if (!meet(1)) {
            break;
        }
    }
}

template <int D, int NT, int FMT, bool SINKS>
cudaError_t launch(const DecodeParams &p, const PageMaps &maps, int num_sms, cudaStream_t stream)
{
    static std::mutex mu;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 64 || !set[dev]) {
            e = cudaFuncSetAttribute(attend_decode_kernel<D, NT, FMT, SINKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)Shape<D, NT, SINKS>::kSmem);
            if (e != cudaSuccess) return e;
            if (dev < 64) set[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * Shape<D, NT, SINKS>::kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<D, NT, SINKS>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_decode_kernel<D, NT, FMT, SINKS>, p, maps);
}

template <int D, bool SINKS>
cudaError_t launch_d(const DecodeParams &p, const PageMaps &maps, int fmt, int num_sms, cudaStream_t stream)
{
    if (p.rows == 8)
        return fmt == SLORA_KV_E4M3 ? launch<D, 1, SLORA_KV_E4M3, SINKS>(p, maps, num_sms, stream)
                                    : launch<D, 1, SLORA_KV_INT8, SINKS>(p, maps, num_sms, stream);
    return fmt == SLORA_KV_E4M3 ? launch<D, 2, SLORA_KV_E4M3, SINKS>(p, maps, num_sms, stream)
                                : launch<D, 2, SLORA_KV_INT8, SINKS>(p, maps, num_sms, stream);
}

}  // namespace

size_t decode_workspace_bytes(int num_sms)
{
    const size_t ctas = (size_t)num_sms * kMaxCtas;
    return (ctas * 2 * kPartStride * 4 + (ctas + 1) * 8 + 255) / 256 * 256;
}

cudaError_t launch_attend_decode(const AttendArgs &a, const PageMaps &maps, int head_dim, int fmt,
                                 int32_t small_rows, void *ws, int num_sms, cudaStream_t stream, int *launches)
{
    DecodeParams p;
    p.a = a;
    p.box_rows = a.c.bt % 16 == 0 ? 16 : 8;
    p.small_rows = small_rows;
    // Rows per unit by the batch's most common kind: every sequence's, or, where longer ones are the
    // other kernel's, the single tokens'.  8 rows have the registers for 3 CTAs per SM, 16 for 2, but
    // read the keys half as often.  24 sequences of 500 to 8000 keys, by 8 and by 16 in us: 8 rows 70
    // and 81, 16 rows 94 and 91, 32 rows 147 and 138; 96 of 16 rows 280 and 224, 4 of 16 rows 41 and
    // 50; 512 single tokens of one row 500 and 696.
    const int64_t most = (int64_t)a.b.max_q * a.group;
    p.rows = (most <= small_rows ? most : a.group) <= 8 ? 8 : 16;
    p.min_tiles = 1 + kUnitCost;
    p.bt_inverse = (uint32_t)(((1ull << 32) + a.c.bt - 1) / a.c.bt);
    p.part = static_cast<float *>(ws);
    p.joins.started = reinterpret_cast<unsigned long long *>(p.part + (size_t)num_sms * kMaxCtas * 2 * kPartStride);
    p.joins.word = p.joins.started + 1;
    cudaError_t e;
    if (head_dim == 128)
        e = a.sinks > 0 ? launch_d<128, true>(p, maps, fmt, num_sms, stream) : launch_d<128, false>(p, maps, fmt, num_sms, stream);
    else
        e = a.sinks > 0 ? launch_d<64, true>(p, maps, fmt, num_sms, stream) : launch_d<64, false>(p, maps, fmt, num_sms, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace kv
}  // namespace slora
