// i8_matmul_tc.cu -- matrix product of 8-bit tokens and 8-bit weights on the
// 5th-generation tensor cores (tcgen05, sm_103a), for five tokens to many.
//
//   acc[t][r] = sum_k W[r][k] X[t][k],  y[t][r] = (float)acc * (sw[r] * sx[t]) + bias[r]
//
// sm_103a multiplies no 8-bit integers on its tensor cores at a useful rate, but every
// int8 is an f16, every product of two is exact in f32, and at most 1024 of them stay
// within 2^24, where f32 holds every whole number.  So the bytes stay bytes in memory
// and L2 and become f16 inside the SM, and a finished f32 accumulator of 1024 k at most
// is turned into int32 and added up in registers: acc is exact for any k.
//
// Design
//  * D[channel][token]: 128 channels are the MMA's M (tensor-memory lanes) of each CTA,
//    the tokens its N.  Up to 32 tokens a CTA works alone; above, CTA pairs share each MMA
//    (cta_group::2, M = 256): each CTA converts its 128 channels and half of the tokens, so
//    a byte converted once feeds twice the products.  A tile holds up to 256 tokens, above
//    128 as two halves with MMAs of their own.
//  * Shared memory moves 128 bytes a cycle, for copies, converters and MMA operands
//    together, and is what runs out first.  So the f16 weights go to tensor memory
//    (tcgen05.st; the MMA's A operand) and only the f16 tokens go back to shared memory.
//    A stage of 128 k of a 256 x 256 pair tile then moves 128 KB in 1024 MMA cycles
//    (measured: 1225 cycles a stage).
//  * Roles (20 warps, with one half 28).  A loader copies 128 bytes of k of each row into a
//    ring by TMA, completing on an mbarrier.  Two groups of four converter warps (with one
//    half: four groups) take stages in turn.  One thread issues the MMAs.  Eight epilogue
//    warps add finished accumulators up, each thread one channel and half the tokens (at
//    most 128 int32 sums in registers), and store: a warp's lanes are channels of one token.
//  * Rows whose k is a multiple of 4 alone: TMA needs a row pitch of whole 16s, which four rows
//    have together.  The matrix is seen as n / 4 rows of 4 k bytes; the rows of one of four
//    classes (row mod 4) lie at a column of it, and a box of 144 bytes from the 16-byte
//    boundary before brings their 128 bytes, which the converters shift into place.  The last
//    n mod 4 rows are copied word by word.  (A bulk copy a row, and four-byte copies for all
//    rows, took three and two times as long as the boxes.)
//  * Tensor memory holds the accumulators, of up to 128 tokens each and used in turn (two; for
//    two halves three), and a buffer of f16 weights for each group of converters.  The two
//    halves of a tile share each stage: the accumulator of one drains while the other's MMAs
//    run, and the third takes the next 1024 k.
//  * Registers go where they are needed (setmaxnreg): the sums.
//  * With fewer tiles than SMs, k is split over the CTAs (or pairs) of a cluster, and their
//    int32 sums are added through distributed shared memory: whole numbers, so the bits do
//    not depend on the split.
//  * Every wait is bounded; one that runs out sets LOOM_DEVERR_TIMEOUT, every role stops at
//    its next wait, copies and MMAs in flight finish, tensor memory is freed, affected y are
//    NaN and acc INT32_MIN.
//
// Measured (tokens x n x k, bf16 outputs)
//   4096 x 16384 x 8192   765 us, 1.44 PFLOP/s (a library's bf16 product of these sizes takes
//                         520 to 565 us).  Bound by the converters' shared-memory traffic (64
//                         stages of 1225 cycles a tile), then by a tile's stores (18000 cycles,
//                         half of them behind the next tile's MMAs), which share those ports.
//   96 x 65536 x 4096     61 us, 4.4 TB/s: 256 tiles are 3.4 waves of 76 pairs and take four, and
//                         each begins and ends by itself.  (An MMA takes 84 cycles or more however few
//                         its tokens, and a stage has eight, 770 cycles measured: full waves of
//                         those would move 6.4 TB/s.)
//   16 x 8192 x 16384     31 us, 4.3 TB/s: 64 tiles split over 128 of the SMs, and an exchange of sums.
//                         (loom_i8_dequant_dot, whole rows on all SMs and no exchange, takes 27 us
//                         for the same sums as [row][vector] f32.)
//   203 x 5001 x 4108     31 us (k = 4112: 25 us): 120 CTAs of 11 stages each; the exchange of
//                         the sums is a third of it.
// All six forms spill some registers (124 to 164 bytes of stores a thread, 312 to 372 of loads).
#include "tc_ptx.cuh"
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int MT_KSTEP = 128;                 // k per stage: two 64-k swizzle atoms of the token operand
constexpr int MT_CHUNK_STEPS = 1024 / MT_KSTEP;   // stages per f32 accumulator
constexpr int MT_M = 128;                     // channels per CTA
constexpr int MT_CONV_WARP = 4, MT_EPI_WARPS = 8;
constexpr int MT_ACC_COLS = 128, MT_A_COLS = 64;   // tensor memory: an accumulator, a weight buffer
constexpr uint32_t MT_TMEM_COLS = 512;
// What goes by the number H of halves of a tile (of at most 128 tokens each).  With one, the
// weights' stream is the bound: four groups of converters keep up with memory, and the
// epilogue's sums are half as many.
template <int H> struct Shape {
    static constexpr int GROUPS = H == 1 ? 4 : 2;     // converter groups of four warps = weight buffers
    static constexpr int DEPTH = H == 1 ? 4 : 3;      // stages of the token operand
    static constexpr int ACCS = H == 1 ? 2 : 3;       // accumulators
    static constexpr int EPI_WARP = MT_CONV_WARP + 4 * GROUPS;
    static constexpr int THREADS = 32 * (EPI_WARP + MT_EPI_WARPS);
    // 896 x 72 >= 128 x 48 + 512 x 64 + 256 x 96;  640 x 96 = 128 x 48 + 256 x 56 + 256 x 160
    static constexpr int LAUNCH_REGS = H == 1 ? 72 : 96;
    static constexpr uint32_t A_COL = ACCS * MT_ACC_COLS;
    static_assert(A_COL + GROUPS * MT_A_COLS <= MT_TMEM_COLS, "tensor memory");
};
constexpr int MT_DEPTH = 4, MT_ACCS = 3;      // the most of either, for the barriers' places
constexpr int MT_MAX_AHEAD = 8;               // stages of bytes in the copy ring
constexpr uint32_t MT_AREA = 1024;            // barriers, tensor-memory slot, abort word
constexpr int MT_GROUP_T = 16;                // token tiles walked together (they share weight rows in L2)
constexpr uint32_t MT_MAX_SMEM = 227u * 1024u;
constexpr uint32_t MT_ROOM = MT_MAX_SMEM - 2 * MT_AREA;    // barriers, and the base's own alignment

__device__ __forceinline__ uint32_t bar_staged(uint32_t area, int s) { return area + 16 + 8 * s; }
__device__ __forceinline__ uint32_t bar_freed(uint32_t area, int s) { return area + 16 + 8 * (MT_MAX_AHEAD + s); }
__device__ __forceinline__ uint32_t bar_full(uint32_t area, int s) { return area + 16 + 8 * (2 * MT_MAX_AHEAD + s); }
__device__ __forceinline__ uint32_t bar_empty(uint32_t area, int s) { return area + 16 + 8 * (2 * MT_MAX_AHEAD + MT_DEPTH + s); }
__device__ __forceinline__ uint32_t bar_acc_full(uint32_t area, int b) { return area + 16 + 8 * (2 * MT_MAX_AHEAD + 2 * MT_DEPTH + b); }
__device__ __forceinline__ uint32_t bar_acc_empty(uint32_t area, int b) { return area + 16 + 8 * (2 * MT_MAX_AHEAD + 2 * MT_DEPTH + MT_ACCS + b); }
__device__ __forceinline__ uint32_t bar_drain(uint32_t area) { return area + 16 + 8 * (2 * MT_MAX_AHEAD + 2 * MT_DEPTH + 2 * MT_ACCS); }

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

// One arrival on the barrier at `bar` of CTA `rank` (CG 1: on this CTA's).  The release is
// the default one, of CTA scope: what the other CTA must see went through the async proxy
// (fence_async_smem) or tensor memory (fence_before) first.  A release of cluster scope
// would wait for the thread's loads in flight (measured: 1100 to 2200 cycles a stage).
template <int CG> __device__ __forceinline__ void arrive(uint32_t bar, uint32_t rank)
{
    if (CG == 1)
        tc::mbar_arrive(bar);
    else
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to(bar, rank)) : "memory");
}

// True in one lane of a converged warp.  Branching on this instruction's predicate (and not on
// a lane number) tells the compiler that one thread runs what follows.
__device__ __forceinline__ bool elected()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// The upper word of tc::smem_desc_sw128, the same for every operand here; the lower word
// is the start address in 16-byte units and a constant.
constexpr uint32_t MT_DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29), MT_DESC_LOW = 1u << 16;

// D += A (tensor memory) x B (shared memory, lower descriptor word `b`).
template <int CG> __device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    if (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
                     "r"(MT_DESC_HIGH)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
                     "r"(MT_DESC_HIGH)
                     : "memory");
}

// Arrives on `bar` (of both CTAs of the pair) when the MMAs issued so far are done.
template <int CG> __device__ __forceinline__ void commit(uint32_t bar, uint32_t pair_mask)
{
    if (CG == 1)
        tc::commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)pair_mask)
                     : "memory");
}

template <int CG> __device__ __forceinline__ void tmem_alloc(uint32_t slot)
{
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(MT_TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(MT_TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG> __device__ __forceinline__ void tmem_free(uint32_t tmem)
{
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(MT_TMEM_COLS) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(MT_TMEM_COLS) : "memory");
}

// Place of 16-byte piece j of row `row` in a stage of bytes: rows of 128 bytes in the TMA's
// 128-byte swizzle.  Eight lanes meet eight different banks when they hold one piece of
// eight rows (the weights' converters) or four pieces of rows r and r ^ 5 (the tokens').
__device__ __forceinline__ uint32_t piece_at(int row, int j) { return (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); }

// 16 bytes -> 16 f16.
__device__ __forceinline__ void to_f16(const int4 &v, uint32_t *h)
{
    tc::i8x4_to_f16x4((uint32_t)v.x, h[0], h[1]);
    tc::i8x4_to_f16x4((uint32_t)v.y, h[2], h[3]);
    tc::i8x4_to_f16x4((uint32_t)v.z, h[4], h[5]);
    tc::i8x4_to_f16x4((uint32_t)v.w, h[6], h[7]);
}

// The channel of a tensor-memory lane among its warp's 32.  Without whole 16-byte pieces the lanes
// take rows of one class by eights: neighbours of a box, on different banks.
template <bool V16> __device__ __forceinline__ int channel_of(int lane) { return V16 ? lane : (lane & 7) * 4 + (lane >> 3); }

struct Tile {
    int64_t m0, t0;     // first channel and token of the tile
};

__device__ __forceinline__ Tile tile_at(const MatmulTcPlan &q, int64_t i)
{
    const int64_t per_group = (int64_t)MT_GROUP_T * q.tiles_m, g = i / per_group, in = i % per_group;
    const int64_t wide = min((int64_t)MT_GROUP_T, (int64_t)q.tiles_t - g * MT_GROUP_T);
    return Tile{in / wide * MT_M * q.cg, (g * MT_GROUP_T + in % wide) * q.tile_t};
}

// This CTA's work: its tiles are first, first + stride, ..., each over k stages [step0, step1).
struct Work {
    int64_t first, stride, tiles;
    int step0, step1;
};

// ---- loaders -----------------------------------------------------------------------
// Rows that are whole 16-byte pieces: one thread, two TMA copies a stage.  Copies in flight
// land before it returns.
template <int CG, int H>
__device__ __forceinline__ void load_role(const MatmulParams &p, const MatmulTcPlan &q, const CUtensorMap *map_w, const CUtensorMap *map_x,
                                          uint32_t area, uint32_t ring, uint32_t pair_rank, const Work &w)
{
    const int rows = q.tile_t / (CG * H);                   // of a half, in this CTA
    const uint64_t once = dev::l2_evict_first_policy(), again = dev::l2_evict_last_policy();
    const uint64_t policy_w = q.tiles_t > 1 ? again : once;
    int s = 0;
    uint32_t phase = 1;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t i = w.first; ok && i < w.tiles; i += w.stride) {
        const Tile t = tile_at(q, i);
        const int m0 = (int)(t.m0 + pair_rank * MT_M), t0 = (int)t.t0 + (int)pair_rank * rows;
        for (int step = w.step0; step < w.step1; ++step, ++issued) {
            ok = tc::role_wait(area + 8, p.error, p.wait_ns, bar_freed(area, s), phase);
            if (!ok)
                break;
            const uint32_t to = ring + (uint32_t)s * q.ahead_bytes;
            dev::mbar_arrive_expect_tx(bar_staged(area, s), q.ahead_bytes);
            tc::tma_load_2d(to, map_w, step * MT_KSTEP, m0, bar_staged(area, s), policy_w);
#pragma unroll
            for (int h = 0; h < H; ++h)
                tc::tma_load_2d(to + (uint32_t)(MT_M + h * rows) * 128, map_x, step * MT_KSTEP, t0 + h * rows * CG, bar_staged(area, s), again);
            if (++s == q.ahead) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok)
        for (int64_t i = issued > q.ahead ? issued - q.ahead : 0; i < issued; ++i)
            dev::mbar_wait_bounded(bar_staged(area, (int)(i % q.ahead)), (uint32_t)(i / q.ahead) & 1u, 1000000000ull);
}

// Rows of any k that is a multiple of 4.  A stage is, for each class of rows (row mod 4), the boxes
// of the weights (32 rows of 144 bytes) and of each half's tokens, and places for the up to three
// last rows of either matrix.
constexpr int MT_PLACE = MT_KSTEP + 16;
constexpr uint32_t MT_CLASS_W = MT_M / 4 * MT_PLACE;
__host__ __device__ constexpr uint32_t class_x(int rows) { return ((uint32_t)rows / 4 * MT_PLACE + 127u) & ~127u; }   // TMA boxes start on 128 bytes
__host__ __device__ constexpr uint32_t last_rows_at(int rows, int halves) { return 4 * (MT_CLASS_W + (uint32_t)halves * class_x(rows)); }
__host__ __device__ constexpr uint32_t quads_stage(int rows, int halves) { return (last_rows_at(rows, halves) + 6 * MT_PLACE + 1023u) & ~1023u; }

// By one thread: the boxes.
template <int CG, int H>
__device__ __forceinline__ void load_quads_role(const MatmulParams &p, const MatmulTcPlan &q, const CUtensorMap *map_w, const CUtensorMap *map_x,
                                                uint32_t area, uint32_t ring, uint32_t pair_rank, const Work &w)
{
    const int rows = q.tile_t / (CG * H);                  // of a half, in this CTA
    const uint32_t x_class = class_x(rows), bytes = (p.n >= 4 ? 4 * MT_CLASS_W : 0) + (p.tokens >= 4 ? (uint32_t)(H * rows * MT_PLACE) : 0);
    const uint64_t policy = dev::l2_evict_last_policy();
    int s = 0;
    uint32_t phase = 1;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t i = w.first; ok && i < w.tiles; i += w.stride) {
        const Tile t = tile_at(q, i);
        const int m4 = (int)((t.m0 + pair_rank * MT_M) / 4), t4 = (int)(t.t0 / 4) + (int)pair_rank * (rows / 4);
        for (int step = w.step0; step < w.step1; ++step, ++issued) {
            ok = tc::role_wait(area + 8, p.error, p.wait_ns, bar_freed(area, s), phase);
            if (!ok)
                break;
            const uint32_t to = ring + (uint32_t)s * q.ahead_bytes, bar = bar_staged(area, s);
            dev::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int x = (c * p.k + step * MT_KSTEP) & ~15;
                if (p.n >= 4)
                    tc::tma_load_2d(to + c * MT_CLASS_W, map_w, x, m4, bar, policy);
                if (p.tokens >= 4)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        tc::tma_load_2d(to + 4 * MT_CLASS_W + (uint32_t)(h * 4 + c) * x_class, map_x, x, t4 + h * CG * (rows / 4), bar, policy);
            }
            if (++s == q.ahead) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok)
        for (int64_t i = issued > q.ahead ? issued - q.ahead : 0; i < issued; ++i)
            dev::mbar_wait_bounded(bar_staged(area, (int)(i % q.ahead)), (uint32_t)(i / q.ahead) & 1u, 1000000000ull);
}

// By one warp: the last rows of both matrices, a word a lane.
template <int CG, int H>
__device__ __forceinline__ void load_last_rows_role(const MatmulParams &p, const MatmulTcPlan &q, uint32_t area, uint32_t ring, int lane, const Work &w)
{
    int s = 0;
    uint32_t phase = 1;
    for (int64_t i = w.first; i < w.tiles; i += w.stride)
        for (int step = w.step0; step < w.step1; ++step) {
            if (!__all_sync(dev::FULL_MASK, tc::role_wait(area + 8, p.error, p.wait_ns, bar_freed(area, s), phase)))
                return;
            const uint32_t to = ring + (uint32_t)s * q.ahead_bytes + last_rows_at(q.tile_t / (CG * H), H);
            const int at = step * MT_KSTEP + 4 * lane;
            if (at < p.k)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int8_t *base = m ? p.x : p.w;
                    const int total = m ? p.tokens : p.n;
                    for (int j = 0; j < (total & 3); ++j) {
                        const int8_t *row = base + (int64_t)((total & ~3) + j) * p.k;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + (uint32_t)(m * 3 + j) * MT_PLACE + 4 * lane +
                                                                                     ((uint32_t)(j * p.k) & 15u)),
                                     "l"(row + at)
                                     : "memory");
                    }
                }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar_staged(area, s)) : "memory");
            if (++s == q.ahead) {
                s = 0;
                phase ^= 1u;
            }
        }
}

// N words from the `shift`-th of N + 3 on.
template <int N> __device__ __forceinline__ void shift_words(uint32_t (&w)[N + 3], int shift)
{
#pragma unroll
    for (int i = 0; i < N + 2; ++i)
        w[i] = (shift & 1) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < N; ++i)
        w[i] = (shift & 2) ? w[i + 2] : w[i];
}

// Whether a phase of `bar` is over, without waiting (try_wait may suspend the thread).
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// ---- converters ----------------------------------------------------------------------
// Group `group` of four warps takes every GROUPS-th of the CTA's `stages`.
template <int CG, int H, bool V16>
__device__ __forceinline__ void convert_role(const MatmulParams &p, const MatmulTcPlan &q, uint32_t area, uint32_t ring, uint32_t operands,
                                             uint32_t tmem, int group, int sub, int lane, uint32_t pair_rank, uint32_t leader, uint32_t stages,
                                             const Work &work)
{
    using S = Shape<H>;
    const int b_rows = q.tile_t / CG;
    // the tokens' pieces of this thread: piece v of rows r0, r0 + 16, ...; eight lanes hold four
    // pieces of rows r and r ^ 5, whose reads and (twice as wide) writes fall on different banks
    const int pair = sub * 2 + (lane >> 4), v = (lane & 3) | ((lane >> 3) & 1) << 2;
    const int r0 = (pair >> 2) * 8 + ((pair & 3) ^ ((lane & 4) ? 5 : 0));
    const uint32_t b_from = MT_M * 128 + piece_at(r0, v);                  // r0 + 16: the same place 16 rows on
    const uint32_t b_to = (uint32_t)((v >> 2) * b_rows * 128 + (r0 >> 3) * 1024 + (r0 & 7) * 128);
    const uint32_t c0 = b_to + ((((v & 3) * 2) ^ (r0 & 7)) << 4), c1 = b_to + ((((v & 3) * 2 + 1) ^ (r0 & 7)) << 4);
    const int row = 32 * sub + channel_of<V16>(lane), key = row & 7;
    // Without whole 16-byte pieces: the word of a place that a row's bytes start at (tiles start
    // at rows of whole 16s, so it stays), and this thread's places in the boxes.
    const int a_shift = (int)((uint32_t)(row * p.k) & 15u) / 4, b_shift = (int)((uint32_t)(r0 * p.k) & 15u) / 4;
    const int half_rows = b_rows / H;
    const uint32_t a_place = (uint32_t)(row & 3) * MT_CLASS_W + (uint32_t)(row >> 2) * MT_PLACE;
    const uint32_t b_place = 4 * MT_CLASS_W + (uint32_t)(r0 & 3) * class_x(half_rows) + (uint32_t)(r0 >> 2) * MT_PLACE + 16 * (uint32_t)v;
    int64_t tile = work.first;
    const int steps = work.step1 - work.step0;
    int step = group % steps;                      // of the stage, from step0
    tile += group / steps * work.stride;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * sub) << 16) + S::A_COL + (uint32_t)group * MT_A_COLS;
    int s = group;
    uint32_t s_phase = 0;
    while (s >= q.ahead) {
        s -= q.ahead;
        s_phase ^= 1u;
    }
    uint32_t it = (uint32_t)group;
    bool staged = false, empty = false;
    for (; it < stages; it += S::GROUPS) {
        const uint32_t d = it % S::DEPTH, turn = it / S::DEPTH;
        // first the token stage, whose last MMAs were behind every earlier stage's conversion: then
        // the ring (of at least DEPTH stages) is at most one phase behind what is asked of it
        bool ok = empty || tc::role_wait(area + 8, p.error, p.wait_ns, bar_empty(area, (int)d), (turn & 1u) ^ 1u);
        ok = ok && (staged || tc::role_wait(area + 8, p.error, p.wait_ns, bar_staged(area, s), s_phase));
        if (!__all_sync(dev::FULL_MASK, ok))
            return;
        // the weight buffer is free when the MMAs of this group's last stage are done: with fewer
        // buffers than token stages, later than what is waited for so far
        const uint32_t old = it - S::GROUPS, old_bar = bar_empty(area, (int)(old % S::DEPTH)), old_phase = (old / S::DEPTH) & 1u;
        bool a_free = S::DEPTH == S::GROUPS || it < S::GROUPS || test_wait(old_bar, old_phase);
        const uint32_t from = ring + (uint32_t)s * q.ahead_bytes;
        uint32_t a_from = from + (V16 ? (uint32_t)row * 128 : 0u);
        const uint32_t to = operands + d * q.stage_bytes;
        if constexpr (V16) {
            for (int r = 0; r < b_rows; r += 64) {
                int4 in[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + 16 * j < b_rows)
                        in[j] = tc::lds128(from + b_from + (uint32_t)(r + 16 * j) * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + 16 * j < b_rows) {
                        uint32_t out[8];
                        to_f16(in[j], out);
                        tc::sts128(to + c0 + (uint32_t)(r + 16 * j) * 128, out[0], out[1], out[2], out[3]);
                        tc::sts128(to + c1 + (uint32_t)(r + 16 * j) * 128, out[4], out[5], out[6], out[7]);
                    }
            }
        } else {
            // what lies past k is some other row's: zero for the tokens, so that it counts for nothing
            const Tile t = tile_at(q, tile);
            const int left = (p.k - (work.step0 + step) * MT_KSTEP - 16 * v) / 4;
            const uint32_t last_rows = from + last_rows_at(half_rows, H);
            const uint32_t a_row = (uint32_t)(t.m0 + pair_rank * MT_M + row - (p.n & ~3));       // of the last rows, from 0
            a_from = a_row < 3 ? last_rows + a_row * MT_PLACE : from + a_place;
#pragma unroll 2
            for (int r = 0; r < b_rows; r += 16) {
                const int h = H == 2 && r >= half_rows ? 1 : 0, in_half = r - h * half_rows;
                const uint32_t b_row = (uint32_t)(t.t0 + (h * CG + (int)pair_rank) * half_rows + in_half + r0 - (p.tokens & ~3));
                const uint32_t at = b_row < 3 ? last_rows + (3 + b_row) * MT_PLACE + 16 * (uint32_t)v
                                                            : from + b_place + (uint32_t)h * 4 * class_x(half_rows) + (uint32_t)in_half / 4 * MT_PLACE;
                const int4 lo = tc::lds128(at), hi = tc::lds128(at + 16);
                uint32_t in[7] = {(uint32_t)lo.x, (uint32_t)lo.y, (uint32_t)lo.z, (uint32_t)lo.w, (uint32_t)hi.x, (uint32_t)hi.y, (uint32_t)hi.z};
                shift_words<4>(in, b_shift);
                uint32_t out[8];
                to_f16(make_int4(left > 0 ? (int)in[0] : 0, left > 1 ? (int)in[1] : 0, left > 2 ? (int)in[2] : 0, left > 3 ? (int)in[3] : 0), out);
                tc::sts128(to + c0 + (uint32_t)r * 128, out[0], out[1], out[2], out[3]);
                tc::sts128(to + c1 + (uint32_t)r * 128, out[4], out[5], out[6], out[7]);
            }
        }
        // the weights: this thread's row, two pieces at a time
        int4 next[2];
        if constexpr (V16) {
            next[0] = tc::lds128(a_from + (uint32_t)((0 ^ key) << 4));
            next[1] = tc::lds128(a_from + (uint32_t)((1 ^ key) << 4));
        } else {
            next[1] = tc::lds128(a_from);
        }
        a_free = a_free || tc::role_wait(area + 8, p.error, p.wait_ns, old_bar, old_phase);
        if (!__all_sync(dev::FULL_MASK, a_free))
            return;
        tc::fence_after();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t out[16];
            if constexpr (V16) {
                to_f16(next[0], out);
                to_f16(next[1], out + 8);
                if (h < 3) {
                    next[0] = tc::lds128(a_from + (uint32_t)(((2 * h + 2) ^ key) << 4));
                    next[1] = tc::lds128(a_from + (uint32_t)(((2 * h + 3) ^ key) << 4));
                }
            } else {
                const int4 a = next[1], b = tc::lds128(a_from + 32 * h + 16);
                next[1] = tc::lds128(a_from + 32 * h + 32);
                uint32_t in[11] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w, (uint32_t)b.x, (uint32_t)b.y, (uint32_t)b.z,
                                   (uint32_t)b.w, (uint32_t)next[1].x, (uint32_t)next[1].y, (uint32_t)next[1].z};
                shift_words<8>(in, a_shift);
                to_f16(make_int4((int)in[0], (int)in[1], (int)in[2], (int)in[3]), out);
                to_f16(make_int4((int)in[4], (int)in[5], (int)in[6], (int)in[7]), out + 8);
            }
            tc::st16(lane_base + 16 * h, out);
        }
        // the next stage's barriers are asked while the stores land
        int s_next = s + S::GROUPS;
        uint32_t s_next_phase = s_phase;
        while (s_next >= q.ahead) {
            s_next -= q.ahead;
            s_next_phase ^= 1u;
        }
        const uint32_t n = it + S::GROUPS;
        empty = test_wait(bar_empty(area, (int)(n % S::DEPTH)), ((n / S::DEPTH) & 1u) ^ 1u);
        staged = empty && test_wait(bar_staged(area, s_next), s_next_phase);
        tc::wait_st();
        tc::fence_before();
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            tc::mbar_arrive(bar_freed(area, s));
            arrive<CG>(bar_full(area, (int)d), leader);
        }
        s = s_next;
        s_phase = s_next_phase;
        for (step += S::GROUPS; step >= steps; tile += work.stride)
            step -= steps;
    }
    // the MMAs' arrivals on this CTA's barriers come before it may leave
    for (; it < stages + S::DEPTH; it += S::GROUPS)
        if (!__all_sync(dev::FULL_MASK, tc::role_wait(area + 8, p.error, p.wait_ns, bar_empty(area, (int)(it % S::DEPTH)), ((it / S::DEPTH) & 1u) ^ 1u)))
            return;
}

// ---- MMA issue -------------------------------------------------------------------------
// By one thread, of the leading CTA of a pair; false when a wait ran out.
template <int CG, int H>
__device__ __forceinline__ bool mma_role(const MatmulParams &p, const MatmulTcPlan &q, uint32_t area, uint32_t operands, uint32_t tmem,
                                         uint32_t pair_mask, int64_t work, int step0, int step1)
{
    using S = Shape<H>;
    const uint32_t rows = (uint32_t)q.tile_t / (CG * H);     // token rows of a half in this CTA
    const uint32_t idesc = tc::idesc_f16(128 * CG, q.tile_t / H), atom = rows * H * 8;   // 16-byte units
    uint32_t acc = 0, acc_phase = 1, s = 0, phase = 0, buf = 0;
    for (; work > 0; --work)
        for (int step = step0; step < step1;) {
            const uint32_t second = acc + 1 == S::ACCS ? 0 : acc + 1, second_phase = second == 0 ? acc_phase ^ 1u : acc_phase;
            const int first = step, last = min(step + MT_CHUNK_STEPS, step1);
#pragma unroll 1
            for (; step < last; ++step) {
                if (!tc::role_wait(area + 8, p.error, p.wait_ns, bar_full(area, (int)s), phase))
                    return false;
                const uint32_t a = tmem + S::A_COL + buf * MT_A_COLS, b = MT_DESC_LOW | ((operands + s * q.stage_bytes) >> 4);
                const int slices = (p.k - step * MT_KSTEP + 15) / 16;    // of 16 k that hold anything
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t u = h == 0 ? acc : second;
                    if (step == first &&
                        !tc::role_wait(area + 8, p.error, p.wait_ns, bar_acc_empty(area, (int)u), h == 0 ? acc_phase : second_phase))
                        return false;
                    tc::fence_after();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < slices)
                            mma<CG>(tmem + u * MT_ACC_COLS, a + 8 * j, b + (j >> 2) * atom + h * rows * 8 + 2 * (j & 3), idesc,
                                    step > first || j > 0);      // the first MMA overwrites the accumulator
                    if (step == last - 1)
                        commit<CG>(bar_acc_full(area, (int)u), pair_mask);
                }
                commit<CG>(bar_empty(area, (int)s), pair_mask);
                buf = buf + 1 == S::GROUPS ? 0 : buf + 1;
                if (++s == S::DEPTH) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            acc += H;
            if (acc >= S::ACCS) {
                acc -= S::ACCS;
                acc_phase ^= 1u;
            }
        }
    return true;
}

// ---- epilogue ------------------------------------------------------------------------
// Up to N tokens from `t` on of one channel.  The element type and whether all N are there are
// decided once, not per element: a branch for each made a tile's stores take 30000 cycles, where
// they now take 18000.  The compiler barrier keeps the next tokens' scales behind this call's
// stores: the running sums leave few registers.
template <int N, typename E, typename F>
__device__ __forceinline__ void put_tokens(const MatmulParams &p, int64_t t, int64_t channel, const int32_t *a, F scale, float sw, float bias, bool ok)
{
    const int64_t stride = p.y_stride, left = p.tokens - t;
    const bool add = p.bias != nullptr, live = channel < p.n;
    auto value = [&](int i) {
        const float f = __fmul_rn((float)a[i], __fmul_rn(sw, scale(i)));
        return dev::from_f32<E>(ok ? (add ? __fadd_rn(f, bias) : f) : __uint_as_float(0x7fc00000u));
    };
    E *y = static_cast<E *>(p.y) + t * stride + channel;
    if (left >= N) {
#pragma unroll
        for (int i = 0; i < N; ++i, y += stride) {
            const E v = value(i);
            if (live)
                *y = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i, y += stride)
            if (i < left) {
                const E v = value(i);
                if (live)
                    *y = v;
            }
    }
}

// scale(i): token t + i's, asked for by whole warps and where there is such a token alone.
template <int N, typename F>
__device__ __forceinline__ void store_tokens(const MatmulParams &p, int64_t t, int64_t channel, const int32_t *a, F scale, float sw, float bias, bool ok)
{
    asm volatile("" ::: "memory");
    if (p.y_dtype == LOOM_F32)
        put_tokens<N, float>(p, t, channel, a, scale, sw, bias, ok);
    else if (p.y_dtype == LOOM_F16)
        put_tokens<N, __half>(p, t, channel, a, scale, sw, bias, ok);
    else
        put_tokens<N, __nv_bfloat16>(p, t, channel, a, scale, sw, bias, ok);
    if (p.acc && channel < p.n)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (t + i < p.tokens)
                p.acc[(t + i) * p.n + channel] = ok ? a[i] : INT32_MIN;
}

// Two runs of 16 columns, waited for together.
__device__ __forceinline__ void ld16x2(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// N sums of one channel, at an address of the cluster's shared memory.
template <int N> __device__ __forceinline__ void read_sums(uint32_t at, int32_t (&v)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v[j]) : "r"(at + 512 * j) : "memory");
}

// N tokens' sums of one channel at `at` (own shared memory, and the same place in the others), of all
// `split` CTAs, and their outputs.  The cluster's network carries about 10 bytes a cycle for each CTA,
// so the own sums are read locally, nothing twice, and each CTA begins with another neighbour.
template <int N, int CG>
__device__ __forceinline__ void store_sums(const MatmulParams &p, uint32_t at, int split, int part, uint32_t pair_rank, int64_t t, int64_t channel,
                                           int lane, float sw, float bias, bool ok)
{
    const float sx = lane < N && t + lane < p.tokens ? p.scale_x[t + lane] : 0.0f;      // a lane's token, on its way with the sums
    int32_t a[N], v[N], u[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a[j]) : "r"(at + 512 * j) : "memory");
    for (int s = 1; s < split; s += 2) {          // two neighbours' in flight together
        const int first = part + s < split ? part + s : part + s - split, second = first + 1 < split ? first + 1 : 0;
        const bool two = s + 1 < split;
        read_sums(map_to(at, (uint32_t)(first * CG) + pair_rank), v);
        if (two)
            read_sums(map_to(at, (uint32_t)(second * CG) + pair_rank), u);
#pragma unroll
        for (int j = 0; j < N; ++j)
            a[j] += v[j] + (two ? u[j] : 0);
    }
    store_tokens<N>(p, t, channel, a, [&](int i) { return __shfl_sync(dev::FULL_MASK, sx, i); }, sw, bias, ok);
}

// Adds a tile's accumulators (one for each half and 1024 k) to `sum`: of this thread's channel,
// `cols` tokens of each half; false when a wait ran out.
template <int CG, int H>
__device__ __forceinline__ bool drain_tile(const MatmulParams &p, uint32_t area, uint32_t from, int cols, int lane, uint32_t leader, uint32_t &acc,
                                           uint32_t &phase, const Work &w, bool ok, int32_t (&sum)[64 * H])
{
    const uint32_t chunks = (uint32_t)(w.step1 - w.step0 + MT_CHUNK_STEPS - 1) / MT_CHUNK_STEPS;
#pragma unroll
    for (int i = 0; i < 64 * H; ++i)
        sum[i] = 0;
    for (uint32_t c = 0; ok && c < chunks; ++c)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            ok = ok && __all_sync(dev::FULL_MASK, tc::role_wait(area + 8, p.error, p.wait_ns, bar_acc_full(area, (int)acc), phase));
            if (!ok)
                break;
            tc::fence_after();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = from + acc * MT_ACC_COLS + 32 * j;
                if (32 * j + 16 < cols) {
                    uint32_t r[32];
                    ld16x2(at, r);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sum[64 * h + 32 * j + i] += __float2int_rn(__uint_as_float(r[i]));
                } else if (32 * j < cols) {
                    uint32_t r[16];
                    tc::ld16(at, r);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum[64 * h + 32 * j + i] += __float2int_rn(__uint_as_float(r[i]));
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                arrive<CG>(bar_acc_empty(area, (int)acc), leader);
            if (++acc == Shape<H>::ACCS) {
                acc = 0;
                phase ^= 1u;
            }
        }
    return ok;
}

template <int CG, int H, bool V16>
__global__ void __launch_bounds__(Shape<H>::THREADS, 1)
    i8_matmul_tc_kernel(const MatmulParams p, const MatmulTcPlan q, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x)
{
    using S = Shape<H>;
    extern __shared__ unsigned char raw[];
    const uint32_t area = (dev::smem_u32(raw) + 1023u) & ~1023u, operands = area + MT_AREA;
    const uint32_t ring = operands + S::DEPTH * q.stage_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t pair_rank = CG == 1 ? 0 : rank & 1u, leader = CG == 1 ? rank : rank & ~1u, pair_mask = 3u << (rank & ~1u);
    const int part = (int)(rank / CG);                       // this CTA's share of k
    Work w;
    {
        const int steps = (p.k + MT_KSTEP - 1) / MT_KSTEP;
        w.step0 = (int)((int64_t)steps * part / q.split);
        w.step1 = (int)((int64_t)steps * (part + 1) / q.split);
        w.first = blockIdx.x / (CG * q.split);
        w.stride = gridDim.x / (CG * q.split);
        w.tiles = (int64_t)q.tiles_m * q.tiles_t;
    }
    const int64_t work = (w.tiles - w.first + w.stride - 1) / w.stride;

    if (threadIdx.x == 0) {
        for (int s = 0; s < q.ahead; ++s) {
            dev::mbar_init(bar_staged(area, s), V16 ? 1 : 1 + 32);
            dev::mbar_init(bar_freed(area, s), 4);
        }
        for (int s = 0; s < S::DEPTH; ++s) {
            dev::mbar_init(bar_full(area, s), 4 * CG);
            dev::mbar_init(bar_empty(area, s), 1);
        }
        for (int b = 0; b < S::ACCS; ++b) {
            dev::mbar_init(bar_acc_full(area, b), 1);
            dev::mbar_init(bar_acc_empty(area, b), MT_EPI_WARPS * CG);
        }
        dev::mbar_init(bar_drain(area), 1);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(area + 8), "r"(0u) : "memory");
        dev::fence_barrier_init();
    }
    if (warp == 1 && lane == 0) {
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (warp == 0)
        tmem_alloc<CG>(area);
    tc::fence_before();
    cluster_sync();
    tc::fence_after();
    dev::follow_previous_kernel();     // nothing above touches global memory
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(area));

    if (warp < MT_CONV_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp > 0) {
            if (!V16 && warp == 1) {
                if (elected())
                    load_quads_role<CG, H>(p, q, &map_w, &map_x, area, ring, pair_rank, w);
            } else if (!V16 && warp == 2) {
                load_last_rows_role<CG, H>(p, q, area, ring, lane, w);
                asm volatile("cp.async.wait_all;" ::: "memory");
            } else if (V16 && warp == 1 && elected()) {
                load_role<CG, H>(p, q, &map_w, &map_x, area, ring, pair_rank, w);
            }
        } else if (CG == 1 || pair_rank == 0) {
            if (elected() && !mma_role<CG, H>(p, q, area, operands, tmem, pair_mask, work, w.step0, w.step1)) {
                // let the MMAs in flight finish before tensor memory is freed
                commit<CG>(bar_drain(area), pair_mask & (0u - pair_mask));   // on this CTA alone
                const uint64_t t0 = dev::global_ns();
                while (!dev::mbar_try_wait(bar_drain(area), 0) && dev::global_ns() - t0 < 1000000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp < S::EPI_WARP) {
        if (H == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        convert_role<CG, H, V16>(p, q, area, ring, operands, tmem, (warp - MT_CONV_WARP) >> 2, warp & 3, lane, pair_rank, leader,
                                 (uint32_t)(work * (w.step1 - w.step0)), w);
        __syncwarp();
    } else {
        if (H == 1)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        const int sub = warp & 3, half = (warp - S::EPI_WARP) >> 2, cols = q.tile_t / (2 * H);   // tokens of a half for each warp
        const uint32_t from = tmem + ((uint32_t)(32 * sub) << 16) + half * cols;
        uint32_t acc = 0, phase = 0;
        bool ok = true;
        int32_t sum[64 * H];
        for (int64_t i = w.first; i < w.tiles; i += w.stride) {
            ok = drain_tile<CG, H>(p, area, from, cols, lane, leader, acc, phase, w, ok, sum);
            if (q.split > 1) {
                // sums of this share of k, [token][128 channels], over the operand stages (all of
                // them are used up: the accumulator is the last thing that read them)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j < cols)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(operands + (uint32_t)((2 * h + half) * cols + j) * 512 +
                                                                         (uint32_t)(32 * sub + lane) * 4),
                                         "r"(sum[64 * h + j])
                                         : "memory");
                break;   // one tile per cluster
            }
            const Tile t = tile_at(q, i);
            const int64_t channel = t.m0 + pair_rank * MT_M + 32 * sub + channel_of<V16>(lane);
            if (channel < p.n) {
                const float sw = p.scale_w[channel], bias = p.bias ? p.bias[channel] : 0.0f;
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (16 * j < cols)
                            {
                            const int64_t token = t.t0 + (2 * h + half) * cols + 16 * j;
                            store_tokens<16>(p, token, channel, sum + 64 * h + 16 * j, [&](int i) { return p.scale_x[token + i]; }, sw, bias, ok);
                        }
            }
        }
        __syncwarp();
    }
    __syncwarp();
    tc::fence_before();
    cluster_sync();      // every CTA's MMAs are done, its sums are in shared memory
    tc::fence_after();
    if (q.split > 1 && warp >= S::EPI_WARP) {
        const int sub = warp & 3, half = (warp - S::EPI_WARP) >> 2;
        const Tile t = tile_at(q, w.first);
        const int64_t channel = t.m0 + pair_rank * MT_M + 32 * sub + channel_of<V16>(lane);
        bool ok = true;
        for (int s = 0; s < CG * q.split; ++s) {
            uint32_t bad;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(bad) : "r"(map_to(area + 8, (uint32_t)s)) : "memory");
            ok = ok && bad == 0;
        }
        const float sw = channel < p.n ? p.scale_w[channel] : 0.0f, bias = channel < p.n && p.bias ? p.bias[channel] : 0.0f;
        const uint32_t at = operands + (uint32_t)(32 * sub + lane) * 4, turn = (uint32_t)(part * 2 + half);
        // groups of tokens, shared out over the CTAs of the split and the two warps of each channel
        if (q.tile_t >= 32 * q.split)
            for (int c = 16 * (int)turn; c < q.tile_t; c += 32 * q.split)
                store_sums<16, CG>(p, at + (uint32_t)c * 512, q.split, part, pair_rank, t.t0 + c, channel, lane, sw, bias, ok);
        else
            for (int c = 4 * (int)turn; c < q.tile_t; c += 8 * q.split)
                store_sums<4, CG>(p, at + (uint32_t)c * 512, q.split, part, pair_rank, t.t0 + c, channel, lane, sw, bias, ok);
        __syncwarp();
    }
    if (q.split > 1)
        cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 0)
        tmem_free<CG>(tmem);
}

// Rows of `pitch` bytes in boxes of `width` bytes of `rows` rows; boxes of 128 bytes swizzled.
bool encode_rows(CUtensorMap *map, const int8_t *base, int64_t pitch, int64_t outer, int width, int rows)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) == cudaSuccess && r == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<Encode>(f)
                   : nullptr;
    }();
    const cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)(outer > 0 ? outer : 1)}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)rows}, unit[2] = {1, 1};
    const CUtensorMapSwizzle swizzle = width == MT_KSTEP ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, strides, box, unit,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int H, bool V16> cudaError_t launch_cg(const MatmulParams &p, const MatmulTcPlan &q, cudaStream_t stream)
{
    const auto kernel = i8_matmul_tc_kernel<CG, H, V16>;
    // setmaxnreg hands out the registers that the launch brought: were there fewer, the
    // epilogue's request would wait for ever
    static std::atomic<uint64_t> done{0};
    if (q.ahead < Shape<H>::DEPTH)     // (no tile of matmul_tc_plan) the converters would take a stage for copied that is not
        return cudaErrorInvalidConfiguration;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), Shape<H>::LAUNCH_REGS, done);
    if (e != cudaSuccess)
        return e;
    CUtensorMap map_w = {}, map_x = {};
    const int rows = q.tile_t / (CG * H);
    if (V16 ? !encode_rows(&map_w, p.w, p.k, p.n, MT_KSTEP, MT_M) || !encode_rows(&map_x, p.x, p.k, p.tokens, MT_KSTEP, rows)
            : !encode_rows(&map_w, p.w, 4 * (int64_t)p.k, p.n / 4, MT_PLACE, MT_M / 4) ||
                  !encode_rows(&map_x, p.x, 4 * (int64_t)p.k, p.tokens / 4, MT_PLACE, rows / 4))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)q.grid);
    cfg.blockDim = dim3(Shape<H>::THREADS);
    cfg.dynamicSmemBytes = q.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)(CG * q.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, q, map_w, map_x);
}

}  // namespace

int matmul_tc_threads(const MatmulTcPlan &q) { return q.halves == 1 ? Shape<1>::THREADS : Shape<2>::THREADS; }

// Tile, split of k and grid.  The time of a choice is its waves of tiles times the stages of
// one tile, plus what a tile (or a split) costs once, in units of a stage.
bool matmul_tc_plan(int64_t tokens, int64_t n, int64_t k, bool vec16, int64_t sms, MatmulTcPlan *out)
{
    MatmulTcPlan best = {};
    double best_cost = 0.0;
    // Pairs save the conversion of half the tokens' bytes and cost an exchange of barriers: 32 tokens
    // of 4096 x 8192 take single CTAs 13.3 us, 33 take pairs 17.0.
    const int cg = tokens <= 32 ? 1 : 2, halves = tokens <= 128 ? 1 : 2;
    const int64_t steps = (k + MT_KSTEP - 1) / MT_KSTEP, tiles_t = (tokens + 255) / 256;
    const int64_t tiles_m = (n + MT_M * cg - 1) / (MT_M * cg), tiles = tiles_m * tiles_t;
    const int64_t quantum = 32 * halves;  // each half's columns, shared by two warps (and CTAs), are whole 16s
    const int64_t tile_t = ((tokens + tiles_t - 1) / tiles_t + quantum - 1) / quantum * quantum;   // up to 256
    // clusters of 1 to 8 of these CTAs (one an SM) that fit GB300's 152 SMs at a time, by
    // cudaOccupancyMaxActiveClusters: a cluster lies within one of the GPU's uneven groups of SMs
    static const int fits[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    for (int split = 1; cg * split <= 8; ++split) {
        const int64_t size = cg * split, slots = fits[size] * sms / 152;
        if (slots < 1 || (split > 1 && (tiles > slots || split > steps)))
            continue;
        const int64_t waves = (tiles + slots - 1) / slots;
        const double cost = (double)waves * ((double)((steps + split - 1) / split) + 2.0) + (split > 1 ? 3.0 + tile_t / 64.0 : 0.0);
        if (best.split == 0 || cost < best_cost) {
            best_cost = cost;
            best.split = split;
            best.grid = (tiles < slots ? tiles : slots) * size;
        }
    }
    if (best.split == 0)
        return false;
    best.cg = cg;
    best.halves = halves;
    best.tile_t = (int32_t)tile_t;
    best.tiles_m = (int32_t)tiles_m;
    best.tiles_t = (int32_t)tiles_t;
    best.stage_bytes = (uint32_t)(tile_t / cg) * 2 * MT_KSTEP;
    best.ahead_bytes = vec16 ? (uint32_t)(MT_M + tile_t / cg) * MT_KSTEP : quads_stage((int)tile_t / (cg * halves), halves);
    const uint32_t operands = (uint32_t)(halves == 1 ? Shape<1>::DEPTH : Shape<2>::DEPTH) * best.stage_bytes;
    const int64_t room = (MT_ROOM - operands) / best.ahead_bytes;
    best.ahead = (int32_t)(room < MT_MAX_AHEAD ? room : MT_MAX_AHEAD);
    uint32_t bytes = operands + (uint32_t)best.ahead * best.ahead_bytes;
    const uint32_t sums = best.split > 1 ? (uint32_t)tile_t * 512u : 0u;
    bytes = bytes > sums ? bytes : sums;
    bytes = bytes > 116u * 1024u ? bytes : 116u * 1024u;   // more than half an SM: one CTA, which owns tensor memory
    best.smem_bytes = 2 * MT_AREA + bytes;
    *out = best;
    return true;
}

cudaError_t launch_matmul_tc(const MatmulParams &p, const MatmulTcPlan &q, bool vec16, cudaStream_t stream)
{
    if (q.cg == 1)
        return vec16 ? launch_cg<1, 1, true>(p, q, stream) : launch_cg<1, 1, false>(p, q, stream);
    if (q.halves == 1)
        return vec16 ? launch_cg<2, 1, true>(p, q, stream) : launch_cg<2, 1, false>(p, q, stream);
    return vec16 ? launch_cg<2, 2, true>(p, q, stream) : launch_cg<2, 2, false>(p, q, stream);
}

}  // namespace loom
