// i4_matvec.cu -- products of a few 8-bit tokens with 4-bit weights that have a scale for each
// group along k, of one matrix or of the experts that each token goes to (sm_103a).
//
//   y[t][r] = sx[t] * sum_g s[r][g] a[t][r][g] + bias[r],  a = sum_{k in g} W[r][k] X[t][k]
//
// Design
//  * Bound: the n k / 2 bytes of W.  One CTA an SM (two for one or two tokens) takes an equal share of the rows (of
//    all rows of the experts that some pair names, counted once for each pass over them), so no partial sums leave
//    a CTA.  A row is gone through once for as many pairs as the launch has columns for (1, 2, 8, 16 or 32): one matrix's
//    as its tokens want, up to 32; the experts' as their average number of pairs wants (i4_shape).
//  * The tensor cores make the sums exact.  A weight's nibble is turned into w + 8 (one XOR) and its bits
//    are taken as a subnormal f16, (w + 8) 2^-24, or four places higher, (w + 8) 2^-20; those of the second kind
//    meet a token's byte / 16.  So eight weights cost five logic instructions and no conversion, and
//    every product is a whole multiple of 2^-24 whose sums over 128 k stay below 2^18 of them:
//    f16 MMAs (m16n8k16) with f32 sums lose nothing.  The 8 too many per weight is taken off by starting the sums
//    at -8 times the sum of the token's bytes.  (Rates measured, products per SM and clock: f16 1000, e4m3 3750, s8
//    260, dp4a 256.  e4m3, whose codes 0 to 15 are whole numbers too, with bytes as two halves: exact, but 28 us
//    for the 20.9 of 8 tokens below.)
//  * A warp takes 64 rows x 128 k at a time: 64 bytes of each row, copied ahead into its own ring of
//    shared memory (cp.async, 16 bytes; 4 where rows do not start on 16 bytes), 16-byte pieces swizzled by
//    row, so that ldmatrix hands each lane whole words of eight neighbouring weights without conflicts.  The
//    order of k inside an MMA follows from that and is the same for the tokens' bytes.
//  * The warps of a team share out k (all of a CTA's where it has one unit of rows, down to one warp where there are as
//    many units as warps); each keeps f32 sums of its rows for up to 32 tokens in registers over its part of k,
//    adding a group's whole number times the scale, and the team adds them up in a fixed order in shared
//    memory, in the stage that each warp read last.
//  * The experts' pairs are sorted by expert in each CTA (counts, a scan, lists in shared memory; up to 32 of them by
//    one warp).  Which column of an MMA a pair takes does not change its sums.
//  * What bounds it: one token the bytes and 4 us to start and end; more of them instructions (500 a stage, of which
//    unpacking and MMAs 243, the tokens' conversion 60 for each eight), 1.3 to 1.8 a clock.  Copies alone take 14 us of
//    the 20.9.  The kernels of 32 columns spill (12 bytes with groups of 128, 80 of 64, 396 of 32).
//
// Measured as nodes of a CUDA graph (8192 x 16384, groups of 128, f16 scales): 1 token 14.7 us (4.7 TB/s), 2 16.5, 3 20.6, 8 20.9,
// 16 25.9, 32 42.8; 16 tokens with groups of 64 29.9, of 32 35.6.  Experts of 2048 x 4096, 8 of 64: 1 token 10.6 us, 4 27, 16 58,
// 32 62.6 (269 MB, 4.3 TB/s).  5 x 5001 x 4104, groups of 32, f32 scales 11.6 us.  (A small call through the binding takes 11 to
// 13 us, the host's part.)
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int I4_ROWS = 64, I4_CHUNK = 128;                      // of a stage: rows, k
constexpr int I4_STAGE = I4_ROWS * I4_CHUNK / 2;                 // bytes
constexpr int I4_DEPTH = 3;                                      // stages of a warp's ring

struct I4Shape {          // of a launch
    int tokens;           // that it is built for: 1 or 2 (dp4a), 8, 16 or 32 (MMA columns)
    int warps;
    int team;             // warps that share out k
    int vec16;            // rows of W start on 16 bytes
    int x8;               // rows of X start on 8 bytes
    int log_group;
    uint32_t scales, sums, ways, lists;   // offsets in shared memory behind the rings
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Eight neighbouring bytes of a token as the B operands of two MMAs: (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16.
__device__ __forceinline__ void token_operands(uint32_t (&b)[4], uint2 x)
{
    const uint32_t u = x.x ^ 0x80808080u, v = x.y ^ 0x80808080u;      // byte + 128: the last bits of 1024 + that
    const uint32_t p = __byte_perm(u, v, 0x5140), q = __byte_perm(u, v, 0x7362);
    const uint32_t one = 0x3c003c00u, sixteenth = 0x2c002c00u, m1152 = 0xe480e480u, m72 = 0xd480d480u;
    b[0] = half2_fma(__byte_perm(p, 0x64646464u, 0x4140), one, m1152);
    b[1] = half2_fma(__byte_perm(p, 0x64646464u, 0x4342), sixteenth, m72);
    b[2] = half2_fma(__byte_perm(q, 0x64646464u, 0x4140), one, m1152);
    b[3] = half2_fma(__byte_perm(q, 0x64646464u, 0x4342), sixteenth, m72);
}

// Nibbles of two halves as (w + 8) 2^-24 and (w + 8) 2^-20.  One instruction, as its two constants are held in
// registers (where the compiler sees them it takes two).
struct Nibbles {
    uint32_t low, low8, high, high8;
};
__device__ __forceinline__ Nibbles nibble_masks()
{
    Nibbles n;
    asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, 0x00080008;\n\tmov.b32 %2, 0x00f000f0;\n\tmov.b32 %3, 0x00800080;"
                 : "=r"(n.low), "=r"(n.low8), "=r"(n.high), "=r"(n.high8));
    return n;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t a, uint32_t x)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(w), "r"(a), "r"(x));
    return d;
}

// ---- what a CTA works on: runs of rows of one matrix, each with the pairs that want it ------------
struct Lists {                 // in shared memory, of the experts' products
    // of each expert that some pair names (the latter two also behind the last): it, its first pair, passes before it
    uint16_t *expert, *first, *passes;
    uint16_t *pair;            // sorted by expert, the missing ones last
    int experts, pairs;        // that are named; that are not missing
};

struct Unit {
    int64_t matrix_row;        // of the weights, counted over all matrices
    int row, rows;             // in its matrix
    int list, count;           // pairs: places in the list (or numbers)
};

// A CTA's share of the rows of the matrices that are wanted, a row counted once for each pass over it, as runs of
// rows of one matrix.
struct Runs {
    int64_t begin, end;        // the share
    int matrix, matrices;      // of the wanted ones: the present run's, all
    int row, rows;             // the run's first row and rows
    int first, pairs;          // its pairs
};

// The run of matrix w.matrix or the next one that has rows; false past the last.
__device__ __forceinline__ bool find_run(Runs &w, const I4Params &p, const Lists &l)
{
    for (; w.matrix < w.matrices; ++w.matrix) {
        const int before = p.ids ? l.passes[w.matrix] : 0, passes = p.ids ? l.passes[w.matrix + 1] - before : 1;
        const int64_t base = (int64_t)before * p.n, b = max(w.begin - base, (int64_t)0), e = min(w.end - base, (int64_t)passes * p.n);
        if (e <= 0)
            break;
        w.row = (int)(passes == 1 ? b : b / passes);
        w.rows = (int)(passes == 1 ? e : e / passes) - w.row;
        if (w.rows > 0) {
            w.first = p.ids ? l.first[w.matrix] : 0;
            w.pairs = p.ids ? l.first[w.matrix + 1] - w.first : p.pairs;
            return true;
        }
    }
    w.matrix = w.matrices;
    return false;
}

__device__ __forceinline__ bool first_run(Runs &w, const I4Params &p, const Lists &l)
{
    w.matrices = p.ids ? l.experts : 1;
    const int64_t all = (int64_t)(p.ids ? l.passes[l.experts] : 1) * p.n;
    if (all * gridDim.x <= 0xffffffffll) {         // (a quotient of 32 bits takes a fifth of one of 64)
        w.begin = (uint32_t)all * blockIdx.x / gridDim.x;
        w.end = (uint32_t)all * (blockIdx.x + 1) / gridDim.x;
    } else {
        w.begin = all * blockIdx.x / gridDim.x;
        w.end = all * (blockIdx.x + 1) / gridDim.x;
    }
    w.matrix = 0;
    if (p.ids) {                               // the last matrix that begins at or before the share
        int step = 1;
        while (2 * step < w.matrices)
            step *= 2;
        for (; step > 0; step /= 2)
            if (w.matrix + step < w.matrices && (int64_t)l.passes[w.matrix + step] * p.n <= w.begin)
                w.matrix += step;
    }
    return find_run(w, p, l);
}

__device__ __forceinline__ bool next_run(Runs &w, const I4Params &p, const Lists &l)
{
    ++w.matrix;
    return find_run(w, p, l);
}

// The units of a team: up to 64 rows with the pairs of one pass, in turn.
struct Walk {
    Runs run;
    int q, units;              // unit of the run, of so many: its parts, each `passes` times
    int passes, part_rows;
    int columns, teams, most;  // most: rows of a unit
    bool more;
};

__device__ __forceinline__ void set_units(Walk &w)
{
    if (!w.more)
        return;
    w.passes = (w.run.pairs + w.columns - 1) / w.columns;
    const int parts = (w.run.rows + w.most - 1) / w.most;
    w.part_rows = (w.run.rows + parts - 1) / parts;
    w.units = (w.run.rows + w.part_rows - 1) / w.part_rows * w.passes;
}

// The unit that the walk stands on; false past the last.
__device__ __forceinline__ bool unit_of(Walk &w, const I4Params &p, const Lists &l, Unit &u)
{
    while (w.more) {
        if (w.q < w.units) {
            const int part = w.passes == 1 ? w.q : w.q / w.passes, pass = w.q - part * w.passes;
            const int r0 = part * w.part_rows;
            u.row = w.run.row + r0;
            u.rows = min(w.part_rows, w.run.rows - r0);
            u.matrix_row = (int64_t)(p.ids ? l.expert[w.run.matrix] : 0) * p.n + u.row;
            u.list = w.run.first + pass * w.columns;
            u.count = min(w.columns, w.run.pairs - pass * w.columns);
            return true;
        }
        w.q -= w.units;
        w.more = next_run(w.run, p, l);
        set_units(w);
    }
    return false;
}

// The row of X of a pair.
__device__ __forceinline__ int x_row(const I4Params &p, int pair)
{
    return p.pairs_per_x == 1 ? pair : (int)((unsigned)pair / (unsigned)p.pairs_per_x);
}

// Sorts the pairs by expert.  counts: [experts] words of scratch.
template <int THREADS> __device__ Lists make_lists(const I4Params &p, uint32_t *scratch, int columns)
{
    __shared__ uint64_t warp_sums[THREADS / 32];
    __shared__ uint32_t missing;
    Lists l;
    uint32_t *counts = scratch;
    l.expert = reinterpret_cast<uint16_t *>(counts + p.experts);
    l.first = l.expert + p.experts;
    l.passes = l.first + p.experts + 1;
    l.pair = l.passes + p.experts + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.pairs <= 32) {            // by one warp, a pair a lane
        __shared__ int totals[2];
        if (warp == 0) {
            int e = lane < p.pairs ? p.ids[lane] : -1;
            if (e >= p.experts) {
                if (blockIdx.x == 0)
                    dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
                e = -1;
            }
            const unsigned same = __match_any_sync(dev::FULL_MASK, e), valid = __ballot_sync(dev::FULL_MASK, e >= 0);
            const bool first = e >= 0 && (same & ((1u << lane) - 1u)) == 0;
            const int own = first ? (__popc(same) + columns - 1) / columns : 0;
            int place = 0, smaller = 0, passes = 0;          // pairs, experts and their passes that come before
            for (int i = 0; i < p.pairs; ++i) {
                const int other = __shfl_sync(dev::FULL_MASK, e, i), p_i = __shfl_sync(dev::FULL_MASK, own, i);
                const bool less = other >= 0 && other < e;
                place += less || (other >= 0 && other == e && i < lane);
                smaller += less && p_i > 0;
                passes += less ? p_i : 0;
            }
            const int pairs = __popc(valid), experts = __popc(__ballot_sync(dev::FULL_MASK, first)), all = __reduce_add_sync(dev::FULL_MASK, own);
            if (first) {
                l.expert[smaller] = (uint16_t)e;
                l.first[smaller] = (uint16_t)place;
                l.passes[smaller] = (uint16_t)passes;
            }
            if (lane < p.pairs)
                l.pair[e >= 0 ? place : pairs + __popc(~valid & ((1u << lane) - 1u))] = (uint16_t)lane;
            if (lane == 0) {
                l.first[experts] = (uint16_t)pairs;
                l.passes[experts] = (uint16_t)all;
                totals[0] = pairs;
                totals[1] = experts;
            }
        }
        __syncthreads();
        l.pairs = totals[0];
        l.experts = totals[1];
        return l;
    }
    for (int e = tid; e < p.experts; e += THREADS)
        counts[e] = 0;
    if (tid == 0)
        missing = 0;
    __syncthreads();
    constexpr int MOST = I4_MAX_PAIRS / THREADS;
    int expert[MOST];
    uint32_t rank[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int at = tid + i * THREADS;
        expert[i] = -1;
        rank[i] = 0;
        if (at < p.pairs) {
            expert[i] = p.ids[at];
            if (expert[i] >= p.experts) {
                if (blockIdx.x == 0)
                    dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
                expert[i] = -1;
            }
            rank[i] = atomicAdd(expert[i] >= 0 ? counts + expert[i] : &missing, 1u);
        }
    }
    __syncthreads();
    // three running sums in one word: pairs, from bit 20 on passes, from bit 40 on experts that have pairs
    constexpr int PER = (I4_MAX_EXPERTS + THREADS - 1) / THREADS;
    uint64_t own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        const uint32_t n = e < p.experts ? counts[e] : 0u;
        own[i] = n ? n | ((uint64_t)((n + columns - 1) / columns) << 20) | (1ull << 40) : 0ull;
        sum += own[i];
    }
    uint64_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t up = __shfl_up_sync(dev::FULL_MASK, run, d);
        run += lane >= d ? up : 0ull;
    }
    if (lane == 31)
        warp_sums[warp] = run;
    __syncthreads();
    uint64_t before = run - sum, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        before += i < warp ? warp_sums[i] : 0ull;
        all += warp_sums[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < p.experts) {
            counts[e] = (uint32_t)before & 0xfffffu;
            if (own[i]) {
                const int at = (int)(before >> 40);
                l.expert[at] = (uint16_t)e;
                l.first[at] = (uint16_t)(before & 0xfffffu);
                l.passes[at] = (uint16_t)((before >> 20) & 0xfffffu);
            }
        }
        before += own[i];
    }
    l.pairs = (int)(all & 0xfffffu);
    l.experts = (int)(all >> 40);
    if (tid == 0) {
        l.first[l.experts] = (uint16_t)l.pairs;
        l.passes[l.experts] = (uint16_t)((all >> 20) & 0xfffffu);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int at = tid + i * THREADS;
        if (at < p.pairs)
            l.pair[(expert[i] >= 0 ? counts[expert[i]] : (uint32_t)l.pairs) + rank[i]] = (uint16_t)at;
    }
    __syncthreads();
    return l;
}

// Missing routes: rows of zeros.
__device__ __forceinline__ void clear_missing(const I4Params &p, const Lists &l)
{
    for (int i = l.pairs; i < p.pairs; ++i) {
        const int64_t at = l.pair[i] * p.y_stride;
        for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < p.n; r += (int64_t)gridDim.x * blockDim.x)
            dev::store_as(p.y, p.y_dtype, at + r, 0.0f);
    }
}

// A warp's copies, which run two stages ahead of its products: 64 bytes of up to 64 rows a stage.  What lies past the
// rows or past k is not copied: it meets zeros, or sums that are thrown away.
struct Copies {
    const char *src;           // of this lane's first row in the stage
    int limit, chunk;          // rows of the unit from that one on
    uint32_t at;               // where the next stage goes, of this lane's first piece
    bool more;
};

// A warp's way through its units, in shared memory (registers hold the sums): where its copies stand, and the units
// that they have begun, for the products (at most two of them ahead).
struct Way {
    Walk walk;
    Unit queue[4];
    int made;
    uint32_t sums;             // where the warp's last sums lie
};

__device__ __forceinline__ void start_unit(Copies &c, Way *way, const I4Params &p, const I4Shape &s, const Lists &l, int chunk, int lane)
{
    Walk w = way->walk;
    Unit u;
    c.more = unit_of(w, p, l, u);
    c.chunk = chunk;
    u.count = c.more ? u.count : 0;
    const int at = way->made;
    __syncwarp();
    if (lane == 0) {
        w.q += w.teams;
        way->walk = w;
        way->queue[at & 3] = u;
        way->made = at + 1;
    }
    __syncwarp();
    if (!c.more)
        return;
    const int r0 = s.vec16 ? lane >> 2 : lane >> 4, row_bytes = p.k / 2;
    c.limit = u.rows - r0;
    c.src = reinterpret_cast<const char *>(p.w) + (u.matrix_row + r0) * row_bytes + chunk * (I4_CHUNK / 2) + (s.vec16 ? 16 * (lane & 3) : 4 * (lane & 15));
}

__device__ __forceinline__ void copy_stage(const Copies &c, const I4Params &p, const I4Shape &s, int lane)
{
    const int row_bytes = p.k / 2, left = row_bytes - c.chunk * (I4_CHUNK / 2);
    if (s.vec16) {
        const int rows = 16 * (lane & 3) < left ? c.limit : 0;
        const uint32_t step = 8u * (uint32_t)row_bytes;
#pragma unroll
        for (int i = 0; i < I4_ROWS / 8; ++i)
            if (8 * i < rows)
                copy_async16(c.at + 512 * i, c.src + (uint64_t)step * i);
    } else if (4 * (lane & 15) < left) {
        const int word = lane & 15, r0 = lane >> 4;
        const uint32_t stage = c.at - (r0 * 64 + (((word >> 2) ^ (r0 >> 1)) << 4) + 4 * (word & 3));
#pragma unroll 8
        for (int r = 0; r < c.limit; r += 2) {
            const int row = r0 + r;
            copy_async4(stage + row * 64 + (((word >> 2) ^ ((row >> 1) & 3)) << 4) + 4 * (word & 3), c.src + r * (int64_t)row_bytes);
        }
    }
}

// NT: MMA columns / 8; FL: steps of 32 k between flushes (a group's, 4 at most); PAIR: 16-row tiles whose MMAs overlap.
template <int NT, int FL, int WARPS, int PAIR>
__global__ void __launch_bounds__(32 * WARPS, 1) i4_matvec_kernel(const I4Params p, const I4Shape s)
{
    extern __shared__ __align__(128) unsigned char i4_shared[];
    constexpr int STEPS = I4_CHUNK / 32, SP = STEPS / FL;            // SP: flushes, and scales of a row, in a stage
    constexpr bool EARLY = NT <= 2 && WARPS == 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
    dev::follow_previous_kernel();

    Lists l = {};
    if (p.ids) {
        l = make_lists<32 * WARPS>(p, reinterpret_cast<uint32_t *>(i4_shared + s.lists), 8 * NT);
        clear_missing(p, l);
    }
    Way *way = reinterpret_cast<Way *>(i4_shared + s.ways) + warp;
    {
        Walk walk;
        walk.more = first_run(walk.run, p, l);
        walk.teams = WARPS / s.team;
        walk.columns = 8 * NT;
        walk.q = warp / s.team;
        // Units of whole 16 rows, 64 at most, so many that the teams take the same number, or one less: each matrix but the
        // first may add one that is not full.  (With 17 units for 16 warps 16 tokens to 8 of 64 experts took 72 us.)
        const int64_t share = walk.run.end - walk.run.begin;
        int matrices = 0;
        if (p.ids)
            for (int m = walk.run.matrix + 1; m < walk.run.matrices && (int64_t)l.passes[m] * p.n < walk.run.end; ++m)
                ++matrices;
        int64_t slots = walk.teams - matrices;
        while (slots <= 0 || share > slots * I4_ROWS)
            slots += walk.teams;
        walk.most = ((int)((share + slots - 1) / slots) + 15) / 16 * 16;
        set_units(walk);
        if (lane == 0) {
            way->walk = walk;
            way->made = 0;
        }
        __syncwarp();
    }
    const int part = warp % s.team;
    const int chunks = (p.k + I4_CHUNK - 1) / I4_CHUNK;
    const int c0 = chunks * part / s.team, c1 = chunks * (part + 1) / s.team;

    const uint32_t ring = dev::smem_u32(i4_shared) + warp * I4_DEPTH * I4_STAGE;
    float *scales = reinterpret_cast<float *>(i4_shared + s.scales) + warp * I4_ROWS * SP;
    const Nibbles n = nibble_masks();
    // ldmatrix: lane's row of a tile, and the piece of 16 bytes that it points at in the first two steps
    const uint32_t place = (lane & 15) * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4);

    Copies ahead;
    const int word = lane & 15;
    const uint32_t first_place = s.vec16 ? (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4)
                                         : (lane >> 4) * 64 + ((word >> 2) << 4) + 4 * (word & 3);
    const uint32_t ring_end = ring + I4_DEPTH * I4_STAGE;
    ahead.at = ring + first_place;
    start_unit(ahead, way, p, s, l, c0, lane);
    const auto copy_next = [&]() {
        if (ahead.more && c0 < c1) {
            copy_stage(ahead, p, s, lane);
            ahead.src += I4_CHUNK / 2;
            if (++ahead.chunk == c1)
                start_unit(ahead, way, p, s, l, c0, lane);
        }
        copies_commit();
        ahead.at += I4_STAGE;
        if (ahead.at >= ring_end)
            ahead.at -= I4_DEPTH * I4_STAGE;
    };
    for (int i = 1; i < I4_DEPTH; ++i)
        copy_next();

    uint32_t stage = ring + place;
    for (int done = 0;; ++done) {
        if (c0 >= c1 && done > 0)                 // (no k: no copies begin a unit)
            start_unit(ahead, way, p, s, l, c0, lane);
        const Unit u = way->queue[done & 3];
        if (u.count == 0)
            break;
        float acc[4][NT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][j][i] = 0.0f;
        const int8_t *xp[NT];                // columns that no pair has take the first one's: their sums are not used
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int col = 8 * j + g < u.count ? 8 * j + g : 0;
            xp[j] = p.x + (int64_t)x_row(p, p.ids ? l.pair[u.list + col] : u.list + col) * p.k + 8 * tig;
        }
        uint2 raw[STEPS][NT];
        const auto load_tokens = [&](int chunk) {
            const int k0 = chunk * I4_CHUNK;
            if (s.x8 && k0 + I4_CHUNK <= p.k) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < STEPS; ++i)
                        raw[i][j] = __ldg(reinterpret_cast<const uint2 *>(xp[j] + k0 + 32 * i));
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < STEPS; ++i) {
                        const int8_t *at = xp[j] + k0 + 32 * i;
                        raw[i][j] = make_uint2(0, 0);
                        if (k0 + 32 * i + 8 * tig < p.k)
                            raw[i][j] = make_uint2(__ldg(reinterpret_cast<const uint32_t *>(at)), __ldg(reinterpret_cast<const uint32_t *>(at) + 1));
                    }
            }
        };
        // a stage's scales: lane's are those of elements lane + 32 i of [64 rows][SP]
        const int64_t scale0 = u.matrix_row * p.groups;
        int scale_row[2 * SP];
#pragma unroll
        for (int i = 0; i < 2 * SP; ++i)
            scale_row[i] = min((lane + 32 * i) / SP, u.rows - 1) * p.groups;
        uint32_t scale[2 * SP];
        const auto load_scales = [&](int chunk) {
            const int group = min((chunk * I4_CHUNK + lane % SP * 32 * FL) >> s.log_group, p.groups - 1);
            if (p.scale_dtype == LOOM_F32) {
                const uint32_t *at = static_cast<const uint32_t *>(p.scale_w) + scale0 + group;
#pragma unroll
                for (int i = 0; i < 2 * SP; ++i)
                    scale[i] = __ldg(at + scale_row[i]);
            } else {
                const unsigned short *at = static_cast<const unsigned short *>(p.scale_w) + scale0 + group;
#pragma unroll
                for (int i = 0; i < 2 * SP; ++i)
                    scale[i] = __ldg(at + scale_row[i]);
            }
        };
        if (c0 < c1) {
            load_tokens(c0);
            load_scales(c0);
        }
        for (int c = c0; c < c1; ++c) {
            copies_wait<I4_DEPTH - 2>();
            __syncwarp();                    // the stage is there, and the last one read by all lanes
            copy_next();
            // (the whole sums are in 2^-24)
            if (p.scale_dtype == LOOM_F16) {
#pragma unroll
                for (int i = 0; i < 2 * SP; ++i)
                    scales[lane + 32 * i] = __half2float(__ushort_as_half((unsigned short)scale[i])) * 16777216.0f;
            } else {
                const int up = p.scale_dtype == LOOM_BF16 ? 16 : 0;
#pragma unroll
                for (int i = 0; i < 2 * SP; ++i)
                    scales[lane + 32 * i] = __uint_as_float(scale[i] << up) * 16777216.0f;
            }
            uint32_t early[EARLY ? 4 : 1][2][4];          // where registers allow it: the stage's weights, whose way takes as long
            if (EARLY) {                                  // as the tokens' conversion
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        load_matrices(early[t % (EARLY ? 4 : 1)][i], (stage ^ (i << 5)) + t * 1024);
            }
            uint32_t b[STEPS][NT][4];
            float start[SP][NT][4];
#pragma unroll
            for (int f = 0; f < SP; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    int sum = 0;
#pragma unroll
                    for (int i = f * FL; i < (f + 1) * FL; ++i) {
                        token_operands(b[i][j], raw[i][j]);
                        sum = __dp4a((int)raw[i][j].x, 0x01010101, __dp4a((int)raw[i][j].y, 0x01010101, sum));
                    }
                    sum += __shfl_xor_sync(dev::FULL_MASK, sum, 1);
                    sum += __shfl_xor_sync(dev::FULL_MASK, sum, 2);
                    const float of = (float)sum * -4.76837158203125e-07f;      // -8 * 2^-24
                    start[f][j][0] = start[f][j][2] = __shfl_sync(dev::FULL_MASK, of, 8 * tig);
                    start[f][j][1] = start[f][j][3] = __shfl_sync(dev::FULL_MASK, of, 8 * tig + 4);
                }
            if (c + 1 < c1) {
                load_tokens(c + 1);
                load_scales(c + 1);
            }
            __syncwarp();
#pragma unroll
            for (int t0 = 0; t0 < 4; t0 += PAIR) {
                if (16 * t0 >= u.rows)
                    break;
                uint32_t w[PAIR][4];
#pragma unroll
                for (int f = 0; f < SP; ++f) {
                    float sum[PAIR][NT][4];
#pragma unroll
                    for (int i = f * FL; i < (f + 1) * FL; ++i)
#pragma unroll
                        for (int t = 0; t < PAIR; ++t) {
                            if (!EARLY && i % 2 == 0)         // two steps (16-byte pieces) of 16 rows at a time
                                load_matrices(w[t], (stage ^ (i << 4)) + (t0 + t) * 1024);
                            const uint32_t *of = EARLY ? early[(t0 + t) % (EARLY ? 4 : 1)][i / 2] : w[t];
                            const uint32_t w0 = of[2 * (i % 2)], w1 = of[2 * (i % 2) + 1];
                            const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
                            const uint32_t a0 = and_xor(w0, n.low, n.low8), a1 = and_xor(w1, n.low, n.low8);
                            const uint32_t a2 = and_xor(w0, n.high, n.high8), a3 = and_xor(w1, n.high, n.high8);
                            const uint32_t e0 = and_xor(v0, n.low, n.low8), e1 = and_xor(v1, n.low, n.low8);
                            const uint32_t e2 = and_xor(v0, n.high, n.high8), e3 = and_xor(v1, n.high, n.high8);
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                if (i == f * FL)
                                    mma(sum[t][j], a0, a1, a2, a3, b[i][j][0], b[i][j][1], start[f][j]);
                                else
                                    mma(sum[t][j], a0, a1, a2, a3, b[i][j][0], b[i][j][1], sum[t][j]);
                                mma(sum[t][j], e0, e1, e2, e3, b[i][j][2], b[i][j][3], sum[t][j]);
                            }
                        }
#pragma unroll
                    for (int t = 0; t < PAIR; ++t) {
                        const float *at = scales + (16 * (t0 + t) + g) * SP + f;
                        const float s0 = at[0], s1 = at[8 * SP];
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            acc[t0 + t][j][0] = fmaf(s0, sum[t][j][0], acc[t0 + t][j][0]);
                            acc[t0 + t][j][1] = fmaf(s0, sum[t][j][1], acc[t0 + t][j][1]);
                            acc[t0 + t][j][2] = fmaf(s1, sum[t][j][2], acc[t0 + t][j][2]);
                            acc[t0 + t][j][3] = fmaf(s1, sum[t][j][3], acc[t0 + t][j][3]);
                        }
                    }
                }
            }
            stage += I4_STAGE;
            if (stage >= ring_end)
                stage -= I4_DEPTH * I4_STAGE;
        }
        const auto finish = [&](float y, int row, int col) {
            const int pair = p.ids ? l.pair[u.list + col] : u.list + col;
            y *= __ldg(p.scale_x + x_row(p, pair));
            if (p.bias)
                y = __fadd_rn(y, __ldg(p.bias + u.matrix_row + row));
            dev::store_as(p.y, p.y_dtype, pair * p.y_stride + u.row + row, y);
        };
        if (s.team == 1) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 8 * j + 2 * tig + i;
                    if (col < u.count) {
                        const int pair = p.ids ? l.pair[u.list + col] : u.list + col;
                        const float sx = __ldg(p.scale_x + x_row(p, pair));
                        const int64_t at = pair * p.y_stride + u.row;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int row = 16 * t + 8 * h + g;
                                if (row < u.rows) {
                                    const float y = acc[t][j][2 * h + i] * sx;
                                    dev::store_as(p.y, p.y_dtype, at + row, p.bias ? __fadd_rn(y, __ldg(p.bias + u.matrix_row + row)) : y);
                                }
                            }
                    }
                }
            continue;
        }
        // The team's sums meet in the stages that were read last, which no copy is under way to, as
        // [rows][columns]; where they do not hold all 64 rows, in two rounds.
        constexpr int ROUNDS = 32 * NT * I4_ROWS > I4_STAGE ? 2 : 1, ROWS = I4_ROWS / ROUNDS, TILES = 4 / ROUNDS;
        const int team_thread = threadIdx.x - 32 * (warp - part), barrier = 1 + warp / s.team;
        const uint32_t offset = (stage == ring + place ? ring_end : stage - place) - I4_STAGE - dev::smem_u32(i4_shared);
        float *own = reinterpret_cast<float *>(i4_shared + offset);
        __syncwarp();                                       // (all lanes have read the stage)
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r * ROWS >= u.rows)
                break;
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float *at = own + (16 * t + g) * 8 * NT + 8 * j + 2 * tig;
                    *reinterpret_cast<float2 *>(at) = make_float2(acc[r * TILES + t][j][0], acc[r * TILES + t][j][1]);
                    *reinterpret_cast<float2 *>(at + 64 * NT) = make_float2(acc[r * TILES + t][j][2], acc[r * TILES + t][j][3]);
                }
            if (lane == 0)
                way->sums = offset;
            asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * s.team) : "memory");
            for (int i = team_thread; i < ROWS * 8 * NT; i += 32 * s.team) {
                const int row = r * ROWS + i / (8 * NT), col = i % (8 * NT);
                if (row < u.rows && col < u.count) {
                    float y = 0.0f;
#pragma unroll 4
                    for (int w = 0; w < s.team; ++w)
                        y += reinterpret_cast<const float *>(i4_shared + (way - part + w)->sums)[i];
                    finish(y, row, col);
                }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * s.team) : "memory");
        }
    }
    copies_wait<0>();
}

// ---- one or two tokens: dp4a ------------------------------------------------------------------
// Lanes across k: 16 bytes of a row (32 weights, one scale) each, so a warp takes 1024 k of R rows at a
// time with the tokens' bytes for them in registers.  A nibble in a byte's upper half is 16 times a signed
// weight, so eight weights cost three logic instructions and two dp4a (8192 x 16384: 14.7 us for one token where the
// tensor cores take 20).  Warps share out k where it is long, rows where it is not; a row's sums over lanes meet in
// shared memory, one place per warp, and are added in a fixed order.
constexpr int DP_CHUNK = 1024;      // k of a warp's access
constexpr int DP_RUN = 512;         // rows whose sums a CTA holds
constexpr int DP_WARPS = 8, DP_THREADS = 32 * DP_WARPS;

// Sums of N values over the warp: afterwards v[0] of lane l is the sum of value l / (32 / N).
template <int N> __device__ __forceinline__ void sum_lanes(float (&v)[N], int lane)
{
    int n = N;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = (lane & m) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(dev::FULL_MASK, send, m);
                }
        } else {
            v[0] += __shfl_xor_sync(dev::FULL_MASK, v[0], m);
        }
    }
}

// T tokens, R rows and KV chunks of k together.  V16: rows start on 16 bytes, and a lane holds 16 neighbouring
// bytes; else the words lane, lane + 32, ... of the chunk.
template <int T, int R, int KV, bool V16> __global__ void __launch_bounds__(DP_THREADS, 2) i4_dp4a_kernel(const I4Params p, const I4Shape s)
{
    extern __shared__ __align__(128) unsigned char i4_shared[];
    constexpr int Q = V16 ? 1 : 4;                                   // scales of a lane's 32 weights
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    dev::follow_previous_kernel();
    Lists l = {};
    if (p.ids) {
        l = make_lists<DP_THREADS>(p, reinterpret_cast<uint32_t *>(i4_shared + s.lists), T);
        clear_missing(p, l);
    }
    float *sums = reinterpret_cast<float *>(i4_shared + s.sums);     // [team][rows of the run][T]
    const int part = warp % s.team, team = warp / s.team, teams = DP_WARPS / s.team;
    const int chunks = (p.k + DP_CHUNK - 1) / DP_CHUNK;
    const int c0 = chunks * part / s.team, c1 = chunks * (part + 1) / s.team;
    const int row_bytes = p.k / 2;
    Runs run;
    for (bool more = first_run(run, p, l); more;) {
        const int rows = min(run.rows, DP_RUN);
        const int64_t matrix_row = (int64_t)(p.ids ? l.expert[run.matrix] : 0) * p.n + run.row;
        const int r0 = rows * team / teams, r1 = rows * (team + 1) / teams;
        for (int pass = 0; pass < run.pairs; pass += T) {
            for (int c = c0; c < c1; c += KV) {
                // the tokens' bytes: of each word's eight the even ones and the odd ones
                uint32_t x[T][KV][8];
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const int pair = min(pass + t, run.pairs - 1);
                    const int8_t *xr = p.x + (int64_t)x_row(p, p.ids ? l.pair[run.first + pair] : pair) * p.k;
#pragma unroll
                    for (int j = 0; j < KV; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int k0 = (c + j) * DP_CHUNK + (V16 ? 32 * lane + 8 * i : 8 * lane + 256 * i);
                            uint32_t a = 0, b = 0;
                            if (c + j < c1 && k0 < p.k) {
                                a = __ldg(reinterpret_cast<const uint32_t *>(xr + k0));
                                b = __ldg(reinterpret_cast<const uint32_t *>(xr + k0) + 1);
                            }
                            x[t][j][2 * i] = __byte_perm(a, b, 0x6420);
                            x[t][j][2 * i + 1] = __byte_perm(a, b, 0x7531);
                        }
                }
                bool there[KV][Q];
                int group[KV][Q];
#pragma unroll
                for (int j = 0; j < KV; ++j)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int k0 = (c + j) * DP_CHUNK + (V16 ? 32 * lane : 8 * lane + 256 * q);
                        there[j][q] = c + j < c1 && k0 < p.k;
                        group[j][q] = there[j][q] ? k0 >> s.log_group : 0;
                    }
                const char *w_row = reinterpret_cast<const char *>(p.w) + (matrix_row + r0) * row_bytes + c * (DP_CHUNK / 2) + (V16 ? 16 : 4) * lane;
                int64_t scale_row = (matrix_row + r0) * p.groups;
                for (int r = r0; r < r1; r += R, w_row += R * (int64_t)row_bytes, scale_row += R * p.groups) {
                    uint4 w[R][KV];
                    uint32_t scale[R][KV][Q];
                    const char *at = w_row;
#pragma unroll
                    for (int i = 0; i < R; ++i) {
#pragma unroll
                        for (int j = 0; j < KV; ++j) {
                            uint32_t *o = &w[i][j].x;
                            w[i][j] = make_uint4(0, 0, 0, 0);
                            if (V16) {
                                if (there[j][0])
                                    w[i][j] = __ldcs(reinterpret_cast<const uint4 *>(at + j * (DP_CHUNK / 2)));
                            } else {
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (there[j][q % Q])
                                        o[q] = __ldcs(reinterpret_cast<const uint32_t *>(at + j * (DP_CHUNK / 2) + 128 * q));
                            }
                        }
                        if (r + i + 1 < r1)        // (past the last row its own again)
                            at += row_bytes;
                    }
                    if (p.scale_dtype == LOOM_F32) {
                        const uint32_t *from = static_cast<const uint32_t *>(p.scale_w) + scale_row;
#pragma unroll
                        for (int i = 0; i < R; ++i) {
#pragma unroll
                            for (int j = 0; j < KV; ++j)
#pragma unroll
                                for (int q = 0; q < Q; ++q)
                                    scale[i][j][q] = __ldg(from + group[j][q]);
                            if (r + i + 1 < r1)
                                from += p.groups;
                        }
                    } else {
                        const unsigned short *from = static_cast<const unsigned short *>(p.scale_w) + scale_row;
#pragma unroll
                        for (int i = 0; i < R; ++i) {
#pragma unroll
                            for (int j = 0; j < KV; ++j)
#pragma unroll
                                for (int q = 0; q < Q; ++q)
                                    scale[i][j][q] = __ldg(from + group[j][q]);
                            if (r + i + 1 < r1)
                                from += p.groups;
                        }
                    }
                    int a[R][KV][Q][T];
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int j = 0; j < KV; ++j) {
                            const uint32_t *word = &w[i][j].x;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t even = (word[q] << 4) & 0xf0f0f0f0u, odd = word[q] & 0xf0f0f0f0u;
#pragma unroll
                                for (int t = 0; t < T; ++t) {
                                    int &sum = a[i][j][q % Q][t];
                                    sum = __dp4a((int)even, (int)x[t][j][2 * q], q < Q ? 0 : sum);
                                    sum = __dp4a((int)odd, (int)x[t][j][2 * q + 1], sum);
                                }
                            }
                        }
                    float v[R * T];
                    const bool half = p.scale_dtype == LOOM_F16;
                    const int up = p.scale_dtype == LOOM_BF16 ? 16 : 0;
#pragma unroll
                    for (int i = 0; i < R * T; ++i)
                        v[i] = 0.0f;
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int j = 0; j < KV; ++j)
#pragma unroll
                            for (int q = 0; q < Q; ++q) {
                                const float f = half ? __half2float(__ushort_as_half((unsigned short)scale[i][j][q])) : __uint_as_float(scale[i][j][q] << up);
#pragma unroll
                                for (int t = 0; t < T; ++t)
                                    v[i * T + t] = fmaf(f, (float)a[i][j][q][t], v[i * T + t]);
                            }
                    sum_lanes<R * T>(v, lane);
                    constexpr int SPAN = 32 / (R * T);
                    const int i = lane / SPAN / T, t = lane / SPAN % T;
                    if (lane % SPAN == 0 && r + i < r1) {
                        float *to = sums + (part * rows + r + i) * T + t;
                        *to = c == c0 ? v[0] : *to + v[0];
                    }
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < rows * T; i += DP_THREADS) {
                const int r = T == 1 ? i : i / T, t = T == 1 ? 0 : i % T;
                if (pass + t < run.pairs) {
                    float y = 0.0f;
                    for (int w = 0; w < s.team && chunks > 0; ++w)
                        y += sums[w * rows * T + i];
                    const int pair = p.ids ? l.pair[run.first + pass + t] : pass + t;
                    y *= __ldg(p.scale_x + x_row(p, pair)) * 0.0625f;
                    if (p.bias)
                        y = __fadd_rn(y, __ldg(p.bias + matrix_row + r));
                    dev::store_as(p.y, p.y_dtype, pair * p.y_stride + run.row + r, y);
                }
            }
            __syncthreads();
        }
        if (rows < run.rows) {
            run.row += rows;
            run.rows -= rows;
        } else {
            more = next_run(run, p, l);
        }
    }
}

template <typename... A> cudaError_t launch_kernel(void (*kernel)(A...), std::atomic<uint64_t> &done, const I4Params &p, const I4Shape &s,
                                                   const loom_launch &L, cudaStream_t stream)
{
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), 0, done);
    return e != cudaSuccess ? e : launch_prepared(kernel, L, stream, p, s);
}

template <int NT, int FL, int WARPS, int PAIR>
cudaError_t launch_mma(const I4Params &p, const I4Shape &s, const loom_launch &L, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_kernel(i4_matvec_kernel<NT, FL, WARPS, PAIR>, done, p, s, L, stream);
}

template <int T, int R, int KV, bool V16>
cudaError_t launch_dp4a(const I4Params &p, const I4Shape &s, const loom_launch &L, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_kernel(i4_dp4a_kernel<T, R, KV, V16>, done, p, s, L, stream);
}

template <int NT, int WARPS> cudaError_t launch_nt(const I4Params &p, const I4Shape &s, const loom_launch &L, cudaStream_t stream)
{
    constexpr int PAIR = NT == 4 ? 1 : NT == 1 && WARPS == 8 ? 4 : 2;
    return p.group == 32 ? launch_mma<NT, 1, WARPS, PAIR>(p, s, L, stream)
                         : p.group == 64 ? launch_mma<NT, 2, WARPS, PAIR>(p, s, L, stream) : launch_mma<NT, 4, WARPS, PAIR>(p, s, L, stream);
}

int log2_floor(int64_t v)
{
    int l = 0;
    while (v >> (l + 1))
        ++l;
    return l;
}

// Bytes of the experts' lists (make_lists).
constexpr int64_t list_bytes(int64_t experts, int64_t pairs) { return (10 * experts + 4 + 2 * pairs + 15) / 16 * 16; }

// What a launch is built for: tokens of the dp4a kernel (1 or 2), or MMA columns (8, 16, 32), for the
// pairs that a matrix has -- on average half as many again of the experts' that are wanted.  The host does not know the ids:
// uneven ones take more passes (64 tokens to 8 of 64 experts 89 us, all tokens to the same 8 46, half of
// the pairs to two experts 150 to 180).
// Its warps and shared memory (the static arrays of make_lists are counted as 256 bytes).
uint32_t i4_shape(int64_t pairs, int64_t n, int64_t k, int64_t group, int64_t experts, int64_t sms, I4Shape *s)
{
    const int64_t named = experts ? (pairs < experts ? pairs : experts) : 1;
    const int64_t each = experts <= 1 ? pairs : pairs <= experts / 4 ? 1 : (3 * pairs + 2 * named - 1) / (2 * named);
    s->tokens = each <= 2 ? (int)each : each <= 8 ? 8 : each <= 16 ? 16 : 32;
    const bool few = s->tokens <= 2;
    // Eight warps with 255 registers each load a stage's weights before they convert its tokens; sixteen hide more where
    // each has rows of its own (measured, 8 tokens: 8192 x 16384 21.3 us by 8 warps, 22.3 by 16, 65536 x 2048 21.1 and
    // 23.3; 32 tokens to 8 of 64 experts of 2048 x 4096 70 and 64).
    const int64_t rows = named * n / sms;
    s->warps = few ? DP_WARPS : s->tokens == 8 && rows >= 12 * I4_ROWS ? 16 : 8;
    const int64_t chunk = few ? DP_CHUNK : I4_CHUNK, chunks = (k + chunk - 1) / chunk;
    // A team for each 48 rows of a CTA or more: its warps meet after each 64 rows, the fewer the cheaper.
    // The dp4a kernel's warps take two chunks each, where there are as many.
    const int64_t units = rows / (3 * I4_ROWS / 4);
    int team = few ? s->warps : s->warps >> log2_floor(units < 1 ? 1 : units > s->warps ? s->warps : units);
    while (team > 1 && team > (few ? chunks / 2 : chunks))
        team /= 2;
    s->team = team;
    s->scales = few ? 0 : (uint32_t)(s->warps * I4_DEPTH * I4_STAGE);
    s->sums = s->scales + (few ? 0 : s->warps * I4_ROWS * 4 * (group == 32 ? 4 : group == 64 ? 2 : 1));
    s->ways = s->sums + (few ? (uint32_t)(s->team * DP_RUN * s->tokens * 4) : 0);
    s->lists = s->ways + (few ? 0 : s->warps * (uint32_t)sizeof(Way));
    return s->lists + (experts ? (uint32_t)list_bytes(experts, pairs) : 0);
}
static_assert(16 * (I4_DEPTH * I4_STAGE + I4_ROWS * 16 + (int)sizeof(Way)) + list_bytes(I4_MAX_EXPERTS, I4_MAX_PAIRS) + 256 <= 227 * 1024, "the most there is");

}  // namespace

void i4_geometry(int64_t pairs, int64_t n, int64_t k, int64_t group, int64_t experts, int64_t sms, loom_launch *out)
{
    I4Shape s;
    *out = loom_launch{};
    out->smem_bytes = i4_shape(pairs, n, k, group, experts, sms, &s);
    const int64_t most = (experts ? (experts < pairs ? experts : pairs) : 1) * n, ctas = s.tokens > 2 ? sms : 2 * sms;
    out->grid[0] = (uint32_t)(most < ctas ? (most > 0 ? most : 1) : ctas);
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->block[0] = 32 * s.warps;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    const int64_t rows = (most + out->grid[0] - 1) / out->grid[0];
    out->units_per_cta = (uint32_t)(rows < 0xffffffffll ? rows : 0xffffffffll);
    out->kernel = LOOM_KERNEL_I4_MATVEC;
}

cudaError_t launch_i4_matvec(const I4Params &p, int64_t sms, const loom_launch &L, cudaStream_t stream)
{
    I4Shape s;
    i4_shape(p.pairs, p.n, p.k, p.group, p.ids ? (p.experts > 0 ? p.experts : 1) : 0, sms, &s);
    s.vec16 = p.k % 32 == 0 && reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    s.x8 = reinterpret_cast<uintptr_t>(p.x) % 8 == 0;
    s.log_group = log2_floor(p.group);
    switch (s.tokens) {
    case 1: return s.vec16 ? launch_dp4a<1, 8, 2, true>(p, s, L, stream) : launch_dp4a<1, 4, 1, false>(p, s, L, stream);
    case 2: return s.vec16 ? launch_dp4a<2, 4, 2, true>(p, s, L, stream) : launch_dp4a<2, 4, 1, false>(p, s, L, stream);
    case 8: return s.warps == 16 ? launch_nt<1, 16>(p, s, L, stream) : launch_nt<1, 8>(p, s, L, stream);
    case 16: return launch_nt<2, 8>(p, s, L, stream);
    default: return launch_nt<4, 8>(p, s, L, stream);
    }
}

}  // namespace loom
