// i4_matvec.cu -- products of a few 8-bit tokens with 4-bit weights that have a scale for each
// group along k, of one matrix or of the experts that each token goes to (sm_103a).
//
//   y[t][r] = sx[t] * sum_g s[r][g] a[t][r][g] + bias[r],  a = sum_{k in g} W[r][k] X[t][k]
//
// Design
//  * Bound: the n k / 2 bytes of W.  One CTA an SM takes an equal share of the rows (of all rows of
//    the experts that some pair names), so no partial sums leave a CTA and every row is read once.
//  * The tensor cores make the sums exact.  A weight's nibble is turned into w + 8 (one XOR) and its bits
//    are taken as a subnormal f16, (w + 8) 2^-24, or four places higher, (w + 8) 2^-20; those of the second kind
//    meet a token's byte / 16.  So eight weights cost five logic instructions and no conversion, and
//    every product is a whole multiple of 2^-24 whose sums over 128 k stay below 2^24 of them:
//    f16 MMAs (m16n8k16) with f32 sums lose nothing.  The 8 too many per weight is taken off by starting the sums
//    at -8 times the sum of the token's bytes.  (Rates measured, per SM and clock: f16 1000 products, s8
//    260, dp4a 256.)
//  * A warp takes 64 rows x 256 k at a time: 128 bytes of each row, copied ahead into its own ring of
//    shared memory (cp.async, 16 bytes; 4 where rows do not start on 16 bytes), 16-byte pieces swizzled by
//    row, so that ldmatrix hands each lane whole words of eight neighbouring weights without conflicts.  The
//    order of k inside an MMA follows from that and is the same for the tokens' bytes.
//  * The warps of a team (8 of them, fewer for short rows) share out k; each keeps f32 sums of its rows
//    for up to 32 tokens in registers over its part of k, adding a group's whole number times the
//    scale, and the team adds them up in a fixed order in shared memory.
//  * The experts' pairs are sorted by expert in each CTA (counts, a scan, lists in shared memory).  Which
//    column of an MMA a pair takes does not change its sums.
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int I4_WARPS = 8, I4_THREADS = 32 * I4_WARPS;
constexpr int I4_ROWS = 64, I4_CHUNK = 256;                      // of a stage: rows, k
constexpr int I4_STAGE = I4_ROWS * I4_CHUNK / 2;                 // bytes
constexpr int I4_HALF = 128;                                     // k between flushes of whole sums

struct I4Shape {          // of a launch
    int team;             // warps that share out k
    int depth;            // stages of a warp's ring, 2 or 3
    int vec16;            // rows of W start on 16 bytes
    int x8;               // rows of X start on 8 bytes
    int log_group;
    uint32_t scales, sums, lists;   // offsets in shared memory behind the rings
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

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

__device__ __forceinline__ uint32_t low_nibbles(uint32_t w) { return (w & 0x000f000fu) ^ 0x00080008u; }
__device__ __forceinline__ uint32_t high_nibbles(uint32_t w) { return (w & 0x00f000f0u) ^ 0x00800080u; }

// A scale's bits (read ahead), and its value times 2^24.
__device__ __forceinline__ uint32_t scale_bits(const void *s, int32_t dtype, int64_t at)
{
    return dtype == LOOM_F32 ? __ldg(static_cast<const uint32_t *>(s) + at) : (uint32_t)__ldg(static_cast<const unsigned short *>(s) + at);
}
__device__ __forceinline__ float scale_value(uint32_t bits, int32_t dtype)
{
    const float v = dtype == LOOM_F32 ? __uint_as_float(bits) : dtype == LOOM_F16 ? __half2float(__ushort_as_half((unsigned short)bits))
                                                                                  : __uint_as_float(bits << 16);
    return v * 16777216.0f;
}

// ---- what a CTA works on: runs of rows of one matrix, each with the pairs that want it ------------
struct Lists {                 // in shared memory, of the experts' products
    uint16_t *expert, *first;  // of each expert that some pair names (first: also behind the last): its first pair
    uint16_t *pair;            // sorted by expert, the missing ones last
    int experts, pairs;        // that are named; that are not missing
};

struct Unit {
    int64_t matrix_row;        // of the weights, counted over all matrices
    int row, rows;             // in its matrix
    int list, count;           // pairs: places in the list (or numbers)
};

struct Walk {
    int64_t begin, end;        // rows of the CTA, counted over the matrices that are wanted
    int64_t at;                // begin of the present run
    int q;                     // unit in it
    int columns, teams;
};

// The unit that the walk stands on; false past the last.
__device__ __forceinline__ bool unit_of(Walk &w, const I4Params &p, const Lists &l, Unit &u)
{
    while (w.at < w.end) {
        const int m = (int)(w.at / p.n), row0 = (int)(w.at % p.n);
        const int rows = (int)min((int64_t)(p.n - row0), w.end - w.at);
        const int first = p.ids ? l.first[m] : 0, pairs = p.ids ? l.first[m + 1] - first : p.pairs;
        const int passes = (pairs + w.columns - 1) / w.columns;
        const int parts = max((rows + I4_ROWS - 1) / I4_ROWS, min(w.teams, (rows + 15) / 16));
        if (w.q < parts * passes) {
            const int part = w.q / passes, pass = w.q % passes;
            const int r0 = (int)((int64_t)rows * part / parts), r1 = (int)((int64_t)rows * (part + 1) / parts);
            u.row = row0 + r0;
            u.rows = r1 - r0;
            u.matrix_row = (int64_t)(p.ids ? l.expert[m] : 0) * p.n + u.row;
            u.list = first + pass * w.columns;
            u.count = min(w.columns, pairs - pass * w.columns);
            return true;
        }
        w.q -= parts * passes;
        w.at += rows;
    }
    return false;
}

// Sorts the pairs by expert.  counts: [experts] words of scratch.
__device__ Lists make_lists(const I4Params &p, uint32_t *scratch)
{
    __shared__ uint32_t warp_sums[I4_WARPS], missing;
    Lists l;
    uint32_t *counts = scratch;
    l.expert = reinterpret_cast<uint16_t *>(counts + p.experts);
    l.first = l.expert + p.experts;
    l.pair = l.first + p.experts + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < p.experts; e += I4_THREADS)
        counts[e] = 0;
    if (tid == 0)
        missing = 0;
    __syncthreads();
    constexpr int MOST = I4_MAX_PAIRS / I4_THREADS;
    int expert[MOST];
    uint32_t rank[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int at = tid + i * I4_THREADS;
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
    // pairs in the low half, experts that have some in the high half
    constexpr int PER = I4_MAX_EXPERTS / I4_THREADS;
    uint32_t own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        own[i] = e < p.experts ? counts[e] : 0u;
        own[i] |= own[i] ? 0x10000u : 0u;
        sum += own[i];
    }
    uint32_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t up = __shfl_up_sync(dev::FULL_MASK, run, d);
        run += lane >= d ? up : 0u;
    }
    if (lane == 31)
        warp_sums[warp] = run;
    __syncthreads();
    uint32_t before = run - sum, all = 0;
#pragma unroll
    for (int i = 0; i < I4_WARPS; ++i) {
        before += i < warp ? warp_sums[i] : 0u;
        all += warp_sums[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < p.experts) {
            counts[e] = before & 0xffffu;
            if (own[i]) {
                l.expert[before >> 16] = (uint16_t)e;
                l.first[before >> 16] = (uint16_t)before;
            }
        }
        before += own[i];
    }
    l.pairs = (int)(all & 0xffffu);
    l.experts = (int)(all >> 16);
    if (tid == 0)
        l.first[l.experts] = (uint16_t)l.pairs;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int at = tid + i * I4_THREADS;
        if (at < p.pairs)
            l.pair[(expert[i] >= 0 ? counts[expert[i]] : (uint32_t)l.pairs) + rank[i]] = (uint16_t)at;
    }
    __syncthreads();
    return l;
}

// The copies of one stage: 128 bytes of up to 64 rows from k = chunk * 256 on.  What lies past the
// rows or past k is not copied: it meets zeros, or sums that are thrown away.
__device__ __forceinline__ void copy_stage(const I4Params &p, const I4Shape &s, const Unit &u, int chunk, uint32_t dst, int lane)
{
    const int64_t row_bytes = p.k / 2;
    const char *src = reinterpret_cast<const char *>(p.w) + u.matrix_row * row_bytes + chunk * (I4_CHUNK / 2);
    const int left = (int)min((int64_t)(I4_CHUNK / 2), row_bytes - (int64_t)chunk * (I4_CHUNK / 2));
    if (s.vec16) {
        const int piece = lane & 7, r0 = lane >> 3;
        if (16 * piece < left) {
#pragma unroll
            for (int i = 0; i < I4_ROWS / 4; ++i) {
                const int r = r0 + 4 * i;
                if (r < u.rows)
                    copy_async16(dst + r * 128 + ((piece ^ (r & 7)) << 4), src + r * row_bytes + 16 * piece);
            }
        }
    } else if (4 * lane < left) {
#pragma unroll 8
        for (int r = 0; r < u.rows; ++r)
            copy_async4(dst + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3), src + r * row_bytes + 4 * lane);
    }
}

// NT: MMA columns / 8; FL: MMA steps of 32 k between flushes (a group's, 4 at most).
template <int NT, int FL> __global__ void __launch_bounds__(I4_THREADS, 1) i4_matvec_kernel(const I4Params p, const I4Shape s)
{
    extern __shared__ __align__(128) unsigned char i4_shared[];
    constexpr int STEPS = I4_HALF / 32, FLUSHES = STEPS / FL;        // of half a stage
    constexpr int SP = 2 * FLUSHES;                                  // scales of a row in a stage
    constexpr int PAIR = NT == 1 ? 4 : NT == 2 ? 2 : 1;              // 16-row tiles whose MMAs overlap
    constexpr int SUM_STRIDE = 8 * NT + 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
    dev::follow_previous_kernel();

    Lists l = {};
    Walk walk;
    walk.teams = I4_WARPS / s.team;
    walk.columns = 8 * NT;
    if (p.ids) {
        l = make_lists(p, reinterpret_cast<uint32_t *>(i4_shared + s.lists));
        const int64_t rows = (int64_t)l.experts * p.n;
        walk.begin = rows * blockIdx.x / gridDim.x;
        walk.end = rows * (blockIdx.x + 1) / gridDim.x;
        for (int i = l.pairs; i < p.pairs; ++i) {                    // missing routes: rows of zeros
            const int64_t at = l.pair[i] * p.y_stride;
            for (int64_t r = (int64_t)blockIdx.x * I4_THREADS + threadIdx.x; r < p.n; r += (int64_t)gridDim.x * I4_THREADS)
                dev::store_as(p.y, p.y_dtype, at + r, 0.0f);
        }
    } else {
        walk.begin = (int64_t)p.n * blockIdx.x / gridDim.x;
        walk.end = (int64_t)p.n * (blockIdx.x + 1) / gridDim.x;
    }
    walk.at = walk.begin;
    walk.q = warp / s.team;
    const int part = warp % s.team;
    const int chunks = (p.k + I4_CHUNK - 1) / I4_CHUNK;
    const int c0 = chunks * part / s.team, c1 = chunks * (part + 1) / s.team;

    const uint32_t ring = dev::smem_u32(i4_shared) + warp * s.depth * I4_STAGE;
    float *scales = reinterpret_cast<float *>(i4_shared + s.scales) + warp * I4_ROWS * SP;
    float *sums = reinterpret_cast<float *>(i4_shared + s.sums);

    // the copies run `depth - 1` stages ahead of the products
    Walk ahead = walk;
    Unit next;
    bool more = unit_of(ahead, p, l, next);
    int next_chunk = c0, next_slot = 0;
    const auto copy_next = [&]() {
        while (more && next_chunk >= c1) {          // (no chunk at all: k = 0)
            ahead.q += ahead.teams;
            more = unit_of(ahead, p, l, next);
            next_chunk = c0;
            if (c0 >= c1)
                more = false;
        }
        if (more) {
            copy_stage(p, s, next, next_chunk, ring + next_slot * I4_STAGE, lane);
            ++next_chunk;
        }
        copies_commit();
        next_slot = next_slot + 1 == s.depth ? 0 : next_slot + 1;
    };
    for (int i = 1; i < s.depth; ++i)
        copy_next();

    int slot = 0;
    Unit u;
    for (; unit_of(walk, p, l, u); walk.q += walk.teams) {
        float acc[4][NT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][j][i] = 0.0f;
        const int8_t *xp[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int col = 8 * j + g;
            xp[j] = nullptr;
            if (col < u.count) {
                const int64_t row = p.ids ? l.pair[u.list + col] / p.pairs_per_x : u.list + col;
                xp[j] = p.x + row * p.k + 8 * tig;
            }
        }
        uint2 raw[STEPS][NT];
        const auto load_tokens = [&](int k0) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    raw[i][j] = make_uint2(0, 0);
                    if (xp[j] && k0 + 32 * i + 8 * tig < p.k) {
                        const int8_t *at = xp[j] + k0 + 32 * i;
                        if (s.x8)
                            raw[i][j] = __ldg(reinterpret_cast<const uint2 *>(at));
                        else
                            raw[i][j] = make_uint2(__ldg(reinterpret_cast<const uint32_t *>(at)), __ldg(reinterpret_cast<const uint32_t *>(at) + 1));
                    }
                }
        };
        uint32_t scale[2 * SP];
        const auto load_scales = [&](int chunk) {
#pragma unroll
            for (int i = 0; i < 2 * SP; ++i) {
                const int at = lane + 32 * i, row = min(at / SP, u.rows - 1);
                const int group = min((chunk * I4_CHUNK + at % SP * 32 * FL) >> s.log_group, p.groups - 1);
                scale[i] = scale_bits(p.scale_w, p.scale_dtype, (u.matrix_row + row) * p.groups + group);
            }
        };
        if (c0 < c1) {
            load_tokens(c0 * I4_CHUNK);
            load_scales(c0);
        }
        for (int c = c0; c < c1; ++c) {
            if (s.depth == 3)
                copies_wait<1>();
            else
                copies_wait<0>();
            __syncwarp();                    // the stage is there, and the last one read by all lanes
            copy_next();
#pragma unroll
            for (int i = 0; i < 2 * SP; ++i)
                scales[lane + 32 * i] = scale_value(scale[i], p.scale_dtype);
            if (c + 1 < c1)
                load_scales(c + 1);
            __syncwarp();
            const uint32_t stage = ring + slot * I4_STAGE;
            slot = slot + 1 == s.depth ? 0 : slot + 1;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int k0 = c * I4_CHUNK + h * I4_HALF;
                if (k0 >= p.k)
                    break;
                uint32_t b[STEPS][NT][4];
                float start[FLUSHES][NT][2];
#pragma unroll
                for (int f = 0; f < FLUSHES; ++f)
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
                        start[f][j][0] = (float)__shfl_sync(dev::FULL_MASK, sum, 8 * tig) * -4.76837158203125e-07f;      // -8 * 2^-24
                        start[f][j][1] = (float)__shfl_sync(dev::FULL_MASK, sum, 8 * tig + 4) * -4.76837158203125e-07f;
                    }
                if (k0 + I4_HALF < min(p.k, c1 * I4_CHUNK))
                    load_tokens(k0 + I4_HALF);
#pragma unroll
                for (int t0 = 0; t0 < 4; t0 += PAIR) {
                    if (16 * t0 >= u.rows)
                        break;
                    uint32_t w[PAIR][4];
#pragma unroll
                    for (int f = 0; f < FLUSHES; ++f) {
                        float sum[PAIR][NT][4];
#pragma unroll
                        for (int t = 0; t < PAIR; ++t)
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                sum[t][j][0] = sum[t][j][2] = start[f][j][0];
                                sum[t][j][1] = sum[t][j][3] = start[f][j][1];
                            }
#pragma unroll
                        for (int i = f * FL; i < (f + 1) * FL; ++i)
#pragma unroll
                            for (int t = 0; t < PAIR; ++t) {
                                if (i % 2 == 0) {       // two steps (16-byte pieces) of 16 rows at a time
                                    const int row = 16 * (t0 + t) + (lane & 15), piece = 4 * h + i + (lane >> 4);
                                    load_matrices(w[t], stage + row * 128 + ((piece ^ (row & 7)) << 4));
                                }
                                const uint32_t w0 = w[t][2 * (i % 2)], w1 = w[t][2 * (i % 2) + 1];
                                const uint32_t a0 = low_nibbles(w0), a1 = low_nibbles(w1), a2 = high_nibbles(w0), a3 = high_nibbles(w1);
                                const uint32_t e0 = low_nibbles(w0 >> 8), e1 = low_nibbles(w1 >> 8), e2 = high_nibbles(w0 >> 8),
                                               e3 = high_nibbles(w1 >> 8);
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    mma(sum[t][j], a0, a1, a2, a3, b[i][j][0], b[i][j][1]);
                                    mma(sum[t][j], e0, e1, e2, e3, b[i][j][2], b[i][j][3]);
                                }
                            }
#pragma unroll
                        for (int t = 0; t < PAIR; ++t) {
                            const int at = (16 * (t0 + t) + g) * SP + h * FLUSHES + f;
                            const float s0 = scales[at], s1 = scales[at + 8 * SP];
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
            }
        }
        // the team's sums, 16 rows at a time
        const int team_thread = threadIdx.x % (32 * s.team), barrier = 1 + warp / s.team;
        float *own = sums + warp * 16 * SUM_STRIDE, *first = sums + (warp - part) * 16 * SUM_STRIDE;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (16 * t >= u.rows)
                break;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float *at = own + g * SUM_STRIDE + 8 * j + 2 * tig;
                *reinterpret_cast<float2 *>(at) = make_float2(acc[t][j][0], acc[t][j][1]);
                *reinterpret_cast<float2 *>(at + 8 * SUM_STRIDE) = make_float2(acc[t][j][2], acc[t][j][3]);
            }
            asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * s.team) : "memory");
            for (int i = team_thread; i < 128 * NT; i += 32 * s.team) {
                const int row = i & 15, col = i >> 4;
                if (16 * t + row < u.rows && col < u.count) {
                    float y = 0.0f;
                    for (int w = 0; w < s.team; ++w)
                        y += first[(16 * w + row) * SUM_STRIDE + col];
                    const int64_t pair = p.ids ? l.pair[u.list + col] : u.list + col;
                    y *= __ldg(p.scale_x + pair / p.pairs_per_x);
                    if (p.bias)
                        y = __fadd_rn(y, __ldg(p.bias + u.matrix_row + 16 * t + row));
                    dev::store_as(p.y, p.y_dtype, pair * p.y_stride + u.row + 16 * t + row, y);
                }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * s.team) : "memory");
        }
    }
    copies_wait<0>();
}

template <int NT, int FL>
cudaError_t launch_one(const I4Params &p, const I4Shape &s, const loom_launch &L, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(i4_matvec_kernel<NT, FL>), 0, done);
    return e != cudaSuccess ? e : launch_prepared(i4_matvec_kernel<NT, FL>, L, stream, p, s);
}

template <int NT> cudaError_t launch_nt(const I4Params &p, const I4Shape &s, const loom_launch &L, cudaStream_t stream)
{
    return p.group == 32 ? launch_one<NT, 1>(p, s, L, stream) : p.group == 64 ? launch_one<NT, 2>(p, s, L, stream) : launch_one<NT, 4>(p, s, L, stream);
}

// MMA columns / 8: for the pairs that a matrix has, on average half as many again.
int i4_columns(int64_t pairs, int64_t experts)
{
    const int64_t each = experts ? (3 * pairs + 2 * experts - 1) / (2 * experts) : pairs;
    return each <= 8 ? 1 : each <= 16 ? 2 : 4;
}

// Shared memory of a launch (the static arrays of make_lists are counted as 256 bytes).
uint32_t i4_smem(int64_t pairs, int64_t k, int64_t group, int64_t experts, I4Shape *s)
{
    const int nt = i4_columns(pairs, experts);
    const int64_t chunks = (k + I4_CHUNK - 1) / I4_CHUNK;
    s->team = chunks >= 8 ? 8 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
    const uint32_t scales = I4_WARPS * I4_ROWS * 4 * (group == 32 ? 8 : group == 64 ? 4 : 2), sums = I4_WARPS * 16 * (8 * nt + 2) * 4;
    const uint32_t lists = experts ? (uint32_t)(((8 * experts + 2 + 2 * pairs) + 15) / 16 * 16) : 0;
    const uint32_t rest = scales + sums + lists;
    s->depth = 3 * I4_WARPS * I4_STAGE + rest + 256 <= 227 * 1024 ? 3 : 2;
    s->scales = (uint32_t)(s->depth * I4_WARPS * I4_STAGE);
    s->sums = s->scales + scales;
    s->lists = s->sums + sums;
    return s->lists + lists;
}

}  // namespace

void i4_geometry(int64_t pairs, int64_t n, int64_t k, int64_t group, int64_t experts, int64_t sms, loom_launch *out)
{
    I4Shape s;
    *out = loom_launch{};
    out->smem_bytes = i4_smem(pairs, k, group, experts, &s);
    const int64_t most = (experts ? experts : 1) * n;
    out->grid[0] = (uint32_t)(most < sms ? (most > 0 ? most : 1) : sms);
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->block[0] = I4_THREADS;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    const int64_t rows = (most + out->grid[0] - 1) / out->grid[0];
    out->units_per_cta = (uint32_t)(rows < 0xffffffffll ? rows : 0xffffffffll);
    out->kernel = LOOM_KERNEL_I4_MATVEC;
}

cudaError_t launch_i4_matvec(const I4Params &p, const loom_launch &L, cudaStream_t stream)
{
    I4Shape s;
    const int32_t experts = p.ids ? (p.experts > 0 ? p.experts : 1) : 0;
    i4_smem(p.pairs, p.k, p.group, experts, &s);
    s.vec16 = p.k % 32 == 0 && reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    s.x8 = reinterpret_cast<uintptr_t>(p.x) % 8 == 0;
    s.log_group = 5;
    while (s.log_group < 30 && (1 << s.log_group) < p.group)
        ++s.log_group;
    switch (i4_columns(p.pairs, experts)) {
    case 1: return launch_nt<1>(p, s, L, stream);
    case 2: return launch_nt<2>(p, s, L, stream);
    default: return launch_nt<4>(p, s, L, stream);
    }
}

}  // namespace loom
