// token_rows.cu -- operators over the rows of an activation matrix (sm_103a):
// tokens to signed bytes, layer norm (forward, forward to signed bytes,
// backward with the gradients of gain and bias).
//
// All are bound by the bytes of the rows, read once and written once.
//  * Forward and quantisation: a row is held in the registers of one CTA (one
//    warp for short rows), so mean, squares about the mean and largest magnitude
//    are taken from registers in turn, each with one reduction, and the row is
//    read once.  Rows beyond 32768 elements are read again for each pass (L2).
//  * Backward: CTAs walk over the rows; a thread keeps the same columns for all
//    of them, so the gain's and bias's gradients grow in its registers, and each
//    CTA leaves one partial sum per column in the workspace.  A second launch adds
//    the partial sums in a fixed order: no atomics, the same bits on every call.
//    Rows wider than 8192 take two passes: the two sums of each row, then blocks
//    of columns (dx alone: both in one launch, a row a CTA).
//  * CTAs walk over the rows and copy them ahead into a ring of shared memory (bulk copies),
//    two rows a turn.
//  * Loads are as wide as every row's start allows: 16 or 8 bytes, else one element.
//
// Measured (bf16 rows x width where no type is given; graph nodes)
//   layer norm 16384 x 8192       84 us, 6.4 TB/s (a copy of the same bytes: 79 us)
//              16384 x 2048       27 us, 4.9 TB/s: a turn's barriers for 8 KiB of rows
//              8000 x 5001        76 us, 2.1 TB/s; 4000 x 5001 f32 40 us, 4.0 TB/s: one element an access
//              2048 x 40000       133 us, 2.5 TB/s: the row read three times, from L2 where it still is there
//              8 x 2048 f32       2.5 us: the launch and three trips to memory
//   to bytes 8192 x 8192          32 us, 6.2 TB/s;  layer norm to bytes 61 us, 3.3 TB/s: three
//                                 reductions a row, one after the other, and what lies between
//   backward 16384 x 4096         75 us, 5.3 TB/s; 16384 x 2048 46 us; 8192 x 8192 83 us
//            1001 x 5001 f32      22 us, 2.7 TB/s: seven rows a CTA, then 12 MB of partial sums written
//                                 and read
//            4096 x 6144          42 us, 3.6 TB/s: 257 to 511 threads a row leave one CTA an SM
//            4096 x 12288         151 us, 2.0 TB/s: x and dy are read twice; dx alone 114 us
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int ROW_WARP_ROWS = 4;      // rows per CTA where a warp takes a whole row

// CTAs of `threads` threads that share an SM: 128 registers a thread.
int64_t rows_per_sm(int64_t threads) { return threads >= 512 ? 1 : 512 / threads; }

constexpr float TINY_AMAX = 7.888609052210118e-31f;   // 2^-100

template <typename E, int V> struct alignas(sizeof(E) * V) Pack {
    E e[V];
};

template <typename E, int V> __device__ __forceinline__ void load_f32(const E *p, float *v)
{
    const Pack<E, V> q = *reinterpret_cast<const Pack<E, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = dev::to_f32(q.e[i]);
}

template <typename E, int V> __device__ __forceinline__ void store_f32(E *p, const float *v)
{
    Pack<E, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i)
        q.e[i] = dev::from_f32<E>(v[i]);
    *reinterpret_cast<Pack<E, V> *>(p) = q;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(dev::FULL_MASK, v, m);
    return v;
}

// Sums over the CTA (or the warp where WARP) of N values at once, behind one barrier; `red` holds
// a float per value and warp and is not written again before every thread has read it.
template <int N, bool WARP> __device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[32])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum(v[i]);
    if (WARP)
        return;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            red[i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum(lane < warps ? red[i][lane] : 0.0f);
}

template <int N, bool WARP> __device__ __forceinline__ void group_maxima(uint32_t (&v)[N], float (*red)[32])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __reduce_max_sync(dev::FULL_MASK, v[i]);
    if (WARP)
        return;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            red[i][threadIdx.x >> 5] = __uint_as_float(v[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __reduce_max_sync(dev::FULL_MASK, lane < warps ? __float_as_uint(red[i][lane]) : 0u);
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The factor of a token's bytes, and its scale, from the bits of its largest magnitude
// (as whole numbers these order like the magnitudes, with NaN above infinity).
__device__ __forceinline__ float byte_factor(uint32_t amax_bits, float &scale, bool &bad)
{
    const float amax = __uint_as_float(amax_bits);
    bad = amax_bits >= 0x7f800000u;
    if (bad || amax < TINY_AMAX) {   // 127 / amax would leave f32 for the smallest
        scale = bad ? __uint_as_float(0x7fc00000u) : 0.0f;
        return 0.0f;
    }
    scale = __fdiv_rn(amax, 127.0f);
    return __fdiv_rn(127.0f, amax);
}

// Packed f32 pairs: two columns in one instruction, each rounded as on its own.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t both(float v) { return dev::pack2(v, v); }

// rint(v inv) of V values, |v inv| < 2^21: added to 1.5 2^23, the product's nearest whole number is in
// the low bits.  (The conversion instruction issues at a quarter of that rate: to bytes,
// 8192 x 8192 bf16 took 47 us by it, and 38 without.)
template <int V> __device__ __forceinline__ Pack<int8_t, V> to_bytes(const float *v, float inv, bool bad)
{
    uint32_t b[V];      // (in two roundings: of f32x2 instructions, product and sum may become one)
#pragma unroll
    for (int i = 0; i < V; ++i)
        b[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.0f));
    Pack<int8_t, V> o;
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint32_t w = __byte_perm(__byte_perm(b[i], b[i + 1], 0x0040), __byte_perm(b[i + 2], b[i + 3], 0x0040), 0x5410), q = bad ? 0u : w;
            memcpy(o.e + i, &q, 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            o.e[i] = bad ? (int8_t)0 : (int8_t)b[i];
    }
    return o;
}

__device__ __forceinline__ float halves_sum(uint64_t v)
{
    float a, b;
    dev::unpack2(v, a, b);
    return a + b;
}

// Column of element i of a thread's N: packs of V columns, `group` packs apart.
template <int V> __device__ __forceinline__ int column(int t, int group, int i) { return (t + i / V * group) * V + i % V; }

// V parameters of columns from c on (`dflt` where there are none).  Wide accesses give them 16
// bytes at a time, which the host has checked: every lane's own 32 bytes one float at a time
// would cost the L1 eight times the accesses.
template <int V> __device__ __forceinline__ void load_params(const float *p, int64_t c, float dflt, float *v)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = dflt;
    } else if (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p + c + i));
            v[i] = q.x;
            v[i + 1] = q.y;
            v[i + 2] = q.z;
            v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = __ldg(p + c + i);
    }
}

// ---- the read-ahead ring of a CTA that walks over rows ---------------------------------
// Rows are copied whole into a ring of shared memory, several ahead, by bulk copies; a row that
// does not start or end on 16 bytes is copied with the bytes around it that share its 16-byte
// blocks.  Blocks that reach past the first or the last row are not the caller's: such a row
// (and every row where there is no ring) is read with plain loads.  So is every row from then on
// when a wait for a copy runs out: the results are the same.  Threads may differ in when they see
// that; the one that issues the copies then issues no more, and waits, with a limit, for those in
// flight, so that none lands in a CTA that has ended.
constexpr uint64_t RING_WAIT_NS = 1000000000ull;
struct Ring {
    uint32_t slots, bars;       // shared-memory addresses
    uint32_t slot_bytes;
    int stages;                 // 0: no ring
    bool late;                  // a copy did not land in time: this thread uses the ring no more
};

template <typename E> struct RowSpan {
    const char *from;           // 16-byte block of the row's start
    uint32_t bytes, offset;     // of the blocks; of the row in them
    bool inside;
};

template <typename E> __device__ __forceinline__ RowSpan<E> span_of(const void *base, int64_t stride, int64_t rows, int32_t width, int64_t row)
{
    const uintptr_t first = reinterpret_cast<uintptr_t>(base), start = first + (uintptr_t)(row * stride) * sizeof(E);
    const uintptr_t end = start + (uintptr_t)width * sizeof(E);
    const uintptr_t last = first + (uintptr_t)((rows - 1) * stride + width) * sizeof(E);
    const uintptr_t lo = start & ~(uintptr_t)15, hi = (end + 15) & ~(uintptr_t)15;
    RowSpan<E> s;
    s.from = reinterpret_cast<const char *>(lo);
    s.bytes = (uint32_t)(hi - lo);
    s.offset = (uint32_t)(start - lo);
    s.inside = lo >= first && hi <= last;
    return s;
}

__device__ __forceinline__ Ring make_ring(const void *raw, int stages, uint32_t slot_bytes)
{
    Ring r;
    r.slots = dev::smem_u32(raw);
    r.slot_bytes = slot_bytes;
    r.bars = r.slots + (uint32_t)stages * slot_bytes;
    r.stages = stages;
    r.late = false;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i)
            dev::mbar_init(r.bars + 8 * i, 1);
        dev::fence_barrier_init();
    }
    __syncthreads();
    return r;
}

// By the issuing thread, once its rows are done: the copies that were in flight when it gave the ring up, from
// `slot` on (where a slot had none, this waits in vain), RING_WAIT_NS for them all.
__device__ __forceinline__ void ring_drain(const Ring &r, int slot, uint32_t parity)
{
    const uint64_t t0 = dev::global_ns();
    for (int i = 0; i < r.stages; ++i) {
        while (!dev::mbar_try_wait(r.bars + 8 * slot, parity) && dev::global_ns() - t0 < RING_WAIT_NS) {
        }
        if (++slot == r.stages) {
            slot = 0;
            parity ^= 1u;
        }
    }
}

// By one thread: the copies into the slot at `to`, completing on `bar`, of a turn's R rows from
// `row` on, of one or two matrices (b: NULL for one).  A slot is R rows of places of `place`
// bytes, one for each matrix.  Not inlined: its 64-bit arithmetic, for one thread, would cost all
// of them registers.
template <typename E, int R>
__device__ __noinline__ void ring_fill(uint32_t bar, uint32_t to, uint32_t place, const void *a, int64_t a_stride, const void *b, int64_t b_stride,
                                          int64_t rows, int32_t width, int64_t row, uint64_t policy)
{
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (row + i < rows) {
            const RowSpan<E> sa = span_of<E>(a, a_stride, rows, width, row + i);
            bytes += sa.inside ? sa.bytes : 0;
            if (b) {
                const RowSpan<E> sb = span_of<E>(b, b_stride, rows, width, row + i);
                bytes += sb.inside ? sb.bytes : 0;
            }
        }
    dev::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (row + i < rows) {
            const RowSpan<E> sa = span_of<E>(a, a_stride, rows, width, row + i);
            if (sa.inside)
                dev::bulk_g2s(to, sa.from, sa.bytes, bar, policy);
            to += place;
            if (b) {
                const RowSpan<E> sb = span_of<E>(b, b_stride, rows, width, row + i);
                if (sb.inside)
                    dev::bulk_g2s(to, sb.from, sb.bytes, bar, policy);
                to += place;
            }
        }
}

// The same for rows of whole 16-byte blocks, all inside: short enough to stand in the loop, where
// the one thread's way to the next barrier is everyone's (16384 x 8192 bf16, layer norm: 94 us by the
// call above, 84 by this).
template <typename E, int R>
__device__ __forceinline__ void ring_fill_whole(uint32_t bar, uint32_t to, uint32_t place, const void *a, int64_t a_stride, const void *b, int64_t b_stride,
                                                int64_t rows, int32_t width, int64_t row, uint64_t policy)
{
    const uint32_t bytes = (uint32_t)width * (uint32_t)sizeof(E), here = R == 1 || row + 1 < rows ? R : 1;
    static_assert(R <= 2, "rows of a turn");
    dev::mbar_arrive_expect_tx(bar, (b ? 2 : 1) * here * bytes);
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < (int)here) {
            dev::bulk_g2s(to + (uint32_t)i * (b ? 2 : 1) * place, static_cast<const E *>(a) + (row + i) * a_stride, bytes, bar, policy);
            if (b)
                dev::bulk_g2s(to + (uint32_t)(2 * i + 1) * place, static_cast<const E *>(b) + (row + i) * b_stride, bytes, bar, policy);
        }
}

template <typename E, int R, bool WHOLE>
__device__ __forceinline__ void ring_fill_rows(uint32_t bar, uint32_t to, uint32_t place, const void *a, int64_t a_stride, const void *b, int64_t b_stride,
                                               int64_t rows, int32_t width, int64_t row, uint64_t policy)
{
    if (WHOLE)
        ring_fill_whole<E, R>(bar, to, place, a, a_stride, b, b_stride, rows, width, row, policy);
    else
        ring_fill<E, R>(bar, to, place, a, a_stride, b, b_stride, rows, width, row, policy);
}

// Where a row is read: in the ring's slot or in memory.  A pointer for both, chosen once a row: a branch at
// each access takes 8000 x 5001 bf16 90 us (backward 144) where this takes 77 (113).
template <typename E> __device__ __forceinline__ const E *row_at(const Ring &r, uint32_t slot_at, const RowSpan<E> &s, const E *row)
{
    return r.stages && !r.late && s.inside ? reinterpret_cast<const E *>(__cvta_shared_to_generic(slot_at + s.offset)) : row;
}

// R rows at a time in the registers of a CTA, which walks over the rows, or one row in a warp's
// (WARP: several rows a CTA, no ring).  What bounds it beside the rows' bytes is instruction
// issue: many columns a thread and two rows a turn spread a turn's reductions over more
// elements, and pairs of columns share their arithmetic.  KEEP: the parameters stay in
// registers; read again for each row they are, for 16-bit rows, four times the row's own bytes.
template <typename E, RowMode M, int V, int EPT, int R, bool WARP, int THREADS, bool KEEP>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) rows_kernel(const RowsParams p, int stages, uint32_t place)
{
    constexpr int NV = EPT / V, NP = KEEP && M != RowMode::Quantize ? EPT : V;
    constexpr bool WHOLE = V * sizeof(E) == 16;             // rows of whole 16-byte blocks
    extern __shared__ __align__(16) unsigned char raw_ring[];
    __shared__ float red[2][3][R][32];
    const int group = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per_cta = WARP ? blockDim.x >> 5 : R;
    const int64_t step = (int64_t)gridDim.x * per_cta;
    int64_t row0 = (int64_t)blockIdx.x * per_cta + (WARP ? threadIdx.x >> 5 : 0);
    Ring ring = {};
    if (!WARP && stages)
        ring = make_ring(raw_ring, stages, R * place);
    dev::follow_previous_kernel();
    const uint64_t policy = dev::l2_evict_first_policy();
    if (!WARP && threadIdx.x == 0 && !p.inject_stall)
        for (int i = 0; i < stages && row0 + i * step < p.rows; ++i)
            ring_fill_rows<E, R, WHOLE>(ring.bars + 8 * i, ring.slots + (uint32_t)i * ring.slot_bytes, place, p.x, p.x_stride, nullptr, 0, p.rows, p.width,
                            row0 + i * step, policy);
    float gain[NP], bias[NP];
    if (KEEP && M != RowMode::Quantize)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (t + j * group) * V;
            if (c < p.width) {
                load_params<V>(p.gain, c, 1.0f, gain + (KEEP ? j * V : 0));
                load_params<V>(p.bias, c, 0.0f, bias + (KEEP ? j * V : 0));
            }
        }
    const float per_width = __fdiv_rn(1.0f, (float)p.width);
    int slot = 0, turn = 0;
    uint32_t parity = 0;
    for (; row0 < p.rows; row0 += step, turn ^= 1) {
        if (!WARP && stages && !ring.late)
            ring.late = !dev::mbar_wait_bounded(ring.bars + 8 * slot, parity, RING_WAIT_NS);
        float v[R][EPT];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r;
            const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
            RowSpan<E> span = {nullptr, 0, 0, true};
            if (!WARP && stages && !WHOLE)
                span = span_of<E>(p.x, p.x_stride, p.rows, p.width, row);
            const E *from = row_at<E>(ring, ring.slots + (uint32_t)slot * ring.slot_bytes + r * place, span, x);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * group) * V;
                if (c < p.width && row < p.rows)
                    load_f32<E, V>(from + c, v[r] + j * V);
                else
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        v[r][j * V + i] = 0.0f;
            }
        }
        // the slot is free behind the first reduction's barrier: every thread has read it
        auto refill = [&]() {
            if (!WARP && stages) {
                if (threadIdx.x == 0 && row0 + stages * step < p.rows && !ring.late)
                    ring_fill_rows<E, R, WHOLE>(ring.bars + 8 * slot, ring.slots + (uint32_t)slot * ring.slot_bytes, place, p.x, p.x_stride, nullptr, 0, p.rows,
                                    p.width, row0 + stages * step, policy);
                if (!ring.late && ++slot == stages) {     // (where late, the place to drain from)
                    slot = 0;
                    parity ^= 1u;
                }
            }
        };
        if (M != RowMode::Quantize) {
            float mean[R], rstd[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint64_t s = 0;
#pragma unroll
                for (int i = 0; i < EPT; i += 2)
                    s = dev::add2(s, dev::pack2(v[r][i], v[r][i + 1]));
                mean[r] = halves_sum(s);
            }
            group_sums<R, WARP>(mean, red[turn][0]);
            refill();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mean[r] *= per_width;
                const uint64_t m = both(mean[r]);
                uint64_t s = 0;
#pragma unroll
                for (int i = 0; i < EPT; i += 2) {
                    const uint64_t d = dev::sub2(dev::pack2(v[r][i], v[r][i + 1]), m);
                    dev::unpack2(d, v[r][i], v[r][i + 1]);       // from here on: about the mean
                    const bool in0 = column<V>(t, group, i) < p.width, in1 = column<V>(t, group, i + 1) < p.width;
                    if (V > 1) {
                        if (in0)                                 // packs are in or out as a whole
                            s = fma2(d, d, s);
                    } else {
                        const uint64_t q = dev::pack2(in0 ? v[r][i] : 0.0f, in1 ? v[r][i + 1] : 0.0f);
                        s = fma2(q, q, s);
                    }
                }
                rstd[r] = halves_sum(s);
            }
            group_sums<R, WARP>(rstd, red[turn][1]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                rstd[r] = rsqrtf(fmaf(rstd[r], per_width, p.eps));
                if (M == RowMode::Norm && t == 0 && row0 + r < p.rows) {
                    if (p.mean)
                        p.mean[row0 + r] = mean[r];
                    if (p.rstd)
                        p.rstd[row0 + r] = rstd[r];
                }
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * group) * V;
                if (c < p.width) {
                    if (!KEEP) {
                        load_params<V>(p.gain, c, 1.0f, gain);
                        load_params<V>(p.bias, c, 0.0f, bias);
                    }
                    const float *g = gain + (KEEP ? j * V : 0), *b = bias + (KEEP ? j * V : 0);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float *o = v[r] + j * V;
                        if constexpr (V == 1) {
                            o[0] = fmaf(o[0] * rstd[r], g[0], b[0]);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; i += 2)
                                dev::unpack2(fma2(mul2(dev::pack2(o[i], o[i + 1]), both(rstd[r])), dev::pack2(g[i], g[i + 1]), dev::pack2(b[i], b[i + 1])),
                                             o[i], o[i + 1]);
                        }
                        if (M == RowMode::Norm && row0 + r < p.rows)
                            store_f32<E, V>(static_cast<E *>(p.y) + (row0 + r) * p.y_stride + c, o);
                    }
                }
            }
        }
        if (M != RowMode::Norm) {
            uint32_t a[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                a[r] = 0;
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    if (M == RowMode::Quantize || column<V>(t, group, i) < p.width)     // (zeros past the tokens' width)
                        a[r] = max(a[r], magnitude_bits(v[r][i]));
            }
            group_maxima<R, WARP>(a, red[turn][2]);
            if (M == RowMode::Quantize)
                refill();
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row0 + r < p.rows) {
                    float scale;
                    bool bad;
                    const float inv = byte_factor(a[r], scale, bad);
                    if (t == 0) {
                        p.scale[row0 + r] = scale;
                        if (bad)
                            dev::flag_error(p.error, LOOM_DEVERR_NONFINITE);
                    }
                    int8_t *q = p.q + (row0 + r) * p.width;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int c = (t + j * group) * V;
                        if (c < p.width) {
                            *reinterpret_cast<Pack<int8_t, V> *>(q + c) = to_bytes<V>(v[r] + j * V, inv, bad);
                        }
                    }
                }
        }
    }
    if (!WARP && ring.late && threadIdx.x == 0 && !p.inject_stall)      // (a stalled test run has none in flight)
        ring_drain(ring, slot, parity);
}

// The same for rows of any length: each pass reads the row again.
template <typename E, RowMode M, int V> __global__ void __launch_bounds__(1024) long_rows_kernel(const RowsParams p)
{
    __shared__ float red[3][1][32];
    const int64_t row = blockIdx.x;
    dev::follow_previous_kernel();
    const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
    const int32_t c0 = threadIdx.x * V, step = blockDim.x * V;
    const float per_width = __fdiv_rn(1.0f, (float)p.width);
    float mean[1] = {0.0f}, rstd[1] = {0.0f}, v[V], gain[V], bias[V];
    if (M != RowMode::Quantize) {
        for (int64_t c = c0; c < p.width; c += step) {
            load_f32<E, V>(x + c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                mean[0] += v[i];
        }
        group_sums<1, false>(mean, red[0]);
        mean[0] *= per_width;
        for (int64_t c = c0; c < p.width; c += step) {
            load_f32<E, V>(x + c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                rstd[0] = fmaf(v[i] - mean[0], v[i] - mean[0], rstd[0]);
        }
        group_sums<1, false>(rstd, red[1]);
        rstd[0] = rsqrtf(fmaf(rstd[0], per_width, p.eps));
    }
    auto output = [&](int64_t c) {      // the row's values, normalised where it asks for that
        load_f32<E, V>(x + c, v);
        if (M != RowMode::Quantize) {
            load_params<V>(p.gain, c, 1.0f, gain);
            load_params<V>(p.bias, c, 0.0f, bias);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = fmaf((v[i] - mean[0]) * rstd[0], gain[i], bias[i]);
        }
    };
    if (M == RowMode::Norm) {
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean[0];
            if (p.rstd)
                p.rstd[row] = rstd[0];
        }
        for (int64_t c = c0; c < p.width; c += step) {
            output(c);
            store_f32<E, V>(static_cast<E *>(p.y) + row * p.y_stride + c, v);
        }
        return;
    }
    uint32_t a[1] = {0};
    for (int64_t c = c0; c < p.width; c += step) {
        output(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
            a[0] = max(a[0], magnitude_bits(v[i]));
    }
    float scale;
    bool bad;
    group_maxima<1, false>(a, red[2]);
    const float inv = byte_factor(a[0], scale, bad);
    if (threadIdx.x == 0) {
        p.scale[row] = scale;
        if (bad)
            dev::flag_error(p.error, LOOM_DEVERR_NONFINITE);
    }
    for (int64_t c = c0; c < p.width; c += step) {
        output(c);
        *reinterpret_cast<Pack<int8_t, V> *>(p.q + row * p.width + c) = to_bytes<V>(v, inv, bad);
    }
}

// Elements per thread and row: 16, two rows a turn, while 256 threads hold a row (so that two CTAs
// share an SM and one computes while the other waits); then 32, one row a turn, with up to 512
// threads of 128 registers, and at last 1024.
constexpr int ROW_EPT = 16, ROW_EPT_WIDE = 32;
inline int rows_ept(int32_t width) { return width <= 256 * ROW_EPT ? ROW_EPT : ROW_EPT_WIDE; }

// The ring of a CTA of which `per_sm` share an SM, with places of row_bytes (and the blocks around
// an unaligned row) for `rows_a_turn` rows of `matrices`: enough stages to keep 112 KiB of an SM in
// flight.  None where no CTA has a second turn.
constexpr int64_t RING_BYTES_SM = 112 * 1024, RING_MAX_STAGES = 8;
struct RingPlan {
    int stages;
    uint32_t place, smem_bytes;
};
RingPlan plan_ring(int64_t rows, int64_t grid, int64_t per_sm, int64_t row_bytes, int matrices, int rows_a_turn)
{
    RingPlan r = {0, 0, 0};
    const int64_t place = (row_bytes + 30) / 16 * 16, slot = place * matrices * rows_a_turn;
    int64_t stages = RING_BYTES_SM / (per_sm * slot);
    const int64_t turns = (rows + grid * rows_a_turn - 1) / (grid > 0 ? grid * rows_a_turn : 1);
    stages = stages < 2 ? 2 : stages > RING_MAX_STAGES ? RING_MAX_STAGES : stages;
    stages = stages < turns ? stages : turns;
    if (stages < 2 || per_sm * (stages * (slot + 8) + 3 * 1024) > 226 * 1024)
        return r;
    r.stages = (int)stages;
    r.place = (uint32_t)place;
    r.smem_bytes = (uint32_t)(stages * (slot + 8));
    return r;
}

// The rings of a launch of the geometry below (none where a warp takes a row).
RingPlan rows_ring(int64_t rows, int32_t width, int64_t row_bytes, const loom_launch &L)
{
    if (width <= 32 * ROW_EPT || L.kernel != LOOM_KERNEL_NORM_ROWS)
        return RingPlan{0, 0, 0};
    return plan_ring(rows, L.grid[0], rows_per_sm(L.block[0]), row_bytes, 1, (int)L.units_per_cta);
}

RingPlan norm_grad_ring(int64_t rows, int32_t width, int64_t row_bytes, const loom_launch &L)
{
    if (width <= 32 * NG_EPT || width > NG_MAX_WIDTH)
        return RingPlan{0, 0, 0};
    return plan_ring(rows, L.grid[0], rows_per_sm(L.block[0]), row_bytes, 2, (int)L.units_per_cta);
}

template <typename... K, typename P> cudaError_t launch_ring(void (*kernel)(K...), const loom_launch &L, const P &p, const RingPlan &r, std::atomic<uint64_t> &done,
                                                             cudaStream_t stream)
{
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), 0, done);
    return e != cudaSuccess ? e : launch_prepared(kernel, L, stream, p, r.stages, r.place);
}

template <typename E, RowMode M, int V, int EPT, int R, bool WARP, int THREADS, bool KEEP>
cudaError_t launch_rows_k(const RowsParams &p, const loom_launch &L, const RingPlan &r, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_ring(rows_kernel<E, M, V, EPT, R, WARP, THREADS, KEEP>, L, p, r, done, stream);
}

template <typename E, RowMode M, int V>
cudaError_t launch_rows_v(const RowsParams &p, const loom_launch &L, cudaStream_t stream)
{
    if (L.kernel == LOOM_KERNEL_NORM_LONG)
        return launch_with(long_rows_kernel<E, M, V>, L, stream, p);
    const RingPlan r = rows_ring(p.rows, p.width, (int64_t)p.width * (int64_t)sizeof(E), L);
    if (p.width <= 32 * ROW_EPT)
        return launch_rows_k<E, M, V, ROW_EPT, 1, true, 32 * ROW_WARP_ROWS, false>(p, L, r, stream);
    if (rows_ept(p.width) == ROW_EPT)
        return launch_rows_k<E, M, V, ROW_EPT, 2, false, 256, true>(p, L, r, stream);
    return p.width <= 512 * ROW_EPT_WIDE ? launch_rows_k<E, M, V, ROW_EPT_WIDE, 1, false, 512, true>(p, L, r, stream)
                                         : launch_rows_k<E, M, V, ROW_EPT_WIDE, 1, false, 1024, false>(p, L, r, stream);
}

template <typename E, int V>
cudaError_t launch_rows_m(const RowsParams &p, RowMode mode, const loom_launch &L, cudaStream_t stream)
{
    switch (mode) {
    case RowMode::Quantize: return launch_rows_v<E, RowMode::Quantize, V>(p, L, stream);
    case RowMode::Norm: return launch_rows_v<E, RowMode::Norm, V>(p, L, stream);
    default: return launch_rows_v<E, RowMode::NormI8, V>(p, L, stream);
    }
}

// ---- backward ------------------------------------------------------------------
// Rows of up to NG_MAX_WIDTH, R at a time: every thread keeps EPT columns of all the rows its CTA
// takes.
template <typename E, int V, int EPT, int R, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512, 1) norm_grad_kernel(const NormGradParams p, int stages, uint32_t place)
{
    constexpr int NV = EPT / V;
    constexpr bool WHOLE = V * sizeof(E) == 16;
    extern __shared__ __align__(16) unsigned char raw_ring[];   // WARP: [warps][2][width] f32 at the end
    __shared__ float red[2][2 * R][32];
    const int group = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int warps = blockDim.x >> 5, mine = WARP ? threadIdx.x >> 5 : 0;
    Ring ring = {};
    if (!WARP && stages)
        ring = make_ring(raw_ring, stages, 2 * R * place);
    uint64_t dg[EPT / 2], db[EPT / 2], gain[EPT / 2];         // pairs of columns
    dev::follow_previous_kernel();
    const int64_t step = (int64_t)gridDim.x * (WARP ? warps : R);
    int64_t row0 = (int64_t)blockIdx.x * (WARP ? warps : R) + mine;
    const uint64_t policy = dev::l2_evict_first_policy();
    if (!WARP && threadIdx.x == 0 && !p.inject_stall)
        for (int i = 0; i < stages && row0 + i * step < p.rows; ++i)
            ring_fill_rows<E, R, WHOLE>(ring.bars + 8 * i, ring.slots + (uint32_t)i * ring.slot_bytes, place, p.x, p.x_stride, p.dy, p.dy_stride, p.rows,
                            p.width, row0 + i * step, policy);
    {
        float g[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            g[i] = 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((t + j * group) * V < p.width)
                load_params<V>(p.gain, (t + j * group) * V, 1.0f, g + j * V);
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) {
            dg[i] = db[i] = 0;
            gain[i] = dev::pack2(g[2 * i], g[2 * i + 1]);
        }
    }
    // the rows' statistics, a turn ahead: a load of their own would stand at each turn's start
    float next_mean[R], next_rstd[R];
    auto stats = [&](int64_t first) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = first + r < p.rows;
            next_mean[r] = in ? p.mean[first + r] : 0.0f;
            next_rstd[r] = in ? p.rstd[first + r] : 0.0f;
        }
    };
    stats(row0);
    const float per_width = __fdiv_rn(1.0f, (float)p.width);
    int slot = 0, turn = 0;
    uint32_t parity = 0;
    for (; row0 < p.rows; row0 += step, turn ^= 1) {
        float rstd[R], sums[2 * R];
        uint64_t xh[R][EPT / 2], g[R][EPT / 2];               // xhat and dy * gain
        float mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = next_mean[r];
            rstd[r] = next_rstd[r];
        }
        stats(row0 + step);
        if (!WARP && stages && !ring.late)
            ring.late = !dev::mbar_wait_bounded(ring.bars + 8 * slot, parity, RING_WAIT_NS);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r;
            const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
            const E *dy = static_cast<const E *>(p.dy) + row * p.dy_stride;
            RowSpan<E> span_x = {nullptr, 0, 0, true}, span_dy = span_x;
            if (!WARP && stages && !WHOLE) {
                span_x = span_of<E>(p.x, p.x_stride, p.rows, p.width, row);
                span_dy = span_of<E>(p.dy, p.dy_stride, p.rows, p.width, row);
            }
            const uint32_t at = ring.slots + (uint32_t)slot * ring.slot_bytes + 2 * r * place;
            float xv[EPT], d[EPT];
            const E *from_x = row_at<E>(ring, at, span_x, x), *from_dy = row_at<E>(ring, at + place, span_dy, dy);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * group) * V;
                if (c < p.width && row < p.rows) {
                    load_f32<E, V>(from_x + c, xv + j * V);
                    load_f32<E, V>(from_dy + c, d + j * V);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        xv[j * V + i] = mean[r];
                        d[j * V + i] = 0.0f;
                    }
                }
            }
            const uint64_t m = both(mean[r]), rs = both(rstd[r]);
            uint64_t s1 = 0, s2 = 0;
#pragma unroll
            for (int i = 0; i < EPT / 2; ++i) {
                const uint64_t dy2 = dev::pack2(d[2 * i], d[2 * i + 1]);
                xh[r][i] = mul2(dev::sub2(dev::pack2(xv[2 * i], xv[2 * i + 1]), m), rs);
                g[r][i] = mul2(dy2, gain[i]);
                s1 = dev::add2(s1, g[r][i]);
                s2 = fma2(g[r][i], xh[r][i], s2);
                dg[i] = fma2(dy2, xh[r][i], dg[i]);
                db[i] = dev::add2(db[i], dy2);
            }
            sums[2 * r] = halves_sum(s1);
            sums[2 * r + 1] = halves_sum(s2);
        }
        if (p.dx || (!WARP && stages))
            group_sums<2 * R, WARP>(sums, red[turn]);      // behind its barrier the slot is free: every thread has read it
        if (!WARP && stages) {
            if (threadIdx.x == 0 && row0 + stages * step < p.rows && !ring.late)
                ring_fill_rows<E, R, WHOLE>(ring.bars + 8 * slot, ring.slots + (uint32_t)slot * ring.slot_bytes, place, p.x, p.x_stride, p.dy, p.dy_stride,
                                p.rows, p.width, row0 + stages * step, policy);
            if (!ring.late && ++slot == stages) {
                slot = 0;
                parity ^= 1u;
            }
        }
        if (p.dx)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row0 + r < p.rows) {
                    // dx = rstd (g - mean(g) - xhat mean(g xhat))
                    const uint64_t a = both(-(sums[2 * r] * per_width)), b = both(-(sums[2 * r + 1] * per_width)), rs = both(rstd[r]);
                    E *dx = static_cast<E *>(p.dx) + (row0 + r) * p.dx_stride;
                    float o[EPT];
#pragma unroll
                    for (int i = 0; i < EPT / 2; ++i)
                        dev::unpack2(mul2(fma2(xh[r][i], b, dev::add2(g[r][i], a)), rs), o[2 * i], o[2 * i + 1]);
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        if ((t + j * group) * V < p.width)
                            store_f32<E, V>(dx + (t + j * group) * V, o + j * V);
                }
    }
    if (!WARP && ring.late && threadIdx.x == 0 && !p.inject_stall)
        ring_drain(ring, slot, parity);
    if (!p.partial)
        return;
    float *out = p.partial + (int64_t)blockIdx.x * 2 * p.width;
    float *shared_sums = reinterpret_cast<float *>(raw_ring);
    float *mine_out = WARP ? shared_sums + (int64_t)mine * 2 * p.width : out;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int c = column<V>(t, group, i);
        float g[2], b[2];
        dev::unpack2(dg[i / 2], g[0], g[1]);
        dev::unpack2(db[i / 2], b[0], b[1]);
        if (c < p.width) {
            mine_out[c] = g[i % 2];
            mine_out[p.width + c] = b[i % 2];
        }
    }
    if (WARP) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.width; i += blockDim.x) {
            float s = 0.0f;
            for (int w = 0; w < warps; ++w)
                s += shared_sums[w * 2 * p.width + i];
            out[i] = s;
        }
    }
}

// dx of one element from its row's two means; the same bits in either kernel below.
__device__ __forceinline__ float dx_of(float d, float xhat, float gain, float rstd, float s1, float s2)
{
    return __fmul_rn(rstd, __fmaf_rn(-xhat, s2, __fmaf_rn(d, gain, -s1)));
}

// Rows wider than the registers of a CTA: the two sums of each row, and, where the columns' sums are
// not wanted (DX), its dx (the row is read again, from L2: no workspace) ...
template <typename E, int V, bool DX> __global__ void __launch_bounds__(1024) long_norm_sums_kernel(const NormGradParams p)
{
    __shared__ float red[2][32];
    const int64_t row = blockIdx.x;
    dev::follow_previous_kernel();
    const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
    const E *dy = static_cast<const E *>(p.dy) + row * p.dy_stride;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float sums[2] = {0.0f, 0.0f}, xv[V], d[V];
    for (int64_t c = threadIdx.x * V; c < p.width; c += blockDim.x * V) {
        float gain[V];
        load_params<V>(p.gain, c, 1.0f, gain);
        load_f32<E, V>(x + c, xv);
        load_f32<E, V>(dy + c, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float g = d[i] * gain[i];
            sums[0] += g;
            sums[1] = fmaf(g, (xv[i] - mean) * rstd, sums[1]);
        }
    }
    group_sums<2, false>(sums, red);
    const float s1 = __fdiv_rn(sums[0], (float)p.width), s2 = __fdiv_rn(sums[1], (float)p.width);
    if constexpr (!DX) {
        if (threadIdx.x == 0) {
            p.row_sums[2 * row] = s1;
            p.row_sums[2 * row + 1] = s2;
        }
    } else {
        // (behind the reduction's barrier every thread has read the row: dx may take its place)
        E *dx = static_cast<E *>(p.dx) + row * p.dx_stride;
        for (int64_t c = threadIdx.x * V; c < p.width; c += blockDim.x * V) {
            float gain[V];
            load_params<V>(p.gain, c, 1.0f, gain);
            load_f32<E, V>(x + c, xv);
            load_f32<E, V>(dy + c, d);
#pragma unroll
            for (int i = 0; i < V; ++i)
                d[i] = dx_of(d[i], (xv[i] - mean) * rstd, gain[i], rstd, s1, s2);
            store_f32<E, V>(dx + c, d);
        }
    }
}

// ... then a block of columns (blockIdx.x: there may be more than 65535, where a grid's y ends) of a
// share of the rows (blockIdx.y).
constexpr int NG_LONG_THREADS = 256;
template <typename E, int V>
__global__ void __launch_bounds__(NG_LONG_THREADS) long_norm_grad_kernel(const NormGradParams p)
{
    const int64_t c = ((int64_t)blockIdx.x * NG_LONG_THREADS + threadIdx.x) * V;
    dev::follow_previous_kernel();
    if (c >= p.width)
        return;
    float dg[V], db[V], gain[V];
    load_params<V>(p.gain, c, 1.0f, gain);
#pragma unroll
    for (int i = 0; i < V; ++i)
        dg[i] = db[i] = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float xv[V], d[V];
        load_f32<E, V>(static_cast<const E *>(p.x) + row * p.x_stride + c, xv);
        load_f32<E, V>(static_cast<const E *>(p.dy) + row * p.dy_stride + c, d);
        const float s1 = p.dx ? p.row_sums[2 * row] : 0.0f, s2 = p.dx ? p.row_sums[2 * row + 1] : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xh = (xv[i] - mean) * rstd;
            dg[i] = fmaf(d[i], xh, dg[i]);
            db[i] += d[i];
            d[i] = dx_of(d[i], xh, gain[i], rstd, s1, s2);
        }
        if (p.dx)
            store_f32<E, V>(static_cast<E *>(p.dx) + row * p.dx_stride + c, d);
    }
    float *out = p.partial + (int64_t)blockIdx.y * 2 * p.width + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        out[i] = dg[i];
        out[p.width + i] = db[i];
    }
}

// Partial column sums [parts][2 width] -> dgain, dbias: 32 columns per CTA, 32 threads per
// column over interleaved parts (the latency of a thread's chain of loads is what this takes),
// added in a fixed order.
constexpr int NG_SUM_COLS = 32, NG_SUM_GROUPS = 32;
__global__ void __launch_bounds__(NG_SUM_COLS *NG_SUM_GROUPS)
    norm_grad_columns_kernel(const float *partial, int64_t parts, int32_t width, float *dgain, float *dbias)
{
    __shared__ float part[NG_SUM_GROUPS][NG_SUM_COLS];
    const int col = threadIdx.x % NG_SUM_COLS, group = threadIdx.x / NG_SUM_COLS;
    const int64_t c = (int64_t)blockIdx.x * NG_SUM_COLS + col;
    dev::follow_previous_kernel();
    float s = 0.0f;
    if (c < 2 * (int64_t)width)
#pragma unroll 8
        for (int64_t q = group; q < parts; q += NG_SUM_GROUPS)
            s += partial[q * 2 * width + c];
    part[group][col] = s;
    __syncthreads();
    if (group == 0 && c < 2 * (int64_t)width) {
#pragma unroll 8
        for (int g = 1; g < NG_SUM_GROUPS; ++g)
            s += part[g][col];
        float *out = c < width ? dgain : dbias;
        if (out)
            out[c < width ? c : c - width] = s;
    }
}

template <typename E, int V, int EPT, int R, bool WARP>
cudaError_t launch_norm_grad_k(const NormGradParams &p, const loom_launch &L, const RingPlan &r, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_ring(norm_grad_kernel<E, V, EPT, R, WARP>, L, p, r, done, stream);
}

template <typename E, int V>
cudaError_t launch_norm_grad_v(const NormGradParams &p, const loom_launch &L, int64_t parts, cudaStream_t stream)
{
    const RingPlan r = norm_grad_ring(p.rows, p.width, (int64_t)p.width * (int64_t)sizeof(E), L);
    if (p.width <= 32 * NG_EPT)
        return launch_norm_grad_k<E, V, NG_EPT, 1, true>(p, L, r, stream);
    if (p.width <= NG_MAX_WIDTH)
        return p.width <= 256 * NG_EPT ? launch_norm_grad_k<E, V, NG_EPT, 2, false>(p, L, r, stream)
                                       : launch_norm_grad_k<E, V, 2 * NG_EPT, 1, false>(p, L, r, stream);
    if (p.dx) {
        if (!p.partial)
            return launch_with(long_norm_sums_kernel<E, V, true>, L, stream, p);
        const cudaError_t e = launch_with(long_norm_sums_kernel<E, V, false>, L, stream, p);
        if (e != cudaSuccess)
            return e;
    }
    loom_launch G = L;
    G.grid[0] = (uint32_t)((p.width / V + NG_LONG_THREADS - 1) / NG_LONG_THREADS);
    G.grid[1] = (uint32_t)parts;
    G.block[0] = NG_LONG_THREADS;
    return launch_with(long_norm_grad_kernel<E, V>, G, stream, p);
}

}  // namespace

int row_vec(int32_t dtype, int32_t width, const void *const *pointers, const int64_t *strides, int n)
{
    const int64_t size = dtype_bytes(dtype);
    for (int64_t bytes = 16; bytes > size; bytes >>= 1) {
        const int64_t v = bytes / size;
        if (v == 2)   // 4-byte loads of 16-bit pairs, 8-byte loads of f32 pairs: one element instead
            break;
        bool ok = width % v == 0;
        for (int i = 0; i < n && ok; ++i)
            ok = reinterpret_cast<uintptr_t>(pointers[i]) % bytes == 0 && strides[i] % v == 0;
        if (ok)
            return (int)v;
    }
    return 1;
}

bool rows_geometry(int64_t rows, int32_t width, int32_t dtype, int64_t sms, loom_launch *out)
{
    *out = loom_launch{};
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->kernel = LOOM_KERNEL_NORM_ROWS;
    out->units_per_cta = 1;
    int64_t threads, grid = rows;
    if (width <= 32 * ROW_EPT) {
        threads = 32 * ROW_WARP_ROWS;
        out->units_per_cta = ROW_WARP_ROWS;
        grid = (rows + ROW_WARP_ROWS - 1) / ROW_WARP_ROWS;
    } else if (width <= 1024 * 32) {
        const int ept = rows_ept(width);
        threads = ((int64_t)width + 32 * ept - 1) / (32 * ept) * 32;
        out->units_per_cta = ept == ROW_EPT ? 2 : 1;         // at a time
        const int64_t most = sms * rows_per_sm(threads);
        grid = (rows + out->units_per_cta - 1) / out->units_per_cta;
        grid = grid < most ? grid : most;
    } else {
        threads = 1024;
        out->kernel = LOOM_KERNEL_NORM_LONG;
    }
    if (grid > 0x7fffffff)
        return false;
    out->grid[0] = (uint32_t)grid;
    out->block[0] = (uint32_t)threads;
    out->smem_bytes = rows_ring(rows, width, width * dtype_bytes(dtype), *out).smem_bytes;
    return true;
}

cudaError_t launch_rows(const RowsParams &p, RowMode mode, int32_t dtype, int vec, const loom_launch &L,
                        cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return vec == 4 ? launch_rows_m<float, 4>(p, mode, L, stream) : launch_rows_m<float, 1>(p, mode, L, stream);
    if (dtype == LOOM_F16)
        return vec == 8   ? launch_rows_m<__half, 8>(p, mode, L, stream)
               : vec == 4 ? launch_rows_m<__half, 4>(p, mode, L, stream)
                          : launch_rows_m<__half, 1>(p, mode, L, stream);
    return vec == 8   ? launch_rows_m<__nv_bfloat16, 8>(p, mode, L, stream)
           : vec == 4 ? launch_rows_m<__nv_bfloat16, 4>(p, mode, L, stream)
                      : launch_rows_m<__nv_bfloat16, 1>(p, mode, L, stream);
}

// Rows at a time and threads of the launch that takes the column sums, and how many of its CTAs share an SM.
struct NormGradShape {
    int64_t rows, threads, per_sm;
};

static NormGradShape norm_grad_shape(int32_t width)
{
    if (width <= 32 * NG_EPT)
        return {8, 256, 4};
    if (width > NG_MAX_WIDTH)
        return {1, NG_LONG_THREADS, 1};
    const int64_t ept = width <= 256 * NG_EPT ? NG_EPT : 2 * NG_EPT, threads = ((int64_t)width + 32 * ept - 1) / (32 * ept) * 32;
    return {ept == NG_EPT ? 2 : 1, threads, rows_per_sm(threads)};
}

int64_t norm_grad_parts(int64_t rows, int32_t width, int64_t sms)
{
    const NormGradShape shape = norm_grad_shape(width);
    const int64_t turns = (rows + shape.rows - 1) / shape.rows, most = shape.per_sm * sms;
    return turns < most ? turns : most;
}

void norm_grad_geometry(int64_t rows, int32_t width, int32_t dtype, int64_t sms, loom_launch *out)
{
    const NormGradShape shape = norm_grad_shape(width);
    const bool wide = width > NG_MAX_WIDTH;            // the rows' own sums come first
    *out = loom_launch{};
    out->grid[0] = (uint32_t)(wide ? rows : norm_grad_parts(rows, width, sms));
    out->block[0] = (uint32_t)(wide ? 1024 : shape.threads);
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->kernel = LOOM_KERNEL_NORM_BACKWARD;
    out->units_per_cta = (uint32_t)shape.rows;
    out->smem_bytes = width <= 32 * NG_EPT ? (uint32_t)(8 * 2 * width * 4) : norm_grad_ring(rows, width, width * dtype_bytes(dtype), *out).smem_bytes;
}

int64_t norm_grad_workspace_bytes(int64_t rows, int32_t width, int64_t sms)
{
    return (norm_grad_parts(rows, width, sms) * 2 * width + (width > NG_MAX_WIDTH ? 2 * rows : 0)) * 4;
}

cudaError_t launch_norm_grad(const NormGradParams &p, int32_t dtype, int vec, const loom_launch &L, int64_t parts,
                             cudaStream_t stream)
{
    if (p.rows > 0) {
        cudaError_t e;
        if (dtype == LOOM_F32)
            e = vec == 4 ? launch_norm_grad_v<float, 4>(p, L, parts, stream) : launch_norm_grad_v<float, 1>(p, L, parts, stream);
        else if (dtype == LOOM_F16)
            e = vec == 8   ? launch_norm_grad_v<__half, 8>(p, L, parts, stream)
                : vec == 4 ? launch_norm_grad_v<__half, 4>(p, L, parts, stream)
                           : launch_norm_grad_v<__half, 1>(p, L, parts, stream);
        else
            e = vec == 8   ? launch_norm_grad_v<__nv_bfloat16, 8>(p, L, parts, stream)
                : vec == 4 ? launch_norm_grad_v<__nv_bfloat16, 4>(p, L, parts, stream)
                           : launch_norm_grad_v<__nv_bfloat16, 1>(p, L, parts, stream);
        if (e != cudaSuccess)
            return e;
    }
    if (!p.dgain && !p.dbias)
        return cudaSuccess;
    loom_launch S = L;
    S.grid[0] = (uint32_t)((2 * (int64_t)p.width + NG_SUM_COLS - 1) / NG_SUM_COLS);
    S.grid[1] = 1;
    S.block[0] = NG_SUM_COLS * NG_SUM_GROUPS;
    S.smem_bytes = 0;
    return launch_with(norm_grad_columns_kernel, S, stream, (const float *)p.partial, parts, p.width, p.dgain,
                       p.dbias);
}

}  // namespace loom
