// i8_matmul.cu -- matrix product of 8-bit tokens and 8-bit weights for few
// tokens: dp4a, the weights streamed once for up to eight tokens (sm_103a).
//
//   acc[t][r] = sum_k W[r][k] X[t][k],  y[t][r] = (float)acc * (sw[r] * sx[t]) + bias[r]
//
// Design
//  * Bound: the n k bytes of W.  A pass takes up to eight tokens (grid.y), each
//    CTA ceil(n / (2 SMs)) whole rows, so no partial sums leave a CTA.
//  * A CTA's work is a list of items -- one chunk of k (KV x 512 bytes, 16 bytes
//    a lane) of R rows -- ordered chunk by chunk and cut into equal ranges, one
//    per warp.  A lane keeps its pieces of all T tokens' chunk in registers over
//    the items of that chunk, so a token's bytes are read once per chunk and
//    warp, not once per row, and R x KV independent 16-byte loads are in flight.
//  * The R x T sums of an item are reduced over the lanes by a butterfly that
//    halves the values a lane carries at each step (R T + few shuffles instead of
//    5 R T) and added to the CTA's totals in shared memory: int32 additions, so
//    their order does not matter.
//  * Rows that are not whole 16-byte pieces (k % 16 != 0, or pointers that are
//    not 16-byte aligned) take the same path with 4-byte loads.
//
//  * Two CTAs share an SM for any number of tokens (128 registers a thread: alone, 8 tokens
//    took 70 us below).
//
// Measured: 8192 x 16384 for 1 token in 20.9 us, the 134 MB of weights at 6.4 TB/s; 4 tokens 25.6 us,
// 8 tokens 43 us (instruction issue: 32 dp4a for each 16 bytes of weights).
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int DP_WARPS = 8;

// 16 bytes of a row for this lane: chunk piece `piece` (512 bytes a warp) at
// `p`, zero past `left` bytes of the row.  V16: lane l holds bytes 16 l .. 16 l + 15;
// else words l, l + 32, l + 64, l + 96 of the piece -- any split of k over lanes
// gives the same sums as long as tokens and weights use the same one.
template <bool V16>
__device__ __forceinline__ int4 load_piece(const int8_t *p, int64_t left, int lane, bool stream)
{
    int4 v = make_int4(0, 0, 0, 0);
    if (V16) {
        if (16 * lane < left) {
            const int4 *q = reinterpret_cast<const int4 *>(p) + lane;
            v = stream ? __ldcs(q) : *q;
        }
    } else {
        const int32_t *q = reinterpret_cast<const int32_t *>(p) + lane;
        int32_t *o = &v.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * (lane + 32 * j) < left)
                o[j] = stream ? __ldcs(q + 32 * j) : q[32 * j];
    }
    return v;
}

__device__ __forceinline__ int32_t dot16(const int4 &a, const int4 &b, int32_t c)
{
    c = __dp4a(a.x, b.x, c);
    c = __dp4a(a.y, b.y, c);
    c = __dp4a(a.z, b.z, c);
    return __dp4a(a.w, b.w, c);
}

// Sums of N (a power of two, <= 32) values over the warp: afterwards v[0] of
// lane l is the sum of value l / (32 / N).
template <int N> __device__ __forceinline__ void warp_sums(int32_t (&v)[N], int lane)
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
                    const int32_t send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(dev::FULL_MASK, send, m);
                }
        } else {
            v[0] += __shfl_xor_sync(dev::FULL_MASK, v[0], m);
        }
    }
}

template <int T, int KV, int R, bool V16>
__global__ void __launch_bounds__(32 * DP_WARPS, 2) i8_matmul_dp4a_kernel(const MatmulParams p)
{
    extern __shared__ int32_t totals[];   // [rows_per_cta][T]
    constexpr int CHUNK = KV * 512;
    static_assert(R * T <= 32, "one value per lane");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * p.rows_per_cta;
    const int rows = (int)min((int64_t)p.rows_per_cta, p.n - row0);
    dev::follow_previous_kernel();
    for (int64_t pass = blockIdx.y; pass * MM_DP4A_PASS < p.tokens; pass += gridDim.y) {
        const int token0 = (int)(pass * MM_DP4A_PASS), nt = min(T, p.tokens - token0);
        for (int i = threadIdx.x; i < rows * T; i += 32 * DP_WARPS)
            totals[i] = 0;
        __syncthreads();
        const int groups = (rows + R - 1) / R, chunks = (p.k + CHUNK - 1) / CHUNK;
        const int64_t items = (int64_t)groups * chunks;
        const int64_t first = items * warp / DP_WARPS, last = items * (warp + 1) / DP_WARPS;
        int4 xv[T][KV];
        int held = -1;
        for (int64_t it = first; it < last; ++it) {
            const int c = (int)(it / groups), g = (int)(it % groups);
            const int64_t k0 = (int64_t)c * CHUNK;
            int4 wv[R][KV];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < KV; ++j)
                    wv[r][j] = load_piece<V16>(p.w + (row0 + g * R + r) * p.k + k0 + 512 * j,
                                               g * R + r < rows ? p.k - k0 - 512 * j : 0, lane, true);
            if (c != held) {
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int j = 0; j < KV; ++j)
                        xv[t][j] = load_piece<V16>(p.x + (int64_t)(token0 + t) * p.k + k0 + 512 * j,
                                                   t < nt ? p.k - k0 - 512 * j : 0, lane, false);
                held = c;
            }
            int32_t v[R * T];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    int32_t s = 0;
#pragma unroll
                    for (int j = 0; j < KV; ++j)
                        s = dot16(wv[r][j], xv[t][j], s);
                    v[r * T + t] = s;
                }
            warp_sums<R * T>(v, lane);
            constexpr int SPAN = 32 / (R * T);
            const int at = g * R * T + lane / SPAN;   // (row, token) of this lane's sum
            if (lane % SPAN == 0 && at < rows * T)
                atomicAdd(totals + at, v[0]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * nt; i += 32 * DP_WARPS) {
            const int t = i / rows, r = i % rows;
            const int64_t row = row0 + r, token = token0 + t;
            const int32_t a = totals[r * T + t];
            if (p.acc)
                p.acc[token * p.n + row] = a;
            dev::store_as(p.y, p.y_dtype, token * p.y_stride + row,
                          dev::dequantized(a, __ldg(p.scale_w + row), p.scale_x[token], p.bias, row));
        }
        __syncthreads();   // before the totals are cleared
    }
}

template <int T, int KV, int R>
cudaError_t launch_t(const MatmulParams &p, bool vec16, const loom_launch &L, cudaStream_t stream)
{
    return vec16 ? launch_with(i8_matmul_dp4a_kernel<T, KV, R, true>, L, stream, p)
                 : launch_with(i8_matmul_dp4a_kernel<T, KV, R, false>, L, stream, p);
}

}  // namespace

cudaError_t launch_matmul_dp4a(const MatmulParams &p, bool vec16, const loom_launch &L, cudaStream_t stream)
{
    switch (matmul_dp4a_tokens(p.tokens)) {
    case 1: return launch_t<1, 4, 4>(p, vec16, L, stream);
    case 2: return launch_t<2, 4, 4>(p, vec16, L, stream);
    case 4: return launch_t<4, 2, 4>(p, vec16, L, stream);
    default: return launch_t<MM_DP4A_PASS, 1, 4>(p, vec16, L, stream);
    }
}

}  // namespace loom
