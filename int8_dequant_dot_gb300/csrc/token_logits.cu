// token_logits.cu -- logits adjusted before a token is chosen: penalties for tokens that were
// seen, biases, a grammar's mask (sm_103a).
//
// Design
//  * Bound: a row's logits in and out.  A row is cut into slices, a CTA each, whose loads of logits are all in flight
//    while it finds out what its tokens have coming: nothing but the history and the bias list
//    stands between a logit's load and its store.
//  * A slice's marks are one word a token in shared memory:
//      bits 0..19 occurrences behind the prompt, bit 20 seen in the prompt, bits 21..31 the bias entry
//    (AL_ENTRY - its place, so that a maximum finds the first of several).  Additions and maxima of whole numbers:
//    their order does not matter.  Every CTA of a row reads all of the row's history and keeps what is its
//    own; that is L2 traffic alone, 1 / 16 of the logits' for a history of 4096 tokens.
//  * Logits without a mark (nearly all) pass as bits.
//  * Slices are cut at 16-byte boundaries of the row's memory, wherever it starts; a row whose copy starts elsewhere in
//    its 16 bytes is taken one element at a time.
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int AL_THREADS = 512;
constexpr int AL_SLICE = 16384;              // most tokens of a slice: 64 KiB of marks, two CTAs an SM
constexpr int AL_LEAST = 2048;               // fewest
constexpr int AL_BATCH = 8;                  // history tokens that a thread loads together
constexpr uint32_t AL_SEEN = 1u << 20, AL_COUNT = AL_SEEN - 1u, AL_ENTRY = 2047;

struct RowSettings {
    float repetition, frequency, presence;
    int length, prompt;
    const uint32_t *mask;    // or NULL
};

__device__ __forceinline__ RowSettings settings_of(const AdjustParams &p, int64_t row, bool report)
{
    RowSettings s;
    s.repetition = p.d_repetition ? p.d_repetition[row] : p.repetition;
    if (!(s.repetition > 0.0f))
        s.repetition = 1.0f;
    s.frequency = p.d_frequency ? p.d_frequency[row] : p.frequency;
    s.presence = p.d_presence ? p.d_presence[row] : p.presence;
    s.length = p.history;
    bool wrong = false;
    if (p.tokens && p.lengths) {
        const int len = p.lengths[row];
        wrong = len < 0 || len > p.history;
        s.length = min(max(len, 0), p.history);
    }
    s.prompt = p.prompts ? min(max(p.prompts[row], 0), s.length) : 0;
    s.mask = nullptr;
    if (p.mask) {
        int64_t m = p.mask_rows ? p.mask_rows[row] : p.masks == 1 ? 0 : row;
        if (m >= p.masks) {
            wrong = true;
            m = -1;
        }
        s.mask = m < 0 ? nullptr : reinterpret_cast<const uint32_t *>(p.mask) + m * ((p.vocab + 31) / 32);
    }
    if (wrong && report && threadIdx.x == 0)
        dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
    return s;
}

__device__ __forceinline__ float adjusted(float l, uint32_t mark, const RowSettings &s, const float *bias)
{
    const uint32_t count = mark & AL_COUNT;
    if (count || (mark & AL_SEEN))
        l = l > 0.0f ? __fdiv_rn(l, s.repetition) : __fmul_rn(l, s.repetition);
    if (count)
        l = __fsub_rn(__fsub_rn(l, __fmul_rn(s.frequency, (float)count)), s.presence);
    if (mark >> 21)
        l = __fadd_rn(l, bias[AL_ENTRY - (mark >> 21)]);
    return l;
}

// The marks of the tokens from `first` on, `n` of them; zeroed before.
__device__ __forceinline__ void set_marks(const AdjustParams &p, const RowSettings &s, int64_t row, uint32_t *marks, uint32_t first, uint32_t n)
{
    const int32_t *tokens = p.tokens + row * p.history_stride;
    for (int i0 = threadIdx.x; i0 < s.length; i0 += AL_BATCH * AL_THREADS) {
        uint32_t at[AL_BATCH];
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j) {
            const int i = i0 + j * AL_THREADS;
            at[j] = i < s.length ? (uint32_t)__ldg(tokens + i) : 0xffffffffu;      // (-1)
        }
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j) {
            const uint32_t t = at[j] - first;       // (those outside the row meet words that nothing reads)
            if (t < n && (int32_t)at[j] >= 0) {
                if (i0 + j * AL_THREADS < s.prompt)
                    atomicOr(marks + t, AL_SEEN);
                else
                    atomicAdd(marks + t, 1u);
            }
        }
    }
    if (p.biases == 0)
        return;
    __syncthreads();
    const int32_t *ids = p.bias_ids + row * p.biases;
    for (int i = threadIdx.x; i < p.biases; i += AL_THREADS) {
        const int32_t id = __ldg(ids + i);
        const uint32_t t = (uint32_t)id - first;
        if (id >= 0 && t < n)
            atomicMax(marks + t, (marks[t] & (AL_SEEN | AL_COUNT)) | ((AL_ENTRY - (uint32_t)i) << 21));
    }
}

template <typename E, int N> struct alignas(sizeof(E) * N) Pack {
    E e[N];
};

// N: elements of an access, 16 bytes or one.  U: accesses of a thread.
template <typename E, int N, int U, bool MARKS>
__global__ void __launch_bounds__(AL_THREADS, 2) adjust_kernel(const AdjustParams p, int slices)
{
    extern __shared__ __align__(16) uint32_t al_marks[];
    constexpr int SLICE = AL_THREADS * N * U;
    typedef Pack<E, N> P;
    if (MARKS)
        for (int i = threadIdx.x; i < SLICE / 4; i += AL_THREADS)
            reinterpret_cast<uint4 *>(al_marks)[i] = make_uint4(0, 0, 0, 0);
    dev::follow_previous_kernel();
    const int64_t row = blockIdx.x / (unsigned)slices;
    const int slice = (int)(blockIdx.x - row * slices);
    const E *x = static_cast<const E *>(p.logits) + row * p.stride;
    E *y = static_cast<E *>(p.y) + row * p.y_stride;
    const bool in_place = x == y;
    const int first = slice * SLICE - (int)(reinterpret_cast<uintptr_t>(x) / sizeof(E) % N);     // the slice's first token
    const auto whole = [&](int t) { return t >= 0 && t <= p.vocab - N; };
    P v[U];
    if (!in_place) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = first + ((int)threadIdx.x + u * AL_THREADS) * N;
            if (whole(t))
                v[u] = *reinterpret_cast<const P *>(x + t);
        }
    }
    const RowSettings s = settings_of(p, row, slice == 0);
    const float *bias = p.bias_values + row * p.biases;
    if (MARKS) {
        __syncthreads();
        set_marks(p, s, row, al_marks, (uint32_t)first, SLICE);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = ((int)threadIdx.x + u * AL_THREADS) * N, t = first + at;
        if (t >= p.vocab || t <= -N)
            continue;
        uint32_t mark[N], any = 0;
        if (MARKS) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (N % 4 == 0) {
                    if (i % 4 == 0)
                        *reinterpret_cast<uint4 *>(mark + i) = *reinterpret_cast<const uint4 *>(al_marks + at + i);
                } else {
                    mark[i] = al_marks[at + i];
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                any |= mark[i];
        }
        uint32_t masked = 0;                    // a bit for each token that may not be chosen
        if (s.mask) {
            const int t0 = max(t, 0), word = t0 >> 5;
            uint32_t low = __ldg(s.mask + word), high = 0;
            if ((t0 & 31) + N > 32 && word + 1 < (p.vocab + 31) / 32)
                high = __ldg(s.mask + word + 1);
            masked = ~(__funnelshift_r(low, high, t0 & 31) << (t0 - t));
        }
        if (whole(t)) {
            if (in_place) {
                if (!any && !(masked & (N < 32 ? (1u << (N % 32)) - 1u : ~0u)))
                    continue;
                v[u] = *reinterpret_cast<const P *>(x + t);
            }
            if (MARKS && any)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (mark[i])
                        v[u].e[i] = dev::from_f32<E>(adjusted(dev::to_f32(v[u].e[i]), mark[i], s, bias));
            if (s.mask)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if ((masked >> i) & 1)
                        v[u].e[i] = dev::from_f32<E>(-INFINITY);
            *reinterpret_cast<P *>(y + t) = v[u];
        } else {                                // the row's first or last tokens
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (t + i >= 0 && t + i < p.vocab) {
                    E l = x[t + i];
                    if (MARKS && mark[i])
                        l = dev::from_f32<E>(adjusted(dev::to_f32(l), mark[i], s, bias));
                    y[t + i] = s.mask && ((masked >> i) & 1) ? dev::from_f32<E>(-INFINITY) : l;
                }
        }
    }
}

template <typename E, int N, int U, bool MARKS> cudaError_t launch_one(const AdjustParams &p, loom_launch L, int slices, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(adjust_kernel<E, N, U, MARKS>), 0, done);
    if (e != cudaSuccess)
        return e;
    L.grid[0] = (uint32_t)(p.rows * slices);
    L.smem_bytes = MARKS ? AL_THREADS * N * U * 4 : 0;
    return launch_prepared(adjust_kernel<E, N, U, MARKS>, L, stream, p, slices);
}

template <typename E, int N, int U> cudaError_t launch_u(const AdjustParams &p, const loom_launch &L, cudaStream_t stream)
{
    constexpr int SLICE = AL_THREADS * N * U;
    // rows that do not all start on an access's boundary reach up to N - 1 places further
    const bool even = reinterpret_cast<uintptr_t>(p.logits) % (N * sizeof(E)) == 0 && p.stride % N == 0;
    const int slices = (p.vocab + (even ? 0 : N - 1) + SLICE - 1) / SLICE;
    if (p.rows * slices > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    return p.tokens || p.bias_ids ? launch_one<E, N, U, true>(p, L, slices, stream) : launch_one<E, N, U, false>(p, L, slices, stream);
}

// Tokens of a slice: shorter ones while there are SMs without one.
int slice_of(int64_t rows, int32_t vocab, int64_t sms)
{
    int slice = AL_SLICE;
    while (slice > AL_LEAST && rows * ((vocab + slice - 1) / slice) < 2 * sms)
        slice /= 2;
    return slice;
}

template <typename E> cudaError_t launch_e(const AdjustParams &p, int slice, const loom_launch &L, cudaStream_t stream)
{
    constexpr int N = 16 / (int)sizeof(E);
    const auto phase = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 16; };
    if (phase(p.logits) != phase(p.y) || (p.stride - p.y_stride) % N)
        return slice > 4096 ? launch_u<E, 1, 16>(p, L, stream) : launch_u<E, 1, 4>(p, L, stream);
    switch (slice / (AL_THREADS * N)) {
    case 8: return launch_u<E, N, 8 * (int)sizeof(E) / 4>(p, L, stream);       // (16-bit types: at most 4)
    case 4: return launch_u<E, N, 4>(p, L, stream);
    case 2: return launch_u<E, N, 2>(p, L, stream);
    default: return launch_u<E, N, 1>(p, L, stream);
    }
}

}  // namespace

bool adjust_geometry(int64_t rows, int32_t vocab, bool marks, int64_t sms, loom_launch *out)
{
    const int slice = slice_of(rows, vocab, sms);
    const int64_t ctas = rows * ((vocab + slice - 1) / slice);
    if (ctas > 0x7fffffff)
        return false;
    *out = loom_launch{};
    out->grid[0] = (uint32_t)ctas;
    out->block[0] = AL_THREADS;
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->smem_bytes = marks ? (uint32_t)slice * 4 : 0;
    out->units_per_cta = (uint32_t)slice;
    out->kernel = LOOM_KERNEL_ADJUST;
    return true;
}

cudaError_t launch_adjust(const AdjustParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    const int slice = (int)L.units_per_cta;
    if (dtype == LOOM_F32)
        return launch_e<float>(p, slice, L, stream);
    return dtype == LOOM_F16 ? launch_e<__half>(p, slice, L, stream) : launch_e<__nv_bfloat16>(p, slice, L, stream);
}

}  // namespace loom
