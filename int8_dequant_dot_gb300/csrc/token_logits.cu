// token_logits.cu -- logits adjusted before a token is chosen: penalties for tokens that were
// seen, biases, a grammar's mask (sm_103a).
//
// A CTA takes a row, slice by slice.  A slice's marks are one word a token in shared memory:
//   bits 0..19 occurrences behind the prompt, bit 20 seen in the prompt, bits 21..31 the bias entry
// (AL_ENTRY - its place, so that a maximum finds the first of several).
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int AL_THREADS = 512;
constexpr int AL_SLICE = 8192;               // tokens whose marks a CTA holds
constexpr uint32_t AL_SEEN = 1u << 20, AL_COUNT = AL_SEEN - 1u, AL_ENTRY = 2047;

struct RowSettings {
    float repetition, frequency, presence;
    int length, prompt;
    const int32_t *mask;     // or NULL
};

__device__ __forceinline__ RowSettings settings_of(const AdjustParams &p, int64_t row)
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
        const int64_t words = (p.vocab + 31) / 32;
        int64_t m = p.mask_rows ? p.mask_rows[row] : p.masks == 1 ? 0 : row;
        if (m >= p.masks) {
            wrong = true;
            m = -1;
        }
        s.mask = m < 0 ? nullptr : p.mask + m * words;
    }
    if (wrong && threadIdx.x == 0)
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

template <typename E> __global__ void __launch_bounds__(AL_THREADS) adjust_kernel(const AdjustParams p)
{
    __shared__ uint32_t marks[AL_SLICE];
    dev::follow_previous_kernel();
    const int64_t row = blockIdx.x;
    const RowSettings s = settings_of(p, row);
    const E *l = static_cast<const E *>(p.logits) + row * p.stride;
    E *y = static_cast<E *>(p.y) + row * p.y_stride;
    const int32_t *tokens = p.tokens + row * p.history_stride;
    const int32_t *ids = p.bias_ids + row * p.biases;
    const float *bias = p.bias_values + row * p.biases;
    for (int first = 0; first < p.vocab; first += AL_SLICE) {
        const int n = min(AL_SLICE, p.vocab - first);
        for (int i = threadIdx.x; i < n; i += AL_THREADS)
            marks[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < s.length; i += AL_THREADS) {
            const uint32_t t = (uint32_t)(tokens[i] - first);
            if (tokens[i] >= 0 && t < (uint32_t)n) {
                if (i < s.prompt)
                    atomicOr(marks + t, AL_SEEN);
                else
                    atomicAdd(marks + t, 1u);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.biases; i += AL_THREADS) {
            const uint32_t t = (uint32_t)(ids[i] - first);
            if (ids[i] >= 0 && t < (uint32_t)n)
                atomicMax(marks + t, (marks[t] & (AL_SEEN | AL_COUNT)) | ((AL_ENTRY - (uint32_t)i) << 21));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += AL_THREADS) {
            const int t = first + i;
            E v = l[t];
            if (marks[i])
                v = dev::from_f32<E>(adjusted(dev::to_f32(v), marks[i], s, bias));
            if (s.mask && !((s.mask[t / 32] >> (t % 32)) & 1))
                v = dev::from_f32<E>(-INFINITY);
            y[t] = v;
        }
        __syncthreads();
    }
}

}  // namespace

bool adjust_geometry(int64_t rows, int32_t, bool, int64_t, loom_launch *out)
{
    *out = loom_launch{};
    out->grid[0] = (uint32_t)rows;
    out->block[0] = AL_THREADS;
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->units_per_cta = 1;
    out->kernel = LOOM_KERNEL_ADJUST;
    return true;
}

cudaError_t launch_adjust(const AdjustParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_with(adjust_kernel<float>, L, stream, p);
    return dtype == LOOM_F16 ? launch_with(adjust_kernel<__half>, L, stream, p) : launch_with(adjust_kernel<__nv_bfloat16>, L, stream, p);
}

}  // namespace loom
