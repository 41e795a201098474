// token_logits.cu -- logits adjusted before a token is chosen: penalties for tokens that were
// seen, biases, a grammar's mask (sm_103a).
//
// Design
//  * Bound: a row's logits in and out.  A row is cut into slices, a CTA each (at 16-byte boundaries of the row's memory,
//    wherever it starts; a row whose copy starts elsewhere in its 16 bytes is taken one element at a time), whose
//    loads are all in flight before anything else is known.  The logits pass through registers as bits, masked or not.
//  * Few tokens of a row have a penalty or a bias.  A slice's CTA goes through the row's history, each warp putting what
//    is the slice's on a list of its own, and marks the list's tokens, one word a token in shared memory:
//    bits 0..19 occurrences behind the prompt, bit 20 seen in the prompt, bits 21..31 the bias entry (AL_ENTRY - its
//    place, so that the largest is the first of several).  Sums and maxima of whole numbers: their order does not
//    matter.  Those that mark a token first stay on the list, and when the slice is copied the lists' tokens are
//    adjusted, out of L2.  (Histories of more than 4096 tokens take the lists a batch at a time, and all of the
//    slice's marks are looked through.)  The lists keep warps full: where 1 token of 19 is a given slice's, 32 of them
//    cost as much as one.
//
// Measured as nodes of a CUDA graph (f32)
//   1 x 32768, history 2000, biases, a mask   3.1 us (a call through the binding 17, the host's part)
//   256 x 131072, history 4096 (2048 on average), 64 biases, masks for half of the rows   52.2 us (copy and mask alone 41;
//   bf16 43.4 us; histories of 5000 64, 8192 74, 16384 97, 131072 273 us)
//   the same in place, history 4096 and a mask of half of the tokens for every row: 78 us, bf16 41 (to another y 55 and 45):
//   what a mask changes is read when that is known, not ahead
// (Tried: marks looked up for every logit, 56 us; a bit a token, numbers by running counts and marks by numbers, 55 us; a
// cluster sharing out the history and marking each other's slices, 96 us, as most tokens of a text are in one slice;
// a second kernel for the marked tokens, 57 us, which finds them in DRAM again; CTAs that load the next slice while they
// adjust one, 76 us.)
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int AL_THREADS = 512;
constexpr int AL_SLICE = 32 * AL_THREADS;    // most tokens of a slice
constexpr int AL_LEAST = 2048;               // fewest
constexpr int AL_BATCH = 8;                  // history tokens that a thread loads together
constexpr uint32_t AL_SEEN = 1u << 20, AL_COUNT = AL_SEEN - 1u, AL_ENTRY = 2047, AL_NONE = 0xffffffffu;

struct RowSettings {
    float repetition, frequency, presence;
    int length, prompt;
    const uint32_t *mask;    // or NULL
};

__device__ __forceinline__ RowSettings settings_of(const AdjustParams &p, int64_t row, bool report)
{
    RowSettings s;
    s.repetition = p.d_repetition ? __ldg(p.d_repetition + row) : p.repetition;
    if (!(s.repetition > 0.0f))
        s.repetition = 1.0f;
    s.frequency = p.d_frequency ? __ldg(p.d_frequency + row) : p.frequency;
    s.presence = p.d_presence ? __ldg(p.d_presence + row) : p.presence;
    s.length = p.history;
    bool wrong = false;
    if (p.tokens && p.lengths) {
        const int len = __ldg(p.lengths + row);
        wrong = len < 0 || len > p.history;
        s.length = min(max(len, 0), p.history);
    }
    s.prompt = p.prompts ? min(max(__ldg(p.prompts + row), 0), s.length) : 0;
    s.mask = nullptr;
    if (p.mask) {
        int64_t m = p.mask_rows ? __ldg(p.mask_rows + row) : p.masks == 1 ? 0 : row;
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

template <typename E, int N> struct alignas(sizeof(E) * N) Pack {
    E e[N];
};

// N: elements of an access, 16 bytes or one.  U: accesses of a thread.
template <typename E, int N, int U, bool MARKS>
__global__ void __launch_bounds__(AL_THREADS, 2) adjust_kernel(const AdjustParams p, int slices)
{
    constexpr int SLICE = AL_THREADS * N * U, WORDS = SLICE / 32, LIST = 32 * AL_BATCH;
    extern __shared__ __align__(16) uint32_t al_shared[];          // the mask's words; marks, then the warps' lists
    uint32_t *mask = al_shared, *marks = al_shared + (WORDS + 4) / 4 * 4;
    typedef Pack<E, N> P;
    if (MARKS)
        for (int i = threadIdx.x; i < SLICE / 4; i += AL_THREADS)
            reinterpret_cast<uint4 *>(marks)[i] = make_uint4(0, 0, 0, 0);
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
    // what the row's length does not matter for is loaded along with it
    const int32_t *tokens = p.tokens + row * p.history_stride, *ids = p.bias_ids + row * p.biases;
    const float *bias = p.bias_values + row * p.biases;
    uint32_t early[AL_BATCH];
    int32_t id = -1;
    if (MARKS) {
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j) {
            const int i = threadIdx.x + j * AL_THREADS;
            early[j] = i < p.history ? (uint32_t)__ldg(tokens + i) : AL_NONE;
        }
        if (threadIdx.x < p.biases)
            id = __ldg(ids + threadIdx.x);
    }
    const RowSettings s = settings_of(p, row, slice == 0);
    const int word0 = max(first, 0) >> 5;
    if (s.mask)
        for (int w = threadIdx.x; w <= WORDS; w += AL_THREADS)
            mask[w] = word0 + w < (p.vocab + 31) / 32 ? __ldg(s.mask + word0 + w) : 0u;
    __syncthreads();

    // The history's tokens of this warp that are the slice's, a batch at a time, on the warp's list as places in the
    // slice, with bit 15 for those of the prompt.  (A row's last slice may begin past the row.)
    const uint32_t begin = (uint32_t)min(max(first, 0), p.vocab), count = (uint32_t)min(first + SLICE, p.vocab) - begin;
    const int lane = threadIdx.x & 31;
    uint16_t *list = reinterpret_cast<uint16_t *>(marks + SLICE) + (threadIdx.x >> 5) * LIST;
    int listed = 0;
    const auto make_list = [&](int i0) {
        listed = 0;
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j) {
            const int i = i0 + j * AL_THREADS;
            if (i - lane >= s.length)
                break;
            const uint32_t token = early[j];
            const bool ours = i < s.length && token - begin < count;
            const unsigned all = __ballot_sync(dev::FULL_MASK, ours);
            if (ours)
                list[listed + __popc(all & ((1u << lane) - 1u))] = (uint16_t)((token - (uint32_t)first) | (i < s.prompt ? 0x8000u : 0u));
            listed += __popc(all);
        }
        __syncwarp();
    };
    const auto load_batch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j)
            early[j] = i0 + j * AL_THREADS < s.length ? (uint32_t)__ldg(tokens + i0 + j * AL_THREADS) : AL_NONE;
    };
    bool fresh_bias[AL_MAX_BIASES / AL_THREADS];
    if (MARKS) {
        for (int i0 = threadIdx.x; i0 - lane < s.length; i0 += AL_BATCH * AL_THREADS) {
            if (i0 >= AL_BATCH * AL_THREADS)
                load_batch(i0);
            make_list(i0);
            if (s.length > AL_BATCH * AL_THREADS) {
                for (int l = lane; l < listed; l += 32) {
                    const uint32_t t = list[l];
                    if (t & 0x8000u)
                        atomicOr(marks + (t & 0x7fffu), AL_SEEN);
                    else
                        atomicAdd(marks + t, 1u);
                }
                __syncwarp();
                continue;
            }
            // those that mark a token first stay on the list
            int kept = 0;
            for (int l = 0; l < listed; l += 32) {
                uint32_t t = 0, old = 1;
                if (l + lane < listed) {
                    t = list[l + lane];
                    old = t & 0x8000u ? atomicOr(marks + (t & 0x7fffu), AL_SEEN) : atomicAdd(marks + t, 1u);
                }
                const unsigned those = __ballot_sync(dev::FULL_MASK, old == 0);
                if (old == 0)
                    list[kept + __popc(those & ((1u << lane) - 1u))] = (uint16_t)(t & 0x7fffu);
                kept += __popc(those);
            }
            listed = kept;
            __syncwarp();
        }
        // the first of several entries stays: theirs are the upper bits, whatever the lower ones count meanwhile
#pragma unroll
        for (int j = 0; j < AL_MAX_BIASES / AL_THREADS; ++j) {
            const int i = threadIdx.x + j * AL_THREADS;
            fresh_bias[j] = false;
            if (i < p.biases) {
                const uint32_t token = (uint32_t)(j == 0 ? id : __ldg(ids + i)), entry = AL_ENTRY - (uint32_t)i;
                uint32_t *mark = marks + (token - (uint32_t)first);
                if (token - begin < count)
                    for (uint32_t old = *mark; (old >> 21) < entry;) {
                        const uint32_t now = atomicCAS(mark, old, (old & (AL_SEEN | AL_COUNT)) | (entry << 21));
                        if (now == old) {
                            fresh_bias[j] = old == 0;
                            break;
                        }
                        old = now;
                    }
            }
        }
    }
    // Whole words of the mask and whole accesses, as most slices of aligned rows are: no place is looked at (256 x 131072
    // f32 52.3 us, without this way 53.2; bf16 43.5 and 45).
    if (N > 1 && (first & 31) == 0 && first + SLICE <= p.vocab) {
        if (!in_place || s.mask) {
            const int shift = (int)threadIdx.x * N & 31;
            const uint32_t *words = mask + ((int)threadIdx.x * N >> 5);
            const E *from = x + first + (int)threadIdx.x * N;
            E *to = y + first + (int)threadIdx.x * N;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s.mask) {
                    const uint32_t free = words[u * (AL_THREADS * N / 32)] >> shift;
                    if (in_place) {
                        if ((~free & ((1u << N) - 1u)) == 0)
                            continue;
                        v[u] = *reinterpret_cast<const P *>(from + u * AL_THREADS * N);
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (!((free >> i) & 1))
                            v[u].e[i] = dev::from_f32<E>(-INFINITY);
                }
                *reinterpret_cast<P *>(to + u * AL_THREADS * N) = v[u];
            }
        }
    } else if (!in_place || s.mask) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = first + ((int)threadIdx.x + u * AL_THREADS) * N;
            if (t >= p.vocab || t <= -N)
                continue;
            uint32_t masked = 0;                // a bit for each token that may not be chosen
            if (s.mask) {
                const int t0 = max(t, 0), word = (t0 >> 5) - word0;
                masked = ~(__funnelshift_r(mask[word], N > 1 ? mask[word + ((t0 & 31) + N > 32)] : 0u, t0 & 31) << (t0 - t));
            }
            if (whole(t)) {
                if (in_place) {
                    if (!(masked & ((1u << N) - 1u)))
                        continue;
                    v[u] = *reinterpret_cast<const P *>(x + t);
                }
                if (s.mask)
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if ((masked >> i) & 1)
                            v[u].e[i] = dev::from_f32<E>(-INFINITY);
                *reinterpret_cast<P *>(y + t) = v[u];
            } else {                            // the row's first or last tokens
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (t + i >= 0 && t + i < p.vocab)
                        y[t + i] = (masked >> i) & 1 ? dev::from_f32<E>(-INFINITY) : x[t + i];
            }
        }
    }
    if (MARKS) {
        __syncthreads();
        const auto adjust = [&](uint32_t place, uint32_t mark) {
            const int t = first + (int)place;
            if (mark && (!s.mask || ((mask[(t >> 5) - word0] >> (t & 31)) & 1)))
                y[t] = dev::from_f32<E>(adjusted(dev::to_f32(x[t]), mark, s, bias));
        };
        if (s.length <= AL_BATCH * AL_THREADS) {
            for (int l = lane; l < listed; l += 32)
                adjust(list[l], marks[list[l]]);
#pragma unroll
            for (int j = 0; j < AL_MAX_BIASES / AL_THREADS; ++j)
                if (fresh_bias[j]) {
                    const uint32_t place = (uint32_t)(j == 0 ? id : __ldg(ids + threadIdx.x + j * AL_THREADS)) - (uint32_t)first;
                    adjust(place, marks[place]);
                }
        } else {                                // a long history's tokens were not kept: all marks are looked through
            for (int i = threadIdx.x; i < SLICE; i += AL_THREADS)
                if (marks[i])
                    adjust(i, marks[i]);
        }
    }
}

// Shared memory of a slice: its mask's words, a word for each token and the warps' lists.
int64_t smem_of(bool marks, int64_t slice) { return (slice / 32 + 4) / 4 * 16 + (marks ? 4 * slice + AL_THREADS * AL_BATCH * 2 : 0); }

template <typename E, int N, int U, bool MARKS> cudaError_t launch_one(const AdjustParams &p, const loom_launch &L, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    static_assert(AL_THREADS * N * U <= 32768, "places have 15 bits");
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(adjust_kernel<E, N, U, MARKS>), 0, done);
    return e != cudaSuccess ? e : launch_prepared(adjust_kernel<E, N, U, MARKS>, L, stream, p, (int)(L.grid[0] / p.rows));
}

template <typename E, int N, int U> cudaError_t launch_u(const AdjustParams &p, const loom_launch &L, cudaStream_t stream)
{
    return p.tokens || p.bias_ids ? launch_one<E, N, U, true>(p, L, stream) : launch_one<E, N, U, false>(p, L, stream);
}

template <typename E> cudaError_t launch_e(const AdjustParams &p, const loom_launch &L, cudaStream_t stream)
{
    constexpr int N = 16 / (int)sizeof(E);
    if (adjust_access(p, (int)sizeof(E)) == AL_APART)
        return L.units_per_cta == 16 * AL_THREADS ? launch_u<E, 1, 16>(p, L, stream) : launch_u<E, 1, 4>(p, L, stream);
    switch (L.units_per_cta / (AL_THREADS * N)) {
    case 8: return launch_u<E, N, 8 * (int)sizeof(E) / 4>(p, L, stream);       // (16-bit types: at most 4)
    case 4: return launch_u<E, N, 4>(p, L, stream);
    case 2: return launch_u<E, N, 2>(p, L, stream);
    default: return launch_u<E, N, 1>(p, L, stream);
    }
}

}  // namespace

int adjust_access(const AdjustParams &p, int bytes)
{
    const auto phase = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 16; };
    const int n = 16 / bytes;
    if (phase(p.logits) != phase(p.y) || (p.stride - p.y_stride) % n)
        return AL_APART;
    return phase(p.logits) == 0 && p.stride % n == 0 ? AL_ALIGNED : AL_ALIKE;
}

bool adjust_geometry(int64_t rows, int32_t vocab, bool marks, int bytes, int access, int64_t sms, loom_launch *out)
{
    int slice = AL_SLICE;                    // shorter ones while there are SMs without one
    while (slice > AL_LEAST && rows * ((vocab + slice - 1) / slice) < 2 * sms)
        slice /= 2;
    // accesses of 16 bytes: one of a thread at least; of one element: 16 or 4
    const int n = 16 / bytes;
    slice = access != AL_APART ? (slice > AL_THREADS * n ? slice : AL_THREADS * n) : slice > AL_LEAST ? 16 * AL_THREADS : 4 * AL_THREADS;
    // rows that do not all start on an access's boundary reach up to n - 1 places further
    const int64_t slices = (vocab + (access == AL_ALIKE ? n - 1 : 0) + slice - 1) / slice;
    if (rows * slices > 0x7fffffff)
        return false;
    *out = loom_launch{};
    out->grid[0] = (uint32_t)(rows * slices);
    out->block[0] = AL_THREADS;
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->smem_bytes = (uint32_t)smem_of(marks, slice);
    out->units_per_cta = (uint32_t)slice;
    out->kernel = LOOM_KERNEL_ADJUST;
    return true;
}

cudaError_t launch_adjust(const AdjustParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (p.logits == p.y && !p.tokens && !p.bias_ids && !p.mask)
        return cudaSuccess;
    if (dtype == LOOM_F32)
        return launch_e<float>(p, L, stream);
    return dtype == LOOM_F16 ? launch_e<__half>(p, L, stream) : launch_e<__nv_bfloat16>(p, L, stream);
}

}  // namespace loom
