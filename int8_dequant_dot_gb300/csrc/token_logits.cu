// token_logits.cu -- logits adjusted before a token is chosen: penalties for tokens that were
// seen, biases, a grammar's mask (sm_103a).
//
// Design
//  * Bound: a row's logits in and out.  Nearly all of them pass as bits, masked or not; few tokens of a row have a
//    penalty or a bias.
//  * Many rows take two kernels.  The first copies and masks, slices of a row a CTA, 16 bytes an access (cut at 16-byte
//    boundaries of the row's memory, wherever it starts; one element at a time where the two rows start differently).
//    The second counts a row's history in a hash table in shared memory, a CTA a row, as the first one's last CTAs
//    run, and then adjusts those tokens alone, 32 a warp at once.  In place and without masks it is the second alone.
//  * A token's mark is one word: bits 0..19 occurrences behind the prompt, bit 20 seen in the prompt, bits 21..31 the bias
//    entry (AL_ENTRY - its place, so that the largest is the first of several).  Sums and maxima of whole numbers: their
//    order does not matter.  Who marks a token first also puts it on the list of what is to be adjusted.
//  * Histories too long for the table have a word for every token instead, those of 2 to 16 CTAs a row
//    interleaved, each of which goes through all of the history.
//  * Few rows (whose slices fit the SMs at once) take one kernel, in which a slice's CTA marks, copies and adjusts.
//
// Measured (f32)
//   1 x 32768, history 2000, biases, a mask   3.4 us
//   256 x 131072, history 4096 (2048 on average), 64 biases, masks for half of the rows   AL_T us (copy and mask alone 41)
// (Tried: the one kernel for many rows, 66 us: its words take the room that loads in flight want of the same memory;
// marks looked up for every logit, 56 us; a cluster sharing out the history and marking each other's slices, 96 us, as
// most tokens of a text are in one slice.)
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int AL_THREADS = 512;
constexpr int AL_SLICE = 32 * AL_THREADS;    // most tokens of a slice
constexpr int AL_LEAST = 2048;               // fewest
constexpr int AL_BATCH = 8;                  // history tokens that a thread loads together
constexpr int AL_HASHED = 10240;             // most tokens and biases that a table takes, which has 5/4 as many places or more
constexpr int AL_DIRECT = 34000;             // most tokens of a CTA that has a word for each
constexpr uint32_t AL_SEEN = 1u << 20, AL_COUNT = AL_SEEN - 1u, AL_ENTRY = 2047, AL_NONE = 0xffffffffu;

struct RowSettings {
    float repetition, frequency, presence;
    int length, prompt;
    const uint32_t *mask;    // or NULL
};

__device__ __forceinline__ RowSettings settings_of(const AdjustParams &p, int64_t row, bool report)
{
    RowSettings s;
    s.repetition = p.d_repetition ? __ldcg(p.d_repetition + row) : p.repetition;
    if (!(s.repetition > 0.0f))
        s.repetition = 1.0f;
    s.frequency = p.d_frequency ? __ldcg(p.d_frequency + row) : p.frequency;
    s.presence = p.d_presence ? __ldcg(p.d_presence + row) : p.presence;
    s.length = p.history;
    bool wrong = false;
    if (p.tokens && p.lengths) {
        const int len = __ldcg(p.lengths + row);
        wrong = len < 0 || len > p.history;
        s.length = min(max(len, 0), p.history);
    }
    s.prompt = p.prompts ? min(max(__ldcg(p.prompts + row), 0), s.length) : 0;
    s.mask = nullptr;
    if (p.mask) {
        int64_t m = p.mask_rows ? __ldcg(p.mask_rows + row) : p.masks == 1 ? 0 : row;
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

// ---- marks of a CTA's tokens --------------------------------------------------------------------
struct Marks {
    uint32_t *marks;         // [places], zero at first
    uint32_t *keys;          // [places] of a table, AL_NONE at first; NULL: a word for every token
    uint32_t places;         // of a table a power of two
    uint32_t first, log_parts, part;       // words: of the tokens first + part, and every 1 << log_parts further
    uint32_t *listed;        // tokens that have a mark
    uint16_t *list;          // their places

    __device__ __forceinline__ void clear() const
    {
        for (uint32_t i = threadIdx.x; i < (places + 3) / 4; i += AL_THREADS)
            reinterpret_cast<uint4 *>(marks)[i] = make_uint4(0, 0, 0, 0);
        if (keys)
            for (uint32_t i = threadIdx.x; i < places / 4; i += AL_THREADS)
                reinterpret_cast<uint4 *>(keys)[i] = make_uint4(AL_NONE, AL_NONE, AL_NONE, AL_NONE);
        if (threadIdx.x == 0)
            *listed = 0;
    }

    // The token's place, or AL_NONE where it is not this CTA's.  (A table is never full.)
    template <bool TABLE> __device__ __forceinline__ uint32_t find(uint32_t token, uint32_t vocab) const
    {
        if (token >= vocab)                                 // (a negative one among them)
            return AL_NONE;
        if (!TABLE) {
            const uint32_t t = token - first, place = t >> log_parts;
            return (t & ((1u << log_parts) - 1u)) == part && place < places ? place : AL_NONE;
        }
        uint32_t at = token * 2654435769u >> (32 - log_parts);          // (of a table: the logarithm of its places)
        for (;;) {
            const uint32_t there = atomicCAS(keys + at, AL_NONE, token);
            if (there == AL_NONE || there == token)
                return at;
            at = (at + 1) & (places - 1);
        }
    }
    template <bool TABLE> __device__ __forceinline__ uint32_t token_of(uint32_t place) const
    {
        return TABLE ? keys[place] : first + part + (place << log_parts);
    }

    // All lanes of a warp together.
    __device__ __forceinline__ void append(uint32_t place, bool fresh) const
    {
        const unsigned all = __ballot_sync(dev::FULL_MASK, fresh);
        if (all == 0)
            return;
        const int lane = threadIdx.x & 31, leader = __ffs(all) - 1;
        uint32_t at = 0;
        if (lane == leader)
            at = atomicAdd(listed, (uint32_t)__popc(all));
        at = __shfl_sync(dev::FULL_MASK, at, leader);
        if (fresh)
            list[at + __popc(all & ((1u << lane) - 1u))] = (uint16_t)place;
    }
    template <bool TABLE> __device__ __forceinline__ void see(uint32_t token, uint32_t vocab, bool prompt) const
    {
        const uint32_t place = find<TABLE>(token, vocab);
        uint32_t old = 1;
        if (place != AL_NONE)
            old = prompt ? atomicOr(marks + place, AL_SEEN) : atomicAdd(marks + place, 1u);
        append(place, old == 0);
    }
    // The first of several entries stays: theirs are the upper bits, whatever the lower ones count meanwhile.
    template <bool TABLE> __device__ __forceinline__ void bias(uint32_t token, uint32_t vocab, int index) const
    {
        const uint32_t place = find<TABLE>(token, vocab), entry = AL_ENTRY - (uint32_t)index;
        bool fresh = false;
        if (place != AL_NONE)
            for (uint32_t old = marks[place]; (old >> 21) < entry;) {
                const uint32_t now = atomicCAS(marks + place, old, (old & (AL_SEEN | AL_COUNT)) | (entry << 21));
                if (now == old) {
                    fresh = old == 0;
                    break;
                }
                old = now;
            }
        append(place, fresh);
    }
};

// What is loaded before the row's length is known.
struct Early {
    uint32_t token[AL_BATCH];
    int32_t id;
};

__device__ __forceinline__ Early load_early(const AdjustParams &p, int64_t row)
{
    Early e;
#pragma unroll
    for (int j = 0; j < AL_BATCH; ++j) {
        const int i = threadIdx.x + j * AL_THREADS;
        e.token[j] = i < p.history ? (uint32_t)__ldcg(p.tokens + row * p.history_stride + i) : AL_NONE;
    }
    e.id = threadIdx.x < p.biases ? __ldcg(p.bias_ids + row * p.biases + threadIdx.x) : -1;
    return e;
}

template <bool TABLE> __device__ __forceinline__ void mark_row(const Marks &m, const AdjustParams &p, const RowSettings &s, int64_t row, const Early &e)
{
    const int32_t *tokens = p.tokens + row * p.history_stride, *ids = p.bias_ids + row * p.biases;
    const int lane = threadIdx.x & 31;
    const uint32_t vocab = (uint32_t)p.vocab;
#pragma unroll
    for (int j = 0; j < AL_BATCH; ++j) {
        const int i = threadIdx.x + j * AL_THREADS;
        if (i - lane < s.length)                            // (a warp's lanes together)
            m.see<TABLE>(i < s.length ? e.token[j] : AL_NONE, vocab, i < s.prompt);
    }
    for (int i0 = threadIdx.x + AL_BATCH * AL_THREADS; i0 - lane < s.length; i0 += AL_BATCH * AL_THREADS) {
        uint32_t at[AL_BATCH];
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j)
            at[j] = i0 + j * AL_THREADS < s.length ? (uint32_t)__ldcg(tokens + i0 + j * AL_THREADS) : AL_NONE;
#pragma unroll
        for (int j = 0; j < AL_BATCH; ++j)
            m.see<TABLE>(at[j], vocab, i0 + j * AL_THREADS < s.prompt);
    }
    for (int i = threadIdx.x; i - lane < p.biases; i += AL_THREADS)
        m.bias<TABLE>((uint32_t)(i < AL_THREADS ? e.id : i < p.biases ? __ldcg(ids + i) : -1), vocab, i);
}

template <typename E, bool TABLE>
__device__ __forceinline__ void adjust_marked(const Marks &m, const AdjustParams &p, const RowSettings &s, int64_t row)
{
    const E *x = static_cast<const E *>(p.logits) + row * p.stride;
    E *y = static_cast<E *>(p.y) + row * p.y_stride;
    const float *bias = p.bias_values + row * p.biases;
    const int n = (int)*m.listed;
    for (int i = threadIdx.x; i < n; i += AL_THREADS) {
        const uint32_t place = m.list[i], t = m.token_of<TABLE>(place);
        if (!s.mask || ((__ldg(s.mask + (t >> 5)) >> (t & 31)) & 1))
            y[t] = dev::from_f32<E>(adjusted(dev::to_f32(x[t]), m.marks[place], s, bias));
    }
}

// ---- a slice of a row, copied and masked; with MARKS adjusted, too ---------------------------------------
template <typename E, int N> struct alignas(sizeof(E) * N) Pack {
    E e[N];
};

// N: elements of an access, 16 bytes or one.  U: accesses of a thread.  `chain`: the second kernel follows, which reads
// what this one's predecessors have written before it waits for this one, so it may start once they have ended.
template <typename E, int N, int U, bool MARKS>
__global__ void __launch_bounds__(AL_THREADS, 2) adjust_slice_kernel(const AdjustParams p, int slices, int chain)
{
    extern __shared__ __align__(16) uint32_t al_shared[];          // marks of the slice, its mask's words, the list
    __shared__ uint32_t listed;
    constexpr int SLICE = AL_THREADS * N * U, WORDS = SLICE / 32 + 1;
    typedef Pack<E, N> P;
    uint32_t *mask = al_shared + (MARKS ? SLICE : 0);
    Marks m = {al_shared, nullptr, (uint32_t)SLICE, 0, 0, 0, &listed, reinterpret_cast<uint16_t *>(mask + WORDS)};
    if (MARKS)
        m.clear();
    if (chain) {
        dev::wait_previous_kernel();
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    } else {
        dev::follow_previous_kernel();
    }
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
    Early early;
    if (MARKS)
        early = load_early(p, row);
    const RowSettings s = settings_of(p, row, slice == 0 && !chain);
    const int word0 = max(first, 0) >> 5;
    if (s.mask) {
#pragma unroll
        for (int i = 0; i < (WORDS + AL_THREADS - 1) / AL_THREADS; ++i) {
            const int w = threadIdx.x + i * AL_THREADS;
            if (w < WORDS)
                mask[w] = word0 + w < (p.vocab + 31) / 32 ? __ldg(s.mask + word0 + w) : 0u;
        }
    }
    if (MARKS || s.mask)
        __syncthreads();
    if (MARKS) {
        m.first = (uint32_t)first;
        mark_row<false>(m, p, s, row, early);
    }
    if (!in_place || s.mask) {
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
        adjust_marked<E, false>(m, p, s, row);
    }
}

// ---- the marked tokens of a row (or of one of its 1 << log_parts parts) -----------------------------------
template <typename E, bool TABLE>
__global__ void __launch_bounds__(AL_THREADS, 2) adjust_marked_kernel(const AdjustParams p, int places, int log_parts, int after_slices)
{
    extern __shared__ __align__(16) uint32_t al_shared[];          // marks, a table's keys, the list
    __shared__ uint32_t listed;
    const int64_t row = blockIdx.x >> (TABLE ? 0 : log_parts);
    const uint32_t part = TABLE ? 0 : blockIdx.x & ((1u << log_parts) - 1u);
    const int room = (places + 3) / 4 * 4;
    const Marks m = {al_shared, TABLE ? al_shared + room : nullptr, (uint32_t)places, 0, (uint32_t)log_parts, part, &listed,
                     reinterpret_cast<uint16_t *>(al_shared + (TABLE ? 2 : 1) * room)};
    m.clear();
    if (!after_slices)
        dev::follow_previous_kernel();
    // After the slices' kernel: its CTAs let this one start when all that came before them had ended, so what
    // only they write (y) is all that has to wait.  Loads that go past the first-level cache, which may be older.
    const Early early = load_early(p, row);
    const RowSettings s = settings_of(p, row, part == 0);
    __syncthreads();
    mark_row<TABLE>(m, p, s, row, early);
    if (after_slices)
        dev::follow_previous_kernel();
    __syncthreads();
    adjust_marked<E, TABLE>(m, p, s, row);
}

// ---- launches -------------------------------------------------------------------------------------------
// Shared memory of a slice: a word and a place on the list for each token, and its mask's words.
int64_t slice_smem(bool marks, int64_t slice) { return (marks ? 6 * slice : 0) + 4 * (slice / 32 + 1); }

// Tokens of a slice: shorter ones while there are SMs without one.
int slice_of(int64_t rows, int32_t vocab, int64_t sms)
{
    int slice = AL_SLICE;
    while (slice > AL_LEAST && rows * ((vocab + slice - 1) / slice) < 2 * sms)
        slice /= 2;
    return slice;
}

// Whether one kernel does it all: its CTAs fit the SMs at once, two each.
bool one_kernel(int64_t rows, int32_t vocab, int slice, int64_t sms) { return rows * ((vocab + slice - 1) / slice) <= 2 * sms; }

template <typename E, int N, int U, bool MARKS>
cudaError_t launch_slices(const AdjustParams &p, loom_launch L, int slices, int chain, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(adjust_slice_kernel<E, N, U, MARKS>), 0, done);
    if (e != cudaSuccess)
        return e;
    if (p.rows * slices > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    L.grid[0] = (uint32_t)(p.rows * slices);
    L.smem_bytes = (uint32_t)slice_smem(MARKS, AL_THREADS * N * U);
    return launch_prepared(adjust_slice_kernel<E, N, U, MARKS>, L, stream, p, slices, chain);
}

template <typename E, int N, int U> cudaError_t launch_u(const AdjustParams &p, const loom_launch &L, bool marks, int chain, cudaStream_t stream)
{
    constexpr int SLICE = AL_THREADS * N * U;
    static_assert(SLICE <= 65536, "the list holds 16 bits a token");
    // rows that do not all start on an access's boundary reach up to N - 1 places further
    const bool even = reinterpret_cast<uintptr_t>(p.logits) % (N * sizeof(E)) == 0 && p.stride % N == 0;
    const int slices = (p.vocab + (even ? 0 : N - 1) + SLICE - 1) / SLICE;
    return marks ? launch_slices<E, N, U, true>(p, L, slices, chain, stream) : launch_slices<E, N, U, false>(p, L, slices, chain, stream);
}

template <typename E, bool TABLE> cudaError_t launch_marked(const AdjustParams &p, loom_launch L, int after_slices, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(adjust_marked_kernel<E, TABLE>), 0, done);
    if (e != cudaSuccess)
        return e;
    int places, log_parts = 0;
    if (TABLE) {
        log_parts = 8;
        while ((1 << log_parts) < (p.history + p.biases) * 5 / 4)
            ++log_parts;
        places = 1 << log_parts;
        L.grid[0] = (uint32_t)p.rows;
        L.smem_bytes = (uint32_t)places * 10;
    } else {
        while (((p.vocab - 1) >> log_parts) + 1 > AL_DIRECT)
            ++log_parts;
        places = ((p.vocab - 1) >> log_parts) + 1;
        if (p.rows << log_parts > 0x7fffffff)
            return cudaErrorInvalidConfiguration;
        L.grid[0] = (uint32_t)(p.rows << log_parts);
        L.smem_bytes = (uint32_t)((places + 3) / 4 * 4) * 6;
    }
    return launch_prepared(adjust_marked_kernel<E, TABLE>, L, stream, p, places, log_parts, after_slices);
}

template <typename E> cudaError_t launch_e(const AdjustParams &p, int slice, bool one, const loom_launch &L, cudaStream_t stream)
{
    constexpr int N = 16 / (int)sizeof(E);
    const bool any = p.tokens || p.bias_ids, in_place = p.logits == p.y;
    const bool slices = !in_place || p.mask || (any && one), chain = any && !one && slices;
    if (slices) {
        const auto phase = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 16; };
        const bool marks = any && one;
        cudaError_t e;
        if (phase(p.logits) != phase(p.y) || (p.stride - p.y_stride) % N)
            e = slice > AL_LEAST ? launch_u<E, 1, 16>(p, L, marks, chain, stream) : launch_u<E, 1, 4>(p, L, marks, chain, stream);
        else if (slice >= 8 * AL_THREADS * N)
            e = launch_u<E, N, 8 * (int)sizeof(E) / 4>(p, L, marks, chain, stream);       // (16-bit types: at most 4)
        else if (slice >= 4 * AL_THREADS * N)
            e = launch_u<E, N, 4>(p, L, marks, chain, stream);
        else if (slice >= 2 * AL_THREADS * N)
            e = launch_u<E, N, 2>(p, L, marks, chain, stream);
        else
            e = launch_u<E, N, 1>(p, L, marks, chain, stream);
        if (e != cudaSuccess || !chain)
            return e;
    }
    if (!any || one)
        return cudaSuccess;
    return p.history + p.biases <= AL_HASHED ? launch_marked<E, true>(p, L, chain, stream) : launch_marked<E, false>(p, L, chain, stream);
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
    out->smem_bytes = (uint32_t)slice_smem(marks && one_kernel(rows, vocab, slice, sms), slice);
    out->units_per_cta = (uint32_t)slice;
    out->kernel = LOOM_KERNEL_ADJUST;
    return true;
}

cudaError_t launch_adjust(const AdjustParams &p, int32_t dtype, int64_t sms, const loom_launch &L, cudaStream_t stream)
{
    const int slice = (int)L.units_per_cta;
    const bool one = one_kernel(p.rows, p.vocab, slice, sms);
    if (dtype == LOOM_F32)
        return launch_e<float>(p, slice, one, L, stream);
    return dtype == LOOM_F16 ? launch_e<__half>(p, slice, one, L, stream) : launch_e<__nv_bfloat16>(p, slice, one, L, stream);
}

}  // namespace loom
