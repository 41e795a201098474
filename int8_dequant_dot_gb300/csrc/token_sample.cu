// token_sample.cu -- the next token of each row of logits, with temperature,
// top-k, top-p and min-p, from given random numbers (sm_103a).
//
// The definition (loom_token.h) is in whole-number weights
//   w[i] = floor(exp((l[i] - m) / T) * 2^31),
// whose sums do not depend on the order they are taken in, so the row can be cut
// and summed at will and the chosen token is still the definition's.
//
// Design
//  * A row is read once: a cluster of 1 to 8 CTAs holds it in shared memory as
//    f32 (slices of up to 49152 logits), and every later pass runs on chip.
//  * No sort of a row.  A histogram over 2048 equal bins of (m - l) / T, which spread the
//    bulk of a row over many bins, finds the bin in which top-k's count or top-p's
//    weight is reached.  Logits whose weight is 0 cannot be chosen and take no part.
//  * Where top-k leaves few logits (with those of its last bin at most 2048), they are
//    gathered in one CTA, which does the rest: up to 512 are sorted, by counting; of more,
//    each cut is found by a histogram and the entries of one bin.
//  * Otherwise the boundary's bin alone is gathered and sorted; one with more logits than
//    2048 (equal ones, mostly) is searched by histograms over their bit patterns, 2048 at a
//    time, until one pattern is left.  Equal logits there: the number that stays follows from
//    the sums alone, and the first ones in index order stay, by a running count over segments
//    of the row.  The draw then sums the kept weight per segment (a warp each), scans over
//    segments and CTAs, and one warp walks the segment that holds floor(u total).
//  * A weight is added to a bin as two 32-bit halves (its upper and lower 16 bits:
//    no slice can overflow them), which shared memory adds natively.
//  * What bounds it is not the row's bytes but, for few rows, the chain of passes, scans and
//    cluster barriers (1000 to 2000 cycles each, most of it waiting for the slowest CTA), and,
//    for many, the instructions of the passes (15 for a weight) of the two CTAs that fit an SM.
//
// Measured (f32, normal logits; top-k 50 / top-p 0.9 / neither)
//   1 x 32768     9.0 / 14.1 / 5.8 us
//   38 x 131072   24 / 45 / 18 us (one wave of clusters)
//   256 x 131072  99 / 203 / 78 us, 1.7 TB/s for the last; greedy 43 us, 3.1 TB/s
//   256 x 131072 bf16  95 / 210 / 75 us; greedy 37 us: the passes over f32 copies are the same
//   256 x 131071  210 us by top-p, 85 us unfiltered (bf16 220 and 85): rows that do not start on 16 bytes
//                 are loaded one element at a time
// (An L2 prefetch of the slices that will follow on the same SMs took 2 us from greedy rows and
// gave 2 us to the others.)
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int SM_THREADS = 512, SM_WARPS = SM_THREADS / 32;
constexpr int SM_BINS = 2048;
constexpr int SM_MAX_CLUSTER = 8;
constexpr int SM_MAX_SLICE = 49152;        // logits of a CTA: 192 KiB
constexpr int SM_SLICE = 16384;            // slices up to this leave room for a second CTA on the SM
constexpr int SM_SHORT_SLICE = 2048;       // not worth another CTA
constexpr int SM_SEGMENTS = 128;           // segments of a slice
constexpr int SM_LIST = SM_BINS;           // logits that one CTA sorts: their list takes the bins' place
constexpr float SM_BIN_SCALE = 95.0f;      // bins per unit of (m - l) / T: weights are above 0 in
                                           // bins below SM_EDGE_BIN and 0 above it
constexpr uint32_t SM_EDGE_BIN = 2041;     // 21.4842 .. 21.4948; 2^-31 is at 21.4876
constexpr uint32_t SM_KEY_NONE = 0x007fffffu;   // key of -infinity

// Bit pattern of a logit whose whole-number order is the logits' order.
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu)); }

// 2^31 for the largest logit, which is finite here.  (What is no number, or -infinity, converts to 0.)
__device__ __forceinline__ uint32_t weight_of(float l, float m, float inv) { return __float2uint_rz(expf((l - m) * inv) * 2147483648.0f); }

// Sum over a warp of what adds up to less than 2^56.
__device__ __forceinline__ uint64_t warp_sum(uint64_t v)
{
    const uint32_t low = __reduce_add_sync(dev::FULL_MASK, (uint32_t)v & 0xffffffu);
    return low + ((uint64_t)__reduce_add_sync(dev::FULL_MASK, (uint32_t)(v >> 24)) << 24);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(dev::smem_u32(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ uint32_t load_remote(const uint32_t *p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ void store_remote(uint32_t *p, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}

__device__ __forceinline__ void store_remote(uint64_t *p, uint32_t rank, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}

__device__ __forceinline__ uint32_t add_remote(uint32_t *p, uint32_t rank, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(p, rank)), "r"(v) : "memory");
    return old;
}

struct Found {            // where a search ended: what lies above bin `bin`
    uint64_t mass_above;
    uint32_t count_above, bin, count;      // count: in the bin (where counts were searched)
};

// What the CTAs of a cluster tell each other has two places, used in turn: one barrier then
// parts the writing of a place from its next writing.
struct alignas(16) Shared {       // (the slice behind it is read 16 bytes at a time)
    union {
        struct {
            uint32_t count[SM_BINS], low[SM_BINS], high[SM_BINS];
        };
        struct {                                // gathered logits: (~key, index) in one word, so that
            uint64_t list_order[SM_LIST];       // their order is that of the words; and their weights
            uint32_t list_w[SM_LIST];
        };
    };
    uint64_t share_mass[2][SM_MAX_CLUSTER];     // per CTA of the cluster
    uint32_t share_count[2][SM_MAX_CLUSTER];
    uint32_t key_max[2][SM_MAX_CLUSTER], key_min[2][SM_MAX_CLUSTER];
    Found found[2];
    uint64_t warp_mass[SM_WARPS];
    uint32_t warp_count[SM_WARPS], warp_a[SM_WARPS], warp_b[SM_WARPS];
    uint64_t seg_mass[SM_SEGMENTS];
    uint64_t word;                              // one thread's to all
    uint32_t seg_ties[SM_SEGMENTS];
    uint32_t list_n;                            // gathered logits of this CTA
};

static_assert(sizeof(Shared) % 16 == 0, "the slice is 16-byte aligned");

struct Row {              // what the threads of a cluster agree on
    Shared *s;
    float *l;             // this CTA's slice
    int n, slice, seg;    // logits of this CTA, of a full slice, of a segment
    uint32_t rank, ranks;
    float m, inv, bins_per_unit;      // largest logit, 1 / T, SM_BIN_SCALE / T
    uint32_t turn;        // which places are used next
};

// f(logit, place) for every logit of the slice, four neighbours a thread at a time (their
// arithmetic overlaps).  The slice is filled up to a multiple of four with -infinity.
template <typename F> __device__ __forceinline__ void for_each(const Row &r, F f)
{
    for (int i = 4 * threadIdx.x; i < r.n; i += 4 * SM_THREADS) {
        const float4 q = *reinterpret_cast<const float4 *>(r.l + i);
        f(q.x, i);
        f(q.y, i + 1);
        f(q.z, i + 2);
        f(q.w, i + 3);
    }
}

// The same with the four together, f(logits, place): for what branches only after its arithmetic.
template <typename F> __device__ __forceinline__ void for_fours(const Row &r, F f)
{
    for (int i = 4 * threadIdx.x; i < r.n; i += 4 * SM_THREADS) {
        const float4 q = *reinterpret_cast<const float4 *>(r.l + i);
        const float l[4] = {q.x, q.y, q.z, q.w};
        f(l, i);
    }
}

__device__ __forceinline__ void agree(const Row &r)
{
    if (r.ranks > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Largest a and smallest b over the cluster.
__device__ __forceinline__ void cluster_max_min(Row &r, uint32_t &a, uint32_t &b)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t turn = r.turn;
    r.turn ^= 1u;
    a = __reduce_max_sync(dev::FULL_MASK, a);
    b = __reduce_min_sync(dev::FULL_MASK, b);
    if (lane == 0) {
        r.s->warp_a[warp] = a;
        r.s->warp_b[warp] = b;
    }
    __syncthreads();
    a = __reduce_max_sync(dev::FULL_MASK, lane < SM_WARPS ? r.s->warp_a[lane] : 0u);
    b = __reduce_min_sync(dev::FULL_MASK, lane < SM_WARPS ? r.s->warp_b[lane] : 0xffffffffu);
    if (threadIdx.x < r.ranks) {
        store_remote(&r.s->key_max[turn][r.rank], threadIdx.x, a);
        store_remote(&r.s->key_min[turn][r.rank], threadIdx.x, b);
    }
    agree(r);
    a = __reduce_max_sync(dev::FULL_MASK, lane < (int)r.ranks ? r.s->key_max[turn][lane] : 0u);
    b = __reduce_min_sync(dev::FULL_MASK, lane < (int)r.ranks ? r.s->key_min[turn][lane] : 0xffffffffu);
}

template <bool BY_MASS> __device__ __forceinline__ void clear_bins(const Row &r)
{
#pragma unroll
    for (int i = threadIdx.x; i < SM_BINS; i += SM_THREADS) {
        if (BY_MASS)
            r.s->low[i] = r.s->high[i] = 0;
        else
            r.s->count[i] = 0;
    }
    __syncthreads();
}

__device__ __forceinline__ void add_to_bin(Shared *s, uint32_t bin, uint32_t w)
{
    atomicAdd(&s->low[bin], w & 0xffffu);
    if (w >> 16)
        atomicAdd(&s->high[bin], w >> 16);
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(dev::FULL_MASK, v); }

// Inclusive scan over the CTA's threads (T uint64_t or uint32_t).
template <typename T> __device__ __forceinline__ T scan(const Row &r, T v)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T *sums = reinterpret_cast<T *>(r.s->warp_mass);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T up = __shfl_up_sync(dev::FULL_MASK, v, d);
        v += lane >= d ? up : (T)0;
    }
    if (lane == 31)
        sums[warp] = v;
    __syncthreads();
    v += warp_sum(lane < warp ? sums[lane] : (T)0);
    __syncthreads();
    return v;
}

// This CTA's mass and count to every CTA, and all of theirs: those of lower ranks, and in all.
struct Shares {
    uint64_t mass_below, mass;
    uint32_t count_below, count;
};
__device__ __forceinline__ Shares share(Row &r, uint64_t mass, uint32_t count)   // values of the last thread
{
    const uint32_t turn = r.turn, lane = threadIdx.x & 31;
    r.turn ^= 1u;
    if (threadIdx.x >= SM_THREADS - 32) {
        mass = __shfl_sync(dev::FULL_MASK, mass, 31);
        count = __shfl_sync(dev::FULL_MASK, count, 31);
        if (lane < r.ranks) {
            store_remote(&r.s->share_mass[turn][r.rank], lane, mass);
            store_remote(&r.s->share_count[turn][r.rank], lane, count);
        }
    }
    agree(r);
    mass = lane < r.ranks ? r.s->share_mass[turn][lane] : 0u;
    count = lane < r.ranks ? r.s->share_count[turn][lane] : 0u;
    return Shares{warp_sum(lane < r.rank ? mass : (uint64_t)0), warp_sum(mass), warp_sum(lane < r.rank ? count : 0u), warp_sum(count)};
}

// The bin in which the running count (or mass) from bin 0 up reaches `target`,
// given that `start` lies above bin 0; bins of all CTAs together.  Each CTA adds up
// its share of the bins.  `all`: what the bins hold.  Where the target is not reached the
// bin is SM_BINS.  Afterwards every CTA may clear its bins.
template <bool BY_MASS> __device__ Found search(Row &r, uint64_t target, Found start, Shares *all = nullptr)
{
    Shared *s = r.s;
    agree(r);   // every histogram is complete
    constexpr int MOST = SM_BINS / SM_THREADS;      // bins per thread with one CTA
    const int bins = SM_BINS / (int)r.ranks;
    const int per = bins >= SM_THREADS ? bins / SM_THREADS : 1;
    const int bin0 = (int)r.rank * bins + (int)threadIdx.x * per;
    uint64_t m[MOST], mass = 0;
    uint32_t c[MOST], count = 0;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        m[j] = 0;
        c[j] = 0;
        if (j < per && (int)threadIdx.x * per + j < bins) {      // all loads of a bin in flight together
            uint32_t low[SM_MAX_CLUSTER], high[SM_MAX_CLUSTER];
#pragma unroll
            for (uint32_t q = 0; q < SM_MAX_CLUSTER; ++q) {
                low[q] = high[q] = 0;
                if (q < r.ranks) {
                    low[q] = load_remote(BY_MASS ? &s->low[bin0 + j] : &s->count[bin0 + j], q);
                    if (BY_MASS)
                        high[q] = load_remote(&s->high[bin0 + j], q);
                }
            }
#pragma unroll
            for (uint32_t q = 0; q < SM_MAX_CLUSTER; ++q)
                if (BY_MASS)
                    m[j] += low[q] + ((uint64_t)high[q] << 16);
                else
                    c[j] += low[q];
        }
        mass += m[j];
        count += c[j];
    }
    const uint64_t own_mass = mass;
    const uint32_t own_count = count;
    if (BY_MASS)
        mass = scan(r, mass);
    else
        count = scan(r, count);
    const uint32_t turn = r.turn;
    if (threadIdx.x == 0) {
        s->found[turn].bin = SM_BINS;               // (the owner writes after the next barrier)
        s->list_n = 0;
    }
    const Shares t = share(r, mass, count);
    if (all)
        *all = t;
    uint64_t above_mass = start.mass_above + t.mass_below + mass - own_mass;
    uint32_t above_count = start.count_above + t.count_below + count - own_count;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const uint64_t before = BY_MASS ? above_mass : above_count, has = BY_MASS ? m[j] : c[j];
        if (before < target && target <= before + has)
            for (uint32_t q = 0; q < r.ranks; ++q) {
                store_remote(&s->found[turn].mass_above, q, above_mass);
                store_remote(&s->found[turn].count_above, q, above_count);
                store_remote(&s->found[turn].bin, q, (uint32_t)(bin0 + j));
                store_remote(&s->found[turn].count, q, c[j]);
            }
        above_mass += m[j];
        above_count += c[j];
    }
    agree(r);
    return s->found[turn];
}

// (fminf takes what is no number, a logit without weight, to the last bin.)
__device__ __forceinline__ uint32_t bin_of(float l, const Row &r)
{
    // (its whole part by an addition: the conversion instruction issues at a quarter of that rate)
    return __float_as_uint(__fadd_rd(fminf((r.m - l) * r.bins_per_unit, (float)(SM_BINS - 1)), 8388608.0f)) & (SM_BINS - 1);
}

// Whether a logit takes part (its weight is above 0), from its bin: the exponential is needed at
// the edge alone.
__device__ __forceinline__ bool takes_part(float l, uint32_t bin, const Row &r)
{
    return bin < SM_EDGE_BIN || (bin == SM_EDGE_BIN && weight_of(l, r.m, r.inv) > 0);
}

struct Boundary {        // the last logit that stays, and how many of its equals
    uint32_t key, keep;
};

// The first `n` words (a power of two) and, where PAIRS, their weights in rising order of the words.
template <bool PAIRS> __device__ void sort_list(Shared *s, int n)
{
    for (int k = 2; k <= n; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < n / 2; i += SM_THREADS) {
                const int a = 2 * i - (i & (j - 1)), b = a + j;
                const uint64_t x = s->list_order[a], y = s->list_order[b];
                if ((x > y) == ((a & k) == 0)) {
                    s->list_order[a] = y;
                    s->list_order[b] = x;
                    if (PAIRS) {
                        const uint32_t w = s->list_w[a];
                        s->list_w[a] = s->list_w[b];
                        s->list_w[b] = w;
                    }
                }
            }
            __syncthreads();
        }
}

__device__ __forceinline__ int power_of_two(int n)
{
    int p = 2;
    while (p < n)
        p <<= 1;
    return p;
}

// The logits of the bins `from` to `to` that take part, listed in the cluster's first CTA (each thread
// asks it for a place) as far as they are at most SM_LIST.  The list takes the place of the
// histograms.  Behind a search, that made its count 0.
__device__ void gather(Row &r, int start, uint32_t from, uint32_t to)
{
    Shared *s = r.s;
    const float low = (float)from, high = (float)(to + 1);
    for_fours(r, [&](const float (&l)[4], int i) {
        bool in[4], any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float at = (r.m - l[j]) * r.bins_per_unit;      // its whole part is the bin
            in[j] = at >= low && at < high;
            any = any || in[j];
        }
        if (any)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j]) {
                    const uint32_t w = weight_of(l[j], r.m, r.inv), e = w > 0 ? add_remote(&s->list_n, 0, 1u) : (uint32_t)SM_LIST;
                    if (e < SM_LIST) {
                        store_remote(&s->list_order[e], 0, ((uint64_t)~key_of(l[j]) << 32) | (uint32_t)(start + i + j));
                        store_remote(&s->list_w[e], 0, w);
                    }
                }
    });
    agree(r);
}

// Sorts the first n words and, where PAIRS, their weights.  A short list is ranked by counting, each
// of its words (all different) against the others by as many threads as there are for it: one
// pass, where the sorting network has a barrier a step.
template <bool PAIRS> __device__ void sorted_list(Shared *s, int n)
{
    if (n <= SM_THREADS) {
        int each = 1;                              // threads of a word: neighbours in a warp
        while (each < 16 && 2 * each * n <= SM_THREADS)
            each *= 2;
        const int e = (int)threadIdx.x / each, part = (int)threadIdx.x % each;
        const uint64_t mine = e < n ? s->list_order[e] : ~0ull;
        const uint32_t w = PAIRS && e < n ? s->list_w[e] : 0u;
        int rank = 0;
#pragma unroll 4
        for (int j = part; j < n; j += each)
            rank += s->list_order[j] < mine;
        for (int d = each >> 1; d > 0; d >>= 1)
            rank += __shfl_xor_sync(dev::FULL_MASK, rank, d);
        __syncthreads();
        if (e < n && part == 0) {
            s->list_order[rank] = mine;
            if (PAIRS)
                s->list_w[rank] = w;
        }
        __syncthreads();
        return;
    }
    const int size = power_of_two(n);
    for (int e = n + threadIdx.x; e < size; e += SM_THREADS) {
        s->list_order[e] = ~0ull;
        s->list_w[e] = 0;
    }
    __syncthreads();
    sort_list<PAIRS>(s, size);
}

// The boundary in bin `f.bin` of the first histogram: `target` is reached there.
template <bool BY_MASS> __device__ Boundary refine(Row &r, int start, uint64_t target, Found f)
{
    uint32_t members = f.count;
    if (BY_MASS || members <= SM_LIST)
        gather(r, start, f.bin, f.bin);
    if (BY_MASS)
        members = load_remote(&r.s->list_n, 0);          // (a barrier follows, before its CTA may change it or end)
    if (members <= SM_LIST) {      // sorted, the boundary is where the running sum gets there
        const uint32_t turn = r.turn;
        r.turn ^= 1u;
        if (r.rank == 0) {
            Shared *s = r.s;
            sorted_list<true>(s, (int)members);
            const int e0 = 4 * (int)threadIdx.x;
            uint64_t mass = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mass += e0 + j < (int)members ? (BY_MASS ? s->list_w[e0 + j] : 1u) : 0u;
            uint64_t run = scan(r, mass);
            run += (BY_MASS ? f.mass_above : f.count_above) - mass;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e0 + j < (int)members) {
                    const uint64_t next = run + (BY_MASS ? s->list_w[e0 + j] : 1u);
                    if (run < target && target <= next) {
                        const uint32_t order = (uint32_t)(s->list_order[e0 + j] >> 32);
                        int first = 0, past = e0 + j;      // the first of its equals
                        while (first < past) {
                            const int mid = (first + past) / 2;
                            if ((uint32_t)(s->list_order[mid] >> 32) < order)
                                first = mid + 1;
                            else
                                past = mid;
                        }
                        for (uint32_t q = 0; q < r.ranks; ++q) {
                            store_remote(&s->found[turn].bin, q, ~order);
                            store_remote(&s->found[turn].count_above, q, (uint32_t)(e0 + j - first + 1));
                        }
                    }
                    run = next;
                }
        }
        agree(r);
        return Boundary{r.s->found[turn].bin, r.s->found[turn].count_above};
    }
    uint32_t hi = 0, lo = 0xffffffffu;
    for_each(r, [&](float l, int) {
        const uint32_t bin = bin_of(l, r);
        if (bin == f.bin && takes_part(l, bin, r)) {
            hi = max(hi, key_of(l));
            lo = min(lo, key_of(l));
        }
    });
    cluster_max_min(r, hi, lo);
    for (int level = 0; level < 3 && hi > lo; ++level) {   // bins of equal size, the largest keys first
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        clear_bins<BY_MASS>(r);
        for_each(r, [&](float l, int) {
            const uint32_t key = key_of(l);
            if (key >= lo && key <= hi && takes_part(l, f.bin, r)) {
                if (BY_MASS)
                    add_to_bin(r.s, (hi - key) >> shift, weight_of(l, r.m, r.inv));
                else
                    atomicAdd(&r.s->count[(hi - key) >> shift], 1u);
            }
        });
        const uint32_t first_bin = f.bin;
        f = search<BY_MASS>(r, target, f);
        hi -= f.bin << shift;
        lo = max(lo, hi - min(hi, (1u << shift) - 1));
        f.bin = first_bin;
    }
    if (!BY_MASS)
        return Boundary{hi, (uint32_t)target - f.count_above};
    const uint64_t w = weight_of(logit_of(hi), r.m, r.inv);
    return Boundary{hi, (uint32_t)((target - f.mass_above + w - 1) / w)};
}

// ---- numbers of 64 bits ------------------------------------------------------------
// The SM's 64-bit floating-point units are few (a logarithm takes 4000 cycles, a product and its
// floor 800), so these are put together from whole numbers and f32.

// The 64-bit floating-point product f total of a positive f below 1 and a total below 2^52, rounded
// down or up to a whole number.
__device__ __forceinline__ uint64_t product(float f, uint64_t total, bool up)
{
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint32_t m = e ? (b & 0x7fffffu) | 0x800000u : b, s = e ? 150 - e : 149;      // f = m 2^-s
    uint64_t low = m * total, high = __umul64hi(m, total);
    const int drop = 22 - __clzll(high << 53 | low >> 11);       // bits past 53: to nearest, ties to even
    if (drop > 0) {
        const uint64_t add = (1ull << (drop - 1)) - 1 + ((low >> drop) & 1);
        low += add;
        high += low < add;
        low &= ~0ull << drop;
    }
    if (s >= 76)
        return up;
    const uint64_t rest = s < 64 ? low & ((1ull << s) - 1) : low | (high & ((1ull << (s - 64)) - 1));
    return (s < 64 ? low >> s | high << (64 - s) : high >> (s - 64)) + (up && rest);
}

// log(w / total), 0 < w <= total < 2^51, to f32's last place but for about 3 cases in 10^5.  With
// w / total = 2^-k a / b and a / b within [2^-1/2, 2^1/2], s = (a - b) / (a + b) is
//   log(a / b) = 2 s (1 + z / 3 + z^2 / 5 + ...),  z = s^2 <= 0.0295,
// in pairs of f32 (value and rest), the higher terms, which count for less, in one.
__device__ float log_of_part(uint32_t w, uint64_t total)
{
    int k = __clzll((long long)w) - __clzll((long long)total);
    uint64_t a = (uint64_t)w << k, b = total;
    if ((float)a > 1.4142135f * (float)b) {
        b *= 2;
        --k;
    } else if (1.4142135f * (float)a < (float)b) {
        a *= 2;
        ++k;
    }
    const int64_t num = (int64_t)(a - b), den = (int64_t)(a + b);
    const float num_hi = (float)num, num_lo = (float)(num - (int64_t)num_hi), den_hi = (float)den, den_lo = (float)(den - (int64_t)den_hi);
    const float s_hi = __fdiv_rn(num_hi, den_hi);
    const float s_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-s_hi, den_hi, num_hi), __fmaf_rn(-s_hi, den_lo, num_lo)), den_hi);
    const float z_hi = __fmul_rn(s_hi, s_hi), z_lo = __fmaf_rn(s_hi, s_hi, -z_hi) + 2.0f * s_hi * s_lo;
    const float tail = 1.0f / 7 + z_hi * (1.0f / 9 + z_hi * (1.0f / 11 + z_hi * (1.0f / 13 + z_hi * (1.0f / 15))));
    const float fifth = 0.2f, fifth_lo = (float)(0.2 - (double)0.2f), third = 1.0f / 3, third_lo = (float)(1.0 / 3 - (double)(1.0f / 3));
    float p = __fmul_rn(z_hi, tail);                          // 1/5 + z tail
    const float q_hi = __fadd_rn(fifth, p), q_lo = __fadd_rn(__fsub_rn(p, __fsub_rn(q_hi, fifth)), fifth_lo);
    p = __fmul_rn(z_hi, q_hi);                                // 1/3 + z q
    float p_lo = __fmaf_rn(z_hi, q_hi, -p) + (z_hi * q_lo + z_lo * q_hi);
    const float t_hi = __fadd_rn(third, p), t_lo = __fadd_rn(__fsub_rn(p, __fsub_rn(t_hi, third)), __fadd_rn(third_lo, p_lo));
    const float y = __fmul_rn(z_hi, t_hi), y_lo = __fmaf_rn(z_hi, t_hi, -y) + (z_hi * t_lo + z_lo * t_hi);
    p = __fmul_rn(s_hi, y);                                   // s + s z t
    p_lo = __fmaf_rn(s_hi, y, -p) + (s_hi * y_lo + s_lo * y);
    const float l_hi = __fadd_rn(s_hi, p), l_lo = __fadd_rn(__fsub_rn(p, __fsub_rn(l_hi, s_hi)), __fadd_rn(s_lo, p_lo));
    if (k == 0)
        return 2.0f * __fadd_rn(l_hi, l_lo);
    const float ln2 = 45426.0f / 65536, ln2_lo = (float)(0.69314718055994530942 - 45426.0 / 65536);   // k ln2 is exact
    const float whole = -(float)k * ln2, sum = __fadd_rn(whole, 2.0f * l_hi);
    return __fadd_rn(sum, __fadd_rn(__fsub_rn(2.0f * l_hi, __fsub_rn(sum, whole)), __fmaf_rn(-(float)k, ln2_lo, 2.0f * l_lo)));
}

// floor(u total) cut to [0, total), and ceil(part total) but at least 1.
__device__ __forceinline__ uint64_t draw_at(float u, uint64_t total)
{
    return u >= 1.0f ? total - 1 : u > 0.0f ? min(product(u, total, false), total - 1) : 0u;
}

__device__ __forceinline__ uint64_t part_of(float part, uint64_t total) { return part > 0.0f ? max((uint64_t)1, product(part, total, true)) : 1u; }

// Mass of all threads.
__device__ uint64_t total_of(Shared *s, uint64_t mass)
{
    const int lane = threadIdx.x & 31;
    mass = warp_sum(mass);
    if (lane == 0)
        s->warp_mass[threadIdx.x >> 5] = mass;
    __syncthreads();
    mass = warp_sum(lane < SM_WARPS ? s->warp_mass[lane] : (uint64_t)0);
    __syncthreads();
    return mass;
}

// The entry of some, each thread having four of them (weights `w`, 0 for none), at which their running
// weight in rising order of `order` reaches `target` (at least 1, and not more than there is), and its
// weight.  `place(j)`, below SM_BINS, rises with the order: the entries of the place in question alone
// are sorted.
struct Entry {
    uint64_t order;
    uint32_t w;
};
template <typename P> __device__ Entry reach(const Row &r, const uint64_t (&order)[4], const uint32_t (&w)[4], uint64_t target, P place)
{
    Shared *s = r.s;
    const int e0 = 4 * (int)threadIdx.x;
    clear_bins<true>(r);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (w[j] > 0)
            add_to_bin(s, place(j), w[j]);
    if (threadIdx.x == 0)
        s->list_n = 0;
    __syncthreads();
    uint64_t m[4], mass = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] = s->low[e0 + j] + ((uint64_t)s->high[e0 + j] << 16);
        mass += m[j];
    }
    uint64_t run = scan(r, mass) - mass;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (run < target && target <= run + m[j]) {
            s->found[0].bin = (uint32_t)(e0 + j);
            s->found[0].mass_above = run;
        }
        run += m[j];
    }
    __syncthreads();                     // (and the bins have been read: the list takes their place)
    const uint32_t bin = s->found[0].bin;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (w[j] > 0 && place(j) == bin) {
            const uint32_t e = atomicAdd(&s->list_n, 1u);
            s->list_order[e] = order[j];
            s->list_w[e] = w[j];
        }
    __syncthreads();
    const int n = (int)s->list_n;
    sorted_list<true>(s, n);
    uint32_t own[4];
    mass = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        own[j] = e0 + j < n ? s->list_w[e0 + j] : 0u;
        mass += own[j];
    }
    run = s->found[0].mass_above + scan(r, mass) - mass;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (run < target && target <= run + own[j]) {
            s->word = s->list_order[e0 + j];
            s->warp_a[0] = own[j];
        }
        run += own[j];
    }
    __syncthreads();
    const Entry found = {s->word, s->warp_a[0]};
    __syncthreads();
    return found;
}

// The whole choice among the `n` logits of a long list, the first `keep` of those of bin `bin` (and
// all of the bins above) being top-k's.  No sort of all: each cut is found by places, a histogram of
// the weights over the bins (top-p) or over ranges of the index (the draw), and one place's entries.
// (Sorted twice, 1000 logits take 20 us longer.)
__device__ void choose_from_long_list(const SampleParams &p, const Row &r, int n, int64_t row, uint32_t bin, int keep, bool by_p, float top_p,
                                      uint32_t least, float u)
{
    Shared *s = r.s;
    uint64_t order[4];
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = (int)threadIdx.x + j * SM_THREADS;
        order[j] = e < n ? s->list_order[e] : ~0ull;
        w[j] = e < n ? s->list_w[e] : 0u;
    }
    auto bin_at = [&](int j) { return bin_of(logit_of(~(uint32_t)(order[j] >> 32)), r); };
    __syncthreads();
    if (threadIdx.x == 0)
        s->list_n = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (w[j] > 0 && bin_at(j) == bin)
            s->list_order[atomicAdd(&s->list_n, 1u)] = order[j];
    __syncthreads();
    if (keep < (int)s->list_n) {
        sorted_list<false>(s, (int)s->list_n);
        const uint64_t last = s->list_order[keep - 1];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = order[j] <= last ? w[j] : 0u;
    }
    __syncthreads();
    if (by_p) {
        const uint64_t target = part_of(top_p, total_of(s, (uint64_t)w[0] + w[1] + w[2] + w[3]));
        const uint64_t last = reach(r, order, w, target, bin_at).order;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = order[j] <= last ? w[j] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = w[j] >= least ? w[j] : 0u;
        order[j] = (uint32_t)order[j];         // the index
    }
    const uint64_t total = total_of(s, (uint64_t)w[0] + w[1] + w[2] + w[3]), at = draw_at(u, total);
    const int shift = max(0, 32 - __clz(p.vocab - 1) - 11);
    const Entry drawn = reach(r, order, w, at + 1, [&](int j) { return (uint32_t)order[j] >> shift; });
    if (threadIdx.x == 0) {
        p.token[row] = (int32_t)drawn.order;
        if (p.logprob)
            p.logprob[row] = log_of_part(drawn.w, total);
    }
}

// The whole choice among the `n` logits of a short list: top-k and top-p along their order, the draw
// along their indices.  Each thread holds four neighbours of the sorted list.
__device__ void choose_from_list(const SampleParams &p, const Row &r, int n, int64_t row, int32_t top_k, bool by_p, float top_p, uint32_t least, float u)
{
    Shared *s = r.s;
    const int e0 = 4 * (int)threadIdx.x;
    sorted_list<true>(s, n);
    uint64_t order[4], mass = 0;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool in = e0 + j < n && e0 + j < top_k;
        order[j] = in ? s->list_order[e0 + j] : ~0ull;
        w[j] = in ? s->list_w[e0 + j] : 0u;
        mass += w[j];
    }
    uint64_t run = scan(r, mass) - mass;       // above this thread's first
    uint64_t target = ~0ull;
    if (by_p) {
        if (threadIdx.x == SM_THREADS - 1)
            s->seg_mass[0] = run + mass;
        __syncthreads();
        target = part_of(top_p, s->seg_mass[0]);
    }
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {              // kept: index and weight in one word
        const bool keep = w[j] > 0 && run < target && w[j] >= least;
        run += w[j];
        order[j] = keep ? (order[j] << 32) | w[j] : ~0ull;
        mine = keep ? e0 + j + 1 : mine;
    }
    // what stays stands at the front, for weights fall along the order
    mine = __reduce_max_sync(dev::FULL_MASK, mine);
    if ((threadIdx.x & 31) == 0)
        s->warp_a[threadIdx.x >> 5] = (uint32_t)mine;
    __syncthreads();
    int kept = 0;
#pragma unroll
    for (int q = 0; q < SM_WARPS; ++q)
        kept = max(kept, (int)s->warp_a[q]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (e0 + j < kept)
            s->list_order[e0 + j] = order[j];
    __syncthreads();
    sorted_list<false>(s, kept);
    mass = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        order[j] = e0 + j < kept ? s->list_order[e0 + j] : ~0ull;
        w[j] = order[j] == ~0ull ? 0u : (uint32_t)order[j];
        mass += w[j];
    }
    run = scan(r, mass) - mass;
    if (threadIdx.x == SM_THREADS - 1)
        s->seg_mass[1] = run + mass;
    __syncthreads();
    const uint64_t total = s->seg_mass[1], at = draw_at(u, total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (run <= at && at < run + w[j]) {
            p.token[row] = (int32_t)(order[j] >> 32);
            if (p.logprob)
                p.logprob[row] = log_of_part(w[j], total);
        }
        run += w[j];
    }
}

template <typename E> __global__ void __launch_bounds__(SM_THREADS, 2) sample_kernel(const SampleParams p, int slice, int seg)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Row r;
    r.s = reinterpret_cast<Shared *>(raw);
    r.l = reinterpret_cast<float *>(raw + sizeof(Shared));
    Shared *s = r.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r.ranks));
    r.rank = cluster_rank();
    r.turn = 0;
    r.slice = slice;
    r.seg = seg;
    const int64_t row = blockIdx.x / r.ranks;
    const int start = (int)r.rank * slice;
    r.n = max(0, min(slice, p.vocab - start));
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");      // waited for behind the loads
    dev::follow_previous_kernel();

    const E *src = static_cast<const E *>(p.logits) + row * p.stride + start;
    // the row's settings, on their way with its logits
    const float t = p.d_temperature ? p.d_temperature[row] : p.temperature, u = p.uniform[row];
    const int32_t top_k = p.d_top_k ? p.d_top_k[row] : p.top_k;
    const float top_p = p.d_top_p ? p.d_top_p[row] : p.top_p, least_p = p.d_min_p ? p.d_min_p[row] : p.min_p;

    // the slice, with NaN as -infinity (fmaxf) and one zero (-0 + 0 = 0)
    float largest = -INFINITY;
    auto put = [&](int i, E v) {
        const float l = fmaxf(__fadd_rn(dev::to_f32(v), 0.0f), -INFINITY);
        r.l[i] = l;
        largest = fmaxf(largest, l);
    };
    constexpr int V = dev::Vec16<E>::N;
    int done = 0;
    if (reinterpret_cast<uintptr_t>(src) % 16 == 0) {
        done = r.n / V * V;
#pragma unroll 4
        for (int i = V * threadIdx.x; i < done; i += V * SM_THREADS) {
            const dev::Vec16<E> v = *reinterpret_cast<const dev::Vec16<E> *>(src + i);
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float4 q;
                q.x = fmaxf(__fadd_rn(dev::to_f32(v.e[j]), 0.0f), -INFINITY);
                q.y = fmaxf(__fadd_rn(dev::to_f32(v.e[j + 1]), 0.0f), -INFINITY);
                q.z = fmaxf(__fadd_rn(dev::to_f32(v.e[j + 2]), 0.0f), -INFINITY);
                q.w = fmaxf(__fadd_rn(dev::to_f32(v.e[j + 3]), 0.0f), -INFINITY);
                *reinterpret_cast<float4 *>(r.l + i + j) = q;
                largest = fmaxf(largest, fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)));
            }
        }
    }
#pragma unroll 8
    for (int i = done + threadIdx.x; i < r.n; i += SM_THREADS)
        put(i, src[i]);
    uint32_t top = key_of(largest), unused = 0xffffffffu;
    if (threadIdx.x < 3 && r.n + (int)threadIdx.x < (r.n + 3) / 4 * 4)
        r.l[r.n + threadIdx.x] = -INFINITY;
    // every CTA of the cluster runs: its shared memory may be written.  (It may end when it is done:
    // the last that any other does with it comes before a barrier of all.)
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    cluster_max_min(r, top, unused);
    if (top == SM_KEY_NONE) {
        if (r.rank == 0 && threadIdx.x == 0) {
            p.token[row] = -1;
            if (p.logprob)
                p.logprob[row] = __uint_as_float(0x7fc00000u);
            dev::flag_error(p.error, LOOM_DEVERR_NO_TOKEN);
        }
        return;
    }
    r.m = logit_of(top);
    if (!(t > 0.0f)) {   // greedy: the first of the largest
        uint32_t none = 0, first = 0xffffffffu;
        for_each(r, [&](float l, int i) {
            if (l == r.m)
                first = min(first, (uint32_t)(start + i));
        });
        cluster_max_min(r, none, first);
        if (r.rank == 0 && threadIdx.x == 0) {
            p.token[row] = (int32_t)first;
            if (p.logprob)
                p.logprob[row] = 0.0f;
        }
        return;
    }
    r.inv = __fdiv_rn(1.0f, t);
    r.bins_per_unit = r.inv * SM_BIN_SCALE;
    if (isinf(r.m) || isinf(r.bins_per_unit)) {
        // The largest logits alone have weight, or (at temperatures near 2^-120) those that differ from
        // them by as little: these are scaled, exactly.
        const bool scaled = !isinf(r.inv) && fabsf(r.m) < 0x1p60f;
        for (int i = threadIdx.x; i < r.n; i += SM_THREADS)
            r.l[i] = scaled ? r.l[i] * 0x1p60f : r.l[i] == r.m ? 0.0f : -INFINITY;
        r.m = scaled ? r.m * 0x1p60f : 0.0f;
        r.inv = scaled ? r.inv * 0x1p-60f : 1.0f;
        r.bins_per_unit = r.inv * SM_BIN_SCALE;
        __syncthreads();
    }

    const float min_p = fminf(fmaxf(least_p, 0.0f), 1.0f);   // NaN: 0
    const uint32_t least = __float2uint_ru(min_p * 2147483648.0f);     // w >= min_p * 2^31 (exact)
    const bool by_k = top_k > 0 && top_k < p.vocab, by_p = top_p < 1.0f;
    Boundary last = {SM_KEY_NONE, 0xffffffffu};   // everything stays
    const Found nothing = {};
    bool cut_k = false;
    if (by_k) {           // counts alone: no exponentials
        clear_bins<false>(r);
        for_fours(r, [&](const float (&l)[4], int) {
            uint32_t bin[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                bin[j] = bin_of(l[j], r);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (takes_part(l[j], bin[j], r))
                    atomicAdd(&s->count[bin[j]], 1u);
        });
        Shares all;
        const Found f = search<false>(r, (uint64_t)top_k, nothing, &all);
        cut_k = all.count > (uint32_t)top_k;
        if (cut_k) {
            // the logits of the bins down to the boundary's, if they are few
            const uint32_t n = f.count_above + f.count;
            if (n <= SM_LIST) {
                gather(r, start, 0, f.bin);
                if (r.rank == 0 && n <= SM_THREADS)
                    choose_from_list(p, r, (int)n, row, top_k, by_p, top_p, least, u);
                else if (r.rank == 0)
                    choose_from_long_list(p, r, (int)n, row, f.bin, top_k - (int)f.count_above, by_p, top_p, least, u);
                return;
            }
            last = refine<false>(r, start, (uint64_t)top_k, f);
        }
    }
    if (by_p) {
        clear_bins<true>(r);
        const float from = logit_of(last.key);         // of the boundary's equals all: the target lies among those that stay
        uint64_t mass = 0;
        for_fours(r, [&](const float (&l)[4], int) {
            uint32_t w[4], bin[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = l[j] >= from ? weight_of(l[j], r.m, r.inv) : 0u;
                bin[j] = bin_of(l[j], r);
                mass += l[j] > from ? w[j] : 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (w[j] > 0)
                    add_to_bin(s, bin[j], w[j]);
        });
        uint64_t all = share(r, scan(r, mass), 0).mass;
        if (cut_k)
            all += (uint64_t)last.keep * weight_of(logit_of(last.key), r.m, r.inv);
        const uint64_t target = part_of(top_p, all);
        last = refine<true>(r, start, target, search<true>(r, target, nothing));
    }

    // kept weight of each segment, its equals of the boundary counted apart
    const float edge = logit_of(last.key);
    uint64_t edge_w = weight_of(edge, r.m, r.inv);
    if (edge_w < least)
        edge_w = 0;
    const int segments = (r.n + seg - 1) / seg;         // (at most SM_SEGMENTS)
    for (int g = warp; g < segments; g += SM_WARPS) {
        uint64_t mass = 0;
        uint32_t ties = 0;
        const int end = min(r.n, (g + 1) * seg);
        for (int i = g * seg + 4 * lane; i < end; i += 128) {
            const float4 q = *reinterpret_cast<const float4 *>(r.l + i);
            const float l[4] = {q.x, q.y, q.z, q.w};
            if (edge_w == 0) {                         // (nothing was cut, or min-p cuts further)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = weight_of(l[j], r.m, r.inv);
                    mass += w >= least ? w : 0u;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = weight_of(l[j], r.m, r.inv);
                    mass += l[j] > edge && w >= least ? w : 0u;
                    ties += l[j] == edge;
                }
            }
        }
        mass = warp_sum(mass);
        if (edge_w > 0)
            ties = warp_sum(ties);
        if (lane == 0) {
            s->seg_mass[g] = mass;
            s->seg_ties[g] = ties;
        }
    }
    __syncthreads();
    uint32_t ties_before = 0, kept_ties = 0;       // the boundary's equals before this thread's segment, and kept in it
    if (edge_w > 0) {
        const uint32_t own_ties = (int)threadIdx.x < segments ? s->seg_ties[threadIdx.x] : 0u, ties = scan(r, own_ties);
        ties_before = ties - own_ties + share(r, 0, ties).count_below;
        kept_ties = ties_before < last.keep ? min(own_ties, last.keep - ties_before) : 0u;
    }
    const uint64_t own_mass = (int)threadIdx.x < segments ? s->seg_mass[threadIdx.x] + kept_ties * edge_w : 0u;
    const uint64_t mass = scan(r, own_mass);       // of the last thread: this CTA's
    const Shares kept = share(r, mass, 0);
    const uint64_t total = kept.mass, before = kept.mass_below + mass - own_mass;
    const uint64_t at = draw_at(u, total);
    if ((int)threadIdx.x < segments && before <= at && at < before + own_mass) {
        s->warp_mass[0] = at - before;      // what to walk into this segment, and with how many equals
        s->warp_count[0] = last.keep > ties_before ? last.keep - ties_before : 0u;
        s->warp_a[0] = threadIdx.x;
    }
    const bool here = __syncthreads_or(threadIdx.x == SM_THREADS - 1 && kept.mass_below <= at && at < kept.mass_below + mass);
    if (here && warp == 0) {
        uint64_t left = s->warp_mass[0];
        uint32_t keep = s->warp_count[0];
        const int g = (int)s->warp_a[0], end = min(r.n, (g + 1) * seg);
        for (int i0 = g * seg; i0 < end; i0 += 128) {      // four neighbours a lane
            const int i = i0 + 4 * lane;
            float l[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (i < end)
                memcpy(l, r.l + i, sizeof(l));             // (filled up with -infinity)
            uint32_t ties = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ties += l[j] == edge;
            uint32_t tie_run = ties;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t q = __shfl_up_sync(dev::FULL_MASK, tie_run, d);
                tie_run += lane >= d ? q : 0u;
            }
            const uint32_t round_ties = __shfl_sync(dev::FULL_MASK, tie_run, 31);
            tie_run -= ties;
            uint32_t w[4];
            uint64_t sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool tie = l[j] == edge, stays = l[j] > edge || (tie && tie_run < keep);
                w[j] = stays ? weight_of(l[j], r.m, r.inv) : 0u;
                w[j] = w[j] >= least ? w[j] : 0u;
                tie_run += tie;
                sum += w[j];
            }
            uint64_t run = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint64_t q = __shfl_up_sync(dev::FULL_MASK, run, d);
                run += lane >= d ? q : 0u;
            }
            const uint32_t past = __ballot_sync(dev::FULL_MASK, run > left);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    run -= sum;
                    int j = 0;
                    while (j < 3 && run + w[j] <= left)
                        run += w[j++];
                    p.token[row] = start + i + j;
                    if (p.logprob)
                        p.logprob[row] = log_of_part(w[j], total);
                }
                break;
            }
            left -= __shfl_sync(dev::FULL_MASK, run, 31);
            keep -= min(keep, round_ties);
        }
    }
}

template <typename E> cudaError_t launch_e(const SampleParams &p, const loom_launch &L, cudaStream_t stream)
{
    const int ranks = (int)L.cluster[0];
    const int slice = ((p.vocab + ranks - 1) / ranks + 15) / 16 * 16;
    const int seg = ((slice + SM_SEGMENTS - 1) / SM_SEGMENTS + 127) / 128 * 128;   // whole rounds of a warp's float4
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(sample_kernel<E>), 0, done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid[0]);
    cfg.blockDim = dim3(L.block[0]);
    cfg.dynamicSmemBytes = L.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<E>, p, slice, seg);
}

}  // namespace

bool sample_geometry(int64_t rows, int32_t vocab, int64_t sms, loom_launch *out)
{
    // Slices of up to SM_SLICE (two CTAs an SM); shorter ones while that leaves SMs without work:
    // a pass over a slice takes as long as it is.
    int ranks = 1;
    while (ranks < SM_MAX_CLUSTER && (vocab > ranks * SM_SLICE || (rows * ranks * 2 <= sms && vocab > ranks * SM_SHORT_SLICE)))
        ranks *= 2;
    if (vocab > ranks * SM_MAX_SLICE || rows * ranks > 0x7fffffff)
        return false;
    *out = loom_launch{};
    out->grid[0] = (uint32_t)(rows * ranks);
    out->block[0] = SM_THREADS;
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = (uint32_t)ranks;
    out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->smem_bytes = (uint32_t)(sizeof(Shared) + ((vocab + ranks - 1) / ranks + 15) / 16 * 16 * sizeof(float));
    out->units_per_cta = 1;
    out->kernel = LOOM_KERNEL_SAMPLE;
    return true;
}

cudaError_t launch_sample(const SampleParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_e<float>(p, L, stream);
    return dtype == LOOM_F16 ? launch_e<__half>(p, L, stream) : launch_e<__nv_bfloat16>(p, L, stream);
}

}  // namespace loom
