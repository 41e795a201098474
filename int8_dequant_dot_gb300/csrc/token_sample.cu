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
//  * No sort.  The k-th logit, and the one where the running weight reaches
//    top_p of the total, are found by histogram: first over 2048 equal bins of
//    (m - l) / T, which spread the bulk of a row over many bins (counts and
//    weights, so one histogram serves both searches), then over the bit patterns
//    of the logits in the bin that holds the boundary, 2048 at a time, until one
//    pattern is left.  Logits whose weight is 0 cannot be chosen and take no part.
//  * Equal logits at the boundary: the number of them that stays follows from the
//    sums alone; the first ones in index order are kept, by a running count over
//    segments of the row.
//  * The draw: kept weight per segment (a warp each), a scan over segments and
//    CTAs, and one warp walks the segment that holds floor(u total).
//  * A weight is added to a bin as two 32-bit halves (its upper and lower 16 bits:
//    no slice can overflow them), which shared memory adds natively.
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int SM_THREADS = 512, SM_WARPS = SM_THREADS / 32;
constexpr int SM_BINS = 2048;
constexpr int SM_MAX_CLUSTER = 8;
constexpr int SM_MAX_SLICE = 49152;        // logits of a CTA: 192 KiB
constexpr int SM_SLICE = 16384;            // slices up to this leave room for a second CTA on the SM
constexpr int SM_SEGMENTS = 128;           // segments of a slice
constexpr uint32_t SM_FULL = 1u << 31;     // the weight of the largest logit
constexpr float SM_BIN_SCALE = 95.0f;      // bins per unit of (m - l) / T: 2^-31 lies in bin 2041
constexpr uint32_t SM_KEY_NONE = 0x007fffffu;   // key of -infinity

// Bit pattern of a logit whose whole-number order is the logits' order.
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float exponent_of(float l, float m, float inv) { return (l - m) * inv; }

__device__ __forceinline__ uint32_t weight_of(float l, float m, float inv)
{
    if (l == m)
        return SM_FULL;
    if (l == -INFINITY)
        return 0;
    return __float2uint_rz(expf(exponent_of(l, m, inv)) * 2147483648.0f);
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

struct Found {            // where a search ended: what lies above bin `bin`
    uint64_t mass_above;
    uint32_t count_above, bin;
};

struct Shared {
    uint32_t count[SM_BINS], low[SM_BINS], high[SM_BINS];
    uint64_t share_mass[SM_MAX_CLUSTER];     // per CTA of the cluster
    uint32_t share_count[SM_MAX_CLUSTER];
    uint32_t key_max[SM_MAX_CLUSTER], key_min[SM_MAX_CLUSTER];
    uint32_t first[SM_MAX_CLUSTER];
    uint32_t ties[SM_MAX_CLUSTER];
    uint64_t mass[SM_MAX_CLUSTER];
    Found found;
    uint64_t warp_mass[SM_WARPS];
    uint32_t warp_count[SM_WARPS], warp_a[SM_WARPS], warp_b[SM_WARPS];
    uint64_t seg_mass[SM_SEGMENTS];
    uint32_t seg_ties[SM_SEGMENTS];
};

struct Row {              // what the threads of a cluster agree on
    Shared *s;
    float *l;             // this CTA's slice
    int n, slice, seg;    // logits of this CTA, of a full slice, of a segment
    uint32_t rank, ranks;
    float m, inv;
};

__device__ __forceinline__ void agree(const Row &r)
{
    if (r.ranks > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Largest a and smallest b over the cluster.
__device__ __forceinline__ void cluster_max_min(const Row &r, uint32_t &a, uint32_t &b)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
        store_remote(&r.s->key_max[r.rank], threadIdx.x, a);
        store_remote(&r.s->key_min[r.rank], threadIdx.x, b);
    }
    agree(r);
    a = 0;
    b = 0xffffffffu;
    for (uint32_t q = 0; q < r.ranks; ++q) {
        a = max(a, r.s->key_max[q]);
        b = min(b, r.s->key_min[q]);
    }
    agree(r);   // before the slots are written again
}

__device__ __forceinline__ void clear_bins(const Row &r)
{
    for (int i = threadIdx.x; i < SM_BINS; i += SM_THREADS)
        r.s->count[i] = r.s->low[i] = r.s->high[i] = 0;
    __syncthreads();
}

__device__ __forceinline__ void add_to_bin(Shared *s, uint32_t bin, uint32_t w)
{
    atomicAdd(&s->count[bin], 1u);
    atomicAdd(&s->low[bin], w & 0xffffu);
    atomicAdd(&s->high[bin], w >> 16);
}

// Inclusive scans over the CTA's threads.
__device__ __forceinline__ void scan(const Row &r, uint64_t &mass, uint32_t &count)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t m = __shfl_up_sync(dev::FULL_MASK, mass, d);
        const uint32_t c = __shfl_up_sync(dev::FULL_MASK, count, d);
        if (lane >= d) {
            mass += m;
            count += c;
        }
    }
    if (lane == 31) {
        r.s->warp_mass[warp] = mass;
        r.s->warp_count[warp] = count;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        mass += r.s->warp_mass[w];
        count += r.s->warp_count[w];
    }
    __syncthreads();
}

// The bin in which the running count (or mass) from bin 0 up reaches `target`,
// given that `start` lies above bin 0; bins of all CTAs together.  Each CTA adds up
// its share of the bins.  Ends agreed: every CTA may clear its bins.
__device__ Found search(const Row &r, bool by_mass, uint64_t target, Found start)
{
    Shared *s = r.s;
    agree(r);   // every histogram is complete
    constexpr int MOST = SM_BINS / SM_THREADS;      // bins per thread with one CTA
    const int share = SM_BINS / (int)r.ranks;
    const int per = share >= SM_THREADS ? share / SM_THREADS : 1;
    const int bin0 = (int)r.rank * share + (int)threadIdx.x * per;
    uint64_t m[MOST], mass = 0;
    uint32_t c[MOST], count = 0;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        m[j] = 0;
        c[j] = 0;
        if (j < per && (int)threadIdx.x * per + j < share)
            for (uint32_t q = 0; q < r.ranks; ++q) {
                c[j] += load_remote(&s->count[bin0 + j], q);
                m[j] += load_remote(&s->low[bin0 + j], q) + ((uint64_t)load_remote(&s->high[bin0 + j], q) << 16);
            }
        mass += m[j];
        count += c[j];
    }
    const uint64_t own_mass = mass;
    const uint32_t own_count = count;
    scan(r, mass, count);
    if (threadIdx.x == SM_THREADS - 1)
        for (uint32_t q = 0; q < r.ranks; ++q) {
            store_remote(&s->share_mass[r.rank], q, mass);
            store_remote(&s->share_count[r.rank], q, count);
        }
    agree(r);
    uint64_t above_mass = start.mass_above + mass - own_mass;
    uint32_t above_count = start.count_above + count - own_count;
    for (uint32_t q = 0; q < r.rank; ++q) {
        above_mass += s->share_mass[q];
        above_count += s->share_count[q];
    }
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const uint64_t before = by_mass ? above_mass : above_count, has = by_mass ? m[j] : c[j];
        if (before < target && target <= before + has)
            for (uint32_t q = 0; q < r.ranks; ++q) {
                store_remote(&s->found.mass_above, q, above_mass);
                store_remote(&s->found.count_above, q, above_count);
                store_remote(&s->found.bin, q, (uint32_t)(bin0 + j));
            }
        above_mass += m[j];
        above_count += c[j];
    }
    agree(r);
    const Found f = s->found;
    agree(r);   // before `found` is written again
    return f;
}

__device__ __forceinline__ uint32_t bin_of(float l, float m, float inv)
{
    return (uint32_t)min(SM_BINS - 1, (int)(-exponent_of(l, m, inv) * SM_BIN_SCALE));
}

struct Boundary {        // the last logit that stays, and how many of its equals
    uint32_t key, keep;
    uint64_t mass;       // kept in all
};

// The boundary in bin `f.bin` of the first histogram: `target` is reached there.
__device__ Boundary refine(const Row &r, bool by_mass, uint64_t target, Found f)
{
    uint32_t hi = 0, lo = 0xffffffffu;
    for (int i = threadIdx.x; i < r.n; i += SM_THREADS) {
        const float l = r.l[i];
        if (weight_of(l, r.m, r.inv) > 0 && bin_of(l, r.m, r.inv) == f.bin) {
            hi = max(hi, key_of(l));
            lo = min(lo, key_of(l));
        }
    }
    cluster_max_min(r, hi, lo);
    for (int level = 0; level < 3 && hi > lo; ++level) {   // bins of equal size, the largest keys first
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        clear_bins(r);
        for (int i = threadIdx.x; i < r.n; i += SM_THREADS) {
            const float l = r.l[i];
            const uint32_t key = key_of(l);
            if (key >= lo && key <= hi) {
                const uint32_t w = weight_of(l, r.m, r.inv);
                if (w > 0)
                    add_to_bin(r.s, (hi - key) >> shift, w);
            }
        }
        f = search(r, by_mass, target, f);
        hi -= f.bin << shift;
        lo = max(lo, hi - min(hi, (1u << shift) - 1));
    }
    const float l = __uint_as_float(hi ^ ((hi >> 31) ? 0x80000000u : 0xffffffffu));
    const uint64_t w = weight_of(l, r.m, r.inv);
    Boundary b;
    b.key = hi;
    b.keep = by_mass ? (uint32_t)((target - f.mass_above + w - 1) / w) : (uint32_t)target - f.count_above;
    b.mass = f.mass_above + b.keep * w;
    return b;
}

template <typename E> __global__ void __launch_bounds__(SM_THREADS) sample_kernel(const SampleParams p, int slice, int seg)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Row r;
    r.s = reinterpret_cast<Shared *>(raw);
    r.l = reinterpret_cast<float *>(raw + sizeof(Shared));
    Shared *s = r.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r.ranks));
    r.rank = cluster_rank();
    r.slice = slice;
    r.seg = seg;
    const int64_t row = blockIdx.x / r.ranks;
    const int start = (int)r.rank * slice;
    r.n = max(0, min(slice, p.vocab - start));
    dev::follow_previous_kernel();

    // the slice, with NaN as -infinity and one zero
    const E *src = static_cast<const E *>(p.logits) + row * p.stride + start;
    uint32_t top = SM_KEY_NONE, unused = 0xffffffffu;
    constexpr int V = dev::Vec16<E>::N;
    if (reinterpret_cast<uintptr_t>(src) % 16 == 0) {
        const int whole = r.n / V;
        for (int i = threadIdx.x; i < whole; i += SM_THREADS) {
            const dev::Vec16<E> v = reinterpret_cast<const dev::Vec16<E> *>(src)[i];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float l = __fadd_rn(dev::to_f32(v.e[j]), 0.0f);
                l = l == l ? l : -INFINITY;
                r.l[i * V + j] = l;
                top = max(top, key_of(l));
            }
        }
        for (int i = whole * V + threadIdx.x; i < r.n; i += SM_THREADS) {
            float l = __fadd_rn(dev::to_f32(src[i]), 0.0f);
            l = l == l ? l : -INFINITY;
            r.l[i] = l;
            top = max(top, key_of(l));
        }
    } else {
        for (int i = threadIdx.x; i < r.n; i += SM_THREADS) {
            float l = __fadd_rn(dev::to_f32(src[i]), 0.0f);
            l = l == l ? l : -INFINITY;
            r.l[i] = l;
            top = max(top, key_of(l));
        }
    }
    agree(r);   // every CTA of the cluster runs: its shared memory may be written
    cluster_max_min(r, top, unused);
    if (top == SM_KEY_NONE) {
        if (r.rank == 0 && threadIdx.x == 0) {
            p.token[row] = -1;
            if (p.logprob)
                p.logprob[row] = __uint_as_float(0x7fc00000u);
            dev::flag_error(p.error, LOOM_DEVERR_NO_TOKEN);
        }
        agree(r);
        return;
    }
    r.m = __uint_as_float(top ^ ((top >> 31) ? 0x80000000u : 0xffffffffu));
    const float t = p.d_temperature ? p.d_temperature[row] : p.temperature;
    if (!(t > 0.0f)) {   // greedy: the first of the largest
        uint32_t none = 0, first = 0xffffffffu;
        for (int i = threadIdx.x; i < r.n; i += SM_THREADS)
            if (r.l[i] == r.m)
                first = min(first, (uint32_t)(start + i));
        cluster_max_min(r, none, first);
        if (r.rank == 0 && threadIdx.x == 0) {
            p.token[row] = (int32_t)first;
            if (p.logprob)
                p.logprob[row] = 0.0f;
        }
        agree(r);
        return;
    }
    r.inv = __fdiv_rn(1.0f, t);

    const int32_t top_k = p.d_top_k ? p.d_top_k[row] : p.top_k;
    const float top_p = p.d_top_p ? p.d_top_p[row] : p.top_p;
    const float min_p = fminf(fmaxf(p.d_min_p ? p.d_min_p[row] : p.min_p, 0.0f), 1.0f);   // NaN: 0
    const double min_w = (double)min_p * 2147483648.0;
    const bool by_k = top_k > 0 && top_k < p.vocab, by_p = top_p < 1.0f;
    Boundary last = {SM_KEY_NONE, 0xffffffffu, 0};   // everything stays
    if (by_k || by_p) {
        clear_bins(r);
        uint64_t mass = 0;
        uint32_t count = 0;
        for (int i = threadIdx.x; i < r.n; i += SM_THREADS) {
            const uint32_t w = weight_of(r.l[i], r.m, r.inv);
            if (w > 0) {
                add_to_bin(s, bin_of(r.l[i], r.m, r.inv), w);
                mass += w;
                ++count;
            }
        }
        scan(r, mass, count);
        if (threadIdx.x == SM_THREADS - 1)
            for (uint32_t q = 0; q < r.ranks; ++q) {
                store_remote(&s->mass[r.rank], q, mass);
                store_remote(&s->ties[r.rank], q, count);
            }
        agree(r);
        uint64_t all = 0;
        uint32_t choices = 0;
        for (uint32_t q = 0; q < r.ranks; ++q) {
            all += s->mass[q];
            choices += s->ties[q];
        }
        const Found nothing = {0, 0, 0};
        Found at_k = nothing, at_p = nothing;
        const bool cut_k = by_k && choices > (uint32_t)top_k;
        if (cut_k)
            at_k = search(r, false, (uint64_t)top_k, nothing);
        // top-p's target needs the mass that top-k leaves, and the first histogram: keep
        // that histogram by searching for the boundary bin once the mass is known; the
        // refinement of top-k overwrites it, so it is built again only when both cut.
        if (cut_k) {
            last = refine(r, false, (uint64_t)top_k, at_k);
            all = last.mass;
            if (by_p) {
                clear_bins(r);
                for (int i = threadIdx.x; i < r.n; i += SM_THREADS) {
                    const float l = r.l[i];
                    if (key_of(l) >= last.key) {
                        const uint32_t w = weight_of(l, r.m, r.inv);
                        if (w > 0)
                            add_to_bin(s, bin_of(l, r.m, r.inv), w);
                    }
                }
            }
        }
        if (by_p) {
            const double want = ceil((double)top_p * (double)all);
            const uint64_t target = want >= 1.0 ? (uint64_t)want : 1u;   // a NaN top_p: the first alone
            at_p = search(r, true, target, nothing);
            last = refine(r, true, target, at_p);
        }
    }

    // kept weight of each segment, its equals of the boundary counted apart
    const float edge = __uint_as_float(last.key ^ ((last.key >> 31) ? 0x80000000u : 0xffffffffu));
    uint64_t edge_w = weight_of(edge, r.m, r.inv);
    if ((double)edge_w < min_w)
        edge_w = 0;
    for (int g = warp; g < SM_SEGMENTS; g += SM_WARPS) {
        uint64_t mass = 0;
        uint32_t ties = 0;
        const int end = min(r.n, (g + 1) * seg);
        for (int i = g * seg + lane; i < end; i += 32) {
            const float l = r.l[i];
            if (l > edge) {
                const uint32_t w = weight_of(l, r.m, r.inv);
                mass += (double)w >= min_w ? w : 0u;
            } else if (l == edge) {
                ++ties;
            }
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            mass += __shfl_xor_sync(dev::FULL_MASK, mass, d);
        ties = __reduce_add_sync(dev::FULL_MASK, ties);
        if (lane == 0) {
            s->seg_mass[g] = mass;
            s->seg_ties[g] = ties;
        }
    }
    __syncthreads();
    uint64_t mass = 0;
    uint32_t ties = threadIdx.x < SM_SEGMENTS ? s->seg_ties[threadIdx.x] : 0u;
    const uint32_t own_ties = ties;
    scan(r, mass, ties);
    if (threadIdx.x == SM_THREADS - 1)
        for (uint32_t q = 0; q < r.ranks; ++q)
            store_remote(&s->ties[r.rank], q, ties);
    agree(r);
    uint32_t ties_before = ties - own_ties;    // of this thread's segment
    for (uint32_t q = 0; q < r.rank; ++q)
        ties_before += s->ties[q];
    const uint32_t kept_ties = ties_before < last.keep ? min(own_ties, last.keep - ties_before) : 0u;
    uint32_t none = 0;
    const uint64_t own_mass = threadIdx.x < SM_SEGMENTS ? s->seg_mass[threadIdx.x] + kept_ties * edge_w : 0u;
    mass = own_mass;
    scan(r, mass, none);
    if (threadIdx.x == SM_THREADS - 1)
        for (uint32_t q = 0; q < r.ranks; ++q)
            store_remote(&s->mass[r.rank], q, mass);
    agree(r);
    uint64_t total = 0, before = mass - own_mass;
    for (uint32_t q = 0; q < r.ranks; ++q) {
        if (q < r.rank)
            before += s->mass[q];
        total += s->mass[q];
    }
    const double drawn = floor((double)p.uniform[row] * (double)total);
    const uint64_t at = drawn >= (double)total ? total - 1 : drawn > 0.0 ? (uint64_t)drawn : 0u;
    if (threadIdx.x < SM_SEGMENTS && before <= at && at < before + own_mass) {
        s->warp_mass[0] = at - before;      // what to walk into this segment, and with how many equals
        s->warp_count[0] = last.keep > ties_before ? last.keep - ties_before : 0u;
        s->warp_a[0] = threadIdx.x;
    }
    uint64_t base = 0;
    for (uint32_t q = 0; q < r.rank; ++q)
        base += s->mass[q];
    const bool here = base <= at && at < base + s->mass[r.rank];
    __syncthreads();
    if (here && warp == 0) {
        uint64_t left = s->warp_mass[0];
        uint32_t keep = s->warp_count[0];
        const int g = (int)s->warp_a[0], end = min(r.n, (g + 1) * seg);
        for (int i0 = g * seg; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            const float l = i < end ? r.l[i] : -INFINITY;
            const uint32_t tie_lanes = __ballot_sync(dev::FULL_MASK, i < end && l == edge);
            const uint32_t mine = __popc(tie_lanes & ((1u << lane) - 1u));
            uint64_t w = 0;
            if (i < end && (l > edge || (l == edge && mine < keep))) {
                w = weight_of(l, r.m, r.inv);
                w = (double)w >= min_w ? w : 0u;
            }
            uint64_t run = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint64_t q = __shfl_up_sync(dev::FULL_MASK, run, d);
                if (lane >= d)
                    run += q;
            }
            const uint32_t past = __ballot_sync(dev::FULL_MASK, run > left);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    p.token[row] = start + i;
                    if (p.logprob)
                        p.logprob[row] = (float)log((double)w / (double)total);
                }
                break;
            }
            left -= __shfl_sync(dev::FULL_MASK, run, 31);
            keep -= min(keep, (uint32_t)__popc(tie_lanes));
        }
    }
    agree(r);   // no CTA ends while another may read its shared memory
}

template <typename E> cudaError_t launch_e(const SampleParams &p, const loom_launch &L, cudaStream_t stream)
{
    const int ranks = (int)L.cluster[0];
    const int slice = ((p.vocab + ranks - 1) / ranks + 15) / 16 * 16;
    const int seg = ((slice + SM_SEGMENTS - 1) / SM_SEGMENTS + 31) / 32 * 32;
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

bool sample_geometry(int64_t rows, int32_t vocab, int32_t, int64_t, loom_launch *out)
{
    int ranks = 1;
    while (ranks < SM_MAX_CLUSTER && vocab > ranks * SM_SLICE)
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
