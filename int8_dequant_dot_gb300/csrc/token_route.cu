// token_route.cu -- routing: the experts of each token and their weights from logits, and the
// gradient of those weights (sm_103a).
//
// Design
//  * A warp takes a token, a lane a run of neighbouring experts in registers (1 to 32 of them), so that a tie's
//    lowest expert is the lowest lane's, and groups of experts mostly are runs of lanes (others go by shared memory).
//  * The choice is that of real numbers, made in f32 where f32 tells: with no bias (or the same for all) the order of scores
//    is that of the logits; else the scores plus bias are ranked with a bound of their error, and a token whose
//    order it leaves open (two neighbours among the chosen and the next one, or groups at the cut, nearer than that)
//    is ranked in 64 bits, of those experts alone that may make a difference, one a lane (all of a token's where they are
//    more than 32, or where there are more than 32 groups).  A sum's bound goes by its own size, so that a finite mask in the
//    bias (-1e9, the lowest f32) opens no other expert's order: 16384 x 256 take 19.8 us with one or with half of them masked, 19.7 without.
//    64-bit units are few on this GPU (2 lanes an SM and clock): all tokens of 16384 x 256 would
//    take 640 us, and a single one in full held up the kernel for 25 us; of normal logits one in a thousand is open.
//  * The chosen ones are found top_k + 1 times as the warp's maximum of the lanes' largest keys.  A key is a float as
//    an ordered whole number whose last 5 to 10 bits are the expert's, so that the maximum names it; a lane has its keys
//    sorted (16 and more are searched) and drops the first.  Where two neighbours differ in those bits alone (1 token
//    in 200 of normal logits) the choice is made again with whole keys, and where f32 leaves sigmoids' order
//    open, in 64 bits for those near the last one chosen.
//    What bounds many tokens is the instructions of that, not the logits' bytes.
//
// Measured as nodes of a CUDA graph: 1 x 64 2.0 us (a call through the binding 13, the host's part); 16384 x 256 f32, sigmoid, top 8:
// 14.4 us, with a bias 19.7, with 4 of 8 groups as well 25.6 (1195 instructions a token, 2.7 a clock); softmax 37.2; with 16 of 64
// groups, all in 64 bits, 600.  Gradient of 16384 x 256: 7.6 us renormalised, 10.2 of a softmax over all.
#include <cfloat>

#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int RT_WARPS = 4, RT_CTAS = 8;

// Places of 64 bits of a warp where f32 may not tell: two for each expert, or 32 groups' bounds and a list of 32 experts.
__host__ __device__ constexpr int exact_places(int experts) { return experts < 16 ? 32 : 2 * experts; }

// +infinity counts as the largest finite f32; NaN (and -infinity) as -infinity.
__device__ __forceinline__ float logit_of(float l) { return isnan(l) ? -INFINITY : fminf(l, FLT_MAX); }

__device__ __forceinline__ double warp_max(double v)
{
    for (int m = 16; m >= 1; m >>= 1)
        v = fmax(v, __shfl_xor_sync(dev::FULL_MASK, v, m));
    return v;
}

__device__ __forceinline__ double warp_sum(double v)
{
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(dev::FULL_MASK, v, m);
    return v;
}

// The place of the largest of v[0..n) (the lowest among equals), or -1 where all are -infinity.
__device__ int warp_argmax(const double *v, int n, int lane)
{
    double best = -INFINITY;
    int at = -1;
    for (int i = lane; i < n; i += 32)
        if (v[i] > best) {
            best = v[i];
            at = i;
        }
    for (int m = 16; m >= 1; m >>= 1) {
        const double b = __shfl_xor_sync(dev::FULL_MASK, best, m);
        const int a = __shfl_xor_sync(dev::FULL_MASK, at, m);
        if (b > best || (b == best && (unsigned)a < (unsigned)at)) {
            best = b;
            at = a;
        }
    }
    return at;
}

__device__ __forceinline__ double score_of(int kind, double l, double m, double sum)
{
    return kind == LOOM_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / sum;
}

// The experts of a token in 64 bits: the chosen one of each lane below top_k, or -1.  choose: [2][experts], the warp's.
// ranked: experts by scores and bias, else by logits; by_sums: groups by scores and bias, else by logits.
template <typename E>
__device__ __noinline__ int route_exactly(const RouteParams &p, const E *l, double *choose, int lane, bool ranked, bool by_sums)
{
    double *group = choose + p.experts;
    double m = -INFINITY, sum = 0;
    for (int e = lane; e < p.experts; e += 32)
        m = fmax(m, (double)logit_of(dev::to_f32(l[e])));
    m = warp_max(m);
    if (p.score == LOOM_SCORE_SOFTMAX && m > -INFINITY) {
        for (int e = lane; e < p.experts; e += 32)
            sum += exp((double)logit_of(dev::to_f32(l[e])) - m);
        sum = warp_sum(sum);
    }
    for (int e = lane; e < p.experts; e += 32) {
        const float v = logit_of(dev::to_f32(l[e]));
        const float b = p.bias ? logit_of(p.bias[e]) : 0.0f;
        choose[e] = v == -INFINITY || b == -INFINITY ? -INFINITY : ranked || by_sums ? score_of(p.score, v, m, sum) + (double)b : (double)v;
    }
    __syncwarp();
    if (p.groups > 1) {
        const int size = p.experts / p.groups;
        for (int g = lane; g < p.groups; g += 32) {
            double a = -INFINITY, b = -INFINITY;
            for (int i = 0; i < size; ++i) {
                const double v = choose[g * size + i];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            group[g] = p.group_best == 2 && b > -INFINITY ? a + b : a;
        }
        __syncwarp();
        for (int i = 0; i < p.top_groups; ++i) {
            const int g = warp_argmax(group, p.groups, lane);
            __syncwarp();
            if (g >= 0 && lane == 0)
                group[g] = NAN;        // kept: never the largest again
            __syncwarp();
        }
        for (int e = lane; e < p.experts; e += 32)
            if (!isnan(group[e / size]))
                choose[e] = -INFINITY;
            else if (!ranked && choose[e] > -INFINITY)
                choose[e] = (double)logit_of(dev::to_f32(l[e]));
        __syncwarp();
    }
    int mine = -1;
    for (int i = 0; i < p.top_k; ++i) {
        const int e = warp_argmax(choose, p.experts, lane);
        if (lane == i)
            mine = e;
        __syncwarp();
        if (e >= 0 && lane == 0)
            choose[e] = -INFINITY;
        __syncwarp();
    }
    return mine;
}

__device__ __forceinline__ float warp_sum_f(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(dev::FULL_MASK, v, m);
    return v;
}

// A float as a whole number of the same order; INT_MIN is what cannot be chosen.
__device__ __forceinline__ int key_of(float v)
{
    const int b = __float_as_int(v);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float float_of(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7fffffff)); }
constexpr int RT_NONE = -0x7fffffff - 1;
constexpr float RT_UNIT = 6.1e-8f;               // a rounding of f32, 2^-24 of its result, with room for those of a bound

__device__ __forceinline__ float warp_max_f(float v) { return float_of(__reduce_max_sync(dev::FULL_MASK, key_of(v))); }      // (of no NaN)

// Falling order of N keys, by the merging network of Batcher (1968).
template <int N> __device__ __forceinline__ void sort_keys(int (&k)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (j + i + q < N && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
                        const int a = k[j + i], b = k[j + i + q];
                        k[j + i] = max(a, b);
                        k[j + i + q] = min(a, b);
                    }
}

// A lane's PER neighbouring values of a row of n, -infinity past it.  `packs`: accesses of several elements are aligned
// and lie in the row or past it as a whole.
template <typename E, int PER> __device__ __forceinline__ void load_run(const E *row, int n, bool packs, int lane, float (&v)[PER])
{
    constexpr int C = PER < 16 / (int)sizeof(E) ? PER : 16 / (int)sizeof(E);
    struct alignas(sizeof(E) * C) Pack {
        E e[C];
    };
    if (packs) {
#pragma unroll
        for (int i = 0; i < PER / C; ++i) {
            const int at = lane * PER + i * C;
            Pack q;
            if (at < n)
                q = *reinterpret_cast<const Pack *>(row + at);
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[i * C + j] = at < n ? dev::to_f32(q.e[j]) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            v[j] = lane * PER + j < n ? dev::to_f32(row[lane * PER + j]) : -INFINITY;
    }
}

template <typename E, int PER> __host__ __device__ bool packs_of(const void *row, int64_t stride, int n)
{
    constexpr int C = PER < 16 / (int)sizeof(E) ? PER : 16 / (int)sizeof(E);
    return reinterpret_cast<uintptr_t>(row) % (sizeof(E) * C) == 0 && stride % C == 0 && n % C == 0;
}

// The experts of a warp whose bits are set (lane's run, PER each), up to 32 of them, on a list in the experts' order;
// returns their number, which may be more.
template <int PER> __device__ __forceinline__ int list_of(unsigned own, int *list, int lane)
{
    int run = __popc(own);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(dev::FULL_MASK, run, d);
        run += lane >= d ? up : 0;
    }
    const int all = __shfl_sync(dev::FULL_MASK, run, 31);
    if (all <= 32) {
        run -= __popc(own);
        for (unsigned left = own; left; left &= left - 1u)
            list[run++] = lane * PER + __ffs(left) - 1;
    }
    __syncwarp();
    return all;
}

// In 64 bits the score and bias of the lane's expert (of no expert: -infinity).  Without a bias softmax scores may
// have any common factor.
template <typename E> __device__ __noinline__ double precise_score(const RouteParams &p, const E *l, int e, int lane)
{
    double m = 0, sum = 1;
    if (p.score == LOOM_SCORE_SOFTMAX) {
        m = -INFINITY;
        for (int i = lane; i < p.experts; i += 32)
            m = fmax(m, (double)logit_of(dev::to_f32(l[i])));
        m = warp_max(m);
        if (p.bias) {
            sum = 0;
            for (int i = lane; i < p.experts; i += 32)
                sum += exp((double)logit_of(dev::to_f32(l[i])) - m);
            sum = warp_sum(sum);
        }
    }
    if (e < 0)
        return -INFINITY;
    return score_of(p.score, (double)logit_of(dev::to_f32(l[e])), m, sum) + (p.bias ? (double)logit_of(p.bias[e]) : 0.0);
}

template <typename E, int PER, bool GROUPS>
__global__ void __launch_bounds__(32 * RT_WARPS, PER <= 8 ? RT_CTAS : 3) route_kernel(const RouteParams p, int close, int packs)
{
    extern __shared__ double route_smem[];           // [warps][exact_places] where f32 may not tell, then the counts
    dev::follow_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *exact = route_smem + (size_t)warp * exact_places(p.experts);
    int *counts = reinterpret_cast<int *>(route_smem + (close ? (size_t)RT_WARPS * exact_places(p.experts) : 0));
    if (p.counts) {
        for (int e = threadIdx.x; e < p.experts; e += 32 * RT_WARPS)
            counts[e] = 0;
        __syncthreads();
    }
    const bool soft = p.score == LOOM_SCORE_SOFTMAX;
    // the bias of the lane's experts, and whether it is the same for all
    float bias[PER];
    bool ranked = false;                             // by scores and bias; else by logits
    if (p.bias) {
        float low = INFINITY, high = -INFINITY;
        load_run<float, PER>(p.bias, p.experts, packs_of<float, PER>(p.bias, 0, p.experts), lane, bias);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            bias[j] = logit_of(bias[j]);
            if (bias[j] > -INFINITY) {
                low = fminf(low, bias[j]);
                high = fmaxf(high, bias[j]);
            }
        }
        low = -warp_max_f(-low);
        high = warp_max_f(high);
        ranked = low < high;
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            bias[j] = 0.0f;
    }
    const bool by_sums = GROUPS && (p.group_best == 2 || ranked);
    const int members = GROUPS ? p.experts / p.groups : PER;
    // groups that are runs of a power of two of whole lanes: of so many, else 0
    const int runs = members % PER == 0 && (members / PER & (members / PER - 1)) == 0 ? members / PER : 0;
    const bool scored = ranked || by_sums;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < p.tokens; t += (int64_t)gridDim.x * RT_WARPS) {
        const E *l = static_cast<const E *>(p.logits) + t * p.stride;
        float v[PER], score[PER];
        load_run<E, PER>(l, p.experts, packs, lane, v);
        float m = -INFINITY, sum = 0.0f, largest = 1.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            v[j] = logit_of(v[j]);
        if (soft && (scored || !p.renormalise)) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                m = fmaxf(m, v[j]);
            m = warp_max_f(m);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                score[j] = v[j] > -INFINITY ? expf(v[j] - m) : 0.0f;
                sum += score[j];
            }
            sum = warp_sum_f(sum);
        }
        if (scored) {
            if (soft) {
                largest = 1.0f / sum;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    score[j] = __fdiv_rn(score[j], sum);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    score[j] = __fdividef(1.0f, 1.0f + __expf(-v[j]));
            }
#pragma unroll
            for (int j = 0; j < PER; ++j)
                score[j] += bias[j];
        }
        // Bound of a score's error.  Sigmoid s: the exponential's 2 + 1.173 |l| units in the last place (2^-23), of
        // which s (1 - s), 0.63 units at most, passes on; a rounding; the quotient's 2 units: below 2^-21.  Softmax:
        // exponential and difference, s |l - m| 2^-24 <= 0.37 2^-24 and 4 2^-24 s; the sum's terms the same on average
        // (their |l - m| is an entropy, below 7) and 37 + 5 roundings; below 2^-18 (s + 2^-7).  And the rounding of its
        // own sum with the bias: a low bias, such as a mask's, makes that of no other one less sure.
        const float of_score = soft ? 3.8146973e-6f * (largest + 0.0078125f) : 4.7683716e-7f;
        const auto told = [&](float a, float b) { return a - b > 2.0f * (of_score + RT_UNIT * fmaxf(fabsf(a), fabsf(b))); };     // a is above b
        const auto reach = [&](float a) { return a - 4.0f * (of_score + RT_UNIT * fabsf(a)); };      // what is below it is below a's
        int key[PER];
        bool open = false;                           // f32 does not tell
#pragma unroll
        for (int j = 0; j < PER; ++j)                // (+ 0: the two zeros are equal)
            key[j] = v[j] == -INFINITY || bias[j] == -INFINITY ? RT_NONE : key_of((ranked ? score[j] : v[j]) + 0.0f);
        if (GROUPS && p.groups > 32) {
            open = true;
        } else if (GROUPS) {
            // lane g has group g's value: its best, or half of its two best ones' sum, which f32 holds whatever they are
            float best1 = -INFINITY, best2 = -INFINITY;
            if (runs > 0) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float q = key[j] == RT_NONE ? -INFINITY : by_sums ? score[j] : v[j];
                    best2 = fmaxf(best2, fminf(best1, q));
                    best1 = fmaxf(best1, q);
                }
                for (int d = 1; d < runs; d <<= 1) {
                    const float o1 = __shfl_xor_sync(dev::FULL_MASK, best1, d), o2 = __shfl_xor_sync(dev::FULL_MASK, best2, d);
                    best2 = fmaxf(fmaxf(best2, o2), fminf(best1, o1));
                    best1 = fmaxf(best1, o1);
                }
                const int at = lane < p.groups ? lane * runs : 0;
                best1 = __shfl_sync(dev::FULL_MASK, best1, at);
                best2 = __shfl_sync(dev::FULL_MASK, best2, at);
            } else {                                 // groups that are no runs of lanes, by way of shared memory
                float *all = reinterpret_cast<float *>(exact);
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (lane * PER + j < p.experts)
                        all[lane * PER + j] = key[j] == RT_NONE ? -INFINITY : by_sums ? score[j] : v[j];
                __syncwarp();
                for (int g = 0; g < p.groups; ++g) {
                    float a = -INFINITY, b = -INFINITY;
                    for (int i = lane; i < members; i += 32) {
                        const float q = all[g * members + i];
                        b = fmaxf(b, fminf(a, q));
                        a = fmaxf(a, q);
                    }
                    const float first = warp_max_f(a);
                    const int from = __ffs(__ballot_sync(dev::FULL_MASK, a == first)) - 1;
                    const float second = warp_max_f(lane == from ? b : a);
                    if (lane == g) {
                        best1 = first;
                        best2 = second;
                    }
                }
                __syncwarp();
            }
            const bool has = lane < p.groups && best1 > -INFINITY;      // (two lowest finite scores make no empty group)
            const float own = !has ? -INFINITY : p.group_best == 1 ? best1 : 0.5f * best1 + (best2 > -INFINITY ? 0.5f * best2 : 0.0f);
            int above = 0;                           // groups that come before this lane's
            for (int g = 0; g < p.groups; ++g) {
                const float other = __shfl_sync(dev::FULL_MASK, own, g);
                above += other > own || (other == own && g < lane);
            }
            bool stays = above < p.top_groups && has;
            // Bound of own's error: of_score and a rounding with the bias (2^-24 of the sum, 6.1e-8 with room) of each one, as
            // much again of the halves' sum, none above the larger's, and of own - off and own + off.
            const float size1 = fabsf(best1), size2 = best2 > -INFINITY ? fabsf(best2) : 0.0f;
            const float off = of_score + 3.0f * RT_UNIT * fmaxf(size1, size2);
            const float lowest = -warp_max_f(stays ? off - own : -INFINITY), highest = warp_max_f(has && !stays ? own + off : -INFINITY);
            if (by_sums && highest > -INFINITY && !(lowest > highest)) {
                // the groups that may be on either side of the cut, in 64 bits: of each those members that may count
                const bool surely = stays && own - off > highest, near = has && !surely && own + off >= lowest;
                const int sure = __popc(__ballot_sync(dev::FULL_MASK, surely));
                float *least = reinterpret_cast<float *>(exact);
                int *list = reinterpret_cast<int *>(exact) + 32;
                const float last = p.group_best == 2 && best2 > -INFINITY ? best2 : best1;
                if (lane < p.groups)
                    least[lane] = !near ? INFINITY : reach(last);
                __syncwarp();
                unsigned wanted = 0;
                int group = lane * PER / members, left = members - (lane * PER - group * members);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (lane * PER + j < p.experts)
                        wanted |= (unsigned)(key[j] != RT_NONE && score[j] >= least[group]) << j;
                    if (--left == 0) {
                        ++group;
                        left = members;
                    }
                }
                __syncwarp();
                const int n = list_of<PER>(wanted, list, lane);
                if (n > 32) {
                    open = true;
                } else {
                    const int e = lane < n ? list[lane] : -1;
                    const double score64 = precise_score<E>(p, l, e, lane);
                    double first = -INFINITY, second = -INFINITY;
                    for (int i = 0; i < n; ++i) {
                        const double q = __shfl_sync(dev::FULL_MASK, score64, i);
                        if (__shfl_sync(dev::FULL_MASK, e, i) / members == lane) {
                            second = fmax(second, fmin(first, q));
                            first = fmax(first, q);
                        }
                    }
                    const double own64 = !near ? -INFINITY : p.group_best == 2 && second > -INFINITY ? first + second : first;
                    int above64 = sure;
                    for (int g = 0; g < p.groups; ++g) {
                        const double other = __shfl_sync(dev::FULL_MASK, own64, g);
                        above64 += other > own64 || (other == own64 && other > -INFINITY && g < lane);
                    }
                    stays = surely || (near && above64 < p.top_groups);
                }
            }
            const unsigned kept = __ballot_sync(dev::FULL_MASK, stays);
            int group = lane * PER / members, left = members - (lane * PER - group * members);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (!((kept >> (group & 31)) & 1u))
                    key[j] = RT_NONE;
                if (--left == 0) {
                    ++group;
                    left = members;
                }
            }
        }
        int mine = -1;
        bool again = false;                          // the first bits of two keys are alike
        float least = -INFINITY;                     // of the chosen ones, not above it
        if (!open) {
            constexpr int LOW = PER * 32 - 1;
            int u[PER], own = RT_NONE, top = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                u[j] = key[j] == RT_NONE ? RT_NONE : (key[j] & ~LOW) | (LOW - (lane * PER + j));
            if (PER <= 8)
                sort_keys(u);
            for (int i = 0; i <= p.top_k; ++i) {
                int best = u[0];
                if (PER > 8)
#pragma unroll
                    for (int j = 1; j < PER; ++j)
                        best = max(best, u[j]);
                top = __reduce_max_sync(dev::FULL_MASK, best);
                if (top == RT_NONE || i == p.top_k)
                    break;
                own = lane == i ? top : own;
                if (best == top) {
                    if (PER <= 8) {
#pragma unroll
                        for (int j = 0; j + 1 < PER; ++j)
                            u[j] = u[j + 1];
                        u[PER - 1] = RT_NONE;
                    } else {
#pragma unroll
                        for (int j = 0; j < PER; ++j)
                            u[j] = u[j] == top ? RT_NONE : u[j];
                    }
                }
            }
            int next = __shfl_down_sync(dev::FULL_MASK, own, 1);
            if (lane == p.top_k - 1)
                next = top;
            const bool pair = own != RT_NONE && next != RT_NONE;
            const bool near = ranked ? !told(float_of(own & ~LOW), float_of(next | LOW))
                                     : (own ^ next) <= LOW && (own ^ next) >= 0;
            again = __any_sync(dev::FULL_MASK, pair && near);
            least = __shfl_sync(dev::FULL_MASK, own == RT_NONE ? -INFINITY : float_of(own & ~LOW), p.top_k - 1);
            mine = own == RT_NONE ? -1 : LOW - (own & LOW);
        }
        if (again) {                                 // whole keys
            int rest[PER], before = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                rest[j] = key[j];
            mine = -1;
            for (int i = 0; i < p.top_k + (ranked ? 1 : 0); ++i) {
                int best = rest[0];
#pragma unroll
                for (int j = 1; j < PER; ++j)
                    best = max(best, rest[j]);
                const int top = __reduce_max_sync(dev::FULL_MASK, best);
                if (top == RT_NONE)
                    break;
                if (ranked && i > 0 && !told(float_of(before), float_of(top))) {
                    open = true;
                    break;
                }
                before = top;
                const int from = __ffs(__ballot_sync(dev::FULL_MASK, best == top)) - 1;
                int at = 0;
#pragma unroll
                for (int j = PER - 1; j >= 0; --j)
                    at = rest[j] == top ? j : at;
                if (lane == from)
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        rest[j] = j == at ? RT_NONE : rest[j];
                at = __shfl_sync(dev::FULL_MASK, from * PER + at, from);
                if (lane == i && i < p.top_k)
                    mine = at;
            }
        }
        if (open) {
            // of those near enough to the least chosen one or above it, the lane's is taken in 64 bits
            int near = 0;
            if (again && least > -INFINITY) {
                unsigned wanted = 0;
                const float from = reach(least);
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    wanted |= (unsigned)(key[j] != RT_NONE && score[j] >= from) << j;
                int *list = reinterpret_cast<int *>(exact);
                near = list_of<PER>(wanted, list, lane);
                if (near <= 32) {
                    const int e = lane < near ? list[lane] : -1;
                    const double of = precise_score<E>(p, l, e, lane);
                    int above = 0;
                    for (int i = 0; i < near; ++i) {
                        const double other = __shfl_sync(dev::FULL_MASK, of, i);
                        above += other > of || (other == of && i < lane);       // (the list is in the experts' order)
                    }
                    __syncwarp();
                    if (lane < near && above < p.top_k)
                        list[above] = e;
                    __syncwarp();
                    mine = lane < p.top_k ? list[lane] : -1;
                    __syncwarp();
                }
            }
            if (near == 0 || near > 32)
                mine = route_exactly<E>(p, l, exact, lane, ranked, by_sums);
        }
        // the weights of the chosen; renormalised, softmax scores are taken relative to the largest of them, and sigmoids
        // far below zero (where they are exponentials) as well
        const float lm = mine >= 0 ? logit_of(dev::to_f32(l[mine])) : -INFINITY;
        float w = 0.0f;
        const float top = p.renormalise ? warp_max_f(lm) : m;
        if (mine >= 0)
            w = soft || (p.renormalise && top < -60.0f) ? expf(lm - top) : __frcp_rn(1.0f + expf(-lm));
        if (p.renormalise)
            w = __fdiv_rn(w, warp_sum_f(w));
        else if (soft)
            w = __fdiv_rn(w, sum);
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = mine;
            p.weights[t * p.top_k + lane] = mine >= 0 ? w * p.factor : 0.0f;
            if (p.counts && mine >= 0)
                atomicAdd(counts + mine, 1);
        }
    }
    if (p.counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.experts; e += 32 * RT_WARPS)
            if (counts[e])
                atomicAdd(p.counts + e, counts[e]);
    }
}

template <typename E, int PER> __device__ __forceinline__ void store_run(E *row, int n, bool packs, int lane, const float (&v)[PER])
{
    constexpr int C = PER < 16 / (int)sizeof(E) ? PER : 16 / (int)sizeof(E);
    struct alignas(sizeof(E) * C) Pack {
        E e[C];
    };
    if (packs) {
#pragma unroll
        for (int i = 0; i < PER / C; ++i) {
            const int at = lane * PER + i * C;
            Pack q;
#pragma unroll
            for (int j = 0; j < C; ++j)
                q.e[j] = dev::from_f32<E>(v[i * C + j]);
            if (at < n)
                *reinterpret_cast<Pack *>(row + at) = q;
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (lane * PER + j < n)
                row[lane * PER + j] = dev::from_f32<E>(v[j]);
    }
}

// A warp a token: the row without the choice (zeros, or the softmax's common part) in packs, then the chosen experts'
// gradients over it, each by its lane.  FULL: a softmax that is not renormalised, which needs all logits; the others
// read the chosen ones alone, and what bounds them is the rows written.
template <typename E, int PER, bool FULL>
__global__ void __launch_bounds__(32 * RT_WARPS, PER <= 8 ? RT_CTAS : 3) route_grad_kernel(const RouteGradParams p, int packs)
{
    dev::follow_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool soft = p.score == LOOM_SCORE_SOFTMAX;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < p.tokens; t += (int64_t)gridDim.x * RT_WARPS) {
        const E *l = static_cast<const E *>(p.logits) + t * p.stride;
        E *d = static_cast<E *>(p.dlogits) + t * p.dstride;
        int e = lane < p.top_k ? __ldg(p.ids + t * p.top_k + lane) : -1;
        float g = lane < p.top_k ? p.factor * __ldg(p.dweights + t * p.top_k + lane) : 0.0f;
        float v[PER], m = -INFINITY, sum = 0.0f;
        if (FULL) {
            load_run<E, PER>(l, p.experts, packs, lane, v);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                v[j] = logit_of(v[j]);
                m = fmaxf(m, v[j]);
            }
            m = warp_max_f(m);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                v[j] = v[j] > -INFINITY ? expf(v[j] - m) : 0.0f;
                sum += v[j];
            }
            sum = warp_sum_f(sum);
        }
        if (e >= p.experts) {
            dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
            e = -1;
        }
        const float le = e >= 0 ? logit_of(dev::to_f32(l[e])) : -INFINITY;
        if (le == -INFINITY) {
            e = -1;
            g = 0.0f;
        }
        // chosen scores; renormalised, relative to their sum, and sigmoids far below zero as the exponentials that they are
        float s = 0.0f, h = g, common = 0.0f;
        if (!FULL && p.renormalise) {
            const float top = warp_max_f(le);
            if (e >= 0)
                s = soft || top < -60.0f ? expf(le - top) : __frcp_rn(1.0f + expf(-le));
            const float all = warp_sum_f(s);
            s = e >= 0 ? __fdiv_rn(s, all) : 0.0f;
            h = g - warp_sum_f(g * s);                      // (h S of the header)
        } else if (e >= 0) {
            s = soft ? __fdiv_rn(expf(le - m), sum) : __frcp_rn(1.0f + expf(-le));
        }
        if (FULL)
            common = warp_sum_f(h * s);
        float part = e >= 0 ? s * h : 0.0f;
        if (!soft)
            part *= __frcp_rn(1.0f + expf(le));             // 1 - score
        // an expert that comes more than once: the sum, by its first lane, in the order of the lanes
        const unsigned same = __match_any_sync(dev::FULL_MASK, e);
        bool first = e >= 0 && (same & ((1u << lane) - 1u)) == 0;
        if (__any_sync(dev::FULL_MASK, e >= 0 && !first)) {
            float total = 0.0f;
            for (int i = 0; i < p.top_k; ++i) {
                const float other = __shfl_sync(dev::FULL_MASK, part, i);
                total += (same >> i) & 1u ? other : 0.0f;
            }
            part = total;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            v[j] = FULL && sum > 0.0f ? -__fdiv_rn(v[j], sum) * common : 0.0f;
        __syncwarp();                                       // (the row may be the logits': they have been read)
        store_run<E, PER>(d, p.experts, packs, lane, v);
        __syncwarp();
        if (first)
            d[e] = dev::from_f32<E>(FULL ? part - s * common : part);
    }
}

}  // namespace

bool route_geometry(int64_t tokens, int32_t experts, bool backward, int64_t sms, loom_launch *out)
{
    *out = loom_launch{};
    const int64_t ctas = (tokens + RT_WARPS - 1) / RT_WARPS, most = 16 * sms;
    out->grid[0] = (uint32_t)(ctas < most ? ctas : most);
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->block[0] = 32 * RT_WARPS;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->smem_bytes = backward ? 0 : (uint32_t)(RT_WARPS * exact_places(experts) * sizeof(double) + experts * sizeof(int));     // (with a bias and counts)
    out->units_per_cta = RT_WARPS;
    out->kernel = backward ? LOOM_KERNEL_ROUTE_BACKWARD : LOOM_KERNEL_ROUTE;
    return true;
}

namespace {

template <typename E, int PER, bool GROUPS> cudaError_t launch_one(const RouteParams &p, loom_launch L, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(route_kernel<E, PER, GROUPS>), 0, done);
    if (e != cudaSuccess)
        return e;
    const bool close = p.bias || GROUPS;            // where f32 may not tell
    L.smem_bytes = (uint32_t)((close ? RT_WARPS * exact_places(p.experts) * sizeof(double) : 0) + (p.counts ? p.experts * sizeof(int) : 0));
    return launch_prepared(route_kernel<E, PER, GROUPS>, L, stream, p, (int)close, (int)packs_of<E, PER>(p.logits, p.stride, p.experts));
}

template <typename E, int PER> cudaError_t launch_per(const RouteParams &p, const loom_launch &L, cudaStream_t stream)
{
    return p.groups > 1 ? launch_one<E, PER, true>(p, L, stream) : launch_one<E, PER, false>(p, L, stream);
}

template <typename E> cudaError_t launch_e(const RouteParams &p, const loom_launch &L, cudaStream_t stream)
{
    const int per = (p.experts + 31) / 32;
    if (per <= 1)
        return launch_per<E, 1>(p, L, stream);
    if (per <= 2)
        return launch_per<E, 2>(p, L, stream);
    if (per <= 4)
        return launch_per<E, 4>(p, L, stream);
    if (per <= 8)
        return launch_per<E, 8>(p, L, stream);
    return per <= 16 ? launch_per<E, 16>(p, L, stream) : launch_per<E, 32>(p, L, stream);
}

template <typename E, int PER> cudaError_t launch_grad(const RouteGradParams &p, const loom_launch &L, cudaStream_t stream)
{
    const int packs = packs_of<E, PER>(p.logits, p.stride, p.experts) && packs_of<E, PER>(p.dlogits, p.dstride, p.experts);
    return p.score == LOOM_SCORE_SOFTMAX && !p.renormalise ? launch_with(route_grad_kernel<E, PER, true>, L, stream, p, packs)
                                                           : launch_with(route_grad_kernel<E, PER, false>, L, stream, p, packs);
}

template <typename E> cudaError_t launch_grad_e(const RouteGradParams &p, const loom_launch &L, cudaStream_t stream)
{
    const int per = (p.experts + 31) / 32;
    if (per <= 1)
        return launch_grad<E, 1>(p, L, stream);
    if (per <= 2)
        return launch_grad<E, 2>(p, L, stream);
    if (per <= 4)
        return launch_grad<E, 4>(p, L, stream);
    if (per <= 8)
        return launch_grad<E, 8>(p, L, stream);
    return per <= 16 ? launch_grad<E, 16>(p, L, stream) : launch_grad<E, 32>(p, L, stream);
}

}  // namespace

cudaError_t launch_route(const RouteParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_e<float>(p, L, stream);
    return dtype == LOOM_F16 ? launch_e<__half>(p, L, stream) : launch_e<__nv_bfloat16>(p, L, stream);
}

cudaError_t launch_route_grad(const RouteGradParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_grad_e<float>(p, L, stream);
    return dtype == LOOM_F16 ? launch_grad_e<__half>(p, L, stream) : launch_grad_e<__nv_bfloat16>(p, L, stream);
}

}  // namespace loom
