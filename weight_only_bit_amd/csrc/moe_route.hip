// Group-limited choice of experts on gfx950.  For one token with scores l_e:
//
//     s_e = 1 / (1 + exp(-l_e)),  or  exp(l_e - max l) / sum exp(l - max l)
//     c_e = s_e + bias_e                                  (the choice; weights use s_e)
//     the kept groups: largest sum of their best one or two c
//     ids: the topk largest c of the kept groups, ties to the lowest index
//     weights = scale * s (over the sum of the chosen s)
//
// s is formed in 64 bits and rounded once to binary32, so c, and with it the order, hardly depends on
// how an exponential is approximated: s is off by 2^-47.9 of its value before that rounding
// (reciprocal 2^-48.6, exponential 2^-50, the rest 2^-53 each), a softmax by 2^-46.9 at worst (its sum's
// additions, 37 at most).  A rounding goes the other way only for an s that near to the middle of two
// binary32 numbers, one value in 2^23 or fewer.
//
// L lanes share a token (16 of them: four tokens a wave).  A group has `span` of them, a
// power of two, and each holds a run of consecutive experts in V registers, so experts
// ascend with (lane, register) and a group's best two meet by cross-lane operands within
// its lanes.  c is held as an unsigned key of the same order, 0 for an expert that cannot
// be chosen.
//
// 16384 tokens of 256 experts 14.7 us (17 MB, a read of which takes 3.9): half of it is the vector ALU, about 1000
// operations of four tokens, some 440 of them the 64-bit scores, and half is left when scores, groups, places and
// sort are all taken out: 1024 workgroups, the four that a CU has room for, load, go through LDS (1.6
// conflict cycles an instruction) and write at the same time, and nothing overlaps.  4096 of 160 6.5 to 6.8;
// one token 3.8, the chain of its places.  A wave a token with library exponentials and divisions,
// groups through LDS and the places searched in all registers 27 us, four tokens a wave 16.2, sorted
// lists 13.9 to 14.4 (14.7 with the exponential's argument unrounded).
#include "moe_choice.hpp"
#include "weight_only_bit.h"
#include "wob_rows.hpp"

#include <type_traits>

namespace wob {

namespace {

// Threads of a workgroup: its lanes' keys and scores fit in static LDS.
template <int V>
constexpr int route_threads() { return V > 16 ? 128 : 256; }

struct RouteSplit { // how a token's experts lie in its lanes
    int span, run;  // lanes of a group, experts of a lane
};

// e^(x + low) for |x| <= 693 and |low| <= 2^-53 |x|: n = round(x log2 e), f = (x + low) log2 e - n in [-1/2, 1/2],
// and 2^f = 1 + f q(f) with the polynomial of degree 9 that meets (2^f - 1) / f at ten Chebyshev
// nodes: off by 2^-50 of the value at most, and by nothing at f = 0.  f is formed with the low part of log2 e
// and without a rounding of the product: rounded to 64 bits first, it cost up to 2^-47 of the value
// where |x| passes 44, a rounded difference of a softmax as much again.  16384 tokens of 256 experts, binary32,
// 14.7 us (14.6 without), softmax 15.6 (14.5 without).
constexpr double LOG2E = 1.44269504088896340736, LOG2E_LOW = 2.0355273740931033e-17;

template <bool LOW = false>
__device__ __forceinline__ double exp_64(double x, double low = 0.0)
{
    constexpr double Q[10] = {0.6931471805599462,    0.24022650695910075,   0.05550410866465167,
                              0.009618129107618665,  0.0013333558200794592, 0.00015403530424776529,
                              1.5252672924850737e-05, 1.3215451633221434e-06, 1.0205905413765595e-07,
                              7.070977866508138e-09};
    const double n = __builtin_rint(x * LOG2E);
    double f = __builtin_fma(x, LOG2E_LOW, __builtin_fma(x, LOG2E, -n));
    if constexpr (LOW)
        f = __builtin_fma(low, LOG2E, f);
    double q = Q[9];
#pragma unroll
    for (int i = 8; i >= 0; --i)
        q = __builtin_fma(q, f, Q[i]);
    return __builtin_amdgcn_ldexp(__builtin_fma(q, f, 1.0), (int)n);
}

// 1 / d for d in [1, 2^1000]: the instruction's estimate (off by 2^-24.3 at most over 2^30 arguments)
// and a Newton step (2^-48.6).
__device__ __forceinline__ double recip_64(double d)
{
    const double r = __builtin_amdgcn_rcp(d);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// From lane ^ D, where lanes whose numbers differ only below D hold the same (see group_reduce).
template <int D>
__device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    static_assert(D <= 8, "within a row of 16");
    if constexpr (D == 1)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
    else if constexpr (D == 2)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
    else if constexpr (D == 4)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);
    else
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true);
}

// v of both lanes that D tells apart, in an order that is the same in both.
template <int D>
__device__ __forceinline__ uint2 both_lanes(uint32_t v)
{
    if constexpr (D == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return uint2{(uint32_t)p[0], (uint32_t)p[1]};
    } else if constexpr (D == 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return uint2{(uint32_t)p[0], (uint32_t)p[1]};
    } else {
        return uint2{v, from_lane<D>(v)}; // (the order does not matter to the sums and maxima here)
    }
}

// The largest of L lanes, in each of them.
template <int L, int D = 1>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    if constexpr (D < L) {
        const uint2 p = both_lanes<D>(v);
        return lanes_max<L, 2 * D>(max(p.x, p.y));
    } else {
        return v;
    }
}

template <int L, int D = 1>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (D < L) {
        const uint2 p = both_lanes<D>(bitcast<uint32_t>(v));
        return lanes_sum<L, 2 * D>(bitcast<float>(p.x) + bitcast<float>(p.y));
    } else {
        return v;
    }
}

template <int L, int D = 1>
__device__ __forceinline__ double lanes_sum64(double v)
{
    if constexpr (D < L) {
        const uint64_t b = bitcast<uint64_t>(v);
        const uint2 lo = both_lanes<D>((uint32_t)b), hi = both_lanes<D>((uint32_t)(b >> 32));
        return lanes_sum64<L, 2 * D>(bitcast<double>((uint64_t)hi.x << 32 | lo.x) +
                                     bitcast<double>((uint64_t)hi.y << 32 | lo.y));
    } else {
        return v;
    }
}

// The two largest keys of `span` lanes, in each of them.
template <int L, int D = 1>
__device__ __forceinline__ void group_best2(uint32_t &first, uint32_t &second, int span)
{
    if constexpr (D < L) {
        if (D < span) { // (uniform)
            const uint2 f = both_lanes<D>(first), s = both_lanes<D>(second);
            second = max(min(f.x, f.y), max(s.x, s.y));
            first = max(f.x, f.y);
            group_best2<L, 2 * D>(first, second, span);
        }
    }
}

// The lowest lane of this lane's L for which `on` holds
// (some lane does).
template <int L>
__device__ __forceinline__ int lowest_lane(bool on)
{
    const uint64_t b = __ballot(on);
    if constexpr (L == 64)
        return __ffsll((unsigned long long)b) - 1;
    const int lane = __lane_id();
    const uint32_t half = lane & 32 ? (uint32_t)(b >> 32) : (uint32_t)b;
    return __ffs(half >> (lane & 16) & 0xFFFFu) - 1;
}

// Batcher's odd-even merge sort of V values as pairs of places.
template <int V>
struct SortNet {
    int n = 0, a[V * 8] = {}, b[V * 8] = {};
    constexpr SortNet()
    {
        for (int p = 1; p < V; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < V; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < V; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[n] = i + j;
                            b[n++] = i + j + k;
                        }
    }
};

template <int DT, int L, int V, bool QUAD>
__global__ __launch_bounds__(route_threads<V>()) void moe_route_kernel(RouteArgs a, RouteSplit split)
{
    constexpr int RT = route_threads<V>(), PITCH = V + (V >= 4 ? 4 : 1); // (neighbours' rows start in other banks)
    __shared__ __align__(16) uint32_t keys[RT * PITCH];
    __shared__ __align__(16) float scores[RT * PITCH];
    const int g = threadIdx.x % L, t = blockIdx.x * (RT / L) + threadIdx.x / L;
    const int span = split.span, run = split.run, size = a.E / a.groups;
    const int group = g / span, from = (g - group * span) * run; // of this lane: the group, the first expert in it
    const int e0 = group * size + from;
    const int have = t < a.T && group < a.groups ? min(run, size - from) : 0; // experts of this lane, or below 1
    const int64_t row = (int64_t)t * a.E + e0;

    float l[V], bias[V];
    if constexpr (QUAD) { // E, size and run are multiples of 4
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            float4_t f = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
            if (v < have) {
                f = logit_value4(a.logits, DT, row + v);
                if (a.bias)
                    b = *reinterpret_cast<const float4_t *>(a.bias + e0 + v);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l[v + i] = f[i];
                bias[v + i] = b[i];
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            l[v] = v < have ? logit_value(a.logits, DT, row + v) : 0.f;
            bias[v] = v < have && a.bias ? a.bias[e0 + v] : 0.f;
        }
    }
    const float none = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < V; ++v)
        l[v] = v < have && l[v] == l[v] ? l[v] : none;

    float p[V];
    if (a.score == WOB_SCORE_SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) // beyond 690 the score is 1 or rounds to 0
            p[v] = (float)recip_64(1.0 + exp_64(-(double)fminf(fmaxf(l[v], -690.f), 690.f)));
    } else {
        uint32_t k = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v)
            k = max(k, order_key(l[v]));
        const float top = order_value(lanes_max<L>(k));
        double q[V], sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            // l - top = d + low exactly.  (No exponential under a condition: 0 gives exactly 1, -693 nothing in
            // 32 bits.)
            const double a = (double)l[v], d = a - (double)top, b = d - a;
            const double low = (a - (d - b)) + (-(double)top - b);
            const bool near = d > -693.0; // (not for infinities)
            q[v] = exp_64<true>(l[v] == top ? 0.0 : near ? d : -693.0, near ? low : 0.0);
            sum += q[v];
        }
        const double r = recip_64(lanes_sum64<L>(sum)); // (1 or more; of a row without an expert nothing is used)
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = (float)(q[v] * r);
    }
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float c = p[v] + bias[v] + 0.f; // (the two zeros are one)
        key[v] = l[v] > none && c > none ? order_key(c) : 0u;
    }

    if (a.groups > 1) {
        uint32_t first = 0u, second = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            second = max(second, min(first, key[v]));
            first = max(first, key[v]);
        }
        group_best2<L>(first, second, span);
        uint32_t value = first;
        if (a.group_top == 2 && second != 0u)
            value = order_key(order_value(first) + order_value(second) + 0.f);
        bool kept = false;
        for (int i = 0; i < a.topk_groups; ++i) {
            const uint32_t best = lanes_max<L>(value);
            const bool take = best != 0u && lowest_lane<L>(value == best) / span == group;
            kept = kept || take;
            value = take ? 0u : value;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = kept ? key[v] : 0u;
    }

    // Every lane sorts its keys; then place after place goes to the largest head, of the lowest
    // lane that has it, and that lane's list moves up.  Which of the lane's experts it was
    // is looked up afterwards, for all places at once: equal keys of a lane come
    // one after the other, the n-th of them is the n-th expert with that key.
    uint32_t *const my_keys = keys + threadIdx.x * PITCH;
    float *const my_scores = scores + threadIdx.x * PITCH;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        my_keys[v] = key[v];
        my_scores[v] = p[v];
    }
    constexpr SortNet<V> net;
#pragma unroll
    for (int i = 0; i < net.n; ++i) {
        const uint32_t x = key[net.a[i]], y = key[net.b[i]];
        key[net.a[i]] = max(x, y);
        key[net.b[i]] = min(x, y);
    }
    constexpr int PL = (CHOICE_MAX + L - 1) / L; // places of a lane: i L + g
    uint32_t chosen[PL];                         // key of the place, 0 for none
    int where[PL];                               // 256 * the lane + which of its equal keys
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        chosen[j] = 0u;
        where[j] = 0;
    }
    uint32_t last = 0u;
    int last_where = -1;
    auto places = [&](auto depth) __attribute__((always_inline)) { // lists no deeper than that are used up
        constexpr int D = decltype(depth)::value;
#pragma unroll
        for (int j = 0; j < PL; ++j)
            for (int i = 0; i < L && j * L + i < a.topk; ++i) {
                const uint32_t best = lanes_max<L>(key[0]);
                const int owner = lowest_lane<L>(key[0] == best);
                last_where = best == last && last_where >> 8 == owner ? last_where + 1 : owner << 8;
                last = best;
                if (g == i) {
                    chosen[j] = best;
                    where[j] = last_where;
                }
                const bool pop = g == owner;
#pragma unroll
                for (int v = 0; v < D - 1; ++v)
                    key[v] = pop ? key[v + 1] : key[v];
                key[D - 1] = pop ? 0u : key[D - 1];
            }
    };
    if constexpr (V > 8) {
        if (a.topk <= 8)
            places(std::integral_constant<int, 8>{});
        else
            places(std::integral_constant<int, V>{});
    } else {
        places(std::integral_constant<int, V>{});
    }
    __builtin_amdgcn_wave_barrier(); // a wave reads only what it wrote, in order
    int id[PL];
    float s[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        id[j] = -1;
        s[j] = 0.f;
        if (j * L >= a.topk)
            continue;
        const int owner = where[j] >> 8, row_at = ((int)threadIdx.x - g + owner) * PITCH;
        int v_at = 0;
        int seen = where[j] & 255;
        bool open = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool match = open && keys[row_at + v] == chosen[j];
            const bool hit = match && seen == 0;
            v_at = hit ? v : v_at;
            open = open && !hit;
            seen -= match;
        }
        if (chosen[j] != 0u) {
            id[j] = owner / span * size + owner % span * run + v_at;
            s[j] = scores[row_at + v_at];
        }
    }
    float total = 1.f;
    if (a.renormalize) {
        total = 0.f;
#pragma unroll
        for (int j = 0; j < PL; ++j)
            total += s[j];
        total = lanes_sum<L>(total);
    }
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        const int place = j * L + g;
        if (t < a.T && place < a.topk) {
            a.ids[(int64_t)t * a.topk + place] = id[j];
            a.weights[(int64_t)t * a.topk + place] = (total > 0.f ? s[j] / total : 0.f) * a.scale;
        }
    }
}

// Lanes and registers for `size` experts in each of `groups`, on L lanes; quads where they can be.
RouteSplit split_of(int L, int groups, int size)
{
    int span = 1;
    while (2 * span * groups <= L)
        span *= 2;
    int run = (size + span - 1) / span;
    if (size % 4 == 0)
        run = (run + 3) / 4 * 4;
    return {span, run};
}

template <int DT, int L, int V>
hipError_t launch_v(const RouteArgs &a, const RouteSplit &split, hipStream_t stream)
{
    if constexpr ((L == 16 && V < 16) || (L == 64 && V < 32))
        if (split.run > V)
            return launch_v<DT, L, 2 * V>(a, split, stream);
    constexpr int RT = route_threads<V>();
    const dim3 grid((unsigned)((a.T + RT / L - 1) / (RT / L)));
    if constexpr (V % 4 == 0) {
        if (a.E / a.groups % 4 == 0) {
            hipLaunchKernelGGL((moe_route_kernel<DT, L, V, true>), grid, dim3(RT), 0, stream, a, split);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((moe_route_kernel<DT, L, V, false>), grid, dim3(RT), 0, stream, a, split);
    return hipGetLastError();
}

// 16 lanes a token, or a whole wave where the tokens do not fill the CUs and a lane would have
// more than four experts.  us, 16 lanes / 64: 256 experts in 8 groups, 1 token 5.9 / 4.7, 1024 7.1 /
// 5.6, 2048 7.2 / 6.3, 4096 7.7 / 8.0, 16384 15.6 / 19.7; 160 in 8, 2048 tokens 6.3 / 5.7, 4096 6.7 / 7.2;
// 64 in one, 1 token 3.1 / 3.5, 1024 3.4 / 3.9.
template <int DT>
hipError_t launch(const RouteArgs &a, hipStream_t stream)
{
    const int size = a.E / a.groups;
    if (a.groups <= 16) {
        const RouteSplit s = split_of(16, a.groups, size);
        if (s.run <= (a.T <= 2048 ? 4 : 16))
            return launch_v<DT, 16, 2>(a, s, stream);
    }
    return launch_v<DT, 64, 2>(a, split_of(64, a.groups, size), stream);
}

} // namespace

hipError_t launch_moe_route(const RouteArgs &a, hipStream_t stream)
{
    if (a.dt == DT_F16)
        return launch<DT_F16>(a, stream);
    if (a.dt == DT_BF16)
        return launch<DT_BF16>(a, stream);
    return launch<DT_F32>(a, stream);
}

} // namespace wob
