// Group-limited choice of experts on gfx950.  For one token with scores l_e:
//
//     s_e = 1 / (1 + exp(-l_e)),  or  exp(l_e - max l) / sum exp(l - max l)
//     c_e = s_e + bias_e                                  (the choice; weights use s_e)
//     the kept groups: largest sum of their best one or two c
//     ids: the topk largest c of the kept groups, ties to the lowest index
//     weights = scale * s (over the sum of the chosen s)
//
// s is formed in 64 bits and rounded once to binary32, so c, and with it the order, is a
// function of the scores that does not depend on how an exponential is approximated: two
// experts whose c differ in the last place are ordered the same everywhere.
//
// L lanes share a token (16 of them: four tokens a wave).  A group has `span` of them, a
// power of two, and each holds a run of consecutive experts in V registers, so experts
// ascend with (lane, register) and a group's best two meet by cross-lane operands within
// its lanes.  c is held as an unsigned key of the same order, 0 for an expert that cannot
// be chosen.
#include "moe_choice.hpp"
#include "weight_only_bit.h"

namespace wob {

namespace {

constexpr int RT = 256; // threads

struct RouteSplit { // how a token's experts lie in its lanes
    int span, run;  // lanes of a group, experts of a lane
};

// 2^x for |x| <= 1000: n = round(x), f = x - n in [-1/2, 1/2], the series of exp(f ln 2) up to
// f^11 (the rest is below 2^-46 of it).
__device__ __forceinline__ double exp2_64(double x)
{
    // (ln 2)^k / k!
    constexpr double C[12] = {1.0,
                              0.693147180559945309417,
                              0.240226506959100712334,
                              0.0555041086648215799531,
                              0.00961812910762847716197,
                              0.00133335581464284434234,
                              0.000154035303933816099544,
                              0.0000152527338040598402800,
                              0.00000132154867901443094884,
                              0.000000101780860092396997275,
                              0.00000000705491162080112332987,
                              0.000000000444553827187081149760};
    const double n = __builtin_rint(x), f = x - n;
    double p = C[11];
#pragma unroll
    for (int i = 10; i >= 0; --i)
        p = __builtin_fma(p, f, C[i]);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / d for d in [1, 2^1000]: the instruction's estimate and two Newton steps.
__device__ __forceinline__ double recip_64(double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

constexpr double LOG2E = 1.44269504088896340736;

__device__ __forceinline__ uint32_t lane_max(uint32_t a, uint32_t b) { return max(a, b); }

// A double from lane ^ D of the group's lanes that hold equal values below D (see group_reduce).
template <int D>
__device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    if constexpr (D == 1)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
    else if constexpr (D == 2)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
    else if constexpr (D == 4)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);
    else if constexpr (D == 8)
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true);
    else
        return (uint32_t)__shfl_xor((int)v, D);
}

template <int L, int D = 1>
__device__ __forceinline__ double group_sum64(double v)
{
    if constexpr (D < L) {
        const uint64_t b = bitcast<uint64_t>(v);
        const uint64_t o = (uint64_t)from_lane<D>((uint32_t)(b >> 32)) << 32 | from_lane<D>((uint32_t)b);
        return group_sum64<L, 2 * D>(v + bitcast<double>(o));
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
            const uint32_t f = from_lane<D>(first), s = from_lane<D>(second);
            second = max(min(first, f), max(second, s));
            first = max(first, f);
            group_best2<L, 2 * D>(first, second, span);
        }
    }
}

// Eight lanes' worth of one token: the lowest lane of this lane's L for which `on` holds
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

template <int DT, int L, int V, bool QUAD>
__global__ __launch_bounds__(RT) void moe_route_kernel(RouteArgs a, RouteSplit split)
{
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
            p[v] = (float)recip_64(1.0 + exp2_64((double)fminf(fmaxf(l[v], -690.f), 690.f) * -LOG2E));
    } else {
        uint32_t k = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v)
            k = max(k, order_key(l[v]));
        const float top = order_value(group_reduce<L>(k, lane_max));
        double q[V], sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            q[v] = exp2_64(fmax(((double)l[v] - (double)top) * LOG2E, -1000.0));
            q[v] = l[v] == none ? 0.0 : l[v] == top ? 1.0 : q[v];
            sum += q[v];
        }
        const double r = recip_64(fmax(group_sum64<L>(sum), 1.0)); // a row with an expert sums to 1 or more
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
            const uint32_t best = group_reduce<L>(value, lane_max);
            const bool take = best != 0u && lowest_lane<L>(value == best) / span == group;
            kept = kept || take;
            value = take ? 0u : value;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = kept ? key[v] : 0u;
    }

    // Place after place: the largest key, the lowest expert that has it, its key cleared.
    constexpr int PL = (CHOICE_MAX + L - 1) / L; // places of a lane: i L + g
    int id[PL];
    float s[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        id[j] = -1;
        s[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        for (int i = 0; i < L && j * L + i < a.topk; ++i) {
            uint32_t best = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v)
                best = max(best, key[v]);
            const uint32_t local = best;
            best = group_reduce<L>(best, lane_max);
            if (!__any(best != 0u))
                break;
            const int owner = lowest_lane<L>(local == best);
            bool open = g == owner && best != 0u; // until the owner has found it
            int e = 0;
            float own = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool hit = open && key[v] == best;
                key[v] = hit ? 0u : key[v];
                e = hit ? v : e;
                own = hit ? p[v] : own;
                open = open && !hit;
            }
            const int at = (int)(threadIdx.x & 63 & ~(L - 1)) + owner;
            e = __shfl(e + e0, at);
            own = __shfl(own, at);
            if (g == i && best != 0u) {
                id[j] = e;
                s[j] = own;
            }
        }
    }
    float total = 1.f;
    if (a.renormalize) {
        total = 0.f;
#pragma unroll
        for (int j = 0; j < PL; ++j)
            total += s[j];
        total = bitcast<float>(group_reduce<L>(bitcast<uint32_t>(total), [](uint32_t x, uint32_t y) {
            return bitcast<uint32_t>(bitcast<float>(x) + bitcast<float>(y));
        }));
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

template <int DT>
hipError_t launch(const RouteArgs &a, hipStream_t stream)
{
    const int size = a.E / a.groups;
    if (a.groups <= 16) {
        const RouteSplit s = split_of(16, a.groups, size);
        if (s.run <= 16)
            return launch_v<DT, 16, 2>(a, s, stream);
    }
    return launch_v<DT, 64, 8>(a, split_of(64, a.groups, size), stream);
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
