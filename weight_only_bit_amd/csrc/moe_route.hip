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
#include "moe_choice.hpp"
#include "weight_only_bit.h"

namespace wob {

namespace {

constexpr int RT = 256;         // threads
constexpr int RT_TOKENS = RT / 64;

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// A wave per token, V scores a lane: expert v 64 + lane.  Keys of 0 stand for experts that
// cannot be chosen.
template <int V>
__global__ __launch_bounds__(RT) void moe_route_kernel(RouteArgs a)
{
    extern __shared__ uint32_t shared_keys[]; // [RT_TOKENS][E], for the groups
    auto umax = [](uint32_t p, uint32_t q) { return max(p, q); };
    auto umin = [](uint32_t p, uint32_t q) { return min(p, q); };
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * RT_TOKENS + wave;
    const bool here = t < a.T;
    const int E = a.E;
    float l[V], p[V];
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 64 * v + lane;
        l[v] = here && e < E ? logit_value(a.logits, a.dt, (int64_t)t * E + e) : -__builtin_inff();
        l[v] = l[v] == l[v] ? l[v] : -__builtin_inff();
    }
    if (a.score == WOB_SCORE_SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = (float)(1.0 / (1.0 + exp(-(double)l[v])));
    } else {
        float top = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            top = fmaxf(top, l[v]);
        top = order_value(group_reduce<64>(order_key(top), umax));
        double q[V], sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            q[v] = l[v] == -__builtin_inff() ? 0.0 : l[v] == top ? 1.0 : exp((double)l[v] - (double)top);
            sum += q[v];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = sum > 0.0 ? (float)(q[v] / sum) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 64 * v + lane;
        const float c = p[v] + (a.bias && e < E ? a.bias[e] : 0.f) + 0.f;
        key[v] = l[v] > -__builtin_inff() && c > -__builtin_inff() ? order_key(c) : 0u;
    }
    if (a.groups > 1) {
        uint32_t *const mine = shared_keys + wave * E;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (64 * v + lane < E)
                mine[64 * v + lane] = key[v];
        __syncthreads();
        const int size = E / a.groups;
        uint32_t first = 0u, second = 0u;
        if (lane < a.groups)
            for (int i = 0; i < size; ++i) {
                const uint32_t k = mine[lane * size + i];
                second = max(second, min(first, k));
                first = max(first, k);
            }
        uint32_t value = first;
        if (a.group_top == 2 && first != 0u && second != 0u)
            value = order_key(order_value(first) + order_value(second) + 0.f);
        uint64_t kept = 0;
        for (int i = 0; i < a.topk_groups; ++i) {
            const uint32_t best = group_reduce<64>(value, umax);
            if (best == 0u)
                break;
            const int g = __ffsll((unsigned long long)__ballot(value == best)) - 1;
            kept |= (uint64_t)1 << g;
            value = lane == g ? 0u : value;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = kept >> (min(64 * v + lane, E - 1) / size) & 1 ? key[v] : 0u;
    }
    int id = -1; // of place `lane`
    float s = 0.f;
    for (int i = 0; i < a.topk; ++i) {
        uint32_t best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            best = max(best, key[v]);
        best = group_reduce<64>(best, umax);
        if (best == 0u)
            break;
        uint32_t e = ~0u;
        float own = 0.f;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] == best) {
                e = (uint32_t)(64 * v + lane);
                own = p[v];
            }
        const uint32_t at = group_reduce<64>(e, umin);
        own = __shfl(own, (int)(at & 63u));
        if (lane == i) {
            id = (int)at;
            s = own;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = at == (uint32_t)(64 * v + lane) ? 0u : key[v];
    }
    if (a.renormalize) {
        const float total = bitcast<float>(group_reduce<64>(bitcast<uint32_t>(s), [](uint32_t x, uint32_t y) {
            return bitcast<uint32_t>(bitcast<float>(x) + bitcast<float>(y));
        }));
        s = total > 0.f ? s / total : 0.f;
    }
    if (here && lane < a.topk) {
        a.ids[(int64_t)t * a.topk + lane] = id;
        a.weights[(int64_t)t * a.topk + lane] = s * a.scale;
    }
}

template <int V>
hipError_t launch(const RouteArgs &a, hipStream_t stream)
{
    if constexpr (V < 16)
        if (a.E > 64 * V)
            return launch<2 * V>(a, stream);
    const size_t lds = a.groups > 1 ? (size_t)RT_TOKENS * a.E * 4 : 0;
    hipLaunchKernelGGL(moe_route_kernel<V>, dim3((unsigned)((a.T + RT_TOKENS - 1) / RT_TOKENS)), dim3(RT),
                       lds, stream, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_moe_route(const RouteArgs &a, hipStream_t stream) { return launch<1>(a, stream); }

} // namespace wob
