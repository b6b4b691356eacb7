// The choice of a token's experts, shared by the stand-alone kernel and the
// mixture-of-experts layer (both give the same bits).
//
// With l_e = logit_e + bias_e in binary32 (NaN counts as -inf):
//     ids     = the topk largest l_e > -inf, largest first, ties to the lowest e
//     weights = exp(l - max l) / sum of exp(l - max l), the sum over the chosen
//               (renormalised) or over all experts
// A place for which no expert above -inf is left has id -1 and weight 0.
// Where the maximum is +inf, exp(l - max) is read as its limit: 1 for the
// experts at +inf and 0 for the others.
//
// L lanes share a token, lane g of them holding experts v L + g in V registers
// as unsigned keys of the same order.  A place costs one maximum of the keys,
// then the lowest index that has it; both are reduced over the lanes with
// cross-lane operands of the vector ALU (no LDS round trip) for L = 16, so four
// tokens of a wave are chosen at once: E = 256, topk = 8, 16384 tokens take
// 16 us (14.4 in a kernel trace), where one token a wave with shuffles took 25.
#pragma once

#include "wob_device.hpp"

namespace wob {

// A float as an unsigned key of the same order (a < b <=> key a < key b; the
// two zeros are made one by the caller's addition of +0).
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = bitcast<uint32_t>(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k)
{
    return bitcast<float>(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu; // order_key(-inf); 0 is below every float

__device__ __forceinline__ float logit_value(const void *p, int dt, int64_t at)
{
    if (dt == DT_F32)
        return static_cast<const float *>(p)[at];
    return act_to_f32(static_cast<const uint16_t *>(p)[at], dt);
}

__device__ __forceinline__ float exp_below(float l, float top)
{
    return l == top ? 1.0f : __expf(l - top);
}

// f over all lanes of a group of L = 16 or 64, the result in every lane.
template <int L, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f)
{
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // lane ^ 1
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // lane ^ 2
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true)); // 7 - lane of 8
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true)); // 15 - lane of 16
    if constexpr (L == 64) {
        v = f(v, (uint32_t)__shfl_xor((int)v, 16));
        v = f(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}

constexpr int CHOICE_MAX = 64; // places of a token, at most

// One group of L lanes (g: the lane's place in it) chooses for one token, whose
// scores begin at `row`.  On return lane g holds places g, g + L, ... in id[] and
// weight[].  Every lane of the wave calls it with the same topk (a group without
// a token passes E = 0).
template <int L, int V>
__device__ __forceinline__ void choose(const void *logits, int dt, int64_t row, const float *bias,
                                       int E, int topk, bool renormalize, int g,
                                       int (&id)[CHOICE_MAX / L], float (&weight)[CHOICE_MAX / L])
{
    auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
    auto umin = [](uint32_t a, uint32_t b) { return min(a, b); };
    auto fadd = [](uint32_t a, uint32_t b) {
        return bitcast<uint32_t>(bitcast<float>(a) + bitcast<float>(b));
    };
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * L + g;
        float l = 0.f;
        if (e < E) {
            l = logit_value(logits, dt, row + e) + (bias ? bias[e] : 0.0f);
            l = l != l ? -__builtin_inff() : l;
        }
        key[v] = e < E ? order_key(l) : 0u;
    }
    auto best_key = [&]() {
        uint32_t k = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            k = max(k, key[v]);
        return group_reduce<L>(k, umax);
    };
    uint32_t k = best_key();
    const float top = order_value(k);
    float total = 0.f;
    if (!renormalize) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > KEY_NEG_INF)
                total += exp_below(order_value(key[v]), top);
        total = bitcast<float>(group_reduce<L>(bitcast<uint32_t>(total), fadd));
    }
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j) {
        id[j] = -1;
        weight[j] = 0.f;
        for (int s = 0; s < L; ++s) {
            if (j * L + s >= topk)
                break;
            if (j + s > 0)
                k = best_key();
            // the lowest expert with that key (the registers hold ascending experts)
            uint32_t e = ~0u;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                e = key[v] == k ? (uint32_t)(v * L + g) : e;
            e = group_reduce<L>(e, umin);
            const bool some = k > KEY_NEG_INF; // an expert above -inf is left
            const float p = some ? exp_below(order_value(k), top) : 0.f;
            if (renormalize)
                total += p;
            if (g == s && some) {
                id[j] = (int)e;
                weight[j] = p;
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                key[v] = some && e == (uint32_t)(v * L + g) ? 0u : key[v];
        }
    }
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j)
        weight[j] = id[j] < 0 ? 0.f : weight[j] / total;
}

} // namespace wob
