// The choice of a token's experts, shared by the stand-alone kernel and the
// mixture-of-experts layer.
//
// With l_e = logit_e + bias_e in binary32 (NaN counts as -inf):
//     ids     = the topk largest l_e > -inf, largest first, ties to the lowest e
//     weights = exp(l - max l) / sum of exp(l - max l), the sum over the chosen
//               (renormalised) or over all experts
// A place for which no expert above -inf is left has id -1 and weight 0.
// Where the maximum is +inf, exp(l - max) is read as its limit: 1 for the
// experts at +inf and 0 for the others.
//
// L lanes share a token, lane g of them holding experts v L + g (QUAD: 4 (v / 4) L +
// 4 g + v % 4, loaded four at a time) in V registers as unsigned keys of the same
// order; reductions over the lanes use cross-lane
// operands of the vector ALU (no LDS round trip) for L = 16, so four tokens of a
// wave are chosen at once.  Two ways to the same result:
//  * one place after the other: the largest key, the lowest expert that has it,
//    and that expert's key cleared (5 V operations a place);
//  * for many registers: the topk largest different keys first, without clearing
//    (the next one below k is the largest key - k in wrapping arithmetic: 1.5 V
//    operations a place), then every lane finds which of its experts reach the last
//    of them and their places by counting.  Equal keys show as a count above
//    the number of places; that wave then goes the first way.
// 16384 tokens, 256 experts, top 8: 9.6 us; the first way alone 14.2, one token a
// wave with shuffles through LDS 25.
#pragma once

#include "wob_device.hpp"
#include "wob_internal.hpp"

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

__device__ __forceinline__ float4_t logit_value4(const void *p, int dt, int64_t at) // at % 4 == 0
{
    if (dt == DT_F32)
        return *reinterpret_cast<const float4_t *>(static_cast<const float *>(p) + at);
    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at);
    return float4_t{act_to_f32((uint16_t)(v.x & 0xFFFFu), dt), act_to_f32((uint16_t)(v.x >> 16), dt),
                    act_to_f32((uint16_t)(v.y & 0xFFFFu), dt), act_to_f32((uint16_t)(v.y >> 16), dt)};
}

// exp(l - top) for l <= top; 1 where both are +inf, 0 for l = -inf below any top.  The
// hardware's exponential of d log2(e): off by 2^-22 and, from the rounding of d and of
// the product, 2^-23 |d| of the value (4e-6 for a score 32 below the largest, where the
// weight itself is 1e-14).  With expf 16384 tokens of 256 experts take 10.8 us instead of
// 10.1, and 11.3 instead of 10.0 with the sum over all experts.
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
// scores begin at `row`: put(place, expert, weight) is called once for every place
// below topk, by some lane of the group.  Every lane of the wave calls with the
// same topk (a group without a token passes E = 0 and ignores what it is told).
template <int L, int V, bool QUAD, class Put>
__device__ __forceinline__ void choose(const void *logits, int dt, int64_t row, const float *bias,
                                       int E, int topk, bool renormalize, int g, Put put)
{
    auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
    auto umin = [](uint32_t a, uint32_t b) { return min(a, b); };
    auto uadd = [](uint32_t a, uint32_t b) { return a + b; };
    auto fadd = [](uint32_t a, uint32_t b) {
        return bitcast<uint32_t>(bitcast<float>(a) + bitcast<float>(b));
    };
    static_assert(!QUAD || V % 4 == 0, "whole loads");
    auto expert = [&](int v) { return QUAD ? 4 * (v / 4) * L + 4 * g + v % 4 : v * L + g; };
    float l[V];
    uint32_t key[V];
    if constexpr (QUAD) { // E % 4 == 0
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const int e = expert(v);
            float4_t f = {0.f, 0.f, 0.f, 0.f};
            if (e < E) {
                f = logit_value4(logits, dt, row + e);
                if (bias)
                    f += *reinterpret_cast<const float4_t *>(bias + e);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                l[v + i] = f[i];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert(v);
            l[v] = e < E ? logit_value(logits, dt, row + e) + (bias ? bias[e] : 0.0f) : 0.f;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool in = expert(v) < E;
        l[v] += 0.0f; // -0 becomes +0: the two are equal scores
        l[v] = in && l[v] == l[v] ? l[v] : -__builtin_inff();
        key[v] = in ? order_key(l[v]) : 0u;
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
            total += exp_below(l[v], top);
        total = bitcast<float>(group_reduce<L>(bitcast<uint32_t>(total), fadd));
    }

    constexpr int NK = 16; // places of the second way, at most
    if constexpr (V >= 8 && V <= 32) {
        if (topk <= NK) {
            uint32_t kept[NK]; // the largest different keys above -inf, zeros behind them
            uint32_t last = k;
            int n = 0;
#pragma unroll
            for (int s = 0; s < NK; ++s) {
                kept[s] = 0u;
                if (s < topk) {
                    uint32_t c = k;
                    if (s > 0) {
                        uint32_t d = key[0] - last;
#pragma unroll
                        for (int v = 1; v < V; ++v)
                            d = max(d, key[v] - last);
                        c = group_reduce<L>(d, umax) + last; // not below `last` if nothing is
                    }
                    const bool on = n == s && c > KEY_NEG_INF && (s == 0 || c < last);
                    kept[s] = on ? c : 0u;
                    last = on ? c : last;
                    n += on;
                }
            }
            uint32_t mine = 0; // bit v: the expert of register v is chosen
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                mine = mine << 1 | (uint32_t)(key[v] >= last);
            mine = n ? mine : 0u;
            const int found = (int)group_reduce<L>((uint32_t)__popc(mine), uadd);
            if (!__any(found != n)) {
                if (renormalize) {
                    total = 0.f;
#pragma unroll
                    for (int s = 0; s < NK; ++s)
                        if (s < topk)
                            total += kept[s] ? exp_below(order_value(kept[s]), top) : 0.f;
                }
                while (__any(mine != 0u)) {
                    if (mine != 0u) {
                        const int v = __ffs(mine) - 1;
                        mine &= mine - 1;
                        float f = l[0];
#pragma unroll
                        for (int i = 1; i < V; ++i)
                            f = v == i ? l[i] : f;
                        const uint32_t own = order_key(f);
                        int place = 0;
#pragma unroll
                        for (int s = 0; s < NK; ++s)
                            place += kept[s] > own;
                        put(place, expert(v), exp_below(f, top) / total);
                    }
                }
                for (int s = n + g; s < topk; s += L)
                    put(s, -1, 0.f);
                return;
            }
        }
    }

    int id[CHOICE_MAX / L];
    float weight[CHOICE_MAX / L];
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j) {
        id[j] = -1;
        weight[j] = 0.f;
    }
    if (renormalize)
        total = 0.f;
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j) {
        for (int s = 0; s < L; ++s) {
            if (j * L + s >= topk)
                break;
            if (j + s > 0)
                k = best_key();
            // the lowest expert with that key (the registers hold ascending experts)
            uint32_t e = ~0u;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                e = key[v] == k ? (uint32_t)expert(v) : e;
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
                key[v] = some && e == (uint32_t)expert(v) ? 0u : key[v];
        }
    }
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j)
        if (j * L + g < topk)
            put(j * L + g, id[j], id[j] < 0 ? 0.f : weight[j] / total);
}

} // namespace wob
