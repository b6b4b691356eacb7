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

template <int DT>
__device__ __forceinline__ float logit_value(const void *p, int64_t at)
{
    if constexpr (DT == DT_F32)
        return static_cast<const float *>(p)[at];
    else
        return act_to_f32<DT>(static_cast<const uint16_t *>(p)[at]);
}

__device__ __forceinline__ float exp_below(float l, float top)
{
    return l == top ? 1.0f : __expf(l - top);
}

// One wave chooses for one token: lane l holds experts l, l + 64, ... in V
// registers.  On return lane s < topk holds place s.
template <int DT, int V>
__device__ __forceinline__ void choose_wave(const void *logits, int64_t row, const float *bias,
                                            int E, int topk, bool renormalize, int &id, float &weight)
{
    const int lane = threadIdx.x & 63;
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        float l = 0.f;
        if (e < E) {
            l = logit_value<DT>(logits, row + e) + (bias ? bias[e] : 0.0f);
            l = l != l ? -__builtin_inff() : l;
        }
        key[v] = e < E ? order_key(l) : 0u;
    }
    uint32_t kmax = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v)
        kmax = max(kmax, key[v]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        kmax = max(kmax, (uint32_t)__shfl_xor((int)kmax, d));
    const float top = order_value(kmax);
    float total = 0.f;
    if (!renormalize) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > KEY_NEG_INF)
                total += exp_below(order_value(key[v]), top);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            total += __shfl_xor(total, d);
    }
    id = -1;
    weight = 0.f;
    for (int s = 0; s < topk; ++s) {
        uint32_t k = 0;
        int e = 0;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) // >= : the lowest index of equal keys stays
            if (key[v] >= k) {
                k = key[v];
                e = v * 64 + lane;
            }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t ok = (uint32_t)__shfl_xor((int)k, d);
            const int oe = __shfl_xor(e, d);
            if (ok > k || (ok == k && oe < e)) {
                k = ok;
                e = oe;
            }
        }
        if (k <= KEY_NEG_INF)
            break; // nothing left (the same in every lane)
        const float p = exp_below(order_value(k), top);
        if (renormalize)
            total += p;
        if (lane == s) {
            id = e;
            weight = p;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == v * 64 + lane)
                key[v] = 0;
    }
    weight = id < 0 ? 0.f : weight / total;
}

} // namespace wob
