// The choice of experts (moe_topk) and the whole mixture-of-experts layer.
#include "moe_choice.hpp"
#include "weight_only_bit.h"
#include "wob_internal.hpp"

namespace wob {

namespace {

constexpr int CH_THREADS = 256;

template <int DT, int L, int V>
__global__ __launch_bounds__(CH_THREADS) void moe_topk_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ ids,
    float *__restrict__ weights, int T, int E, int topk, bool renormalize)
{
    const int t = blockIdx.x * (CH_THREADS / L) + threadIdx.x / L, g = threadIdx.x % L;
    int id[CHOICE_MAX / L];
    float w[CHOICE_MAX / L];
    choose<DT, L, V>(logits, (int64_t)t * E, bias, t < T ? E : 0, topk, renormalize, g, id, w);
    if (t >= T)
        return;
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j)
        if (j * L + g < topk) {
            ids[(int64_t)t * topk + j * L + g] = id[j];
            weights[(int64_t)t * topk + j * L + g] = w[j];
        }
}

template <int DT, int L, int V>
hipError_t launch_topk_v(const void *logits, const float *bias, int32_t *ids, float *weights, int T,
                         int E, int topk, bool renormalize, hipStream_t stream)
{
    // 16 lanes a token up to 256 experts, a whole wave beyond
    if (E > L * V) {
        if constexpr (L == 16 && V < 16)
            return launch_topk_v<DT, 16, 2 * V>(logits, bias, ids, weights, T, E, topk, renormalize,
                                                stream);
        else if constexpr (L == 16)
            return launch_topk_v<DT, 64, 8>(logits, bias, ids, weights, T, E, topk, renormalize,
                                            stream);
        else if constexpr (V < 64)
            return launch_topk_v<DT, 64, 2 * V>(logits, bias, ids, weights, T, E, topk, renormalize,
                                                stream);
    }
    constexpr int PER = CH_THREADS / L; // tokens per workgroup
    hipLaunchKernelGGL((moe_topk_kernel<DT, L, V>), dim3((T + PER - 1) / PER), dim3(CH_THREADS), 0,
                       stream, logits, bias, ids, weights, T, E, topk, renormalize);
    return hipGetLastError();
}

// Workspace of the layer: the choice, the activated rows of stage 1, then the
// stages' own scratch.
struct LayerWs {
    int32_t *ids;
    float *weights;
    uint16_t *a;
    uint8_t *stage;
};

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t layer_rows_at(int64_t P) { return 2 * round256(4 * (size_t)P); }
size_t layer_stage_at(int64_t P, int64_t I)
{
    return layer_rows_at(P) + round256(2 * (size_t)P * (size_t)I);
}

LayerWs carve_layer(void *ws, int64_t P, int64_t I)
{
    uint8_t *b = static_cast<uint8_t *>(ws);
    LayerWs w;
    w.ids = reinterpret_cast<int32_t *>(b);
    w.weights = reinterpret_cast<float *>(b + round256(4 * (size_t)P));
    w.a = reinterpret_cast<uint16_t *>(b + layer_rows_at(P));
    w.stage = b + layer_stage_at(P, I);
    return w;
}

} // namespace

hipError_t launch_moe_topk(const void *logits, int dt, const float *bias, int32_t *ids,
                           float *weights, int T, int E, int topk, bool renormalize,
                           hipStream_t stream)
{
    if (dt == DT_F16)
        return launch_topk_v<DT_F16, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize, stream);
    if (dt == DT_BF16)
        return launch_topk_v<DT_BF16, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize,
                                         stream);
    return launch_topk_v<DT_F32, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize, stream);
}

size_t moe_layer_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    return layer_stage_at(T * topk, I) + moe_stage2_workspace_bytes(T, topk, E, H);
}

hipError_t launch_mxfp4_moe_layer(const MoeLayerArgs &a, void *workspace, hipStream_t stream)
{
    const LayerWs w = carve_layer(workspace, (int64_t)a.T * a.topk, a.I);
    hipError_t e = launch_moe_topk(a.logits, a.logits_dt, a.bias, w.ids, w.weights, a.T, a.E, a.topk,
                                   a.renormalize, stream);
    if (e != hipSuccess)
        return e;
    e = launch_mxfp4_moe(a.x, w.ids, a.w1, a.w1s, w.a, a.T, a.topk, a.E, 2 * a.I, a.H,
                         WOB_ACT_SILU_MUL, 32, w.stage, stream);
    if (e != hipSuccess)
        return e;
    return launch_mxfp4_moe_stage2(w.a, w.ids, w.weights, a.w2, a.w2s, a.y, a.T, a.topk, a.E, a.H,
                                   a.I, w.stage, stream);
}

} // namespace wob
