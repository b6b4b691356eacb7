// The norms around a block with its gate and residual scale, on gfx950, in one pass:
//
//     t = y,  or  y / sqrt(mean(y^2) + eps) * post_weight      (the norm after the block)
//     h = residual + (alpha * gate) * t                        (gate absent: 1)
//     n = h / sqrt(mean(h^2) + eps) * weight                   (the norm before the next)
//
// in binary32; h is rounded once to the residual's type, n once to its own, or to 8-bit rows
// or MXFP4 blocks, the operands of the products that follow.
//
// Bound by memory: y, residual and a gate per element are read once, h and n written once;
// the row stays in registers across both sums.
#include "weight_only_bit.h"
#include "wob_rows.hpp"

#include <algorithm>

namespace wob {

namespace {

// NT threads share a row, V pieces of eight elements a thread: piece j of thread t is j NT + t.
// residual_out may be residual: a thread reads its pieces before it writes them.
template <int DT, int RDT, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_kernel(NormArgs a)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, ES = elem_size<DT>(), RES = elem_size<RDT>();
    __shared__ uint32_t part[4][NT / 64];
    const int t = threadIdx.x % NT, pieces = a.H / RV;
    int turn = 0; // reductions take four slots in turn: none is written while it is read
    for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT; row < a.T;
         row += (int64_t)gridDim.x * ROWS) {
        float h[V][RV];
        const uint8_t *r = static_cast<const uint8_t *>(a.residual) + row * a.H * RES;
        if (a.y) {
            const uint8_t *y = static_cast<const uint8_t *>(a.y) + row * a.ldy * ES;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces) {
                    load8<DT>(y + (int64_t)p * RV * ES, h[j]);
#pragma unroll
                    for (int i = 0; i < RV; ++i)
                        sum = __builtin_fmaf(h[j][i], h[j][i], sum);
                }
            }
            float rstd = 1.0f;
            if (a.post)
                rstd = 1.0f / __builtin_sqrtf(row_sum<NT>(sum, part[turn++ & 3]) / (float)a.H + a.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces) {
                    float v[RV], g[RV];
                    if (a.post) {
                        load8<DT>(static_cast<const uint8_t *>(a.post) + (int64_t)p * RV * ES, v);
#pragma unroll
                        for (int i = 0; i < RV; ++i)
                            h[j][i] *= rstd * v[i];
                    }
                    load8<RDT>(r + (int64_t)p * RV * RES, v);
                    if (a.gate) {
                        load8<DT>(static_cast<const uint8_t *>(a.gate) + (row * a.ldg + (int64_t)p * RV) * ES, g);
#pragma unroll
                        for (int i = 0; i < RV; ++i)
                            h[j][i] = __builtin_fmaf(a.alpha * g[i], h[j][i], v[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < RV; ++i)
                            h[j][i] = __builtin_fmaf(a.alpha, h[j][i], v[i]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces)
                    load8<RDT>(r + (int64_t)p * RV * RES, h[j]);
            }
        }
        if (a.residual_out) {
            uint8_t *out = static_cast<uint8_t *>(a.residual_out) + row * a.H * RES;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces)
                    store8<RDT>(out + (int64_t)p * RV * RES, h[j]);
            }
        }
        if (!a.weight)
            continue;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j * NT + t < pieces)
#pragma unroll
                for (int i = 0; i < RV; ++i)
                    sum = __builtin_fmaf(h[j][i], h[j][i], sum);
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<NT>(sum, part[turn++ & 3]) / (float)a.H + a.eps);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = j * NT + t;
            if (p < pieces) {
                float w[RV];
                load8<DT>(static_cast<const uint8_t *>(a.weight) + (int64_t)p * RV * ES, w);
#pragma unroll
                for (int i = 0; i < RV; ++i)
                    h[j][i] *= rstd * w[i];
                top = max(top, magnitude8(h[j]));
            }
        }
        if (a.quant == WOB_QUANT_NONE) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces)
                    store8<DT>(static_cast<uint8_t *>(a.n) + (row * a.H + (int64_t)p * RV) * ES, h[j]);
            }
        } else if (a.quant == WOB_QUANT_INT8) {
            const Int8Row s = int8_row(row_max<NT>(top, part[turn++ & 3]));
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces)
                    static_cast<uint2 *>(a.n)[row * pieces + p] = int8_codes8(h[j], s);
            }
            if (t == 0)
                static_cast<float *>(a.n_scale)[row] = s.scale;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = j * NT + t;
                if (p < pieces) { // H % 32 == 0: a quad of lanes has a block or none
                    uint32_t b;
                    static_cast<uint32_t *>(a.n)[row * pieces + p] = mxfp4_codes8(h[j], b);
                    if ((t & 3) == 0)
                        static_cast<uint8_t *>(a.n_scale)[(row * pieces + p) >> 2] = (uint8_t)b;
                }
            }
        }
    }
}

template <int DT, int RDT, int NT, int V>
hipError_t launch_rows(const NormArgs &a, hipStream_t stream)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    const int64_t grid = std::min<int64_t>((a.T + ROWS - 1) / ROWS, (int64_t)1 << 20);
    hipLaunchKernelGGL((residual_norm_kernel<DT, RDT, NT, V>), dim3((unsigned)grid), dim3(NT * ROWS), 0,
                       stream, a);
    return hipGetLastError();
}

template <int DT, int RDT>
hipError_t launch(const NormArgs &a, hipStream_t stream)
{
    if (a.H <= 512)
        return launch_rows<DT, RDT, 64, 1>(a, stream);
    if (a.H <= 2048)
        return launch_rows<DT, RDT, 256, 1>(a, stream);
    if (a.H <= 8192)
        return launch_rows<DT, RDT, 256, 4>(a, stream);
    return launch_rows<DT, RDT, 1024, 4>(a, stream);
}

} // namespace

hipError_t launch_residual_norm(const NormArgs &a, int dt, int residual_dt, hipStream_t stream)
{
    if (dt == DT_F16)
        return residual_dt == DT_F16 ? launch<DT_F16, DT_F16>(a, stream) : launch<DT_F16, DT_F32>(a, stream);
    if (dt == DT_BF16)
        return residual_dt == DT_BF16 ? launch<DT_BF16, DT_BF16>(a, stream) : launch<DT_BF16, DT_F32>(a, stream);
    return launch<DT_F32, DT_F32>(a, stream);
}

} // namespace wob
