// MXFP4 x MXFP4 product on gfx950:
//     y[m][n] = sum_k x[m][k] * w[n][k],   x = e2m1 * 2^(x_scale - 127), w likewise
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes E2M1 operands and their E8M0 scales
// as they are stored: lane l = 32 h + r supplies the 16 code bytes and the one
// scale byte of block h (of the step's two blocks of 32 k) of row r, and the
// product of every pair is exact before the fp32 sum.
#include "wob_device.hpp"
#include "wob_internal.hpp"

namespace wob {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int FMT_FP4 = 4; // operand format E2M1 of the f8f6f4 matrix instructions
constexpr int E8M0_ONE = 127;

__device__ __forceinline__ i32x8 fp4_operand(const u32x4 &v)
{
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ void store4(void *y, int ydt, size_t at, float a, float b, float c,
                                       float d)
{
    if (ydt == DT_F32)
        *reinterpret_cast<float4_t *>(static_cast<float *>(y) + at) = float4_t{a, b, c, d};
    else if (ydt == DT_F16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            uint2{f32x2_to_act2<DT_F16>(a, b), f32x2_to_act2<DT_F16>(c, d)};
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            uint2{f32x2_to_act2<DT_BF16>(a, b), f32x2_to_act2<DT_BF16>(c, d)};
}

// One wave per 32 x 32 outputs, operands straight from global memory.  A
// holds weight rows and B activation rows, so a lane ends with four runs of
// four consecutive n of one output row: one vector store each (N % 8 == 0).
__global__ __launch_bounds__(64) void mxfp4_gemm_kernel(const uint8_t *__restrict__ x,
                                                        const uint8_t *__restrict__ xs,
                                                        const uint8_t *__restrict__ w,
                                                        const uint8_t *__restrict__ ws,
                                                        void *__restrict__ y, int ydt, int M, int N,
                                                        int K)
{
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 32;
    const int KB = K >> 5;
    const size_t wr = (size_t)min(n0 + r, N - 1), xr = (size_t)min(m0 + r, M - 1);
    const u32x4 *wc = reinterpret_cast<const u32x4 *>(w) + wr * KB;
    const u32x4 *xc = reinterpret_cast<const u32x4 *>(x) + xr * KB;
    const uint8_t *wsr = ws + wr * KB, *xsr = xs + xr * KB;
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = 0.f;
    for (int j = 0; j < KB; j += 2) {
        const bool in = j + h < KB; // an odd block count leaves the upper lanes without a block
        const int b = min(j + h, KB - 1);
        u32x4 wv = wc[b];
        const u32x4 xv = xc[b];
        const int sw = in ? wsr[b] : E8M0_ONE, sx = in ? xsr[b] : E8M0_ONE;
        if (!in)
            wv = u32x4{0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(wv), fp4_operand(xv), acc,
                                                             FMT_FP4, FMT_FP4, 0, sw, 0, sx);
    }
    const int m = m0 + r;
    if (m >= M)
        return;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int n = n0 + 8 * g + 4 * h;
        if (n < N)
            store4(y, ydt, (size_t)m * N + n, acc[4 * g], acc[4 * g + 1], acc[4 * g + 2],
                   acc[4 * g + 3]);
    }
}

} // namespace

size_t mxfp4_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mxfp4_gemm(const uint8_t *x, const uint8_t *xs, const uint8_t *w,
                             const uint8_t *ws, void *y, int ydt, int M, int N, int K, void *,
                             hipStream_t stream)
{
    hipLaunchKernelGGL(mxfp4_gemm_kernel, dim3((N + 31) / 32, (M + 31) / 32), dim3(64), 0, stream,
                       x, xs, w, ws, y, ydt, M, N, K);
    return hipGetLastError();
}

} // namespace wob
