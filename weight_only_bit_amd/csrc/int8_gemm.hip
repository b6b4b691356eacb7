// 8-bit product on gfx950:
//     y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k]  (+ bias[n])
//
// The sums are exact in 32 bits (K 2^14 < 2^31); they are converted to binary32, scaled
// twice, added to the bias and rounded once to y's type.  A holds weight rows and B
// activation rows, so a lane ends with runs of four consecutive n of one output row.
#include "wob_rows.hpp"

namespace wob {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// Four consecutive outputs of a row.
__device__ __forceinline__ void store4(void *y, int ydt, size_t at, const float4_t &v)
{
    if (ydt == DT_F32)
        *reinterpret_cast<float4_t *>(static_cast<float *>(y) + at) = v;
    else if (ydt == DT_F16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            uint2{f32x2_to_act2<DT_F16>(v[0], v[1]), f32x2_to_act2<DT_F16>(v[2], v[3])};
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            uint2{f32x2_to_act2<DT_BF16>(v[0], v[1]), f32x2_to_act2<DT_BF16>(v[2], v[3])};
}

// Four sums of row m (scale xs), columns n .. n + 3, scaled.
__device__ __forceinline__ float4_t scaled4(const i32x4 &sum, float xs, const float *ws, const float *bias, int n)
{
    const float4_t w = *reinterpret_cast<const float4_t *>(ws + n);
    float4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = (float)sum[e] * xs * w[e];
    if (bias)
        v += *reinterpret_cast<const float4_t *>(bias + n);
    return v;
}

// A workgroup of 2 x 2 waves owns 64 weight rows x 64 activation rows, a wave a block of
// 32 x 32; operands straight from memory.
__global__ __launch_bounds__(256) void int8_simple_kernel(const int8_t *__restrict__ x,
                                                          const float *__restrict__ xs,
                                                          const int8_t *__restrict__ w,
                                                          const float *__restrict__ ws,
                                                          const float *__restrict__ bias,
                                                          void *__restrict__ y, int ydt, int M, int N, int K)
{
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5, wave = threadIdx.x >> 6;
    const int tiles_n = (N + 63) / 64, n0 = blockIdx.x % tiles_n * 64 + (wave & 1) * 32;
    const int m0 = blockIdx.x / tiles_n * 64 + (wave >> 1) * 32;
    const int8_t *wr = w + (size_t)min(n0 + r, N - 1) * K, *xr = x + (size_t)min(m0 + r, M - 1) * K;
    i32x16 acc = {};
    for (int k = 16 * h; k < K + 16 * h; k += 32) {
        i32x4 a = {}, b = {};
        if (k < K) { // the last step may be half a step
            a = *reinterpret_cast<const i32x4 *>(wr + k);
            b = *reinterpret_cast<const i32x4 *>(xr + k);
        }
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
    }
    const int m = m0 + r;
    if (m >= M)
        return;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int n = n0 + 8 * g + 4 * h;
        if (n < N)
            store4(y, ydt, (size_t)m * N + n,
                   scaled4(i32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]}, xs[m], ws, bias, n));
    }
}

} // namespace

size_t int8_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8_gemm(const Int8GemmArgs &a, int M, int N, int K, void *workspace, hipStream_t stream)
{
    hipLaunchKernelGGL(int8_simple_kernel, dim3((unsigned)((int64_t)((N + 63) / 64) * ((M + 63) / 64))), dim3(256), 0, stream, a.x,
                       a.xs, a.w, a.ws, a.bias, a.y, a.ydt, M, N, K);
    return hipGetLastError();
}

} // namespace wob
