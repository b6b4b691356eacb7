// MXFP4 quantisation on gfx950: 16- or 32-bit rows -> E2M1 codes with one
// E8M0 scale per 32 elements (OCP Microscaling Formats, MXFP4).
//
// For each block of 32 elements v_i of a row, with amax = max |v_i|:
//     X   = clamp(floor(log2 amax) - 2, -127, 127)    (2 = the exponent of E2M1's 4.0)
//     b   = X + 127                                   (E8M0 byte)
//     q_i = the E2M1 value nearest to v_i * 2^-X, ties to the even code,
//           held at +-6; the sign of v_i is kept, also that of a zero
// amax = 0 gives b = 0.  A block that holds a NaN or an infinity has no finite
// scale: it gets b = 255 (NaN) and codes 0, so it reads back as NaN.
//
// floor(log2 amax) is the exponent field of amax as binary32 (a binary32
// subnormal has field 0 and meets the clamp), so no logarithm is taken.
#include "wob_device.hpp"
#include "wob_internal.hpp"

namespace wob {

namespace {

constexpr int QT = 256; // threads per workgroup
constexpr int QE = 8;   // elements per thread: a quarter of a block

// n / d for n < 2^31: (n * m) >> (31 + l), l = ceil(log2 d), m = ceil(2^(31+l) / d) < 2^32.
struct FastDiv {
    uint32_t m, d;
    int s;
    explicit FastDiv(uint32_t div) : d(div)
    {
        int l = 0;
        while (((uint64_t)1 << l) < div)
            ++l;
        m = (uint32_t)((((uint64_t)1 << (31 + l)) + div - 1) / div);
        s = 31 + l;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const
    {
        return (uint32_t)(((uint64_t)n * m) >> s);
    }
};

// Eight consecutive elements in binary32 (exact for every input type).
template <int DT>
__device__ __forceinline__ void load8(const void *p, float (&v)[QE])
{
    if constexpr (DT == DT_F32) {
        const float4_t *s = static_cast<const float4_t *>(p);
        const float4_t a = s[0], b = s[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 a = *static_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = act_to_f32<DT>((uint16_t)(a[i] & 0xFFFFu));
            v[2 * i + 1] = act_to_f32<DT>((uint16_t)(a[i] >> 16));
        }
    }
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true)); // 1,0,3,2
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true)); // 2,3,0,1
}

// Thread u takes elements 8 u .. 8 u + 7 of the rows laid end to end; a quad
// of lanes shares a block (K % 32 == 0, so no block crosses a row, and the
// number of threads with work is a multiple of 4).
//
// Bound by memory: 16384 x 5376 fp32 70 us (399 MB, 5.7 TB/s), bf16 39 us, 2048 x 5376
// 9.9 and 7.2 (graph replays).  Two or four units a thread: 71.6 and 74.2 for the first,
// 37.8 and 38.4 for the second; four fp32 elements a thread, so that a load covers whole
// lines: 70.0.
template <int DT, bool STRIDED>
__global__ __launch_bounds__(QT) void mxfp4_quantize_kernel(const void *__restrict__ x, int64_t ldx,
                                                            uint32_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scale,
                                                            int64_t units, FastDiv row_units)
{
    const int64_t u = (int64_t)blockIdx.x * QT + threadIdx.x;
    if (u >= units)
        return;
    int64_t at = u * QE;
    if constexpr (STRIDED) {
        const uint32_t r = row_units.div((uint32_t)u);
        at = (int64_t)r * ldx + (int64_t)((uint32_t)u - r * row_units.d) * QE;
    }
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    float v[QE];
    load8<DT>(static_cast<const uint8_t *>(x) + at * ES, v);
    uint32_t top = 0; // magnitudes order as their bit patterns do, NaN above infinity
#pragma unroll
    for (int i = 0; i < QE; ++i)
        top = max(top, bitcast<uint32_t>(v[i]) & 0x7FFFFFFFu);
    top = quad_max(top);
    const uint32_t field = top >> 23;
    const uint32_t b = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
    const float s = e8m0_to_f32(b == 255u ? 127u : b);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    codes[u] = b == 255u ? 0u : c;
    if ((threadIdx.x & 3) == 0)
        scale[u >> 2] = (uint8_t)b;
}

template <int DT>
hipError_t launch(const void *x, int64_t ldx, uint8_t *codes, uint8_t *scale, int64_t R, int64_t K,
                  hipStream_t stream)
{
    const int64_t units = R * (K / QE);
    const dim3 grid((unsigned)((units + QT - 1) / QT));
    const FastDiv fd((uint32_t)(K / QE));
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
    if (ldx == K || R == 1)
        hipLaunchKernelGGL((mxfp4_quantize_kernel<DT, false>), grid, dim3(QT), 0, stream, x, ldx, c,
                           scale, units, fd);
    else
        hipLaunchKernelGGL((mxfp4_quantize_kernel<DT, true>), grid, dim3(QT), 0, stream, x, ldx, c,
                           scale, units, fd);
    return hipGetLastError();
}

} // namespace

hipError_t launch_mxfp4_quantize(const void *x, int dt, int64_t ldx, uint8_t *codes, uint8_t *scale,
                                 int64_t R, int64_t K, hipStream_t stream)
{
    if (dt == DT_F16)
        return launch<DT_F16>(x, ldx, codes, scale, R, K, stream);
    if (dt == DT_BF16)
        return launch<DT_BF16>(x, ldx, codes, scale, R, K, stream);
    return launch<DT_F32>(x, ldx, codes, scale, R, K, stream);
}

} // namespace wob
