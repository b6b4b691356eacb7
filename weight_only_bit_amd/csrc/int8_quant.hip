// Rows in 8 bits on gfx950: one binary32 scale a row, codes half to even.
//
//     v_k   = x_k, or silu(x_k) * x_{K + k} (the gate and up halves of a row of 2 K)
//     scale = max |v| / 127,   code_k = round(v_k * (127 / max |v|))
//
// and the codes read back as values.  Bound by memory: x is read once, the row stays in
// registers between its maximum and its codes.
#include "weight_only_bit.h"
#include "wob_rows.hpp"

#include <algorithm>
#include <type_traits>

namespace wob {

namespace {

// silu(g) * u in binary32: e^-g by the hardware's 2^t, with the rounding of t = -g log2 e made good by one
// term of the exponential (alone it costs 2^-24 |g|), and the hardware's reciprocal.  Both are off by 2^-23 at
// most, the whole by 9.5 * 2^-24.  t stays below 128, past which the added term takes e to infinity.
// 1 / (1 + e) leaves binary32's normal numbers, which the reciprocal does not, from g = -87.3 on:
// it is taken 4 times as large, and g a quarter, which is exact from 2^-124 on.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float t = __builtin_amdgcn_fmed3f(g * -1.44269504f, -200.f, 127.99999f);
    const float rest = __builtin_fmaf(t, 1.90465421e-9f, __builtin_fmaf(t, -0.693147182f, -g)); // -g - t ln 2
    float e = __builtin_amdgcn_exp2f(t);
    e = __builtin_fmaf(e, rest, e);
    return 0.25f * g * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.25f, 0.25f)) * u;
}

// NT threads share a row, V pieces of eight elements a thread: piece j of thread t is j NT + t.
// All loads of a row are issued before the first of them is used where they take fewer than 64 registers of a
// thread, else piece by piece.
//
// 2048 x 21504 bf16 gated (220 MB) 38 to 40 us, 5.6 TB/s, with 512 x 6 (36 to 38 with the bare exponential and
// reciprocal in silu_mul; then 42 when read ordinarily, 1024 x 3 and x 4 45 to 47, 768 x 4 46, 512 x 8 46).  Rows too short for a wave share one: 65536 x 16 bf16 3.5 us with
// 8 threads a row, 4.9 with 16, 12.4 with 64; 65536 x 128 7.6 with 16, 15.7 with 64.  Longer ones, us:
// 32768 x 768 64 x 2 16.0, 256 x 1 25.9; 8192 x 2208 256 x 2 13.2, 512 x 1 17.3, one row of 2880 2.3 and
// 2.2; 2048 x 5376 512 x 2 8.5, 256 x 3 8.4, one row 2.3 and 2.5.
template <int DT, bool ACT, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void int8_quantize_kernel(
    const void *__restrict__ x, int64_t ldx, u32x2 *__restrict__ codes, float *__restrict__ scale,
    int64_t R, int K, bool once)
{
    static_assert(NT <= 64 || NT >= 256, "rows that share a workgroup share no barrier");
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, ES = elem_size<DT>();
    __shared__ uint32_t part[NT < 64 ? 1 : NT / 64];
    const int t = threadIdx.x % NT, pieces = K / RV;
    const int64_t r = (int64_t)blockIdx.x * ROWS + row_in_block<NT>();
    if (r >= R) // (NT < 256: lanes or waves without a row; no barrier follows there)
        return;
    auto each = [&](auto f) __attribute__((always_inline)) { // f(j, p) for every piece p of this thread
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j * NT + t < pieces)
                f(j, j * NT + t);
    };
    const uint8_t *const row = static_cast<const uint8_t *>(x) + r * ldx * ES, *const ups = row + (int64_t)K * ES;
    Raw8<DT> raw[V], up[V];
    float v[V][RV];
    uint32_t top = 0;
    auto load = [&](int j, int p, auto nt) __attribute__((always_inline)) {
        load_raw8<DT, decltype(nt)::value>(row + (uint32_t)(p * RV) * ES, raw[j]);
        if constexpr (ACT)
            load_raw8<DT, decltype(nt)::value>(ups + (uint32_t)(p * RV) * ES, up[j]);
    };
    auto values = [&](int j, int) __attribute__((always_inline)) {
        unpack8<DT>(raw[j], v[j]);
        if constexpr (ACT) {
            float u[RV];
            unpack8<DT>(up[j], u);
#pragma unroll
            for (int i = 0; i < RV; ++i)
                v[j][i] = silu_mul(v[j][i], u[i]);
        }
        top = max(top, magnitude8(v[j]));
    };
    auto read = [&](auto nt) __attribute__((always_inline)) {
        if constexpr (V * ES * (ACT ? 2 : 1) < 32) {
            each([&](int j, int p) __attribute__((always_inline)) { load(j, p, nt); });
            each(values);
        } else {
            each([&](int j, int p) __attribute__((always_inline)) {
                load(j, p, nt);
                values(j, p);
            });
        }
    };
    if (once) // nontemporally (see launch_rows)
        read(std::true_type{});
    else
        read(std::false_type{});
    const Int8Row s = int8_row(row_max<NT>(top, part));
    each([&](int j, int p) __attribute__((always_inline)) { codes[r * pieces + p] = int8_codes8(v[j], s); });
    if (t == 0)
        scale[r] = s.scale;
}

template <int DT, bool ACT, int NT, int V>
hipError_t launch_rows(const void *x, int64_t ldx, int8_t *codes, float *scale, int64_t R, int K,
                       hipStream_t stream)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    constexpr int64_t MOST = (int64_t)1 << 21; // rows of a launch: 2^31 threads at most
    // Rows that the last-level cache (256 MB) cannot hold are read nontemporally, gated ones from half of it
    // on, where it costs 6 % if they are in the cache and gains 13 % if they are not.  us, ordinary and nontemporal, x in the caches before / not: gated 84 MB 18.5, 19.0 / 22.4, 19.8,
    // 168 MB 33.8, 36.0 / 41.6, 36.1, 336 MB 80, 70; plain 168 MB 38, 44 / 46.4, 44.0.
    const bool once = R * K * (ACT ? 2 : 1) * elem_size<DT>() > (int64_t)(ACT ? 128 : 256) << 20;
    for (int64_t r0 = 0; r0 < R; r0 += MOST) {
        const int64_t rows = std::min(R - r0, MOST);
        hipLaunchKernelGGL((int8_quantize_kernel<DT, ACT, NT, V>), dim3((unsigned)((rows + ROWS - 1) / ROWS)),
                           dim3(NT * ROWS), 0, stream,
                           static_cast<const uint8_t *>(x) + r0 * ldx * elem_size<DT>(), ldx,
                           reinterpret_cast<u32x2 *>(codes + r0 * K), scale + r0, rows, K, once);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <int DT, bool ACT>
hipError_t launch(const void *x, int64_t ldx, int8_t *codes, float *scale, int64_t R, int K,
                  hipStream_t stream)
{
    if (K <= 64)
        return launch_rows<DT, ACT, 8, 1>(x, ldx, codes, scale, R, K, stream);
    if (K <= 128)
        return launch_rows<DT, ACT, 16, 1>(x, ldx, codes, scale, R, K, stream);
    if (K <= 256)
        return launch_rows<DT, ACT, 32, 1>(x, ldx, codes, scale, R, K, stream);
    if (K <= 512)
        return launch_rows<DT, ACT, 64, 1>(x, ldx, codes, scale, R, K, stream);
    if (K <= 1024)
        return launch_rows<DT, ACT, 64, 2>(x, ldx, codes, scale, R, K, stream);
    if (K <= 2048)
        return launch_rows<DT, ACT, 256, 1>(x, ldx, codes, scale, R, K, stream);
    if (K <= 4096)
        return launch_rows<DT, ACT, 256, 2>(x, ldx, codes, scale, R, K, stream);
    if (K <= 8192)
        return launch_rows<DT, ACT, 512, 2>(x, ldx, codes, scale, R, K, stream);
    if (K <= 16384)
        return launch_rows<DT, ACT, 512, 4>(x, ldx, codes, scale, R, K, stream);
    if (K <= 24576)
        return launch_rows<DT, ACT, 512, 6>(x, ldx, codes, scale, R, K, stream);
    if (K <= 32768)
        return launch_rows<DT, ACT, 1024, 4>(x, ldx, codes, scale, R, K, stream);
    return launch_rows<DT, ACT, 1024, 8>(x, ldx, codes, scale, R, K, stream);
}

// Eight elements a thread: 2048 x 21504 into bf16 (132 MB) 20 us, 6.5 TB/s, past the caches (26 with
// ordinary stores).
template <int DT>
__global__ __launch_bounds__(256) void int8_dequant_kernel(const uint2 *__restrict__ codes,
                                                           const float *__restrict__ scale,
                                                           void *__restrict__ out, int64_t R, int pieces)
{
    const int64_t n = R * pieces;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const uint2 c = codes[i];
        const float s = scale[i / pieces];
        float v[RV];
#pragma unroll
        for (int e = 0; e < RV; ++e)
            v[e] = (float)(int8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3))) * s;
        store8<DT>(static_cast<uint8_t *>(out) + i * RV * elem_size<DT>(), v);
    }
}

template <int DT>
hipError_t launch_dequant(const int8_t *codes, const float *scale, void *out, int64_t R, int K,
                          hipStream_t stream)
{
    const int64_t blocks = (R * (K / RV) + 255) / 256;
    hipLaunchKernelGGL(int8_dequant_kernel<DT>, dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)),
                       dim3(256), 0, stream, reinterpret_cast<const uint2 *>(codes), scale, out, R, K / RV);
    return hipGetLastError();
}

} // namespace

hipError_t launch_int8_quantize(const void *x, int dt, int64_t ldx, int act, int8_t *codes,
                                float *scale, int64_t R, int K, hipStream_t stream)
{
    if (act == WOB_ACT_SILU_MUL) {
        if (dt == DT_F16)
            return launch<DT_F16, true>(x, ldx, codes, scale, R, K, stream);
        if (dt == DT_BF16)
            return launch<DT_BF16, true>(x, ldx, codes, scale, R, K, stream);
        return launch<DT_F32, true>(x, ldx, codes, scale, R, K, stream);
    }
    if (dt == DT_F16)
        return launch<DT_F16, false>(x, ldx, codes, scale, R, K, stream);
    if (dt == DT_BF16)
        return launch<DT_BF16, false>(x, ldx, codes, scale, R, K, stream);
    return launch<DT_F32, false>(x, ldx, codes, scale, R, K, stream);
}

hipError_t launch_int8_dequant(const int8_t *codes, const float *scale, void *out, int dt, int64_t R,
                               int K, hipStream_t stream)
{
    if (dt == DT_F16)
        return launch_dequant<DT_F16>(codes, scale, out, R, K, stream);
    if (dt == DT_BF16)
        return launch_dequant<DT_BF16>(codes, scale, out, R, K, stream);
    return launch_dequant<DT_F32>(codes, scale, out, R, K, stream);
}

} // namespace wob
