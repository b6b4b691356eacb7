// Rows shared by the threads of a workgroup: loads, reductions and the 8- and 4-bit
// forms that the quantising kernels write.
#pragma once

#include "wob_device.hpp"
#include "wob_internal.hpp"

namespace wob {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int RV = 8; // consecutive elements of a thread: 16 bytes of 16-bit values

// Eight consecutive elements as they are stored, and in binary32 (exact for every input type).
template <int DT>
struct Raw8 {
    u32x4 v[DT == DT_F32 ? 2 : 1];
};

// NT: nontemporal, for rows that no cache holds.
template <int DT, bool NT = false>
__device__ __forceinline__ void load_raw8(const void *p, Raw8<DT> &r)
{
    const u32x4 *s = static_cast<const u32x4 *>(p);
#pragma unroll
    for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) {
        if constexpr (NT)
            r.v[i] = __builtin_nontemporal_load(s + i);
        else
            r.v[i] = s[i];
    }
}

template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT> &r, float (&v)[RV])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_F32) {
            v[i] = bitcast<float>(r.v[0][i]);
            v[4 + i] = bitcast<float>(r.v[1][i]);
        } else {
            v[2 * i] = act_to_f32<DT>((uint16_t)(r.v[0][i] & 0xFFFFu));
            v[2 * i + 1] = act_to_f32<DT>((uint16_t)(r.v[0][i] >> 16));
        }
    }
}

template <int DT>
__device__ __forceinline__ void load8(const void *p, float (&v)[RV])
{
    Raw8<DT> r;
    load_raw8<DT>(p, r);
    unpack8<DT>(r, v);
}

// Eight consecutive elements, each rounded once to the type.  Nontemporal: rows that are read, changed
// and written are faster so at every size, in the caches or not (norms of 2048 x 5376 bf16 16.9 us
// to 15.9 and 21.5 to 20.2, 8-bit rows of that size into bf16 6.1 to 5.0 and 9.1 to 6.3).
template <int DT>
__device__ __forceinline__ void store8(void *p, const float (&v)[RV])
{
    if constexpr (DT == DT_F32) {
        float4_t *d = static_cast<float4_t *>(p);
        const float4_t lo{v[0], v[1], v[2], v[3]}, hi{v[4], v[5], v[6], v[7]};
        __builtin_nontemporal_store(lo, d);
        __builtin_nontemporal_store(hi, d + 1);
    } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = f32x2_to_act2<DT>(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(o, static_cast<u32x4 *>(p));
    }
}

template <int DT>
constexpr int elem_size() { return DT == DT_F32 ? 4 : 2; }

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true)); // 1,0,3,2
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true)); // 2,3,0,1
}

// f of v and lane ^ D's v for D = 16 and 32, where f does not mind the order of its operands: the
// swap of two copies' halves leaves both halves' values in every lane, without the way through LDS.
template <int D, class F>
__device__ __forceinline__ uint32_t join_halves(uint32_t v, F f)
{
    static_assert(D == 16 || D == 32, "rows of 16 lanes or halves of a wave");
    if constexpr (D == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return f((uint32_t)p[0], (uint32_t)p[1]);
    } else {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return f((uint32_t)p[0], (uint32_t)p[1]);
    }
}

// f over the NT threads that share a row, the result in every one of them.  NT = 8, 16, 32, 64: lanes of
// a wave; more: the waves' results meet in `part` (NT / 64 words of LDS that nothing else
// is read from until the next barrier).
template <int NT, class F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, uint32_t *part, F f)
{
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // lane ^ 1
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // lane ^ 2
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true)); // 7 - lane of 8
    if constexpr (NT > 8)
        v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true)); // 15 - lane of 16
    if constexpr (NT > 16)
        v = join_halves<16>(v, f);
    if constexpr (NT > 32)
        v = join_halves<32>(v, f);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i)
            v = f(v, part[i]);
    }
    return v;
}

template <int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *part)
{
    return row_reduce<NT>(v, part, [](uint32_t a, uint32_t b) { return max(a, b); });
}

template <int NT>
__device__ __forceinline__ float row_sum(float v, uint32_t *part)
{
    return bitcast<float>(row_reduce<NT>(bitcast<uint32_t>(v), part, [](uint32_t a, uint32_t b) {
        return bitcast<uint32_t>(bitcast<float>(a) + bitcast<float>(b));
    }));
}

// The row of this thread in its workgroup: uniform in a wave where a wave has no more than one.
template <int NT>
__device__ __forceinline__ int row_in_block()
{
    const int r = threadIdx.x / NT;
    return NT < 64 ? r : __builtin_amdgcn_readfirstlane(r);
}

// The largest magnitude as a bit pattern (magnitudes order as their patterns do, NaN
// above infinity).
__device__ __forceinline__ uint32_t magnitude8(const float (&v)[RV])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < RV; ++i)
        top = max(top, bitcast<uint32_t>(v[i]) & 0x7FFFFFFFu);
    return top;
}

// A row in 8 bits: scale = amax / 127, code = round(v * (127 / amax)), half to even.  Rows
// with a NaN or an infinity get a NaN scale and codes 0, rows of zeros scale 0 and codes 0.
// v * (127 / amax) is at most 127 (1 + 2^-23), so no code passes 127.  127 / amax would pass
// binary32's range below 2^-121: such rows are taken 2^64 times as large, which is exact.
struct Int8Row {
    float scale, lift, inv;
};

__device__ __forceinline__ Int8Row int8_row(uint32_t top)
{
    const float amax = bitcast<float>(top);
    Int8Row r;
    r.lift = amax < 0x1p-100f ? 0x1p64f : 1.0f;
    const bool finite = top < 0x7F800000u;
    r.scale = finite ? amax / 127.0f : bitcast<float>(0x7FC00000u);
    r.inv = finite && top != 0u ? 127.0f / (amax * r.lift) : 0.0f;
    return r;
}

// Eight codes; 0 for a row that is not finite.  |v inv| is below 2^22, so adding 1.5 * 2^23
// rounds it to a whole number, half to even, and leaves that number's two's complement in the
// low bits, from which permutes take the bytes: 2.75 operations a code, against 7 with a
// rounding, a conversion and shifts.  The product is rounded by itself, not fused.
__device__ __forceinline__ u32x2 int8_codes8(const float (&v)[RV], const Int8Row &r)
{
#pragma clang fp contract(off)
    if (r.inv == 0.0f)
        return u32x2{0u, 0u};
    uint32_t q[RV];
    const bool tiny = r.lift != 1.0f;
#pragma unroll
    for (int i = 0; i < RV; ++i) {
        float f = v[i];
        if (tiny)
            f *= r.lift;
        f = f * r.inv;
        q[i] = bitcast<uint32_t>(f + 12582912.0f);
    }
    auto four = [&](int i) {
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[i + 3], q[i + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(q[i + 1], q[i], 0x0C0C0400u), 0x05040100u);
    };
    return u32x2{four(0), four(4)};
}

// A quarter of an MXFP4 block: the eight codes of this lane and the block's E8M0 byte (see
// mx_quant.hip).  The four lanes of a quad hold the block and call together.
__device__ __forceinline__ uint32_t mxfp4_codes8(const float (&v)[RV], uint32_t &b)
{
    const uint32_t field = quad_max(magnitude8(v)) >> 23;
    b = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
    const float s = e8m0_to_f32(b == 255u ? 127u : b);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    return b == 255u ? 0u : c;
}

} // namespace wob
