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
#include <type_traits>

namespace wob {

namespace {

// NT threads share a row, V pieces of eight elements a thread: piece j of thread t is j NT + t.
// All loads of a row are issued before the first of them is used, as far as registers reach.
// residual_out may be residual: a thread reads its pieces before it writes them.
//
// 16384 x 5376 fp16 with a gate per element (881 MB) 138 us, 6.4 TB/s; 2048 x 5376 bf16 with a
// 32-bit residual into 8 bits 27.  With ordinary loads and stores 151 and 28; with y read, summed
// and only then the residual and the gate read, and several rows a workgroup (whose addresses took
// 40 registers), 222 and 41.  Threads x pieces for the two and one row (ordinary): 256 x 3 153, 29.2, 4.5;
// 384 x 2 151, 29.9, 3.9; 512 x 2 152, 28.2, 3.7; 1024 x 1 157, 30.4, 3.6.  Rows too short for a wave
// share one: 65536 x 64 bf16 7.3 us with 8 threads a row, 9.5 with 16, 21.5 with 64; 65536 x 128 14.5 with
// 16, 24.3 with 64.  32768 x 768 64 x 2 36.8, 256 x 1 45.9; 16384 x 2048 256 x 1 46.5, 64 x 4 48.5; one row of
// 2880 512 x 1 2.7, 256 x 2 3.05.
template <int DT, int RDT, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_kernel(NormArgs a)
{
    static_assert(NT <= 64 || NT >= 256, "rows that share a workgroup share no barrier");
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, ES = elem_size<DT>(), RES = elem_size<RDT>();
    __shared__ uint32_t part[3][NT < 64 ? 1 : NT / 64];
    const int t = threadIdx.x % NT, pieces = a.H / RV;
    const int64_t row = a.row0 + (int64_t)blockIdx.x * ROWS + row_in_block<NT>();
    if (row >= a.T) // (NT < 256: lanes or waves without a row; no barrier follows there)
        return;
    // f(j, p) for every piece p = j NT + t of this thread, or for those from j0 on before j1
    auto some = [&](int j0, int j1, auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= j0 && j < j1 && j * NT + t < pieces)
                f(j, j * NT + t);
    };
    auto each = [&](auto f) __attribute__((always_inline)) { some(0, V, f); };
    auto row_of = [&](const void *base, int64_t ld, int size) __attribute__((always_inline)) {
        return static_cast<const uint8_t *>(base) + row * ld * size;
    };
    Raw8<RDT> r[V];
    Raw8<DT> y[V], gate[V], post[V], weight[V];
    auto load_gate = [&](auto nt) __attribute__((always_inline)) {
        each([&](int j, int p) {
            load_raw8<DT, decltype(nt)::value>(row_of(a.gate, a.ldg, ES) + (uint32_t)(p * RV) * ES, gate[j]);
        });
    };
    auto load_weights = [&](const void *w, Raw8<DT> (&to)[V]) __attribute__((always_inline)) {
        each([&](int j, int p) { load_raw8<DT>(static_cast<const uint8_t *>(w) + (uint32_t)(p * RV) * ES, to[j]); });
    };
    constexpr bool EARLY = V < 4, GATE_EARLY = EARLY || DT != DT_F32; // (else they do not fit the registers)
    auto load_rows = [&](auto nt) __attribute__((always_inline)) {
        constexpr bool NONT = decltype(nt)::value;
        if (a.y)
            each([&](int j, int p) { load_raw8<DT, NONT>(row_of(a.y, a.ldy, ES) + (uint32_t)(p * RV) * ES, y[j]); });
        each([&](int j, int p) { load_raw8<RDT, NONT>(row_of(a.residual, a.H, RES) + (uint32_t)(p * RV) * RES, r[j]); });
        if (GATE_EARLY && a.gate) {
            if (NONT && a.ldg)
                load_gate(std::true_type{});
            else
                load_gate(std::false_type{});
        }
    };
    if (a.once)
        load_rows(std::true_type{});
    else
        load_rows(std::false_type{});
    if (EARLY && a.post)
        load_weights(a.post, post);
    if (EARLY && a.weight)
        load_weights(a.weight, weight);

    float h[V][RV];
    if (a.y) {
        each([&](int j, int) { unpack8<DT>(y[j], h[j]); });
        if (a.post) {
            float sum = 0.f;
            each([&](int j, int) {
#pragma unroll
                for (int i = 0; i < RV; ++i)
                    sum = __builtin_fmaf(h[j][i], h[j][i], sum);
            });
            const float rstd = 1.0f / __builtin_sqrtf(row_sum<NT>(sum, part[0]) / (float)a.H + a.eps);
            if (!EARLY)
                load_weights(a.post, post);
            each([&](int j, int) {
                float w[RV];
                unpack8<DT>(post[j], w);
#pragma unroll
                for (int i = 0; i < RV; ++i)
                    h[j][i] *= rstd * w[i];
            });
        }
        // A gate that is not here yet comes two pieces at a time: with all of them 24 registers went through
        // memory (1024 x 32768 binary32 with a gate per element and both norms 155 us, now 144, one row 13.2, 10.6).
        constexpr int STEP = GATE_EARLY ? V : 2;
#pragma unroll
        for (int j0 = 0; j0 < V; j0 += STEP) {
            if (!GATE_EARLY && a.gate)
                some(j0, j0 + STEP, [&](int j, int p) {
                    load_raw8<DT>(row_of(a.gate, a.ldg, ES) + (uint32_t)(p * RV) * ES, gate[j]);
                });
            some(j0, j0 + STEP, [&](int j, int) {
                float v[RV];
                unpack8<RDT>(r[j], v);
                if (a.gate) {
                    float g[RV];
                    unpack8<DT>(gate[j], g);
#pragma unroll
                    for (int i = 0; i < RV; ++i)
                        h[j][i] = __builtin_fmaf(a.alpha * g[i], h[j][i], v[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < RV; ++i)
                        h[j][i] = __builtin_fmaf(a.alpha, h[j][i], v[i]);
                }
            });
        }
    } else {
        each([&](int j, int) { unpack8<RDT>(r[j], h[j]); });
    }
    if (a.residual_out)
        each([&](int j, int p) {
            uint8_t *const to = static_cast<uint8_t *>(a.residual_out) + (row * a.H + (uint32_t)(p * RV)) * RES;
            store8<RDT>(to, h[j]);
        });
    if (!a.weight)
        return;
    float sum = 0.f;
    each([&](int j, int) {
#pragma unroll
        for (int i = 0; i < RV; ++i)
            sum = __builtin_fmaf(h[j][i], h[j][i], sum);
    });
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<NT>(sum, part[1]) / (float)a.H + a.eps);
    if (!EARLY)
        load_weights(a.weight, weight);
    each([&](int j, int) {
        float w[RV];
        unpack8<DT>(weight[j], w);
#pragma unroll
        for (int i = 0; i < RV; ++i)
            h[j][i] *= rstd * w[i];
    });
    if (a.quant == WOB_QUANT_NONE) {
        each([&](int j, int p) {
            uint8_t *const to = static_cast<uint8_t *>(a.n) + (row * a.H + (uint32_t)(p * RV)) * ES;
            store8<DT>(to, h[j]);
        });
    } else if (a.quant == WOB_QUANT_INT8) {
        uint32_t top = 0;
        each([&](int j, int) { top = max(top, magnitude8(h[j])); });
        const Int8Row s = int8_row(row_max<NT>(top, part[2]));
        each([&](int j, int p) { static_cast<u32x2 *>(a.n)[row * pieces + p] = int8_codes8(h[j], s); });
        if (t == 0)
            static_cast<float *>(a.n_scale)[row] = s.scale;
    } else {
        each([&](int j, int p) { // H % 32 == 0: a quad of lanes has a block or none
            uint32_t b;
            static_cast<uint32_t *>(a.n)[row * pieces + p] = mxfp4_codes8(h[j], b);
            if ((t & 3) == 0)
                static_cast<uint8_t *>(a.n_scale)[(row * pieces + p) >> 2] = (uint8_t)b;
        });
    }
}

template <int DT, int RDT, int NT, int V>
hipError_t launch_rows(NormArgs a, hipStream_t stream)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    constexpr int64_t MOST = (int64_t)1 << 21; // rows of a launch: 2^31 threads at most
    // Rows that the last-level cache (256 MB) cannot hold are read nontemporally.  us, ordinary and
    // nontemporal, operands in the caches before / not: 84 MB 28.7, 33.3 / 34.2, 33.6, 168 MB 53.7,
    // 63.2 / 63.4, 61.4, 336 MB 120.5, 118.2 / 123.0, 120.2.
    const int64_t operands = (a.y ? elem_size<DT>() : 0) + (a.gate && a.ldg ? elem_size<DT>() : 0) + elem_size<RDT>();
    a.once = a.T * a.H * operands > (int64_t)256 << 20;
    for (a.row0 = 0; a.row0 < a.T; a.row0 += MOST) {
        const int64_t rows = std::min(a.T - a.row0, MOST);
        hipLaunchKernelGGL((residual_norm_kernel<DT, RDT, NT, V>), dim3((unsigned)((rows + ROWS - 1) / ROWS)),
                           dim3(NT * ROWS), 0, stream, a);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <int DT, int RDT>
hipError_t launch(const NormArgs &a, hipStream_t stream)
{
    if (a.H <= 64)
        return launch_rows<DT, RDT, 8, 1>(a, stream);
    if (a.H <= 128)
        return launch_rows<DT, RDT, 16, 1>(a, stream);
    if (a.H <= 256)
        return launch_rows<DT, RDT, 32, 1>(a, stream);
    if (a.H <= 512)
        return launch_rows<DT, RDT, 64, 1>(a, stream);
    if (a.H <= 1024)
        return launch_rows<DT, RDT, 64, 2>(a, stream);
    if (a.H <= 2048)
        return launch_rows<DT, RDT, 256, 1>(a, stream);
    if (a.H <= 4096)
        return launch_rows<DT, RDT, 512, 1>(a, stream);
    if (a.H <= 8192)
        return launch_rows<DT, RDT, 512, 2>(a, stream);
    if (a.H <= 16384)
        return launch_rows<DT, RDT, 1024, 2>(a, stream);
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
