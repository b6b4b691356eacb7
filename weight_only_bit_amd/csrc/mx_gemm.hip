// MXFP4 x MXFP4 product on gfx950:
//     y[m][n] = sum_k x[m][k] * w[n][k],   x = e2m1 * 2^(x_scale - 127), w likewise
//
// The scaled matrix instructions take E2M1 operands and their E8M0 scales as
// they are stored: a lane supplies the 16 code bytes and the one scale byte
// of one block (32 k) of one row, and every product is exact before the fp32
// sum.  A holds weight rows and B activation rows, so a lane ends with runs of
// four consecutive n of one output row.  Which blocks of a row meet in one
// instruction is free as long as both operands agree.
//
// Two kernels:
//  * few rows (M <= 16 MT): a workgroup owns 16 weight rows and its waves split
//    K; codes go from memory straight into registers
//    (v_mfma_scale_f32_16x16x128_f8f6f4); bound by the weights' bytes.
//  * tiles: both operands through LDS (v_mfma_scale_f32_32x32x64_f8f6f4), K
//    optionally split over workgroups with an fp32 sum in a second kernel.
#include "wob_device.hpp"
#include "wob_internal.hpp"
#include "wob_tile.hpp"

#include <algorithm>
#include <type_traits>

namespace wob {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int FMT_FP4 = 4; // operand format E2M1 of the f8f6f4 matrix instructions
constexpr uint32_t ONE_X4 = 0x7F7F7F7Fu; // four scale bytes of 1.0

__device__ __forceinline__ i32x8 fp4_operand(const u32x4 &v)
{
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// Four consecutive outputs of a row, rounded once to y's type.
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

// ---- Few rows --------------------------------------------------------------
//
// Workgroup: 16 weight rows; wave v of W takes the K steps j = v, v + W, ...
// (128 k: lane (r, q) = (lane % 16, lane / 16) holds block 4 j + q of row r),
// so the waves of a workgroup read neighbouring 64-byte pieces of the same
// lines.  A lane's codes stream through a ring of FR_D slots.  The scale bytes
// of the 16 weight rows are one contiguous stretch of memory (as are those of
// the M activation rows): they are copied to LDS once, after the first loads
// are under way.
constexpr int FR_ROWS = 16;
constexpr int FR_D = 4;

template <int MT>
struct FewSlot {
    u32x4 w, x[MT];
};

template <int MT, int W>
__global__ __launch_bounds__(64 * W) void mxfp4_few_kernel(const uint8_t *__restrict__ x,
                                                           const uint8_t *__restrict__ xs,
                                                           const uint8_t *__restrict__ w,
                                                           const uint8_t *__restrict__ ws,
                                                           void *__restrict__ y, int ydt, int M,
                                                           int N, int K)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * FR_ROWS;
    const int KB = K >> 5, steps = (KB + 3) >> 2;
    const int rows = min(FR_ROWS, N - n0);
    const u32x4 *wr = reinterpret_cast<const u32x4 *>(w) + (size_t)(n0 + min(r, rows - 1)) * KB;
    const u32x4 *xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xr[t] = reinterpret_cast<const u32x4 *>(x) + (size_t)min(16 * t + r, M - 1) * KB;
    const int mine = (steps - wave + W - 1) / W; // steps of this wave
    auto load = [&](int i, FewSlot<MT> &s) __attribute__((always_inline)) {
        int b = min(4 * (wave + W * i) + q, KB - 1);
        asm volatile("" : "+v"(b)); // one address per slot, not one pointer kept per slot
        s.w = __builtin_nontemporal_load(wr + b);
#pragma unroll
        for (int t = 0; t < MT; ++t)
            s.x[t] = xr[t][b];
    };
    FewSlot<MT> ring[FR_D];
#pragma unroll
    for (int d = 0; d < FR_D; ++d)
        load(min(d, max(mine - 1, 0)), ring[d]);
    // scale bytes: 8-byte units (N % 8 == 0) of the weight rows, bytes of x
    {
        const uint64_t *src = reinterpret_cast<const uint64_t *>(ws + (size_t)n0 * KB);
        uint64_t *dst = reinterpret_cast<uint64_t *>(smem);
        for (int i = tid; i < rows * KB / 8; i += 64 * W)
            dst[i] = src[i];
        uint8_t *xd = smem + FR_ROWS * KB;
        const int nb = M * KB, nd = nb >> 2;
        for (int i = tid; i < nd; i += 64 * W)
            reinterpret_cast<uint32_t *>(xd)[i] = reinterpret_cast<const uint32_t *>(xs)[i];
        if (tid < (nb & 3))
            xd[4 * nd + tid] = xs[4 * nd + tid];
    }
    __syncthreads();
    const uint8_t *wsl = smem + min(r, rows - 1) * KB;
    const uint8_t *xsl[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xsl[t] = smem + FR_ROWS * KB + min(16 * t + r, M - 1) * KB;
    float4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int i, const FewSlot<MT> &s) __attribute__((always_inline)) {
        const int b = 4 * (wave + W * i) + q;
        const bool in = b < KB; // the last step may leave some lanes without a block
        const int bc = in ? b : KB - 1;
        u32x4 wv = s.w;
        uint32_t sw = wsl[bc];
        if (!in) {
            wv = u32x4{0, 0, 0, 0};
            sw = 127u;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            uint32_t sx = xsl[t][bc];
            sx = in ? sx : 127u;
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fp4_operand(wv), fp4_operand(s.x[t]), acc[t], FMT_FP4, FMT_FP4, 0, (int)sw, 0,
                (int)sx);
        }
    };
    int i = 0;
    for (; i + FR_D < mine; i += FR_D) {
#pragma unroll
        for (int d = 0; d < FR_D; ++d) {
            if (i + d < mine)
                multiply(i + d, ring[d]);
            __builtin_amdgcn_sched_barrier(0);
            load(min(i + d + FR_D, mine - 1), ring[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < FR_D; ++d)
        if (i + d < mine)
            multiply(i + d, ring[d]);
    // Sum over the waves in wave order.  Lane (r, q) holds n = 4 q + e of
    // output row 16 t + r in acc[t][e].
    __syncthreads();
    float4_t *part = reinterpret_cast<float4_t *>(smem);
#pragma unroll
    for (int t = 0; t < MT; ++t)
        part[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int o = tid; o < 64 * MT; o += 64 * W) {
        float4_t v = part[o];
#pragma unroll
        for (int k = 1; k < W; ++k)
            v += part[k * MT * 64 + o];
        const int m = 16 * (o >> 6) + (o & 15), n = 4 * ((o >> 4) & 3);
        if (m < M && n < rows)
            store4(y, ydt, (size_t)m * N + n0 + n, v);
    }
}

template <int MT, int W>
size_t few_lds(int M, int K)
{
    const size_t scales = (size_t)(FR_ROWS + M) * (K >> 5), sums = (size_t)W * MT * 1024;
    return (std::max(scales, sums) + 15) & ~(size_t)15;
}

template <int MT, int W>
hipError_t launch_few(const uint8_t *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                      void *y, int ydt, int M, int N, int K, hipStream_t stream)
{
    auto kern = mxfp4_few_kernel<MT, W>;
    static std::atomic<uint64_t> lds_set{0};
    const size_t lds = few_lds<MT, W>(M, K);
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), 160 * 1024, lds_set);
        e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kern, dim3((N + FR_ROWS - 1) / FR_ROWS), dim3(64 * W), lds, stream, x, xs, w,
                       ws, y, ydt, M, N, K);
    return hipGetLastError();
}

// ---- Tiles -----------------------------------------------------------------
//
// A workgroup of 4 waves (WN along n, 4 / WN along m) owns TN weight rows x TM
// activation rows; a wave owns NB x MB blocks of 32 x 32 outputs.  K advances
// in spans of 256 (128 code bytes and 8 scale bytes a row), double buffered in
// LDS: the codes are copied by global_load_lds_dwordx4 (8 rows of 128 bytes,
// whole cache lines, per wave instruction), the scales pass through registers.
// A span is four MFMA steps of 64 k: in step s the lane half h = lane / 32
// supplies block 4 h + s of its row, so the four scale bytes a lane needs in a
// span are one dword of its row's eight, and the instruction selects byte s.
//
// LDS row R (weight rows, then activation rows) is 128 bytes; its 16-byte
// piece p lies at position p ^ ((R >> 1) & 7), so the 16 rows that one piece
// is read from at a time cover all 64 banks.
template <int WN_, int NB_, int MB_>
struct MxTile {
    static constexpr int WN = WN_, WM = 4 / WN_, NB = NB_, MB = MB_;
    static constexpr int TN = 32 * NB * WN, TM = 32 * MB * WM, ROWS = TN + TM;
    static constexpr int BUF = ROWS * 128;          // codes of one span
    static constexpr int LDS = 2 * BUF + 2 * ROWS * 8;
    static constexpr int ND = ROWS / 32;            // copies per wave and span
    static constexpr int SR = (ROWS + 255) / 256;   // scale rows per thread
    static_assert(LDS <= 160 * 1024, "tile fits the LDS");
};

constexpr int MX_SPAN = 256;

// The eight scale bytes of blocks b .. b + 7 of a row at p (KB blocks); bytes
// past the row read as 1.0.
__device__ __forceinline__ uint2 scale8(const uint8_t *row, int b, int KB)
{
    uint2 v;
    if (b + 8 <= KB) {
        __builtin_memcpy(&v, row + b, 8); // K % 256 != 0 leaves rows unaligned
    } else {
        v = uint2{ONE_X4, ONE_X4};
        for (int i = 0; b + i < KB; ++i) {
            const uint32_t s = row[b + i];
            if (i < 4)
                v.x = (v.x & ~(0xFFu << (8 * i))) | (s << (8 * i));
            else
                v.y = (v.y & ~(0xFFu << (8 * i - 32))) | (s << (8 * i - 32));
        }
    }
    return v;
}

template <class T>
__global__ __launch_bounds__(256) void mxfp4_tile_kernel(
    const uint8_t *__restrict__ x, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ w,
    const uint8_t *__restrict__ ws, void *__restrict__ y, int ydt, float *__restrict__ part, int M,
    int N, int K, int tiles_m, int tiles, int splits, int nxcd)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int id = xcd_tile(tiles * splits, nxcd);
    if (id < 0)
        return;
    // activation tiles fastest, then weight tiles, then K parts
    const int split = id / tiles, tile = id - split * tiles;
    const int n0 = tile / tiles_m * T::TN, m0 = tile % tiles_m * T::TM;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % T::WN, wm = wave / T::WN;
    const int KB = K >> 5, S = (KB + 7) >> 3;
    const int s_begin = (int)((int64_t)S * split / splits);
    const int s_end = (int)((int64_t)S * (split + 1) / splits);
    const uint32_t rowb = (uint32_t)K >> 1;

    // Copy d of wave v fills LDS rows 8 (4 d + v) .. + 7: lane L the position
    // L % 8 of row L / 8.  Rows past the matrix repeat its last row (never
    // stored), pieces past the row its last piece (zeroed before use).
    uint32_t row_at[T::ND];
#pragma unroll
    for (int d = 0; d < T::ND; ++d) {
        const int R = 8 * (4 * d + wave) + (lane >> 3);
        row_at[d] = (uint32_t)(32 * d < T::TN ? min(n0 + R, N - 1) : min(m0 + R - T::TN, M - 1)) * rowb;
    }
    const uint32_t piece = 16u * (uint32_t)((lane & 7) ^ ((lane >> 4) | ((wave & 1) << 2)));
    const uint32_t lds0 = (uint32_t)(size_t)(lds_ptr_t *)smem;
    auto copy = [&](int d, int buf, uint32_t k) __attribute__((always_inline)) {
        lds_dma16(32 * d < T::TN ? w : x, row_at[d] + k,
                  lds0 + (uint32_t)(buf * T::BUF + (4 * d + wave) * 1024));
    };
    auto copy_at = [&](int span) { return min((uint32_t)span * 128u + piece, rowb - 16u); };

    // Scales: thread t moves the eight bytes of rows t, t + 256.
    const uint8_t *srow[T::SR];
#pragma unroll
    for (int i = 0; i < T::SR; ++i) {
        const int R = min(tid + 256 * i, T::ROWS - 1);
        srow[i] = R < T::TN ? ws + (size_t)min(n0 + R, N - 1) * KB
                            : xs + (size_t)min(m0 + R - T::TN, M - 1) * KB;
    }
    uint2 *sl = reinterpret_cast<uint2 *>(smem + 2 * T::BUF);
    auto scales_in = [&](int span, uint2 (&v)[T::SR]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::SR; ++i)
            v[i] = scale8(srow[i], 8 * span, KB);
    };
    auto scales_out = [&](int buf, const uint2 (&v)[T::SR]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::SR; ++i)
            if (T::ROWS % 256 == 0 || tid + 256 * i < T::ROWS)
                sl[buf * T::ROWS + tid + 256 * i] = v[i];
    };

    float16_t acc[T::NB][T::MB];
#pragma unroll
    for (int a = 0; a < T::NB; ++a)
#pragma unroll
        for (int b = 0; b < T::MB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[a][b][e] = 0.f;

    const int an = 32 * T::NB * wn + r, bm = T::TN + 32 * T::MB * wm + r; // this lane's first LDS rows
    uint32_t at[4]; // position of piece 4 h + s in a row of this lane
#pragma unroll
    for (int s = 0; s < 4; ++s)
        at[s] = 16u * (uint32_t)((4 * h + s) ^ ((r >> 1) & 7));

    auto operands = [&](int buf, int s, u32x4 (&a)[T::NB], u32x4 (&b)[T::MB]) __attribute__((always_inline)) {
        const uint8_t *base = smem + buf * T::BUF + at[s];
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
            a[i] = *reinterpret_cast<const u32x4 *>(base + (an + 32 * i) * 128);
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
            b[i] = *reinterpret_cast<const u32x4 *>(base + (bm + 32 * i) * 128);
    };

    if (s_begin < s_end) {
        const uint32_t k = copy_at(s_begin);
#pragma unroll
        for (int d = 0; d < T::ND; ++d)
            copy(d, 0, k);
        uint2 v[T::SR];
        scales_in(s_begin, v);
        scales_out(0, v);
        __builtin_amdgcn_s_waitcnt(0);
        barrier_only();
    }
    auto run_span = [&](int span, auto tail) __attribute__((always_inline)) {
        const int buf = (span - s_begin) & 1;
        const int next = min(span + 1, s_end - 1); // the last span copies itself again
        const uint32_t k = copy_at(next);
        const int left = KB - 8 * span; // blocks of a partial span
        uint32_t sa[T::NB], sb[T::MB];
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
            sa[i] = reinterpret_cast<const uint32_t *>(sl + buf * T::ROWS)[2 * (an + 32 * i) + h];
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
            sb[i] = reinterpret_cast<const uint32_t *>(sl + buf * T::ROWS)[2 * (bm + 32 * i) + h];
        u32x4 a[2][T::NB], b[2][T::MB];
        operands(buf, 0, a[0], b[0]);
        uint2 sv[T::SR];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = s & 1;
            if (s < 3)
                operands(buf, s + 1, a[c ^ 1], b[c ^ 1]);
#pragma unroll
            for (int d = 0; d < T::ND; ++d)
                if (d * 4 / T::ND == s)
                    copy(d, buf ^ 1, k);
            if (s == 3)
                scales_in(next, sv);
            if constexpr (decltype(tail)::value) { // blocks past the row: zero weights
                const bool in = 4 * h + s < left;
#pragma unroll
                for (int i = 0; i < T::NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a[c][i][e] = in ? a[c][i][e] : 0u;
            }
            auto mul = [&](auto sel) __attribute__((always_inline)) {
                constexpr int SEL = decltype(sel)::value;
#pragma unroll
                for (int i = 0; i < T::NB; ++i)
#pragma unroll
                    for (int j = 0; j < T::MB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            fp4_operand(a[c][i]), fp4_operand(b[c][j]), acc[i][j], FMT_FP4, FMT_FP4,
                            SEL, (int)sa[i], SEL, (int)sb[j]);
            };
            if (s == 0)
                mul(std::integral_constant<int, 0>{});
            else if (s == 1)
                mul(std::integral_constant<int, 1>{});
            else if (s == 2)
                mul(std::integral_constant<int, 2>{});
            else
                mul(std::integral_constant<int, 3>{});
        }
        scales_out(buf ^ 1, sv);
        __builtin_amdgcn_s_waitcnt(0); // the copies and the scales of the next span are in LDS
        barrier_only();
    };
    const int full = KB & 7 ? min(s_end, S - 1) : s_end; // spans before a row's partial last one
    for (int span = s_begin; span < full; ++span)
        run_span(span, std::false_type{});
    if (full < s_end)
        run_span(full, std::true_type{});

    // acc[i][j][4 g + e] is n = 32 i + 8 g + 4 h + e of the wave's rows, m = 32 j + r
#pragma unroll
    for (int j = 0; j < T::MB; ++j) {
        const int m = m0 + bm - T::TN + 32 * j;
        if (m >= M)
            continue;
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int n = n0 + 32 * (T::NB * wn + i) + 8 * g + 4 * h;
                const float4_t v{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                                 acc[i][j][4 * g + 3]};
                if (n >= N)
                    continue;
                if (splits > 1)
                    *reinterpret_cast<float4_t *>(part + ((size_t)split * M + m) * N + n) = v;
                else
                    store4(y, ydt, (size_t)m * N + n, v);
            }
    }
}

// y = the sum of the K parts, in part order.
__global__ __launch_bounds__(256) void mxfp4_sum_kernel(const float4_t *__restrict__ part,
                                                        void *__restrict__ y, int ydt, int64_t n4,
                                                        int splits)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4)
        return;
    float4_t v = part[i];
    for (int s = 1; s < splits; ++s)
        v += part[(size_t)s * n4 + i];
    store4(y, ydt, (size_t)i * 4, v);
}

template <class T>
hipError_t launch_tile(const uint8_t *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                       void *y, int ydt, int M, int N, int K, int splits, void *workspace,
                       hipStream_t stream)
{
    auto kern = mxfp4_tile_kernel<T>;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), T::LDS, lds_set);
        e != hipSuccess)
        return e;
    const int tiles_m = (M + T::TM - 1) / T::TM;
    const int64_t tiles = (int64_t)tiles_m * ((N + T::TN - 1) / T::TN);
    const int nxcd = device_topology().xcds;
    const int64_t grid = (int64_t)nxcd * ((tiles * splits + nxcd - 1) / nxcd);
    if (grid > INT32_MAX / 256)
        return hipErrorInvalidValue;
    float *part = static_cast<float *>(workspace);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), (size_t)T::LDS, stream, x, xs, w, ws, y,
                       ydt, part, M, N, K, tiles_m, (int)tiles, splits, nxcd);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1)
        return e;
    const int64_t n4 = (int64_t)M * N / 4;
    hipLaunchKernelGGL(mxfp4_sum_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream,
                       reinterpret_cast<const float4_t *>(part), y, ydt, n4, splits);
    return hipGetLastError();
}

using TileL = MxTile<2, 4, 4>; // 256 x 256
using TileS = MxTile<2, 1, 2>; // 64 weight rows x 128 activation rows

bool few_rows(int64_t M, int64_t K) { return M <= 16 && (16 + M) * (K >> 5) <= 64 * 1024; }
bool large_tile(int64_t M, int64_t N) { return ((M + 255) / 256) * ((N + 255) / 256) >= 128; }

// K parts so that about two workgroups reach each CU, at least four spans each.
int split_count(int64_t M, int64_t N, int64_t K)
{
    if (few_rows(M, K) || large_tile(M, N))
        return 1;
    const int64_t tiles = ((M + TileS::TM - 1) / TileS::TM) * ((N + TileS::TN - 1) / TileS::TN);
    const int64_t spans = (K + MX_SPAN - 1) / MX_SPAN;
    return (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, spans / 4, 16}));
}

} // namespace

size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    const int s = split_count(M, N, K);
    return s > 1 ? (size_t)s * (size_t)M * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_mxfp4_gemm(const uint8_t *x, const uint8_t *xs, const uint8_t *w,
                             const uint8_t *ws, void *y, int ydt, int M, int N, int K,
                             void *workspace, hipStream_t stream)
{
    if (few_rows(M, K)) {
        // waves per workgroup: about 16 per CU in all, at least four steps each
        const int64_t groups = (N + FR_ROWS - 1) / FR_ROWS, steps = (K + 127) / 128;
        if (groups * 8 <= 4096 && steps >= 64)
            return launch_few<1, 16>(x, xs, w, ws, y, ydt, M, N, K, stream);
        if (groups * 4 <= 4096 && steps >= 32)
            return launch_few<1, 8>(x, xs, w, ws, y, ydt, M, N, K, stream);
        return launch_few<1, 4>(x, xs, w, ws, y, ydt, M, N, K, stream);
    }
    if (large_tile(M, N))
        return launch_tile<TileL>(x, xs, w, ws, y, ydt, M, N, K, 1, workspace, stream);
    return launch_tile<TileS>(x, xs, w, ws, y, ydt, M, N, K, split_count(M, N, K), workspace, stream);
}

} // namespace wob
