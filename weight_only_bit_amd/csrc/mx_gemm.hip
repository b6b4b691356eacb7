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
//  * few rows (M <= 16): waves own 16 weight rows each and may split K; the
//    weights' codes go from memory straight into registers
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
// M <= 16.  A wave owns 16 weight rows; W waves share them and split K, in pairs
// of steps of 128 k (in a step lane (r, q) = (lane % 16, lane / 16) holds block
// 4 j + q of row r, so a pair is one whole cache line of each row), and their
// sums are joined in LDS.  A workgroup has G such groups of rows.  The weights'
// codes go from memory into registers, FR_D loads of a lane ahead; only the x
// operand and the scales pass through LDS: the activation rows (pitch 16 mod 128
// bytes, which makes their reads conflict-free) and the scale bytes, each of them
// one contiguous stretch of memory, copied once, with their loads ahead of the
// codes' so that they land first.
//
// Bound by the weights' bytes.  Measured (graph replay over copies larger than
// the caches, us; 1 x 16384 x 5376 / 1 x 43008 x 5376 / 1 x 5376 x 21504 / 16 x
// 16384 x 5376 / 13 x 5760 x 2880 / 4 x 2048 x 2048):
//   x straight from memory, W = 8, G = 1      14.9 / 28.2 / 21.0 / 20.6 / 6.6 / 3.5
//   W = 8, G = 2, single steps, nontemporal   13.9 / 35.4 / 19.4 / 15.7 / 7.7 / 6.2
//   W = 8, G = 2, pairs, ring of 8            11.1 / 26.3 / 16.8 / 13.2 / 4.7 / 5.7
//   W = 8, G = 2, pairs, ring of 6            10.2 / 23.4 / 17.0 / 12.0 / 4.3 / 5.1
//   W = 4, G = 1, pairs, ring of 4            10.5 / 24.1 / 20.1 / 20.8 / 5.0 / 2.9
// (a plain read of the first shape's 47 MB takes 8.4).  Nontemporal loads gave up
// the other half of a line; rings of 4 and 12 were no better than 6.
constexpr int FR_ROWS = 16;
constexpr int FR_D = 6;  // loads ahead
constexpr int FR_CH = 2; // neighbouring steps of a wave

__host__ __device__ inline int few_pitch(int K) { return (K / 2 + 127 - 16) / 128 * 128 + 16; }
__host__ __device__ inline size_t few_scales_at(int M, int K) { return (size_t)M * few_pitch(K); }
inline size_t few_lds(int M, int K, int W, int G)
{
    const size_t staged = few_scales_at(M, K) + (((size_t)M * (K >> 5) + 15) & ~(size_t)15) +
                          (size_t)G * FR_ROWS * (K >> 5);
    const size_t sums = W > 1 ? (size_t)W * G * 1024 : 0;
    return (std::max(staged, sums) + 15) & ~(size_t)15;
}

template <int W, int G>
__global__ __launch_bounds__(64 * W * G) void mxfp4_few_kernel(const uint8_t *__restrict__ x,
                                                               const uint8_t *__restrict__ xs,
                                                               const uint8_t *__restrict__ w,
                                                               const uint8_t *__restrict__ ws,
                                                               void *__restrict__ y, int ydt, int M,
                                                               int N, int K)
{
    constexpr int NT = 64 * W * G;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), k = wave % W, g = wave / W;
    const int KB = K >> 5, steps = (KB + 3) >> 2, pitch = few_pitch(K);
    const int nw = blockIdx.x * FR_ROWS * G, n0 = nw + FR_ROWS * g;
    const int rows = min(FR_ROWS * G, N - nw); // of the workgroup
    uint8_t *const xsl = smem + few_scales_at(M, K);
    uint8_t *const wsl = xsl + ((M * KB + 15) & ~15);

    // Staging, 16 bytes a thread (8 for the weights' scales: N % 8 == 0; 4 and
    // single bytes for x's), the first round's loads ahead of the codes'.
    const int nx = M * KB, nws = rows * KB >> 3, nxs = nx >> 2;
    const u32x4 *xg = reinterpret_cast<const u32x4 *>(x);
    const uint64_t *wsg = reinterpret_cast<const uint64_t *>(ws + (size_t)nw * KB);
    const uint32_t *xsg = reinterpret_cast<const uint32_t *>(xs);
    const u32x4 x_first = xg[min(tid, nx - 1)];
    const uint64_t ws_first = wsg[min(tid, nws - 1)];
    const uint32_t xs_first = nxs ? xsg[min(tid, nxs - 1)] : 0u;

    const u32x4 *wr = reinterpret_cast<const u32x4 *>(w) + (size_t)min(n0 + r, N - 1) * KB;
    const int mine = FR_CH * (((steps + FR_CH - 1) / FR_CH - k + W - 1) / W); // steps of this wave
    auto block = [&](int i) __attribute__((always_inline)) { // this lane's in step i
        return 4 * (FR_CH * (k + W * (i / FR_CH)) + i % FR_CH) + q;
    };
    u32x4 ring[FR_D];
    auto load = [&](int i, u32x4 &s) __attribute__((always_inline)) {
        int b = min(block(i), KB - 1);
        asm volatile("" : "+v"(b)); // one address per load, not one pointer kept per slot
        s = wr[b];
    };
#pragma unroll
    for (int d = 0; d < FR_D; ++d)
        load(min(d, max(mine - 1, 0)), ring[d]);
    __builtin_amdgcn_sched_barrier(0);

    auto put_x = [&](int i, const u32x4 &v) __attribute__((always_inline)) {
        const int m = M == 1 ? 0 : i / KB; // uniform
        *reinterpret_cast<u32x4 *>(smem + (size_t)m * pitch + (size_t)(i - m * KB) * 16) = v;
    };
    if (tid < nx)
        put_x(tid, x_first);
    if (tid < nws)
        reinterpret_cast<uint64_t *>(wsl)[tid] = ws_first;
    if (tid < nxs)
        reinterpret_cast<uint32_t *>(xsl)[tid] = xs_first;
    for (int i = tid + NT; i < nx; i += NT)
        put_x(i, xg[i]);
    for (int i = tid + NT; i < nws; i += NT)
        reinterpret_cast<uint64_t *>(wsl)[i] = wsg[i];
    for (int i = tid + NT; i < nxs; i += NT)
        reinterpret_cast<uint32_t *>(xsl)[i] = xsg[i];
    if (tid < (nx & 3))
        xsl[4 * nxs + tid] = xs[4 * nxs + tid];
    __syncthreads();

    const uint8_t *wrow = wsl + (min(n0 + r, N - 1) - nw) * KB;
    const uint8_t *xrow = smem + (size_t)min(r, M - 1) * pitch, *xsrow = xsl + min(r, M - 1) * KB;
    float4_t acc{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int i, u32x4 wv) __attribute__((always_inline)) {
        const int b = block(i);
        const bool in = b < KB; // the last steps may leave some lanes without a block
        const int bc = in ? b : KB - 1;
        const u32x4 xv = *reinterpret_cast<const u32x4 *>(xrow + 16 * bc);
        const int sw = wrow[bc], sx = xsrow[bc]; // (the row's own: a NaN there is the result's)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            wv[e] = in ? wv[e] : 0u;
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wv), fp4_operand(xv), acc,
                                                               FMT_FP4, FMT_FP4, 0, sw, 0, sx);
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
    // Lane (r, q) holds n = 4 q + e of output row r in acc[e]; the waves of a
    // group are summed in order.
    if constexpr (W > 1) {
        __syncthreads();
        float4_t *part = reinterpret_cast<float4_t *>(smem);
        part[wave * 64 + lane] = acc;
        __syncthreads();
        if (k != 0)
            return;
#pragma unroll
        for (int j = 1; j < W; ++j)
            acc += part[(wave + j) * 64 + lane];
    }
    const int n = n0 + 4 * q;
    if (r < M && n < N)
        store4(y, ydt, (size_t)r * N + n, acc);
}

template <int W, int G>
hipError_t launch_few(const uint8_t *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                      void *y, int ydt, int M, int N, int K, hipStream_t stream)
{
    auto kern = mxfp4_few_kernel<W, G>;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), 160 * 1024, lds_set);
        e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kern, dim3((N + FR_ROWS * G - 1) / (FR_ROWS * G)), dim3(64 * W * G),
                       few_lds(M, K, W, G), stream, x, xs, w, ws, y, ydt, M, N, K);
    return hipGetLastError();
}

// ---- Tiles -----------------------------------------------------------------
//
// A workgroup of 4 waves (WN along n, 4 / WN along m) owns TN weight rows x TM
// activation rows; a wave owns NB x MB blocks of 32 x 32 outputs.  K advances
// in stages of 128 (64 code bytes a row).  GS of them form a group, which is copied
// as one piece of 64 GS bytes a row; NG groups are in LDS at a time.  Four stages, a
// span of 512, share the 16 scale bytes a row has per 512 k.  Codes and scales
// are copied by global_load_lds (1 KB of codes, or 16 rows x 16 scale bytes, per wave
// instruction), NG - 1 groups ahead of their use.
//
// The copies' cost is one cache look-up a row and instruction, 59 B/ns a CU with 64
// bytes of a row and 113 with whole lines.  Groups of two stages (whole lines) against
// single ones: 100 x 5376 x 21504 23.4 us and 25.0, 200 x 16384 x 2880 18.2 and 21.0,
// 100 x 5760 x 2880 11.2 and 11.9.  (Of the first's times plain reads of its codes in
// that order are 13.9 and 16.2; eight waves instead of four change nothing.)  The 256 x
// 256 tile has no room for three groups of two.
//
// Copied from rows K / 32 bytes apart, the scales cost as many cache look-ups a
// row as the codes do.  Packed: a kernel before this one lays the scales out span
// by span, the 16 bytes of successive rows side by side, so that one copy takes
// 64 rows.  2048 x 16384 x 5376: scales 8 bytes a row at a time 118 us, 16 bytes
// 114, packed 110 with the packing; 100 x 5376 x 21504, where the scales are
// a larger share, 2.4 us less straight than packed.  (Whole: see tile_scales.)
//
// 2048 x 16384 x 5376, 107 us: 3.4 PFLOP/s, MFMA busy 53 % of the time.  Timing-only
// forms: the MFMAs alone, from registers, 47 us; with the reads of their operands from
// LDS 60; all but the copies and the stores 75; without the packing 101.  So the
// pipeline's waits and barriers take 15, the copies about 15, the stores of 67 MB 9 to 11
// (nothing multiplies meanwhile on the CU, and 48 of the 512 registers of the 256 x 256
// tile spill where they begin), the packing 5.6.  The clock is at 1.6 GHz meanwhile: with
// zero codes, which switch little, the same launches take 92.  x straight from memory
// into registers, which halves the traffic of LDS, brings nothing.
//
// A stage is two MFMA steps of 64 k: in step j the lane half h = lane / 32
// supplies block 2 h + j of its row, so a lane needs bytes 2 h, 2 h + 1 of each
// of the span's four scale dwords: a byte permute packs those of two stages into
// one register, and the instruction selects the byte.
//
// LDS row R (weight rows, then activation rows) holds 64 GS bytes of a group; its
// 16-byte piece p lies at position p ^ swizzle(R), so the rows that one piece
// is read from at a time cover all 64 banks.
//
// Order within a group (see run_span): its steps but the last read the next
// step's operands and multiply; then group g + 1's copies are waited for, a barrier
// makes them visible and frees group g's place (every wave has its last operands in
// registers), and the last step reads group g + 1's first operands and starts the
// copies of group g + NG while it multiplies.  No operand read and no copy is
// waited for in the step that issues it.
template <int WN_, int NB_, int MB_, int GS_, int NG_>
struct MxTile {
    static constexpr int WN = WN_, WM = 4 / WN_, NB = NB_, MB = MB_, GS = GS_, NG = NG_;
    static constexpr int TN = 32 * NB * WN, TM = 32 * MB * WM, ROWS = TN + TM;
    static constexpr int SEG = 64 * GS;                  // code bytes of a row in a group
    static constexpr int GROUP = ROWS * SEG;             // code bytes of one group
    static constexpr int ND = GROUP / 4096;              // code copies per wave and group
    static constexpr int SROWS = (ROWS + 255) & ~255;    // scale rows in LDS
    static constexpr int LDS = NG * GROUP + 2 * SROWS * 16;
    // Scales::Whole: the most spans of a part
    static constexpr int SPANS = (160 * 1024 - NG * GROUP) / (ROWS * 16);
    static constexpr int WSTAGE = LDS / 4 & ~15;         // LDS of one wave in the epilogue
    static_assert(ROWS % 64 == 0 && (GS == 1 ? NG == 4 : GS == 2 && NG == 3) && LDS <= 160 * 1024, "tile geometry");
};

constexpr int MX_SPAN = 512;

// As lds_dma16 with 4 bytes per lane (lane L's bytes land at `lds_addr` + 4 L).
__device__ __forceinline__ void lds_dma4(const void *sbase_any, uint32_t voff, uint32_t lds_addr)
{
    const uint64_t b = reinterpret_cast<uint64_t>(sbase_any);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const void *sbase = reinterpret_cast<const void *>(((uint64_t)hi << 32) | (uint64_t)lo);
    uint32_t saved;
    asm volatile("s_mov_b32 %0, m0\n\t"
                 "s_mov_b32 m0, %1\n\t"
                 "global_load_lds_dword %2, %3\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(saved)
                 : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(sbase)
                 : "memory");
}

// Scale bytes b .. b + 15 of a row of KB, zeros past its end (a finite scale, met by
// zero codes).
__device__ __forceinline__ u32x4 span_scales(const uint8_t *row, int b, int KB)
{
    u32x4 v = {0, 0, 0, 0};
    if (KB >= 16) {
        // unaligned, which global loads allow; at the end the row's last 16, shifted
        const int past = max(b + 16 - KB, 0);
        unsigned __int128 t;
        __builtin_memcpy(&t, row + b - past, 16);
        t >>= 8 * past;
        __builtin_memcpy(&v, &t, 16);
    } else {
        for (int i = b; i < KB; ++i) {
            const uint32_t s = (uint32_t)row[i] << (8 * (i & 3));
#pragma unroll
            for (int e = 0; e < 4; ++e) // no indexing by a variable: v stays in registers
                v[e] |= (i - b) >> 2 == e ? s : 0u;
        }
    }
    return v;
}

// Packed scales: span u of row r at ((u * rows) + r) * 16.  One thread per 16 bytes,
// the spans of a row side by side, so the reads are contiguous.
__global__ __launch_bounds__(256) void mxfp4_pack_scales_kernel(const uint8_t *__restrict__ ws,
                                                                const uint8_t *__restrict__ xs,
                                                                u32x4 *__restrict__ out, int N, int M,
                                                                int KB, int spans)
{
    const int rows = N + M;
    const uint32_t i0 = blockIdx.x * 256 + threadIdx.x;
    const int r = (int)(i0 / (uint32_t)spans), u = (int)(i0 - (uint32_t)r * (uint32_t)spans);
    if (r >= rows)
        return;
    const uint8_t *row = r < N ? ws + (size_t)r * KB : xs + (size_t)(r - N) * KB;
    out[(size_t)u * rows + r] = span_scales(row, 16 * u, KB);
}

// How the scales come into LDS: copied span by span from the rows themselves
// (K % 128 == 0, so a row's scale bytes are whole dwords) or from packed ones,
// or loaded by the workgroup at its start, all spans of its part.
enum class Scales { Straight, Packed, Whole };

// A wave's outputs (n from nw, m from mw) through its part of LDS, 32 output
// rows at a time: rows of 32 NB n are written as the accumulators hold them
// (acc[i][k][4 g + e] is n = 32 i + 8 g + 4 h + e, m = 32 k + r) and read back
// 16 bytes a lane, so a store covers whole runs of a row.  The LDS serves a
// wave's accesses in order, and no other wave uses this part.
template <class T, int DT>
__device__ __forceinline__ void store_wave(const float16_t (&acc)[T::NB][T::MB], void *y, int M, int N,
                                           int nw, int mw, uint8_t *stage)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2, ROW = 32 * T::NB * ES, PITCH = ROW + 16;
    constexpr int VECS = ROW / 16, RPI = 64 / VECS; // 16-byte pieces of a row; rows per instruction
    static_assert(32 * PITCH <= T::WSTAGE && 64 % VECS == 0, "staging space");
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int n = nw + lane % VECS * (16 / ES);
#pragma unroll
    for (int k = 0; k < T::MB; ++k) {
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4_t v{acc[i][k][4 * g], acc[i][k][4 * g + 1], acc[i][k][4 * g + 2],
                                 acc[i][k][4 * g + 3]};
                uint8_t *to = stage + r * PITCH + (32 * i + 8 * g + 4 * h) * ES;
                if constexpr (DT == DT_F32)
                    *reinterpret_cast<float4_t *>(to) = v;
                else
                    *reinterpret_cast<uint2 *>(to) =
                        uint2{f32x2_to_act2<DT>(v[0], v[1]), f32x2_to_act2<DT>(v[2], v[3])};
            }
#pragma unroll
        for (int q = 0; q < 32 / RPI; ++q) {
            const int row = q * RPI + lane / VECS, m = mw + 32 * k + row;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(stage + row * PITCH + lane % VECS * 16);
            if (m < M && n < N) // N % 8 == 0: a piece is whole
                *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(y) + ((size_t)m * N + n) * ES) = v;
        }
    }
}

// Packed: ws holds the packed scales of weight rows, then activation rows.
template <class T, Scales SC>
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
    const int KB = K >> 5, S = (KB + 15) >> 4; // blocks, spans of a row
    const int s_begin = (int)((int64_t)S * split / splits);
    const int s_end = (int)((int64_t)S * (split + 1) / splits); // > s_begin: splits <= S
    constexpr int GS = T::GS, NG = T::NG, GPS = 4 / GS; // stages of a group, groups in LDS, groups of a span
    const int groups = GPS * (s_end - s_begin);
    const uint32_t rowb = (uint32_t)K >> 1;
    constexpr int ND = T::ND;
    constexpr bool PACKED = SC == Scales::Packed, WHOLE = SC == Scales::Whole;
    constexpr int NSC = WHOLE ? 0 : PACKED ? T::SROWS / 256 : T::ROWS / 64; // scale copies per wave and span
    constexpr auto part_of = [](int w) { return w * ND / (2 * GS); }; // copies before part w of a group's 2 GS

    // Code copy d of wave v fills LDS rows RI (4 d + v) .. + RI - 1: lane L the
    // position L % LR of row L / LR.  Rows past the matrix repeat its last row
    // (never stored), pieces past the row its last piece (zeroed before use).
    constexpr int LR = 4 * GS, RI = 64 / LR; // lanes of a row, rows of a copy
    uint32_t row_at[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const int R = RI * (4 * d + wave) + lane / LR;
        row_at[d] = (uint32_t)(4 * RI * d < T::TN ? min(n0 + R, N - 1) : min(m0 + R - T::TN, M - 1)) * rowb;
    }
    static_assert(T::TN % (4 * RI) == 0, "a copy has rows of one operand");
    // position of a row's piece: piece ^ swizzle(row)
    auto swizzle = [](int R) __attribute__((always_inline)) { return GS == 1 ? (R >> 2) & 3 : (R >> 1) & 7; };
    const uint32_t piece = 16u * (uint32_t)(lane % LR ^ swizzle(RI * wave + lane / LR));
    const uint32_t lds0 = (uint32_t)(size_t)(lds_ptr_t *)smem;
    auto code_copy = [&](int g, int b, int d) __attribute__((always_inline)) { // group g into buffer b
        const int from = GPS * s_begin + min(g, groups - 1); // past the end: the last group again
        const uint32_t k = min((uint32_t)from * (uint32_t)T::SEG + piece, rowb - 16u);
        const uint32_t to = lds0 + (uint32_t)(b * T::GROUP + wave * 1024);
        lds_dma16(4 * RI * d < T::TN ? w : x, row_at[d] + k, to + (uint32_t)(4096 * d));
    };

    // Scale copy i of wave v fills LDS scale rows 64 (4 i + v) .. + 63 (Packed:
    // lane L all 16 bytes of row L) or 16 (4 i + v) .. + 15 (lane L dword L % 4 of
    // row L / 4, a dword past the row its last one: a finite scale or a NaN that
    // the row's result has anyway).
    constexpr int SC0 = NG * T::GROUP, SBUF = (WHOLE ? T::ROWS : T::SROWS) * 16;
    uint32_t scale_at[NSC + 1];
    const uint32_t spr = (uint32_t)KB >> 2; // scale dwords per row
#pragma unroll
    for (int i = 0; i < NSC; ++i) {
        if constexpr (PACKED) {
            const int R = 64 * (4 * i + wave) + lane;
            scale_at[i] = 16u * (uint32_t)(R < T::TN ? min(n0 + R, N - 1) : N + min(m0 + R - T::TN, M - 1));
        } else {
            const int R = 16 * (4 * i + wave) + (lane >> 2);
            scale_at[i] =
                (uint32_t)(64 * i < T::TN ? min(n0 + R, N - 1) : min(m0 + R - T::TN, M - 1)) * (uint32_t)KB;
        }
    }
    auto scale_copy = [&](int u, int i) __attribute__((always_inline)) {
        const int from = min(s_begin + u, s_end - 1);
        const uint32_t to = lds0 + (uint32_t)(SC0 + (u & 1) * SBUF);
        if constexpr (PACKED)
            lds_dma16(ws + (size_t)from * (size_t)(N + M) * 16, scale_at[i],
                      to + (uint32_t)(wave * 1024 + 4096 * i));
        else
            lds_dma4(64 * i < T::TN ? ws : xs,
                     scale_at[i] + 4u * min(4u * (uint32_t)from + (uint32_t)(lane & 3), spr - 1u),
                     to + (uint32_t)(wave * 256 + 1024 * i));
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
    uint32_t at[GS][2]; // position of piece 4 p + 2 h + j in a row of this lane
#pragma unroll
    for (int p = 0; p < GS; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            at[p][j] = 16u * (uint32_t)((4 * p + 2 * h + j) ^ swizzle(r));

    struct Operands {
        u32x4 a[T::NB], b[T::MB];
    };
    constexpr int NR = T::NB + T::MB;
    // operand i (weight blocks, then activation blocks) of step j of stage p of the group in buffer b
    auto read_operand = [&](int b, int p, int j, int i, Operands &o) __attribute__((always_inline)) {
        const uint8_t *base = smem + b * T::GROUP + at[p][j];
        if (i < T::NB)
            o.a[i] = *reinterpret_cast<const u32x4 *>(base + (an + 32 * i) * T::SEG);
        else
            o.b[i - T::NB] = *reinterpret_cast<const u32x4 *>(base + (bm + 32 * (i - T::NB)) * T::SEG);
    };
    // A lane's scale bytes of span u, in step order.
    struct Scales {
        u32x4 v[NR];
    };
    const uint32_t pick = h ? 0x07060302u : 0x05040100u; // bytes 2 h, 2 h + 1 of both dwords
    auto read_scale = [&](int u, int i, Scales &o) __attribute__((always_inline)) {
        const u32x4 *base = reinterpret_cast<const u32x4 *>(smem + SC0 + (WHOLE ? min(u, s_end - s_begin - 1) : u & 1) * SBUF);
        o.v[i] = base[i < T::NB ? an + 32 * i : bm + 32 * (i - T::NB)];
    };

    Operands op[2];
    Scales sc;
    {
#pragma unroll
        for (int g = 0; g < NG - 1; ++g) {
            if (g == 0)
#pragma unroll
                for (int i = 0; i < NSC; ++i)
                    scale_copy(0, i);
#pragma unroll
            for (int d = 0; d < ND; ++d)
                code_copy(g, g, d);
        }
#pragma unroll
        for (int d = 0; d < part_of(1); ++d)
            code_copy(NG - 1, NG - 1, d);
        if constexpr (WHOLE) {
            const int total = (s_end - s_begin) * T::ROWS;
            constexpr int B = 4; // loads of a thread under way at a time
            for (int i0 = tid; i0 < total; i0 += 256 * B) {
                u32x4 v[B];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int i = min(i0 + 256 * j, total - 1), u = i / T::ROWS, R = i - u * T::ROWS;
                    v[j] = span_scales(R < T::TN ? ws + (size_t)min(n0 + R, N - 1) * KB
                                                 : xs + (size_t)min(m0 + R - T::TN, M - 1) * KB,
                                       16 * (s_begin + u), KB);
                }
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (i0 + 256 * j < total)
                        reinterpret_cast<u32x4 *>(smem + SC0)[i0 + 256 * j] = v[j];
            }
            __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): written before the barrier
        }
        // group 0 and the first scales have landed
        wait_vmcnt<(NG - 2) * ND + part_of(1)>();
        barrier_only();
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            read_scale(0, i, sc);
            read_operand(0, 0, 0, i, op[0]);
        }
    }
    int cur = 0; // the buffer of the group at hand (NG = 4: of the span's first one, always 0)

    // Span u of this part (stages 4 u .. 4 u + 3).  TAIL: the row's partial last
    // span; nothing follows it.
    auto run_span = [&](int u, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        uint32_t sv8[2][NR]; // the scale bytes of each operand, in step order
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            sv8[0][i] = __builtin_amdgcn_perm(sc.v[i][1], sc.v[i][0], pick);
            sv8[1][i] = __builtin_amdgcn_perm(sc.v[i][3], sc.v[i][2], pick);
        }
        const int left = KB - 16 * (s_begin + u); // blocks of a partial span
        auto step = [&](auto sel) __attribute__((always_inline)) {
            constexpr int SEL = decltype(sel)::value, j = SEL & 1, p = SEL >> 1;
            // stage p = GS q + s of the span; a group's last step is its (2 GS)th
            constexpr int q = p / GS, s = p % GS, in_group = SEL % (2 * GS);
            constexpr bool END = in_group == 2 * GS - 1;
            const int g = GPS * u + q;
            auto buffer = [&](int k) __attribute__((always_inline)) { // of the group k after this one
                if constexpr (NG == GPS)
                    return (q + k) & (NG - 1);
                const int b = cur + k;
                return b >= NG ? b - NG : b;
            };
            Operands &now = op[j], &next = op[j ^ 1];
            if constexpr (END) {
                // group g + 1 has landed (and in the span's last group the next span's
                // scales, started in its first): the codes of groups g + 2 ..
                // g + NG - 1 may be in flight, and the scales that were started among them
                constexpr bool AMONG = GS == 1 ? p == 1 || p == 2 : p == 1;
                if constexpr (TAIL)
                    wait_vmcnt<0>();
                else
                    wait_vmcnt<(NG - 2) * ND + (AMONG ? NSC : 0)>();
                __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): this wave's reads of group g
                barrier_only();
            }
            if constexpr (TAIL) { // blocks past the row: zero weights
                const bool in = 4 * p + 2 * h + j < left;
#pragma unroll
                for (int i = 0; i < T::NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        now.a[i][e] = in ? now.a[i][e] : 0u;
            }
            // The step's other work, one piece at a time between the MFMAs: the
            // next step's operands, (SEL 7) the next span's scales, then copies.
            // In the partial last span only the rest of its own fourth stage is
            // still to be copied.
            constexpr bool LAST = TAIL && (GS != 1 || SEL != 0);
            constexpr int PART = END ? 0 : in_group + 1, C0 = part_of(PART), C1 = part_of(PART + 1);
            constexpr int RS = SEL == 7 && !TAIL ? NR : 0, SCC = SEL == 1 && !TAIL ? NSC : 0;
            constexpr int SIDE = NR + RS + SCC + (LAST ? 0 : C1 - C0), NM = T::NB * T::MB;
            auto side = [&](int i) __attribute__((always_inline)) {
                if (i < NR)
                    read_operand(buffer(END ? 1 : 0), END ? 0 : s + j, j ^ 1, i, next);
                else if (i < NR + RS)
                    read_scale(u + 1, i - NR, sc);
                else if (i < NR + RS + SCC)
                    scale_copy(u + 1, i - NR - RS);
                else
                    code_copy(END ? g + NG : g + NG - 1, buffer(END ? 0 : NG - 1), C0 + i - NR - RS - SCC);
            };
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int i = m / T::MB, k = m % T::MB;
                __builtin_amdgcn_sched_barrier(0);
                acc[i][k] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fp4_operand(now.a[i]), fp4_operand(now.b[k]), acc[i][k], FMT_FP4, FMT_FP4, SEL & 3,
                    (int)sv8[SEL >> 2][i], SEL & 3, (int)sv8[SEL >> 2][T::NB + k]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int z = 0; z < SIDE; ++z)
                    if (z >= m * SIDE / NM && z < (m + 1) * SIDE / NM)
                        side(z);
            }
            if constexpr (END && NG != GPS)
                cur = buffer(1);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        if (TAIL && left <= 4)
            return; // (the same for the whole workgroup)
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        if (TAIL && left <= 8)
            return;
        step(std::integral_constant<int, 4>{});
        step(std::integral_constant<int, 5>{});
        if (TAIL && left <= 12)
            return;
        step(std::integral_constant<int, 6>{});
        step(std::integral_constant<int, 7>{});
    };
    const int full = (KB & 15 ? min(s_end, S - 1) : s_end) - s_begin;
    for (int u = 0; u < full; ++u)
        run_span(u, std::false_type{});
    if (full < s_end - s_begin)
        run_span(full, std::true_type{});
    wait_vmcnt<0>(); // copies past the end: none is in flight when the workgroup ends

    // Every wave has read its last operands (the barrier of the last stage came
    // before them, so one more): the stage buffers become staging space.
    barrier_only();
    uint8_t *stage = smem + wave * T::WSTAGE;
    if (splits > 1)
        store_wave<T, DT_F32>(acc, part + (size_t)split * M * N, M, N, n0 + 32 * T::NB * wn,
                              m0 + 32 * T::MB * wm, stage);
    else if (ydt == DT_F32)
        store_wave<T, DT_F32>(acc, y, M, N, n0 + 32 * T::NB * wn, m0 + 32 * T::MB * wm, stage);
    else if (ydt == DT_F16)
        store_wave<T, DT_F16>(acc, y, M, N, n0 + 32 * T::NB * wn, m0 + 32 * T::MB * wm, stage);
    else
        store_wave<T, DT_BF16>(acc, y, M, N, n0 + 32 * T::NB * wn, m0 + 32 * T::MB * wm, stage);
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
    constexpr int B = 4; // parts under way at a time
    for (int s0 = 1; s0 < splits; s0 += B) {
        float4_t a[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            a[j] = part[(size_t)min(s0 + j, splits - 1) * n4 + i];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s0 + j < splits)
                v += a[j];
    }
    store4(y, ydt, (size_t)i * 4, v);
}

size_t parts_bytes(int64_t M, int64_t N, int splits)
{
    return splits > 1 ? (size_t)splits * (size_t)M * (size_t)N * sizeof(float) : 0; // N % 8 == 0
}

template <class T, Scales SC>
hipError_t launch_tile(const uint8_t *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                       void *y, int ydt, int M, int N, int K, int splits, void *workspace, hipStream_t stream)
{
    auto kern = mxfp4_tile_kernel<T, SC>;
    const int spans = (K + MX_SPAN - 1) / MX_SPAN, part_spans = (spans + splits - 1) / splits;
    const int lds = SC == Scales::Whole ? std::max(T::LDS, T::NG * T::GROUP + part_spans * T::ROWS * 16) : T::LDS;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), 160 * 1024, lds_set);
        e != hipSuccess)
        return e;
    const int tiles_m = (M + T::TM - 1) / T::TM;
    const int64_t tiles = (int64_t)tiles_m * ((N + T::TN - 1) / T::TN);
    const int nxcd = device_topology().xcds;
    const int64_t grid = (int64_t)nxcd * ((tiles * splits + nxcd - 1) / nxcd);
    if (grid > INT32_MAX / 256)
        return hipErrorInvalidValue;
    float *part = static_cast<float *>(workspace);
    if constexpr (SC == Scales::Packed) {
        uint8_t *scales = static_cast<uint8_t *>(workspace) + parts_bytes(M, N, splits);
        hipLaunchKernelGGL(mxfp4_pack_scales_kernel,
                           dim3((unsigned)(((int64_t)(M + N) * spans + 255) / 256)), dim3(256), 0, stream,
                           ws, xs, reinterpret_cast<u32x4 *>(scales), N, M, K >> 5, spans);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        ws = scales;
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), (size_t)lds, stream, x, xs, w, ws, y,
                       ydt, part, M, N, K, tiles_m, (int)tiles, splits, nxcd);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1)
        return e;
    const int64_t n4 = (int64_t)M * N / 4;
    hipLaunchKernelGGL(mxfp4_sum_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream,
                       reinterpret_cast<const float4_t *>(part), y, ydt, n4, splits);
    return hipGetLastError();
}

template <class T, class... A>
hipError_t launch_scales(Scales scales, A... a)
{
    if (scales == Scales::Straight)
        return launch_tile<T, Scales::Straight>(a...);
    if (scales == Scales::Packed)
        return launch_tile<T, Scales::Packed>(a...);
    return launch_tile<T, Scales::Whole>(a...);
}

using TileL = MxTile<2, 4, 4, 1, 4>; // 256 x 256
using TileM = MxTile<2, 2, 2, 2, 3>; // 128 x 128
using TileS = MxTile<2, 1, 2, 2, 3>; // 64 weight rows x 128 activation rows
using TileN = MxTile<2, 1, 1, 2, 3>; // 64 x 64

// Spans of a part of the 64 x 128 tile, at most (see plan): their scales always fit.
constexpr int SMALL_SPANS = 11;
static_assert(TileS::SPANS >= SMALL_SPANS, "no packed form of the 64 x 128 tile");

// Rows and scales of x must leave the LDS room for a second workgroup.
bool few_rows(int64_t M, int64_t K) { return M <= 16 && K <= 65536 && few_lds((int)M, (int)K, 8, 2) <= 80 * 1024; }
enum class Path { Few, Large, Medium, Small, Narrow };

struct Plan {
    Path path;
    Scales scales;
    int splits;
};

// K parts for `tiles` tiles so that up to one workgroup reaches each CU, at least
// two spans each.  A part costs its sums' way through memory and the launch that
// adds them, about 4.5 us, so there is one only where it takes five spans off the
// longest workgroup.  us, in parts / whole: 100 x 5376 x 21504 24.1 / 63.9, 32 x 5376 x
// 21504 21.6 / 37.6, 100 x 2048 x 4096 (eight spans in four) 9.2 / 11.5, 48 x 5376 x 5376
// 10.9 / 12.4; where the rule says whole: 100 x 5760 x 2880 13.4 / 13.0, 20 x 8192 x 3584 9.7 /
// 9.2, but 100 x 4096 x 3584 (seven spans in three) 10.8 / 11.4.  Two workgroups on each CU
// bring nothing, one / two: 100 x 16384 x 5376 18.6 / 22.8, 64 x 16384 x 5376 15.0 / 20.7, 100 x
// 5376 x 21504 24.1 / 28.3 (32 x 5376 x 21504 21.6 / 20.7).
int k_parts(int64_t tiles, int64_t K)
{
    const int64_t spans = (K + MX_SPAN - 1) / MX_SPAN;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({256 / tiles, spans / 2, 16}));
    return spans - (spans + parts - 1) / parts >= 5 ? (int)parts : 1;
}

template <class T>
int64_t tile_count(int64_t M, int64_t N) { return ((M + T::TM - 1) / T::TM) * ((N + T::TN - 1) / T::TN); }

// Rows whose scale bytes are not whole dwords are loaded at the start where a part's fit:
// 700 x 2048 x 992 6.8 us and 9.0 packed, 36 x 1768 x 4960 8.8 and 10.9, 100 x 5760 x 4000 16.0 and
// 16.9.  Others are copied as they are used: 100 x 5760 x 2944 8.4 and 9.6 loaded at the
// start, 200 x 16384 x 2944 14.1 and 15.9.
template <class T>
Scales tile_scales(int64_t K, int parts)
{
    const int64_t spans = (K + MX_SPAN - 1) / MX_SPAN;
    if (K % 128 == 0)
        return Scales::Straight;
    return (spans + parts - 1) / parts <= T::SPANS ? Scales::Whole : Scales::Packed;
}

// The 256 x 256 tile: a round of one a CU takes as long as 2.5 of the 128 x 128 tile, a
// quarter of it.  Rounds of both, us: 1 and 3, 48.1 and 60.0 (2048 x 6144 x 5376); 1 and 2, 45.4
// and 40.6 (2048 x 4096 x 5376); 2 and 5, 86.2 and 90.1 (2048 x 8704 x 5376), 67.9 and 67.8 (1100 x
// 16384 x 2880); 2 and 4, 58.7 and 54.3 (1030 x 14000 x 2880).
bool large_tile(int64_t M, int64_t N)
{
    const int64_t large = (tile_count<TileL>(M, N) + 255) / 256, medium = (tile_count<TileM>(M, N) + 255) / 256;
    return 2 * medium >= 5 * large;
}

Plan plan(int64_t M, int64_t N, int64_t K)
{
    if (few_rows(M, K))
        return {Path::Few, Scales::Straight, 1};
    if (large_tile(M, N))
        return {Path::Large, Scales::Packed, 1};
    const int64_t spans = (K + MX_SPAN - 1) / MX_SPAN;
    const int small = k_parts(tile_count<TileS>(M, N), K);
    // A tile of twice the weight rows reads x half as often.  It is taken where the
    // small tile's parts are still long (100 x 5376 x 21504, 14 spans a part: 23.4 us and
    // 26.2 with the small one, 200 x 5376 x 21504, 42: 31.5 and 55.4; but 100 x 5376 x 10752,
    // 7 spans, 17.8 and 17.0, 100 x 16384 x 5376, 11, 20.6 and 18.1), and where its
    // workgroups are on the CUs all at once and the small one's are not (200 x 16384 x 2880
    // 18.2 and 20.7, 1000 x 4096 x 5376 20.4 and 24.0) or fill their second round (1024 x
    // 8192 x 5376, 512 workgroups, 39.9 and 46.0; but 600 x 8192 x 2880, 320, 27.2 and 25.9,
    // 250 x 24576 x 2880, 384, 31.5 and 30.1).  Up to 64 rows, where half of it is
    // idle, it brings little or loses (64 x 16384 x 5376 18.6 and 15.9).
    const int64_t medium = tile_count<TileM>(M, N);
    const bool fills = tile_count<TileS>(M, N) > 256 && (medium <= 256 || medium > 384);
    if (M > 64 && (spans > SMALL_SPANS * (int64_t)small || fills))
        return {Path::Medium, tile_scales<TileM>(K, k_parts(medium, K)), k_parts(medium, K)};
    // 17 to 64 rows: 32 x 5760 x 2880 7.8 us and 9.2 in the small tile, 64 x 16384 x 5376 14.8 and 16.0,
    // 32 x 5376 x 21504 19.5 and 20.7 (128 weight rows: 9.8, 17.9, 18.7).
    if (M <= 64)
        return {Path::Narrow, tile_scales<TileN>(K, small), small};
    return {Path::Small, tile_scales<TileS>(K, small), small};
}

} // namespace

size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M == 0 || N == 0)
        return 0;
    const Plan p = plan(M, N, K);
    const int64_t spans = (K + MX_SPAN - 1) / MX_SPAN;
    return parts_bytes(M, N, p.splits) + (p.scales == Scales::Packed ? (size_t)(M + N) * (size_t)spans * 16 : 0);
}

hipError_t launch_mxfp4_gemm(const uint8_t *x, const uint8_t *xs, const uint8_t *w,
                             const uint8_t *ws, void *y, int ydt, int M, int N, int K,
                             void *workspace, hipStream_t stream)
{
    const Plan p = plan(M, N, K);
    if (p.path == Path::Few) {
        // Two groups of eight waves where one group a workgroup would be more than one a CU,
        // and K gives the waves work; else one group, of four waves below 4096.  us, two
        // groups / one:
        //   256 workgroups of one group: 1 x 4096 x 14336 12.1 / 9.2, 8 x 4096 x 4096 6.9 / 5.5,
        //   16 x 4096 x 8192 11.1 / 9.9
        //   more: 1 x 5376 x 21504 17.0 / 17.8, 16 x 6144 x 8192 11.7 / 12.1, 8 x 16384 x 5376
        //   11.2 / 12.4; but 1 x 16384 x 5376 10.7 / 10.4, 1 x 43008 x 5376 23.7 / 22.1
        //   below 4096 (one group of four waves), more than 8 rows: 16 x 4104 x 2880 4.8 / 5.5,
        //   13 x 5760 x 2880 5.2 / 5.7, 16 x 8192 x 2880 5.2 / 6.7; up to 8: 8 x 43008 x 2880
        //   16.1 / 15.1, 1 x 16384 x 2880 7.4 / 6.8 (but 8 x 8192 x 2880 4.8 / 5.2)
        //   up to 2048: 1 x 43008 x 2048 19.7 / 11.3, 16 x 43008 x 2048 20.5 / 15.1,
        //   1 x 2048 x 2048 4.9 / 2.9
        const int groups = (N + FR_ROWS - 1) / FR_ROWS;
        if (groups > 256 && (K >= 4096 || (K > 2048 && M > 8)))
            return launch_few<8, 2>(x, xs, w, ws, y, ydt, M, N, K, stream);
        if (K >= 4096)
            return launch_few<8, 1>(x, xs, w, ws, y, ydt, M, N, K, stream);
        return launch_few<4, 1>(x, xs, w, ws, y, ydt, M, N, K, stream);
    }
    if (p.path == Path::Large)
        return launch_tile<TileL, Scales::Packed>(x, xs, w, ws, y, ydt, M, N, K, 1, workspace, stream);
    if (p.path == Path::Medium)
        return launch_scales<TileM>(p.scales, x, xs, w, ws, y, ydt, M, N, K, p.splits, workspace, stream);
    if (p.path == Path::Narrow)
        return launch_scales<TileN>(p.scales, x, xs, w, ws, y, ydt, M, N, K, p.splits, workspace, stream);
    if (p.scales == Scales::Straight)
        return launch_tile<TileS, Scales::Straight>(x, xs, w, ws, y, ydt, M, N, K, p.splits, workspace, stream);
    return launch_tile<TileS, Scales::Whole>(x, xs, w, ws, y, ydt, M, N, K, p.splits, workspace, stream);
}

} // namespace wob
