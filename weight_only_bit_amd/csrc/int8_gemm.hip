// 8-bit product on gfx950:
//     y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k]  (+ bias[n])
//
// The sums are exact in 32 bits (K 2^14 < 2^31), so their order and their split do not
// show in the result; they are converted to binary32, scaled twice, added to the bias
// and rounded once to y's type.  A holds weight rows and B activation rows, so a lane ends
// with runs of four consecutive n of one output row.  Which 16 k of a row meet in one
// instruction is free as long as both operands agree.
//
// Two kernels:
//  * few rows (M <= 16): waves own 8 or 16 weight rows each and may split K; the weights go
//    from memory straight into registers (v_mfma_i32_16x16x64_i8); bound by their bytes.
//  * tiles: both operands through LDS (v_mfma_i32_32x32x32_i8), K optionally split over
//    workgroups with a sum in a second kernel.
#include "wob_rows.hpp"
#include "wob_tile.hpp"

#include <math.h>

#include <algorithm>
#include <type_traits>

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

// Four sums of one row, scaled: binary32 steps in the order that the contract names.
__device__ __forceinline__ float4_t scaled4(const i32x4 &sum, float xs, const float4_t &ws)
{
    float4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = (float)sum[e] * xs * ws[e];
    return v;
}

// ---- Few rows --------------------------------------------------------------
//
// M <= 16.  A wave owns 8 weight rows, with M > 8 (WIDE) 16; W waves share them and split K,
// and their sums are joined in LDS.  A workgroup has G such groups of rows.  The weights go from
// memory into registers, FR_D loads of a lane ahead; only x passes through LDS, with its loads ahead of the
// weights' so that they land first.  Its pitch is 16 mod 128 bytes: the same piece of all rows lies in
// different banks, but neighbouring pieces of neighbouring rows meet (2.3 conflict cycles a LDS instruction
// with 13 rows, none with one, whose reads are the same in every lane).
//
// A load is one whole cache line of each of 8 weight rows: lane (r, q) = (lane % 16, lane / 16)
// holds piece 4 (r / 8) + q of the line of row r % 8.  With up to 8 activation rows that is the
// instruction's first operand as it is: its rows 0 to 7 and 8 to 15 are the same weight rows with
// the two halves of 128 k, its column j is activation row j % 8 with half j / 8, and of
// its sums the two 8 x 8 blocks of equal halves are used.  WIDE: the second load holds rows 8 + r %
// 8 with the halves swapped, so lanes r < 8 of the one and r >= 8 of the other are rows 0 to 15 with the
// first half, and the rest are rows r ^ 8 with the second.
//
// Bound by the weights' bytes: 1 x 16384 x 5376 (88 MB) 16.3 us, a plain read of as many 14.7 to 15.2;
// 1 x 43008 x 5376 (231 MB) 40, a read 33.6; 13 x 5760 x 2880 (17 MB) 7.0, a read 3.9 (graph replays over
// copies larger than the caches; in the last of them a workgroup stages 37 KB of x for 69 KB of weights
// before its first product).  With half lines of 16 rows a load 17.8, 48 and 7.3.  Nothing reads a
// line twice, so the loads are nontemporal: past the caches / with three sets of weights 8 x 16384 x
// 5376 19.6 / 18.3, ordinary 20.9 / 17.2; 4 x 10752 x 5376 15.2 / 14.6, 16.5 / 13.1; 13 x 5760 x 2880 7.1 /
// 6.5, 7.8 / 6.9.
constexpr int FR_D = 6; // loads ahead

__host__ __device__ inline int few_pitch(int K) { return (K + 127 - 16) / 128 * 128 + 16; }

template <int W, int G, bool WIDE>
__global__ __launch_bounds__(64 * W * G) void int8_few_kernel(Int8GemmArgs a, int M, int N, int K,
                                                             int rows)
{
    constexpr int NT = 64 * W * G, L = WIDE ? 2 : 1, U = FR_D / L; // loads of a line, lines ahead
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), k = wave % W, g = wave / W;
    const int KB = K >> 4, lines = (KB + 7) >> 3, pitch = few_pitch(K);
    const int n0 = blockIdx.x * rows + 8 * L * g, n_end = min((blockIdx.x + 1) * rows, N); // (rows <= 8 L G)

    // Staging of x, 16 bytes a thread, the first round's loads ahead of the weights'.
    const int nx = M * KB;
    const u32x4 *xg = reinterpret_cast<const u32x4 *>(a.x);
    const u32x4 x_first = xg[min(tid, nx - 1)];

    const u32x4 *wr[L];
#pragma unroll
    for (int l = 0; l < L; ++l)
        wr[l] = reinterpret_cast<const u32x4 *>(a.w) + (size_t)min(n0 + 8 * l + r % 8, n_end - 1) * KB;
    const int mine = (lines - k + W - 1) / W; // lines of this wave
    u32x4 ring[U][L];
    auto load = [&](int i, u32x4 (&s)[L]) __attribute__((always_inline)) { // line i of this wave
#pragma unroll
        for (int l = 0; l < L; ++l) {
            int b = min(8 * (k + W * i) + 4 * (r / 8 ^ l) + q, KB - 1);
            asm volatile("" : "+v"(b)); // one address per load, not one pointer kept per slot
            s[l] = __builtin_nontemporal_load(wr[l] + b);
        }
    };
#pragma unroll
    for (int d = 0; d < U; ++d)
        load(min(d, max(mine - 1, 0)), ring[d]);
    __builtin_amdgcn_sched_barrier(0);

    auto put_x = [&](int i, const u32x4 &v) __attribute__((always_inline)) {
        const int m = M == 1 ? 0 : i / KB;
        *reinterpret_cast<u32x4 *>(smem + (size_t)m * pitch + (size_t)(i - m * KB) * 16) = v;
    };
    if (tid < nx)
        put_x(tid, x_first);
    for (int i = tid + NT; i < nx; i += NT)
        put_x(i, xg[i]);
    __syncthreads();

    const uint8_t *xrow = smem + (size_t)min(WIDE ? r : r % 8, M - 1) * pitch;
    i32x4 acc[L] = {};
    auto multiply = [&](int i, const u32x4 (&s)[L]) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = 8 * (k + W * i) + 4 * (WIDE ? l : r / 8) + q;
            const bool in = b < KB; // the last line may leave some lanes without a piece
            const bool first = !WIDE || (r < 8) == (l == 0); // which load has it
            u32x4 wv;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                wv[e] = in ? (first ? s[0][e] : s[L - 1][e]) : 0u;
            const i32x4 xv = *reinterpret_cast<const i32x4 *>(xrow + 16 * min(b, KB - 1));
            acc[l] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bitcast<i32x4>(wv), xv, acc[l], 0, 0, 0);
        }
    };
    int i = 0;
    for (; i + U < mine; i += U) {
#pragma unroll
        for (int d = 0; d < U; ++d) {
            if (i + d < mine)
                multiply(i + d, ring[d]);
            __builtin_amdgcn_sched_barrier(0);
            load(min(i + d + U, mine - 1), ring[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < U; ++d)
        if (i + d < mine)
            multiply(i + d, ring[d]);
    // Lane (r, q) holds the instruction's rows 4 q + e of its column r: the sums of both halves
    // and of all waves of a group meet at the lane of their first half.
    __syncthreads();
    i32x4 *const part = reinterpret_cast<i32x4 *>(smem) + g * W * L * 64;
#pragma unroll
    for (int l = 0; l < L; ++l)
        part[(k * L + l) * 64 + (lane ^ 32 * l)] = acc[l];
    __syncthreads();
    const int n = n0 + 4 * q;
    if (k != 0 || r >= M || n >= n_end || (!WIDE && (r >= 8 || q >= 2)))
        return;
    i32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < W; ++j)
        sum += part[j * L * 64 + lane] + part[j * L * 64 + lane + (WIDE ? 64 : 2 * 16 + 8)];
    float4_t v = scaled4(sum, a.xs[r], *reinterpret_cast<const float4_t *>(a.ws + n));
    if (a.bias)
        v += *reinterpret_cast<const float4_t *>(a.bias + n);
    store4(a.y, a.ydt, (size_t)r * N + n, v);
}

template <int W, int G, bool WIDE>
hipError_t launch_few(const Int8GemmArgs &a, int M, int N, int K, int rows, hipStream_t stream)
{
    auto kern = int8_few_kernel<W, G, WIDE>;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), 160 * 1024, lds_set);
        e != hipSuccess)
        return e;
    const size_t lds = std::max((size_t)M * few_pitch(K), (size_t)W * G * (WIDE ? 2 : 1) * 1024); // x, then the sums
    hipLaunchKernelGGL(kern, dim3((N + rows - 1) / rows), dim3(64 * W * G), lds, stream, a, M, N, K, rows);
    return hipGetLastError();
}

// ---- Tiles -----------------------------------------------------------------
//
// A workgroup of 4 waves (WN along n, 4 / WN along m) owns TN weight rows x TM activation
// rows; a wave owns NB x MB blocks of 32 x 32 outputs.  K advances in stages of 64 (64
// bytes a row).  GS of them form a group, which is copied as one piece of 64 GS bytes a
// row.  LDS holds NH half groups (the weight rows' bytes and the activation rows' are halves
// of a group) in a ring: half i of the sequence A0 B0 A1 B1 .. lies in place i % NH, and is
// copied by global_load_lds (1 KB a wave instruction) as soon as half i - NH has been used.
//
// A stage is two MFMA steps of 32 k: in step j the lane half h = lane / 32 supplies the 16
// bytes of piece 2 h + j of its row.  LDS row R (weight rows, then activation rows) holds
// 64 GS bytes of a group; its 16-byte piece p lies at position p ^ swizzle(R), so the rows
// that one piece is read from at a time cover all 64 banks.
//
// Order within a group: its steps but the last read the next step's operands and multiply;
// then group g + 1's copies are waited for, a barrier makes them visible and frees group g's
// places (every wave has its last operands in registers), and the last step reads group
// g + 1's first operands and starts the copies into group g's places while it multiplies;
// the steps of group g + 1 go on with them.
//
// Copies cost one cache look-up a row and instruction, so whole lines (GS = 2) are copied, and the
// 256 x 256 tile, of which two groups fit, gets half a third.  2048 x 16384 x 5376, us: four groups of
// 64 bytes a row 175 to 191, five 179, two of 128 bytes 174 to 187, two and a half 158 to 160.  The
// other tiles are bound by bytes; rings of an odd number of halves are faster for them too, deeper ones
// and eight waves of half the blocks are not: 64 x 16384 x 5376 in the 64 x 64 tile (nontemporal) 8 halves
// 21.8, 9 18.7, 10 21.6, 11 18.5, 13 18.7; 100 x 5376 x 21504 in the 128 x 128 tile 6 34.6, 7 33.6, 8 34.5, 9 33.2.
//
// 2048 x 16384 x 5376, 150 to 165 us (2.2 to 2.4 POPS; the library's product of the operands without
// scales 164): the power limit.  MFMA busy 61 % at 1.75 GHz; with zero codes, which switch nothing,
// the same launches take 117, and an order of reads and copies that takes 4 off that takes
// nothing off this.  Timing-only forms: no stores 148 to 158, no copies 142 to 149, neither 121 to
// 127, the MFMAs alone, from registers, 108 (72 at 2.4 GHz).
template <int WN_, int NB_, int MB_, int GS_, int NH_>
struct Int8Tile {
    static constexpr int WN = WN_, WM = 4 / WN_, NB = NB_, MB = MB_, GS = GS_, NH = NH_;
    static constexpr int TN = 32 * NB * WN, TM = 32 * MB * WM, ROWS = TN + TM;
    static constexpr int SEG = 64 * GS;                  // bytes of a row in a group
    static constexpr int GROUP = ROWS * SEG;             // bytes of one group
    static constexpr int ND = GROUP / 4096;              // copies per wave and group
    static constexpr int NDA = TN * SEG / 4096;          // of them weight rows
    static constexpr int RING = NH * GROUP / 2;
    static constexpr int SCALES = 4 * (2 * TN + TM);     // scales and bias of the tile, in the epilogue
    static constexpr int WSTAGE = 32 * (128 * NB + 16);  // LDS of one wave in the epilogue
    static constexpr int LDS = std::max(RING, SCALES + 4 * WSTAGE);
    static_assert(ROWS % 64 == 0 && (GS == 1 || GS == 2) && NH >= 4 && LDS <= 160 * 1024, "tile geometry");
    static_assert(NH % 2 == 0 || TN == TM, "halves of one size");
};

// lds_dma16, or the same with a nontemporal load.
template <bool NT>
__device__ __forceinline__ void copy_weights(const int8_t *w, uint32_t at, uint32_t lds_addr)
{
    if constexpr (!NT) {
        lds_dma16(w, at, lds_addr);
    } else {
        const uint64_t b = reinterpret_cast<uint64_t>(w); // uniform: in scalar registers
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
        uint32_t saved;
        asm volatile("s_mov_b32 %0, m0\n\t"
                     "s_mov_b32 m0, %1\n\t"
                     "global_load_lds_dwordx4 %2, %3 nt\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(at), "s"((uint64_t)hi << 32 | lo)
                     : "memory");
    }
}

// A wave's outputs (n from nw, m from mw) through its part of LDS, 32 output rows at a
// time: rows of 32 NB n are written as the accumulators hold them (acc[i][k][4 g + e] is n =
// 32 i + 8 g + 4 h + e, m = 32 k + r) and read back 16 bytes a lane, so a store covers
// whole runs of a row.  The LDS serves a wave's accesses in order, and no other wave uses
// this part.  RAW: the sums themselves, as one of the K parts.  (The columns' scales in registers:
// 2048 x 16384 x 5376 with zero codes 122 us to 117.)
template <class T, int DT, bool RAW, bool BIAS>
__device__ __forceinline__ void store_wave(const i32x16 (&acc)[T::NB][T::MB], void *y, int M, int N, int nw, int mw,
                                           const float *ws, const float *bias, const float *xs, uint8_t *stage)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2, ROW = 32 * T::NB * ES, PITCH = ROW + 16;
    constexpr int VECS = ROW / 16, RPI = 64 / VECS; // 16-byte pieces of a row; rows per instruction
    static_assert(32 * PITCH <= T::WSTAGE && 64 % VECS == 0, "staging space");
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int n = nw + lane % VECS * (16 / ES);
    float4_t wv[4 * T::NB]; // scales of this lane's columns, for all its rows
    if constexpr (!RAW)
#pragma unroll
        for (int i = 0; i < 4 * T::NB; ++i)
            wv[i] = *reinterpret_cast<const float4_t *>(ws + 8 * i + 4 * h);
#pragma unroll
    for (int k = 0; k < T::MB; ++k) {
        const float x = RAW ? 0.f : xs[32 * k + r];
#pragma unroll
        for (int i = 0; i < T::NB; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            i32x16 block = acc[i][k];
            // 256 accumulators stay in the accumulator registers up to their use (taken out for
            // all stores at once, half of them went through memory)
            if constexpr (T::NB * T::MB == 16)
                asm volatile("" : "+a"(block));
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const i32x4 sum{block[4 * g], block[4 * g + 1], block[4 * g + 2], block[4 * g + 3]};
                const int at = 32 * i + 8 * g + 4 * h;
                uint8_t *to = stage + r * PITCH + at * ES;
                if constexpr (RAW) {
                    *reinterpret_cast<i32x4 *>(to) = sum;
                } else {
                    float4_t v = scaled4(sum, x, wv[4 * i + g]);
                    if constexpr (BIAS)
                        v += *reinterpret_cast<const float4_t *>(bias + at);
                    if constexpr (DT == DT_F32)
                        *reinterpret_cast<float4_t *>(to) = v;
                    else
                        *reinterpret_cast<uint2 *>(to) =
                            uint2{f32x2_to_act2<DT>(v[0], v[1]), f32x2_to_act2<DT>(v[2], v[3])};
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 32 / RPI; ++q) {
            const int row = q * RPI + lane / VECS, m = mw + 32 * k + row;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(stage + row * PITCH + lane % VECS * 16);
            if (m < M && n < N) // N % 8 == 0: a piece is whole
            {
                u32x4 *const to = reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(y) + ((size_t)m * N + n) * ES);
                if constexpr (RAW)
                    *to = v;
                else
                    __builtin_nontemporal_store(v, to);
            }
        }
    }
}

// NT: weights are copied nontemporally, but for the halves that fill the ring at the start (see launch_once).
template <class T, bool NT>
__global__ __launch_bounds__(256) void int8_tile_kernel(Int8GemmArgs a, int *__restrict__ part, int M, int N, int K,
                                                        int tiles_m, int tiles, int splits, int nxcd)
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
    constexpr int GS = T::GS, NH = T::NH, STEPS = 2 * GS, ND = T::ND, NDA = T::NDA;
    constexpr bool ODD = NH % 2 != 0;
    const int row_groups = (K + T::SEG - 1) / T::SEG;
    const int g_begin = (int)((int64_t)row_groups * split / splits);
    const int g_end = (int)((int64_t)row_groups * (split + 1) / splits); // > g_begin: splits <= row_groups
    const int groups = g_end - g_begin;
    const uint32_t rowb = (uint32_t)K;
    constexpr auto part_of = [](int w) { return w * ND / STEPS; }; // copies before part w of STEPS

    // Copy d of wave v fills LDS rows RI (4 d + v) .. + RI - 1: lane L the position L % LR of
    // row L / LR.  Rows past the matrix repeat its last row (never stored), pieces past the
    // row its last piece (zeroed before use).
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
    struct Place { // of a group's halves in LDS
        int a, b;
    };
    auto half_size = [](bool second) { return second ? T::TM * T::SEG : T::TN * T::SEG; };
    auto following = [&](Place p) __attribute__((always_inline)) { // of the next group
        if constexpr (!ODD) {
            const int a = p.a + T::GROUP == T::RING ? 0 : p.a + T::GROUP;
            return Place{a, a + half_size(false)};
        }
        auto two_on = [](int at) { return at + T::GROUP >= T::RING ? at + T::GROUP - T::RING : at + T::GROUP; };
        return Place{two_on(p.a), two_on(p.b)};
    };
    // Copy d of those into the places of group g, once they are free: the next halves of the
    // sequence that are not in LDS, A and B of group g + NH / 2 (NH odd: B of that one and A of
    // the one after it).
    auto copy = [&](int g, const Place &p, int d, auto nt) __attribute__((always_inline)) {
        const bool second = d >= (ODD ? ND / 2 : NDA); // into place b
        const bool b_rows = ODD ? !second : second;
        const int i = ODD ? (second ? d - ND / 2 : d + ND / 2) : d;
        // past the end: the last group again
        const int from = g_begin + min(g + NH / 2 + (ODD && second), groups - 1);
        const uint32_t k = min((uint32_t)from * (uint32_t)T::SEG + piece, rowb - 16u);
        const int to = (second ? p.b : p.a) + 4096 * (second ? d - (ODD ? ND / 2 : NDA) : d) + wave * 1024;
        if (b_rows)
            lds_dma16(a.x, row_at[i] + k, lds0 + (uint32_t)to);
        else
            copy_weights<decltype(nt)::value>(a.w, row_at[i] + k, lds0 + (uint32_t)to);
    };

    i32x16 acc[T::NB][T::MB] = {};

    const int an = 32 * T::NB * wn + r, bm = 32 * T::MB * wm + r; // this lane's first rows in LDS
    uint32_t at[GS][2]; // position of piece 4 p + 2 h + j in a row of this lane
#pragma unroll
    for (int p = 0; p < GS; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            at[p][j] = 16u * (uint32_t)((4 * p + 2 * h + j) ^ swizzle(r));

    struct Operands {
        i32x4 a[T::NB], b[T::MB];
    };
    constexpr int NR = T::NB + T::MB, NM = T::NB * T::MB;
    // operand i (weight blocks, then activation blocks) of step s of the group at p
    auto read_operand = [&](const Place &p, int s, int i, Operands &o) __attribute__((always_inline)) {
        const uint32_t lane_at = at[s >> 1][s & 1];
        if (i < T::NB)
            o.a[i] = *reinterpret_cast<const i32x4 *>(smem + p.a + lane_at + (an + 32 * i) * T::SEG);
        else
            o.b[i - T::NB] = *reinterpret_cast<const i32x4 *>(smem + p.b + lane_at + (bm + 32 * (i - T::NB)) * T::SEG);
    };

    Operands op[2];
    Place now_at = {0, half_size(false)}; // of the group at hand
    // of the group before it, whose places are being filled again; of group -1 the last ones
    Place before = {(NH - 2) * (T::GROUP / 2), (NH - 2) * (T::GROUP / 2) + half_size(false)};
    {
        // halves 0 .. NH - 3, as the ones that groups -NH / 2 .. -2 (NH odd: and half of one before
        // them) leave their places to
        Place p = now_at;
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < NH - 2; ++i) {
                const bool second = i % 2 != 0;
#pragma unroll
                for (int d = 0; d < ND / 2; ++d) {
                    const uint32_t k = min((uint32_t)(g_begin + min(i / 2, groups - 1)) * (uint32_t)T::SEG + piece, rowb - 16u);
                    lds_dma16(second ? a.x : a.w, row_at[second ? d + ND / 2 : d] + k,
                              lds0 + (uint32_t)(i * (T::GROUP / 2) + 4096 * d + wave * 1024));
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < NH / 2 - 1; ++g) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    copy(g - NH / 2, p, d, std::false_type{});
                p = following(p);
            }
        }
#pragma unroll
        for (int d = 0; d < part_of(1); ++d)
            copy(-1, before, d, std::bool_constant<NT>{});
        wait_vmcnt<(NH - 4) * ND / 2 + part_of(1)>(); // group 0 has landed
    }
    barrier_only();
#pragma unroll
    for (int i = 0; i < NR; ++i)
        read_operand(now_at, 0, i, op[0]);

    // Group g of this part.  TAIL: the row's partial last group; nothing follows it.
    auto run_group = [&](int g, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        const int left = (int)((rowb - (uint32_t)(g_begin + g) * (uint32_t)T::SEG) >> 4); // pieces of a partial group
        const Place after = following(now_at);
        auto step = [&](auto sel) __attribute__((always_inline)) {
            constexpr int S = decltype(sel)::value;
            constexpr bool END = S == STEPS - 1;
            Operands &now = op[S & 1], &next = op[(S & 1) ^ 1];
            if constexpr (END && !TAIL) {
                // group g + 1 has landed: the halves behind it may be in flight
                wait_vmcnt<(NH - 4) * ND / 2>();
                __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): this wave's reads of group g
                barrier_only();
            }
            if constexpr (TAIL) { // pieces past the row: zero weights
                const bool in = 4 * (S >> 1) + 2 * h + (S & 1) < left;
#pragma unroll
                for (int i = 0; i < T::NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        now.a[i][e] = in ? now.a[i][e] : 0;
            }
            // The step's other work, one piece at a time between the MFMAs: the next step's
            // operands, then copies: those into the places of group g - 1, in the last step the
            // first ones into the places of g.
            constexpr int PART = END ? 0 : S + 1, C0 = part_of(PART), C1 = part_of(PART + 1);
            constexpr int READS = TAIL && END ? 0 : NR, SIDE = READS + (TAIL ? 0 : C1 - C0);
            auto side = [&](int i) __attribute__((always_inline)) {
                if (i < READS)
                    read_operand(END ? after : now_at, END ? 0 : S + 1, i, next);
                else
                    copy(END ? g : g - 1, END ? now_at : before, C0 + i - READS, std::bool_constant<NT>{});
            };
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int i = m / T::MB, k = m % T::MB;
                __builtin_amdgcn_sched_barrier(0);
                acc[i][k] = __builtin_amdgcn_mfma_i32_32x32x32_i8(now.a[i], now.b[k], acc[i][k], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int z = 0; z < SIDE; ++z)
                    if (z >= m * SIDE / NM && z < (m + 1) * SIDE / NM)
                        side(z);
            }
        };
        step(std::integral_constant<int, 0>{});
        if (TAIL && left <= 1)
            return; // (the same for the whole workgroup)
        step(std::integral_constant<int, 1>{});
        if constexpr (GS == 2) {
            if (TAIL && left <= 4)
                return;
            step(std::integral_constant<int, 2>{});
            if (TAIL && left <= 5)
                return;
            step(std::integral_constant<int, 3>{});
        }
        before = now_at;
        now_at = after;
    };
    // the part's last group is run as a tail where the row ends inside it
    const int full = rowb % T::SEG && g_end == row_groups ? groups - 1 : groups;
    for (int g = 0; g < full; ++g)
        run_group(g, std::false_type{});
    if (full < groups)
        run_group(full, std::true_type{});

    // The scales (and the bias) of the tile's rows and columns, for the epilogue.
    const bool raw = splits > 1;
    float tile_ws = 0.f, tile_bias = 0.f, tile_xs = 0.f;
    if (!raw) {
        if (tid < T::TN)
            tile_ws = a.ws[min(n0 + tid, N - 1)];
        if (a.bias && tid < T::TN)
            tile_bias = a.bias[min(n0 + tid, N - 1)];
        if (tid < T::TM)
            tile_xs = a.xs[min(m0 + tid, M - 1)];
    }
    wait_vmcnt<0>(); // copies past the end: none is in flight when their place is used again
    // Every wave has read its last operands (the barrier of the last group came before them, so
    // one more): the buffers become staging space.
    barrier_only();
    float *const sws = reinterpret_cast<float *>(smem), *const sb = sws + T::TN, *const sx = sb + T::TN;
    uint8_t *const stage = smem + T::SCALES + wave * T::WSTAGE;
    const int nw = n0 + 32 * T::NB * wn, mw = m0 + 32 * T::MB * wm;
    if (raw) {
        store_wave<T, DT_F32, true, false>(acc, part + (size_t)split * M * N, M, N, nw, mw, nullptr, nullptr, nullptr, stage);
        return;
    }
    if (tid < T::TN) {
        sws[tid] = tile_ws;
        sb[tid] = tile_bias;
    }
    if (tid < T::TM)
        sx[tid] = tile_xs;
    __syncthreads();
    const float *const pw = sws + 32 * T::NB * wn, *const pb = sb + 32 * T::NB * wn, *const px = sx + 32 * T::MB * wm;
    auto store = [&](auto biased) __attribute__((always_inline)) {
        constexpr bool B = decltype(biased)::value;
        if (a.ydt == DT_F32)
            store_wave<T, DT_F32, false, B>(acc, a.y, M, N, nw, mw, pw, pb, px, stage);
        else if (a.ydt == DT_F16)
            store_wave<T, DT_F16, false, B>(acc, a.y, M, N, nw, mw, pw, pb, px, stage);
        else
            store_wave<T, DT_BF16, false, B>(acc, a.y, M, N, nw, mw, pw, pb, px, stage);
    };
    if (a.bias)
        store(std::true_type{});
    else
        store(std::false_type{});
}

// y from the sum of the K parts; n4 = N / 4.  100 x 5376 in five parts 4.3 to 4.9 us (12 MB), in six 4.5 (all
// of them loaded at once instead of four at a time 4.5).
__global__ __launch_bounds__(256) void int8_sum_kernel(Int8GemmArgs a, const i32x4 *__restrict__ part, int64_t total4,
                                                       int n4, int splits)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total4)
        return;
    const int64_t m = i / n4;
    const int n = (int)(i - m * n4) * 4;
    const float4_t ws = *reinterpret_cast<const float4_t *>(a.ws + n);
    float4_t bias = {};
    if (a.bias)
        bias = *reinterpret_cast<const float4_t *>(a.bias + n);
    const float xs = a.xs[m];
    i32x4 v = part[i];
    constexpr int B = 4; // parts under way at a time
    for (int s0 = 1; s0 < splits; s0 += B) {
        i32x4 p[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            p[j] = part[(size_t)min(s0 + j, splits - 1) * total4 + i];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s0 + j < splits)
                v += p[j];
    }
    float4_t y = scaled4(v, xs, ws);
    if (a.bias)
        y += bias;
    store4(a.y, a.ydt, (size_t)i * 4, y);
}

hipError_t launch_sum(const Int8GemmArgs &a, const int *part, int M, int N, int splits, hipStream_t stream)
{
    const int64_t total4 = (int64_t)M * N / 4;
    hipLaunchKernelGGL(int8_sum_kernel, dim3((unsigned)((total4 + 255) / 256)), dim3(256), 0, stream, a,
                       reinterpret_cast<const i32x4 *>(part), total4, N / 4, splits);
    return hipGetLastError();
}

template <class T, bool NT = false>
hipError_t launch_tile(const Int8GemmArgs &a, int M, int N, int K, int splits, void *workspace, hipStream_t stream)
{
    auto kern = int8_tile_kernel<T, NT>;
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
    int *part = static_cast<int *>(workspace);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), (size_t)T::LDS, stream, a, part, M, N, K, tiles_m,
                       (int)tiles, splits, nxcd);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || splits == 1 ? e : launch_sum(a, part, M, N, splits, stream);
}

using TileL = Int8Tile<2, 4, 4, 2, 5>;  // 256 x 256
using TileW = Int8Tile<4, 2, 4, 2, 6>;  // 256 weight rows x 128 activation rows
using TileM = Int8Tile<2, 2, 2, 2, 9>;  // 128 x 128
using TileS = Int8Tile<2, 1, 2, 2, 10>; // 64 weight rows x 128 activation rows
using TileN = Int8Tile<2, 1, 1, 2, 11>; // 64 x 64

// ---- Choice ----------------------------------------------------------------
//
// The form and its K parts are the ones with the smallest estimate, in us, from what was measured
// (graph replays over copies larger than the caches, 5200 triples of a shape, a form and parts, M 1 to
// 2048, N x K of 512 x 512 to 65528 x 16384; profiles/int8_product_forms.txt):
//   tiles: rounds of 256 workgroups, each `start` and `per_k` a 1000 k of a part, the latter a third
//          less on an empty card, but at least the weights' bytes;
//   parts: their sum's launch and its bytes;
//   few rows: the weights' bytes and the staging of x by a CU's workgroups.
// On average the choice is 0.9 % slower than the best form and parts measured, at worst 21 % (2 x 28672
// x 8192, few rows 8 x 1 49 us, 4 x 1 40).  The 128 x 128 tile's bytes at 0.17, 0.18, 0.19, 0.20, 0.21 us a million: 1.3 %,
// 1.0, 0.9, 0.9, 1.0 on average, 30 % at worst, then 21.
enum class Path { Few, Large, Wide, Medium, Small, Narrow };

struct Plan {
    Path path;
    int splits; // Few: weight rows of a workgroup
};

// Waves that share rows and groups of rows of a workgroup.  us, 4 x 1, 8 x 1, 2 x 4: 1 x 1024 x 8192 5.3,
// 5.3, 6.5; 1 x 2048 x 2048 3.4, 4.1, 3.9; 1 x 5376 x 5376 8.3, 8.1, 7.4; 1 x 16384 x 5376 16.9, 16.2, 17.4;
// 1 x 43008 x 5376 38.9, 39.8, 41.4; 8 x 16384 x 5376 25.1, 24.4, 18.4.  Wide, 8 x 1 and 4 x 2: 16 x 2048 x 2048 4.4,
// 4.7; 13 x 5760 x 2880 7.5, 6.8; 13 x 43008 x 5376 51, 48.
struct FewForm {
    int waves, groups;
};
FewForm few_form(int64_t M, int64_t N, int64_t K)
{
    if (M > 8)
        return N <= 4096 ? FewForm{8, 1} : FewForm{4, 2};
    if (N <= 4096) // few workgroups: more waves of them
        return {4, 1};
    if (M <= 2 && N > 8192 && K >= 5120) // x is small enough for each workgroup of 8 rows to stage
        return {8, 1};
    return {2, 4};
}

struct TileCost {
    Path path;
    int tn, tm;
    float start, per_k, per_mb; // us a round, a round and 1000 k, a million bytes of weights
};
constexpr TileCost TILE_COSTS[] = {
    {Path::Large, TileL::TN, TileL::TM, 7.9f, 13.f, 0.24f},  {Path::Wide, TileW::TN, TileW::TM, 6.2f, 7.9f, 0.21f},
    {Path::Medium, TileM::TN, TileM::TM, 5.4f, 5.1f, 0.19f}, {Path::Small, TileS::TN, TileS::TM, 4.6f, 3.6f, 0.17f},
    {Path::Narrow, TileN::TN, TileN::TM, 3.4f, 2.4f, 0.17f},
};
constexpr int MOST_PARTS = 16, PART_K = 512; // parts, at most; k of a part, at least

// Weight rows of a workgroup of few rows: what its groups hold, at most as many that every CU gets the
// same number of them.
int few_block(int64_t M, int64_t N, int64_t K)
{
    const int most = few_form(M, N, K).groups * (M > 8 ? 16 : 8);
    for (int64_t per = 1;; ++per) {
        const int64_t rows = 8 * ((N + 2048 * per - 1) / (2048 * per));
        if (rows <= 32)
            return (int)std::min<int64_t>(rows, most);
    }
}

Plan plan(int64_t M, int64_t N, int64_t K)
{
    Plan best = {Path::Narrow, 1};
    float least = INFINITY;
    for (const TileCost &t : TILE_COSTS) {
        const int64_t tiles = ((M + t.tm - 1) / t.tm) * ((N + t.tn - 1) / t.tn);
        const int64_t most = std::min<int64_t>({256 / tiles, K / PART_K, MOST_PARTS});
        for (int64_t parts = 1; parts == 1 || parts <= most; ++parts) {
            const int64_t rounds = (tiles * parts + 255) / 256, k = (K + parts - 1) / parts;
            const float busy = (float)(tiles * parts) / (float)(256 * rounds);
            float us = (float)rounds * t.start + std::max((float)rounds * t.per_k * 1e-3f * (float)k * (0.65f + 0.35f * busy),
                                                          t.per_mb * 1e-6f * (float)(N * K));
            if (parts > 1)
                us += 1.8f + 0.33f * ((float)parts + 0.5f) * (float)(M * N) * 4e-6f;
            if (us < least) {
                least = us;
                best = {t.path, (int)parts};
            }
        }
    }
    if (M <= 16 && M * few_pitch((int)K) <= 80 * 1024) { // x leaves the LDS room for a second workgroup
        const int rows = few_block(M, N, K);
        const int64_t per_cu = ((N + rows - 1) / rows + 255) / 256;
        // (8 x 1 with many workgroups: the others hide it)
        const float stage = M <= 8 && rows == 8 && N > 8192 ? 0.005e-3f : 0.035e-3f;
        if (2.8f + 0.17e-6f * (float)(N * K) + stage * (float)(M * K * per_cu) < least)
            best = {Path::Few, rows};
    }
    return best;
}

// Weights of more than half of the last-level cache (256 MB) that one tile of activation rows reads are
// copied nontemporally.  us, ordinary and nontemporal, past the caches / three sets of weights: 32 x 43008
// x 5376 54.4, 50.8 / 53.3, 48.5; 100 x 43008 x 5376 65.1, 61.4 / 64.7, 61.5; but 64 x 16384 x 5376 23.7, 22.8 /
// 17.8, 21.4; 100 x 8192 x 5376 19.8, 21.3 / 17.2, 20.8; two tiles: 200 x 16384 x 5376 33.1, 34.7.
// The halves that fill the ring at the start are ordinary copies in every tile.  Past the caches, ordinary, all
// nontemporal, all but those: 64 x 64 tile 40 x 131072 x 4096 125.2, 117.3, 107.1, 64 x 26624 x 5376 40.1, 38.1, 36.9; 128 x
// 128 100 x 131072 x 4096 139.6, 133.9, 125.3, 100 x 262144 x 624 (lines that two groups share) 75.4, 90.7, 74.0; 64 x 128
// 100 x 131072 x 4096 152.3, 147.2, 139.4, 100 x 262144 x 624 98.4, 113.4, 97.4.
template <class T>
hipError_t launch_once(const Int8GemmArgs &a, int M, int N, int K, int splits, void *workspace, hipStream_t stream)
{
    return M <= T::TM && (int64_t)N * K > (int64_t)128 << 20 ? launch_tile<T, true>(a, M, N, K, splits, workspace, stream)
                                                             : launch_tile<T>(a, M, N, K, splits, workspace, stream);
}

} // namespace

size_t int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M == 0 || N == 0)
        return 0;
    const Plan p = plan(M, N, K);
    return p.path != Path::Few && p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(int) : 0;
}

hipError_t launch_int8_gemm(const Int8GemmArgs &a, int M, int N, int K, void *workspace, hipStream_t stream)
{
    const Plan p = plan(M, N, K);
    switch (p.path) {
    case Path::Few:
        switch (const FewForm f = few_form(M, N, K); 16 * f.waves + f.groups) {
        case 16 * 8 + 1:
            return M > 8 ? launch_few<8, 1, true>(a, M, N, K, p.splits, stream)
                         : launch_few<8, 1, false>(a, M, N, K, p.splits, stream);
        case 16 * 4 + 1:
            return launch_few<4, 1, false>(a, M, N, K, p.splits, stream);
        case 16 * 4 + 2:
            return launch_few<4, 2, true>(a, M, N, K, p.splits, stream);
        default:
            return launch_few<2, 4, false>(a, M, N, K, p.splits, stream);
        }
    case Path::Large:
        return launch_tile<TileL>(a, M, N, K, p.splits, workspace, stream);
    case Path::Wide:
        return launch_tile<TileW>(a, M, N, K, p.splits, workspace, stream);
    case Path::Medium:
        return launch_once<TileM>(a, M, N, K, p.splits, workspace, stream);
    case Path::Small:
        return launch_once<TileS>(a, M, N, K, p.splits, workspace, stream);
    default:
        return launch_once<TileN>(a, M, N, K, p.splits, workspace, stream);
    }
}

} // namespace wob
