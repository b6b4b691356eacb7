// The choice of experts (moe_topk) and the whole mixture-of-experts layer.
#include "moe_choice.hpp"
#include "weight_only_bit.h"
#include "wob_internal.hpp"

#include <algorithm>

namespace wob {

namespace {

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int CH_THREADS = 256;

template <int DT, int L, int V, bool QUAD>
__global__ __launch_bounds__(CH_THREADS) void moe_topk_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ ids,
    float *__restrict__ weights, int T, int E, int topk, bool renormalize)
{
    const int t = blockIdx.x * (CH_THREADS / L) + threadIdx.x / L, g = threadIdx.x % L;
    choose<L, V, QUAD>(logits, DT, (int64_t)t * E, bias, t < T ? E : 0, topk, renormalize, g,
                 [&](int place, int id, float w) {
                     if (t < T) {
                         ids[(int64_t)t * topk + place] = id;
                         weights[(int64_t)t * topk + place] = w;
                     }
                 });
}

template <int DT, int L, int V>
hipError_t launch_topk_v(const void *logits, const float *bias, int32_t *ids, float *weights, int T,
                         int E, int topk, bool renormalize, hipStream_t stream)
{
    // 16 lanes a token up to 256 experts, a whole wave beyond
    if (E > L * V) {
        if constexpr (L == 16 && V < 16)
            return launch_topk_v<DT, 16, 2 * V>(logits, bias, ids, weights, T, E, topk, renormalize,
                                                stream);
        else if constexpr (L == 16)
            return launch_topk_v<DT, 64, 8>(logits, bias, ids, weights, T, E, topk, renormalize,
                                            stream);
        else if constexpr (V < 64)
            return launch_topk_v<DT, 64, 2 * V>(logits, bias, ids, weights, T, E, topk, renormalize,
                                                stream);
    }
    constexpr int PER = CH_THREADS / L; // tokens per workgroup
    const dim3 grid((unsigned)((T + PER - 1) / PER));
    if constexpr (V % 4 == 0) {
        if (E % 4 == 0) {
            hipLaunchKernelGGL((moe_topk_kernel<DT, L, V, true>), grid, dim3(CH_THREADS), 0, stream, logits,
                               bias, ids, weights, T, E, topk, renormalize);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((moe_topk_kernel<DT, L, V, false>), grid, dim3(CH_THREADS), 0, stream, logits, bias,
                       ids, weights, T, E, topk, renormalize);
    return hipGetLastError();
}

// ---- The layer for a few tokens --------------------------------------------
//
// Bound by the bytes of the chosen experts' weights, read once a unit.  The pairs
// p = (token, place) are grouped into units of up to 8 pairs of one expert;
//
//  route: one workgroup makes the choice and writes the units (one token: the up
//         kernel does it itself, since its pairs are its units);
//  up:    a[p] = weight_p * silu(gate) * up, rounded once to bf16, the operand type of the
//         second product's instructions (with the rounding of y the result is off by
//         2.3e-3 of its 2-norm, where y alone rounded is by 1.7e-3);
//  down:  the rows pre[p] = W2 a[p] in fp32;
//  join:  y[t] = the sum of its pairs' rows, in order of places.
//
// (For the fewest tokens down and join are one kernel, see moe_token_down_kernel.)
//
// Up and down are one kernel: a workgroup takes one unit and G groups of 16
// weight rows (up: 16 gate rows and the 16 up rows beside them); W waves share a
// group and split K.  Every load that the workgroup needs for its first 128 W SPW
// elements of K is under way as soon as the unit's entry is known.  Many short
// workgroups with few registers (64: 32 waves a CU) took 105 us for 32 tokens where
// long ones that stream several units through a ring of registers took 145 to 160
// (each unit then waits for a whole memory round trip: too few waves to hide it).
// 32 experts, top 4, H = I = 2880, graph replay over three copies, us for 1 / 4 / 8 /
// 16 / 32 tokens, with down by units and join throughout:
//   W = 8, G = 1, SPW = 3    20.1 / 47.5 / 69.9 / 92.9 / 121
//   W = 4, G = 2, SPW = 3    21.7 / 50.7 / 71.2 / 90.8 / 105
//   W = 8, G = 2, SPW = 3    23.1 / 55.7 / 77.7 / 97.6 / 115
//   W = 12, G = 1, SPW = 2   24.8 / 60.3 / - / - / 145
// (plain reads of the weights alone: 9 / 26 / 42 / 55 / 61).  The narrow form has
// twice the workgroups, each with its own copy of the rows: better until the rows
// weigh.
//
// Codes are dequantised with v_cvt_scalef32_pk_bf16_fp4 into the A operand of
// v_mfma_f32_16x16x32_bf16 (lane (r, q) holds row r, block 4 j + q of the 128-k step
// j: word s of its 16 code bytes feeds MFMA s of the step) with the unit's pairs as
// B columns, their rows staged in LDS.
constexpr int FE_NARROW = 8;    // tokens with W = 8, G = 1, at most; more: W = 4, G = 2
constexpr int FE_UNIT = 8;      // pairs of a unit, at most
constexpr int MF_TOKENS = 64;   // tokens, at most: 16 lanes each in the choice
constexpr int MF_PAIRS = 512;   // pairs, at most: the lists' room
constexpr int MF_EXPERTS = 256; // experts, at most: 16 scores a lane
constexpr int RT_THREADS = 1024;
constexpr size_t FEW_LDS = 150 * 1024; // of a workgroup, at most, besides its lists
static_assert(RT_THREADS / 16 >= MF_TOKENS, "every token has its lanes");

struct alignas(16) FewUnit {
    int32_t expert, pairs, pad[2];
    uint16_t pair[FE_UNIT];
    float weight[FE_UNIT];
};

struct FewWs {
    int32_t *units;  // their number
    int32_t *ids;    // [P] the chosen experts
    FewUnit *unit;   // [P]: every unit has a pair
    uint16_t *a;     // [P][I]
    float *pre;      // [P][H]
};

size_t few_a_at(int64_t P) { return round256(16 + (4 + sizeof(FewUnit)) * (size_t)P); }
size_t few_pre_at(int64_t P, int64_t I) { return few_a_at(P) + round256(2 * (size_t)P * (size_t)I); }
size_t few_bytes(int64_t P, int64_t H, int64_t I) { return few_pre_at(P, I) + 4 * (size_t)P * (size_t)H; }

FewWs carve_few(void *ws, int64_t P, int64_t I)
{
    uint8_t *b = static_cast<uint8_t *>(ws);
    FewWs w;
    w.units = reinterpret_cast<int32_t *>(b);
    w.unit = reinterpret_cast<FewUnit *>(b + 16);
    w.ids = reinterpret_cast<int32_t *>(b + 16 + sizeof(FewUnit) * (size_t)P);
    w.a = reinterpret_cast<uint16_t *>(b + few_a_at(P));
    w.pre = reinterpret_cast<float *>(b + few_pre_at(P, I));
    return w;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct FewArgs {
    const uint16_t *x;
    const void *logits;
    const float *bias;
    const uint8_t *w, *ws; // up: [E][2I][H/2] and scales; down: [E][H][I/2]
    FewWs f;
    uint16_t *y;
    int dt, T, topk, E, H, I, renormalize;
    int K, N, slices; // this kernel's row length, output columns and workgroups per unit
};

// The choice of all tokens and the units, in order of experts.  A wave lists an
// expert's pairs by ballots over the pairs.
template <int V>
__global__ __launch_bounds__(RT_THREADS) void moe_few_route_kernel(const FewArgs p)
{
    __shared__ int32_t sid[MF_PAIRS], hits[MF_EXPERTS], first[MF_EXPERTS];
    __shared__ float sw[MF_PAIRS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, P = p.T * p.topk;
    for (int e = tid; e < p.E; e += RT_THREADS)
        hits[e] = 0;
    __syncthreads();
    const int t = tid >> 4, g = tid & 15;
    choose<16, V, false>(p.logits, p.dt, (int64_t)t * p.E, p.bias, t < p.T ? p.E : 0, p.topk,
                  p.renormalize != 0, g, [&](int place, int id, float w) {
                      if (t < p.T) {
                          const int i = t * p.topk + place;
                          sid[i] = id;
                          sw[i] = w;
                          p.f.ids[i] = id;
                          if (id >= 0)
                              atomicAdd(&hits[id], 1);
                      }
                  });
    __syncthreads();
    if (wave == 0) { // units before each expert's
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const int e = e0 + lane, mine = e < p.E ? (hits[e] + FE_UNIT - 1) / FE_UNIT : 0;
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d);
                upto += lane >= d ? o : 0;
            }
            if (e < p.E)
                first[e] = n + upto - mine;
            n += __shfl(upto, 63);
        }
        if (lane == 0)
            *p.f.units = n;
    }
    __syncthreads();
    for (int e = wave; e < p.E; e += RT_THREADS / 64) {
        const int c = hits[e];
        if (c == 0)
            continue;
        for (int u = lane; u * FE_UNIT < c; u += 64) {
            p.f.unit[first[e] + u].expert = e;
            p.f.unit[first[e] + u].pairs = min(FE_UNIT, c - u * FE_UNIT);
        }
        int rank = 0;
        for (int i0 = 0; i0 < P; i0 += 64) {
            const bool hit = i0 + lane < P && sid[i0 + lane] == e;
            const uint64_t mask = __ballot(hit);
            const int at = rank + __popcll(mask & (((uint64_t)1 << lane) - 1));
            if (hit) {
                FewUnit &u = p.f.unit[first[e] + at / FE_UNIT];
                u.pair[at % FE_UNIT] = (uint16_t)(i0 + lane);
                u.weight[at % FE_UNIT] = sw[i0 + lane];
            }
            rank += __popcll(mask);
        }
    }
}

// Bytes between staged rows, 16 mod 128, which makes the operand reads conflict-free
// (K % 64 == 0).  Token by token the rows are rounded up to whole steps; in units each
// has at least one block of zeros behind it, which is what blocks past the row read.
__host__ __device__ inline int few_pitch(int K) { return ((K + 127) & ~127) * 2 + 16; }
__host__ __device__ inline int unit_pitch(int K) { return 2 * K + 144; }
__host__ __device__ inline int few_rows(int T) { return T < FE_UNIT ? T : FE_UNIT; } // a unit's pairs have different tokens
template <bool UP, int W, int G>
size_t few_lds(int T, int K)
{
    const size_t staged = (size_t)few_rows(T) * unit_pitch(K) + (size_t)G * (UP ? 32 : 16) * (K >> 5);
    const size_t sums = (size_t)G * W * (UP ? 2 : 1) * 1024;
    return (std::max(staged, sums) + 15) & ~(size_t)15;
}

// One 128-k step of 16 weight rows against the columns: word s of the lane's
// codes times the column's k = 32 b + 8 s .. + 7.
__device__ __forceinline__ void step16(const u32x4 &codes, float scale, const u32x4 (&x)[4], f32x4 &acc)
{
#pragma unroll
    for (int s = 0; s < 4; ++s)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bitcast<bf168_t>(fp4_word_bf16x8(codes[s], scale)),
                                                      bitcast<bf168_t>(x[s]), acc, 0, 0, 0);
}

// UP: gate and up rows, rows of x, activated rows of a; else rows of W2, rows of
// a, fp32 rows of pre.  ONE: one token, and the choice made here (UP).
template <bool UP, bool ONE, int V, int W, int G, int SPW>
__global__ __launch_bounds__(64 * W * G, 8) void moe_few_kernel(const FewArgs p)
{
    constexpr int NT = 64 * W * G;
    constexpr int NR = UP ? 2 : 1; // 16-row operands of a group
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), k = wave % W, g = wave / W;
    const int KB = p.K >> 5, steps = (KB + 3) >> 2, pitch = unit_pitch(p.K);
    const int un = blockIdx.x / p.slices, slice = blockIdx.x - un * p.slices;

    int e, pairs;
    __shared__ int32_t pair_of[FE_UNIT], row_of[FE_UNIT]; // pairs, their rows of the input
    __shared__ float weight_of[FE_UNIT];
    if constexpr (ONE) {
        // places with an expert come first, so place i is unit i
        __shared__ int32_t id[CHOICE_MAX];
        __shared__ float wt[CHOICE_MAX];
        if (wave == 0)
            choose<16, V, false>(p.logits, p.dt, 0, p.bias, lane < 16 ? p.E : 0, p.topk, p.renormalize != 0,
                          lane & 15, [&](int place, int c, float w) {
                              if (lane < 16) {
                                  id[place] = c;
                                  wt[place] = w;
                              }
                          });
        __syncthreads();
        if (blockIdx.x == 0) {
            int n = 0;
            for (int i = 0; i < p.topk; ++i)
                n += id[i] >= 0;
            if (tid == 0)
                *p.f.units = n;
            if (tid < p.topk) {
                p.f.ids[tid] = id[tid];
                FewUnit u;
                u.expert = id[tid];
                u.pairs = 1;
                u.pair[0] = (uint16_t)tid;
                p.f.unit[tid] = u;
            }
        }
        e = __builtin_amdgcn_readfirstlane(id[un]);
        if (e < 0)
            return;
        pairs = 1;
        if (tid == 0) {
            pair_of[0] = un;
            row_of[0] = 0;
            weight_of[0] = wt[un];
        }
    } else {
        // the unit's entry is requested with the number of units, not after it (it is
        // in the table, but holds nothing past the last unit)
        const FewUnit *u = p.f.unit + un;
        const int units = *p.f.units, expert = u->expert, n = u->pairs;
        const int pair = u->pair[tid & (FE_UNIT - 1)];
        const float weight = u->weight[tid & (FE_UNIT - 1)];
        if (un >= units)
            return;
        e = __builtin_amdgcn_readfirstlane(expert);
        pairs = __builtin_amdgcn_readfirstlane(n);
        if (tid < pairs) {
            pair_of[tid] = pair;
            row_of[tid] = UP ? pair / p.topk : pair;
            weight_of[tid] = weight;
        }
    }

    // Codes: scalar bases, 32-bit lane offsets.
    const int c0 = (slice * G + g) * 16;  // this group's columns (may lie past the last)
    const int cc = min(c0, p.N - 16);
    const size_t row = (size_t)e * NR * p.N + cc;
    const uint8_t *const w0 = p.w + row * (size_t)KB * 16, *const w1 = w0 + (size_t)p.N * KB * 16;
    const int rounds = (steps + W * SPW - 1) / (W * SPW);
    auto block = [&](int round, int j) __attribute__((always_inline)) { // this lane's
        return 4 * ((round * W + k) * SPW + j) + q;
    };
    u32x4 c[NR][SPW];
    auto load = [&](int round) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            const uint32_t at = 16u * (uint32_t)(r * KB + min(block(round, j), KB - 1));
            c[0][j] = *reinterpret_cast<const u32x4 *>(w0 + at);
            if constexpr (UP)
                c[1][j] = *reinterpret_cast<const u32x4 *>(w1 + at);
        }
    };
    load(0);
    // Scale bytes: the 16 rows of an operand are KB 16-byte units in a row.
    uint8_t *const sl = smem + (size_t)few_rows(p.T) * pitch;
    const int su = NR * G * KB;
    auto scale_unit = [&](int i) __attribute__((always_inline)) {
        const int op = i / KB, at = i - op * KB, n = min((slice * G + op / NR) * 16, p.N - 16);
        return reinterpret_cast<const u32x4 *>(
            p.ws + ((size_t)e * NR * p.N + (size_t)(op % NR) * p.N + n) * KB)[at];
    };
    const u32x4 sv = scale_unit(min(tid, su - 1));
    __syncthreads(); // the pairs are listed
    const int nv = pitch / 16, nx = p.K / 8; // 16-byte units of a staged row, of a row
    const uint16_t *const rows = UP ? p.x : p.f.a;
    auto x_unit = [&](int i) __attribute__((always_inline)) {
        const int m = i / nv, at = i - m * nv;
        u32x4 v{0, 0, 0, 0};
        if (at < nx)
            v = reinterpret_cast<const u32x4 *>(rows + (size_t)row_of[m] * p.K)[at];
        return v;
    };
    constexpr int XB = 2; // units of a thread under way at a time
    for (int i0 = tid; i0 < pairs * nv; i0 += XB * NT) {
        u32x4 v[XB];
#pragma unroll
        for (int i = 0; i < XB; ++i)
            v[i] = x_unit(min(i0 + i * NT, pairs * nv - 1));
#pragma unroll
        for (int i = 0; i < XB; ++i)
            if (i0 + i * NT < pairs * nv)
                reinterpret_cast<u32x4 *>(smem)[i0 + i * NT] = v[i];
    }
    if (tid < su)
        reinterpret_cast<u32x4 *>(sl)[tid] = sv;
    for (int i = tid + NT; i < su; i += NT)
        reinterpret_cast<u32x4 *>(sl)[i] = scale_unit(i);
    __syncthreads();

    const uint8_t *const xr = smem + (size_t)min(r, pairs - 1) * pitch;
    const uint8_t *const sr = sl + (size_t)(NR * 16 * g + r) * KB;
    f32x4 acc[NR];
#pragma unroll
    for (int o = 0; o < NR; ++o)
        acc[o] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int round = 0; round < rounds; ++round) {
        if (round > 0)
            load(round);
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            // (past the row: zero codes under one of the row's own scale bytes, so a NaN
            // there is the row's result anyway, and the zeros behind the staged row, not
            // the row, which may hold an infinity: 0 x infinity is NaN)
            const int b = block(round, j), bc = min(b, KB - 1), bx = min(b, KB);
            u32x4 x[4];
#pragma unroll
            for (int s = 0; s < 4; ++s)
                x[s] = *reinterpret_cast<const u32x4 *>(xr + 64 * bx + 16 * s);
#pragma unroll
            for (int o = 0; o < NR; ++o) {
                u32x4 v = c[o][j];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    v[s] = b < KB ? v[s] : 0u;
                step16(v, e8m0_to_f32(sr[o * 16 * KB + bc]), x, acc[o]);
            }
        }
    }

    // The waves' sums in order of K; lane (r, q) holds columns 4 q + i of pair r.
    __syncthreads();
    f32x4 *const part = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int o = 0; o < NR; ++o)
        part[(wave * NR + o) * 64 + lane] = acc[o];
    __syncthreads();
    if (k != 0 || r >= pairs || c0 >= p.N)
        return;
#pragma unroll
    for (int o = 0; o < NR; ++o)
        for (int j = 1; j < W; ++j)
            acc[o] += part[((wave + j) * NR + o) * 64 + lane];
    const int pair = pair_of[r];
    const size_t to = (size_t)pair * p.N + c0 + 4 * q;
    if constexpr (UP) {
        const float wt = weight_of[r];
        float a[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a[j] = wt * (acc[0][j] / (1.0f + expf(-acc[0][j])) * acc[NR - 1][j]);
        *reinterpret_cast<uint2 *>(p.f.a + to) =
            uint2{f32x2_to_act2<DT_BF16>(a[0], a[1]), f32x2_to_act2<DT_BF16>(a[2], a[3])};
    } else {
        *reinterpret_cast<f32x4 *>(p.f.pre + to) = acc[0];
    }
}

// Up to 4 tokens, and up to 8 with rows of up to 2048, in place of down and join: y[t][c .. c + 15] =
// the sum of W2_e a[p] over the token's places, by one workgroup of W waves; the places'
// rows laid end to end are one long K.  An expert of two tokens is read twice, most of it
// from caches; the fp32 rows and a launch go.  The layer in us, this and the other way:
//   32 experts, top 4, H = I = 2880            T = 1 17.5 / 19.8, 4 45.4 / 47.3, 6 62.2 / 60.4, 8 71.0 / 69.2
//   64 experts, top 8, H = 2048, I = 1408      T = 1 19.9 / 22.7, 4 41.3 / 48.8, 8 57.9 / 65.8, 12 73.2 / 68.8
//   8 experts, top 2, H = 4096, I = 1792       T = 1 13.7 / 16.3, 4 24.4 / 27.3, 8 36.7 / 36.7
//   128 experts, top 8, H = 4096, I = 1536     T = 4 77.6 / 93.0, 8 142 / 164, 16 196 / 183
//   4 experts, top 4 (all of them), 2880       T = 4 27.2 / 24.2
// One token has 16 waves (eight: 18.8 for the first), more have eight (T = 4 of the
// third: 16 waves 27.0); six steps of a wave at a time instead of two 18.3 for the first.
constexpr int TD_SPW = 2; // steps of a wave at a time

size_t token_down_lds(int topk, int K) { return (size_t)topk * (few_pitch(K) + (K >> 5) * 16); }

template <bool ONE, int W>
__global__ __launch_bounds__(64 * W) void moe_token_down_kernel(const FewArgs p)
{
    constexpr int SPW = TD_SPW, NT = 64 * W;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[W * 16];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int k = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int KB = p.K >> 5, steps = (KB + 3) >> 2, pitch = few_pitch(p.K), c0 = blockIdx.x * 16;
    const int32_t *const ids = p.f.ids + blockIdx.y * p.topk; // this token's
    const uint16_t *const rows = p.f.a + (size_t)blockIdx.y * p.topk * p.K;

    // Staged: all places' rows (those without an expert hold anything and are not used).
    const int nv = pitch / 16, nx = p.K / 8, rows16 = p.topk * nv, su = p.topk * KB;
    auto a_unit = [&](int i) __attribute__((always_inline)) {
        const int m = i / nv, at = i - m * nv;
        u32x4 v{0, 0, 0, 0};
        if (at < nx)
            v = reinterpret_cast<const u32x4 *>(rows + (size_t)m * p.K)[at];
        return v;
    };
    auto scale_unit = [&](int i) __attribute__((always_inline)) {
        const int m = i / KB, e = max(ids[m], 0);
        return reinterpret_cast<const u32x4 *>(p.ws + ((size_t)e * p.N + c0) * KB)[i - m * KB];
    };
    constexpr int XB = 2; // units of a thread under way at a time
    u32x4 av[XB];
#pragma unroll
    for (int i = 0; i < XB; ++i)
        av[i] = a_unit(min(tid + i * NT, rows16 - 1));
    const u32x4 sv = scale_unit(min(tid, su - 1));
    // places with an expert: the first ones (of one token: its units, a scalar load)
    const int total =
        steps * (ONE ? *p.f.units
                     : __popcll(__ballot(lane < p.topk && ids[min(lane, p.topk - 1)] >= 0)));

    u32x4 c[SPW];
    auto load = [&](int round) __attribute__((always_inline)) {
        const int i0 = (round * W + k) * SPW;
        int place = i0 / steps, at = i0 - place * steps;
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            const int e = max(ids[min(place, p.topk - 1)], 0);
            const uint8_t *base = p.w + ((size_t)e * p.N + c0) * KB * 16;
            c[j] = *reinterpret_cast<const u32x4 *>(base + 16u * (uint32_t)(r * KB + min(4 * at + q, KB - 1)));
            if (++at == steps) {
                at = 0;
                ++place;
            }
        }
    };
    load(0);

#pragma unroll
    for (int i = 0; i < XB; ++i)
        if (tid + i * NT < rows16)
            reinterpret_cast<u32x4 *>(smem)[tid + i * NT] = av[i];
    for (int i = tid + XB * NT; i < rows16; i += NT)
        reinterpret_cast<u32x4 *>(smem)[i] = a_unit(i);
    uint8_t *const sl = smem + (size_t)p.topk * pitch;
    if (tid < su)
        reinterpret_cast<u32x4 *>(sl)[tid] = sv;
    for (int i = tid + NT; i < su; i += NT)
        reinterpret_cast<u32x4 *>(sl)[i] = scale_unit(i);
    __syncthreads();

    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    for (int round = 0; round * W * SPW < total; ++round) {
        if (round > 0)
            load(round);
        const int i0 = (round * W + k) * SPW;
        int place = i0 / steps, at = i0 - place * steps;
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            if (i0 + j < total) {
                const int b = 4 * at + q;
                const uint8_t *const xr = smem + (size_t)place * pitch + 64 * b;
                u32x4 x[4], v = c[j];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    x[s] = *reinterpret_cast<const u32x4 *>(xr + 16 * s);
                    v[s] = b < KB ? v[s] : 0u;
                }
                step16(v, e8m0_to_f32(sl[(size_t)(place * 16 + r) * KB + min(b, KB - 1)]), x, acc);
            }
            if (++at == steps) {
                at = 0;
                ++place;
            }
        }
    }
    // the waves' sums in order of K; every column of the instruction is the token's
    if (r == 0)
        *reinterpret_cast<f32x4 *>(part + k * 16 + 4 * q) = acc;
    __syncthreads();
    if (tid < 16) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += part[w * 16 + tid];
        p.y[(size_t)blockIdx.y * p.N + c0 + tid] = (uint16_t)f32x2_to_act2<DT_BF16>(v, v);
    }
}

// y[t][h .. h + 3] = the sum of token t's rows of pre, in order of places.
__global__ __launch_bounds__(256) void moe_few_join_kernel(const float *__restrict__ pre,
                                                           const int32_t *__restrict__ ids,
                                                           uint16_t *__restrict__ y, int topk, int H)
{
    const int t = blockIdx.y, h = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (h >= H)
        return;
    f32x4 v{0.f, 0.f, 0.f, 0.f};
    const int32_t *const id = ids + t * topk;
    const float *const row = pre + (size_t)t * topk * H + h;
    constexpr int B = 8; // places under way at a time (a place without an expert has no row: not added)
    for (int s0 = 0; s0 < topk; s0 += B) {
        f32x4 a[B];
        bool on[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int s = min(s0 + i, topk - 1);
            a[i] = *reinterpret_cast<const f32x4 *>(row + (size_t)s * H);
            on[i] = s0 + i < topk && id[s] >= 0;
        }
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (on[i])
                v += a[i];
    }
    *reinterpret_cast<uint2 *>(y + (size_t)t * H + h) =
        uint2{f32x2_to_act2<DT_BF16>(v[0], v[1]), f32x2_to_act2<DT_BF16>(v[2], v[3])};
}

// Whether the kernels above take the layer: their lists and the staged rows fit, and
// there are few pairs.  Up to 8 tokens an expert's pairs are one unit, so its weights are
// read once.  With more an expert of c pairs has them read (most of it from caches)
// ceil(c / 8) times, where the tile kernels of the two stages read them once and take
// 32 rows at a time; and rows that leave a CU room for fewer than three workgroups
// make each unit slower.  us, here / by the stages (graph replay):
//   H x I         E   pairs: us
//   2880 x 2880   4   128: 55 / 91   256: 82 / 95
//                 8   256: 96 / 97   320: 105 / 100   384: 126 / 99   512: 148 / 102
//                16   256: 110 / 127   320: 130 / 126   384: 145 / 126   512: 172 / 137
//                32   256: 137 / 164   320: 149 / 169   384: 172 / 168   512: 207 / 170
//                64   320: 213 / 311   512: 276 / 312
//   2048 x 1408  64   384: 106 / 115   512: 126 / 118;   128   512: 169 / 193
//   2048 x 768   32   384: 60 / 49;   64   384: 76 / 78;   128   512: 118 / 113
//   4096 x 1792   8    64: 47 / 65   128: 63 / 67   256: 96 / 76
//                16   256: 111 / 75;   32   256: 140 / 127;   64   256: 199 / 217   384: 231 / 220
//   5120 x 2048  16    64: 88 / 93   128: 113 / 94
//   7168 x 2048   8    64: 79 / 94;   64   128: 344 / 386   256: 411 / 400   512: 575 / 406
//   2048 x 7168  32   128: 205 / 228
//   8192 x 3584   8    32: 116 / 124    64: 150 / 127
bool layer_few(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    const int64_t P = T * topk;
    if (T > MF_TOKENS || P > MF_PAIRS || E > MF_EXPERTS || H > 32768 || I > 32768)
        return false;
    const size_t lds = std::max(few_lds<true, 4, 2>((int)T, (int)H), few_lds<false, 4, 2>((int)T, (int)I));
    if (lds > FEW_LDS)
        return false;
    return T <= FE_UNIT || P <= (3 * lds <= 160 * 1024 ? std::max<int64_t>(256, 10 * E) : std::max<int64_t>(96, 4 * E));
}

template <bool UP, bool ONE, int V, int W, int G, int SPW>
hipError_t launch_few_as(FewArgs a, hipStream_t stream)
{
    auto kern = moe_few_kernel<UP, ONE, V, W, G, SPW>;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), FEW_LDS, lds_set);
        e != hipSuccess)
        return e;
    // units: at most one for every pair, one for every expert and FE_UNIT of its pairs
    const int P = a.T * a.topk, units = std::min(P, a.E * ((a.T + FE_UNIT - 1) / FE_UNIT));
    a.slices = (a.N + 16 * G - 1) / (16 * G);
    const size_t lds = few_lds<UP, W, G>(a.T, a.K);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units * a.slices)), dim3(64 * W * G), lds, stream, a);
    return hipGetLastError();
}

// Steps of a wave at a time: two where those cover K, so that no wave is left without any
// (8 tokens, 64 experts, top 6, H = 2048, I = 2880: 75.3 us, with three 83.8).
template <bool UP, bool ONE, int V, int W, int G>
hipError_t launch_few_steps(const FewArgs &a, hipStream_t stream)
{
    if (a.K <= 2 * W * 128)
        return launch_few_as<UP, ONE, V, W, G, 2>(a, stream);
    return launch_few_as<UP, ONE, V, W, G, 3>(a, stream);
}

template <bool UP, bool ONE, int V>
hipError_t launch_few(const FewArgs &a, hipStream_t stream)
{
    if constexpr (!ONE)
        if (a.T > FE_NARROW)
            return launch_few_steps<UP, false, V, 4, 2>(a, stream);
    return launch_few_steps<UP, ONE, V, 8, 1>(a, stream);
}

// Whether the second product is made token by token.
bool token_down(int T, int topk, int I)
{
    return (T <= 4 || (T <= 8 && I <= 2048)) && token_down_lds(topk, I) <= FEW_LDS;
}

template <bool ONE, int W>
hipError_t launch_token_down(const FewArgs &a, hipStream_t stream)
{
    auto kern = moe_token_down_kernel<ONE, W>;
    static std::atomic<uint64_t> lds_set{0};
    if (const hipError_t e = lds_optin(reinterpret_cast<const void *>(kern), FEW_LDS, lds_set);
        e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(a.N / 16), (unsigned)a.T), dim3(64 * W),
                       token_down_lds(a.topk, a.K), stream, a);
    return hipGetLastError();
}

hipError_t launch_layer_few(const MoeLayerArgs &m, void *workspace, hipStream_t stream)
{
    FewArgs a;
    a.x = static_cast<const uint16_t *>(m.x);
    a.logits = m.logits;
    a.bias = m.bias;
    a.f = carve_few(workspace, m.T * m.topk, m.I);
    a.y = static_cast<uint16_t *>(m.y);
    a.dt = m.logits_dt;
    a.T = m.T;
    a.topk = m.topk;
    a.E = m.E;
    a.H = m.H;
    a.I = m.I;
    a.renormalize = m.renormalize;
    hipError_t e = hipSuccess;
    if (m.T > 1) {
        if (m.E <= 32)
            hipLaunchKernelGGL(moe_few_route_kernel<2>, dim3(1), dim3(RT_THREADS), 0, stream, a);
        else
            hipLaunchKernelGGL(moe_few_route_kernel<16>, dim3(1), dim3(RT_THREADS), 0, stream, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    a.w = m.w1;
    a.ws = m.w1s;
    a.K = m.H;
    a.N = m.I;
    if (m.T > 1)
        e = launch_few<true, false, 1>(a, stream);
    else if (m.E <= 32)
        e = launch_few<true, true, 2>(a, stream);
    else
        e = launch_few<true, true, 16>(a, stream);
    if (e != hipSuccess)
        return e;
    a.w = m.w2;
    a.ws = m.w2s;
    a.K = m.I;
    a.N = m.H;
    if (token_down(m.T, m.topk, m.I))
        return m.T == 1 ? launch_token_down<true, 16>(a, stream) : launch_token_down<false, 8>(a, stream);
    e = launch_few<false, false, 1>(a, stream);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(moe_few_join_kernel, dim3((unsigned)((m.H + 1023) / 1024), (unsigned)m.T), dim3(256), 0,
                       stream, a.f.pre, a.f.ids, a.y, m.topk, m.H);
    return hipGetLastError();
}

// ---- The layer ---------------------------------------------------------------

// Workspace of the layer for more tokens: the choice, the activated rows of
// stage 1, then the stages' own scratch.
struct LayerWs {
    int32_t *ids;
    float *weights;
    uint16_t *a;
    uint8_t *stage;
};

size_t layer_rows_at(int64_t P) { return 2 * round256(4 * (size_t)P); }
size_t layer_stage_at(int64_t P, int64_t I)
{
    return layer_rows_at(P) + round256(2 * (size_t)P * (size_t)I);
}

LayerWs carve_layer(void *ws, int64_t P, int64_t I)
{
    uint8_t *b = static_cast<uint8_t *>(ws);
    LayerWs w;
    w.ids = reinterpret_cast<int32_t *>(b);
    w.weights = reinterpret_cast<float *>(b + round256(4 * (size_t)P));
    w.a = reinterpret_cast<uint16_t *>(b + layer_rows_at(P));
    w.stage = b + layer_stage_at(P, I);
    return w;
}

} // namespace

hipError_t launch_moe_topk(const void *logits, int dt, const float *bias, int32_t *ids,
                           float *weights, int T, int E, int topk, bool renormalize,
                           hipStream_t stream)
{
    if (dt == DT_F16)
        return launch_topk_v<DT_F16, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize, stream);
    if (dt == DT_BF16)
        return launch_topk_v<DT_BF16, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize,
                                         stream);
    return launch_topk_v<DT_F32, 16, 1>(logits, bias, ids, weights, T, E, topk, renormalize, stream);
}

size_t moe_layer_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    if (layer_few(T, topk, E, H, I))
        return few_bytes(T * topk, H, I);
    return layer_stage_at(T * topk, I) + moe_stage2_workspace_bytes(T, topk, E, H);
}

hipError_t launch_mxfp4_moe_layer(const MoeLayerArgs &a, void *workspace, hipStream_t stream)
{
    if (layer_few(a.T, a.topk, a.E, a.H, a.I))
        return launch_layer_few(a, workspace, stream);
    const LayerWs w = carve_layer(workspace, (int64_t)a.T * a.topk, a.I);
    hipError_t e = launch_moe_topk(a.logits, a.logits_dt, a.bias, w.ids, w.weights, a.T, a.E, a.topk,
                                   a.renormalize, stream);
    if (e != hipSuccess)
        return e;
    e = launch_mxfp4_moe(a.x, w.ids, a.w1, a.w1s, w.a, a.T, a.topk, a.E, 2 * a.I, a.H,
                         WOB_ACT_SILU_MUL, 32, w.stage, stream);
    if (e != hipSuccess)
        return e;
    return launch_mxfp4_moe_stage2(w.a, w.ids, w.weights, a.w2, a.w2s, a.y, a.T, a.topk, a.E, a.H,
                                   a.I, w.stage, stream);
}

} // namespace wob
