// The choice of experts (moe_topk) and the whole mixture-of-experts layer.
#include "moe_choice.hpp"
#include "weight_only_bit.h"
#include "wob_internal.hpp"

#include <algorithm>

namespace wob {

namespace {

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int CH_THREADS = 256;

template <int DT, int L, int V>
__global__ __launch_bounds__(CH_THREADS) void moe_topk_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ ids,
    float *__restrict__ weights, int T, int E, int topk, bool renormalize)
{
    const int t = blockIdx.x * (CH_THREADS / L) + threadIdx.x / L, g = threadIdx.x % L;
    int id[CHOICE_MAX / L];
    float w[CHOICE_MAX / L];
    choose<L, V>(logits, DT, (int64_t)t * E, bias, t < T ? E : 0, topk, renormalize, g, id, w);
    if (t >= T)
        return;
#pragma unroll
    for (int j = 0; j < CHOICE_MAX / L; ++j)
        if (j * L + g < topk) {
            ids[(int64_t)t * topk + j * L + g] = id[j];
            weights[(int64_t)t * topk + j * L + g] = w[j];
        }
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
    hipLaunchKernelGGL((moe_topk_kernel<DT, L, V>), dim3((T + PER - 1) / PER), dim3(CH_THREADS), 0,
                       stream, logits, bias, ids, weights, T, E, topk, renormalize);
    return hipGetLastError();
}

// ---- The layer for a few tokens --------------------------------------------
//
// Bound by the bytes of the chosen experts' weights, each read once, in two
// kernels:
//
//  up:   a workgroup takes one expert and MU_COLS columns of it.  It makes the
//        choice of all tokens itself (its scores are a few KB in the cache;
//        a kernel of its own would cost a launch), lists the expert's tokens,
//        stages their rows of x in LDS, and streams the gate and up rows of its
//        columns: a wave owns 16 gate rows and the 16 up rows beside them, W = 4
//        waves share them and split K.  The activated and already weighted row
//            a[p] = weight_p * silu(gate) * up          (rounded once to bf16)
//        of each pair p = (token, place) goes to the workspace.
//  down: a workgroup takes 16 rows of W2 in every chosen expert, so that a token's
//        sum over its experts stays in one workgroup: no atomics, no third pass,
//        and the order of the sum is fixed.  Its 16 waves are 4 parts of K x 4
//        sets of experts.
//
// Both dequantise with v_cvt_scalef32_pk_bf16_fp4 into the A operand of
// v_mfma_f32_16x16x32_bf16 (lane (r, q) holds row r, block 4 j + q of the 128-k step
// j: word s of its 16 code bytes feeds MFMA s of the step) with the tokens as B
// columns: with one to a dozen tokens per expert the matrix unit does the work of
// 16 for the same cost, and the vector unit only dequantises.
constexpr int MU_W = 4, MU_G = 2; // up: waves of a group of rows, groups
constexpr int MU_COLS = 16 * MU_G, MU_THREADS = 64 * MU_W * MU_G;
constexpr int MU_D = 6;           // steps of a lane in flight
constexpr int MD_W = 4, MD_S = 4; // down: parts of K, sets of experts
constexpr int MD_WAVES = MD_W * MD_S, MD_THREADS = 64 * MD_WAVES;
constexpr int MF_TOKENS = 32;     // tokens, at most (a 16-lane group each in the up kernel)
constexpr int MF_PAIRS = 512;     // pairs, at most
constexpr int MF_EXPERTS = 256;   // experts, at most (16 scores a lane)
constexpr int MF_LDS = 64 * 1024;

// What the up kernel leaves for the down kernel: the pairs grouped by expert
// and one unit per expert and 16 of its pairs.
struct FewWs {
    int32_t *units;  // their number
    int4 *unit;      // {expert, first place in sorted, pairs, 0}
    int32_t *sorted; // pairs by expert
    uint16_t *a;     // [P][I]
};
size_t max_units(int64_t P) { return (size_t)P; } // every unit has a pair

FewWs carve_few(void *ws, int64_t P)
{
    uint8_t *b = static_cast<uint8_t *>(ws);
    FewWs w;
    w.units = reinterpret_cast<int32_t *>(b);
    w.unit = reinterpret_cast<int4 *>(b + 16);
    w.sorted = reinterpret_cast<int32_t *>(b + 16 + 16 * max_units(P));
    w.a = reinterpret_cast<uint16_t *>(b + round256(16 + 20 * max_units(P)));
    return w;
}
size_t few_bytes(int64_t P, int64_t I) { return round256(16 + 20 * max_units(P)) + 2 * (size_t)P * (size_t)I; }

// Bytes between staged rows of x: K rounded up to whole steps (zeros), 16 mod
// 128, which makes the operand reads conflict-free.
__host__ __device__ inline int up_pitch(int H) { return ((H + 127) & ~127) * 2 + 16; }
// Staged rows: at most 8, and as many as leave the LDS room for two workgroups.
inline size_t up_lds(int rows, int H, int P)
{
    const size_t staged = (size_t)rows * up_pitch(H) + (size_t)MU_G * 32 * (H >> 5);
    const size_t sums = (size_t)MU_G * MU_W * 2 * 1024;
    return ((std::max(staged, sums) + 15) & ~(size_t)15) + 12 * (size_t)P + 16;
}
inline int up_rows(int T, int H, int P)
{
    int rows = T > 4 ? 8 : T > 2 ? 4 : T;
    while (rows > 0 && up_lds(rows, H, P) > (size_t)MF_LDS)
        rows >>= 1;
    return rows;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// One 128-k step of 16 weight rows against the columns: word s of the lane's
// codes times the column's k = 32 b + 8 s .. + 7.
__device__ __forceinline__ void step16(const u32x4 &codes, float scale, const u32x4 (&x)[4], f32x4 &acc)
{
#pragma unroll
    for (int s = 0; s < 4; ++s)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bitcast<bf168_t>(fp4_word_bf16x8(codes[s], scale)),
                                                      bitcast<bf168_t>(x[s]), acc, 0, 0, 0);
}

struct UpArgs {
    const uint16_t *x;
    const void *logits;
    const float *bias;
    const uint8_t *w, *ws;
    FewWs out;
    int dt, T, topk, E, H, I, renormalize, slices, rows;
};

template <int V>
__global__ __launch_bounds__(MU_THREADS) void moe_up_kernel(const UpArgs p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), k = wave % MU_W, g = wave / MU_W;
    const int P = p.T * p.topk, KB = p.H >> 5, steps = (KB + 3) >> 2, pitch = up_pitch(p.H);
    const size_t staged = (size_t)p.rows * pitch + (size_t)MU_G * 32 * KB;
    const size_t sums = (size_t)MU_G * MU_W * 2 * 1024;
    int32_t *const sid = reinterpret_cast<int32_t *>(smem + ((max(staged, sums) + 15) & ~(size_t)15));
    float *const sw = reinterpret_cast<float *>(sid + P);
    int32_t *const list = sid + 2 * P, *const count = sid + 3 * P;
    const int slot = blockIdx.x / p.slices, slice = blockIdx.x - slot * p.slices;

    // The choice: 16 lanes a token.
    {
        const int t = tid >> 4, gl = tid & 15;
        int id[CHOICE_MAX / 16];
        float wt[CHOICE_MAX / 16];
        choose<16, V>(p.logits, p.dt, (int64_t)t * p.E, p.bias, t < p.T ? p.E : 0, p.topk,
                      p.renormalize != 0, gl, id, wt);
        if (t < p.T) {
#pragma unroll
            for (int j = 0; j < CHOICE_MAX / 16; ++j)
                if (16 * j + gl < p.topk) {
                    sid[t * p.topk + 16 * j + gl] = id[j];
                    sw[t * p.topk + 16 * j + gl] = wt[j];
                }
        }
        if (tid == 0)
            *count = 0;
    }
    __syncthreads();

    if (blockIdx.x == 0) {
        // The pairs by expert (then by pair) and the units of up to 16 of them, each
        // pair counting those before it; `list` holds a pair's rank in its expert.
        for (int i = tid; i < P; i += MU_THREADS) {
            int rank = 0;
            for (int j = 0; j < i; ++j)
                rank += sid[j] == sid[i];
            list[i] = rank;
        }
        __syncthreads();
        int units = 0;
        for (int i = tid; i < P; i += MU_THREADS) {
            const int e = sid[i], rank = list[i];
            if (e < 0)
                continue;
            int lower = 0, all = 0, u = rank / 16;
            for (int j = 0; j < P; ++j) {
                const int o = sid[j];
                const bool below = o >= 0 && o < e;
                lower += below;
                all += o == e;
                u += below && list[j] % 16 == 0;
            }
            p.out.sorted[lower + rank] = i;
            if (rank % 16 == 0) {
                p.out.unit[u] = int4{e, lower + rank, min(16, all - rank), 0};
                units = max(units, u + 1);
            }
        }
        if (units)
            atomicMax(count, units);
        __syncthreads();
        if (tid == 0) {
            *p.out.units = *count;
            *count = 0;
        }
        __syncthreads();
    }

    // This workgroup's expert: with at most as many experts as pairs the slot is
    // the expert, else the pair, and the first pair of an expert stands for it.
    const int e = p.E <= P ? slot : sid[slot];
    bool earlier = false;
    for (int i = tid; i < P; i += MU_THREADS) {
        if (e < 0 || sid[i] != e)
            continue;
        earlier |= i < slot;
        list[atomicAdd(count, 1)] = i; // (in any order: each pair's row is computed on its own)
    }
    const int again = __syncthreads_or(p.E > P && earlier);
    const int rows = *count;
    if (rows == 0 || again)
        return;

    // Weight rows: this lane's gate row and the up row beside it (I % 32 == 0
    // except for a last half slice: rows past it are clamped, not stored).
    const int c0 = slice * MU_COLS + 16 * g;
    const int gr = min(c0, p.I - 16) + r;
    const size_t er = (size_t)e * 2 * (size_t)p.I;
    const u32x4 *wg = reinterpret_cast<const u32x4 *>(p.w) + (er + gr) * (size_t)KB;
    const u32x4 *wu = wg + (size_t)p.I * KB;
    const int mine = 2 * (((steps + 1) / 2 - k + MU_W - 1) / MU_W); // neighbouring steps in pairs
    auto block = [&](int i) __attribute__((always_inline)) {
        return 4 * (2 * (k + MU_W * (i / 2)) + i % 2) + q;
    };
    u32x4 rg[MU_D], ru[MU_D];
    auto load = [&](int i, int d) __attribute__((always_inline)) {
        int b = min(block(i), KB - 1);
        asm volatile("" : "+v"(b));
        rg[d] = wg[b];
        ru[d] = wu[b];
    };
    uint8_t *const sl = smem + (size_t)p.rows * pitch; // scales: per group 16 gate, 16 up rows
    const int nv = pitch / 16, nx = p.H / 8;           // 16-byte units of a staged row, of x's

    for (int m0 = 0; m0 < rows; m0 += p.rows) {
        const int mr = min(p.rows, rows - m0);
        if (m0 > 0)
            __syncthreads(); // the previous pass's sums have been read
        auto x_unit = [&](int i) __attribute__((always_inline)) {
            const int m = i / nv, c = i - m * nv;
            u32x4 v{0, 0, 0, 0};
            if (c < nx)
                v = reinterpret_cast<const u32x4 *>(p.x + (size_t)(list[m0 + m] / p.topk) * p.H)[c];
            return v;
        };
        // rows of x and the scales are requested ahead of the codes and land first
        constexpr int XB = 2;
        u32x4 xv[XB];
#pragma unroll
        for (int b = 0; b < XB; ++b)
            xv[b] = x_unit(min(tid + b * MU_THREADS, mr * nv - 1));
        // 16 rows of scales are 16 KB bytes in a row, 16-byte aligned
        const int su = 2 * MU_G * KB; // 16-byte units
        auto s_unit = [&](int i) __attribute__((always_inline)) {
            const int part = i / KB, c = i - part * KB; // group, gate / up
            const size_t row = er + (size_t)(part & 1) * p.I + min(slice * MU_COLS + 16 * (part >> 1), p.I - 16);
            return reinterpret_cast<const u32x4 *>(p.ws + row * KB)[c];
        };
        const u32x4 sv = s_unit(min(tid, su - 1));
#pragma unroll
        for (int d = 0; d < MU_D; ++d)
            load(min(d, max(mine - 1, 0)), d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < XB; ++b)
            if (tid + b * MU_THREADS < mr * nv)
                reinterpret_cast<u32x4 *>(smem)[tid + b * MU_THREADS] = xv[b];
        if (tid < su)
            reinterpret_cast<u32x4 *>(sl)[tid] = sv;
        for (int i = tid + XB * MU_THREADS; i < mr * nv; i += MU_THREADS)
            reinterpret_cast<u32x4 *>(smem)[i] = x_unit(i);
        for (int i = tid + MU_THREADS; i < su; i += MU_THREADS)
            reinterpret_cast<u32x4 *>(sl)[i] = s_unit(i);
        __syncthreads();

        const uint8_t *xr = smem + (size_t)min(r, mr - 1) * pitch;
        const uint8_t *sg = sl + (size_t)(32 * g + r) * KB, *sup = sg + (size_t)16 * KB;
        f32x4 ag{0.f, 0.f, 0.f, 0.f}, au{0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](int i, int d) __attribute__((always_inline)) {
            const int b = block(i);
            const bool in = b < KB;
            const int bc = in ? b : KB - 1;
            // (past the row: zero codes under the row's own scale; x is zero there)
            u32x4 cg = rg[d], cu = ru[d], xo[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                cg[s] = in ? cg[s] : 0u;
                cu[s] = in ? cu[s] : 0u;
                xo[s] = *reinterpret_cast<const u32x4 *>(xr + 64 * min(b, 4 * steps - 1) + 16 * s);
            }
            step16(cg, e8m0_to_f32(sg[bc]), xo, ag);
            step16(cu, e8m0_to_f32(sup[bc]), xo, au);
        };
        int i = 0;
        for (; i + MU_D < mine; i += MU_D) {
#pragma unroll
            for (int d = 0; d < MU_D; ++d) {
                if (i + d < mine)
                    multiply(i + d, d);
                __builtin_amdgcn_sched_barrier(0);
                load(min(i + d + MU_D, mine - 1), d);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < MU_D; ++d)
            if (i + d < mine)
                multiply(i + d, d);

        // Sums over the parts of K in order; lane (r, q) holds columns 4 q + e of
        // row r of the pass.
        __syncthreads();
        f32x4 *part = reinterpret_cast<f32x4 *>(smem);
        part[(2 * wave + 0) * 64 + lane] = ag;
        part[(2 * wave + 1) * 64 + lane] = au;
        __syncthreads();
        if (k == 0) {
#pragma unroll
            for (int j = 1; j < MU_W; ++j) {
                ag += part[(2 * (wave + j) + 0) * 64 + lane];
                au += part[(2 * (wave + j) + 1) * 64 + lane];
            }
            const int n = c0 + 4 * q;
            if (r < mr && n < p.I) {
                const int pair = list[m0 + r];
                const float wt = sw[pair];
                float a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[j] = wt * (ag[j] / (1.0f + expf(-ag[j])) * au[j]);
                *reinterpret_cast<uint2 *>(p.out.a + (size_t)pair * p.I + n) =
                    uint2{f32x2_to_act2<DT_BF16>(a[0], a[1]), f32x2_to_act2<DT_BF16>(a[2], a[3])};
            }
        }
    }
}

struct DownArgs {
    const uint8_t *w, *ws;
    FewWs in;
    uint16_t *y;
    int T, topk, H, I, P;
};

// The down kernel's ring holds pairs of steps: two code loads, the eight scale
// bytes of the pair and the B operands of both steps.
struct DownSlot {
    u32x4 w[2], x[2][4];
    uint64_t s;
};
constexpr int MD_D = 2; // pairs of steps in flight

__global__ __launch_bounds__(MD_THREADS) void moe_down_kernel(const DownArgs p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), k = wave % MD_W, set = wave / MD_W;
    const int KB = p.I >> 5, h0 = blockIdx.x * 16;
    const int per = ((KB + 7) / 8 - k + MD_W - 1) / MD_W; // pairs of steps of this wave and unit
    float *const sums = reinterpret_cast<float *>(smem);  // [wave][T][16]
    float *const ys = sums + wave * p.T * 16;
    for (int i = lane; i < p.T * 16; i += 64)
        ys[i] = 0.f;
    const int units = *p.in.units;
    int4 *const table = reinterpret_cast<int4 *>(sums + MD_WAVES * p.T * 16);
    int32_t *const sorted = reinterpret_cast<int32_t *>(table + p.P);
    for (int i = tid; i < units; i += MD_THREADS)
        table[i] = p.in.unit[i];
    for (int i = tid; i < p.P; i += MD_THREADS)
        sorted[i] = p.in.sorted[i]; // (places behind the last pair with an expert are not used)
    __syncthreads();
    const int mine = set < units ? (units - set + MD_S - 1) / MD_S : 0;
    const int items = mine * per; // unit by unit
    const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
        p.in.a, 0, (int)((uint32_t)p.P * (uint32_t)p.I * 2u), 0x00020000);

    // The unit that loads are issued for, and the unit whose products are summed.
    struct Unit {
        int n, expert, pairs, pair; // number, its expert, pairs, this lane's pair
    };
    auto unit = [&](int n) __attribute__((always_inline)) {
        const int4 u = table[set + MD_S * min(n, mine - 1)];
        return Unit{n, u.x, u.z, sorted[u.y + min(r, u.z - 1)]};
    };
    DownSlot ring[MD_D];
    Unit lu, cu;
    int lc = 0, cc = 0; // pair of steps within the unit
    auto load = [&](DownSlot &s) __attribute__((always_inline)) {
        const size_t row = (size_t)lu.expert * p.H + h0 + r;
        const int b = 8 * (k + MD_W * lc);
        const u32x4 *w = reinterpret_cast<const u32x4 *>(p.w) + row * KB;
        const uint8_t *sc = p.ws + row * KB;
        __builtin_memcpy(&s.s, sc + min(b, KB - 8), 8); // the row's last eight where b + 8 > KB
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int bj = b + 4 * j + q;
            s.w[j] = w[min(bj, KB - 1)];
            // columns without a pair and blocks past the row read as zero
            const uint32_t at = r < lu.pairs && bj < KB
                                    ? ((uint32_t)lu.pair * (uint32_t)p.I + 32u * (uint32_t)bj) * 2u
                                    : 0xFFFFFF00u;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                s.x[j][t] = __builtin_amdgcn_raw_buffer_load_b128(rows, at + 16u * (uint32_t)t, 0, 0);
        }
        if (++lc == per) {
            lc = 0;
            lu = unit(lu.n + 1);
        }
    };
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const DownSlot &s) __attribute__((always_inline)) {
        const int b = 8 * (k + MD_W * cc);
        const uint64_t v = s.s >> (8 * max(b - (KB - 8), 0));
#pragma unroll
        for (int j = 0; j < 2; ++j)
            step16(s.w[j], e8m0_to_f32((uint32_t)(v >> (32 * j + 8 * q)) & 0xFFu), s.x[j], acc);
        if (++cc == per) {
            if (r < cu.pairs) { // this lane's token: rows 4 q .. + 3 of its outputs
                f32x4 *to = reinterpret_cast<f32x4 *>(ys + (cu.pair / p.topk) * 16) + q;
                *to += acc;
            }
            acc = f32x4{0.f, 0.f, 0.f, 0.f};
            cc = 0;
            cu = unit(cu.n + 1);
        }
    };
    if (items > 0) {
        lu = cu = unit(0);
#pragma unroll
        for (int d = 0; d < MD_D; ++d)
            load(ring[d]);
        int i = 0;
        for (; i + MD_D <= items; i += MD_D) {
#pragma unroll
            for (int d = 0; d < MD_D; ++d) {
                multiply(ring[d]);
                __builtin_amdgcn_sched_barrier(0);
                load(ring[d]); // past the last item: the last unit's again
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < MD_D; ++d)
            if (i + d < items)
                multiply(ring[d]);
    }
    __syncthreads();
    for (int i = tid; i < p.T * 16; i += MD_THREADS) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < MD_WAVES; ++j)
            v += sums[j * p.T * 16 + i];
        p.y[(size_t)(i >> 4) * p.H + h0 + (i & 15)] = f32_to_act<DT_BF16>(v);
    }
}

// Whether the two kernels above take the layer: their scores, tables and staged
// rows fit, and a row of W2 has the eight scale bytes that one load takes.
bool layer_few(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    return T <= MF_TOKENS && T * topk <= MF_PAIRS && E <= MF_EXPERTS && I >= 256 && H <= 32768 &&
           up_rows((int)T, (int)H, (int)(T * topk)) > 0;
}

hipError_t launch_layer_few(const MoeLayerArgs &a, void *workspace, hipStream_t stream)
{
    const int P = a.T * a.topk;
    UpArgs u;
    u.x = static_cast<const uint16_t *>(a.x);
    u.logits = a.logits;
    u.bias = a.bias;
    u.w = a.w1;
    u.ws = a.w1s;
    u.out = carve_few(workspace, P);
    u.dt = a.logits_dt;
    u.T = a.T;
    u.topk = a.topk;
    u.E = a.E;
    u.H = a.H;
    u.I = a.I;
    u.renormalize = a.renormalize;
    u.slices = (a.I + MU_COLS - 1) / MU_COLS;
    u.rows = up_rows(a.T, a.H, P);
    const size_t lds = up_lds(u.rows, a.H, P);
    const unsigned grid = (unsigned)(std::min(a.E, P) * u.slices);
    if (a.E <= 32)
        hipLaunchKernelGGL(moe_up_kernel<2>, dim3(grid), dim3(MU_THREADS), lds, stream, u);
    else
        hipLaunchKernelGGL(moe_up_kernel<16>, dim3(grid), dim3(MU_THREADS), lds, stream, u);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    DownArgs d;
    d.w = a.w2;
    d.ws = a.w2s;
    d.in = u.out;
    d.y = static_cast<uint16_t *>(a.y);
    d.T = a.T;
    d.topk = a.topk;
    d.H = a.H;
    d.I = a.I;
    d.P = P;
    hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(a.H / 16)), dim3(MD_THREADS),
                       (size_t)MD_WAVES * a.T * 64 + (size_t)P * 20, stream, d);
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
        return few_bytes(T * topk, I);
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
