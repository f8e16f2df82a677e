// Products of 8-bit codes with one scale per activation row and one per weight
// row: out[m, n] = a_scale[m] * w_scale[n] * sum_k a[m, k] * w[n, k].  The sum
// is a 32-bit integer and exact (K < 131072), so its order does not matter;
// the two scales are applied in fp32 and the result rounded once.
//
// moe_linear_i8 is the dense form.  The experts' FFNs run over the row blocks of
// moe_route: gate/up with SwiGLU into fp32 h, a row-wise quantisation of h, and
// down; the shared expert's rows are dense row blocks in front of the routed ones.
//
// An MFMA operand is a 16 x 64 tile: lane l holds row l % 16, K 16*(l/16) .. +15,
// 16 bytes, for the weights (A operand) and the activations (B operand) alike.
// Weights in tiles (moe_i8_prepack) are read in that order; the rows of
// activations, and of a large dense product both operands, go through LDS.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_lds.h"
#include "moe_lora.h"

namespace moeq4 {

// D = A(16x64) * B(64x16) + C.  Lane l supplies A[l%16][16*(l/16) .. +16] and
// B[16*(l/16) .. +16][l%16]; it holds D[4*(l/16) + i][l%16], i = 0..3.
__device__ __forceinline__ i32x4_t mfma_i8(i32x4_t a, i32x4_t b, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// One part of a launch: the dense rows (the shared expert's, or a linear's) or
// the routed rows.
struct PartI8 {
    const int8_t* a;
    const float* a_scale;
    I8MatDev w, w2;         // w2: the up matrices of gate/up
    int M, N, K;            // M: rows of a dense part
    void* out;              // bf16, or fp32 h of gate/up
    int8_t* low;            // low bytes of a bf16 out (low_byte), or NULL
};

struct ProductArgs {
    PartI8 dense, routed;
    int dense_blocks, dense_tiles, routed_tiles;
    int dense_wgs, k;
    const int32_t* block_expert;
    const int32_t* block_row;
    const int32_t* offsets;
    const int32_t* n_blocks;
    const int32_t* sorted_assign;   // gate/up: row -> assignment
};

// Shares of the row blocks among the XCDs that have one column tile in common.
__host__ __device__ constexpr int xcd_shares(int tiles) { return tiles == 2 || tiles == 4 ? 8 / tiles : 1; }

// ---- Dense product of few tiles: a workgroup per 16 x 16 tile, K split over its 8 waves,
// each with kFewAhead steps of 64 K in flight straight from memory; the waves' integer sums
// meet in LDS.  Bound by the latency of one round of loads.
constexpr int kFewWaves = 8, kFewAhead = 8;

// The adapters' part of MF x NF pieces by K-splitting waves, behind the product's first loads: each wave
// takes every eighth step of ranks of every adapter among 16 rows, two of them at a time.
template <int MF, int NF>
__device__ __forceinline__ void few_lora(const LoraDev& l, int M, int N, int m0, int n0, int wave,
                                         f32x4_t (&v)[MF][NF]) {
    const int lane = __lane_id();
    int of[MF];
    unsigned long long left[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
#pragma unroll
        for (int n = 0; n < NF; ++n) v[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        of[m] = lora_of(l, m0 + m * 16 + lane % 16, M);
        left[m] = __ballot(of[m] >= 0);
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        int j = 0, step = l.steps, turn = 0;   // the item at hand: a step of adapter j
        // this wave's next item, false when there is none
        auto next = [&](int& at_j, int& at_step) {
            for (;;) {
                if (step == l.steps) {
                    if (!left[m]) return false;
                    j = __builtin_amdgcn_readlane(of[m], __builtin_ctzll(left[m]));
                    left[m] &= ~__ballot(of[m] == j);
                    step = 0;
                }
                at_j = j;
                at_step = step++;
                if (turn++ % kFewWaves == wave) return true;
            }
        };
        for (;;) {
            int j0 = 0, j1 = 0, t0 = 0, t1 = 0;
            if (!next(j0, t0)) break;
            const bool two = next(j1, t1);
            if (!two) {
                j1 = j0;
                t1 = t0;
            }
            const u32x4_t u0 = lora_u(l, m0 / 16 + m, t0, lane), u1 = lora_u(l, m0 / 16 + m, t1, lane);
            u32x4_t b0[NF], b1[NF];
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                b0[n] = lora_b(l, j0, N, n0 + n * 16, t0, lane);
                b1[n] = lora_b(l, j1, N, n0 + n * 16, t1, lane);
            }
            // lanes 32 .. 63 multiply what u's rounding left
            uint32_t infinite = 0;
#pragma unroll
            for (int n = 0; n < NF; ++n) infinite |= lora_infinite(b0[n]) | lora_infinite(b1[n]);
            if (__builtin_expect(lane >= 32 && infinite, 0)) {
#pragma unroll
                for (int n = 0; n < NF; ++n) {
                    b0[n] = lora_without(b0[n], 0);
                    b1[n] = lora_without(b1[n], 0);
                }
            }
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                lora_add(b0[n], u0, of[m] == j0, v[m][n]);
                lora_add(b1[n], u1, two && of[m] == j1, v[m][n]);
            }
        }
    }
}

// LORA: the rows' adapters are added in fp32, before the one rounding.
template <bool LORA>
__global__ __launch_bounds__(kFewWaves* WAVE) void linear_few_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, int M, int K, I8MatDev w, int N,
    uint16_t* __restrict__ out, LoraDev lora) {
    __shared__ i32x4_t s_part[kFewWaves - 1][WAVE];
    __shared__ f32x4_t s_lora[LORA ? kFewWaves : 1][WAVE];
    const int lane = threadIdx.x % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int n_tiles = (N + 15) / 16;
    const int m0 = blockIdx.x / n_tiles * 16, n0 = blockIdx.x % n_tiles * 16;
    // rows behind the last read the last; their results go nowhere
    const int row = row_at<LORA>(lora, m0 + lane % 16, M);
    const int8_t* pa = a + (size_t)row * K + lane / 16 * 16;
    const int8_t* pw = w.codes + (size_t)n0 * K +
                       (w.tiles ? (size_t)lane * 16
                                : (size_t)min(lane % 16, N - 1 - n0) * K + lane / 16 * 16);
    const int w_step = w.tiles ? 1024 : 64;
    const int steps = K / 64, s0 = steps * wave / kFewWaves, s1 = steps * (wave + 1) / kFewWaves;
    auto add_lora = [&]() {
        f32x4_t v[1][1];
        few_lora<1, 1>(lora, M, N, m0, n0, wave, v);
        s_lora[wave][lane] = v[0][0];
    };
    if constexpr (LORA)
        if (s0 == s1) add_lora();   // fewer steps than waves
    i32x4_t acc = {0, 0, 0, 0};
    for (int s = s0; s < s1; s += kFewAhead) {
        i32x4_t va[kFewAhead], vw[kFewAhead];
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i)
            if (s + i < s1) {
                vw[i] = *(const i32x4_t*)(pw + (size_t)(s + i) * w_step);
                va[i] = *(const i32x4_t*)(pa + (size_t)(s + i) * 64);
            }
        if constexpr (LORA)
            if (s == s0) add_lora();   // while the first loads are in flight
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i)
            if (s + i < s1) acc = mfma_i8(vw[i], va[i], acc);
    }
    if (wave) s_part[wave - 1][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 0; i < kFewWaves - 1; ++i) acc += s_part[i][lane];
    const int c = n0 + lane / 16 * 4;
    if (m0 + lane % 16 >= M || c >= N) return;
    const float as = a_scale[row];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)acc[i] * as * w.scales[min(c + i, N - 1)];
    if constexpr (LORA) {
        f32x4_t t = s_lora[0][lane];
#pragma unroll
        for (int i = 1; i < kFewWaves; ++i) t += s_lora[i][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += t[i];
    }
    uint16_t* o = out + (size_t)row * N + c;
    if (N % 4 == 0) {
        *(u32x2_t*)o = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < N) o[i] = (uint16_t)pack_bf16x2(v[i], 0.f);
    }
}

// ---- Dense product of some ten to some hundred rows: a workgroup per 16 MF x 16 NF tile, K
// split over its 8 waves as above, so every byte of a tile's rows goes once from the caches to
// registers, without LDS or barriers until the waves' sums meet.  A wave takes 128 K at a
// time, D of them ahead: the two halves of an activation row's cache line are requested one
// after the other, while the line is in L1 (64 K at a time and deeper 128x2048x7168 took
// 11.6 us, this 10.5; with contiguous rows it would take 7.8).  Bound by those half lines.
template <int MF, int NF, int D, bool LORA>
__global__ __launch_bounds__(kFewWaves* WAVE) void linear_split_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, int M, int K, I8MatDev w, int N,
    uint16_t* __restrict__ out, int n_tiles, LoraDev lora) {
    constexpr int W = kFewWaves, P = MF * NF, ROUND = P < W ? P : W;   // pieces of 16 x 16, and those joined at a time
    static_assert(P % ROUND == 0, "whole rounds");
    constexpr uint32_t kPast = 0xC0000000u;   // past every buffer (both are below 2^31 bytes)
    __shared__ i32x4_t s_part[W][ROUND][WAVE];
    __shared__ f32x4_t s_lora[LORA ? W : 1][LORA ? P : 1][WAVE];
    const int lane = threadIdx.x % WAVE, fr = lane % 16, fp = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int m0 = (int)(blockIdx.x / n_tiles) * MF * 16, n0 = (int)(blockIdx.x % n_tiles) * NF * 16;
    const buf_rsrc_t ra = make_buf(a, (uint32_t)M * (uint32_t)K);
    const buf_rsrc_t rw = make_buf(w.codes, (uint32_t)N * (uint32_t)K);
    const uint32_t w_step = w.tiles ? 1024u : 64u;
    uint32_t oa[MF], ow[NF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const uint32_t r = m0 + m * 16 + fr;
        oa[m] = r < (uint32_t)M ? (uint32_t)row_at<LORA>(lora, r, M) * (uint32_t)K + fp * 16 : kPast;
    }
#pragma unroll
    for (int n = 0; n < NF; ++n) {
        const uint32_t c = n0 + n * 16;
        ow[n] = w.tiles ? (c < (uint32_t)N ? c * (uint32_t)K + lane * 16 : kPast)
                        : (c + fr < (uint32_t)N ? (c + fr) * (uint32_t)K + fp * 16 : kPast);
    }
    const int steps = K / 64, pairs = (steps + 1) / 2, s0 = pairs * wave / W, s1 = pairs * (wave + 1) / W;
    i32x4_t va[D][2][MF], vw[D][2][NF];
    auto load = [&](int slot, int s) {
        const uint32_t past0 = s < s1 ? 0u : kPast, past1 = s < s1 && 2 * s + 1 < steps ? 0u : kPast;
#pragma unroll
        for (int n = 0; n < NF; ++n) {
            vw[slot][0][n] = __builtin_bit_cast(i32x4_t, buf_load16_u(rw, ow[n] | past0, (uint32_t)(2 * s) * w_step));
            vw[slot][1][n] = __builtin_bit_cast(i32x4_t, buf_load16_u(rw, ow[n] | past1, (uint32_t)(2 * s + 1) * w_step));
        }
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            va[slot][0][m] = __builtin_bit_cast(i32x4_t, buf_load16_u(ra, oa[m] | past0, (uint32_t)s * 128u));
            va[slot][1][m] = __builtin_bit_cast(i32x4_t, buf_load16_u(ra, oa[m] | past1, (uint32_t)s * 128u + 64u));
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, s0 + d);
    if constexpr (LORA) {
        f32x4_t v[MF][NF];
        few_lora<MF, NF>(lora, M, N, m0, n0, wave, v);
#pragma unroll
        for (int p = 0; p < P; ++p) s_lora[wave][p][lane] = v[p % MF][p / MF];
    }
    i32x4_t acc[NF][MF];
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[n][m] = i32x4_t{0, 0, 0, 0};
    for (int s = s0; s < s1; s += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m)
#pragma unroll
                    for (int q = 0; q < 2; ++q) acc[n][m] = mfma_i8(vw[d][q][n], va[d][q][m], acc[n][m]);
            load(d, s + d + D);
        }
    }
#pragma unroll
    for (int p0 = 0; p0 < P; p0 += ROUND) {
        if (p0) __syncthreads();
#pragma unroll
        for (int i = 0; i < ROUND; ++i) s_part[wave][i][lane] = acc[(p0 + i) / MF][(p0 + i) % MF];
        __syncthreads();
        if (wave < ROUND) {
            i32x4_t sum = s_part[0][wave][lane];
#pragma unroll
            for (int i = 1; i < W; ++i) sum += s_part[i][wave][lane];
            const int p = p0 + wave, r = m0 + p % MF * 16 + fr, c = n0 + p / MF * 16 + fp * 4;
            if (r < M && c < N) {
                const int row = row_at<LORA>(lora, r, M);
                const float as = a_scale[row];
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)sum[i] * as * w.scales[min(c + i, N - 1)];
                if constexpr (LORA) {
                    f32x4_t t = s_lora[0][p][lane];
#pragma unroll
                    for (int i = 1; i < W; ++i) t += s_lora[i][p][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += t[i];
                }
                uint16_t* o = out + (size_t)row * N + c;
                if (N % 4 == 0) {
                    *(u32x2_t*)o = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < N) o[i] = (uint16_t)pack_bf16x2(v[i], 0.f);
                }
            }
        }
    }
}

// ---- Dense product of many rows: tiles through LDS ----
// A workgroup of WM x WN waves owns a BM x BN tile; a wave WM-th of its rows and
// WN-th of its columns, MF x NF products of 16 x 16.  KS blocks of 64 K of both
// operands (one stage) go straight from memory into LDS, ST - 1 stages ahead of the
// one that is multiplied: a stage of the 256 x 256 tile is 1024 cycles of products,
// and a load takes two to four times that under full traffic.  Stages past K are
// zeros and multiplied like the others.  A stage keeps rows of 64 KS bytes, so that with
// KS 2 a load takes whole cache lines of 8 rows (half lines of 16 took 4 to 10 % longer
// from K 4096 on), and their 16-byte pieces permuted: place j of row r holds piece
// j ^ (r / 2 % (4 KS)), chosen on the source side (a load writes LDS in lane order), so
// that neighbouring rows of a fragment read lie in different banks (with r / 4 half of
// the LDS cycles were conflicts).  A workgroup requests its next tile's first stages
// during the last products of a tile.  8192 x 4096 x 4096 takes 120 us (2290 TOP/s), MFMA
// 56 % busy at 2.0 GHz; with codes of zero, at a higher clock, 92.  Where a CU has one tile
// or few it is bound by what L2 gives a CU, 40 to 48 bytes a ns in every form here.
// Waits count this wave's own loads (KS * (LA + LB) a stage): the kernel must not spill,
// which the build checks.
template <int WM, int MF, int WN, int NF, int ST, int KS, bool LORA>
__global__ __launch_bounds__(WM* WN* WAVE) void linear_tiles_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, int M, int K, I8MatDev w, int N,
    uint16_t* __restrict__ out, int m_tiles, int n_tiles, LoraDev lora) {
    constexpr int BM = WM * MF * 16, BN = WN * NF * 16, WAVES = WM * WN;
    constexpr int LA = BM / 16 / WAVES, LB = BN / 16 / WAVES;   // 1 KB loads per wave and block
    static_assert(BM / 16 % WAVES == 0 && BN / 16 % WAVES == 0, "whole loads per wave");
    constexpr uint32_t kPast = 0xC0000000u;   // past every buffer (both are below 2^31 bytes)
    // an array for each stage: loads into one would otherwise hold up reads of the others
#define MOE_STAGE(i) \
    __shared__ __attribute__((aligned(16))) int8_t s_a##i[ST > i ? BM * 64 * KS : 16], s_b##i[ST > i ? BN * 64 * KS : 16]
    MOE_STAGE(0);
    MOE_STAGE(1);
    MOE_STAGE(2);
    MOE_STAGE(3);
    MOE_STAGE(4);
    MOE_STAGE(5);
    MOE_STAGE(6);
    MOE_STAGE(7);
#undef MOE_STAGE
    static_assert(ST >= 4 && ST <= 8 && ST * KS % 2 == 0, "a stage for each array; fragments alternate");
    auto s_a = [&](int i) {
        return i == 0 ? s_a0 : i == 1 ? s_a1 : i == 2 ? s_a2 : i == 3 ? s_a3 : i == 4 ? s_a4 : i == 5 ? s_a5 : i == 6 ? s_a6 : s_a7;
    };
    auto s_b = [&](int i) {
        return i == 0 ? s_b0 : i == 1 ? s_b1 : i == 2 ? s_b2 : i == 3 ? s_b3 : i == 4 ? s_b4 : i == 5 ? s_b5 : i == 6 ? s_b6 : s_b7;
    };
    const int lane = threadIdx.x % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int wm = wave % WM, wn = wave / WM;
    // Workgroups go round the 8 XCDs in launch order; each XCD takes a contiguous share of
    // the tiles, in bands of 4 row tiles, so that its L2 holds what its tiles share, and
    // its workgroups go through that share.
    const int total = m_tiles * n_tiles;
    const int xcd = blockIdx.x % 8, stride = gridDim.x / 8;
    const int first = xcd * (total / 8) + min(xcd, total % 8);
    const int mine = total / 8 + (xcd < total % 8 ? 1 : 0);
    int in = blockIdx.x / 8;
    if (in >= mine) return;
    auto corner = [&](int i, int& m0, int& n0) {
        const int id = first + i;
        const int band = id / (4 * n_tiles), rest = id - band * 4 * n_tiles;
        const int rows_in = min(4, m_tiles - band * 4);
        m0 = (band * 4 + rest % rows_in) * BM;
        n0 = rest / rows_in * BN;
    };

    const buf_rsrc_t ra = make_buf(a, (uint32_t)M * (uint32_t)K);
    const buf_rsrc_t rb = make_buf(w.codes, (uint32_t)N * (uint32_t)K);
    // row and K piece of this lane's place in a load; the second load of 128 K holds rows 8 .. 15
    const int lr = lane / (4 * KS), piece = (lane % (4 * KS)) ^ (lr / 2 % 4);
    uint32_t va[LA][KS], vb[LB][KS];
    auto sources = [&](int m0, int n0) {
#pragma unroll
        for (int i = 0; i < LA; ++i)
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t r = m0 + (i * WAVES + wave) * 16 + lr + j * 8;
                va[i][j] = r < (uint32_t)M
                               ? (uint32_t)row_at<LORA>(lora, r, M) * (uint32_t)K + (piece ^ j * 4) * 16
                               : kPast;
            }
#pragma unroll
        for (int i = 0; i < LB; ++i)
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t r = n0 + (i * WAVES + wave) * 16 + lr + j * 8, p = piece ^ j * 4;
                vb[i][j] = r >= (uint32_t)N ? kPast
                           : w.tiles ? (r - r % 16) * (uint32_t)K + p / 4 * 1024 + p % 4 * 256 + r % 16 * 16
                                     : r * (uint32_t)K + p * 16;
            }
    };
    const int blocks = K / 64, steps = (blocks + KS - 1) / KS;
    const uint32_t b_step = (w.tiles ? 1024 : 64) * KS;
    // K behind the last block is zeros: the second half of 128, or all
    uint32_t half[KS];
#pragma unroll
    for (int j = 0; j < KS; ++j) half[j] = KS == 2 && (piece ^ j * 4) >= 4 ? kPast : 0u;
    auto load = [&](int st, int s) {
        const bool in = s * KS < blocks, whole = s * KS + KS <= blocks;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            const uint32_t past = whole ? 0u : in ? half[j] : kPast;
#pragma unroll
            for (int i = 0; i < LA; ++i)
                buf_to_lds16(ra, s_a(st) + ((i * WAVES + wave) * KS + j) * 1024, va[i][j] | past,
                             (uint32_t)s * (64u * KS));
#pragma unroll
            for (int i = 0; i < LB; ++i)
                buf_to_lds16(rb, s_b(st) + ((i * WAVES + wave) * KS + j) * 1024, vb[i][j] | past,
                             (uint32_t)s * b_step);
        }
    };
    i32x4_t acc[NF][MF];
    const int fr = lane % 16, fp = lane / 16;
    const int at = fr * 64 * KS + (fp ^ (fr / 2 % (4 * KS))) * 16;
    auto read_b = [&](int st, int q, int n) {
        return *(const i32x4_t*)(s_b(st) + (wn * NF + n) * 1024 * KS + (at ^ q * 64));
    };
    auto read_a = [&](int st, int q, int m) {
        return *(const i32x4_t*)(s_a(st) + (wm * MF + m) * 1024 * KS + (at ^ q * 64));
    };
    // While it multiplies a block a wave reads, in the order below, the row fragments it
    // lacks and the next block's columns and first FA row fragments, so that the products
    // go on at once behind a barrier: the next stage landed a barrier earlier.
    constexpr int FA = MF < 4 ? MF : 4;
    i32x4_t fb[2][NF], fa[2][FA];
    int m0, n0, m1 = 0, n1 = 0;
    corner(in, m0, n0);
    // the adapters of the tile's rows, and of this wave's row tiles
    constexpr int QL = (BM + WAVE - 1) / WAVE;
    int all[LORA ? QL : 1], of[LORA ? MF : 1];
    if constexpr (LORA) {
#pragma unroll
        for (int q = 0; q < QL; ++q) {
            const int j = lora_of(lora, m0 + q * WAVE + lane, M);
            all[q] = q * WAVE + lane < BM ? j : -1;
        }
#pragma unroll
        for (int m = 0; m < MF; ++m) of[m] = lora_of(lora, m0 + (wm * MF + m) * 16 + fr, M);
    }
    sources(m0, n0);
#pragma unroll
    for (int st = 0; st < ST - 1; ++st) load(st, st);
    wait_loads<(ST - 3) * KS * (LA + LB)>();
    bare_barrier_i8();
#pragma unroll
    for (int n = 0; n < NF; ++n) fb[0][n] = read_b(0, 0, n);
#pragma unroll
    for (int m = 0; m < FA; ++m) fa[0][m] = read_a(0, 0, m);
    const int rounds = (steps + ST - 1) / ST;
    for (;;) {
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int m = 0; m < MF; ++m) acc[n][m] = i32x4_t{0, 0, 0, 0};
        in += stride;
        const bool more = !LORA && in < mine;   // with adapters a workgroup has one tile
        if (more) corner(in, m1, n1);
        for (int round = 0; round < rounds; ++round) {
            int s = round * ST + ST - 1;   // stage that the step requests
#pragma unroll
            for (int st = 0; st < ST; ++st) {
                load((st + ST - 1) % ST, s + st);
                if (st == 0 && round == rounds - 1) {   // from here on the next tile's stages
                    if (more) sources(m1, n1);
                    s = more ? -1 : steps;   // no tile: zeros
                }
                __builtin_amdgcn_sched_barrier(0);   // the requests go out first
#pragma unroll
                for (int q = 0; q < KS; ++q) {
                    const int c = (st * KS + q) % 2;
                    const int nst = q + 1 < KS ? st : (st + 1) % ST, nq = (q + 1) % KS;
#pragma unroll
                    for (int m = 0; m < MF; ++m) {
                        const i32x4_t f = m < FA ? fa[c][m] : read_a(st, q, m);
#pragma unroll
                        for (int n = 0; n < NF; ++n) acc[n][m] = mfma_i8(fb[c][n], f, acc[n][m]);
                    }
#pragma unroll
                    for (int n = 0; n < NF; ++n) fb[1 - c][n] = read_b(nst, nq, n);
#pragma unroll
                    for (int m = 0; m < FA; ++m) fa[1 - c][m] = read_a(nst, nq, m);
                    constexpr int kRead = 0x100, kMul = 0x8;
#pragma unroll
                    for (int m = 0; m < MF; m += 2) {
                        if (m + 4 < MF) __builtin_amdgcn_sched_group_barrier(kRead, 2, 0);
                        else if (m + 2 >= MF) __builtin_amdgcn_sched_group_barrier(kRead, NF + FA, 0);
                        __builtin_amdgcn_sched_group_barrier(kMul, 2 * NF, 0);
                    }
                }
                wait_loads<(ST - 3) * KS * (LA + LB)>();
                bare_barrier_i8();
            }
        }
        // The tile's values.  Where rows of out start at 16 bytes they go through the wave's
        // share of the last stage (the next tile's stages lie in the others), 16 rows at a
        // time, so that a store covers whole 128-byte lines; a wave's LDS operations complete
        // in order, so no barrier is needed inside it.
        constexpr int kLdc = NF * 16 + 8;   // bf16 of a staged row, padded against bank conflicts
        constexpr int kHalf = WAVES / 2, kRows = 16;
        uint16_t* s_o = (uint16_t*)(wave < kHalf ? s_a(ST - 1) + wave * (BM * 64 * KS / kHalf)
                                                 : s_b(ST - 1) + (wave - kHalf) * (BN * 64 * KS / kHalf));
        static_assert(kRows * kLdc * 2 <= (BM < BN ? BM : BN) * 64 * KS / kHalf && kRows * NF * 2 % WAVE == 0,
                      "a wave's staged rows fit its share");
        const bool wide = N % 8 == 0;
        int rows[MF];
        float as[MF], ws[NF][4];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            rows[m] = row_at<LORA>(lora, m0 + (wm * MF + m) * 16 + fr, M);
            as[m] = a_scale[rows[m]];
        }
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ws[n][i] = w.scales[min(n0 + (wn * NF + n) * 16 + fp * 4 + i, N - 1)];
        // the tile's values, in the sums' registers
        auto value = [&](int n, int m) { return __builtin_bit_cast(f32x4_t, acc[n][m]); };
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                f32x4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)acc[n][m][i] * as[m] * ws[n][i];
                acc[n][m] = __builtin_bit_cast(i32x4_t, v);
            }
        bool infinite = false;   // whether a b of this wave's columns has an infinity or NaN
        if constexpr (LORA) {
            // One adapter after another among the tile's rows, ST steps of ranks at a time: its
            // columns, and once the rows' u, go through LDS, where the product's stages were.
            int here = lane;   // nothing of this is computed before the product's loop, which needs the registers
            asm volatile("" : "+v"(here));
            const int tiles_in = min(BM / 16, (M - m0 + 15) / 16), cols_in = min(BN, N - n0);
            const buf_rsrc_t ru = make_buf((const char*)lora.u + lora_u_at(m0 / 16, 0, lora.steps, 0),
                                           (uint32_t)lora_u_bytes(tiles_in, lora.steps));
            unsigned long long left[QL];
            for (int base = 0; base < lora.steps; base += ST) {
#pragma unroll
                for (int q = 0; q < QL; ++q) left[q] = __ballot(all[q] >= 0);
                bool first = true;
                for (;;) {
                    int j = -1;
#pragma unroll
                    for (int q = QL - 1; q >= 0; --q)
                        if (left[q]) j = __builtin_amdgcn_readlane(all[q], __builtin_ctzll(left[q]));
                    if (j < 0) break;
#pragma unroll
                    for (int q = 0; q < QL; ++q) left[q] &= ~__ballot(all[q] == j);
                    wait_loads<0>();
                    __syncthreads();   // what the stages held has been read
                    if (first) {
#pragma unroll
                        for (int st = 0; st < ST; ++st)
                            for (int t = wave; t < BM / 16; t += WAVES)
                                if (base + st < lora.steps)   // zeros for tiles behind the last row's
                                    buf_to_lds16(ru, s_a(st) + t * 1024,
                                                 (uint32_t)lora_u_at(t, base + st, lora.steps, here), 0);
                        first = false;
                    }
                    const buf_rsrc_t rl = make_buf(lora.b + ((size_t)j * N + n0) * lora.rank,
                                                   (uint32_t)(cols_in * lora.rank) * 2u);
#pragma unroll
                    for (int st = 0; st < ST; ++st)
                        for (int t = wave; t < BN / 32; t += WAVES) {   // 32 columns of 16 ranks
                            const int rr = (base + st) * 16 + here / 16 % 2 * 8;
                            const uint32_t c = t * 32 + here / 32 * 16 + here % 16;
                            if (base + st < lora.steps)
                                buf_to_lds16(rl, s_b(st) + t * 1024, rr < lora.rank ? (c * lora.rank + rr) * 2u : kPast, 0);
                        }
                    wait_loads<0>();
                    __syncthreads();
#pragma unroll
                    for (int st = 0; st < ST; ++st) {
                        if (base + st >= lora.steps) break;
                        u32x4_t b[NF], u[MF];
#pragma unroll
                        for (int n = 0; n < NF; ++n)
                            b[n] = *(const u32x4_t*)(s_b(st) + (wn * NF + n) * 512 + here % 32 * 16);
#pragma unroll
                        for (int m = 0; m < MF; ++m)
                            u[m] = *(const u32x4_t*)(s_a(st) + (wm * MF + m) * 1024 + here * 16);
                        uint32_t any = 0;
#pragma unroll
                        for (int n = 0; n < NF; ++n) any |= lora_infinite(b[n]);
                        if (__builtin_expect(__ballot(any) != 0, 0)) {   // as 1 and -1 here, the rest behind the stores
                            infinite = true;
#pragma unroll
                            for (int n = 0; n < NF; ++n) b[n] = lora_without(b[n], 0x3F80u);
                        }
#pragma unroll
                        for (int m = 0; m < MF; ++m) {
                            const bf16x8_t um = lora_only(of[m] == j, u[m]);
#pragma unroll
                            for (int n = 0; n < NF; ++n)
                                acc[n][m] = __builtin_bit_cast(
                                    i32x4_t, mfma_16x16x32(__builtin_bit_cast(bf16x8_t, b[n]), um, value(n, m)));
                        }
                    }
                }
            }
        }
        if constexpr (LORA) __syncthreads();   // the stores go through a stage
        // the stores' places are not those of the scales above: kept over the adapters they need registers
        if constexpr (LORA) asm volatile("" : "+s"(m0), "+s"(n0));
#pragma unroll
        for (int mb = 0; mb < MF; mb += kRows / 16) {
#pragma unroll
            for (int mi = 0; mi < kRows / 16; ++mi) {
                const int m = mb + mi, r = m0 + (wm * MF + m) * 16 + fr;
#pragma unroll
                for (int n = 0; n < NF; ++n) {
                    const int c = n0 + (wn * NF + n) * 16 + fp * 4;
                    const f32x4_t v = value(n, m);
                    const u32x2_t o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    if (wide) {
                        *(u32x2_t*)(s_o + (mi * 16 + fr) * kLdc + n * 16 + fp * 4) = o;
                    } else if (r < M) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + i < N) out[(size_t)rows[m] * N + c + i] = (uint16_t)(o[i / 2] >> 16 * (i % 2));
                    }
                }
            }
            if (wide) {
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < kRows * NF * 2 / WAVE; ++i) {
                    const int p = i * WAVE + lane, row = p / (NF * 2), c8 = p % (NF * 2) * 8;
                    const int r = m0 + (wm * MF + mb) * 16 + row, c = n0 + wn * NF * 16 + c8;
                    const int at = LORA ? __shfl(rows[mb], row, WAVE) : r;   // one row tile: kRows 16
                    if (r < M && c < N)
                        *(u32x4_t*)(out + (size_t)at * N + c) = *(const u32x4_t*)(s_o + row * kLdc + c8);
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
        if constexpr (LORA)
            if (__builtin_expect(infinite, 0))
                lora_add_infinite(lora, M, N, m0 + wm * MF * 16, MF * 16, n0 + wn * NF * 16, min(n0 + (wn + 1) * NF * 16, N), out);
        if (!more) break;
        m0 = m1;
        n0 = n1;
        // The staging place is the next request's.  Stores still in flight only make the
        // counted waits of the next tile stricter.
        bare_barrier_i8();
    }
    wait_loads<0>();
}

// ---- The experts' products with weights streamed into registers ----
// A workgroup of 4 waves owns BM = 16 MF rows of a block and 64 NT weight rows, a wave
// 16 NT of them (GATEUP: half the gate's, half the up's).  Each weight row is read once
// per block, so the weights go straight into registers, D steps of 64 K ahead, 64 KB
// and more in flight on a CU, which the latency of HBM under load (2 us and more)
// needs.  (Through an LDS ring as above 2048 tokens took 147 us for gate/up instead of
// 120; a variant without its products took as long.)  The rows' codes are shared by the
// waves: Q steps of 64 K at a time go straight into LDS, the next Q while these are
// multiplied, laid out as in the tile kernel; small chunks leave room for three
// workgroups on a CU, which cover each other's waits (Q = 8: two).  Bound by HBM: 541 MB
// of gate and up weights of 256 experts (512 tokens) in 100 us are 5.4 TB/s, of the 6.2 a
// plain read reaches.
template <int MF, int NT, int D, int Q, bool GATEUP>
__global__ __launch_bounds__(4 * WAVE, 2) void grouped_stream_kernel(ProductArgs p, uint32_t dense_rows,
                                                                     uint32_t routed_rows) {
    constexpr int BM = MF * 16, NW = GATEUP ? NT / 2 : NT, COLS = 4 * NW * 16;
    constexpr int LA = Q * MF / 4;   // 1 KB loads of a wave and chunk
    static_assert(Q % D == 0 && Q * MF % 4 == 0, "a slot for each step of a chunk, whole loads");
    constexpr uint32_t kPast = 0xC0000000u;
    constexpr int ES = GATEUP ? 4 : 2, ROW = NW * 16 * ES, STRIDE = ROW + 16;   // bytes of staged rows
    constexpr int A0 = Q * BM * 64, STAGE = 4 * 16 * STRIDE;
    __shared__ __attribute__((aligned(16))) int8_t s_a0[A0 > STAGE ? A0 : STAGE], s_a1[A0];
    __shared__ __attribute__((aligned(16))) float s_as[BM], s_ws[4][NT * 16];
    const int lane = threadIdx.x % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int dense_wgs = p.dense_wgs;
    const bool dense = (int)blockIdx.x < dense_wgs;
    const int id = dense ? blockIdx.x : blockIdx.x - dense_wgs;
    const int tiles = dense ? p.dense_tiles : p.routed_tiles;
    const PartI8& part = dense ? p.dense : p.routed;
    // Workgroups go round the 8 XCDs: with 8 column tiles, or a multiple, the blocks of an
    // expert meet its tile in one XCD's L2; with 2 or 4 an XCD takes a contiguous share of
    // the blocks besides.
    int block = id / tiles, tile = id - block * tiles;
    if (const int shares = xcd_shares(tiles); shares > 1) {
        const int n = dense ? p.dense_blocks : *p.n_blocks, per = (n + shares - 1) / shares;
        const int x = id % 8;
        tile = x % tiles;
        block = x / tiles * per + id / 8;
        if (id / 8 >= per || block >= n) return;
    }
    const int n0 = tile * COLS;
    int e = 0, row0 = block * BM, rows = part.M - row0;
    if (!dense) {
        e = p.block_expert[block];
        if (e < 0) return;
        row0 = p.block_row[block];
        rows = p.offsets[e + 1] - row0;
    }
    rows = min(rows, BM);
    const int K = part.K, N = part.N, blocks = K / 64;
    const size_t expert = (size_t)e * N * K;
    const buf_rsrc_t rg = make_buf(part.w.codes + expert, (uint32_t)N * (uint32_t)K);
    const buf_rsrc_t ru = make_buf(GATEUP ? part.w2.codes + expert : nullptr, (uint32_t)N * (uint32_t)K);
    const uint32_t w_step = part.w.tiles ? 1024u : 64u;
    uint32_t vw[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint32_t c = n0 + (wave * NW + n % NW) * 16;
        vw[n] = c >= (uint32_t)N ? kPast
                : part.w.tiles   ? c * (uint32_t)K + lane * 16
                                 : (c + lane % 16) * (uint32_t)K + lane / 16 * 16;
    }
    i32x4_t w[D][NT];
    auto load_w = [&](int slot, int s) {
        const uint32_t past = s < blocks ? 0u : kPast;   // steps behind the last are zeros
#pragma unroll
        for (int n = 0; n < NT; ++n)
            w[slot][n] = __builtin_bit_cast(
                i32x4_t, buf_load16_u(GATEUP && n >= NW ? ru : rg, vw[n] | past, (uint32_t)s * w_step));
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load_w(d, d);

    const buf_rsrc_t ra = make_buf(part.a, (dense ? dense_rows : routed_rows) * (uint32_t)K);
    const int lr = lane / 4, piece = (lane % 4) ^ (lr / 2 % 4);
    const int group = wave % MF;   // the 16 rows that this wave loads
    int src = row0 + min(group * 16 + lr, rows - 1);
    if (GATEUP && !dense) src = p.sorted_assign[src] / p.k;
    const uint32_t va = group * 16 + lr < rows ? (uint32_t)src * (uint32_t)K + piece * 16 : kPast;
    auto load_a = [&](int8_t* to, int chunk) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int q = (i * 4 + wave) / MF;
            const uint32_t k = (uint32_t)(chunk * Q + q);
            const uint32_t past = k < (uint32_t)blocks ? 0u : kPast;
            buf_to_lds16(ra, to + (q * MF + group) * 1024, va | past, k * 64u);
        }
    };
    const int fr = lane % 16, fp = lane / 16;
    const int at = fr * 64 + (fp ^ (fr / 2 % 4)) * 16;
    i32x4_t acc[NT][MF];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[n][m] = i32x4_t{0, 0, 0, 0};
    auto chunk_products = [&](const int8_t* sa, int8_t* other, int chunk) {
        load_a(other, chunk + 1);
        // Before this chunk's weights: the wait below counts on it.  All but vector memory
        // instructions may be moved across.
        __builtin_amdgcn_sched_barrier(0x38E);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            i32x4_t fa[MF];
#pragma unroll
            for (int m = 0; m < MF; ++m) fa[m] = *(const i32x4_t*)(sa + (q * MF + m) * 1024 + at);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m) acc[n][m] = mfma_i8(w[q % D][n], fa[m], acc[n][m]);
            load_w(q % D, chunk * Q + q + D);
        }
        // the next chunk's rows were requested before this chunk's weights: they have landed
        // once only the last D steps' weights are in flight
        wait_loads<D * NT>();
        bare_barrier_i8();
    };
    load_a(s_a0, 0);
    // The scales, so that nothing waits for memory behind the products (there each 16 rows'
    // waited for two dependent loads: 2048 tokens 123.5 -> 122 us, down 73.5 -> 71.8).
    const int col0 = n0 + wave * NW * 16;
    {
        const float as = part.a_scale[src];
        float ws = 0.f;
        if (lane < NT * 16 && col0 < N) {
            const float* scales = GATEUP && lane / 16 >= NW ? part.w2.scales : part.w.scales;
            ws = scales[(size_t)e * N + col0 + lane % (NW * 16)];
        }
        s_as[group * 16 + lr] = as;
        if (lane < NT * 16) s_ws[wave][lane] = ws;
    }
    wait_loads<0>();
    __syncthreads();
    const int chunks = (blocks + Q - 1) / Q;
    for (int c = 0; c < chunks; c += 2) {
        chunk_products(s_a0, s_a1, c);
        if (c + 1 < chunks) chunk_products(s_a1, s_a0, c + 1);
    }
    // The values, 16 rows of the wave at a time through its share of the LDS (the run-out
    // loads into it have landed), so that a store covers whole lines; a wave's LDS operations
    // complete in order, so no barrier is needed inside it.
    static_assert(16 * ROW / 16 % WAVE == 0, "whole stores");
    if (col0 >= N) return;   // N is a multiple of 64: the wave's columns are all in or all out
    int8_t* s_o = s_a0 + wave * 16 * STRIDE;
    // The low bytes likewise, through the other rows' place.  2048 skewed tokens: down 60.5 -> 70.6
    // us and the combine that reads them 15.2 -> 20.5; whole lines behind a barrier 69.8.
    constexpr int LSTRIDE = NW * 16 + 16;
    static_assert(GATEUP || 4 * 16 * LSTRIDE <= A0, "low bytes fit");
    int8_t* s_l = s_a1 + wave * 16 * LSTRIDE;
    const bool low = !GATEUP && part.low;
    f32x4_t ws[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) ws[n] = *(const f32x4_t*)(s_ws[wave] + n * 16 + fp * 4);
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const float as = s_as[m * 16 + fr];
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            f32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = (float)acc[n][m][i] * as * ws[n][i];
                if (GATEUP)
                    v[i] = silu_f32(v[i]) * ((float)acc[n + (GATEUP ? NW : 0)][m][i] * as * ws[n + (GATEUP ? NW : 0)][i]);
            }
            int8_t* to = s_o + fr * STRIDE + (n * 16 + fp * 4) * ES;
            if constexpr (GATEUP) {
                *(f32x4_t*)to = v;
            } else {
                const u32x2_t o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                *(u32x2_t*)to = o;
                if (low) {
                    uint32_t b = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        b |= (uint32_t)(low_byte(v[i], o[i / 2] >> 16 * (i % 2) & 0xFFFF) & 255) << 8 * i;
                    *(uint32_t*)(s_l + fr * LSTRIDE + n * 16 + fp * 4) = b;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 16 * ROW / 16 / WAVE; ++i) {
            const int piece16 = i * WAVE + lane, row = piece16 / (ROW / 16), at16 = piece16 % (ROW / 16) * 16;
            if (m * 16 + row < rows)
                *(i32x4_t*)((int8_t*)part.out + ((size_t)(row0 + m * 16 + row) * N + col0) * ES + at16) =
                    *(const i32x4_t*)(s_o + row * STRIDE + at16);
        }
        if (low) {
            const int row = lane / NW, at16 = lane % NW * 16;
            if (row < 16 && m * 16 + row < rows)
                *(i32x4_t*)(part.low + (size_t)(row0 + m * 16 + row) * N + col0 + at16) =
                    *(const i32x4_t*)(s_l + row * LSTRIDE + at16);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Row-wise quantisation of h, the routed rows and then the shared expert's.  V > 0: a wave
// per row, V pieces of 4 values a lane in registers (rows up to 256 V); V = 0: a workgroup
// per row, read twice.  Bound by the launch and, from some 10 MB, by the caches h lies in.
constexpr int kQuantWaves = 4;
template <int V>
__global__ __launch_bounds__(kQuantWaves* WAVE) void quant_h_kernel(
    const float* __restrict__ h, const float* __restrict__ h_sh, int n_routed, int n_sh, int I,
    int I_sh, int8_t* __restrict__ q, int8_t* __restrict__ q_sh, float* __restrict__ scale,
    float* __restrict__ scale_sh) {
    constexpr bool kWave = V > 0;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
    const int at = kWave ? blockIdx.x * kQuantWaves + wave : blockIdx.x;
    if (at >= n_routed + n_sh) return;
    const bool routed = at < n_routed;
    const int r = routed ? at : at - n_routed;
    const int K = routed ? I : I_sh;
    const float* src = (routed ? h : h_sh) + (size_t)r * K;
    int8_t* dst = (routed ? q : q_sh) + (size_t)r * K;
    const int tid = kWave ? lane : (int)threadIdx.x;
    constexpr int STEP = kWave ? WAVE * 4 : kQuantWaves * WAVE * 4;
    f32x4_t v[kWave ? V : 1];
    float top = 0.f;
    if constexpr (kWave) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * STEP + tid * 4;
            v[i] = c < K ? *(const f32x4_t*)(src + c) : f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max_abs(top, v[i][j]);
    } else {
        for (int c = tid * 4; c < K; c += STEP) {
            const f32x4_t t = *(const f32x4_t*)(src + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max_abs(top, t[j]);
        }
    }
#pragma unroll
    for (int off = WAVE / 2; off >= 1; off >>= 1) top = max_abs(top, shfl_xor(top, off));
    if constexpr (!kWave) {
        __shared__ float s_top[kQuantWaves];
        if (lane == 0) s_top[wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kQuantWaves; ++i) top = max_abs(top, s_top[i]);
    }
    float to_code;
    const float s = row_scale(top, &to_code);
    if (tid == 0) (routed ? scale : scale_sh)[r] = s;
    auto put = [&](int c, const f32x4_t& t) {
        *(uint32_t*)(dst + c) = row_codes(t[0], t[1], t[2], t[3], to_code);
    };
    if constexpr (kWave) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * STEP + tid * 4 < K) put(i * STEP + tid * 4, v[i]);
    } else {
        for (int c = tid * 4; c < K; c += STEP) put(c, *(const f32x4_t*)(src + c));
    }
}

// Rows to 16 x 64 tiles: piece (n, k / 16) of 16 bytes to its place.
__global__ void prepack_i8_kernel(const i32x4_t* __restrict__ src, size_t pieces, int K,
                                  i32x4_t* __restrict__ dst) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= pieces) return;
    // i counts destination pieces: tile (row tile, K step), then 16-K piece, then row
    const size_t tile = i / 64;
    const int in = (int)(i % 64), steps = K / 64;
    const size_t rt = tile / steps;   // 16-row tile over all experts (N is a multiple of 16)
    const int s = (int)(tile % steps);
    dst[i] = src[(rt * 16 + in % 16) * (size_t)(K / 16) + s * 4 + in / 16];
}

hipError_t launch_prepack_i8(const int8_t* src, int n_exp, int N, int K, int8_t* dst,
                             hipStream_t stream) {
    // a row tile is K pieces, from one contiguous range to the other: whole tiles, up to 2^30
    // pieces a launch (a grid of 2^32 threads would be cut without an error)
    const size_t pieces = (size_t)n_exp * N * K / 16;
    const size_t most = (size_t)K * (K < 1 << 30 ? (1 << 30) / K : 1);
    for (size_t p0 = 0; p0 < pieces; p0 += most) {
        const size_t n = pieces - p0 < most ? pieces - p0 : most;
        prepack_i8_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>((const i32x4_t*)src + p0, n, K,
                                                                           (i32x4_t*)dst + p0);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

size_t linear_i8_ws_bytes(int, int, int) { return 0; }

constexpr int kCUs = 256, kLdsBytes = 160 * 1024;   // of an MI355X, of a CU

static int cdiv(int a, int b) { return (a + b - 1) / b; }

// T: tokens, n: routed rows.
template <int MF, int NT, int D, int Q, bool GATEUP>
static void launch_grouped_stream(ProductArgs& p, int routed_blocks, int T, int n, hipStream_t stream) {
    constexpr int cols = (GATEUP ? NT / 2 : NT) * 64;
    p.dense_blocks = p.dense.out ? cdiv(p.dense.M, MF * 16) : 0;
    p.dense_tiles = p.dense.out ? cdiv(p.dense.N, cols) : 1;
    p.routed_tiles = cdiv(p.routed.N, cols);
    auto wgs = [](int blocks, int tiles) {   // whole shares
        const int shares = xcd_shares(tiles);
        return cdiv(blocks, shares) * shares * tiles;
    };
    p.dense_wgs = wgs(p.dense_blocks, p.dense_tiles);
    const unsigned grid = (unsigned)(p.dense_wgs + wgs(routed_blocks, p.routed_tiles));
    grouped_stream_kernel<MF, NT, D, Q, GATEUP>
        <<<grid, 4 * WAVE, 0, stream>>>(p, (uint32_t)T, (uint32_t)(GATEUP ? T : n));
}

template <bool LORA>
static hipError_t launch_linear(const int8_t* a, const float* a_scale, int M, int K, const I8MatDev& w,
                                int N, uint16_t* out, const LoraDev& lora, hipStream_t stream) {
#define MOE_TILES(WM, MF, WN, NF, ST, KS)                                                         \
    {                                                                                         \
        const int mt = cdiv(M, WM * MF * 16), nt = cdiv(N, WN * NF * 16);                     \
        const int lds = (WM * MF + WN * NF) * 1024 * ST * KS, most = kCUs * (kLdsBytes / lds);     \
        const int grid = LORA || mt * nt < most ? (mt * nt + 7) / 8 * 8 : most;                       \
        linear_tiles_kernel<WM, MF, WN, NF, ST, KS, LORA><<<grid, WM * WN * WAVE, 0, stream>>>(   \
            a, a_scale, M, K, w, N, out, mt, nt, lora);                                       \
    }
    // The smallest tile that still makes no more than one round of the CUs (the larger ones
    // read less but leave CUs idle; us measured, small against next larger).  K over 8 waves:
    //   16 x 16: 17x2048x7168 6.5 / 7.6, but two rounds 32x4096x4096 7.3 / 5.8;
    //   16 x 32: 64x2048x7168 7.8 / 10.5;  32 x 32: 128x2048x7168 10.5 / 12.5, 64x4096x4096
    //     7.5 / 8.8;  32 x 64: 256x2048x7168 12.7 / 16.9, 128x4096x4096 8.9 / 11.0, 512 rows
    //     by 64 x 64 no faster than through LDS.  Weights in rows come as half lines too:
    //     256x1001x4096 10.0 by 32 x 32 against 9.0 through LDS.
    // K by one workgroup, through LDS:
    //   32 x 64: 333x1001x2048 6.2 / 8.4;  64 x 64: 128x8192x7168 19.4 / 27;
    //   128 x 64: 333x4096x4096 17.2 / 24, 1000x2048x2048 11.2 / 15;
    // beyond that 128 x 128, 256 x 128 or 256 x 256, by rounds that take 2, 3 and 5 (K 2048:
    //   14.7, 20 to 25 and 37 us), the larger where they are even:
    //   1024x4096x2048 14.7 / 18.0 / 27, 2048x4096x4096 45.9 / 38.2 / 47.7,
    //   4096x2048x7168 75.7 / 63.0 / 75.9, 4096x4096x2048 53.3 / 43.8 / 37.3.
    auto tiles = [&](int bm, int bn) { return (long long)cdiv(M, bm) * cdiv(N, bn); };
    auto rounds = [&](int bm, int bn) { return (tiles(bm, bn) + kCUs - 1) / kCUs; };
    const long long c128 = 2 * rounds(128, 128), c192 = 3 * rounds(256, 128), c256 = 5 * rounds(256, 256);
#define MOE_SPLIT(MF, NF, D)                                                                  \
    linear_split_kernel<MF, NF, D, LORA>                                                      \
        <<<(unsigned)tiles(MF * 16, NF * 16), kFewWaves * WAVE, 0, stream>>>(                 \
            a, a_scale, M, K, w, N, out, cdiv(N, NF * 16), lora)
    if (M <= 16 || tiles(16, 16) <= kCUs)
        linear_few_kernel<LORA>
            <<<(unsigned)tiles(16, 16), kFewWaves * WAVE, 0, stream>>>(a, a_scale, M, K, w, N, out, lora);
    else if (tiles(16, 32) <= kCUs) MOE_SPLIT(1, 2, 2);
    else if (w.tiles && tiles(32, 32) <= kCUs) MOE_SPLIT(2, 2, 1);
    else if (w.tiles && tiles(32, 64) <= kCUs) MOE_SPLIT(2, 4, 1);
    else if (tiles(32, 64) <= kCUs) MOE_TILES(1, 2, 2, 2, 8, 1)
    else if (tiles(64, 64) <= kCUs) MOE_TILES(2, 2, 2, 2, 4, 2)
    else if (tiles(128, 64) <= kCUs) MOE_TILES(2, 4, 2, 2, 4, 2)
    else if (c256 <= c192 && c256 <= c128) MOE_TILES(2, 8, 4, 4, 4, 1)
    else if (c192 <= c128) MOE_TILES(2, 8, 4, 2, 4, 1)
    else MOE_TILES(2, 4, 4, 2, 4, 2)
#undef MOE_SPLIT
#undef MOE_TILES
    return hipGetLastError();
}

hipError_t launch_linear_i8(const int8_t* a, const float* a_scale, int M, int K, const I8MatDev& w,
                            int N, uint16_t* out, void*, hipStream_t stream) {
    return launch_linear<false>(a, a_scale, M, K, w, N, out, LoraDev{}, stream);
}

hipError_t launch_linear_lora_i8(const int8_t* a, const float* a_scale, int M, int K, const I8MatDev& w,
                                 int N, const LoraDev& lora, uint16_t* out, hipStream_t stream) {
    return launch_linear<true>(a, a_scale, M, K, w, N, out, lora, stream);
}

GemmI8Ws gemm_i8_ws_layout(int T, int H, int I, int I_sh, int k) {
    GemmI8Ws L{};
    const size_t n = (size_t)T * k;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 256);
        return at;
    };
    L.h = take(n * I * 4);
    L.h_sh = take((size_t)T * I_sh * 4);
    const size_t end = o;
    o = 0;   // down writes the low bytes when the activations have become codes
    L.low = take(n * H);
    L.low_sh = take(I_sh ? (size_t)T * H : 0);
    if (o < end) o = end;
    L.q = take(n * I);
    L.q_sh = take((size_t)T * I_sh);
    L.scale = take(n * 4);
    L.scale_sh = take(I_sh ? (size_t)T * 4 : 0);
    L.total = o;
    return L;
}

hipError_t launch_grouped_i8(const GemmI8Problem& g, void* ws, bool want_low, hipStream_t stream) {
    const GemmI8Ws L = gemm_i8_ws_layout(g.T, g.H, g.I, g.I_sh, g.k);
    char* base = (char*)ws;
    float *h = (float*)(base + L.h), *h_sh = (float*)(base + L.h_sh);
    int8_t *q = (int8_t*)(base + L.q), *q_sh = (int8_t*)(base + L.q_sh);
    float *scale = (float*)(base + L.scale), *scale_sh = (float*)(base + L.scale_sh);
    ProductArgs p{};
    p.k = g.k;
    p.block_expert = g.r.block_expert;
    p.block_row = g.r.block_row;
    p.offsets = g.r.offsets;
    p.n_blocks = g.r.n_blocks;
    p.sorted_assign = g.r.sorted_assign;
    p.routed = PartI8{g.x, g.x_scale, g.gate, g.up, 0, g.I, g.H, h, nullptr};
    if (g.I_sh) p.dense = PartI8{g.x, g.x_scale, g.sh_gate, g.sh_up, g.T, g.I_sh, g.H, h_sh, nullptr};
    const int n = g.T * g.k;
    // Rows / 16, weight rows of a wave / 16, steps ahead, steps of a chunk; us measured at H
    // 2048, I 512, 256 experts, k 8.  Gate/up: 64 tokens 1,2,4,4 76; 512 tokens 2,2,4,4 94
    // (2,4,4,4 103, 1,2,4,4 99, 4,4,2,2 105); 2048 tokens 4,4,2,2 120, skewed 90 (2,2,4,4 138
    // and 115, 2,4,4,4 129 and 106, 4,4,2,8 132 and 104).  Down, without low bytes: 64 tokens 1,2,4,4 42; 512
    // tokens 2,4,2,4 52 (1,2,4,4 54, 4,4,4,4 55); 2048 tokens 4,4,4,4 72, skewed 58 (2,4,2,4 76
    // and 63, 4,4,4,8 77 and 67).  Blocks of 32 rows that are mostly full take the wider waves.
    const bool full = n > 32 * g.E;
    if (g.block_rows == 16) launch_grouped_stream<1, 2, 4, 4, true>(p, g.max_blocks, g.T, n, stream);
    else if (g.block_rows == 32 && !full) launch_grouped_stream<2, 2, 4, 4, true>(p, g.max_blocks, g.T, n, stream);
    else if (g.block_rows == 32) launch_grouped_stream<2, 4, 4, 4, true>(p, g.max_blocks, g.T, n, stream);
    else launch_grouped_stream<4, 4, 2, 2, true>(p, g.max_blocks, g.T, n, stream);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int n_sh = g.I_sh ? g.T : 0, widest = g.I > g.I_sh ? g.I : g.I_sh;
#define MOE_QUANT(V)                                                                              \
    quant_h_kernel<V><<<V ? cdiv(n + n_sh, kQuantWaves) : n + n_sh, kQuantWaves * WAVE, 0, stream>>>( \
        h, h_sh, n, n_sh, g.I, g.I_sh, q, q_sh, scale, scale_sh)
    if (widest <= 256) MOE_QUANT(1);
    else if (widest <= 512) MOE_QUANT(2);
    else if (widest <= 1024) MOE_QUANT(4);
    else if (widest <= 2048) MOE_QUANT(8);
    else MOE_QUANT(0);
#undef MOE_QUANT
    if ((err = hipGetLastError()) != hipSuccess) return err;
    int8_t* low = want_low ? (int8_t*)(base + L.low) : nullptr;
    int8_t* low_sh = want_low ? (int8_t*)(base + L.low_sh) : nullptr;
    p.routed = PartI8{q, scale, g.down, {}, 0, g.H, g.I, g.expert_out, low};
    if (g.I_sh) p.dense = PartI8{q_sh, scale_sh, g.sh_down, {}, g.T, g.H, g.I_sh, g.shared_out, low_sh};
    if (g.block_rows == 16) launch_grouped_stream<1, 2, 4, 4, false>(p, g.max_blocks, g.T, n, stream);
    else if (g.block_rows == 32) launch_grouped_stream<2, 4, 2, 4, false>(p, g.max_blocks, g.T, n, stream);
    else launch_grouped_stream<4, 4, 4, 4, false>(p, g.max_blocks, g.T, n, stream);
    return hipGetLastError();
}

}  // namespace moeq4
