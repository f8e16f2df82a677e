// A few tokens (1 to 64) together through the whole 4-bit layer: the selection (inside the
// first kernel, or a launch of its own), gate/up, and down with the weighted sum.
//
//   y_t = sum_j w_tj FFN_e(t,j)(x_t) + g_t FFN_shared(x_t),  FFN(x) = (silu(x Wg^T) * x Wu^T) Wd^T
//
// A weight tile is the A operand of the matrix instruction, 16 rows by 32 K, and up to 16 tokens of
// an expert are the columns of B.  So a weight costs its read and its dequantization, 17
// instructions for 8, for 16 tokens as for one; both sides of the sums are bf16 exactly as the
// format says (w = bf16(q * s + b), x), products and sums fp32.  h already holds the token's
// weight, and is kept as two bf16 (16 bits), so that y has the one rounding of its own.
//
// Up to 8 tokens, two launches (2048 wide, 256 experts of 512 and a shared one, scales packed, 8 a token):
//   batch_gateup_kernel: every workgroup selects and groups for itself, then its waves split K.
//   batch_down_kernel: a workgroup owns 8 columns of y for all tokens, and the products' columns are
//     the tokens, so the sum over the experts stays in the accumulators.  The 16 x 16 product is
//     used as two of 8 x 8: rows and columns 8 .. 15 hold the same columns of y and tokens at a
//     K 128 further on.
//   1, 2, 4, 8 tokens 13.0 + 6.6, 15.4 + 8.2, 17.9 + 11.2 and 26.5 + 20.4 us, for weights that 6.2
//   TB/s read in 2.6, 4.8, 9.2 and 16.5; in the form below 18.2 + 9.9 for 2, 18.1 + 10.9 for 4, 23.9 +
//   16.6 for 8, each with 7 to 9 us of selection and join.
//   Wider than 2048 (up to 4 tokens 4096) x does not fit the first launch's 32 KB, and every task fetches it
//   in parts: 8 tokens 85 us in all 4096 wide and 143 7168 wide, where moe_layer_q4 takes 64 and 99.
// More tokens, four launches: batch_select_kernel (4.7 us), batch_tiles_kernel for gate/up and for down,
//   batch_join_kernel (4.6).  16 tokens 30.7 + 17.8 us (floor 14.5 + 7.2), 32 tokens 48.0 + 29.3 (31 +
//   16), 64 tokens of skewed experts 29.4 + 18.1 (10 + 5).
// What bounds them: 5 us of a launch are its own, 6 to 8 pass before a workgroup's first product (list, tile,
// operands, first weights, each a trip to memory), then dequantization (34 ns a word and wave on a
// SIMD) and the 24 bytes a ns that a compute unit gets from memory take about as long as each other.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_lds.h"
#include "moe_score.h"

namespace moeq4 {

constexpr int kBdWaves = 16;             // waves of a down workgroup
constexpr int kBdAhead = 2;

// h as two bf16: the value and what its rounding left.
__device__ __forceinline__ void split_bf16(float v, uint16_t* hi, uint16_t* lo) {
    const __bf16 h = (__bf16)v;
    *hi = __builtin_bit_cast(uint16_t, h);
    *lo = __builtin_bit_cast(uint16_t, (__bf16)bf16_rest(v, *hi));
}

template <int EPL>
__device__ __forceinline__ void batch_select_token(const BatchArgs& p, int t, int32_t* idx, float* w,
                                                   uint32_t* scr) {
    const float* row = p.logits + (size_t)t * p.E;
    if (p.scored) score_topk_token<EPL>(row, p.bias, p.E, p.k, p.rule, idx, w);
    else topk_token<EPL>(row, p.E, p.k, idx, w, scr, (int*)(scr + p.k), (float*)(scr + 2 * p.k));
}

// One wave a token, for batches whose selection is not repeated in every workgroup.
constexpr int kBsWaves = 4;
template <int EPL>
__global__ __launch_bounds__(kBsWaves* WAVE) void batch_select_kernel(BatchArgs p) {
    __shared__ uint32_t s_scr[kBsWaves][3 * kScoredMaxK];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int t = blockIdx.x * kBsWaves + wave;
    if (t >= p.T) return;
    batch_select_token<EPL>(p, t, p.topk_idx + (size_t)t * p.k, p.topk_w + (size_t)t * p.k, s_scr[wave]);
}

// Sum of v over this lane and the lanes below it.
__device__ __forceinline__ int wave_incl_sum_i32(int v, int lane) {
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int o = __shfl_up(v, off, WAVE);
        v += lane >= off ? o : 0;
    }
    return v;
}

// The lowest 16 set bits of m, which has more than 16.
__device__ __forceinline__ unsigned long long lowest_16(unsigned long long m) {
    int bits = 0;
#pragma unroll
    for (int b = 32; b; b >>= 1)
        if (__popcll(m & ((1ull << (bits + b)) - 1)) <= 16) bits += b;
    return m & ((1ull << bits) - 1);
}

// Entries: an expert with up to 16 of its tokens, which are the columns of its products.  Up to
// kBatchDense tokens every entry's columns are the tokens as they come; of more, an entry's own
// tokens in order, and an expert of more than 16 has several entries.
constexpr int kBatchDense = 16;
__device__ __forceinline__ unsigned long long shared_mask(int T, int v) {
    const unsigned long long all = ~0ull >> (64 - T);
    return T <= kBatchDense ? all : all & (0xFFFFull << 16 * v);
}
__device__ __forceinline__ void list_tokens(unsigned long long mask, uint8_t* tok, int lane) {
    if (mask >> lane & 1) tok[__popcll(mask & lanemask_lt())] = (uint8_t)lane;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Where rows row .. + 3 (row a multiple of 4) of column c lie in an entry's h: for each 128 rows the B
// operands of the down products, four of 1 KB, lane after lane, so that a load of one is contiguous.
__device__ __forceinline__ size_t h_place(int row, int c) {
    return (size_t)(row / 128) * 2048 + ((row % 32) / 8 * 64 + (row % 128) / 32 * 16 + c) * 8 + row % 8;
}

// dequant_word's weights from a code read as a subnormal fp16, q 2^-24 or, 4 bits up, q 2^-20: 17
// instructions, and 30.5 ns for a word in each lane of a SIMD's wave where the fp8 conversions take
// 35.3.  s: the scale times 2^24 and 2^20, which is exact below 2^103.
__device__ __forceinline__ bf16x8_t dequant_half(uint32_t w, f32x2_t s, float b) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    const uint32_t w8 = w >> 8;
    const f16x2_t q04 = __builtin_bit_cast(f16x2_t, w & 0x000F000Fu), q15 = __builtin_bit_cast(f16x2_t, w & 0x00F000F0u);
    const f16x2_t q26 = __builtin_bit_cast(f16x2_t, w8 & 0x000F000Fu), q37 = __builtin_bit_cast(f16x2_t, w8 & 0x00F000F0u);
    u32x4_t r;
    r[0] = pack_bf16x2(__builtin_fmaf((float)q04[0], s[0], b), __builtin_fmaf((float)q15[0], s[1], b));
    r[1] = pack_bf16x2(__builtin_fmaf((float)q26[0], s[0], b), __builtin_fmaf((float)q37[0], s[1], b));
    r[2] = pack_bf16x2(__builtin_fmaf((float)q04[1], s[0], b), __builtin_fmaf((float)q15[1], s[1], b));
    r[3] = pack_bf16x2(__builtin_fmaf((float)q26[1], s[0], b), __builtin_fmaf((float)q37[1], s[1], b));
    return __builtin_bit_cast(bf16x8_t, r);
}

// x of `rows` tokens (their numbers in tok, or `dense`), chunks c0 .. + len of 128 K, to LDS: 1 KB for 4
// tokens of a chunk.  16 bytes of token r, piece j of a chunk lie at place j ^ r, so that the 16
// tokens' pieces that a product reads at once are in different banks.
__device__ __forceinline__ void stage_x(buf_rsrc_t rx, bool dense, const uint8_t* tok, int rows, int H, char* to,
                                        int c0, int len, int wave, int waves, int lane) {
    const int nq = (rows + 3) / 4, g = lane / 16, c = lane % 16;
    for (int i = wave; i < len * nq; i += waves) {
        const int q = i / nq, r = (i - q * nq) * 4 + g;
        const int kk = (c0 + q) * 128 + (c ^ r) * 8;
        const int t = dense ? r : tok[r];
        const bool in = r < rows && kk < H;
        buf_to_lds16(rx, to + i * 1024, in ? ((uint32_t)t * H + kk) * 2 : 0xFFFFFFF0u, 0);
    }
}

// The list of entries from the tokens' experts, in LDS; returns their number.  Begins and ends with a
// barrier.
template <int NW, typename Idx>
__device__ __forceinline__ int group_tokens(const BatchArgs& p, const Idx* s_idx, unsigned long long* s_mask,
                                            int* s_total, uint4* s_list) {
    constexpr int THREADS = NW * WAVE;
    const int tid = threadIdx.x, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int n = p.T * p.k;
    for (int e = tid; e < p.E; e += THREADS) s_mask[e] = 0;
    __syncthreads();
    for (int a = tid; a < n; a += THREADS) atomicOr(&s_mask[s_idx[a]], 1ull << (a / p.k));
    __syncthreads();
    int used = 0;
    for (int e0 = 0; e0 < p.E; e0 += THREADS) {
        const int e = e0 + tid;
        unsigned long long m = e < p.E ? s_mask[e] : 0ull;
        const int mine = !m ? 0 : p.T <= kBatchDense ? 1 : (__popcll(m) + 15) / 16;
        const int upto = wave_incl_sum_i32(mine, lane);
        if (lane == WAVE - 1) s_total[wave] = upto;
        __syncthreads();
        int before = upto - mine, all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int v = s_total[w];
            before += w < wave ? v : 0;
            all += v;
        }
        for (int i = 0; i < mine; ++i) {
            const unsigned long long part = i + 1 < mine ? lowest_16(m) : m;
            s_list[used + before + i] = uint4{(uint32_t)e, 0, (uint32_t)part, (uint32_t)(part >> 32)};
            m &= ~part;
        }
        used += all;
        __syncthreads();
    }
    return used;
}

// ---- up to kBatchColumns tokens ----
//
// Selects too; x of all tokens is in LDS, read in the order of the B operand, where lanes that fetched
// their 16 bytes of 16 rows from memory held up the weights' loads.  x_kb: LDS for x, in pieces of 4 tokens by 128 K; T tokens' pieces of per_seg chunks fit.
// rt_log: a task is 16 << rt_log rows of an entry, 16 a wave, and the other waves split K.  A
// workgroup's tasks lie together, and the waves fetch the next task's weights before they are done
// with this one's.
constexpr int kBgWaves = 8;
// Waves that a SIMD's registers hold: three workgroups' with scales and biases in one word, else two.
constexpr int bg_per_simd(int epl, bool sb) { return sb && epl <= 8 ? 6 : 4; }

template <int EPL, bool SB>
__global__ __launch_bounds__(kBgWaves* WAVE, bg_per_simd(EPL, SB)) void batch_gateup_kernel(BatchArgs p, int x_kb, int rt_log) {
    constexpr int NW = kBgWaves, THREADS = NW * WAVE;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    __shared__ int s_total[NW];
    const int T = p.T, k = p.k, n = T * k, H = p.H;
    char* s_x = s_dyn;
    f32x4_t* s_part = (f32x4_t*)(s_x + x_kb * 1024);                 // [2][NW][2][WAVE]
    uint4* s_list = (uint4*)(s_part + 2 * NW * 2 * WAVE);
    float* s_w = (float*)(s_list + p.tiles);
    int32_t* s_idx = (int32_t*)(s_w + n);
    const int tid = threadIdx.x, lane = tid % WAVE, g = lane / 16, c = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int chunks = (H + 127) / 128, nq = (T + 3) / 4, per_seg = x_kb / nq;
    const buf_rsrc_t rx = make_buf(p.x, (uint32_t)T * H * 2);
    auto stage = [&](int c0) {
        stage_x(rx, true, nullptr, T, H, s_x, c0, min(per_seg, chunks - c0), wave, NW, lane);
    };
    stage(0);
    int staged = 0;   // first chunk of x in LDS

    // ---- selection and grouping, whose masks and scratch lie where the waves' sums will ----
    static_assert(NW * 4096 >= 1024 * 8 + NW * 3 * kScoredMaxK * 4, "scratch behind the masks");
    if (wave < T)
        batch_select_token<EPL>(p, wave, s_idx + wave * k, s_w + wave * k,
                                (uint32_t*)((unsigned long long*)s_part + p.E) + wave * 3 * kScoredMaxK);
    const int used = group_tokens<NW>(p, s_idx, (unsigned long long*)s_part, s_total, s_list);
    if (blockIdx.x == 0) {
        for (int u = tid; u < used; u += THREADS) p.list[u] = s_list[u];
        if (tid == 0) *p.n_list = used;
        for (int a = tid; a < n; a += THREADS) {
            p.topk_idx[a] = s_idx[a];
            p.topk_w[a] = s_w[a];
        }
    }

    // ---- tasks: row tiles of the shared expert's entries, then of the list's ----
    const int KS = NW >> rt_log, rt = wave & ((1 << rt_log) - 1), ks = wave >> rt_log;
    const int ks_log = 31 - __builtin_clz(KS);
    const int sh_n = p.I_sh ? 1 : 0;
    const int sh_tiles = p.I_sh >> (4 + rt_log), tiles = p.I >> (4 + rt_log);
    const int tasks = sh_n * sh_tiles + used * tiles;
    const int last = (int)((long long)tasks * (blockIdx.x + 1) / gridDim.x);
    const int G = H / 64;
    const bool half_chunk = H % 128 != 0;   // the last chunk's groups g >= 2 lie behind K
    int task = (int)((long long)tasks * blockIdx.x / gridDim.x);
    int v = 0, tile = 0;
    if (task < last) {
        const int r = task - sh_n * sh_tiles;
        v = r < 0 ? task / sh_tiles : sh_n + r / tiles;
        tile = r < 0 ? task - v * sh_tiles : r - (v - sh_n) * tiles;
    }
    struct Entry {
        int expert;
        uint32_t mask;
    };
    auto entry = [&](int v) {
        Entry o{0, 0xFFu >> (8 - T)};
        if (v >= sh_n) {
            const uint4 ent = s_list[v - sh_n];
            o.expert = __builtin_amdgcn_readfirstlane((int)ent.x);
            o.mask = (uint32_t)__builtin_amdgcn_readfirstlane((int)ent.z);
        }
        return o;
    };

    // ---- the wave's weights: a sequence of chunks of its rows and K, from task to task ----
    struct Chunk {
        u32x4_t wg, wu;
        uint32_t sg, su, bg, bu;      // SB: scale and bias in sg, su
    };
    int l_task = task, l_v = v, l_tile = tile, l_seg = 0, l_q = 0, l_qb = 0;
    bool l_new = true;
    Entry l_ent;
    const char *gc = nullptr, *uc = nullptr, *gs = nullptr, *us = nullptr, *gb = nullptr, *ub = nullptr;
    uint32_t w_at = 0, s_at = 0;      // of the chunk, within the expert
    const int layout = p.gate.layout;
    const uint32_t w_step = layout ? 4096u : 64u, s_step = SB ? 512u : 4u;
    const uint32_t w_lane = code_word(layout, c, g * 4, H) * 4, s_lane = SB ? (g / 2 * 64 + c) * 4 : (c * G + g / 2) * 2;
    const uint32_t w_half = g >= 2 ? (layout ? 2048u : 32u) : 0u, s_half = g >= 2 ? (SB ? 256u : 2u) : 0u;
    auto fetch = [&](Chunk& o) {
        while (l_q >= l_qb) {         // the next segment, task or entry
            if (l_task >= last) return;
            const bool sh = l_v < sh_n;
            if (l_new) {
                l_ent = entry(l_v);
                l_new = false;
                const QMatDev& mg = sh ? p.sh_gate : p.gate;
                const QMatDev& mu = sh ? p.sh_up : p.up;
                const size_t row = (size_t)l_ent.expert * (sh ? p.I_sh : p.I);
                const size_t ce = row * (H / 2), se = row * G * (SB ? 4 : 2);
                gc = (const char*)mg.codes + ce;
                uc = (const char*)mu.codes + ce;
                gs = (const char*)mg.scales + se;
                us = (const char*)mu.scales + se;
                gb = (const char*)mg.biases + se;
                ub = (const char*)mu.biases + se;
            }
            const int c0 = l_seg * per_seg, len = min(per_seg, chunks - c0);
            l_q = c0 + (len * ks >> ks_log);
            l_qb = c0 + (len * (ks + 1) >> ks_log);
            const uint32_t stripe = (l_tile << rt_log) + rt, block = stripe / 4;   // 16 and 64 rows
            w_at = block * H * 32 + stripe % 4 * (layout ? 512u : H * 8) + l_q * w_step;
            s_at = SB ? (block * G * 64 + stripe % 4 * 16) * 4 + l_q * s_step : stripe * G * 32 + l_q * s_step;
            if (c0 + len < chunks) {
                ++l_seg;
            } else {
                l_seg = 0;
                ++l_task;
                if (++l_tile == (sh ? sh_tiles : tiles)) {
                    l_tile = 0;
                    ++l_v;
                    l_new = true;
                }
            }
        }
        uint32_t w = w_at + w_lane, s = s_at + s_lane;
        if (half_chunk && l_q == chunks - 1) {   // weights of the row again: they meet zeros in LDS
            w -= w_half;
            s -= s_half;
        }
        o.wg = *(const u32x4_t*)(gc + w);
        o.wu = *(const u32x4_t*)(uc + w);
        if constexpr (SB) {
            o.sg = *(const uint32_t*)(gs + s);
            o.su = *(const uint32_t*)(us + s);
        } else {
            o.sg = *(const uint16_t*)(gs + s);
            o.su = *(const uint16_t*)(us + s);
            o.bg = *(const uint16_t*)(gb + s);
            o.bu = *(const uint16_t*)(ub + s);
        }
        ++l_q;
        w_at += w_step;
        s_at += s_step;
    };
    Chunk w0 = {}, w1 = {};
    fetch(w0);
    fetch(w1);
    wait_loads<0>();
    __syncthreads();
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    int turn = 0;   // the task's number here: the waves that join its sums, where these lie
    // columns behind the last token read any one's x
    const int cx = c < nq * 4 ? c : 0, x_low = (cx & 3) * 16;
    const char* x_lane = s_x + cx / 4 * 1024 + cx % 4 * 256 + (g * 4 ^ (cx & 12)) * 16;
    for (; task < last; ++v, tile = 0) {
        const Entry ent = entry(v);
        const bool sh = v < sh_n;
        for (const int n_tiles = sh ? sh_tiles : tiles; tile < n_tiles && task < last; ++tile, ++task, ++turn) {
            const bool joins = ks == (turn & (KS - 1));
            float wt = 1.f;   // the weight of the column's token
            bool on = false;
            for (int c0 = 0; c0 < chunks; c0 += per_seg) {
                const int len = min(per_seg, chunks - c0);
                if (c0 != staged) {
                    __syncthreads();
                    stage(c0);
                    staged = c0;
                    wait_loads<0>();
                    __syncthreads();
                }
                if (joins && c0 == 0) {
                    on = ent.mask >> c & 1;
                    const int t = on ? c : 0;
                    if (sh) {
                        if (p.shared_gate) wt = p.shared_gate[t];
                    } else {
                        int a = -1;   // the lanes of a column share the search
#pragma unroll 2
                        for (int j = g; j < k; j += 4)
                            if (s_idx[t * k + j] == ent.expert) a = t * k + j;
                        a = max(a, __shfl_xor(a, 16));
                        a = max(a, __shfl_xor(a, 32));
                        wt = on ? s_w[a] : 0.f;
                    }
                }
                const int q1 = c0 + (len * (ks + 1) >> ks_log);
                for (int q = c0 + (len * ks >> ks_log); q < q1; ++q) {
                    Chunk w2 = w1;
                    fetch(w2);
                    const char* xq = x_lane + (q - c0) * nq * 1024;
                    const float sg = bf16_to_f32((uint16_t)w0.sg), su = bf16_to_f32((uint16_t)w0.su);
                    const float bg = bf16_to_f32((uint16_t)(SB ? w0.sg >> 16 : w0.bg));
                    const float bu = bf16_to_f32((uint16_t)(SB ? w0.su >> 16 : w0.bu));
                    const f32x2_t dg = {sg * 0x1p24f, sg * 0x1p20f}, du = {su * 0x1p24f, su * 0x1p20f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8_t b = *(const bf16x8_t*)(xq + (x_low ^ i * 16));
                        acc[0] = mfma_16x16x32(dequant_half(w0.wg[i], dg, bg), b, acc[0]);
                        acc[1] = mfma_16x16x32(dequant_half(w0.wu[i], du, bu), b, acc[1]);
                    }
                    w0 = w1;
                    w1 = w2;
                }
            }
            // the waves' sums over K in order; 4 rows of one token a lane
            f32x4_t* part = s_part + (turn & 1) * NW * 2 * WAVE;
            part[(wave * 2 + 0) * WAVE + lane] = acc[0];
            part[(wave * 2 + 1) * WAVE + lane] = acc[1];
            acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            wait_lds();
            bare_barrier_i8();
            if (joins && on) {
                f32x4_t gsum = {0.f, 0.f, 0.f, 0.f}, usum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
                for (int i = 0; i < KS; ++i) {
                    const int w = rt + (i << rt_log);
                    gsum += part[(w * 2 + 0) * WAVE + lane];
                    usum += part[(w * 2 + 1) * WAVE + lane];
                }
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split_bf16(wt * (silu_f32(gsum[i]) * usum[i]), &hi[i], &lo[i]);
                const int row0 = ((tile << rt_log) + rt) * 16;
                const size_t at_h = (sh ? p.sh_h : (size_t)(v - sh_n) * ((p.I + 127) / 128) * 2048) +
                                    h_place(row0 + g * 4, c);
                *(u32x2_t*)(p.h_hi + at_h) = u32x2_t{(uint32_t)hi[0] | (uint32_t)hi[1] << 16,
                                                     (uint32_t)hi[2] | (uint32_t)hi[3] << 16};
                *(u32x2_t*)(p.h_lo + at_h) = u32x2_t{(uint32_t)lo[0] | (uint32_t)lo[1] << 16,
                                                     (uint32_t)lo[2] | (uint32_t)lo[3] << 16};
            }
        }
    }
}

// A workgroup owns 8 columns of y; its waves take 256 K of an entry at a time, whose columns are the
// tokens (kBatchDense), so the sum over the entries stays in the accumulators.
__global__ __launch_bounds__(kBdWaves* WAVE) void batch_down_kernel(BatchArgs p) {
    __shared__ f32x4_t s_part[kBdWaves][WAVE];
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int T = p.T, H = p.H, I = p.I, I_sh = p.I_sh;
    const int g = lane / 16, c = lane % 8, half = lane % 16 / 8;
    const int col = blockIdx.x * 8 + c;
    const int per = (I + 255) / 256, per_sh = (I_sh + 255) / 256;
    const int routed = *p.n_list * per, steps = routed + per_sh;
    u32x4_t wv[kBdAhead];
    float sc[kBdAhead], bi[kBdAhead];
    u32x4_t hi[kBdAhead][4], lo[kBdAhead][4];
    auto load = [&](int s, int step) {
        const bool in = step < steps, sh = step >= routed;
        const int u = in && !sh ? step / per : 0;
        const int d = sh ? step - routed : step - u * per;
        uint4 ent = {0, 0, 0xFF, 0};
        if (in && !sh) ent = p.list[u];
        const int K = sh ? I_sh : I, kb = d * 256 + half * 128 + g * 32;
        const bool on = in && kb < K && c < T && (ent.z >> c & 1);   // the entry's token
        const size_t h_at = (sh ? p.sh_h : (size_t)u * ((I + 127) / 128) * 2048) + (size_t)(d * 2 + half) * 2048 +
                  (g * 16 + c) * 8;
        const QMatDev& m = sh ? p.sh_down : p.down;
        const size_t row = (size_t)ent.x * H + col;
        wv[s] = in && kb < K ? *(const u32x4_t*)(m.codes + (size_t)ent.x * H * (K / 8) +
                                                 code_word(m.layout, col, kb / 8, K))
                             : u32x4_t{0, 0, 0, 0};
        sc[s] = in && kb < K ? bf16_to_f32(m.scales[row * (K / 64) + kb / 64]) : 0.f;
        bi[s] = in && kb < K ? bf16_to_f32(m.biases[row * (K / 64) + kb / 64]) : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[s][i] = on ? *(const u32x4_t*)(p.h_hi + h_at + i * 512) : u32x4_t{0, 0, 0, 0};
            lo[s][i] = on ? *(const u32x4_t*)(p.h_lo + h_at + i * 512) : u32x4_t{0, 0, 0, 0};
        }
    };
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kBdAhead; ++s) load(s, wave + s * kBdWaves);
    for (int step = wave; step < steps; step += kBdAhead * kBdWaves) {
#pragma unroll
        for (int s = 0; s < kBdAhead; ++s) {
            const f32x2_t d = {sc[s] * 0x1p24f, sc[s] * 0x1p20f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x8_t w = dequant_half(wv[s][i], d, bi[s]);
                acc = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, hi[s][i]), acc);
                acc = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, lo[s][i]), acc);
            }
            load(s, step + (s + kBdAhead) * kBdWaves);
        }
    }
    // the waves' sums in order; rows and columns 0 .. 7 and 8 .. 15 hold two parts of K
    s_part[wave][lane] = acc;
    __syncthreads();
    if (tid < 64) {
        const int r = tid % 8, t = tid / 8;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kBdWaves; ++w)
            y += s_part[w][r / 4 * 16 + t][r % 4] + s_part[w][(r + 8) / 4 * 16 + 8 + t][r % 4];
        if (t < T) p.y[(size_t)t * H + blockIdx.x * 8 + r] = (uint16_t)pack_bf16x2(y, 0.f);
    }
}

// ---- more tokens: gate/up (DOWN 0) and down (DOWN 1), whose work is a list of tiles ----
//
// A tile is one wave's: 16 rows of an entry's gate and up, or 32 of its down, times the whole K, so
// that nothing is joined and waves do not wait for each other (K over 8 waves, a barrier a task:
// 32 tokens 56 + 38 us instead of 52 + 32).  A workgroup takes a run of tiles, which belong to one
// or two entries, whose B operands (x, or h as written) lie in LDS for all of its waves; where an
// entry's do not fit, a part of K after another.  kBmAhead chunks of a wave's weights are in flight,
// 2 KB each: 32 tokens 49 + 30 us, with 12 waves 52 + 31, with four chunks and 12 waves 53 + 32; 16
// tokens take 30 + 18 in each but the last, 30 + 19.  The next tile's weights before this one's end
// gained nothing.
constexpr int kBmWaves = 16, kBmAhead = 2;

template <bool DOWN, bool SB>
__global__ __launch_bounds__(kBmWaves* WAVE) void batch_tiles_kernel(BatchArgs p, int x_kb) {
    constexpr int NW = kBmWaves, THREADS = NW * WAVE, ROWS = DOWN ? 32 : 16;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    __shared__ uint8_t s_tok[NW][WAVE];
    __shared__ int s_total[NW];
    const int T = p.T, E = p.E, k = p.k, n = T * k, H = p.H;
    const bool dense = T <= kBatchDense;
    char* s_x = s_dyn;
    uint4* s_list = (uint4*)(s_x + x_kb * 1024);
    uint16_t* s_idx = (uint16_t*)(s_list + p.tiles);
    const int tid = threadIdx.x, lane = tid % WAVE, g = lane / 16, c = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    int used;
    if constexpr (DOWN) {
        used = *p.n_list;
    } else {
        for (int a = tid; a < n; a += THREADS) s_idx[a] = (uint16_t)p.topk_idx[a];
        used = group_tokens<NW>(p, s_idx, (unsigned long long*)s_x, s_total, s_list);
        if (blockIdx.x == 0) {
            for (int u = tid; u < used; u += THREADS) p.list[u] = s_list[u];
            if (tid == 0) *p.n_list = used;
        }
    }
    const int sh_n = !p.I_sh ? 0 : dense ? 1 : (T + 15) / 16;
    // of an entry v, the shared expert's first: tiles, chunks of K, its B operand's size in LDS
    auto tiles_of = [&](int v) { return (DOWN ? H : v < sh_n ? p.I_sh : p.I) / ROWS; };
    auto k_of = [&](int v) { return !DOWN ? H : v < sh_n ? p.I_sh : p.I; };
    auto mask_of = [&](int v) {
        if (v < sh_n) return shared_mask(T, v);
        u32x4_t ent;
        if constexpr (DOWN) {   // another kernel's: through scalar loads
            typedef const __attribute__((address_space(4))) u32x4_t* scalar_t;
            ent = ((scalar_t)(uintptr_t)p.list)[v - sh_n];
        } else {
            ent = *(const u32x4_t*)(s_list + (v - sh_n));
        }
        return (unsigned long long)(uint32_t)__builtin_amdgcn_readfirstlane(ent[3]) << 32 |
               (uint32_t)__builtin_amdgcn_readfirstlane(ent[2]);
    };
    auto expert_of = [&](int v) {
        if (v < sh_n) return 0;
        if constexpr (DOWN) {
            typedef const __attribute__((address_space(4))) u32x4_t* scalar_t;
            return (int)((scalar_t)(uintptr_t)p.list)[v - sh_n][0];
        } else {
            return __builtin_amdgcn_readfirstlane((int)s_list[v - sh_n].x);
        }
    };
    auto piece_of = [&](unsigned long long mask) {   // KB of a chunk
        return DOWN ? 8 : ((dense ? T : __popcll(mask)) + 3) / 4;
    };
    const buf_rsrc_t rx = make_buf(p.x, (uint32_t)T * H * 2);
    // the B operand of entry v, chunks c0 .. + len, to `at`
    auto stage = [&](int v, unsigned long long mask, char* at, int c0, int len) {
        if constexpr (DOWN) {   // as it lies: for each chunk the four KB of h's upper parts, then the lower
            const size_t h0 = v < sh_n ? p.sh_h + (size_t)v * ((p.I_sh + 127) / 128) * 2048
                                       : (size_t)(v - sh_n) * ((p.I + 127) / 128) * 2048;
            const bool on = dense ? mask >> c & 1 : c < __popcll(mask);
            const int K = k_of(v);
            const buf_rsrc_t rh = make_buf(p.h_hi + h0, ((K + 127) / 128) * 4096);
            const buf_rsrc_t rl = make_buf(p.h_lo + h0, ((K + 127) / 128) * 4096);
            for (int i = wave; i < len * 8; i += NW) {
                const int q = c0 + i / 8;
                const bool in = on && q * 128 + g * 32 < K;
                buf_to_lds16(i & 4 ? rl : rh, at + i * 1024, in ? (q * 4 + i % 4) * 1024 + lane * 16 : 0xFFFFFFF0u, 0);
            }
        } else {
            if (!dense) list_tokens(mask, s_tok[wave], lane);
            stage_x(rx, dense, s_tok[wave], dense ? T : __popcll(mask), H, at, c0, len, wave, NW, lane);
        }
    };
    const int total = sh_n * ((DOWN ? H : p.I_sh) / ROWS) + used * ((DOWN ? H : p.I) / ROWS);
    int pos = (int)((long long)total * blockIdx.x / gridDim.x);
    const int last = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
    int v, tile;
    {
        const int sh_all = sh_n * ((DOWN ? H : p.I_sh) / ROWS), r = pos - sh_all, per = (DOWN ? H : p.I) / ROWS;
        v = r < 0 ? pos / ((DOWN ? H : p.I_sh) / ROWS) : sh_n + r / per;
        tile = r < 0 ? pos % ((DOWN ? H : p.I_sh) / ROWS) : r % per;
    }
    while (pos < last) {
        // ---- as many tiles as the B operands that fit into LDS have ----
        __syncthreads();
        int count = 0, per_seg = 1 << 30;
        {
            int room = x_kb, vv = v, from = tile;
            while (count < last - pos) {
                const unsigned long long mask = mask_of(vv);
                const int piece = piece_of(mask), chunks = (k_of(vv) + 127) / 128;
                const int here = min(tiles_of(vv) - from, last - pos - count);
                if (piece * chunks > room) {
                    if (count) break;
                    per_seg = x_kb / piece / kBmAhead * kBmAhead;   // one entry's, a part of K after another
                    count = min(here, NW);
                    break;
                }
                stage(vv, mask, s_x + (x_kb - room) * 1024, 0, chunks);
                room -= piece * chunks;
                count += here;
                ++vv;
                from = 0;
            }
        }
        for (int i0 = 0; i0 < count; i0 += NW) {
            const bool mine = i0 + wave < count;
            // this wave's tile
            int vv = v, tl = tile + min(i0 + wave, count - 1);
            const char* xb = s_x;
            unsigned long long mask = mask_of(vv);
            while (tl >= tiles_of(vv)) {
                tl -= tiles_of(vv);
                xb += piece_of(mask) * ((k_of(vv) + 127) / 128) * 1024;
                mask = mask_of(++vv);
            }
            const bool sh = vv < sh_n;
            const int K = k_of(vv), N = DOWN ? H : sh ? p.I_sh : p.I, chunks = (K + 127) / 128, G = K / 64;
            const int row0 = tl * ROWS, piece = piece_of(mask), expert = expert_of(vv);
            const size_t row = (size_t)expert * N;
            const QMatDev& m0 = DOWN ? (sh ? p.sh_down : p.down) : (sh ? p.sh_gate : p.gate);
            const QMatDev& m1 = DOWN ? m0 : (sh ? p.sh_up : p.up);
            const int layout = m0.layout;
            const size_t w0 = row * (K / 2) + (size_t)code_word(layout, row0, 0, K) * 4;
            const size_t w1 = DOWN ? row * (K / 2) + (size_t)code_word(layout, row0 + 16, 0, K) * 4 : w0;
            const size_t sc0 = SB ? ((row + row0) / 64 * G * 64 + row0 % 64) * 4 : (row + row0) * G * 2;
            const size_t sc1 = DOWN ? sc0 + 32 * G : sc0;
            const char *c0p = (const char*)m0.codes + w0, *c1p = (const char*)m1.codes + w1;
            const char *s0p = (const char*)m0.scales + sc0, *s1p = (const char*)m1.scales + sc1;
            const char *b0p = (const char*)m0.biases + sc0, *b1p = (const char*)m1.biases + sc1;
            const uint32_t w_step = layout ? 4096u : 64u, s_step = SB ? 512u : 4u;
            const uint32_t w_lane = code_word(layout, c, g * 4, K) * 4;
            const uint32_t s_lane = SB ? (g / 2 * 64 + c) * 4 : (c * G + g / 2) * 2;
            const bool half = K % 128 != 0;   // the last chunk's groups g >= 2 lie behind K
            u32x4_t wa[kBmAhead], wb[kBmAhead];
            uint32_t sa[kBmAhead], sb[kBmAhead], ba[kBmAhead], bb[kBmAhead];
            auto fetch = [&](int s, int q) {
                if (q >= chunks) return;
                uint32_t w = w_lane + q * w_step, a = s_lane + q * s_step;
                if (half && q == chunks - 1 && g >= 2) {   // weights of the row again: they meet zeros in LDS
                    w -= layout ? 2048u : 32u;
                    a -= SB ? 256u : 2u;
                }
                wa[s] = *(const u32x4_t*)(c0p + w);
                wb[s] = *(const u32x4_t*)(c1p + w);
                if constexpr (SB) {
                    sa[s] = *(const uint32_t*)(s0p + a);
                    sb[s] = *(const uint32_t*)(s1p + a);
                } else {
                    sa[s] = *(const uint16_t*)(s0p + a);
                    sb[s] = *(const uint16_t*)(s1p + a);
                    ba[s] = *(const uint16_t*)(b0p + a);
                    bb[s] = *(const uint16_t*)(b1p + a);
                }
            };
            if (mine) {
                fetch(0, 0);
                fetch(1, 1);
            }
            // the token of this lane's column
            bool on = mine && (dense ? mask >> c & 1 : c < __popcll(mask));
            int t = c, at = 0;
            if (!dense) {
                list_tokens(mask, s_tok[wave], lane);
                t = on ? s_tok[wave][c] : 0;
            }
            float wt = 1.f;
            if constexpr (DOWN) {
                if (!sh && on) at = p.assign[(vv - sh_n) * 16 + c];
            } else if (sh) {
                if (on && p.shared_gate) wt = p.shared_gate[t];
            } else {
                at = -1;   // its place among the token's experts: the lanes of a column share the search
#pragma unroll 2
                for (int j = g; j < k && on; j += 4)
                    if (s_idx[t * k + j] == expert) at = t * k + j;
                at = max(at, __shfl_xor(at, 16));
                at = max(at, __shfl_xor(at, 32));
                if (on) wt = p.topk_w[at];
                if (on && tl == 0 && g == 0) p.assign[(vv - sh_n) * 16 + c] = at;
            }
            f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const int cx = DOWN || c < piece * 4 ? c : 0;   // columns behind the last token read any one's x
            const uint32_t x_lane = DOWN ? lane * 16 : cx / 4 * 1024 + cx % 4 * 256 + (g * 4 ^ (cx & 12)) * 16;
            const uint32_t x_low = DOWN ? 0 : (cx & 3) * 16;
            for (int k0 = 0; k0 < chunks; k0 += per_seg) {
                const int k1 = per_seg < chunks - k0 ? k0 + per_seg : chunks;
                if (per_seg < chunks) {   // the same for all waves
                    __syncthreads();
                    stage(v, mask, s_x, k0, k1 - k0);
                }
                if (i0 == 0) {
                    wait_loads<0>();
                    __syncthreads();
                }
                if (!mine) continue;
                // slots by chunk: a segment's first chunk is a multiple of kBmAhead
                for (int q0 = k0; q0 < k1; q0 += kBmAhead) {
#pragma unroll
                    for (int s = 0; s < kBmAhead; ++s) {
                        if (q0 + s >= k1) break;
                        const char* xq = xb + (q0 + s - k0) * piece * 1024 + x_lane;
                        const float f0 = bf16_to_f32((uint16_t)sa[s]), f1 = bf16_to_f32((uint16_t)sb[s]);
                        const float e0 = bf16_to_f32((uint16_t)(SB ? sa[s] >> 16 : ba[s]));
                        const float e1 = bf16_to_f32((uint16_t)(SB ? sb[s] >> 16 : bb[s]));
                        const f32x2_t d0 = {f0 * 0x1p24f, f0 * 0x1p20f}, d1 = {f1 * 0x1p24f, f1 * 0x1p20f};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bf16x8_t a0 = dequant_half(wa[s][i], d0, e0), a1 = dequant_half(wb[s][i], d1, e1);
                            const bf16x8_t b = *(const bf16x8_t*)(xq + (DOWN ? i * 1024 : (int)(x_low ^ i * 16)));
                            acc[0] = mfma_16x16x32(a0, b, acc[0]);
                            acc[1] = mfma_16x16x32(a1, b, acc[1]);
                            if constexpr (DOWN) {
                                const bf16x8_t l = *(const bf16x8_t*)(xq + 4096 + i * 1024);
                                acc[0] = mfma_16x16x32(a0, l, acc[0]);
                                acc[1] = mfma_16x16x32(a1, l, acc[1]);
                            }
                        }
                        fetch(s, q0 + s + kBmAhead);
                    }
                }
            }
            if (on) {
                if constexpr (DOWN) {   // fp32 rows: of the token's expert, or the token's shared expert
                    float* o = p.rows + (size_t)(sh ? n + t : at) * H + row0 + g * 4;
                    *(f32x4_t*)o = acc[0];
                    *(f32x4_t*)(o + 16) = acc[1];
                } else {
                    uint16_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) split_bf16(wt * (silu_f32(acc[0][i]) * acc[1][i]), &hi[i], &lo[i]);
                    const size_t at_h = (sh ? p.sh_h + (size_t)vv * ((p.I_sh + 127) / 128) * 2048
                                            : (size_t)(vv - sh_n) * ((p.I + 127) / 128) * 2048) +
                                        h_place(row0 + g * 4, c);
                    *(u32x2_t*)(p.h_hi + at_h) = u32x2_t{(uint32_t)hi[0] | (uint32_t)hi[1] << 16,
                                                         (uint32_t)hi[2] | (uint32_t)hi[3] << 16};
                    *(u32x2_t*)(p.h_lo + at_h) = u32x2_t{(uint32_t)lo[0] | (uint32_t)lo[1] << 16,
                                                         (uint32_t)lo[2] | (uint32_t)lo[3] << 16};
                }
            }
        }
        pos += count;
        tile += count;
        while (pos < last && tile >= tiles_of(v)) tile -= tiles_of(v++);
    }
}

// y = the sum of a token's rows, the shared expert's last, rounded once.
__global__ __launch_bounds__(256) void batch_join_kernel(const float* rows, int T, int k, int H, int shared, uint16_t* y) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= (size_t)T * H) return;
    const int t = (int)(i / H), h = (int)(i - (size_t)t * H);
    const float* row = rows + (size_t)t * k * H + h;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (shared) v = *(const f32x4_t*)(rows + ((size_t)T * k + t) * H + h);
#pragma unroll 8
    for (int j = 0; j < k; ++j) v += *(const f32x4_t*)(row + (size_t)j * H);
    *(u32x2_t*)(y + i) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Tokens whose gate/up workgroups each repeat the selection, a wave for each, and whose down products
// keep the sum over the experts in the accumulators.
constexpr int kBatchColumns = 8;

static int batch_tiles(int T, int E, int k) {   // entries of the list at most
    const int n = T * k, slots = E < n ? E : n;
    return slots + (T > kBatchDense ? n / 16 : 0);
}

BatchWs batch_ws_layout(int T, int H, int I, int I_sh, int E, int k) {
    BatchWs w{};
    const size_t n = (size_t)T * k;
    w.tiles = batch_tiles(T, E, k);
    w.sh_h = (size_t)w.tiles * ((I + 127) / 128) * 2048;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 256);
        return at;
    };
    const size_t values = w.sh_h + (size_t)((T + 15) / 16) * ((I_sh + 127) / 128) * 2048;
    w.h_hi = take(values * 2);
    w.h_lo = take(values * 2);
    w.list = take((size_t)w.tiles * 16);
    w.n_list = take(4);
    w.assign = take((size_t)w.tiles * 16 * 4);
    w.rows = take(T > kBatchColumns ? (n + T) * H * 4 : 0);
    w.idx = take(n * 4);
    w.w = take(n * 4);
    w.total = o;
    return w;
}

template <int EPL>
static void launch_batch_gateup(const BatchArgs& a, hipStream_t stream) {
    const int chunks = (a.H + 127) / 128;
    // a wave takes two chunks of K or more, where there are so many
    const int rt_log = chunks >= 8 ? 0 : chunks >= 4 ? 1 : 2;
    const int x_all = (a.T + 3) / 4 * chunks, x_kb = x_all < 32 ? x_all : 32;
    const int tasks = (a.I_sh >> (4 + rt_log)) + a.tiles * (a.I >> (4 + rt_log));
    const size_t lds = (size_t)x_kb * 1024 + kBgWaves * 4096 + (size_t)a.tiles * 16 + (size_t)a.T * a.k * 8;
    const bool packed = a.gate.layout == 2;
    // a task each for as many workgroups as the chip holds (160 KB of LDS a compute unit), else runs of
    // tasks for two a compute unit: 2 tokens' 544 tasks 15.5 us at once, 16.8 in runs, 4 tokens' 1000
    // tasks 18.6 in runs for 768 workgroups and 16.4 for 512
    const int most = bg_per_simd(EPL, packed) == 6 && lds + 64 <= 160 * 1024 / 3 ? 768 : 512;
    const int grid = tasks <= most ? tasks : 512;
    if (packed)
        batch_gateup_kernel<EPL, true><<<grid, kBgWaves * WAVE, lds, stream>>>(a, x_kb, rt_log);
    else
        batch_gateup_kernel<EPL, false><<<grid, kBgWaves * WAVE, lds, stream>>>(a, x_kb, rt_log);
}

hipError_t launch_decode_batch(const BatchArgs& a, hipStream_t stream) {
    const int epl = (a.E + WAVE - 1) / WAVE;
    hipError_t err;
    if (a.T <= kBatchColumns) {
        if (epl <= 1) launch_batch_gateup<1>(a, stream);
        else if (epl <= 2) launch_batch_gateup<2>(a, stream);
        else if (epl <= 4) launch_batch_gateup<4>(a, stream);
        else if (epl <= 8) launch_batch_gateup<8>(a, stream);
        else launch_batch_gateup<16>(a, stream);
        if ((err = hipGetLastError()) != hipSuccess) return err;
        batch_down_kernel<<<a.H / 8, kBdWaves * WAVE, 0, stream>>>(a);
        return hipGetLastError();
    }
    const int sel = (a.T + kBsWaves - 1) / kBsWaves;
    if (epl <= 1) batch_select_kernel<1><<<sel, kBsWaves * WAVE, 0, stream>>>(a);
    else if (epl <= 2) batch_select_kernel<2><<<sel, kBsWaves * WAVE, 0, stream>>>(a);
    else if (epl <= 4) batch_select_kernel<4><<<sel, kBsWaves * WAVE, 0, stream>>>(a);
    else if (epl <= 8) batch_select_kernel<8><<<sel, kBsWaves * WAVE, 0, stream>>>(a);
    else batch_select_kernel<16><<<sel, kBsWaves * WAVE, 0, stream>>>(a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    // a workgroup for each compute unit; 160 KB of LDS less the lists
    constexpr int kGrid = 256, kLds = 156 * 1024;
    const size_t lists = (size_t)a.tiles * 16 + (size_t)a.T * a.k * 2;
    const int x_kb = (int)((kLds - lists) / 1024) < 128 ? (int)((kLds - lists) / 1024) : 128;
    const size_t lds = (size_t)x_kb * 1024 + lists;
    if (a.gate.layout == 2)
        batch_tiles_kernel<false, true><<<kGrid, kBmWaves * WAVE, lds, stream>>>(a, x_kb);
    else
        batch_tiles_kernel<false, false><<<kGrid, kBmWaves * WAVE, lds, stream>>>(a, x_kb);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    batch_tiles_kernel<true, false><<<kGrid, kBmWaves * WAVE, 128 * 1024, stream>>>(a, 128);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    const unsigned blocks = (unsigned)(((size_t)a.T * a.H / 4 + 255) / 256);
    batch_join_kernel<<<blocks, 256, 0, stream>>>(a.rows, a.T, a.k, a.H, a.I_sh > 0, a.y);
    return hipGetLastError();
}

}  // namespace moeq4
