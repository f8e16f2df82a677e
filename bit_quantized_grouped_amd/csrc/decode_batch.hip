// A few tokens (1 to 64) together through the whole 4-bit layer: the selection (inside the
// first kernel, or a launch of its own), gate/up, and down with the weighted sum.
//
//   y_t = sum_j w_tj FFN_e(t,j)(x_t) + g_t FFN_shared(x_t),  FFN(x) = (silu(x Wg^T) * x Wu^T) Wd^T
//
// Each chosen expert's weights are read once, whatever number of its tokens: a weight tile
// is the A operand of the matrix instruction, 16 rows by 32 K, and the expert's tokens are
// the 16 columns of B.  So a weight costs its dequantization, 19 instructions for 8, and the
// number of tokens nothing; both sides of the sum are bf16 exactly as the format says
// (w = bf16(q * s + b), x), products and sums in fp32.
//
//   batch_gateup_kernel: every workgroup groups the T * k assignments by expert in LDS (a
//     64-bit mask of tokens for each expert, a scan over the experts), then takes row tiles
//     of the experts in turn, its waves splitting rows and K, and writes h = w * silu(g) * u.
//     h already holds the token's weight, and is kept as two bf16 (16 bits), so that y
//     has the one rounding of its own.  Workgroup 0 also writes the grouping for down.
//   batch_down_kernel: a workgroup owns 8 columns of y for all tokens and sums over all
//     experts: the products' columns are the tokens, so the sum over experts stays in the
//     accumulators.  The 16 x 16 product is used as two of 8 x 8: rows and columns 8 .. 15
//     hold the same 8 columns of y and tokens at a K 128 further on.
#include <type_traits>

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
    const uint16_t bits = __builtin_bit_cast(uint16_t, h);
    const float rest = (bits & 0x7F80u) == 0x7F80u ? 0.f : v - (float)h;   // an infinity has no rest
    *hi = bits;
    *lo = __builtin_bit_cast(uint16_t, (__bf16)rest);
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

// EPL > 0: selects too, for at most 8 tokens.  x_kb: LDS for x, in pieces of 4 tokens by 128 K.
// rt_log: a task is 16 << rt_log rows of an entry, 16 a wave, and the other waves split K.  A
// workgroup's tasks lie together, so that x changes seldom, and the waves fetch the next task's
// weights before they are done with this one's.
template <int EPL, bool SB>
__global__ __launch_bounds__(EPL ? 512 : 1024, 4) void batch_gateup_kernel(BatchArgs p, int x_kb, int rt_log) {
    constexpr int NW = EPL ? 8 : 16, THREADS = NW * WAVE;
    typedef typename std::conditional<(EPL > 0), int32_t, uint16_t>::type idx_t;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    __shared__ uint8_t s_tok[NW][WAVE];
    __shared__ int s_total[NW];
    const int T = p.T, E = p.E, k = p.k, n = T * k, H = p.H;
    const bool dense = T <= kBatchDense;
    char* s_x = s_dyn;
    f32x4_t* s_part = (f32x4_t*)(s_x + x_kb * 1024);                 // [2][NW][2][WAVE]
    uint4* s_list = (uint4*)(s_part + 2 * NW * 2 * WAVE);            // expert, -, mask of tokens
    float* s_w = (float*)(s_list + p.tiles);                         // EPL > 0 only
    idx_t* s_idx = (idx_t*)(s_w + (EPL ? n : 0));
    unsigned long long* s_mask = (unsigned long long*)s_part;        // [E], before the products
    const int tid = threadIdx.x, lane = tid % WAVE, g = lane / 16, c = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int chunks = (H + 127) / 128;
    const buf_rsrc_t rx = make_buf(p.x, (uint32_t)T * H * 2);

    // x of the entry's `rows` tokens, chunks c0 .. + len: 16 bytes of token r, piece j of a chunk lie at
    // place j ^ r, so that the 16 tokens' pieces that a product reads at once are in different banks
    auto stage_x = [&](int rows, int c0, int len) {
        const int nq = (rows + 3) / 4;
        for (int i = wave; i < len * nq; i += NW) {
            const int q = i / nq, r = (i - q * nq) * 4 + g;
            const int kk = (c0 + q) * 128 + (c ^ r) * 8;
            const int t = dense ? r : s_tok[wave][r];
            const bool in = r < rows && kk < H;
            buf_to_lds16(rx, s_x + i * 1024, in ? ((uint32_t)t * H + kk) * 2 : 0xFFFFFFF0u, 0);
        }
    };
    int staged = -1;   // entry and segment of x in LDS
    if (dense) {
        const int s = x_kb / ((T + 3) / 4);
        stage_x(T, 0, s < chunks ? s : chunks);
        staged = 0;
    }

    // ---- selection and grouping ----
    for (int e = tid; e < E; e += THREADS) s_mask[e] = 0;
    if constexpr (EPL > 0) {
        static_assert(NW * 4096 >= 1024 * 8 + NW * 3 * kScoredMaxK * 4, "scratch behind the masks");
        if (wave < T)
            batch_select_token<EPL>(p, wave, s_idx + wave * k, s_w + wave * k,
                                    (uint32_t*)(s_mask + E) + wave * 3 * kScoredMaxK);
    } else {
        for (int a = tid; a < n; a += THREADS) s_idx[a] = (uint16_t)p.topk_idx[a];
    }
    __syncthreads();
    for (int a = tid; a < n; a += THREADS) atomicOr(&s_mask[s_idx[a]], 1ull << (a / k));
    __syncthreads();
    int used = 0;
    for (int e0 = 0; e0 < E; e0 += THREADS) {
        const int e = e0 + tid;
        unsigned long long m = e < E ? s_mask[e] : 0ull;
        const int mine = !m ? 0 : dense ? 1 : (__popcll(m) + 15) / 16;
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
    if (blockIdx.x == 0) {
        for (int u = tid; u < used; u += THREADS) p.list[u] = s_list[u];
        if (tid == 0) *p.n_list = used;
        if constexpr (EPL > 0)
            for (int a = tid; a < n; a += THREADS) {
                p.topk_idx[a] = s_idx[a];
                p.topk_w[a] = s_w[a];
            }
    }

    // ---- tasks: row tiles of the shared expert's entries, then of the list's ----
    const int KS = NW >> rt_log, rt = wave & ((1 << rt_log) - 1), ks = wave >> rt_log;
    const int ks_log = 31 - __builtin_clz(KS);
    const int sh_n = !p.I_sh ? 0 : dense ? 1 : (T + 15) / 16;
    const int sh_tiles = p.I_sh >> (4 + rt_log), tiles = p.I >> (4 + rt_log);
    const int tasks = sh_n * sh_tiles + used * tiles;
    const int last = (int)((long long)tasks * (blockIdx.x + 1) / gridDim.x);
    const int G = H / 64;
    const float unit_inv = 1.0f / fp8_unit();
    const bool half_chunk = H % 128 != 0;   // the last chunk's groups g >= 2 lie behind K
    int task = (int)((long long)tasks * blockIdx.x / gridDim.x);
    int v = 0, tile = 0;
    if (task < last) {
        const int r = task - sh_n * sh_tiles;
        v = r < 0 ? task / sh_tiles : sh_n + r / tiles;
        tile = r < 0 ? task - v * sh_tiles : r - (v - sh_n) * tiles;
    }
    struct Entry {
        int expert, rows, nq, per_seg;   // nq: pieces of 4 tokens; per_seg: chunks of x in LDS
        unsigned long long mask;
    };
    auto entry = [&](int v) {
        Entry o;
        if (v < sh_n) {
            o.expert = 0;
            o.mask = shared_mask(T, v);
        } else {
            const uint4 ent = s_list[v - sh_n];
            o.expert = __builtin_amdgcn_readfirstlane((int)ent.x);
            o.mask = (unsigned long long)(uint32_t)__builtin_amdgcn_readfirstlane((int)ent.w) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)ent.z);
        }
        o.rows = dense ? T : __popcll(o.mask);
        o.nq = (o.rows + 3) / 4;
        o.per_seg = o.nq == 1 ? x_kb : o.nq == 2 ? x_kb / 2 : o.nq == 3 ? x_kb / 3 : x_kb / 4;
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
            const int c0 = l_seg * l_ent.per_seg, len = min(l_ent.per_seg, chunks - c0);
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
        if (half_chunk && l_q == chunks - 1) {   // an address of the row, whose weights are not used
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
    if (dense) {
        wait_loads<0>();
        __syncthreads();
    }
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    int turn = 0;   // the task's number here: the waves that join its sums, where these lie
    for (; task < last; ++v, tile = 0) {
        const Entry ent = entry(v);
        const bool sh = v < sh_n;
        // columns behind the last token read any one's x
        const int cx = c < ent.nq * 4 ? c : 0;
        const char* x_lane = s_x + cx / 4 * 1024 + cx % 4 * 256 + (g * 4 ^ (cx & 12)) * 16;
        const int x_low = (cx & 3) * 16;
        for (const int n_tiles = sh ? sh_tiles : tiles; tile < n_tiles && task < last; ++tile, ++task, ++turn) {
            const bool joins = ks == (turn & (KS - 1));
            float wt = 1.f;   // the weight of the column's token
            bool on = false;
            for (int c0 = 0; c0 < chunks; c0 += ent.per_seg) {
                const int len = min(ent.per_seg, chunks - c0), want = (dense ? 0 : v) * chunks + c0;
                if (want != staged) {
                    __syncthreads();
                    if (!dense) list_tokens(ent.mask, s_tok[wave], lane);
                    stage_x(ent.rows, c0, len);
                    staged = want;
                    wait_loads<0>();
                    __syncthreads();
                }
                if (joins && c0 == 0) {
                    on = dense ? ent.mask >> c & 1 : c < ent.rows;
                    const int t = !on ? 0 : dense ? c : s_tok[wave][c];
                    if (sh) {
                        if (p.shared_gate) wt = p.shared_gate[t];
                    } else {
                        int a = -1;   // the lanes of a column share the search
#pragma unroll 2
                        for (int j = g; j < k; j += 4)
                            if (s_idx[t * k + j] == ent.expert) a = t * k + j;
                        a = max(a, __shfl_xor(a, 16));
                        a = max(a, __shfl_xor(a, 32));
                        wt = on ? EPL ? s_w[a] : p.topk_w[a] : 0.f;
                    }
                }
                const int q1 = c0 + (len * (ks + 1) >> ks_log);
                for (int q = c0 + (len * ks >> ks_log); q < q1; ++q) {
                    Chunk w2 = w1;
                    fetch(w2);
                    const char* xq = x_lane + (q - c0) * ent.nq * 1024;
                    float sg = bf16_to_f32((uint16_t)w0.sg) * unit_inv, su = bf16_to_f32((uint16_t)w0.su) * unit_inv;
                    float bg = bf16_to_f32((uint16_t)(SB ? w0.sg >> 16 : w0.bg));
                    float bu = bf16_to_f32((uint16_t)(SB ? w0.su >> 16 : w0.bu));
                    if (half_chunk && q == chunks - 1) {
                        sg = g >= 2 ? 0.f : sg;
                        su = g >= 2 ? 0.f : su;
                        bg = g >= 2 ? 0.f : bg;
                        bu = g >= 2 ? 0.f : bu;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8_t b = *(const bf16x8_t*)(xq + (x_low ^ i * 16));
                        acc[0] = mfma_16x16x32(dequant_word(w0.wg[i], sg, bg), b, acc[0]);
                        acc[1] = mfma_16x16x32(dequant_word(w0.wu[i], su, bu), b, acc[1]);
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
                const size_t at_h = (sh ? p.sh_h + (size_t)v * ((p.I_sh + 127) / 128) * 2048
                                        : (size_t)(v - sh_n) * ((p.I + 127) / 128) * 2048) +
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
    const float unit_inv = 1.0f / fp8_unit();
    u32x4_t wv[kBdAhead];
    float sc[kBdAhead], bi[kBdAhead];
    bool on[kBdAhead];         // the lane's token is the entry's, and its K in range
    size_t h_at[kBdAhead];
    auto load = [&](int s, int step) {
        const bool in = step < steps, sh = step >= routed;
        const int u = in && !sh ? step / per : 0;
        const int d = sh ? step - routed : step - u * per;
        uint4 ent = {0, 0, 0xFF, 0};
        if (in && !sh) ent = p.list[u];
        const int K = sh ? I_sh : I, kb = d * 256 + half * 128 + g * 32;
        on[s] = in && kb < K && c < T && (ent.z >> c & 1);
        h_at[s] = (sh ? p.sh_h : (size_t)u * ((I + 127) / 128) * 2048) + (size_t)(d * 2 + half) * 2048 +
                  (g * 16 + c) * 8;
        const QMatDev& m = sh ? p.sh_down : p.down;
        const size_t row = (size_t)ent.x * H + col;
        wv[s] = in && kb < K ? *(const u32x4_t*)(m.codes + (size_t)ent.x * H * (K / 8) +
                                                 code_word(m.layout, col, kb / 8, K))
                             : u32x4_t{0, 0, 0, 0};
        sc[s] = in && kb < K ? bf16_to_f32(m.scales[row * (K / 64) + kb / 64]) : 0.f;
        bi[s] = in && kb < K ? bf16_to_f32(m.biases[row * (K / 64) + kb / 64]) : 0.f;
    };
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kBdAhead; ++s) load(s, wave + s * kBdWaves);
    for (int step = wave; step < steps; step += kBdAhead * kBdWaves) {
#pragma unroll
        for (int s = 0; s < kBdAhead; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4_t hi = on[s] ? *(const u32x4_t*)(p.h_hi + h_at[s] + i * 512) : u32x4_t{0, 0, 0, 0};
                const u32x4_t lo = on[s] ? *(const u32x4_t*)(p.h_lo + h_at[s] + i * 512) : u32x4_t{0, 0, 0, 0};
                const bf16x8_t w = dequant_word(wv[s][i], sc[s] * unit_inv, bi[s]);
                acc = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, hi), acc);
                acc = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, lo), acc);
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

// ---- Down for more tokens: a workgroup owns 64 columns and a share of the entries' 128-K blocks, so
// that h is read by H / 64 workgroups instead of H / 8.  The 64 columns' codes of a block are two
// runs of 2 KB (tiles), its h four contiguous KB twice; a wave's blocks lie together, and an entry's sums go to
// the tokens' rows in the wave's part of LDS.  The workgroups' sums meet in batch_join_kernel.
constexpr int kBpWaves = 8;

// VEC: K a multiple of 128, so that the two scales of a row and block are one load.
template <bool VEC>
__global__ __launch_bounds__(kBpWaves* WAVE) void batch_down_split_kernel(BatchArgs p, int splits) {
    extern __shared__ __attribute__((aligned(16))) float s_y[];   // [waves][T][64 + 4]
    __shared__ uint8_t s_tok[kBpWaves][WAVE];
    constexpr int LDY = 68;
    const int tid = threadIdx.x, lane = tid % WAVE, g = lane / 16, c = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int T = p.T, H = p.H, I = p.I, I_sh = p.I_sh;
    const bool dense = T <= kBatchDense;
    const int cols = H / 64, cg = blockIdx.x % cols, split = blockIdx.x / cols;
    const int per = (I + 127) / 128, per_sh = (I_sh + 127) / 128;
    const float unit_inv = 1.0f / fp8_unit();
    const int sh_steps = !I_sh ? 0 : (dense ? 1 : (T + 15) / 16) * per_sh;
    const int steps = sh_steps + *p.n_list * per;
    const int share = splits * kBpWaves, mine = split * kBpWaves + wave;
    const int first = (int)((long long)steps * mine / share), last = (int)((long long)steps * (mine + 1) / share);
    float* y = s_y + wave * T * LDY;
    // the next block to fetch: block d of entry u, the shared expert's below 0
    int step = first, u, d;
    if (first < sh_steps) {
        u = first / per_sh;
        d = first - u * per_sh;
        u -= sh_steps / per_sh;
    } else {
        u = (first - sh_steps) / per;
        d = first - sh_steps - u * per;
    }
    // the list 64 entries at a time, one a lane
    int list0 = u < 0 ? 0 : u;
    auto fetch_list = [&]() {
        return list0 + lane < p.tiles ? p.list[list0 + lane] : uint4{0, 0, 0, 0};
    };
    uint4 window = first < last ? fetch_list() : uint4{0, 0, 0, 0};
    u32x4_t wv[2][4], hi[2][4], lo[2][4];
    uint32_t sc[2][4], bi[2][4];
    unsigned long long mask[2];
    bool valid[2], ends[2];       // a block is there; it is the entry's last of this wave
    auto load = [&](int s) {
        const bool on = step < last, sh = u < 0;
        const int K = sh ? I_sh : I;
        uint32_t e = 0;
        if (sh) {
            mask[s] = shared_mask(T, u + (dense ? 1 : (T + 15) / 16));
        } else {
            if (u >= list0 + WAVE && on) {
                list0 = u;
                window = fetch_list();
            }
            e = __builtin_amdgcn_readlane(window.x, u - list0);
            mask[s] = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane(window.w, u - list0) << 32 |
                      (uint32_t)__builtin_amdgcn_readlane(window.z, u - list0);
        }
        const QMatDev& m = sh ? p.sh_down : p.down;
        const bool in = on && d * 128 + g * 32 < K;
        // four column tiles of 16: 512 bytes apart in tiles, 2 K words in rows
        const uint32_t* codes = m.codes + (size_t)e * H * (K / 8) + code_word(m.layout, cg * 64, d * 16, K);
        const uint32_t w_lane = code_word(m.layout, c, g * 4, K);
        const uint32_t t_step = m.layout ? 128u : 2u * K;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            wv[s][t] = in ? *(const u32x4_t*)(codes + (w_lane + t * t_step)) : u32x4_t{0, 0, 0, 0};
        const uint32_t groups = K / 64;
        const size_t s0 = ((size_t)e * H + cg * 64) * groups + d * 2;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t at = (t * 16 + c) * groups;
            if constexpr (VEC) {   // the groups of both halves of the wave
                sc[s][t] = on ? *(const uint32_t*)(m.scales + s0 + at) : 0u;
                bi[s][t] = on ? *(const uint32_t*)(m.biases + s0 + at) : 0u;
            } else {               // this lane's
                sc[s][t] = in ? (m.scales + s0)[at + g / 2] : 0u;
                bi[s][t] = in ? (m.biases + s0)[at + g / 2] : 0u;
            }
        }
        const size_t h0 = (sh ? p.sh_h + (size_t)(u + (dense ? 1 : (T + 15) / 16)) * per_sh * 2048
                              : (size_t)u * per * 2048) + (size_t)d * 2048;
        const bool col = in && (dense ? mask[s] >> c & 1 : c < __popcll(mask[s]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[s][i] = col ? *(const u32x4_t*)(p.h_hi + h0 + (i * 512 + lane * 8)) : u32x4_t{0, 0, 0, 0};
            lo[s][i] = col ? *(const u32x4_t*)(p.h_lo + h0 + (i * 512 + lane * 8)) : u32x4_t{0, 0, 0, 0};
        }
        valid[s] = on;
        ++step;
        ++d;
        ends[s] = step >= last || d == (sh ? per_sh : per);
        if (d == (sh ? per_sh : per)) {
            d = 0;
            ++u;
        }
    };
    f32x4_t acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int i = lane; i < T * LDY / 4; i += WAVE) ((f32x4_t*)y)[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // two slots, each fetched before the other's products: the first round's first slot holds nothing
    valid[0] = false;
    do {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            load(1 - s);
            if (!valid[s]) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float sv = VEC ? __builtin_bit_cast(float, g < 2 ? sc[s][t] << 16 : sc[s][t] & 0xFFFF0000u)
                                     : bf16_to_f32((uint16_t)sc[s][t]);
                const float bv = VEC ? __builtin_bit_cast(float, g < 2 ? bi[s][t] << 16 : bi[s][t] & 0xFFFF0000u)
                                     : bf16_to_f32((uint16_t)bi[s][t]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf16x8_t w = dequant_word(wv[s][t][i], sv * unit_inv, bv);
                    acc[t] = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, hi[s][i]), acc[t]);
                    acc[t] = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, lo[s][i]), acc[t]);
                }
            }
            if (ends[s]) {   // to the tokens' rows: the lanes have different places
                int row = c;
                bool col = mask[s] >> c & 1;
                if (!dense) {
                    list_tokens(mask[s], s_tok[wave], lane);
                    col = c < __popcll(mask[s]);
                    row = col ? s_tok[wave][c] : 0;
                }
                if (col) {
                    float* o = y + row * LDY + g * 4;
#pragma unroll
                    for (int t = 0; t < 4; ++t) *(f32x4_t*)(o + t * 16) = *(const f32x4_t*)(o + t * 16) + acc[t];
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();   // the next entry's tokens take these ones' place
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
        }
    } while (valid[0]);
    __syncthreads();
    for (int i = tid; i < T * 64; i += kBpWaves * WAVE) {
        const int t = i / 64, n = i % 64;
        float v = s_y[t * LDY + n];
#pragma unroll
        for (int w = 1; w < kBpWaves; ++w) v += s_y[(w * T + t) * LDY + n];
        p.y_part[((size_t)split * T + t) * H + cg * 64 + n] = v;
    }
}

// The shares' sums, in order, rounded once.
__global__ __launch_bounds__(256) void batch_join_kernel(const float* part, int splits, size_t n, uint16_t* y) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4_t v = *(const f32x4_t*)(part + i);
#pragma unroll 8
    for (int s = 1; s < splits; ++s) v += *(const f32x4_t*)(part + s * n + i);
    *(u32x2_t*)(y + i) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Shares of the experts: a workgroup for each compute unit.
static int batch_splits(int H) {
    const int s = 256 / (H / 64);
    return s < 1 ? 1 : s < 16 ? s : 16;
}

// Tokens whose selection every gate/up workgroup repeats, one a wave.
constexpr int kBatchOwnSelect = 8;
// Tokens whose down products keep the sum over the experts in the accumulators.
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
    w.y_part = take((size_t)batch_splits(H) * T * H * 4);
    w.idx = take(n * 4);
    w.w = take(n * 4);
    w.total = o;
    return w;
}

template <int EPL>
static void launch_batch_gateup(const BatchArgs& a, hipStream_t stream) {
    constexpr int NW = EPL ? 8 : 16;
    const int chunks = (a.H + 127) / 128;
    // a wave takes two chunks of K or more, where there are so many
    const int rt_log = (chunks >= 8 ? 0 : chunks >= 4 ? 1 : 2) + (EPL || chunks < 8 ? 0 : 1);
    const int want = (a.T < 16 ? (a.T + 3) / 4 : 4) * chunks, most = EPL ? 32 : 64;
    const int x_kb = want < most ? want : most;
    const int sh_n = a.T > kBatchDense ? (a.T + 15) / 16 : 1;
    const int tasks = (sh_n * a.I_sh + a.tiles * a.I) >> (4 + rt_log), resident = EPL ? 512 : 256;
    const int grid = tasks < resident ? tasks : resident;
    const size_t lds = (size_t)x_kb * 1024 + NW * 4096 + (size_t)a.tiles * 16 + (size_t)a.T * a.k * (EPL ? 8 : 2);
    if (a.gate.layout == 2)
        batch_gateup_kernel<EPL, true><<<grid, NW * WAVE, lds, stream>>>(a, x_kb, rt_log);
    else
        batch_gateup_kernel<EPL, false><<<grid, NW * WAVE, lds, stream>>>(a, x_kb, rt_log);
}

hipError_t launch_decode_batch(const BatchArgs& a, hipStream_t stream) {
    const int epl = (a.E + WAVE - 1) / WAVE;
    hipError_t err;
    if (a.T > kBatchOwnSelect) {
        const int grid = (a.T + kBsWaves - 1) / kBsWaves;
#define MOE_SEL(N) batch_select_kernel<N><<<grid, kBsWaves * WAVE, 0, stream>>>(a)
        if (epl <= 1) MOE_SEL(1);
        else if (epl <= 2) MOE_SEL(2);
        else if (epl <= 4) MOE_SEL(4);
        else if (epl <= 8) MOE_SEL(8);
        else MOE_SEL(16);
#undef MOE_SEL
        if ((err = hipGetLastError()) != hipSuccess) return err;
        launch_batch_gateup<0>(a, stream);
    } else if (epl <= 1) launch_batch_gateup<1>(a, stream);
    else if (epl <= 2) launch_batch_gateup<2>(a, stream);
    else if (epl <= 4) launch_batch_gateup<4>(a, stream);
    else if (epl <= 8) launch_batch_gateup<8>(a, stream);
    else launch_batch_gateup<16>(a, stream);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    if (a.T > kBatchColumns) {
        const int splits = batch_splits(a.H), grid2 = a.H / 64 * splits;
        const size_t lds2 = (size_t)kBpWaves * a.T * 68 * 4;
        // pairs of scales as one load: even rows, and arrays that start at 4 bytes
        auto even = [](const QMatDev& m) { return ((uintptr_t)m.scales | (uintptr_t)m.biases) % 4 == 0; };
        if (a.I % 128 == 0 && a.I_sh % 128 == 0 && even(a.down) && even(a.sh_down))
            batch_down_split_kernel<true><<<grid2, kBpWaves * WAVE, lds2, stream>>>(a, splits);
        else
            batch_down_split_kernel<false><<<grid2, kBpWaves * WAVE, lds2, stream>>>(a, splits);
        if ((err = hipGetLastError()) != hipSuccess) return err;
        const size_t n_y = (size_t)a.T * a.H;
        batch_join_kernel<<<(unsigned)((n_y / 4 + 255) / 256), 256, 0, stream>>>(a.y_part, splits, n_y, a.y);
        return hipGetLastError();
    }
    batch_down_kernel<<<a.H / 8, kBdWaves * WAVE, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moeq4
