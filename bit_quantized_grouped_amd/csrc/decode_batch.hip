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
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_score.h"

namespace moeq4 {

constexpr int kBgWaves = 8;              // waves of a gate/up workgroup
constexpr int kBgThreads = kBgWaves * WAVE;
constexpr int kBgResident = 512;        // workgroups that the chip holds, two a compute unit
constexpr int kBgAhead = 2;              // 128-K chunks of a wave in flight
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

// EPL 0: the experts are chosen already.  rt: row tiles of 16 that a workgroup's waves take side
// by side (1, 2 or 4); 8 / rt waves split K.  More than 16 tokens of an expert take its rows again
// from the caches for each 16: the shared expert mostly, whose rows are few beside the others'.
template <int EPL, bool SB>
__global__ __launch_bounds__(kBgThreads, 4) void batch_gateup_kernel(BatchArgs p, int rt_log) {
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    __shared__ f32x4_t s_part[kBgWaves][2][WAVE];
    __shared__ uint32_t s_scr[EPL ? kBgWaves : 1][3 * kScoredMaxK];
    __shared__ int s_tok[kBgWaves][WAVE];
    __shared__ int s_total[kBgWaves];
    const int T = p.T, E = p.E, k = p.k, n = T * k, H = p.H;
    const int slots = E < n ? E : n;
    uint4* s_list = (uint4*)s_dyn;                             // expert, first row, mask of tokens
    unsigned long long* s_mask = (unsigned long long*)(s_list + slots);
    int* s_idx = (int*)(s_mask + E);
    float* s_w = (float*)(s_idx + n);                          // EPL > 0 only
    const float* wts = EPL ? s_w : p.topk_w;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);

    // ---- selection and grouping ----
    for (int e = tid; e < E; e += kBgThreads) s_mask[e] = 0;
    if constexpr (EPL > 0) {
        for (int t = wave; t < T; t += kBgWaves)
            batch_select_token<EPL>(p, t, s_idx + t * k, s_w + t * k, s_scr[wave]);
    } else {
        for (int a = tid; a < n; a += kBgThreads) s_idx[a] = p.topk_idx[a];
    }
    __syncthreads();
    for (int a = tid; a < n; a += kBgThreads) atomicOr(&s_mask[s_idx[a]], 1ull << (a / k));
    __syncthreads();
    int used = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += kBgThreads) {
        const int e = e0 + tid;
        const unsigned long long m = e < E ? s_mask[e] : 0ull;
        const int mine = m ? 1 << 16 | __popcll(m) : 0;   // experts and rows, both below 2^16
        const int upto = wave_incl_sum_i32(mine, lane);
        if (lane == WAVE - 1) s_total[wave] = upto;
        __syncthreads();
        int before = upto - mine, all = 0;
#pragma unroll
        for (int w = 0; w < kBgWaves; ++w) {
            const int v = s_total[w];
            before += w < wave ? v : 0;
            all += v;
        }
        if (m)
            s_list[used + (before >> 16)] =
                uint4{(uint32_t)e, (uint32_t)(rows + (before & 0xFFFF)), (uint32_t)m, (uint32_t)(m >> 32)};
        used += all >> 16;
        rows += all & 0xFFFF;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int u = tid; u < used; u += kBgThreads) p.list[u] = s_list[u];
        if (tid == 0) *p.n_list = used;
        if constexpr (EPL > 0)
            for (int a = tid; a < n; a += kBgThreads) {
                p.topk_idx[a] = s_idx[a];
                p.topk_w[a] = s_w[a];
            }
    }

    // ---- row tiles: the shared expert's, then those of the experts in turn ----
    const int RT = 1 << rt_log, KS = kBgWaves >> rt_log;
    const int rt = wave & (RT - 1), ks = wave >> rt_log;
    const int g = lane / 16, c = lane % 16;
    const int sh_tiles = p.I_sh >> (4 + rt_log), tiles = p.I >> (4 + rt_log);
    const int tasks = sh_tiles + used * tiles;
    const int chunks = (H + 127) / 128, q0 = chunks * ks / KS, q1 = chunks * (ks + 1) / KS;
    const float unit_inv = 1.0f / fp8_unit();
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const bool sh = task < sh_tiles;
        const int u = sh ? 0 : (task - sh_tiles) / tiles;
        const int tile = sh ? task : task - sh_tiles - u * tiles;
        const int N = sh ? p.I_sh : p.I;
        const uint4 ent = s_list[u];
        const int e = sh ? 0 : __builtin_amdgcn_readfirstlane((int)ent.x);
        unsigned long long mask = (unsigned long long)(uint32_t)__builtin_amdgcn_readfirstlane((int)ent.w) << 32 |
                                  (uint32_t)__builtin_amdgcn_readfirstlane((int)ent.z);
        if (sh) mask = ~0ull >> (64 - T);
        const int cnt = __popcll(mask);
        const QMatDev& mg = sh ? p.sh_gate : p.gate;
        const QMatDev& mu = sh ? p.sh_up : p.up;
        const int row0 = ((tile << rt_log) + rt) * 16;
        const size_t grow = (size_t)e * N + row0 + c;
        const size_t ebase = (size_t)e * N * (H / 8);
        const uint32_t w_at = code_word(mg.layout, row0 + c, g * 4, H), w_step = mg.layout ? 1024u : 16u;
        const uint32_t *gc = mg.codes + ebase + w_at, *uc = mu.codes + ebase + w_at;
        const int G = H / 64;
        const size_t s_at = SB ? ((grow / 64) * G + g / 2) * 64 + grow % 64 : grow * G + g / 2;
        // the expert's tokens, in order: the wave's own list
        if (mask >> lane & 1) s_tok[wave][__popcll(mask & lanemask_lt())] = lane;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (int t0 = 0; t0 < cnt; t0 += 16) {
            const int at = t0 + c;
            const bool mine = at < cnt;
            const int t = mine ? s_tok[wave][at] : 0;
            const uint16_t* x0 = p.x + (size_t)t * H;
            u32x4_t wg[kBgAhead], wu[kBgAhead], xv[kBgAhead][4];
            float sg[kBgAhead], bg[kBgAhead], su[kBgAhead], bu[kBgAhead];
            auto load = [&](int s, int q) {
                const int kb = q * 128 + g * 32;
                const bool in = q < q1 && kb < H;
                wg[s] = in ? *(const u32x4_t*)(gc + (size_t)q * w_step) : u32x4_t{0, 0, 0, 0};
                wu[s] = in ? *(const u32x4_t*)(uc + (size_t)q * w_step) : u32x4_t{0, 0, 0, 0};
                if constexpr (SB) {
                    const uint32_t a = in ? ((const uint32_t*)mg.scales)[s_at + (size_t)q * 128] : 0u;
                    const uint32_t b = in ? ((const uint32_t*)mu.scales)[s_at + (size_t)q * 128] : 0u;
                    sg[s] = bf16_to_f32((uint16_t)a);
                    bg[s] = bf16_to_f32((uint16_t)(a >> 16));
                    su[s] = bf16_to_f32((uint16_t)b);
                    bu[s] = bf16_to_f32((uint16_t)(b >> 16));
                } else {
                    sg[s] = in ? bf16_to_f32(mg.scales[s_at + q * 2]) : 0.f;
                    bg[s] = in ? bf16_to_f32(mg.biases[s_at + q * 2]) : 0.f;
                    su[s] = in ? bf16_to_f32(mu.scales[s_at + q * 2]) : 0.f;
                    bu[s] = in ? bf16_to_f32(mu.biases[s_at + q * 2]) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    xv[s][i] = in && mine ? *(const u32x4_t*)(x0 + kb + 8 * i) : u32x4_t{0, 0, 0, 0};
            };
            f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int s = 0; s < kBgAhead; ++s) load(s, q0 + s);
            for (int q = q0; q < q1; q += kBgAhead) {
#pragma unroll
                for (int s = 0; s < kBgAhead; ++s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8_t b = __builtin_bit_cast(bf16x8_t, xv[s][i]);
                        acc[0] = mfma_16x16x32(dequant_word(wg[s][i], sg[s] * unit_inv, bg[s]), b, acc[0]);
                        acc[1] = mfma_16x16x32(dequant_word(wu[s][i], su[s] * unit_inv, bu[s]), b, acc[1]);
                    }
                    load(s, q + s + kBgAhead);
                }
            }
            // the waves' sums over K in order; 4 rows of one token a lane
            __syncthreads();
            s_part[wave][0][lane] = acc[0];
            s_part[wave][1][lane] = acc[1];
            __syncthreads();
            if (ks == 0 && mine) {
                f32x4_t gs = s_part[rt][0][lane], us = s_part[rt][1][lane];
                for (int i = 1; i < KS; ++i) {
                    gs += s_part[rt + i * RT][0][lane];
                    us += s_part[rt + i * RT][1][lane];
                }
                float wt = 1.f;
                if (sh) {
                    if (p.shared_gate) wt = p.shared_gate[t];
                } else {
                    for (int j = 0; j < k; ++j)
                        if (s_idx[t * k + j] == e) wt = wts[t * k + j];
                }
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split_bf16(wt * (silu_f32(gs[i]) * us[i]), &hi[i], &lo[i]);
                const size_t at_h = (sh ? (size_t)n * p.I + (size_t)t * N : (size_t)(ent.y + at) * N) + row0 + g * 4;
                *(u32x2_t*)(p.h_hi + at_h) = u32x2_t{(uint32_t)hi[0] | (uint32_t)hi[1] << 16,
                                                     (uint32_t)hi[2] | (uint32_t)hi[3] << 16};
                *(u32x2_t*)(p.h_lo + at_h) = u32x2_t{(uint32_t)lo[0] | (uint32_t)lo[1] << 16,
                                                     (uint32_t)lo[2] | (uint32_t)lo[3] << 16};
            }
        }
        __syncthreads();
    }
}

// NT: tiles of 8 tokens.
template <int NT>
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
    const size_t sh_h = (size_t)T * p.k * I;
    u32x4_t wv[kBdAhead];
    float sc[kBdAhead], bi[kBdAhead];
    unsigned long long mask[kBdAhead];
    size_t h_at[kBdAhead];   // the lane's place in h's first row of the expert
    int K[kBdAhead], kb[kBdAhead];
    auto load = [&](int s, int step) {
        const bool on = step < steps, sh = step >= routed;
        const int u = on && !sh ? step / per : 0;
        const int d = sh ? step - routed : step - u * per;
        uint4 ent = {0, 0, 0, 0};
        if (on && !sh) ent = p.list[u];
        mask[s] = !on ? 0ull : sh ? ~0ull >> (64 - T) : (unsigned long long)ent.w << 32 | ent.z;
        K[s] = sh ? I_sh : I;
        kb[s] = d * 256 + half * 128 + g * 32;
        h_at[s] = (sh ? sh_h : (size_t)ent.y * I) + kb[s];
        const QMatDev& m = sh ? p.sh_down : p.down;
        const bool in = on && kb[s] < K[s];
        const size_t row = (size_t)ent.x * H + col;
        wv[s] = in ? *(const u32x4_t*)(m.codes + (size_t)ent.x * H * (K[s] / 8) +
                                       code_word(m.layout, col, kb[s] / 8, K[s]))
                   : u32x4_t{0, 0, 0, 0};
        sc[s] = in ? bf16_to_f32(m.scales[row * (K[s] / 64) + kb[s] / 64]) : 0.f;
        bi[s] = in ? bf16_to_f32(m.biases[row * (K[s] / 64) + kb[s] / 64]) : 0.f;
    };
    f32x4_t acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kBdAhead; ++s) load(s, wave + s * kBdWaves);
    for (int step = wave; step < steps; step += kBdAhead * kBdWaves) {
#pragma unroll
        for (int s = 0; s < kBdAhead; ++s) {
            bf16x8_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = dequant_word(wv[s][i], sc[s] * unit_inv, bi[s]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (!(mask[s] >> (nt * 8) & 0xFF)) continue;
                const int t = nt * 8 + c;
                const bool on = (mask[s] >> t & 1) && kb[s] < K[s];
                const size_t at = h_at[s] + (size_t)__popcll(mask[s] & ((1ull << t) - 1)) * K[s];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4_t hi = on ? *(const u32x4_t*)(p.h_hi + at + 8 * i) : u32x4_t{0, 0, 0, 0};
                    const u32x4_t lo = on ? *(const u32x4_t*)(p.h_lo + at + 8 * i) : u32x4_t{0, 0, 0, 0};
                    acc[nt] = mfma_16x16x32(a[i], __builtin_bit_cast(bf16x8_t, hi), acc[nt]);
                    acc[nt] = mfma_16x16x32(a[i], __builtin_bit_cast(bf16x8_t, lo), acc[nt]);
                }
            }
            load(s, step + (s + kBdAhead) * kBdWaves);
        }
    }
    // the waves' sums in order; rows and columns 0 .. 7 and 8 .. 15 hold two parts of K
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        __syncthreads();
        s_part[wave][lane] = acc[nt];
        __syncthreads();
        if (tid < 64) {
            const int r = tid % 8, t = tid / 8;
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kBdWaves; ++w)
                y += s_part[w][r / 4 * 16 + t][r % 4] + s_part[w][(r + 8) / 4 * 16 + 8 + t][r % 4];
            if (nt * 8 + t < T)
                p.y[(size_t)(nt * 8 + t) * H + blockIdx.x * 8 + r] = (uint16_t)pack_bf16x2(y, 0.f);
        }
    }
}

// ---- Down for more tokens: a workgroup owns 64 columns and a share of the experts, so that h is
// read by H / 64 workgroups instead of H / 8.  A wave takes 128 K of an expert at a time: the
// 64 columns' codes are two runs of 2 KB (tiles), and the product's columns are the expert's
// tokens one after another, whose sums then go to the tokens' rows in the wave's part of
// LDS.  The workgroups' sums meet in batch_join_kernel.
constexpr int kBpWaves = 8, kBpAhead = 3;

// An entry of the list of chosen experts, through scalar loads: the list is another kernel's.
struct BatchEntry {
    uint32_t expert, row;
    unsigned long long mask;   // its tokens
    bool shared;
};
__device__ __forceinline__ BatchEntry batch_entry(const uint4* list, int u) {
    typedef const __attribute__((address_space(4))) u32x4_t* scalar_t;
    const u32x4_t v = ((scalar_t)(uintptr_t)list)[u];
    return BatchEntry{v[0], v[1], (unsigned long long)v[3] << 32 | v[2], false};
}

// VEC: K a multiple of 128, so that the two scales of a row and step are one load.
template <bool VEC>
__global__ __launch_bounds__(kBpWaves* WAVE) void batch_down_split_kernel(BatchArgs p, int splits) {
    extern __shared__ __attribute__((aligned(16))) float s_y[];   // [waves][T][64 + 4]
    __shared__ int s_tok[kBpWaves][WAVE];
    constexpr int LDY = 68;
    const int tid = threadIdx.x, lane = tid % WAVE, g = lane / 16, c = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int T = p.T, H = p.H, I = p.I, I_sh = p.I_sh;
    const int cols = H / 64, cg = blockIdx.x % cols, split = blockIdx.x / cols;
    const int per = (I + 127) / 128, per_sh = (I_sh + 127) / 128;
    const float unit_inv = 1.0f / fp8_unit();
    const size_t sh_h = (size_t)T * p.k * I;
    const int routed = *p.n_list * per, steps = routed + per_sh;
    // this wave's steps lie together, so that an expert's sums stay in registers
    const int share = splits * kBpWaves, mine = split * kBpWaves + wave;
    const int first = (int)((long long)steps * mine / share), last = (int)((long long)steps * (mine + 1) / share);
    float* y = s_y + wave * T * LDY;
    for (int i = lane; i < T * LDY; i += WAVE) y[i] = 0.f;
    u32x4_t wv[kBpAhead][4], hi[kBpAhead][4], lo[kBpAhead][4];
    uint32_t sc[kBpAhead][4], bi[kBpAhead][4];
    BatchEntry ent[kBpAhead];
    int block[kBpAhead], K[kBpAhead];   // uniform over the wave, as the entry
    auto load_h = [&](int s, int at, bool on, u32x4_t (&h)[4], u32x4_t (&l)[4]) {
        const int kb = block[s] * 128 + g * 32;
        // a routed expert's rows lie in order, the shared one's by token
        const size_t from = (ent[s].shared ? sh_h : (size_t)ent[s].row * I) + (size_t)at * K[s] + kb;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = on && kb < K[s] ? *(const u32x4_t*)(p.h_hi + from + 8 * i) : u32x4_t{0, 0, 0, 0};
            l[i] = on && kb < K[s] ? *(const u32x4_t*)(p.h_lo + from + 8 * i) : u32x4_t{0, 0, 0, 0};
        }
    };
    auto load = [&](int s, int step) {
        const bool on = step < last, sh = step >= routed;
        const int u = on && !sh ? step / per : 0;
        const int d = sh ? step - routed : step - u * per;
        ent[s] = batch_entry(p.list, u);
        if (sh) ent[s] = BatchEntry{0, 0, ~0ull >> (64 - T), true};
        if (!on) ent[s].mask = 0;
        K[s] = sh ? I_sh : I;
        block[s] = d;
        const QMatDev& m = sh ? p.sh_down : p.down;
        const uint32_t* codes = m.codes + (size_t)ent[s].expert * H * (K[s] / 8);
        const bool in = on && d * 128 + g * 32 < K[s];
        // four column tiles of 16: 512 bytes apart in tiles, 2 K words in rows
        const uint32_t at0 = code_word(m.layout, cg * 64 + c, d * 16 + g * 4, K[s]);
        const uint32_t t_step = m.layout ? 128u : 2u * K[s];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            wv[s][t] = in ? *(const u32x4_t*)(codes + (at0 + t * t_step)) : u32x4_t{0, 0, 0, 0};
        const uint32_t groups = K[s] / 64;
        const size_t s0 = ((size_t)ent[s].expert * H + cg * 64) * groups + d * 2;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t at = (t * 16 + c) * groups;
            if constexpr (VEC) {   // the groups of both halves of the wave
                sc[s][t] = on ? *(const uint32_t*)(m.scales + s0 + at) : 0u;
                bi[s][t] = on ? *(const uint32_t*)(m.biases + s0 + at) : 0u;
            } else {               // this lane's
                sc[s][t] = in ? m.scales[s0 + at + g / 2] : 0u;
                bi[s][t] = in ? m.biases[s0 + at + g / 2] : 0u;
            }
        }
        load_h(s, c, c < __popcll(ent[s].mask), hi[s], lo[s]);
    };
    f32x4_t acc[4];
    auto multiply = [&](int s, const u32x4_t (&h)[4], const u32x4_t (&l)[4]) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float sv = VEC ? __builtin_bit_cast(float, g < 2 ? sc[s][t] << 16 : sc[s][t] & 0xFFFF0000u)
                                 : bf16_to_f32((uint16_t)sc[s][t]);
            const float bv = VEC ? __builtin_bit_cast(float, g < 2 ? bi[s][t] << 16 : bi[s][t] & 0xFFFF0000u)
                                 : bf16_to_f32((uint16_t)bi[s][t]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x8_t w = dequant_word(wv[s][t][i], sv * unit_inv, bv);
                acc[t] = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, h[i]), acc[t]);
                acc[t] = mfma_16x16x32(w, __builtin_bit_cast(bf16x8_t, l[i]), acc[t]);
            }
        }
    };
    // the sums of the expert's tokens t0 .. + 15 to the tokens' rows: the lanes have different places
    auto flush = [&](unsigned long long mask, int t0) {
        if (mask >> lane & 1) s_tok[wave][__popcll(mask & lanemask_lt())] = lane;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (t0 + c < __popcll(mask)) {
            float* o = y + s_tok[wave][t0 + c] * LDY + g * 4;
#pragma unroll
            for (int t = 0; t < 4; ++t) *(f32x4_t*)(o + t * 16) = *(const f32x4_t*)(o + t * 16) + acc[t];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();   // the next expert's tokens take these ones' place
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kBpAhead; ++s) load(s, first + s);
    for (int step = first; step < last; step += kBpAhead) {
#pragma unroll
        for (int s = 0; s < kBpAhead; ++s) {
            if (step + s >= last) break;
            const unsigned long long mask = ent[s].mask;
            const int cnt = __popcll(mask);
            multiply(s, hi[s], lo[s]);
            // the expert's last block of this wave, or more tokens than one product's columns
            if (cnt > 16 || step + s + 1 == last || (block[s] + 1) * 128 >= K[s]) flush(mask, 0);
            for (int t0 = 16; t0 < cnt; t0 += 16) {
                u32x4_t h[4], l[4];
                load_h(s, t0 + c, t0 + c < cnt, h, l);
                multiply(s, h, l);
                flush(mask, t0);
            }
            load(s, step + s + kBpAhead);
        }
    }
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
    for (int s = 1; s < splits; ++s) v += *(const f32x4_t*)(part + s * n + i);
    *(u32x2_t*)(y + i) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Shares of the experts: a workgroup for each compute unit.
static int batch_splits(int H) {
    const int s = 256 / (H / 64);
    return s < 1 ? 1 : s < 16 ? s : 16;
}

// Tokens whose selection every gate/up workgroup repeats, one or two a wave.
constexpr int kBatchOwnSelect = 8;
constexpr int kBatchColumns = 8;

BatchWs batch_ws_layout(int T, int H, int I, int I_sh, int E, int k) {
    BatchWs w{};
    const size_t n = (size_t)T * k, slots = (size_t)E < n ? E : n;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 256);
        return at;
    };
    const size_t values = n * I + (size_t)T * I_sh;
    w.h_hi = take(values * 2);
    w.h_lo = take(values * 2);
    w.list = take(slots * 16);
    w.n_list = take(4);
    w.y_part = take((size_t)batch_splits(H) * T * H * 4);
    w.idx = take(n * 4);
    w.w = take(n * 4);
    w.total = o;
    return w;
}

template <int EPL>
static void launch_batch_gateup(const BatchArgs& a, int grid, size_t lds, int rt_log, hipStream_t stream) {
    if (a.gate.layout == 2)
        batch_gateup_kernel<EPL, true><<<grid, kBgThreads, lds, stream>>>(a, rt_log);
    else
        batch_gateup_kernel<EPL, false><<<grid, kBgThreads, lds, stream>>>(a, rt_log);
}

hipError_t launch_decode_batch(const BatchArgs& a, hipStream_t stream) {
    const int n = a.T * a.k, slots = a.E < n ? a.E : n;
    const int epl = (a.E + WAVE - 1) / WAVE;
    const bool own = a.T <= kBatchOwnSelect;
    hipError_t err;
    if (!own) {
        const int grid = (a.T + kBsWaves - 1) / kBsWaves;
#define MOE_SEL(N) batch_select_kernel<N><<<grid, kBsWaves * WAVE, 0, stream>>>(a)
        if (epl <= 1) MOE_SEL(1);
        else if (epl <= 2) MOE_SEL(2);
        else if (epl <= 4) MOE_SEL(4);
        else if (epl <= 8) MOE_SEL(8);
        else MOE_SEL(16);
#undef MOE_SEL
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    // Rows of a task: few tasks a workgroup leave compute units idle in the last round, tasks of few
    // rows split K over more waves, each of which waits for its loads once: kStart chunks' time.
    constexpr int kStart = 4;
    int rt_log = 0, grid = 0;
    long long best = 0;
    for (int i = 0; i < 3; ++i) {
        const int tasks = (a.I_sh + slots * a.I) >> (4 + i), rounds = (tasks + kBgResident - 1) / kBgResident;
        const long long cost = (long long)rounds * (8 * kStart + (((a.H + 127) / 128) << i));
        if (i == 0 || cost < best) {
            best = cost;
            rt_log = i;
            grid = tasks < kBgResident ? tasks : kBgResident;
        }
    }
    const size_t lds = (size_t)slots * 16 + (size_t)a.E * 8 + (size_t)n * (own ? 8 : 4);
    if (own) {
        if (epl <= 1) launch_batch_gateup<1>(a, grid, lds, rt_log, stream);
        else if (epl <= 2) launch_batch_gateup<2>(a, grid, lds, rt_log, stream);
        else if (epl <= 4) launch_batch_gateup<4>(a, grid, lds, rt_log, stream);
        else if (epl <= 8) launch_batch_gateup<8>(a, grid, lds, rt_log, stream);
        else launch_batch_gateup<16>(a, grid, lds, rt_log, stream);
    } else launch_batch_gateup<0>(a, grid, lds, rt_log, stream);
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
    const int cols = a.H / 8;
    if (a.T <= 8) batch_down_kernel<1><<<cols, kBdWaves * WAVE, 0, stream>>>(a);
    else if (a.T <= 16) batch_down_kernel<2><<<cols, kBdWaves * WAVE, 0, stream>>>(a);
    else if (a.T <= 32) batch_down_kernel<4><<<cols, kBdWaves * WAVE, 0, stream>>>(a);
    else batch_down_kernel<8><<<cols, kBdWaves * WAVE, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moeq4
