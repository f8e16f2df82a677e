// Per-token scored selection by one wave: scores (softmax or sigmoid of the
// logits), a selection bias, groups of experts, top-k and weights.
//
//   score_e  = fp32(sigmoid(l_e)), or fp32(exp(l_e - max l) / sum_i exp(l_i - max l))
//   choice_e = score_e + bias_e (one fp32 addition)
//   worth_g  = the group's best choice, or its two best choices' fp32 sum
//   the topk_groups groups of most worth stay, then the k experts of largest
//   choice among them; ties go to the lowest index throughout
//   weight_j = scale * score_j [/ max(sum of the chosen scores, 1e-30)]
//
// A selection hangs on the last bit of a score, so a score is formed in 64 bits
// and rounded once: it is then the nearest fp32 value whatever the order of the
// sum, but for values within 1e-15 of themselves of a rounding border.  A NaN logit
// or choice counts as -inf; a row of -inf alone has scores 0 and takes the lowest
// indices.
#pragma once

#include "moe_i8.h"
#include "moe_topk.h"

namespace moeq4 {

// Keys of the value that counts as the lowest: above 0, which marks an absent expert.
__device__ __forceinline__ uint32_t choice_key(float v) {
    return float_key(v != v ? -__builtin_huge_valf() : v);
}

// Sum over the wave in a fixed order, returned uniform (row_shr 1, 2, 4, 8 and
// row_bcast 15, 31 as in wave_incl_sum, both halves moved).
__device__ __forceinline__ double wave_sum_f64(double v) {
#define MOE_DPP_ADD64(ctrl, rows)                                                           \
    {                                                                                       \
        const uint64_t u = __builtin_bit_cast(uint64_t, v);                                 \
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, ctrl, rows, 0xf, false); \
        const uint32_t hi =                                                                 \
            __builtin_amdgcn_update_dpp(0, (int)(u >> 32), ctrl, rows, 0xf, false);         \
        v += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);                           \
    }
    MOE_DPP_ADD64(0x111, 0xf)
    MOE_DPP_ADD64(0x112, 0xf)
    MOE_DPP_ADD64(0x114, 0xf)
    MOE_DPP_ADD64(0x118, 0xf)
    MOE_DPP_ADD64(0x142, 0xa)
    MOE_DPP_ADD64(0x143, 0xc)
#undef MOE_DPP_ADD64
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)u, WAVE - 1);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), WAVE - 1);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 1 / d for finite d >= 1: the hardware's estimate and two Newton steps, within 2^-52.
__device__ __forceinline__ double recip_f64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// a / b for 0 <= a < 2^16, 1 <= b < 2^16 without an integer division's thirty instructions:
// (a + 1/2) / b is at least 1 / 2b from a whole number, the rounding far nearer.
__device__ __forceinline__ int small_div(int a, int b) {
    return (int)(((float)a + 0.5f) * __builtin_amdgcn_rcpf((float)b));
}

// Lane l holds experts l*EPL .. l*EPL+EPL-1; absent and dropped experts get key 0.
template <int EPL>
__device__ __forceinline__ void drop_groups(uint32_t (&key)[EPL], int E, const ScoreRule& rule) {
    const int lane = __lane_id();
    const int gs = rule.group_size, span = (int)((unsigned)gs / EPL);
    if ((unsigned)gs % EPL == 0) {
        // whole groups in `span` neighbouring lanes: every lane gathers its group's two best,
        // by a butterfly where span is a power of two and lane by lane otherwise
        uint32_t m1 = 0, m2 = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m2 = max(m2, min(m1, key[j]));
            m1 = max(m1, key[j]);
        }
        const int mine = small_div(lane, span);
        if ((span & (span - 1)) == 0) {
            for (int off = 1; off < span; off <<= 1) {
                const uint32_t o1 = shfl_xor(m1, off), o2 = shfl_xor(m2, off);
                m2 = max(max(m2, o2), min(m1, o1));
                m1 = max(m1, o1);
            }
        } else {
            const uint32_t l1 = m1, l2 = m2;
            m1 = m2 = 0;
            for (int i = 0; i < span; ++i) {
                const int from = mine * span + i;   // past lane 63 for lanes without experts only
                const uint32_t o1 = __shfl(l1, from, WAVE), o2 = __shfl(l2, from, WAVE);
                m2 = max(max(m2, o2), min(m1, o1));
                m1 = max(m1, o1);
            }
        }
        uint32_t worth = rule.top2 ? choice_key(key_float(m1) + key_float(m2)) : m1;
        if (lane * EPL >= E) worth = 0;
        bool keep = false;
        for (int r = 0; r < rule.topk_groups; ++r) {
            const uint32_t m = wave_max_u32(worth);
            const int g = __builtin_amdgcn_readlane(mine, __builtin_ctzll(__ballot(worth == m)));
            if (mine == g) {
                keep = true;
                worth = 0;
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = keep ? key[j] : 0u;
        return;
    }
    // any other size: one or two wave maxima per group, lane g keeps group g's worth
    uint32_t worth = 0;
    for (int g = 0; g < rule.n_groups; ++g) {
        const int lo = g * gs, hi = lo + gs;
        uint32_t m1 = 0, m2 = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            const uint32_t kj = e >= lo && e < hi ? key[j] : 0u;
            m2 = max(m2, min(m1, kj));
            m1 = max(m1, kj);
        }
        const uint32_t best = wave_max_u32(m1);
        uint32_t w = best;
        if (rule.top2) {
            // the second best: the winner's lane offers its own second
            const int win = __builtin_ctzll(__ballot(m1 == best));
            const uint32_t next = wave_max_u32(lane == win ? m2 : m1);
            w = choice_key(key_float(best) + key_float(next));
        }
        if (lane == g) worth = w;
    }
    uint64_t kept = 0;
    for (int r = 0; r < rule.topk_groups; ++r) {
        const uint32_t m = wave_max_u32(worth);
        const int g = __builtin_ctzll(__ballot(worth == m));
        kept |= 1ull << g;
        if (lane == g) worth = 0;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const int g = e < E ? small_div(e, gs) : 0;
        key[j] = (kept >> g) & 1 ? key[j] : 0u;
    }
}

template <int EPL>
__device__ __forceinline__ void score_topk_token(const float* __restrict__ row,
                                                 const float* __restrict__ bias, int E, int k,
                                                 const ScoreRule& rule, int32_t* out_idx,
                                                 float* out_w, int* lds_idx = nullptr) {
    const int lane = __lane_id();
    const float ninf = -__builtin_huge_valf();
    float l[EPL], sc[EPL];
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const float v = e < E ? row[e] : ninf;
        l[j] = v != v ? ninf : v;
    }
    if (rule.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)   // below -700 a score is 0 in fp32
            sc[j] = (float)recip_f64(1.0 + exp(fmin(-(double)l[j], 700.0)));
    } else {
        float best = l[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) best = fmaxf(best, l[j]);
        best = key_float(wave_max_u32(float_key(best)));
        double p[EPL], part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            // an infinite maximum: its holders share the whole score (+inf), or no one has any
            if (__builtin_isinf(best)) p[j] = best > 0.f && l[j] == best ? 1.0 : 0.0;
            else p[j] = exp((double)l[j] - (double)best);
            part += p[j];
        }
        part = wave_sum_f64(part);   // at least 1, or 0 for a row of -inf alone
        const double inv = part > 0.0 ? recip_f64(part) : 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) sc[j] = (float)(p[j] * inv);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const float b = bias && e < E ? bias[e] : 0.f;
        key[j] = e < E ? choice_key(sc[j] + b) : 0u;
    }
    if (rule.topk_groups < rule.n_groups) drop_groups<EPL>(key, E, rule);
    int my_e = 0;
    float my_s = 0.f, sum = 0.f;
    for (int r = 0; r < k; ++r) {
        uint32_t bk = key[0];
        float bs = sc[0];
        int bj = 0;
#pragma unroll
        for (int j = 1; j < EPL; ++j) {
            const bool gt = key[j] > bk;   // strict: the lower index wins a tie
            bk = gt ? key[j] : bk;
            bs = gt ? sc[j] : bs;
            bj = gt ? j : bj;
        }
        const uint32_t m = wave_max_u32(bk);
        const int w = __builtin_ctzll(__ballot(bk == m));   // lowest lane holding m
        const int jw = __builtin_amdgcn_readlane(bj, w);
        const float s = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, bs), w));
        sum += s;
        if (lane == r) {
            my_e = w * EPL + jw;
            my_s = s;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = (lane == w && j == jw) ? 0u : key[j];
    }
    if (lane < k) {
        const float wgt = rule.renormalise ? my_s / fmaxf(sum, 1e-30f) : my_s;
        out_idx[lane] = my_e;
        out_w[lane] = wgt * rule.scale;
        if (lds_idx) lds_idx[lane] = my_e;
    }
    __builtin_amdgcn_wave_barrier();
}

// Routing arrays of one token from its k chosen experts and weights in LDS, by all
// `threads` threads of a workgroup (the experts differ, so an assignment's row is
// the number of chosen experts below its own).
__device__ __forceinline__ void write_one_token(const RoutingDev& r, int E, int k, int max_blocks,
                                                const int* s_idx, const float* s_w, int tid,
                                                int threads) {
    for (int e = tid; e <= E; e += threads) {
        int off = 0, cnt = 0;
        for (int j = 0; j < k; ++j) {
            off += s_idx[j] < e ? 1 : 0;
            cnt += s_idx[j] == e ? 1 : 0;
        }
        r.offsets[e] = off;
        if (e < E) r.counts[e] = cnt;
    }
    for (int j = tid; j < k; j += threads) {
        const int e = s_idx[j];
        int row = 0;
        for (int i = 0; i < k; ++i) row += s_idx[i] < e ? 1 : 0;
        r.topk_idx[j] = e;
        r.topk_w[j] = s_w[j];
        r.sorted_assign[row] = j;
        r.assign_row[j] = row;
        r.block_expert[row] = e;
        r.block_row[row] = row;
    }
    for (int b = k + tid; b < max_blocks; b += threads) {
        r.block_expert[b] = -1;
        r.block_row[b] = -1;
    }
    if (tid == 0) r.n_blocks[0] = k;
}

}  // namespace moeq4
