// Log probabilities of rows of logits z[0 .. V): of a given token, the entropy, and the n most
// probable tokens.
//
//   m = max z,  S = sum exp(z - m),  D = sum (z - m) exp(z - m)
//   log p_i = z_i - m - log S,  entropy = log S - D / S
//
// One pass over the row.  A thread keeps its own running m, S and D over pieces of 16 bytes
// (a new maximum scales the sums: S' = f S, D' = f (D + (m - m') S), f = exp(m - m')), and its
// largest value with the piece that holds it.  The n best tokens lie with the n threads of
// the best maxima: when the row is through, the workgroup orders the threads' maxima, and
// reads again only those n threads' pieces (n / 512 of the row), for values from the n-th
// best maximum on.  Keys order by value, then by the lower index, so they all differ and
// neither ties nor sorted rows change the amount of work much.
//
// Few rows are split over workgroups, whose results a second kernel joins.
// Bound by vector instructions for bf16, about 14 a value with the exponential as four, which 2048
// rows of 131072 need 90 us for where their bytes need 85: 117 us in all back to back, 132 to 135 under
// the tracer, where the figures below are from.  Few rows are bound by
// latency: one of 131072 takes 8.9 us, 1.6 of them for its values, and 3.5 for the join.
// The next pieces' loads before the present ones' sums, 1024 threads and 256 a workgroup were tried: 150, 191
// and 135 us, 192 rows of 150001 in 21.1, 21.7 and 30.1 where 512 threads take 22.0.
#include "moe_i8.h"
#include "moe_score.h"

namespace moeq4 {

constexpr int kLpThreads = 512, kLpWaves = kLpThreads / WAVE;
constexpr int kLpPieces = 4;          // 16-byte pieces of a thread in flight
constexpr int kLpCands = 1024;        // values that may be gathered for the last ordering
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Value and index in one key: larger values first, among equals the lower index.  0: none.
__device__ __forceinline__ uint64_t token_key(float z, uint32_t index) {
    return (uint64_t)choice_key(z) << 32 | (0xFFFFFFFFu - index);
}

// The sums of a part of a row, in powers of two: S = sum 2^t, D = sum t 2^t, t = (z - m) log2(e).
struct LpSums {
    float m, s, d;
};

// a's sums for the maximum m >= a.m.  A part without a number has m = -inf and sums 0, or NaN if it
// held one.  A factor of 0 leaves nothing, however far below m the part lies; m = +inf: NaN.
__device__ __forceinline__ LpSums lp_scaled(const LpSums& a, float m) {
    if (m == -__builtin_huge_valf()) return a;
    const float t = (a.m - m) * kLog2e, f = __builtin_amdgcn_exp2f(t);
    return LpSums{m, f * a.s, f == 0.f ? 0.f * a.s : f * (a.d + t * a.s)};
}

// Sum over the wave, in one order.
__device__ __forceinline__ float wave_sum_f32(float v) {
#define MOE_DPP_ADD(ctrl) \
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xf, 0xf, true))
    MOE_DPP_ADD(0x111);   // row_shr:1
    MOE_DPP_ADD(0x112);   // row_shr:2
    MOE_DPP_ADD(0x114);   // row_shr:4
    MOE_DPP_ADD(0x118);   // row_shr:8
    MOE_DPP_ADD(0x142);   // row_bcast:15
    MOE_DPP_ADD(0x143);   // row_bcast:31
#undef MOE_DPP_ADD
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The lanes' sums together: one exponential a lane, for the maximum of all.
__device__ __forceinline__ LpSums lp_wave(const LpSums& a) {
    const float m = key_float(wave_max_u32(choice_key(a.m)));
    const LpSums o = lp_scaled(a, m);
    return LpSums{m, wave_sum_f32(o.s), wave_sum_f32(o.d)};
}

// Keys above `mine` among `lists` lists of n in descending order.
__device__ __forceinline__ int keys_above(const uint64_t* keys, int lists, int n, uint64_t mine) {
    int above = 0;
    const int top = 1 << (31 - __builtin_clz(n));
    for (int l = 0; l < lists; l += 8) {   // eight searches at a time: each waits for LDS at every step
        int at[8] = {};
        for (int step = top; step; step >>= 1) {
            uint64_t key[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) key[i] = keys[min(l + i, lists - 1) * n + min(at[i] + step, n) - 1];
#pragma unroll
            for (int i = 0; i < 8; ++i) at[i] += (key[i] > mine) & (at[i] + step <= n) & (l + i < lists) ? step : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) above += at[i];
    }
    return above;
}

// Four or eight values of a 16-byte piece.
template <bool BF16>
__device__ __forceinline__ float piece_value(const u32x4_t& v, int i) {
    const uint32_t w = v[BF16 ? i / 2 : i];
    return __builtin_bit_cast(float, !BF16 ? w : i % 2 ? w & 0xFFFF0000u : w << 16);
}

// Where a row's pieces lie.  Piece 0 starts at the 16-byte border at or below the row's first
// value; pieces lo .. hi - 1 are whole, the first and last one may not be.
template <bool BF16>
struct LpRow {
    static constexpr int PER = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
    const char* base;   // piece 0
    int off, V;         // values of piece 0 before the row
    __device__ LpRow(const void* row, int V_) : V(V_) {
        const uint64_t at = (uint64_t)row;
        off = (int)(at % 16) / SIZE;
        base = (const char*)(at - at % 16);
    }
    __device__ int pieces() const { return (int)(((long long)off + V + PER - 1) / PER); }
    __device__ int lo() const { return off ? 1 : 0; }
    __device__ int hi() const { return (int)(((long long)off + V) / PER); }
    __device__ u32x4_t whole(int f) const { return *(const u32x4_t*)(base + (size_t)f * 16); }
    // any piece, value by value; -inf outside the row
    __device__ u32x4_t edge(int f) const {
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const long long at = (long long)f * PER + i - off;
            const bool in = at >= 0 && at < V;
            const char* p = base + (size_t)f * 16 + i * SIZE;
            if constexpr (BF16) {
                const uint32_t b = in ? *(const uint16_t*)p : 0xFF80u;
                v[i / 2] = i % 2 ? v[i / 2] | b << 16 : b;
            } else {
                v[i] = in ? *(const uint32_t*)p : 0xFF800000u;
            }
        }
        return v;
    }
    __device__ bool inside(int f, int i) const {
        const long long at = (long long)f * PER + i - off;
        return at >= 0 && at < V;
    }
    __device__ uint32_t index(int f, int i) const { return (uint32_t)((long long)f * PER + i - off); }
};

// The lanes' keys in descending order.
__device__ __forceinline__ uint64_t wave_sort_keys(uint64_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= WAVE; size <<= 1) {
#pragma unroll
        for (int step = size >> 1; step >= 1; step >>= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)v, step, WAVE);
            const bool first = (lane & step) == 0, down = (lane & size) == 0;
            const bool keep_max = first == down;
            v = keep_max == (v > o) ? v : o;
        }
    }
    return v;
}

struct LpArgs {
    const void* logits;
    long long ld;
    const int32_t* target;
    int T, V, n, splits;
    float *logprob, *entropy;
    int32_t* top_idx;
    float* top_logprob;
    LpSums* sums;      // workspace [T, splits]
    uint64_t* keys;    // workspace [T, splits, n], each list in order, 0 behind its end
};

// The target's logit, in thread 0, fetched before it is needed.
template <bool BF16>
__device__ __forceinline__ float lp_target(const LpArgs& p, int row, int tid) {
    if (tid || !p.logprob) return 0.f;
    const int t = p.target[row];
    if (t < 0 || t >= p.V) return 0.f;
    const size_t at = (size_t)row * p.ld + t;
    return BF16 ? bf16_to_f32(((const uint16_t*)p.logits)[at]) : ((const float*)p.logits)[at];
}

// The row's results from its sums and the n best keys in order.
template <bool BF16>
__device__ __forceinline__ void lp_write(const LpArgs& p, int row, const LpSums& all, const uint64_t* best,
                                         float z_target, int tid) {
    const float ninf = -__builtin_huge_valf();
    const bool none = all.m == ninf && all.s == 0.f;   // -inf alone
    const float log_s = __builtin_logf(all.s);
    auto lp = [&](float z) { return none ? ninf : z - all.m - log_s; };
    if (tid < p.n) {
        const uint64_t key = best[tid];
        const size_t at = (size_t)row * p.n + tid;
        if (p.top_idx) p.top_idx[at] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
        if (p.top_logprob) p.top_logprob[at] = lp(key_float((uint32_t)(key >> 32)));
    }
    if (tid == 0) {
        if (p.entropy) p.entropy[row] = none ? 0.f : log_s - kLn2 * (all.d / all.s);
        if (p.logprob) {
            const int t = p.target[row];
            p.logprob[row] = t >= 0 && t < p.V ? lp(z_target) : 0.f;
        }
    }
}

template <bool BF16>
__global__ __launch_bounds__(kLpThreads) void logprobs_kernel(LpArgs p) {
    __shared__ LpSums s_sums[kLpWaves];
    __shared__ uint64_t s_lists[kLpWaves * kLogprobsMaxTop];
    __shared__ uint64_t s_cand[kLpCands];
    __shared__ uint64_t s_best[kLogprobsMaxTop];
    __shared__ uint64_t s_limit;
    __shared__ int s_count;
    __shared__ int s_from[kLogprobsMaxTop];
    using Row = LpRow<BF16>;
    constexpr int PER = Row::PER;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const float ninf = -__builtin_huge_valf();
    const int row = blockIdx.x / p.splits, part = blockIdx.x % p.splits;
    const Row r((const char*)p.logits + (size_t)row * p.ld * Row::SIZE, p.V);
    // this workgroup's whole pieces; the row's ends go with its first and last part
    const int lo = r.lo(), span = r.hi() - lo;
    const int f0 = lo + (int)((long long)span * part / p.splits);
    const int f1 = lo + (int)((long long)span * (part + 1) / p.splits);
    // piece that thread 0 (the row's first) or thread 1 (its last) takes besides; -1: none
    int extra = -1;
    if (tid == 0 && part == 0 && lo > 0) extra = 0;
    if (tid == 1 && part == p.splits - 1 && r.pieces() > r.hi() && (r.hi() > 0 || lo == 0)) extra = r.pieces() - 1;

    LpSums a = {ninf, 0.f, 0.f};
    float best = ninf;
    int best_f = -1;
    u32x4_t best_v = {0, 0, 0, 0};
    auto piece_max = [&](const u32x4_t& v) {
        float t = piece_value<BF16>(v, 0);
#pragma unroll
        for (int i = 1; i < PER; ++i) t = fmaxf(t, piece_value<BF16>(v, i));
        return fmaxf(t, ninf);   // NaN alone counts as -inf here
    };
    auto take_best = [&](const u32x4_t& v, int f, float t) {
        const bool more = best_f < 0 || t > best;
        best = more ? t : best;
        best_f = more ? f : best_f;
#pragma unroll
        for (int i = 0; i < 4; ++i) best_v[i] = more ? v[i] : best_v[i];
    };
    auto rescale = [&](float m) {
        if (m > a.m) {
            if (a.m != ninf) {
                const float t = (a.m - m) * kLog2e, f = __builtin_amdgcn_exp2f(t);
                a.d = f == 0.f ? 0.f * a.s : f * (a.d + t * a.s);
                a.s *= f;
            }
            a.m = m;
        }
    };
    auto add = [&](const u32x4_t& v) {
        const float ref = a.m == ninf ? 0.f : a.m;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float t = (piece_value<BF16>(v, i) - ref) * kLog2e;
            const float e = __builtin_amdgcn_exp2f(t);
            a.s += e;
            a.d = __builtin_fmaf(fmaxf(t, -1e4f), e, a.d);   // -inf times 0 is 0 here
        }
    };
    if (extra >= 0) {
        const u32x4_t v = r.edge(extra);
        const float t = piece_max(v);
        if (extra == 0) take_best(v, extra, t);   // the row's last piece comes last: lower indices first
        rescale(t);
        add(v);
    }
    for (int f = f0 + tid; f < f1; f += kLpThreads * kLpPieces) {
        u32x4_t v[kLpPieces];
        constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (int i = 0; i < kLpPieces; ++i) {
            const int at = f + i * kLpThreads;
            v[i] = at < f1 ? r.whole(at) : u32x4_t{kNone, kNone, kNone, kNone};
        }
        float t[kLpPieces], m = ninf;
#pragma unroll
        for (int i = 0; i < kLpPieces; ++i) {
            t[i] = piece_max(v[i]);
            m = fmaxf(m, t[i]);
        }
        if (p.n) {
#pragma unroll
            for (int i = 0; i < kLpPieces; ++i) take_best(v[i], f + i * kLpThreads, t[i]);
        }
        rescale(m);
#pragma unroll
        for (int i = 0; i < kLpPieces; ++i) add(v[i]);
    }
    if (extra > 0) {
        const u32x4_t v = r.edge(extra);
        take_best(v, extra, piece_max(v));
    }

    const float z_target = p.splits == 1 ? lp_target<BF16>(p, row, tid) : 0.f;

    // ---- the sums of the workgroup, in a fixed order ----
    a = lp_wave(a);
    if (lane == 0) s_sums[wave] = a;

    // ---- the n best: threads' maxima, then the values of the best n threads ----
    if (p.n) {
        uint64_t key = 0;
        if (best_f >= 0) {
            int at = -1;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) {
                const float z = piece_value<BF16>(best_v, i);
                const bool is = r.inside(best_f, i) && (z == best || (best == ninf && z != z));
                at = is ? i : at;
            }
            if (at >= 0) key = token_key(best, r.index(best_f, at));
        }
        const uint64_t sorted = wave_sort_keys(key, lane);
        if (lane < p.n) s_lists[wave * p.n + lane] = sorted;
        if (tid == 0) {
            s_limit = 1;   // fewer than n threads with a value: all of them
            s_count = 0;
        }
        if (tid < p.n) s_from[tid] = -1;
        __syncthreads();
        const int all = kLpWaves * p.n;
        if (tid < all) {
            const uint64_t mine = s_lists[tid];
            const int rank = keys_above(s_lists, kLpWaves, p.n, mine);
            if (mine && rank < p.n) {
                // the thread of this maximum
                const uint32_t index = 0xFFFFFFFFu - (uint32_t)mine;
                const int f = (int)(((long long)index + r.off) / PER);
                s_from[rank] = f >= f0 && f < f1 ? (f - f0) % kLpThreads : f == 0 && lo > 0 ? 0 : 1;
                if (rank == p.n - 1) s_limit = mine;
            }
        }
        __syncthreads();
        const uint64_t limit = s_limit;
        // every value of those threads' pieces, `use` for each from the limit on
        auto scan = [&](auto use) {
            for (int w = wave; w < p.n; w += kLpWaves) {
                const int t = __builtin_amdgcn_readfirstlane(s_from[w]);
                if (t < 0) continue;
                const int ends = (t == 0 && part == 0 && lo > 0 ? 1 : 0) +
                                 (t == 1 && part == p.splits - 1 && r.pieces() > r.hi() &&
                                  (r.hi() > 0 || lo == 0) ? 1 : 0);
                for (int f = f0 + t + lane * kLpThreads; f - lane * kLpThreads < f1; f += WAVE * kLpThreads) {
                    if (f >= f1) continue;
                    const u32x4_t v = r.whole(f);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const uint64_t k = token_key(piece_value<BF16>(v, i), r.index(f, i));
                        if (k >= limit) use(k);
                    }
                }
                if (ends && lane == 0) {
                    const int f = t == 0 ? 0 : r.pieces() - 1;
                    const u32x4_t v = r.edge(f);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const uint64_t k = token_key(piece_value<BF16>(v, i), r.index(f, i));
                        if (r.inside(f, i) && k >= limit) use(k);
                    }
                }
            }
        };
        scan([&](uint64_t k) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kLpCands) s_cand[at] = k;
        });
        if (tid < p.n) s_best[tid] = 0;
        __syncthreads();
        const int count = s_count;
        if (count <= kLpCands) {
            // keys differ: a key's rank is its place
            for (int c = tid; c < count; c += kLpThreads) {
                const uint64_t mine = s_cand[c];
                int rank = 0;
                for (int i = 0; i < count; ++i) rank += s_cand[i] > mine ? 1 : 0;
                if (rank < p.n) s_best[rank] = mine;
            }
        } else {
            // many large values with few threads: the largest below the one before, n times
            uint64_t last = ~0ull;
            for (int j = 0; j < p.n; ++j) {
                uint64_t top = 0;
                scan([&](uint64_t k) { top = k < last && k > top ? k : top; });
#pragma unroll
                for (int off = 1; off < WAVE; off <<= 1) {
                    const uint64_t o = __shfl_xor((unsigned long long)top, off, WAVE);
                    top = o > top ? o : top;
                }
                __syncthreads();
                if (lane == 0) s_lists[wave] = top;
                __syncthreads();
                last = 0;
                for (int w = 0; w < kLpWaves; ++w) last = s_lists[w] > last ? s_lists[w] : last;
                if (tid == 0) s_best[j] = last;
            }
        }
    }
    __syncthreads();
    LpSums total = {s_sums[0].m, 0.f, 0.f};
#pragma unroll
    for (int w = 1; w < kLpWaves; ++w) total.m = fmaxf(total.m, s_sums[w].m);
#pragma unroll
    for (int w = 0; w < kLpWaves; ++w) {
        const LpSums o = lp_scaled(s_sums[w], total.m);
        total.s += o.s;
        total.d += o.d;
    }
    if (p.splits == 1) {
        lp_write<BF16>(p, row, total, s_best, z_target, tid);
        return;
    }
    if (tid == 0) p.sums[blockIdx.x] = total;
    if (tid < p.n) p.keys[(size_t)blockIdx.x * p.n + tid] = s_best[tid];
}

// A row's parts joined; splits * n <= kLpCands.
template <bool BF16>
__global__ __launch_bounds__(kLpThreads) void logprobs_join_kernel(LpArgs p) {
    __shared__ uint64_t s_keys[kLpCands];
    __shared__ uint64_t s_best[kLogprobsMaxTop];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % WAVE;
    const int all = p.splits * p.n;
    const float ninf = -__builtin_huge_valf(), z_target = lp_target<BF16>(p, row, tid);
    // every wave joins the sums, a part a lane
    const LpSums total = lp_wave(lane < p.splits ? p.sums[(size_t)row * p.splits + lane] : LpSums{ninf, 0.f, 0.f});
    for (int i = tid; i < all; i += kLpThreads) s_keys[i] = p.keys[(size_t)row * all + i];
    __syncthreads();
    for (int c = tid; c < all; c += kLpThreads) {
        const uint64_t mine = s_keys[c];
        if (!mine) continue;
        const int rank = keys_above(s_keys, p.splits, p.n, mine);
        if (rank < p.n) s_best[rank] = mine;
    }
    __syncthreads();
    lp_write<BF16>(p, row, total, s_best, z_target, tid);
}

// Workgroups a row is split over: as many as give each compute unit at most one, of 16384 values at
// least.  What a workgroup does behind its values (5 us where they are read in 4) costs more than
// idle compute units: 48 rows of 100003 fp32 take 12.8 us with 5 parts and 14.1 with 6, 96 rows of
// 150001 bf16 15.3 with 2 and 17.2 with 3, and one row of 131072 8.9 + 3.5 with 8 and 9.4 + 6.0 with 32.
static int lp_splits(int T, int V, int n) {
    int s = T < 256 ? 256 / T : 1;
    const int most = V / 16384 > 0 ? V / 16384 : 1, room = n ? kLpCands / n : kLpCands;
    s = s < most ? s : most;
    s = s < room ? s : room;
    return s < 64 ? s : 64;
}

size_t logprobs_ws_bytes(int T, int V, int n) {
    const int s = lp_splits(T, V, n);
    return s == 1 ? 0 : align_up((size_t)T * s * sizeof(LpSums), 256) + align_up((size_t)T * s * n * 8, 256);
}

hipError_t launch_logprobs(const void* logits, bool bf16, long long ld, const int32_t* target, int T, int V,
                           int n, float* logprob, float* entropy, int32_t* top_idx, float* top_logprob,
                           void* ws, hipStream_t stream) {
    const int splits = lp_splits(T, V, n);
    for (int t = 0; t < T; t += kItemsALaunch) {   // one part where rows are split
        const int rows = T - t < kItemsALaunch ? T - t : kItemsALaunch;
        LpArgs p = {(const char*)logits + (size_t)t * ld * (bf16 ? 2 : 4), ld, target ? target + t : nullptr,
                    rows, V, n, splits, logprob ? logprob + t : nullptr, entropy ? entropy + t : nullptr,
                    top_idx ? top_idx + (size_t)t * n : nullptr,
                    top_logprob ? top_logprob + (size_t)t * n : nullptr, nullptr, nullptr};
        if (splits > 1) {
            p.sums = (LpSums*)ws;
            p.keys = (uint64_t*)((char*)ws + align_up((size_t)T * splits * sizeof(LpSums), 256));
        }
        const unsigned grid = (unsigned)rows * splits;
        if (bf16) logprobs_kernel<true><<<grid, kLpThreads, 0, stream>>>(p);
        else logprobs_kernel<false><<<grid, kLpThreads, 0, stream>>>(p);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        if (splits == 1) continue;
        if (bf16) logprobs_join_kernel<true><<<rows, kLpThreads, 0, stream>>>(p);
        else logprobs_join_kernel<false><<<rows, kLpThreads, 0, stream>>>(p);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace moeq4
