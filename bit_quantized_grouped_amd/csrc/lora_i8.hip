// The adapters' first product: u[m, r] = scale_j * a_scale[m] * sum_k A_j[r, k] a[m, k] for the
// rows m that have an adapter j = adapter[m] (codes a as bf16, which holds them exactly;
// products exact, sums fp32), written as two bf16 in the order of the second product's operand
// (moe_lora.h).
//
// A workgroup multiplies 16 RT ranks of one adapter by up to 16 MT rows that have it, its waves
// splitting K; their sums meet in LDS.  Bound by reading A, once for each such set of rows, so
// where tiles of 16 rows as they come could read more than kDirectBytes (rows of many adapters,
// or many rows), a kernel in front puts the rows in order of their adapters.  Otherwise a
// workgroup finds the adapters of its 16 rows itself, and rows of others are zeros.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_lora.h"

namespace moeq4 {

// Eight codes as bf16.
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t lo, uint32_t hi) {
    bf16x8_t r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = i < 4 ? lo : hi;
        r[i] = (__bf16)(float)(int)(int8_t)(w >> 8 * (i % 4));
    }
    return r;
}

struct ShrinkArgs {
    const int8_t* a;
    const float* a_scale;
    const uint16_t* A;
    const float* scales;
    const int32_t* adapter;
    uint16_t* u;
    int M, K, n, rank, steps;      // steps of 16 ranks
    const int32_t* order;          // grouped: rows by adapter, and the blocks of kSgRows of them
    const int4* blocks;            // (adapter, first place in order, rows, -)
    const int* n_blocks;
};

// One adapter's product with the rows row[m] (below 0: none) of the lanes, whose u goes to
// place[m]; W waves.  Of the 16 ranks of a step those of part `part` of 1 << parts_log.
template <int MT, int RT, int W, int AHEAD>
__device__ __forceinline__ void shrink_rows(const ShrinkArgs& p, int j, int t0, const int (&row)[MT],
                                            const int (&place)[MT], f32x4_t (*s_part)[RT][WAVE],
                                            int part = 0, int parts_log = 0) {
    const int lane = threadIdx.x % WAVE, fr = lane % 16, fp = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int steps = p.K / 64, s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
    const uint16_t* Aj = p.A + ((size_t)j * p.rank + t0 * 16 + fr) * p.K + fp * 16;
    f32x4_t acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    u32x4_t w[AHEAD][RT][2], c[AHEAD][MT];
    auto load = [&](int q, int s) {
        const bool in = s < s1;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[q][t][i] = in && (t0 + t) * 16 + fr < p.rank && fr >> (4 - parts_log) == part
                                 ? *(const u32x4_t*)(Aj + (size_t)t * 16 * p.K + s * 64 + 8 * i)
                                 : u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < MT; ++m)
            c[q][m] = in && row[m] >= 0 ? *(const u32x4_t*)(p.a + (size_t)row[m] * p.K + s * 64 + fp * 16)
                                        : u32x4_t{0, 0, 0, 0};
    };
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) load(q, s0 + q);
    for (int s = s0; s < s1; s += AHEAD) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8_t b = codes_bf16(c[q][m][2 * i], c[q][m][2 * i + 1]);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[m][t] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, w[q][t][i]), b, acc[m][t]);
                }
            load(q, s + q + AHEAD);
        }
    }
    const float scale = p.scales[j];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (!__ballot(row[m] >= 0)) continue;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t) s_part[wave][t][lane] = acc[m][t];
        __syncthreads();
        for (int t = wave; t < RT; t += W) {
            if (t0 + t >= p.steps) break;
            f32x4_t v = s_part[0][t][lane];
#pragma unroll
            for (int i = 1; i < W; ++i) v += s_part[i][t][lane];
            const int r = place[m];
            if (row[m] >= 0 && fp * 4 >> (4 - parts_log) == part) {
                v *= p.a_scale[row[m]] * scale;
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    hi[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    lo[i] = pack_bf16x2(bf16_rest(v[2 * i], (uint16_t)hi[i]),
                                        bf16_rest(v[2 * i + 1], (uint16_t)(hi[i] >> 16)));
                }
                // ranks 4 fp .. + 3: half of what lane r % 16 + 16 (fp / 2) of the operand holds
                char* o = (char*)p.u + lora_u_at(r / 16, t0 + t, p.steps, r % 16 + fp / 2 * 16) + fp % 2 * 8;
                *(u32x2_t*)o = u32x2_t{hi[0], hi[1]};
                *(u32x2_t*)(o + 32 * 16) = u32x2_t{lo[0], lo[1]};
            }
        }
    }
}

// 16 rows as they come, every gridDim.y-th of their adapters, a part of one step of ranks.  A compute
// unit fetches no more than about 24 bytes a ns, so few workgroups take four ranks each: 48 rows of
// 48 adapters of rank 16, K 4096, 8.4 us with whole steps, 7.1 by eights, 6.6 by
// fours; one row, K 2048, 4.5, 4.4 and 4.3.
constexpr int kSdWaves = 16;
__global__ __launch_bounds__(kSdWaves* WAVE) void lora_shrink_kernel(ShrinkArgs p, int parts_log) {
    __shared__ f32x4_t s_part[kSdWaves][1][WAVE];
    const int r = blockIdx.x * 16 + threadIdx.x % 16;
    int of = r < p.M ? p.adapter[r] : -1;
    of = of >= 0 && of < p.n ? of : -1;
    unsigned long long left = __ballot(of >= 0) & 0xFFFF;
    for (int turn = 0; left; ++turn) {
        const int j = __builtin_amdgcn_readlane(of, __builtin_ctzll(left));
        left &= ~__ballot(of == j);
        if (turn % (int)gridDim.y != (int)blockIdx.y) continue;
        const int row[1] = {of == j ? r : -1};
        shrink_rows<1, 1, kSdWaves, 4>(p, j, blockIdx.z >> parts_log, row, row, s_part,
                                       blockIdx.z & ((1 << parts_log) - 1), parts_log);
    }
}

// A block of rows of one adapter, RT steps of ranks.
constexpr int kSgWaves = 8, kSgRows = 32;
template <int RT>
__global__ __launch_bounds__(kSgWaves* WAVE) void lora_shrink_grouped_kernel(ShrinkArgs p) {
    __shared__ f32x4_t s_part[kSgWaves][RT][WAVE];
    if ((int)blockIdx.x >= *p.n_blocks) return;
    const int4 b = p.blocks[blockIdx.x];
    int row[kSgRows / 16], place[kSgRows / 16];
#pragma unroll
    for (int m = 0; m < kSgRows / 16; ++m) {
        const int at = m * 16 + threadIdx.x % 16;
        place[m] = b.y + at;
        row[m] = at < b.z ? p.order[place[m]] : -1;
    }
    shrink_rows<kSgRows / 16, RT, kSgWaves, 1>(p, b.x, blockIdx.y * RT, row, place, s_part);
}

// Rows in order of their adapters, those without one last, and the adapters' rows in blocks, by
// one workgroup: counts, a scan over the adapters, places.  The order inside an adapter is any:
// what a row gets does not depend on it.
constexpr int kGroupThreads = 1024, kGroupMax = 4096;   // adapters whose counts fit LDS
constexpr int kGroupRows = 8;                           // rows of a thread that it holds together

__global__ __launch_bounds__(kGroupThreads) void lora_group_kernel(const int32_t* adapter, int M, int n,
                                                                   int32_t* order, int32_t* of, int4* blocks,
                                                                   int* n_blocks) {
    __shared__ int s_at[kGroupMax + 1];      // counts, then the next place of each adapter's rows
    __shared__ int s_block[kGroupMax + 1];   // blocks up to and with each adapter
    __shared__ int s_first[kGroupMax + 1];
    __shared__ int2 s_wave[kGroupThreads / WAVE];
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    for (int j = tid; j <= n; j += kGroupThreads) s_at[j] = 0;
    int id[kGroupRows];
    auto read = [&](int m0) {
#pragma unroll
        for (int i = 0; i < kGroupRows; ++i) {
            const int j = adapter[min(m0 + i * kGroupThreads + tid, M - 1)];
            id[i] = j >= 0 && j < n ? j : n;
        }
    };
    // `use` for a wave's 64 rows at a time: they are of one adapter mostly, and move the count at once
    auto each = [&](int m0, auto use) {
#pragma unroll
        for (int i = 0; i < kGroupRows; ++i) {
            const int m = m0 + i * kGroupThreads + tid;
            if (m - lane >= M) break;
            const bool on = m < M;
            int at = 0;
            if (__ballot(on && id[i] == __builtin_amdgcn_readfirstlane(id[i])) == ~0ull) {
                if (lane == 0) at = atomicAdd(&s_at[id[i]], WAVE);
                at = __builtin_amdgcn_readfirstlane(at) + lane;
            } else if (on) {
                at = atomicAdd(&s_at[id[i]], 1);
            }
            if (on) use(m, at, id[i]);
        }
    };
    constexpr int kChunk = kGroupRows * kGroupThreads;
    read(0);
    __syncthreads();
    for (int m0 = 0; m0 < M; m0 += kChunk) {
        if (m0) read(m0);
        each(m0, [](int, int, int) {});
    }
    __syncthreads();
    int2 base = {0, 0};   // rows and blocks of the adapters before
    for (int j0 = 0; j0 <= n; j0 += kGroupThreads) {
        const int j = j0 + tid, count = j <= n ? s_at[j] : 0;
        const int mine = j < n ? (count + kSgRows - 1) / kSgRows : 0;
        int2 upto = {count, mine};
#pragma unroll
        for (int off = 1; off < WAVE; off <<= 1) {
            const int2 o = {__shfl_up(upto.x, off, WAVE), __shfl_up(upto.y, off, WAVE)};
            if (lane >= off) upto = {upto.x + o.x, upto.y + o.y};
        }
        if (lane == WAVE - 1) s_wave[wave] = upto;
        __syncthreads();
        int2 at = base;
        for (int w = 0; w < kGroupThreads / WAVE; ++w) {
            const int2 v = s_wave[w];
            if (w < wave) at = {at.x + v.x, at.y + v.y};
            base = {base.x + v.x, base.y + v.y};
        }
        if (j <= n) {
            s_at[j] = s_first[j] = at.x + upto.x - count;
            s_block[j] = at.y + upto.y;
        }
        __syncthreads();
    }
    if (tid == 0) *n_blocks = base.y;
    for (int b = tid; b < base.y; b += kGroupThreads) {
        int lo = 0, hi = n - 1;   // the first adapter whose blocks reach past b
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (s_block[mid] > b) hi = mid;
            else lo = mid + 1;
        }
        const int first = s_first[lo] + (b - (lo ? s_block[lo - 1] : 0)) * kSgRows;
        blocks[b] = int4{lo, first, min(kSgRows, s_first[lo + 1] - first), 0};
    }
    for (int m0 = 0; m0 < M; m0 += kChunk) {
        if (M > kChunk) read(m0);
        each(m0, [&](int m, int at, int j) {
            order[at] = m;
            of[at] = j;
        });
    }
}

// Bytes of A that workgroups of 16 rows may read at most, if their rows' adapters are mixed, before the
// rows are put in order.  With the product, K = N = 4096, in order and as they come, 16 adapters of
// rank 16: 1024 mixed rows (134 MB) 45 and 64 us, 1024 in runs 45 and 37; 512 rows 37 and 42, in runs 38
// and 30; 256 rows 31 and 34, in runs 31 and 27.  Which of the two the rows are is on the device, so the
// rule is for the mixed ones, which lose more (64) than runs do (45 for 37).  6 adapters of rank 64, which the caches hold, 512 mixed
// rows (100 MB) 51 and 49, in runs 51 and 35.
constexpr double kDirectBytes = 128e6;

static bool lora_grouped(int M, int K, int n, int rank) {
    if (n > kGroupMax) return false;
    const int most = n < 16 ? n : 16;
    return (double)((M + 15) / 16) * most * rank * K * 2 > kDirectBytes;
}

struct LoraWs {
    size_t u, order, of, blocks, n_blocks, total;
};

// Room for either form: the workspace's size does not depend on the number of adapters.
static LoraWs lora_ws(int M, int rank) {
    LoraWs w{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 256);
        return at;
    };
    const size_t tiles = ((size_t)M + 15) / 16;
    w.u = take(lora_u_bytes(tiles, (rank + 15) / 16));
    w.order = take((size_t)M * 4);
    w.of = take((size_t)M * 4);
    w.blocks = take(((size_t)M / kSgRows + (M < kGroupMax ? M : kGroupMax) + 1) * 16);
    w.n_blocks = take(4);
    w.total = o;
    return w;
}

size_t linear_lora_ws_bytes(int M, int, int rank) { return lora_ws(M, rank).total; }

hipError_t launch_lora_shrink(const int8_t* a, const float* a_scale, int M, int K, const uint16_t* A,
                              const float* scales, int n, int rank, const int32_t* adapter, void* ws,
                              LoraDev* out, hipStream_t stream) {
    const LoraWs L = lora_ws(M, rank);
    char* base = (char*)ws;
    const int steps = (rank + 15) / 16;
    ShrinkArgs p = {a, a_scale, A, scales, adapter, (uint16_t*)(base + L.u), M, K, n, rank, steps,
                    (const int32_t*)(base + L.order), (const int4*)(base + L.blocks),
                    (const int*)(base + L.n_blocks)};
    if (lora_grouped(M, K, n, rank)) {
        lora_group_kernel<<<1, kGroupThreads, 0, stream>>>(adapter, M, n, (int32_t*)(base + L.order),
                                                           (int32_t*)(base + L.of), (int4*)(base + L.blocks), (int*)(base + L.n_blocks));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const unsigned blocks = M / kSgRows + (M < n ? M : n);
        if (steps <= 1) lora_shrink_grouped_kernel<1><<<dim3(blocks), kSgWaves * WAVE, 0, stream>>>(p);
        else if (steps <= 2) lora_shrink_grouped_kernel<2><<<dim3(blocks), kSgWaves * WAVE, 0, stream>>>(p);
        else lora_shrink_grouped_kernel<4><<<dim3(blocks, (steps + 3) / 4), kSgWaves * WAVE, 0, stream>>>(p);
    } else {
        const int tiles = (M + 15) / 16, rows = M < 16 ? M : 16, most = rows < n ? rows : n;
        int turns = 2048 / (tiles * steps);
        turns = turns < 1 ? 1 : turns < most ? turns : most;
        int parts_log = 0;
        while (parts_log < 2 && tiles * turns * steps << parts_log < 256) ++parts_log;
        lora_shrink_kernel<<<dim3(tiles, turns, steps << parts_log), kSdWaves * WAVE, 0, stream>>>(p, parts_log);
    }
    out->u = p.u;
    const bool grouped = lora_grouped(M, K, n, rank);
    out->order = grouped ? p.order : nullptr;
    out->of = grouped ? (const int32_t*)(base + L.of) : adapter;
    out->n = n;
    out->rank = rank;
    out->steps = steps;
    return hipGetLastError();
}

}  // namespace moeq4
