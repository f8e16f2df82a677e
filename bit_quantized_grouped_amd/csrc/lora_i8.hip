// The adapters' first product: u[m, r] = scale_j * a_scale[m] * sum_k A_j[r, k] a[m, k] for the
// rows m that have an adapter j = adapter[m] (codes a as bf16, which holds them exactly;
// products exact, sums fp32).
//
// A workgroup takes 16 MT rows, every gridDim.y-th of the adapters among them, and a part of
// K, which its 8 waves split once more; their sums meet in LDS.  Rows of other adapters are
// zeros in the products.  Bound by reading A, once for each tile of rows that has the adapter.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_lora.h"

namespace moeq4 {

constexpr int kLsWaves = 8;

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

// RT: tiles of 16 ranks.
template <int MT, int RT>
__global__ __launch_bounds__(kLsWaves* WAVE) void lora_shrink_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, int M, int K, const uint16_t* __restrict__ A,
    const float* __restrict__ scales, const int32_t* __restrict__ adapter, int n, int R,
    float* __restrict__ u) {
    __shared__ f32x4_t s_part[kLsWaves][RT][WAVE];
    const int lane = threadIdx.x % WAVE, fr = lane % 16, fp = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int m0 = blockIdx.x * 16 * MT;
    const int steps = K / 64, share = kLsWaves * gridDim.z, at = blockIdx.z * kLsWaves + wave;
    const int s0 = (int)((long long)steps * at / share), s1 = (int)((long long)steps * (at + 1) / share);
    int of[MT];
    unsigned long long left[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m0 + m * 16 + fr;
        const int j = r < M ? adapter[r] : -1;
        of[m] = j >= 0 && j < n ? j : -1;
        left[m] = __ballot(of[m] >= 0) & 0xFFFF;
    }
    for (int turn = 0;; ++turn) {
        // the next adapter among the rows
        int j = -1;
#pragma unroll
        for (int m = MT - 1; m >= 0; --m)
            if (left[m]) j = __builtin_amdgcn_readlane(of[m], __builtin_ctzll(left[m]));
        if (j < 0) break;
        bool mine[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            mine[m] = of[m] == j;
            left[m] &= ~__ballot(mine[m]);
        }
        if (turn % (int)gridDim.y != (int)blockIdx.y) continue;
        f32x4_t acc[MT][RT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        const uint16_t* Aj = A + (size_t)j * R * K;
        for (int s = s0; s < s1; ++s) {
            const int kb = s * 64 + fp * 16;
            u32x4_t w[RT][2], c[MT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int r = t * 16 + fr;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[t][i] = r < R ? *(const u32x4_t*)(Aj + (size_t)r * K + kb + 8 * i) : u32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
                c[m] = mine[m] ? *(const u32x4_t*)(a + (size_t)(m0 + m * 16 + fr) * K + kb) : u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8_t b = codes_bf16(c[m][2 * i], c[m][2 * i + 1]);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[m][t] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, w[t][i]), b, acc[m][t]);
                }
        }
        const float scale = scales[j];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (!__ballot(mine[m])) continue;
            __syncthreads();
#pragma unroll
            for (int t = 0; t < RT; ++t) s_part[wave][t][lane] = acc[m][t];
            __syncthreads();
            for (int t = wave; t < RT; t += kLsWaves) {
                f32x4_t v = s_part[0][t][lane];
#pragma unroll
                for (int w = 1; w < kLsWaves; ++w) v += s_part[w][t][lane];
                const int row = m0 + m * 16 + fr, r = t * 16 + fp * 4;
                if (mine[m] && r < R)
                    *(f32x4_t*)(u + ((size_t)blockIdx.z * M + row) * R + r) = v * (a_scale[row] * scale);
            }
        }
    }
}

static int lora_row_tiles(int M) { return M >= 1024 ? 4 : 1; }

// Parts of K, so that a few rows still reach many compute units.
static int lora_parts(int M, int K) {
    const int tiles = (M + 15) / 16;
    int parts = M >= 1024 ? 2 : 32 / tiles;
    const int most = K / 512 > 0 ? K / 512 : 1;
    parts = parts < 1 ? 1 : parts;
    parts = parts < most ? parts : most;
    return parts < 8 ? parts : 8;
}

size_t linear_lora_ws_bytes(int M, int K, int rank) {
    return align_up((size_t)lora_parts(M, K) * M * rank * 4, 256);
}

template <int MT>
static void launch_shrink(dim3 grid, const int8_t* a, const float* a_scale, int M, int K, const uint16_t* A,
                          const float* scales, const int32_t* of, int n, int R, float* u, hipStream_t stream) {
#define MOE_SHRINK(RT) \
    lora_shrink_kernel<MT, RT><<<grid, kLsWaves * WAVE, 0, stream>>>(a, a_scale, M, K, A, scales, of, n, R, u)
    if (R <= 16) MOE_SHRINK(1);
    else if (R <= 32) MOE_SHRINK(2);
    else if (R <= 64) MOE_SHRINK(4);
    else MOE_SHRINK(8);
#undef MOE_SHRINK
}

hipError_t launch_lora_shrink(const int8_t* a, const float* a_scale, int M, int K, const uint16_t* A,
                              const float* scales, int n, int rank, const int32_t* adapter, void* ws,
                              LoraDev* out, hipStream_t stream) {
    const int mt = lora_row_tiles(M), tiles = (M + 16 * mt - 1) / (16 * mt), parts = lora_parts(M, K);
    int turns = 1024 / (tiles * parts);
    turns = turns < 1 ? 1 : turns;
    const int rows = 16 * mt < M ? 16 * mt : M, most = rows < n ? rows : n;
    turns = turns < most ? turns : most;
    float* u = (float*)ws;
    const dim3 grid(tiles, turns, parts);
    if (mt == 1) launch_shrink<1>(grid, a, a_scale, M, K, A, scales, adapter, n, rank, u, stream);
    else launch_shrink<4>(grid, a, a_scale, M, K, A, scales, adapter, n, rank, u, stream);
    out->u = u;
    out->of = adapter;
    out->n = n;
    out->rank = rank;
    out->parts = parts;
    out->part = (size_t)M * rank;
    return hipGetLastError();
}

}  // namespace moeq4
