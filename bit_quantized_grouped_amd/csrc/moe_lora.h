// Low-rank adapters beside the dense product of 8-bit codes: what the product's kernels add.
//
// u[m] = scale_j * a_scale[m] * (A_j a[m]), j = adapter[m], comes from the shrink kernel
// (lora_i8.hip) in fp32, in `parts` pieces of K that are added here.  The expansion B_j u is a
// matrix product of bf16: 16 columns of out are the rows of its A operand (B_j as it is), 16
// rows of out its columns, and a step of its K of 32 holds 16 ranks twice: with u rounded to
// bf16, and with what that rounding left, so that u counts to 16 bits.  Rows of another
// adapter have zeros, and keep their sums whatever the adapter holds.
#pragma once

#include "moe_device.h"
#include "moe_i8.h"

namespace moeq4 {

// Ranks rr .. rr + 7 of a row's u as bf16, or the rest of their rounding.
__device__ __forceinline__ bf16x8_t lora_u(const LoraDev& l, size_t row, int rr, bool on, bool rest) {
    f32x4_t v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (on) {
        const float* u = l.u + row * l.rank + rr;
        for (int i = 0; i < l.parts; ++i, u += l.part) {
            v[0] += *(const f32x4_t*)u;
            v[1] += *(const f32x4_t*)(u + 4);
        }
    }
    bf16x8_t r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v[i / 4][i % 4];
        const __bf16 h = (__bf16)x;
        r[i] = rest ? (__bf16)(x - (float)h) : h;
    }
    return r;
}

// Ranks rr .. rr + 7 of column n of adapter j.
__device__ __forceinline__ bf16x8_t lora_b(const LoraDev& l, int j, int N, int n, int rr) {
    u32x4_t v = {0, 0, 0, 0};
    if (n < N && rr < l.rank) v = *(const u32x4_t*)(l.b + ((size_t)j * N + n) * l.rank + rr);
    return __builtin_bit_cast(bf16x8_t, v);
}

// Adapter of row r, or -1.
__device__ __forceinline__ int lora_of(const LoraDev& l, int r, int M) {
    const int j = r < M ? l.of[r] : -1;
    return j >= 0 && j < l.n ? j : -1;
}

// One adapter's part of the pieces at rows m0 .. +15 and columns n0 + 16 i: v[i] is D of the
// 16 x 16 product, column n0 + 16 i + 4 (lane / 16) + 0..3, row m0 + lane % 16.  j: the adapter,
// `of`: the one of this lane's row.
template <int NF>
__device__ __forceinline__ void lora_expand(const LoraDev& l, int j, int of, int N, int m0, int n0,
                                            f32x4_t (&v)[NF]) {
    const int lane = __lane_id(), fr = lane % 16, fp = lane / 16;
    const bool mine = of == j;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        f32x4_t t = v[i];
        for (int r0 = 0; r0 < l.rank; r0 += 16) {
            const int rr = r0 + fp % 2 * 8;
            const bf16x8_t b = lora_b(l, j, N, n0 + i * 16 + fr, rr);
            const bf16x8_t u = lora_u(l, (size_t)(m0 + fr), rr, mine && rr < l.rank, fp >= 2);
            t = mfma_16x16x32(b, u, t);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i][q] = mine ? t[q] : v[i][q];
    }
}

}  // namespace moeq4
