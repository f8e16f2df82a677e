// Low-rank adapters beside the dense product of 8-bit codes: what the product's kernels add.
//
// u[m] = scale_j * a_scale[m] * (A_j a[m]), j = adapter[m], comes from the shrink kernel
// (lora_i8.hip).  The expansion B_j u is a matrix product of bf16: 16 columns of out are the
// rows of its A operand (B_j as it is), 16 rows of out its columns, and a step of its K of
// 32 holds 16 ranks twice: with u rounded to bf16, and with what that rounding left, so that u
// counts to 16 bits.  u lies in that operand's order, a kilobyte for 16 rows and 16 ranks.
// Rows of another adapter have zeros there, and keep their sums whatever the adapter holds.
#pragma once

#include "moe_device.h"
#include "moe_i8.h"

namespace moeq4 {

// Bytes of u of a number of tiles of 16 rows, and the byte among them where 16 ranks of a tile lie.
__host__ __device__ constexpr size_t lora_u_bytes(size_t tiles, int steps) { return tiles * steps * (WAVE * 16); }
__host__ __device__ constexpr size_t lora_u_at(size_t m_tile, int step, int steps, int lane) {
    return ((m_tile * steps + step) * WAVE + lane) * 16;
}

// 16 ranks of the rows of a tile of 16, as they lie.
__device__ __forceinline__ u32x4_t lora_u(const LoraDev& l, int m_tile, int step, int lane) {
    return *(const u32x4_t*)((const char*)l.u + lora_u_at(m_tile, step, l.steps, lane));
}

__device__ __forceinline__ bf16x8_t lora_only(bool mine, const u32x4_t& u) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mine ? u[i] : 0u;
    return __builtin_bit_cast(bf16x8_t, v);
}

// The same 16 ranks of 16 columns of adapter j, from column n0 on.
__device__ __forceinline__ u32x4_t lora_b(const LoraDev& l, int j, int N, int n0, int step,
                                           int lane) {
    const int n = n0 + lane % 16, rr = step * 16 + lane / 16 % 2 * 8;
    u32x4_t v = {0, 0, 0, 0};
    if (n < N && rr < l.rank) v = *(const u32x4_t*)(l.b + ((size_t)j * N + n) * l.rank + rr);
    return v;
}

// Row at place r of the product's order; places behind the last have the last row.
template <bool LORA>
__device__ __forceinline__ int row_at(const LoraDev& l, int r, int M) {
    r = min(r, M - 1);
    if constexpr (LORA) return l.order ? l.order[r] : r;
    return r;
}

// Adapter of the row at place r, or -1.
__device__ __forceinline__ int lora_of(const LoraDev& l, int r, int M) {
    const int j = l.of[min(r, M - 1)];
    return r < M && j >= 0 && j < l.n ? j : -1;
}

// No infinity or NaN among eight bf16.
__device__ __forceinline__ bool lora_finite(const u32x4_t& v) {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ok = ok && (v[i] & 0x7F80u) != 0x7F80u && (v[i] & 0x7F800000u) != 0x7F800000u;
    return ok;
}

// v += b u in the rows that are `mine`.
__device__ __forceinline__ void lora_add(const u32x4_t& b, const u32x4_t& u, bool mine, f32x4_t& v) {
    const f32x4_t t = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, b), lora_only(mine, u), v);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = mine ? t[q] : v[q];
}

}  // namespace moeq4
