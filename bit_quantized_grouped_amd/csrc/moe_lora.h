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

// Infinities and NaN in b reach their columns of their adapter's rows alone, as by the formula.
// Two things stand against that: zeros in other rows' places (0 times an infinity is NaN), and
// what u's rounding left, which may be 0 or of the other sign.

// Bits 15 and 31 are set for the infinities and NaN among two bf16: an exponent of all ones carries.
__device__ __forceinline__ uint32_t lora_infinite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ uint32_t lora_infinite(const u32x4_t& v) {
    return lora_infinite(v[0]) | lora_infinite(v[1]) | lora_infinite(v[2]) | lora_infinite(v[3]);
}

// b with `instead` and its sign for every such value.
__device__ __forceinline__ u32x4_t lora_without(const u32x4_t& b, uint32_t instead) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t is = lora_infinite(b[i]), all = (is >> 15) * 0xFFFFu;
        v[i] = (b[i] & ~all) | (all & ((b[i] & 0x80008000u) | instead * 0x10001u));
    }
    return v;
}

// What such values of their adapters' b add to rows at places r0 .. + rows and columns n0 .. n1 - 1 of
// out, where they counted as finite values of their sign: infinities and NaN, after the rounding as
// before it.  By one wave, which has stored these.  Slow, and rarely called.
__device__ __forceinline__ void lora_add_infinite(const LoraDev& l, int M, int N, int r0, int rows, int n0, int n1,
                                                  uint16_t* out) {
    __threadfence();   // the values that other lanes stored
    for (int r = r0 + __lane_id(); r < min(r0 + rows, M); r += WAVE) {
        const int j = lora_of(l, r, M);
        if (j < 0) continue;
        uint16_t* o = out + (size_t)row_at<true>(l, r, M) * N;
        const uint16_t* b = l.b + ((size_t)j * N + n0) * l.rank;
        for (int c = n0; c < n1; ++c, b += l.rank) {
            float sum = 0.f;
            for (int k = 0; k < l.rank; k += 8) {
                if (!lora_infinite(*(const u32x4_t*)(b + k))) continue;
                const uint16_t* u = (const uint16_t*)((const char*)l.u + lora_u_at(r / 16, k / 16, l.steps, r % 16 + k / 8 % 2 * 16));
                for (int i = 0; i < 8; ++i)
                    if (lora_infinite(b[k + i])) sum += bf16_to_f32(b[k + i]) * bf16_to_f32(u[i]);
            }
            if (sum != 0.f) o[c] = (uint16_t)pack_bf16x2(bf16_to_f32(o[c]) + sum, 0.f);
        }
    }
}

// v += b u in the rows that are `mine`.
__device__ __forceinline__ void lora_add(const u32x4_t& b, const u32x4_t& u, bool mine, f32x4_t& v) {
    const f32x4_t t = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, b), lora_only(mine, u), v);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = mine ? t[q] : v[q];
}

}  // namespace moeq4
