// Internal interface and device helpers of the 8-bit operators (norm_i8.hip,
// gemm_i8.hip, the scored routing of route.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_launch.h"

namespace moeq4 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Widest row of the norm and the row quantisation: 16 waves of 2 pieces of 8 a lane.
constexpr int kMaxNormWidth = 16384;

struct I8MatDev {
    const int8_t* codes;
    const float* scales;   // [n_exp, N]
    int tiles;             // 0: rows [N, K]; 1: 16 x 64 tiles (moe_i8_prepack)
};

constexpr int kScoredMaxK = 64;        // one slot per lane of the selecting wave
constexpr int kScoredMaxGroups = 64;   // one group per lane

// Selection rule of the scored routing (moe_score_rule with its checks done).
struct ScoreRule {
    int sigmoid;       // 0: softmax
    int n_groups, topk_groups, group_size;
    int top2;          // a group's worth: its two best choices' sum, else its best choice
    int renormalise;
    float scale;
};

#ifdef __HIPCC__
// Four values rounded to nearest even as 8-bit codes, the first in the low byte.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
    const int ia = (int)__builtin_rintf(a), ib = (int)__builtin_rintf(b);
    const int ic = (int)__builtin_rintf(c), id = (int)__builtin_rintf(d);
    return (uint32_t)(ia & 255) | (uint32_t)(ib & 255) << 8 | (uint32_t)(ic & 255) << 16 |
           (uint32_t)id << 24;
}
#endif

#ifdef __HIPCC__
// The larger of `top` and |v|; NaN wins over every number (fmaxf would drop it).
__device__ __forceinline__ float max_abs(float top, float v) {
    return __builtin_elementwise_maximum(top, __builtin_fabsf(v));
}

// Scale of a row of largest magnitude `top`, and the factor from its values to codes, 0 where
// the codes are 0.  A row below 2^-119 counts as zeros: 127 / top would pass fp32's range.  The
// scale of a row with an infinity or NaN is infinite or NaN, so all of it comes back as NaN.
__device__ __forceinline__ float row_scale(float top, float* to_code) {
    const bool tiny = top < 0x1p-119f;
    *to_code = top >= 0x1p-119f && top <= 0x1.fffffep127f ? 127.0f / top : 0.f;
    return tiny ? 0.f : top / 127.0f;
}

// Codes of four values of a row by row_scale's factor.
__device__ __forceinline__ uint32_t row_codes(float a, float b, float c, float d, float to_code) {
    const uint32_t p = pack_codes(a * to_code, b * to_code, c * to_code, d * to_code);
    return to_code > 0.f ? p : 0u;   // a NaN has no code
}
#endif

#ifdef __HIPCC__
// The byte that a value loses when it is rounded to bf16: its fp32 bits are the bf16's and 256
// times this, within half a step of 24 bits (2^-16 of the value; a value midway between two
// bf16 keeps 127 of 128: 2^-15).  A bf16 value itself has 0.
__device__ __forceinline__ int low_byte(float v, uint32_t bf16) {
    const int off = (int)(__builtin_bit_cast(uint32_t, v) - (bf16 << 16));
    return max(-128, min(127, (off + 128) >> 8));
}

// Bits of the fp32 value of a bf16 in the high half of `high` and its low byte.
__device__ __forceinline__ uint32_t with_low_byte(uint32_t high, int low) {
    return high + ((uint32_t)low << 8);
}
#endif

// A grid dimension ends below 2^32 threads.  Work of up to 1024 threads an item goes by so many
// items a launch.
constexpr int kItemsALaunch = 1 << 21;

// norm_i8.hip
hipError_t launch_norm_i8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                          float eps, int T, int H, uint16_t* sum, uint16_t* y, int8_t* q,
                          float* q_scale, hipStream_t stream);
hipError_t launch_quant_i8(const uint16_t* x, int R, int K, int8_t* q, float* scale,
                           hipStream_t stream);
hipError_t launch_dequant_i8(const int8_t* q, const float* scale, int R, int K, uint16_t* out,
                             hipStream_t stream);

// route.hip
size_t scored_ws_bytes(int T, int E, int k);
hipError_t launch_route_i8(const float* logits, int T, int E, int k, int block_rows, int max_blocks,
                           const RoutingDev& r, void* ws, hipStream_t stream);
hipError_t launch_route_scored(const float* logits, const float* bias, const ScoreRule& rule, int T,
                               int E, int k, int block_rows, int max_blocks, const RoutingDev& r,
                               void* ws, hipStream_t stream);

// gemm_i8.hip
hipError_t launch_prepack_i8(const int8_t* src, int n_exp, int N, int K, int8_t* dst,
                             hipStream_t stream);
size_t linear_i8_ws_bytes(int M, int N, int K);
hipError_t launch_linear_i8(const int8_t* a, const float* a_scale, int M, int K, const I8MatDev& w,
                            int N, uint16_t* out, void* ws, hipStream_t stream);
struct GemmI8Problem {
    const int8_t* x;          // [T, H]
    const float* x_scale;     // [T]
    int T, H, I, I_sh, E, k, block_rows, max_blocks;
    RoutingDev r;
    I8MatDev gate, up, down, sh_gate, sh_up, sh_down;
    uint16_t* expert_out;
    uint16_t* shared_out;
};
// Workspace: SwiGLU activations fp32 (routed rows, then the shared expert's),
// their 8-bit codes and one scale per row; and the low bytes of the outputs
// (low_byte), where the activations were.
struct GemmI8Ws {
    size_t h, h_sh, low, low_sh, q, q_sh, scale, scale_sh, total;
};
GemmI8Ws gemm_i8_ws_layout(int T, int H, int I, int I_sh, int k);
// want_low: the outputs' low bytes too, into the workspace
hipError_t launch_grouped_i8(const GemmI8Problem& p, void* ws, bool want_low, hipStream_t stream);

// combine.hip: the weighted sum over outputs with their low bytes
hipError_t launch_combine_low(const uint16_t* expert_out, const int8_t* low, const uint16_t* shared_out,
                              const int8_t* shared_low, const int32_t* assign_row, const float* topk_w,
                              int T, int H, int k, uint16_t* y, hipStream_t stream);

// decode_i8.hip: moe_layer_i8 of few tokens; a single one's routing arrays included
bool decode_i8_fits(const GemmI8Problem& p);
hipError_t launch_decode_i8(const GemmI8Problem& p, const float* logits, const float* bias,
                            const ScoreRule* rule, void* ws, uint16_t* y, hipStream_t stream);

}  // namespace moeq4
