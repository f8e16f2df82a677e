// Root-mean-square norm with the residual's addition and an 8-bit output, the
// row-wise 8-bit quantisation alone, and the way back to bf16.
//
//   v = x + residual (fp32), m = mean(v^2), y = v * weight / sqrt(m + eps),
//   scale = max|y| / 127, q = rne(y * (127 / max|y|)); a row of zeros has scale 0, one with a
//   NaN the scale NaN.
//
// max|y| = max|v * weight| / sqrt(m + eps), so the sum of squares and the
// maximum come out of one pass over registers and one joint reduction: a row
// is read once and written once.
#include "moe_device.h"
#include "moe_i8.h"

namespace moeq4 {

constexpr int kNormRows = 4;   // rows per workgroup where one wave takes a row

__device__ __forceinline__ void unpack_bf16x8(u32x4_t w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4_t pack_bf16x8(const float (&f)[8]) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return w;
}

template <bool STREAM>
__device__ __forceinline__ u32x4_t load_piece(const uint16_t* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load((const u32x4_t*)p);
    else return *(const u32x4_t*)p;
}

// NW waves per row, V 8-element pieces per lane, NORM false: quantisation only.
// STREAM: the inputs are read, and y written, with the non-temporal hint.
template <int NW, int V, bool NORM, bool STREAM>
__global__ __launch_bounds__(NW == 1 ? kNormRows * WAVE : NW * WAVE) void norm_i8_kernel(
    const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight, float eps,
    int T, int H, uint16_t* sum, uint16_t* y, int8_t* q, float* q_scale) {
    // sum may be x or residual: a lane stores only what it has loaded itself
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
    const int t = NW == 1 ? blockIdx.x * kNormRows + wave : blockIdx.x;
    if (NW == 1 && t >= T) return;
    const int tid = NW == 1 ? lane : (int)threadIdx.x;
    const size_t row = (size_t)t * H;
    float f[V][8], w[V][8];
    float sq = 0.f, top = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NW * WAVE + tid) * 8;
        u32x4_t a = {0, 0, 0, 0};
        if (c < H) a = load_piece<STREAM>(x + row + c);
        unpack_bf16x8(a, f[v]);
        if (NORM) {
            u32x4_t wv = {0, 0, 0, 0};
            if (c < H) wv = *(const u32x4_t*)(weight + c);
            unpack_bf16x8(wv, w[v]);
            if (residual && c < H) {
                float r[8];
                unpack_bf16x8(load_piece<STREAM>(residual + row + c), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[v][i] += r[i];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (NORM) {
                sq = __builtin_fmaf(f[v][i], f[v][i], sq);
                w[v][i] *= f[v][i];
                top = max_abs(top, w[v][i]);
            } else {
                top = max_abs(top, f[v][i]);
            }
        }
#pragma unroll
    for (int off = WAVE / 2; off >= 1; off >>= 1) {
        if (NORM) sq += shfl_xor(sq, off);
        top = max_abs(top, shfl_xor(top, off));
    }
    if (NW > 1) {
        __shared__ float s_sq[NW], s_top[NW];
        if (lane == 0) {
            s_sq[wave] = sq;
            s_top[wave] = top;
        }
        __syncthreads();
        sq = s_sq[0];
        top = s_top[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
            sq += s_sq[i];
            top = max_abs(top, s_top[i]);
        }
    }
    const float inv = NORM ? 1.0f / sqrtf(sq / (float)H + eps) : 1.0f;
    top *= inv;
    float to_code;
    const float scale = row_scale(top, &to_code);
    if (q_scale && tid == 0) q_scale[t] = scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NW * WAVE + tid) * 8;
        if (c >= H) break;
        // the sum is read again a block later, y and the codes by the next kernel
        if (NORM && sum) __builtin_nontemporal_store(pack_bf16x8(f[v]), (u32x4_t*)(sum + row + c));
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = NORM ? w[v][i] * inv : f[v][i];
        if (NORM && y) {
            if (STREAM) __builtin_nontemporal_store(pack_bf16x8(o), (u32x4_t*)(y + row + c));
            else *(u32x4_t*)(y + row + c) = pack_bf16x8(o);
        }
        if (q) {
            u32x2_t p;
            p[0] = row_codes(o[0], o[1], o[2], o[3], to_code);
            p[1] = row_codes(o[4], o[5], o[6], o[7], to_code);
            *(u32x2_t*)(q + row + c) = p;
        }
    }
}

template <bool NORM>
static hipError_t launch_rows(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                              float eps, int T_all, int H, uint16_t* sum, uint16_t* y, int8_t* q,
                              float* q_scale, hipStream_t stream) {
    // Inputs that do not fit half of the Infinity Cache (256 MB) are not there any more,
    // wherever they come from; read without allocating in it they leave the codes there for
    // the next kernel.  8191 x 7168 with the residual (by 4 waves a row): 90 us against 102, and
    // reading the codes back 28 against 38; 2048 x 2048, whose inputs are there: 11.4 against 8.3.
    const bool big = (residual ? 4ll : 2ll) * T_all * H > (128ll << 20);
#define MOE_NORM_S(NW, V, S)                                                                    \
    norm_i8_kernel<NW, V, NORM, S><<<NW == 1 ? (T + kNormRows - 1) / kNormRows : T,             \
                                     NW == 1 ? kNormRows * WAVE : NW * WAVE, 0, stream>>>(      \
        x + t0 * H, at(residual, t0 * H), weight, eps, T, H, at(sum, t0 * H), at(y, t0 * H),    \
        at(q, t0 * H), at(q_scale, t0))
#define MOE_NORM(NW, V)                      \
    {                                        \
        if (big) MOE_NORM_S(NW, V, true);    \
        else MOE_NORM_S(NW, V, false);       \
    }
    // Wider rows by several waves, one or two pieces a lane: their loads and stores are the chain
    // of a call of few rows.  One row of 2048 by 4 waves 2.5 us, by one 3.9 (2048 rows 8.6, 9.2);
    // 64 rows of 7168 by 8 waves 4.3, by 4 4.9 (8191 rows 84, 90; by 16 88).
    auto at = [](auto* p, size_t by) { return p ? p + by : p; };
    for (size_t t0 = 0; t0 < (size_t)T_all; t0 += kItemsALaunch) {
        const int T = (int)min((size_t)T_all - t0, (size_t)kItemsALaunch);
        if (H <= 512) MOE_NORM(1, 1)
        else if (H <= 1024) MOE_NORM(1, 2)
        else if (H <= 2048) MOE_NORM(4, 1)
        else if (H <= 4096) MOE_NORM(8, 1)
        else if (H <= 8192) MOE_NORM(8, 2)
        else MOE_NORM(16, 2)   // up to kMaxNormWidth
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
#undef MOE_NORM
#undef MOE_NORM_S
    return hipSuccess;
}

hipError_t launch_norm_i8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                          float eps, int T, int H, uint16_t* sum, uint16_t* y, int8_t* q,
                          float* q_scale, hipStream_t stream) {
    return launch_rows<true>(x, residual, weight, eps, T, H, sum, y, q, q_scale, stream);
}

hipError_t launch_quant_i8(const uint16_t* x, int R, int K, int8_t* q, float* scale,
                           hipStream_t stream) {
    return launch_rows<false>(x, nullptr, nullptr, 0.f, R, K, nullptr, nullptr, q, scale, stream);
}

// A wave takes a row, or 1024 codes of one where rows alone are few waves: 16 codes in,
// 16 bf16 out per lane and step.  Bound by HBM (8191 x 7168 codes 28 us, 6.3 TB/s); parts
// shorten 64 rows of 7168 from 5.1 to 2.5 us, at 8192 x 2048 they cost 11.0 against 9.9.
constexpr uint32_t kDequantWaves = 4, kDequantPart = WAVE * 16;
constexpr int kDequantPartRows = 2048;
__global__ __launch_bounds__(kDequantWaves * WAVE) void dequant_i8_kernel(
    const int8_t* __restrict__ q, const float* __restrict__ scale, uint32_t R, uint32_t K,
    uint32_t parts, uint16_t* __restrict__ out) {
    const uint32_t lane = threadIdx.x % WAVE;
    const uint32_t at = blockIdx.x * kDequantWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const uint32_t r = at / parts;
    if (r >= R) return;
    const float s = scale[r];
    const int8_t* src = q + (size_t)r * K;
    uint16_t* dst = out + (size_t)r * K;
    const uint32_t part = at - r * parts, end = parts > 1 ? min(K, (part + 1) * kDequantPart) : K;
#pragma unroll 4
    for (uint32_t c = part * kDequantPart + lane * 16; c < end; c += WAVE * 16) {
        const i32x4_t w = *(const i32x4_t*)(src + c);
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = (float)((w[i / 4] << (24 - 8 * (i % 4))) >> 24) * s;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            u32x4_t o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(f[8 * p + 2 * i], f[8 * p + 2 * i + 1]);
            *(u32x4_t*)(dst + c + 8 * p) = o;
        }
    }
}

hipError_t launch_dequant_i8(const int8_t* q, const float* scale, int R, int K, uint16_t* out,
                             hipStream_t stream) {
    const uint32_t parts = R < kDequantPartRows ? ((uint32_t)K + kDequantPart - 1) / kDequantPart : 1;
    const int most = parts > 1 ? (int)(16u * kItemsALaunch / parts) : kItemsALaunch;   // parts are at most 2^21
    for (size_t r0 = 0; r0 < (size_t)R; r0 += most) {
        const int rows = R - (long long)r0 < most ? R - (int)r0 : most;
        const long long waves = (long long)rows * parts;
        dequant_i8_kernel<<<(unsigned)((waves + kDequantWaves - 1) / kDequantWaves), kDequantWaves * WAVE,
                            0, stream>>>(q + r0 * K, scale + r0, rows, K, parts, out + r0 * K);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace moeq4
