// A few tokens, each on its own, through the layer over 8-bit codes: two launches for one
// token, and the routing in front for more.
//
//   decode_i8_gateup_kernel: a workgroup owns 16 columns of one slot (a chosen
//     expert, or the shared expert) of one token; for a single token its wave 0
//     selects the experts itself (the same selection as the routing call), then its
//     waves split K, stream the gate's and up's tiles, and join their integer sums
//     through LDS: h = silu(g) * u in fp32.  One more workgroup writes the routing
//     arrays of a single token.
//   decode_i8_down_kernel: a workgroup owns 8 columns of a token's output; its waves
//     take a slot each, quantise the slot's h to codes (scale max|h| / 127 as in
//     the grouped path), stream the slot's 8 down rows, and y is the weighted sum
//     over the slots in slot order, the shared expert last, rounded once.
//
// Bound by bytes and by the chain of waits: the selection must end before a weight
// address is known, and down starts after all of gate/up.  Tokens that share an expert
// read it once each, so this form is for few tokens, of many or of small experts; it has
// two launches less than the grouped one and no expert_out.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_score.h"

namespace moeq4 {

// Waves that split K in gate/up, and the 64-K steps whose loads a wave has in flight: at H =
// 2048 8 x 4 takes 6.6 us, 4 x 8 7.4, 16 x 2 8.7.
constexpr int kDgWaves = 8;
constexpr int kDgAhead = 4;
constexpr int kDdAhead = 8;     // the same of a wave of down
constexpr int kDdMaxWaves = 16;

struct DecodeI8Args {
    GemmI8Problem p;
    const float* logits;
    const float* bias;
    ScoreRule rule;
    int scored;                // 0: moe_route's selection
    float* h;                  // [k][I], fp32
    float* h_sh;               // [I_sh]
    uint16_t* y;
};

__device__ __forceinline__ i32x4_t mfma16(i32x4_t a, i32x4_t b, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// EPL 0: the experts are chosen already, in p.r.
template <int EPL>
__global__ __launch_bounds__(kDgWaves* WAVE) void decode_i8_gateup_kernel(DecodeI8Args d) {
    __shared__ int s_idx[kScoredMaxK];
    __shared__ float s_w[kScoredMaxK];
    __shared__ uint32_t s_scr[3 * kScoredMaxK];
    __shared__ i32x4_t s_part[kDgWaves][2][4];
    const GemmI8Problem& p = d.p;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int k = p.k, H = p.H, token = blockIdx.y;
    const int tiles = p.I / 16, routed = k * tiles, all = routed + p.I_sh / 16;
    const int id = blockIdx.x;
    const bool shared = id >= routed && id < all;
    if constexpr (EPL > 0) if (!shared) {
        if (wave == 0) {
            if (d.scored) score_topk_token<EPL>(d.logits, d.bias, p.E, k, d.rule, s_idx, s_w);
            else
                topk_token<EPL>(d.logits, p.E, k, s_idx, s_w, s_scr, (int*)(s_scr + k),
                                (float*)(s_scr + 2 * k));
        }
        __syncthreads();
        if (id == all) {
            write_one_token(p.r, p.E, k, p.max_blocks, s_idx, s_w, tid, kDgWaves * WAVE);
            return;
        }
    }
    const int slot = shared ? k : id / tiles;
    const int tile = shared ? id - routed : id - slot * tiles;
    const int e = shared ? 0
                         : __builtin_amdgcn_readfirstlane(EPL > 0 ? s_idx[slot]
                                                                  : p.r.topk_idx[token * k + slot]);
    const I8MatDev& mg = shared ? p.sh_gate : p.gate;
    const I8MatDev& mu = shared ? p.sh_up : p.up;
    const int N = shared ? p.I_sh : p.I, c0 = tile * 16;
    const size_t base = (size_t)e * N * H + (size_t)c0 * H;
    const int8_t *wg = mg.codes + base, *wu = mu.codes + base;
    const uint32_t w_lane =
        mg.tiles ? lane * 16 : (uint32_t)(lane % 16) * (uint32_t)H + (lane / 16) * 16;
    const uint32_t w_step = mg.tiles ? 1024u : 64u;
    const int8_t* x = p.x + (size_t)token * H + (lane / 16) * 16;
    const int steps = H / 64, s0 = steps * wave / kDgWaves, s1 = steps * (wave + 1) / kDgWaves;
    i32x4_t ag = {0, 0, 0, 0}, au = {0, 0, 0, 0};
    for (int s = s0; s < s1; s += kDgAhead) {
        i32x4_t g[kDgAhead], u[kDgAhead], a[kDgAhead];
#pragma unroll
        for (int i = 0; i < kDgAhead; ++i)
            if (s + i < s1) {
                const uint32_t o = w_lane + (uint32_t)(s + i) * w_step;
                g[i] = __builtin_nontemporal_load((const i32x4_t*)(wg + o));
                u[i] = __builtin_nontemporal_load((const i32x4_t*)(wu + o));
                a[i] = *(const i32x4_t*)(x + (s + i) * 64);
            }
#pragma unroll
        for (int i = 0; i < kDgAhead; ++i)
            if (s + i < s1) {
                ag = mfma16(g[i], a[i], ag);
                au = mfma16(u[i], a[i], au);
            }
    }
    // every column of the products is the token: lanes 0, 16, 32, 48 hold rows 0 .. 15
    if (lane % 16 == 0) {
        s_part[wave][0][lane / 16] = ag;
        s_part[wave][1][lane / 16] = au;
    }
    __syncthreads();
    if (tid < 16) {
        int g = 0, u = 0;
#pragma unroll
        for (int w = 0; w < kDgWaves; ++w) {
            g += s_part[w][0][tid / 4][tid % 4];
            u += s_part[w][1][tid / 4][tid % 4];
        }
        const float xs = p.x_scale[token];
        const size_t col = (size_t)e * N + c0 + tid;
        const float gv = (float)g * xs * mg.scales[col], uv = (float)u * xs * mu.scales[col];
        (shared ? d.h_sh + (size_t)token * N : d.h + (size_t)(token * k + slot) * N)[c0 + tid] = silu_f32(gv) * uv;
    }
}

__global__ __launch_bounds__(kDdMaxWaves* WAVE) void decode_i8_down_kernel(DecodeI8Args d, int ldq) {
    extern __shared__ __attribute__((aligned(16))) int8_t s_q[];   // [waves][ldq] codes of a wave's slot
    __shared__ float s_y[kDdMaxWaves][8];
    const GemmI8Problem& p = d.p;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int waves = blockDim.x / WAVE;
    const int k = p.k, slots = k + (p.I_sh ? 1 : 0), token = blockIdx.y;
    // 8 of a tile's 16 columns: twice the workgroups, one for each CU at H = 2048
    const int c0 = blockIdx.x * 8, cols = c0 / 16 * 16;
    const bool on = (lane % 16) / 8 == (int)blockIdx.x % 2;
    int8_t* q = s_q + wave * ldq;
    float y = 0.f;   // lanes 0 .. 7: column c0 + lane
    for (int j = wave; j < slots; j += waves) {
        const bool shared = j == k;
        const int K = shared ? p.I_sh : p.I;
        const int e = shared ? 0 : __builtin_amdgcn_readfirstlane(p.r.topk_idx[token * k + j]);
        const I8MatDev& m = shared ? p.sh_down : p.down;
        const int8_t* w = m.codes + (size_t)e * p.H * K + (size_t)cols * K;
        const uint32_t w_lane =
            m.tiles ? lane * 16 : (uint32_t)(lane % 16) * (uint32_t)K + (lane / 16) * 16;
        const uint32_t w_step = m.tiles ? 1024u : 64u;
        const float* h = shared ? d.h_sh + (size_t)token * K : d.h + (size_t)(token * k + j) * K;
        const int steps = K / 64;
        i32x4_t wv[kDdAhead];
#pragma unroll
        for (int i = 0; i < kDdAhead; ++i)
            if (i < steps && on)
                wv[i] = __builtin_nontemporal_load((const i32x4_t*)(w + (w_lane + i * w_step)));
            else
                wv[i] = i32x4_t{0, 0, 0, 0};
        // the slot's row: maximum, then codes into LDS while the first weights arrive
        constexpr int KEEP = 2;   // pieces of 256 values that stay in registers
        f32x4_t v[KEEP];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = i * 256 + lane * 4;
            v[i] = c < K ? *(const f32x4_t*)(h + c) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < 4; ++b) top = max_abs(top, v[i][b]);
        }
        for (int c = KEEP * 256 + lane * 4; c < K; c += 256) {
            const f32x4_t t = *(const f32x4_t*)(h + c);
#pragma unroll
            for (int b = 0; b < 4; ++b) top = max_abs(top, t[b]);
        }
#pragma unroll
        for (int off = WAVE / 2; off >= 1; off >>= 1) top = max_abs(top, shfl_xor(top, off));
        float to_code;
        const float scale = row_scale(top, &to_code);
        auto put = [&](int c, const f32x4_t& t) {
            *(uint32_t*)(q + c) = row_codes(t[0], t[1], t[2], t[3], to_code);
        };
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = i * 256 + lane * 4;
            if (c < K) put(c, v[i]);
        }
        for (int c = KEEP * 256 + lane * 4; c < K; c += 256) put(c, *(const f32x4_t*)(h + c));
        // a wave's LDS operations complete in program order: no barrier inside the wave
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        i32x4_t acc = {0, 0, 0, 0};
        for (int s = 0; s < steps; s += kDdAhead) {
            if (s) {
#pragma unroll
                for (int i = 0; i < kDdAhead; ++i)
                    if (s + i < steps && on)
                        wv[i] = __builtin_nontemporal_load(
                            (const i32x4_t*)(w + (w_lane + (uint32_t)(s + i) * w_step)));
            }
#pragma unroll
            for (int i = 0; i < kDdAhead; ++i)
                if (s + i < steps)
                    acc = mfma16(wv[i], *(const i32x4_t*)(q + (s + i) * 64 + (lane / 16) * 16), acc);
        }
        __builtin_amdgcn_wave_barrier();   // the next slot's codes take this one's place
        // column c of 8 into lane c: the tile's c + 8 or c lies in lane 16 * (column / 4),
        // element column % 4
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = __shfl(acc[i], ((lane % 8 + c0 % 16) / 4) * 16, WAVE);
            sum = lane % 4 == i ? t : sum;
        }
        const float wgt = shared ? 1.f : p.r.topk_w[token * k + j];
        const float ws = m.scales[(size_t)e * p.H + c0 + lane % 8];
        y += wgt * ((float)sum * scale * ws);
    }
    if (lane < 8) s_y[wave][lane] = y;
    __syncthreads();
    if (tid < 8) {
        float t = 0.f;
        for (int w = 0; w < waves; ++w) t += s_y[w][tid];
        d.y[(size_t)token * p.H + c0 + tid] = (uint16_t)pack_bf16x2(t, 0.f);
    }
}

// LDS of the down kernel: a wave's codes.  Wider layers take the grouped path.
constexpr int kDecodeI8MaxInter = 4096;

// More than one token: as long as reading again what tokens share, experts chosen by several
// (by chance: the tokens choose alike) and the shared expert, costs less than the grouped
// path's two launches more and its start.  That is some 40 MB, 8 us (us by this path and by
// the grouped one): E 256, k 8, H 2048, I 512, with a shared expert, 6 tokens (27 MB) 40.5 and
// 42.5, 8 (43 MB) 50.3 and 48.0; E 128, k 6, H 1024, I 448, 12 (30 MB) 29.7 and 30.7, 16 (50 MB)
// 35.1 and 33.8; E 16, k 2, H 1024, I 256, 8 (4 MB) 11.7 and 19.3, 32 (38 MB) 16.6 and 20.3.
constexpr int kDecodeI8MaxTokens = 64;
constexpr double kDecodeI8Again = 40e6;

bool decode_i8_fits(const GemmI8Problem& p) {
    if (p.k > kScoredMaxK || p.I > kDecodeI8MaxInter || p.I_sh > kDecodeI8MaxInter) return false;
    if (p.T == 1) return true;
    if (p.T > kDecodeI8MaxTokens) return false;
    double missed = 1.0;   // the share of experts that no token chooses
    for (int t = 0; t < p.T; ++t) missed *= 1.0 - (double)p.k / p.E;
    const double again = (double)p.T * p.k - p.E * (1.0 - missed);
    return 3.0 * p.H * (again * p.I + (p.T - 1.0) * p.I_sh) <= kDecodeI8Again;
}

hipError_t launch_decode_i8(const GemmI8Problem& p, const float* logits, const float* bias,
                            const ScoreRule* rule, void* ws, uint16_t* y, hipStream_t stream) {
    const GemmI8Ws L = gemm_i8_ws_layout(p.T, p.H, p.I, p.I_sh, p.k);
    DecodeI8Args d{};
    d.p = p;
    d.logits = logits;
    d.bias = bias;
    d.scored = rule != nullptr;
    if (rule) d.rule = *rule;
    d.h = (float*)((char*)ws + L.h);
    d.h_sh = (float*)((char*)ws + L.h_sh);
    d.y = y;
    const int grid = p.k * (p.I / 16) + p.I_sh / 16;
    const int epl = (p.E + WAVE - 1) / WAVE;
#define MOE_GU(N) \
    decode_i8_gateup_kernel<N><<<dim3(grid + (N > 0 ? 1 : 0), p.T), kDgWaves * WAVE, 0, stream>>>(d)
    if (p.T > 1) MOE_GU(0);
    else if (epl <= 1) MOE_GU(1);
    else if (epl <= 2) MOE_GU(2);
    else if (epl <= 4) MOE_GU(4);
    else if (epl <= 8) MOE_GU(8);
    else MOE_GU(16);
#undef MOE_GU
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int slots = p.k + (p.I_sh ? 1 : 0), waves = slots < kDdMaxWaves ? slots : kDdMaxWaves;
    const int ldq = p.I > p.I_sh ? p.I : p.I_sh;
    decode_i8_down_kernel<<<dim3(p.H / 8, p.T), waves * WAVE, (size_t)waves * ldq, stream>>>(d, ldq);
    return hipGetLastError();
}

}  // namespace moeq4
