// One token through the layer over 8-bit codes: two launches.
//
//   decode_i8_gateup_kernel: a workgroup owns 16 columns of one slot (a chosen
//     expert, or the shared expert); its wave 0 selects the token's experts itself
//     (the same selection as the routing call), then its waves split K, stream the
//     gate's and up's tiles, and join their integer sums through LDS:
//     h = silu(g) * u in fp32.  One more workgroup writes the routing arrays.
//   decode_i8_down_kernel: a workgroup owns 16 columns of the output; its waves
//     take a slot each, quantise the slot's h to codes (scale max|h| / 127 as in
//     the grouped path), stream the slot's 16 down rows, and y is the weighted sum
//     over the slots in slot order, the shared expert last, rounded once.
//
// Bound by bytes and by the chain of waits: the selection must end before a weight
// address is known, and down starts after all of gate/up.
#include "moe_device.h"
#include "moe_i8.h"
#include "moe_score.h"

namespace moeq4 {

constexpr int kDgWaves = 4;     // waves that split K in gate/up
constexpr int kDgAhead = 8;     // 64-K steps whose loads a wave has in flight
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

template <int EPL>
__global__ __launch_bounds__(kDgWaves* WAVE) void decode_i8_gateup_kernel(DecodeI8Args d) {
    __shared__ int s_idx[kScoredMaxK];
    __shared__ float s_w[kScoredMaxK];
    __shared__ uint32_t s_scr[3 * kScoredMaxK];
    __shared__ i32x4_t s_part[kDgWaves][2][4];
    const GemmI8Problem& p = d.p;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int k = p.k, H = p.H;
    const int tiles = p.I / 16, routed = k * tiles, all = routed + p.I_sh / 16;
    const int id = blockIdx.x;
    const bool shared = id >= routed && id < all;
    if (!shared) {
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
    const int e = shared ? 0 : __builtin_amdgcn_readfirstlane(s_idx[slot]);
    const I8MatDev& mg = shared ? p.sh_gate : p.gate;
    const I8MatDev& mu = shared ? p.sh_up : p.up;
    const int N = shared ? p.I_sh : p.I, c0 = tile * 16;
    const size_t base = (size_t)e * N * H + (size_t)c0 * H;
    const int8_t *wg = mg.codes + base, *wu = mu.codes + base;
    const uint32_t w_lane =
        mg.tiles ? lane * 16 : (uint32_t)(lane % 16) * (uint32_t)H + (lane / 16) * 16;
    const uint32_t w_step = mg.tiles ? 1024u : 64u;
    const int8_t* x = p.x + (lane / 16) * 16;
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
        const float xs = p.x_scale[0];
        const size_t col = (size_t)e * N + c0 + tid;
        const float gv = (float)g * xs * mg.scales[col], uv = (float)u * xs * mu.scales[col];
        (shared ? d.h_sh : d.h + (size_t)slot * N)[c0 + tid] = silu_f32(gv) * uv;
    }
}

__global__ __launch_bounds__(kDdMaxWaves* WAVE) void decode_i8_down_kernel(DecodeI8Args d, int ldq) {
    extern __shared__ __attribute__((aligned(16))) int8_t s_q[];   // [waves][ldq] codes of a wave's slot
    __shared__ float s_y[kDdMaxWaves][16];
    const GemmI8Problem& p = d.p;
    const int tid = threadIdx.x, lane = tid % WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int waves = blockDim.x / WAVE;
    const int k = p.k, slots = k + (p.I_sh ? 1 : 0);
    const int c0 = blockIdx.x * 16;
    int8_t* q = s_q + wave * ldq;
    float y = 0.f;   // lanes 0 .. 15: column c0 + lane
    for (int j = wave; j < slots; j += waves) {
        const bool shared = j == k;
        const int K = shared ? p.I_sh : p.I;
        const int e = shared ? 0 : __builtin_amdgcn_readfirstlane(p.r.topk_idx[j]);
        const I8MatDev& m = shared ? p.sh_down : p.down;
        const int8_t* w = m.codes + (size_t)e * p.H * K + (size_t)c0 * K;
        const uint32_t w_lane =
            m.tiles ? lane * 16 : (uint32_t)(lane % 16) * (uint32_t)K + (lane / 16) * 16;
        const uint32_t w_step = m.tiles ? 1024u : 64u;
        const float* h = shared ? d.h_sh : d.h + (size_t)j * K;
        const int steps = K / 64;
        i32x4_t wv[kDgAhead];
#pragma unroll
        for (int i = 0; i < kDgAhead; ++i)
            if (i < steps)
                wv[i] = __builtin_nontemporal_load((const i32x4_t*)(w + (w_lane + i * w_step)));
        // the slot's row: maximum, then codes into LDS while the first weights arrive
        constexpr int KEEP = 2;   // pieces of 256 values that stay in registers
        f32x4_t v[KEEP];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = i * 256 + lane * 4;
            v[i] = c < K ? *(const f32x4_t*)(h + c) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(v[i][b]));
        }
        for (int c = KEEP * 256 + lane * 4; c < K; c += 256) {
            const f32x4_t t = *(const f32x4_t*)(h + c);
#pragma unroll
            for (int b = 0; b < 4; ++b) top = fmaxf(top, fabsf(t[b]));
        }
#pragma unroll
        for (int off = WAVE / 2; off >= 1; off >>= 1) top = fmaxf(top, shfl_xor(top, off));
        const float to_code = top > 0.f ? 127.0f / top : 0.f;
        auto put = [&](int c, const f32x4_t& t) {
            *(uint32_t*)(q + c) =
                pack_codes(t[0] * to_code, t[1] * to_code, t[2] * to_code, t[3] * to_code);
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
        for (int s = 0; s < steps; s += kDgAhead) {
            if (s) {
#pragma unroll
                for (int i = 0; i < kDgAhead; ++i)
                    if (s + i < steps)
                        wv[i] = __builtin_nontemporal_load(
                            (const i32x4_t*)(w + (w_lane + (uint32_t)(s + i) * w_step)));
            }
#pragma unroll
            for (int i = 0; i < kDgAhead; ++i)
                if (s + i < steps)
                    acc = mfma16(wv[i], *(const i32x4_t*)(q + (s + i) * 64 + (lane / 16) * 16), acc);
        }
        __builtin_amdgcn_wave_barrier();   // the next slot's codes take this one's place
        // column c of 16 into lane c: it lies in lane 16 * (c / 4), element c % 4
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = __shfl(acc[i], (lane / 4) % 4 * 16, WAVE);
            sum = lane % 4 == i ? t : sum;
        }
        const float wgt = shared ? 1.f : p.r.topk_w[j];
        const float ws = m.scales[(size_t)e * p.H + c0 + lane % 16];
        y += wgt * ((float)sum * (top / 127.0f) * ws);
    }
    if (lane < 16) s_y[wave][lane] = y;
    __syncthreads();
    if (tid < 16) {
        float t = 0.f;
        for (int w = 0; w < waves; ++w) t += s_y[w][tid];
        d.y[c0 + tid] = (uint16_t)pack_bf16x2(t, 0.f);
    }
}

// LDS of the down kernel: a wave's codes.  Wider layers take the grouped path.
constexpr int kDecodeI8MaxInter = 4096;

bool decode_i8_fits(const GemmI8Problem& p) {
    return p.T == 1 && p.k <= kScoredMaxK && p.I <= kDecodeI8MaxInter && p.I_sh <= kDecodeI8MaxInter;
}

hipError_t launch_decode_i8(const GemmI8Problem& p, const float* logits, const float* bias,
                            const ScoreRule* rule, void* ws, uint16_t* y, hipStream_t stream) {
    const GemmI8Ws L = gemm_i8_ws_layout(1, p.I, p.I_sh, p.k);
    DecodeI8Args d{};
    d.p = p;
    d.logits = logits;
    d.bias = bias;
    d.scored = rule != nullptr;
    if (rule) d.rule = *rule;
    d.h = (float*)((char*)ws + L.h);
    d.h_sh = (float*)((char*)ws + L.h_sh);
    d.y = y;
    const int grid = p.k * (p.I / 16) + p.I_sh / 16 + 1;
    const int epl = (p.E + WAVE - 1) / WAVE;
#define MOE_GU(N) decode_i8_gateup_kernel<N><<<grid, kDgWaves * WAVE, 0, stream>>>(d)
    if (epl <= 1) MOE_GU(1);
    else if (epl <= 2) MOE_GU(2);
    else if (epl <= 4) MOE_GU(4);
    else if (epl <= 8) MOE_GU(8);
    else MOE_GU(16);
#undef MOE_GU
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int slots = p.k + (p.I_sh ? 1 : 0), waves = slots < kDdMaxWaves ? slots : kDdMaxWaves;
    const int ldq = p.I > p.I_sh ? p.I : p.I_sh;
    decode_i8_down_kernel<<<p.H / 16, waves * WAVE, (size_t)waves * ldq, stream>>>(d, ldq);
    return hipGetLastError();
}

}  // namespace moeq4
