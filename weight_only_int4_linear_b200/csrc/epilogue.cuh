// Epilogues of the fused linear layer, the gated feed-forward projection and
// their backward pass: activation functions, and what each output element
// goes through after its FP32 sum.
#pragma once
#include "common.cuh"

#include "../../include/w4a16_fused.h"

#include <cfloat>

namespace w4a16 {

// What follows the product X . W_hat^T.  gated == 0: Y = act(sum + bias) + residual, each optional.
// gated == 1: the weight holds I gate rows and then I up rows, Y[m][j] = act(sum_j) * sum_{I + j}, and GU
// (nullable) keeps both sums.  Everything in FP32, one rounding to BF16 at each store.
struct FusedEpilogue {
    const uint16_t* bias;      // [N] or null
    const uint16_t* residual;  // [M][N] or null; may be Y itself
    uint16_t* GU;              // [M][2 I] or null
    int act;
    int gated;
};

// 1 / (1 + e^-x), for x above kFar: past it e^-x nears 2^126, where __fdividef gives 0, and e^x itself is the value to
// 2^-125.  __expf's error grows as 2^-22 |x|, far below the 2^-8 of the BF16 store.
constexpr float kFar = -87.f;
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;

// Phi(x) and e^(-x^2/2): the lower tail Phi(-|x|) = e^(-x^2/2) R(t), t = 1 / (1 + 0.35 |x|), R the polynomial of degree
// 7 with the least relative error against Phi(-|x|) e^(x^2/2) over 0 <= |x| <= 14 (3.1e-7, fitted by weighted least
// squares; 6.2e-7 with FP32 coefficients), so the tail keeps its relative accuracy where 1 + erf would cancel.  A
// fifth of erfcf's instructions, with which the epilogue of a 256 x 256 tile outlasted the tile's products at K = 4096.
__device__ constexpr float kTail[8] = {-2.7316276828059927e-05f, 0.14027035236358643f, 0.13335497677326202f,
                                       0.15596191585063934f,     -0.0170243252068758f, 0.24064184725284576f,
                                       -0.20211991667747498f,    0.048942599445581436f};
__device__ __forceinline__ float normal_cdf(float x, float& e) {
    const float t = __fdividef(1.f, fmaf(0.35f, fabsf(x), 1.f));
    e = __expf(-0.5f * x * x);
    float r = kTail[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) r = fmaf(r, t, kTail[i]);
    const float h = e * r;
    return x < 0.f ? h : 1.f - h;
}
// Two FP32 values in one 64-bit register, for the packed instructions (half the issue slots of the epilogues).
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ float ex2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_f(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max(x, 0), NaN for NaN (fmaxf gives the other operand).
__device__ __forceinline__ float max0_nan(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}

// The activations of a pair, with one exponential e^-|u| each.  It is taken 2^16 times larger, so that it flushes to
// zero only where the result is below half of BF16's smallest step; adding 16 to its exponent costs 2^-20.5 of it.
//   x sigmoid(u), u of x's sign, t = e^-|u|:  (max(x, 0) + min(x, 0) t) / (1 + t)      (SILU: u = x)
//   x Phi(x), tail h = Phi(-|x|):             max(x, 0) - |x| h                        (zero from |x| = 16 on)
// None cancels for negative x.  min(x, 0) ends at FP32's lowest number, so that an overflowed sum of -infinity gives the
// limit 0 and not infinity times zero.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float finite_min0(float x) { return fmaxf(fminf(x, 0.f), -FLT_MAX); }
__device__ __forceinline__ uint64_t x_sigmoid2(float x, float y, float u, float v) {
    const uint64_t t = pack2(ex2_f(fmaf(-fabsf(u), kLog2e, 16.f)), ex2_f(fmaf(-fabsf(v), kLog2e, 16.f)));
    const uint64_t down = pack2(0x1p-16f, 0x1p-16f);
    float d, e;
    unpack2(fma2(t, down, pack2(1.f, 1.f)), d, e);
    const uint64_t n = fma2(mul2(pack2(finite_min0(x), finite_min0(y)), t), down, pack2(fmaxf(x, 0.f), fmaxf(y, 0.f)));
    return mul2(n, pack2(rcp_f(d), rcp_f(e)));
}
__device__ __forceinline__ void silu2(float& x, float& y) { unpack2(x_sigmoid2(x, y, x, y), x, y); }
__device__ __forceinline__ void gelu_tanh2(float& x, float& y) {  // 0.5 (1 + tanh u) = sigmoid(2 u)
    const uint64_t p = pack2(x, y);
    float u, v;
    unpack2(mul2(fma2(mul2(p, p), pack2(2.f * kGeluC * kGeluA, 2.f * kGeluC * kGeluA), pack2(2.f * kGeluC, 2.f * kGeluC)), p),
            u, v);
    unpack2(x_sigmoid2(x, y, u, v), x, y);
}
__device__ __forceinline__ void gelu2(float& x, float& y) {
    const float ax = fminf(fabsf(x), 16.f), ay = fminf(fabsf(y), 16.f);
    const uint64_t t = pack2(rcp_f(fmaf(0.35f, ax, 1.f)), rcp_f(fmaf(0.35f, ay, 1.f)));
    const uint64_t q = pack2(ax, ay);
    float d, e;
    unpack2(fma2(mul2(q, q), pack2(-0.5f * kLog2e, -0.5f * kLog2e), pack2(16.f, 16.f)), d, e);
    uint64_t r = pack2(kTail[7] * 0x1p-16f, kTail[7] * 0x1p-16f);
#pragma unroll
    for (int i = 6; i >= 0; --i) r = fma2(r, t, pack2(kTail[i] * 0x1p-16f, kTail[i] * 0x1p-16f));
    float g, h;
    unpack2(mul2(pack2(ex2_f(d), ex2_f(e)), r), g, h);
    x = fmaf(-ax, g, max0_nan(x));  // ax is 16 for NaN
    y = fmaf(-ay, h, max0_nan(y));
}

// x[j] = act(x[j]), T even; the choice is uniform over the grid.
template <int T>
__device__ __forceinline__ void act_all(float (&x)[T], int act) {
    switch (act) {
        case W4A16_ACT_RELU:
#pragma unroll
            for (int j = 0; j < T; ++j) x[j] = x[j] < 0.f ? 0.f : x[j];  // NaN stays NaN
            break;
        case W4A16_ACT_SILU:
#pragma unroll
            for (int j = 0; j < T; j += 2) silu2(x[j], x[j + 1]);
            break;
        case W4A16_ACT_GELU:
#pragma unroll
            for (int j = 0; j < T; j += 2) gelu2(x[j], x[j + 1]);
            break;
        case W4A16_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < T; j += 2) gelu_tanh2(x[j], x[j + 1]);
            break;
        default: break;
    }
}
__device__ __forceinline__ float act_f(float x, int act) {
    float v[2] = {x, x};
    act_all<2>(v, act);
    return v[0];
}

// f[j] = act(x[j]), d[j] = act'(x[j]).  1 - s loses bits only where it is a small part of act'.
template <int T>
__device__ __forceinline__ void act_grads(const float (&x)[T], int act, float (&f)[T], float (&d)[T]) {
    switch (act) {
        case W4A16_ACT_RELU:
#pragma unroll
            for (int j = 0; j < T; ++j) {
                f[j] = x[j] < 0.f ? 0.f : x[j];
                d[j] = x[j] > 0.f ? 1.f : 0.f;  // 0 at 0
            }
            break;
        case W4A16_ACT_SILU:
#pragma unroll
            for (int j = 0; j < T; ++j) {
                const float s = x[j] < kFar ? __expf(x[j]) : sigmoid_f(x[j]);
                f[j] = x[j] * s;
                d[j] = s + f[j] * (1.f - s);
            }
            break;
        case W4A16_ACT_GELU:
#pragma unroll
            for (int j = 0; j < T; ++j) {
                float e;
                const float p = normal_cdf(x[j], e);
                f[j] = x[j] * p;
                d[j] = p + x[j] * kRsqrt2Pi * e;
            }
            break;
        case W4A16_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < T; ++j) {
                const float x2 = x[j] * x[j], u = 2.f * kGeluC * (x[j] + kGeluA * x2 * x[j]);
                const float s = u < kFar ? __expf(u) : sigmoid_f(u);
                f[j] = x[j] * s;
                // s (1 - s) vanishes long before the cubic factor overflows: past |x| = 30 it is zero in FP32
                d[j] = fabsf(x[j]) > 30.f ? s : s + f[j] * (1.f - s) * 2.f * kGeluC * (1.f + 3.f * kGeluA * x2);
            }
            break;
        default:
#pragma unroll
            for (int j = 0; j < T; ++j) {
                f[j] = x[j];
                d[j] = 1.f;
            }
    }
}

// One output of the plain epilogue from its sum v.
__device__ __forceinline__ float linear_epilogue(float v, const FusedEpilogue& e, float bias, float residual) {
    return act_f(v + bias, e.act) + residual;
}

// BF16 load from L2, never the non-coherent path: the residual may be Y, which this kernel writes.
__device__ __forceinline__ float load_bf16(const uint16_t* p) { return bf16_bits_to_float(__ldcg(p)); }

// Host side (epilogue.cu): the split-K slots of the decode GEMVs added and finished.
// One token: slots [tile][slot][128] in two regions, as decode_cc_reduce_kernel reads them.
int launch_cc_epilogue(const float* partial, const FusedEpilogue& e, uint16_t* Y, int64_t N, int cpt, int row_tiles,
                       int tiles_a, int cpt_b, cudaStream_t stream);
// 2-16 tokens: slots [tile][max_slots][M][128], every row tile's sums in slots.
int launch_deal_epilogue(const float* partial, const FusedEpilogue& e, uint16_t* Y, int64_t N, int M, int G,
                         int units_base, int units_rem, int max_slots, cudaStream_t stream);

// The FP16-operand GEMM (gemm_h.cu), any M, K a multiple of 128, groups of 32, 64 or 128.
size_t gemm_h_workspace_bytes(int64_t M, int64_t N, int64_t K, int group, bool backward, int num_sms);
int launch_gemm_h(const uint16_t* X, const float* xscale, int64_t M, int64_t K, int group, const uint32_t* qweight,
                  const uint16_t* scales, const int32_t* zeros, int64_t N, const FusedEpilogue& e, uint16_t* Y,
                  void* workspace, cudaStream_t stream);
// dX = dY . W_hat (times inv_s per column).  With dH (then dY == null): dY = [dG | dU] formed from dH and GU and
// also written to dGU.
int launch_gemm_h_dx(const uint16_t* dY, const uint16_t* dH, const uint16_t* GU, int act, uint16_t* dGU, int64_t M,
                     int64_t N, int group, const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros,
                     int64_t K, const float* inv_s, uint16_t* dX, void* workspace, cudaStream_t stream);
}  // namespace w4a16
