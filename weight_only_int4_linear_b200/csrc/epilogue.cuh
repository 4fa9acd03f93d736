// Epilogues of the fused linear layer, the gated feed-forward projection and
// their backward pass: activation functions, and what each output element
// goes through after its FP32 sum.
#pragma once
#include "common.cuh"

#include "../../include/w4a16_fused.h"

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
// 2^-125.  __expf's error grows as 2^-22 |x|, far below the 2^-9 of the BF16 store.
constexpr float kFar = -87.f;
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float silu_f(float x) { return x < kFar ? x * __expf(x) : x * sigmoid_f(x); }
// Phi(x) and e^(-x^2/2): the lower tail Phi(-|x|) = e^(-x^2/2) R(t), t = 1 / (1 + 0.35 |x|), R the polynomial of degree
// 7 with the least relative error against Phi(-|x|) e^(x^2/2) over 0 <= |x| <= 14 (3.1e-7, fitted by weighted least
// squares; 6.2e-7 with FP32 coefficients), so the tail keeps its relative accuracy where 1 + erf would cancel.  A
// fifth of erfcf's instructions, with which the epilogue of a 256 x 256 tile outlasted the tile's products at K = 4096.
__device__ __forceinline__ float normal_cdf(float x, float& e) {
    const float t = __fdividef(1.f, fmaf(0.35f, fabsf(x), 1.f));
    e = __expf(-0.5f * x * x);
    float r = 0.048942599445581436f;
    r = fmaf(r, t, -0.20211991667747498f);
    r = fmaf(r, t, 0.24064184725284576f);
    r = fmaf(r, t, -0.0170243252068758f);
    r = fmaf(r, t, 0.15596191585063934f);
    r = fmaf(r, t, 0.13335497677326202f);
    r = fmaf(r, t, 0.14027035236358643f);
    r = fmaf(r, t, -2.7316276828059927e-05f);
    const float h = e * r;
    return x < 0.f ? h : 1.f - h;
}
// GELU by the normal distribution and by a sigmoid (0.5 (1 + tanh u) = sigmoid(2 u)): neither form cancels for
// negative x.
__device__ __forceinline__ float gelu_f(float x) {
    float e;
    return x * normal_cdf(x, e);
}
__device__ __forceinline__ float gelu_tanh_f(float x) {
    const float u = 2.f * kGeluC * (x + kGeluA * x * x * x);
    return u < kFar ? x * __expf(u) : x * sigmoid_f(u);
}

// x[j] = act(x[j]); the choice is uniform over the grid.
template <int T>
__device__ __forceinline__ void act_all(float (&x)[T], int act) {
    switch (act) {
        case W4A16_ACT_RELU:
#pragma unroll
            for (int j = 0; j < T; ++j) x[j] = x[j] < 0.f ? 0.f : x[j];  // NaN stays NaN
            break;
        case W4A16_ACT_SILU:
#pragma unroll
            for (int j = 0; j < T; ++j) x[j] = silu_f(x[j]);
            break;
        case W4A16_ACT_GELU:
#pragma unroll
            for (int j = 0; j < T; ++j) x[j] = gelu_f(x[j]);
            break;
        case W4A16_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < T; ++j) x[j] = gelu_tanh_f(x[j]);
            break;
        default: break;
    }
}
__device__ __forceinline__ float act_f(float x, int act) {
    float v[1] = {x};
    act_all<1>(v, act);
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

// One output of the plain epilogue: n the weight row, off = m N + n.
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
                         int units_base, int units_rem, int max_slots, int row_tiles, cudaStream_t stream);

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
