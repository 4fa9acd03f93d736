// Entry points of w4a16_fused.h: host-side validation and dispatch.
#include "common.cuh"
#include "epilogue.cuh"

namespace w4a16 {
namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_fused_shape(int64_t M, int64_t N, int64_t K, int group) {
    if (M < 1 || N < 1 || K < 1) return W4A16_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return W4A16_ERR_ARG;
    if (K % kGroup != 0) return W4A16_ERR_SHAPE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

bool known_act(int act) { return act >= W4A16_ACT_NONE && act <= W4A16_ACT_GELU_TANH; }

enum Path { kCc, kSub, kMt, kGemm };

// The integer GEMVs where they exist (their conditions are those of w4a16_linear and w4a16_linear_g): up to 16 tokens
// they are ahead of the GEMM, whose tiles hold 64 tokens (5120 x 5120, 28672 x 8192, gated 5120 x 51200 and 8192 x
// 57344, us a call with 8 tokens: 10.7 / 34.6 / 39.2 / 61.1 against 15.8 / 51 / 58 / 92; with 16 tokens 14.1 / 47.0 /
// 55.0 / 90.1 against 15.9 / 51.1 / 57.9 / 92.5).
Path forward_path(int64_t M, int64_t K, int group, bool scaled) {
    const bool blocks = (K / kGroup) % 8 == 0;
    if (M == 1 && group == kGroup && blocks) return kCc;
    if (M == 1 && group < kGroup && K % 512 == 0 && !scaled) return kSub;
    if (M > 1 && M <= 16 && group == kGroup && blocks) return kMt;
    return kGemm;
}

size_t path_bytes(Path p, int64_t M, int64_t N, int64_t K, int group) {
    switch (p) {
        case kSub: return decode_sub_workspace_bytes(N, K, group);
        case kGemm: return gemm_h_workspace_bytes(M, N, K, group, false, num_sms_current());
        default: return plan_decode(M, N, K, num_sms_current()).workspace_bytes();
    }
}

int forward_entry(const uint16_t* X, const float* inv_s, int64_t M, int64_t K, int group, const uint32_t* qweight,
                  const uint16_t* scales, const int32_t* zeros, int64_t N, const FusedEpilogue& e, uint16_t* Y,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!X || !qweight || !scales || !zeros || !Y || !known_act(e.act)) return W4A16_ERR_ARG;
    int st = check_fused_shape(M, N, K, group);
    if (st != W4A16_OK) return st;
    if (e.gated && N % 2 != 0) return W4A16_ERR_SHAPE;
    if (misaligned(X) || misaligned(inv_s) || misaligned(qweight) || misaligned(scales) || misaligned(zeros) ||
        misaligned(Y) || misaligned(e.bias) || misaligned(e.residual) || misaligned(e.GU))
        return W4A16_ERR_ALIGN;
    if ((st = check_device()) != W4A16_OK) return st;
    const Path p = forward_path(M, K, group, inv_s != nullptr);
    DecodePlan plan{};
    if (p == kCc || p == kMt) plan = plan_decode(M, N, K, num_sms_current());
    const size_t need = p == kCc || p == kMt ? plan.workspace_bytes() : path_bytes(p, M, N, K, group);
    if (!workspace || workspace_bytes < need) return W4A16_ERR_WORKSPACE;
    if (misaligned(workspace)) return W4A16_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    if (p == kGemm) return launch_gemm_h(X, inv_s, M, K, group, qweight, scales, zeros, N, e, Y, workspace, s);
    if (p == kSub) return launch_decode_sub(X, M, K, group, qweight, scales, zeros, N, Y, workspace, s, &e);
    return launch_decode(X, inv_s, M, K, qweight, scales, zeros, N, Y, workspace, plan, s, nullptr, nullptr, &e);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

size_t w4a16_fused_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
    if (check_fused_shape(M, N, K, group) != W4A16_OK) return 0;
    check_device();  // caches the SM count the plans depend on
    // what any call of up to M tokens needs: every path's size grows with its tokens, but not from one path to the next
    size_t need = 0;
    for (const int64_t m : {(int64_t)1, M < 16 ? M : 16, M})
        for (const bool scaled : {false, true}) {
            const size_t b = path_bytes(forward_path(m, K, group, scaled), m, N, K, group);
            if (b > need) need = b;
        }
    return need;
}

size_t w4a16_dx_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
    if (check_fused_shape(M, N, K, group) != W4A16_OK) return 0;
    check_device();
    return gemm_h_workspace_bytes(M, N, K, group, true, num_sms_current());
}

int w4a16_linear_fused(const uint16_t* X, const float* inv_s, int64_t M, int64_t K, int group,
                       const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros, int64_t N,
                       const uint16_t* bias, int act, const uint16_t* residual, uint16_t* Y, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const FusedEpilogue e{bias, residual, nullptr, act, 0};
    return forward_entry(X, inv_s, M, K, group, qweight, scales, zeros, N, e, Y, workspace, workspace_bytes, stream);
}

int w4a16_gated(const uint16_t* X, const float* inv_s, int64_t M, int64_t K, int group, const uint32_t* qweight,
                const uint16_t* scales, const int32_t* zeros, int64_t N, int act, uint16_t* H, uint16_t* GU,
                void* workspace, size_t workspace_bytes, void* stream) {
    const FusedEpilogue e{nullptr, nullptr, GU, act, 1};
    return forward_entry(X, inv_s, M, K, group, qweight, scales, zeros, N, e, H, workspace, workspace_bytes, stream);
}

int w4a16_linear_dx(const uint16_t* dY, int64_t M, int64_t N, int group, const uint32_t* qweight,
                    const uint16_t* scales, const int32_t* zeros, int64_t K, const float* inv_s, uint16_t* dX,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (!dY || !qweight || !scales || !zeros || !dX) return W4A16_ERR_ARG;
    int st = check_fused_shape(M, N, K, group);
    if (st != W4A16_OK) return st;
    if (misaligned(dY) || misaligned(inv_s) || misaligned(qweight) || misaligned(scales) || misaligned(zeros) ||
        misaligned(dX))
        return W4A16_ERR_ALIGN;
    if ((st = check_device()) != W4A16_OK) return st;
    if (!workspace || workspace_bytes < gemm_h_workspace_bytes(M, N, K, group, true, num_sms_current()))
        return W4A16_ERR_WORKSPACE;
    if (misaligned(workspace)) return W4A16_ERR_ALIGN;
    return launch_gemm_h_dx(dY, nullptr, nullptr, 0, nullptr, M, N, group, qweight, scales, zeros, K, inv_s, dX,
                            workspace, (cudaStream_t)stream);
}

int w4a16_gated_backward(const uint16_t* dH, const uint16_t* GU, int64_t M, int64_t N, int act, int group,
                         const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros, int64_t K,
                         const float* inv_s, uint16_t* dGU, uint16_t* dX, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (!dH || !GU || !qweight || !scales || !zeros || !dGU || !dX || !known_act(act)) return W4A16_ERR_ARG;
    int st = check_fused_shape(M, N, K, group);
    if (st != W4A16_OK) return st;
    if (N % 2 != 0) return W4A16_ERR_SHAPE;
    if (misaligned(dH) || misaligned(GU) || misaligned(inv_s) || misaligned(qweight) || misaligned(scales) ||
        misaligned(zeros) || misaligned(dGU) || misaligned(dX))
        return W4A16_ERR_ALIGN;
    if ((st = check_device()) != W4A16_OK) return st;
    if (!workspace || workspace_bytes < gemm_h_workspace_bytes(M, N, K, group, true, num_sms_current()))
        return W4A16_ERR_WORKSPACE;
    if (misaligned(workspace)) return W4A16_ERR_ALIGN;
    return launch_gemm_h_dx(nullptr, dH, GU, act, dGU, M, N, group, qweight, scales, zeros, K, inv_s, dX, workspace,
                            (cudaStream_t)stream);
}

}  // extern "C"
