// Split-K sums of the decode GEMVs with the fused epilogues.
//
// The GEMVs leave FP32 partial sums of every weight row in slots; these
// kernels add a row's slots in slot order (the same bits on every run) and
// finish the output: bias, activation and residual, or the gated product of
// row j and row I + j, which may lie in row tiles of different CTAs.  They
// are dependent launches, bound by latency: the slots of the largest layer
// (a few MB) are read from L2.
#include "decode_units.cuh"
#include "epilogue.cuh"
#include "sm100.cuh"

namespace w4a16 {
namespace {

constexpr int kEpThreads = 256;
constexpr int kEpRows = 128;   // rows per slot
template <int H>
constexpr int kCcLoads = 32 / H;  // slot loads in flight per thread (with 32 registers; the gated kernel holds more state)

struct CcSlots {
    const float* partial;
    int cpt, tiles_a, cpt_b;
};

// One token.  An item is R = 256 / (H P) outputs; H = 2 for the gated product (the output's gate row and up row
// are summed by different threads), P threads share a row's slots (part p takes slots p, p + P, ...).
// At most 32 registers, so that its CTAs fit beside the four GEMV CTAs of an SM and wait there.
template <int P, int H>
__global__ void __launch_bounds__(kEpThreads, 8) cc_epilogue_kernel(const CcSlots c, const FusedEpilogue e,
                                                                 uint16_t* Y, int outs) {
    constexpr int R = kEpThreads / (P * H);
    __shared__ float s_part[P * H][R];
    pdl_launch_dependents();
    pdl_wait_primary();  // the sums, and the residual of an earlier kernel
    const int r = threadIdx.x % R, q = threadIdx.x / R;  // q = h P + p
    const int p = q % P, h = q / P;
    for (int j0 = blockIdx.x * R; j0 < outs; j0 += gridDim.x * R) {
        const int j = j0 + r;
        float acc = 0.f;
        if (j < outs) {
            const int n = h * outs + j;
            const int tile = n / kEpRows;
            const int64_t first = tile < c.tiles_a
                                      ? (int64_t)tile * c.cpt
                                      : (int64_t)c.tiles_a * c.cpt + (int64_t)(tile - c.tiles_a) * c.cpt_b;
            const int nslots = tile < c.tiles_a ? c.cpt : c.cpt_b;
            const float* pb = c.partial + first * kEpRows + n % kEpRows;
            for (int k0 = p; k0 < nslots; k0 += kCcLoads<H> * P) {
                float v[kCcLoads<H>];
#pragma unroll
                for (int i = 0; i < kCcLoads<H>; ++i) {
                    const int k = k0 + i * P;
                    v[i] = k < nslots ? __ldcg(pb + (int64_t)k * kEpRows) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < kCcLoads<H>; ++i) acc += v[i];
            }
        }
        s_part[q][r] = acc;
        __syncthreads();
        if (q == 0 && j < outs) {
            float sum[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
                sum[i] = s_part[i * P][r];
#pragma unroll
                for (int k = 1; k < P; ++k) sum[i] += s_part[i * P + k][r];
            }
            if constexpr (H == 2) {
                if (e.GU) {
                    e.GU[j] = float_to_bf16_bits(sum[0]);
                    e.GU[outs + j] = float_to_bf16_bits(sum[1]);
                }
                Y[j] = float_to_bf16_bits(act_f(sum[0], e.act) * sum[1]);
            } else {
                const float b = e.bias ? load_bf16(e.bias + j) : 0.f, res = e.residual ? load_bf16(e.residual + j) : 0.f;
                Y[j] = float_to_bf16_bits(linear_epilogue(sum[0], e, b, res));
            }
        }
        __syncthreads();
    }
}

struct DealSlots {
    const float* partial;
    int M, G, units_base, units_rem, max_slots;
};

// Row n's sum of token m: the slots of the CTAs that held units of its row tile, in order, L loads in flight.
template <int L>
__device__ __forceinline__ float deal_sum(const DealSlots& s, int m, int n) {
    const int tile = n / kEpRows;
    const int first = cta_of_unit((int64_t)tile * s.G, s.units_base, s.units_rem);
    const int last = cta_of_unit((int64_t)tile * s.G + s.G - 1, s.units_base, s.units_rem);
    const float* pb = s.partial + (((int64_t)tile * s.max_slots) * s.M + m) * kEpRows + n % kEpRows;
    const int64_t stride = (int64_t)s.M * kEpRows;
    float acc = 0.f;
    for (int k0 = 0; k0 <= last - first; k0 += L) {
        float v[L];
#pragma unroll
        for (int k = 0; k < L; ++k) v[k] = k0 + k <= last - first ? __ldcg(pb + (k0 + k) * stride) : 0.f;
#pragma unroll
        for (int k = 0; k < L; ++k) acc += v[k];
    }
    return acc;
}

// 2-16 tokens: one output per thread and step, consecutive threads on consecutive rows.  At most 32 registers, to fit
// beside the GEMV's CTAs: with 40 (16 loads in flight) 2 tokens on 8192 x 57344 took 67.6 us instead of 58.0.  8 loads
// (4 with two sums at hand) take 2 tokens on 4096 x 4096 from 8.7 us to 7.7.
template <bool GATED>
__global__ void __launch_bounds__(kEpThreads, 8) deal_epilogue_kernel(const DealSlots s, const FusedEpilogue e,
                                                                   uint16_t* Y, int outs) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t total = (int64_t)s.M * outs;
    for (int64_t i = (int64_t)blockIdx.x * kEpThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kEpThreads) {
        const int m = (int)(i / outs), j = (int)(i - (int64_t)m * outs);
        if constexpr (GATED) {
            const float g = deal_sum<4>(s, m, j), u = deal_sum<4>(s, m, outs + j);
            if (e.GU) {
                e.GU[(int64_t)m * 2 * outs + j] = float_to_bf16_bits(g);
                e.GU[(int64_t)m * 2 * outs + outs + j] = float_to_bf16_bits(u);
            }
            Y[i] = float_to_bf16_bits(act_f(g, e.act) * u);
        } else {
            const float b = e.bias ? load_bf16(e.bias + j) : 0.f, res = e.residual ? load_bf16(e.residual + i) : 0.f;
            Y[i] = float_to_bf16_bits(linear_epilogue(deal_sum<8>(s, m, j), e, b, res));
        }
    }
}

template <class Kern, class... Args>
int launch_dependent(Kern kernel, int64_t grid, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kEpThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

}  // namespace

int launch_cc_epilogue(const float* partial, const FusedEpilogue& e, uint16_t* Y, int64_t N, int cpt, int row_tiles,
                       int tiles_a, int cpt_b, cudaStream_t stream) {
    const int sms = num_sms_current();
    if (tiles_a < 0) tiles_a = row_tiles;  // one region
    const CcSlots c{partial, cpt, tiles_a, cpt_b};
    // four parts where a row has more slots than two parts load in one round trip; at most one CTA per SM, so
    // that the next call's GEMV CTAs find their places
    const bool four = (cpt > cpt_b ? cpt : cpt_b) > (e.gated ? 2 * kCcLoads<2> : 2 * kCcLoads<1>);
    const int outs = (int)(e.gated ? N / 2 : N);
    const int R = kEpThreads / ((four ? 4 : 2) * (e.gated ? 2 : 1));
    const int64_t items = ceil_div(outs, R), grid = items < sms ? items : sms;
    if (e.gated)
        return four ? launch_dependent(cc_epilogue_kernel<4, 2>, grid, stream, c, e, Y, outs)
                    : launch_dependent(cc_epilogue_kernel<2, 2>, grid, stream, c, e, Y, outs);
    return four ? launch_dependent(cc_epilogue_kernel<4, 1>, grid, stream, c, e, Y, outs)
                : launch_dependent(cc_epilogue_kernel<2, 1>, grid, stream, c, e, Y, outs);
}

int launch_deal_epilogue(const float* partial, const FusedEpilogue& e, uint16_t* Y, int64_t N, int M, int G,
                         int units_base, int units_rem, int max_slots, cudaStream_t stream) {
    const DealSlots s{partial, M, G, units_base, units_rem, max_slots};
    const int outs = (int)(e.gated ? N / 2 : N);
    const int64_t items = ceil_div((int64_t)M * outs, kEpThreads), cap = (int64_t)num_sms_current() * 8;
    const int64_t grid = items < cap ? items : cap;
    return e.gated ? launch_dependent(deal_epilogue_kernel<true>, grid, stream, s, e, Y, outs)
                   : launch_dependent(deal_epilogue_kernel<false>, grid, stream, s, e, Y, outs);
}

}  // namespace w4a16
