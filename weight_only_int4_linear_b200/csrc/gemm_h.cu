// The tensor-core GEMM of the fused operators, in both directions of the layer:
//   forward   Y[m][n]  = epilogue( sum_k X[m][k] W[n][k] )     (contraction along K)
//   backward  dX[m][k] = sum_n dY[m][n] W[n][k]                (contraction along N)
// from the same packed codes, W = (q - z) s dequantised tile by tile on chip.
//
// Arithmetic.  Both operands are FP16, prepared so that nothing that matters
// leaves FP16's range:
//   * weights: row n is scaled by 2^-e_n, e_n chosen from the row's own scales
//     and zero points so that |W'| < 2^15.  q - z is formed exactly (1024 + q as
//     a bit pattern, one packed subtraction) and multiplied once by
//     s' = s 2^-e_n (8 significant bits, exact in FP16): one rounding of at most 2^-11
//     of the value.  Backward, 2^e_n cannot leave the sum, so it goes into dY's
//     column n.
//   * tokens: row m is scaled by 2^-a_m so that its largest value is in
//     [2^14, 2^15); BF16 values (8 significant bits) are then exact down to 2^-29
//     of the row's maximum and are off by up to 2^-39 of it below.
// Groups and rows of zeros do not enter e_n (preparation, below).  Sums run in FP32 in tensor memory over the whole contraction, without a fold
// per group, and the exponents come back in the epilogue.  Against rounding
// (q - z) s to BF16 (2^-8) this keeps the outputs' error at that of their own
// rounding.
//
// Tile: 256 output rows (weight rows, or K columns backward) x NT tokens by a
// cluster of two CTAs with the pair MMA (M = 256); each CTA dequantises its 128
// rows and holds half of the tile's tokens.
//   * Forward, 8 code words are 64 consecutive k of one row: the K-major operand
//     (K order (0,4,1,5,2,6,3,7) in every 8-block, which the token operand is
//     prepared in), in shared memory, or for NT <= 128 in tensor memory.
//   * Backward, the same words are 64 consecutive output rows of one contraction
//     step: the MN-major operand in shared memory, its rows in that order, which
//     the epilogue undoes in its addresses.
//
// Work: full waves of tiles run whole, so that the clusters sweep the same
// operands together (L2); the last, partial wave's tiles, where it pays, are cut
// along the contraction into equal ranges over the clusters (as many as get at least
// 256 of contraction each), whose FP32 partial tiles a dependent kernel adds in a fixed
// order.
//
// Gated weights (I gate rows, then I up rows) are read interleaved by a 3-D
// tensor map, row 2 j + p = row p I + j, so that a pair of neighbouring lanes
// holds both sums of an output.
//
// Warps (Cfg): groups of four dequantiser warps, which take the stages in turn (a
// stage's dequantisation is a chain of waits -- copy, loads, stores, proxy fence --
// longer than its MMAs); epilogue warps, one or two per TMEM lane quadrant; TMA
// warps for tokens and for codes and meta words (with one thread issuing every copy
// its instruction latency, about 800 cycles a stage, bounded the kernel); one MMA
// warp (rank 0).  Two accumulators: a tile's epilogue overlaps the next one's MMAs.
//
// What bounds it (1.87 GHz, MMAs of K = 16 measured at 128.5 / 65 / 45 cycles for
// 256 / 128 / 64 tokens): with 256 tokens the MMAs, 514 of the 516-560 cycles a stage
// of 64 takes -- 1.51 PFLOP/s on 8192 x 57344 backward and 1.58 forward, 1.63-1.74 on
// 8192 x 10240 backward, until the power limit lowers the clock.  With few tokens the
// dequantisers: forward 790 cycles per 128 k (2.8 TB/s of codes), backward 490 per 64.
#include "decode_units.cuh"
#include "epilogue.cuh"
#include "sm100.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace w4a16 {
namespace {

constexpr int kBM = 128;                       // output rows per CTA
constexpr int kTileRows = 2 * kBM;             // per cluster
constexpr int kBK = 64;                        // contraction per 128-byte operand line
constexpr int kTopExp = 15;                    // scaled operands stay below 2^15

enum Mode { kLinear = 0, kGated = 1, kDx = 2 };

template <int MODE, int NT>
struct Cfg {
    // Up to 128 tokens forward, the dequantised rows go to tensor memory (a thread's row is a TMEM lane), which leaves
    // shared memory to codes and tokens, in stages of 128 k: with few tokens the MMAs take a third of a stage of 64
    // (45 cycles each), and what bounds it is the fixed cost of a stage in every role.
    static constexpr bool kTs = MODE != kDx && NT <= 128;
    static constexpr int kHalves = kTs ? 2 : 1;         // operand lines (64 of contraction) per stage
    static constexpr int kStageK = kHalves * kBK;
    static constexpr int kDqGroups = kTs ? 4 : 3;       // of 4 warps
    static constexpr int kTmaPairs = kTs ? 2 : 1;       // a warp for tokens, one for codes and meta words
    static constexpr int kEpiWarps = kTs ? 4 : 8;       // one or two per TMEM lane quadrant
    static constexpr int kEpiWarp = 4 * kDqGroups, kTmaWarp = kEpiWarp + kEpiWarps, kMmaWarp = kTmaWarp + 2 * kTmaPairs;
    static constexpr int kThreads = (kMmaWarp + 1) * 32;
    static constexpr int kXHalf = NT / 2 * kBK * 2, kXBytes = kHalves * kXHalf;
    static constexpr int kCodeBytes = kBM * kStageK / 2;
    static constexpr int kMetaBytes = kHalves * 1024;   // forward 128 rows x groups in the stage, backward 64 x in 128 columns
    static constexpr int kCodeOff = kXBytes + (kTs ? 0 : kBM * kBK * 2), kMetaOff = kCodeOff + kCodeBytes;
    static constexpr int kStageBytes = kMetaOff + kMetaBytes;
    // Stages: a multiple of the dequantiser groups and of the TMA pairs.  A warp then comes back to a stage on every
    // round of the ring, and the parity it waits for cannot stand for an older round (copies complete in any order).
    static constexpr int kFit = 226 * 1024 / kStageBytes;
    static constexpr int kStages = (kTs || kFit < 9 ? kFit : 9) / kDqGroups * kDqGroups;
    static constexpr int kSlots = kTs ? (512 - 2 * NT) / (kHalves * 32) : kStages;  // dequantised tiles: TMEM, or in the stage
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024;           // + alignment slack
    static constexpr uint32_t kTmemCols = kTs ? 512 : 2 * NT;                       // two accumulators, then the slots
    static_assert(kStages % kDqGroups == 0 && kStages % kTmaPairs == 0 && kStages >= kSlots && kSlots > 1, "rings");
    static_assert(kStageBytes % 1024 == 0 && kSmem + 512 + 2 * NT * 4 <= 232448, "shared memory per CTA");
};

// Instruction descriptor, kind::f16 with FP16 A and B and an FP32 accumulator; A MN-major for the backward.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn) {
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand, 128-byte swizzle: atoms of 64 rows x 8 contraction steps (1024 B, one 128-byte line per
// step, 16-byte chunk c of step k at c ^ (k % 8)); the next 8 steps 1024 B on, the next 64 rows 8 KB on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)(8192 >> 4) << 16;  // leading byte offset: next 64 rows
    d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: next 8 steps
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Pair MMA with the rows' operand in tensor memory (each CTA's own 128 rows) and the other in shared memory.
__device__ __forceinline__ void umma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// x f 2^t: the power in two exact factors around f, so that only the result can leave the FP32 range.  Past +-252 the
// callers' results are zero or infinite either way.
__device__ __forceinline__ float scale2(float x, int t, float f = 1.f) {
    t = min(max(t, -252), 252);
    const int h = t >> 1;
    return x * __uint_as_float((uint32_t)(h + 127) << 23) * f * __uint_as_float((uint32_t)(t - h + 127) << 23);
}

// FP32 -> BF16 bits, nearest even, as one conversion instruction.
__device__ __forceinline__ uint16_t to_bf16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// Output row v of a gated weight's interleaved order -> weight row.
__device__ __forceinline__ int64_t gated_row(int64_t v, int64_t I) { return (v & 1) * I + (v >> 1); }

// ------------------------------------------------------------------ preparation
//
// Meta words, [K / group][Rp] (Rp: rows padded to 256): low half s' = s 2^-e (FP16), high half 1024 + z (FP16,
// exact for |z| <= 1024).  A zero point beyond that leaves 0x7FFF (a NaN) in the high half and e in the low
// half: the dequantiser then forms the value in binary64 from the stored scale and zero point.  Rows past the
// matrix get zero words (s' = 0).  exps[v] = e of row v.
constexpr int kPrepThreads = 256;
// Rows per block: 16, two per warp (33 tokens on 8192 x 10240 take 29.0 us, with 32 rows 31.4, with 8 rows 29.6 and 48
// tokens on 5120 x 51200 83 instead of 75: half lines are written), or 8 where 16 leave SMs without a second block
// (1097 x 28416 in groups of 32: 23 us with 16 rows).
constexpr int kMetaWords = 4096;  // held in shared memory at a time: a block's rows of 256 or 512 groups

//
// A group whose codes all equal its zero point holds only zeros, and its scale says nothing about them (the quantiser
// stores 1): it must not set the exponent.  Codes are read where that could matter: in rows whose groups' bounds lie more
// than 2^kSpread apart, and backward, where a row of zeros would scale its token's whole gradient, in rows whose first
// eight codes are zeros.  A group then left above the row's exponent is one of zeros, and its word is 0.
struct MetaArgs {
    const uint32_t* qweight;
    const uint16_t* scales;
    const int32_t* zeros;
    uint32_t* meta;
    int16_t* exps;  // [Rp] e; kZeroRow (backward) for a row of zeros
    uint8_t* pows;  // [Rp] (backward) the FP32 exponent field of 2^e: 0 for a row of zeros, 255 where 2^e is no normal number
    int R, Rp, GQ, words;  // words: of codes per group
    int64_t I;             // gated: rows per half, else 0
};
constexpr int kSpread = 4;
constexpr int kZeroRow = -32768, kLeastExp = -10000;  // kLeastExp: between kZeroRow's sums and those of any other row

__device__ __forceinline__ int bf16_exponent(uint32_t bits) {  // floor(log2 |x|), or above it for subnormals
    const int ef = (int)((bits >> 7) & 0xFF);
    return ef == 0 ? -126 : ef - 127;
}
constexpr int kNothing = -100000;  // exponent of zero

// Exponent bound of a group: its values are below 2^bound.  |q - z| <= max(|z|, |15 - z|) < 2^bits.
__device__ __forceinline__ int group_bound(uint32_t scale, int z) {
    if ((scale & 0x7FFFu) == 0) return kNothing;
    const uint32_t mag = z < 8 ? 15u - (uint32_t)z : (uint32_t)z;
    return bf16_exponent(scale) + 1 + ((uint32_t)z < 16u ? 4 : 32 - __clz(mag));
}

// The largest bound, from t down, of a row's groups that hold a value other than zero; called by a whole warp.
__device__ __noinline__ int live_bound(const uint4* codes, const uint16_t* scales, const int32_t* zeros, int groups,
                                       int quads, int t) {
    const int lane = threadIdx.x & 31;
    while (t != kNothing) {
        bool live = false;
        int next = kNothing;  // the largest bound below t
        for (int g = lane; g < groups; g += 32) {
            const int z = __ldg(zeros + g), b = group_bound(__ldg(scales + g), z);
            if (b < t) next = max(next, b);
            if (b != t || live) continue;
            live = (uint32_t)z >= 16u;
            for (int i = 0; i < quads && !live; ++i) {
                const uint4 v = __ldg(codes + (int64_t)g * quads + i);
                const uint32_t zero = 0x11111111u * (uint32_t)z;
                live = v.x != zero || v.y != zero || v.z != zero || v.w != zero;
            }
        }
        if (__any_sync(0xFFFFFFFFu, live)) return t;
        t = __reduce_max_sync(0xFFFFFFFFu, next);
    }
    return t;
}

// Rows of up to kMetaWords / ROWS groups are read once: scale and zero point wait in shared memory for the row's exponent.
template <int ROWS, bool BACK>
__device__ __forceinline__ void meta_block(const MetaArgs& a, int block) {
    constexpr int kMetaGroups = kMetaWords / ROWS;
    __shared__ uint32_t s_raw[ROWS][kMetaGroups + 1];  // scale bits, zero point << 16 (0x7FFF: beyond 1024)
    __shared__ int s_exp[ROWS];
    __shared__ uint32_t s_word[BACK ? ROWS : 1];  // backward: the rows' first codes
    constexpr int RW = ROWS / (kPrepThreads / 32), U = 4 / RW;  // rows per warp, groups of each in flight per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v0 = block * ROWS, r0 = warp * RW;
    int64_t first[RW];  // the row's first group, -1 past the matrix
    int top[RW], low[RW];  // largest and smallest exponent bound of the row's groups
    uint32_t usual[RW], least[RW];  // largest and smallest scale of the groups with a zero point in 0 .. 15
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int v = v0 + r0 + i;
        first[i] = v < a.R ? (a.I ? gated_row(v, a.I) : (int64_t)v) * a.GQ : -1;
        top[i] = kNothing;
        low[i] = -kNothing;
        usual[i] = 0u;
        least[i] = 0xFFFFFFFFu;
        if (BACK && lane == 0 && v < a.R)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&s_word[r0 + i])),
                         "l"(a.qweight + first[i] * a.words)
                         : "memory");
    }
    // groups g0 .. g1 - 1 of the warp's rows into shared memory, U groups of each in flight per lane
    auto read = [&](int g0, int g1) {
        for (int gb = g0; gb < g1; gb += 32 * U) {
            uint32_t sb[RW][U];
            int z[RW][U];
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int l = 0; l < U; ++l) {
                    const int g = gb + 32 * l + lane;
                    const bool ok = first[i] >= 0 && g < g1;
                    sb[i][l] = ok ? __ldg(a.scales + first[i] + g) : 0u;
                    z[i][l] = ok ? __ldg(a.zeros + first[i] + g) : 0;
                }
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int l = 0; l < U; ++l) {
                    const int g = gb + 32 * l + lane, zz = z[i][l];
                    if (g >= g1) continue;
                    uint32_t zw = (uint32_t)zz << 16;
                    if ((uint32_t)zz < 16u) {
                        usual[i] = max(usual[i], sb[i][l] & 0x7FFFu);
                        least[i] = min(least[i], sb[i][l] & 0x7FFFu);
                    } else {
                        const int b = group_bound(sb[i][l], zz);
                        top[i] = max(top[i], b);
                        low[i] = min(low[i], b);
                        if (zz < -1024 || zz > 1024) zw = 0x7FFF0000u;
                    }
                    s_raw[r0 + i][g - g0] = sb[i][l] | zw;
                }
        }
    };
    for (int g0 = 0; g0 < a.GQ; g0 += kMetaGroups) read(g0, min(g0 + kMetaGroups, a.GQ));
    if (BACK) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    auto set_exp = [&](int r, int t) {  // of the block's row r, its bound t
        const int e = t == kNothing ? 0 : t - kTopExp;
        const bool none = BACK && t == kNothing;
        s_exp[r] = e;
        a.exps[v0 + r] = (int16_t)(none ? kZeroRow : e);
        if (BACK) a.pows[v0 + r] = (uint8_t)(none ? 0 : e >= -126 && e <= 127 ? e + 127 : 255);
    };
    auto look_at = [&](int64_t group0, int t) {
        return live_bound(reinterpret_cast<const uint4*>(a.qweight + group0 * a.words), a.scales + group0, a.zeros + group0,
                          a.GQ, a.words / 4, t);
    };
    uint32_t look = 0u;  // backward: the rows whose codes are looked at, after the loop (fewer registers held over the call)
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        if (least[i] <= 0x7FFFu) {
            top[i] = max(top[i], group_bound(usual[i], 0));
            low[i] = min(low[i], group_bound(least[i], 0));  // kNothing for a scale of 0: the row is looked at
        }
        int t = __reduce_max_sync(0xFFFFFFFFu, top[i]);
        const bool apart = t - __reduce_min_sync(0xFFFFFFFFu, low[i]) > kSpread;
        if constexpr (BACK) {
            look |= apart ? 1u << i : 0u;
            if (lane == 0) s_exp[r0 + i] = t;
        } else {
            if (apart) t = look_at(first[i], t);
            if (lane == 0) set_exp(r0 + i, t);
        }
    }
    if constexpr (BACK) {
        __syncwarp();
        const int v = v0 + r0 + lane;  // lane r: the warp's row r
        bool zeros = false;
        if (lane < RW && v < a.R) {
            const uint32_t z0 = a.GQ <= kMetaGroups ? s_raw[r0 + lane][0] >> 16 : (uint32_t)__ldg(a.zeros + (int64_t)v * a.GQ);
            zeros = s_word[r0 + lane] == 0x11111111u * z0;
        }
        look |= __ballot_sync(0xFFFFFFFFu, zeros);
        for (; look; look &= look - 1u) {
            const int r = r0 + __ffs(look) - 1, t = look_at((int64_t)(v0 + r) * a.GQ, s_exp[r]);
            __syncwarp();
            if (lane == 0) s_exp[r] = t;
        }
        __syncwarp();
        if (lane < RW) set_exp(r0 + lane, s_exp[r0 + lane]);
    }
    for (int g0 = 0; g0 < a.GQ; g0 += kMetaGroups) {
        const int g1 = min(g0 + kMetaGroups, a.GQ);
        if (a.GQ > kMetaGroups) {
            __syncthreads();  // the preceding words are out
            read(g0, g1);
        }
        __syncthreads();
        const int rr = lane % ROWS, gs = lane / ROWS;  // row, and group within the warp's
        constexpr int GW = 32 / ROWS;
        const int e = s_exp[rr];
        // A positive scale whose 2^-e multiple is a normal FP16 number below 2^11, as that of every group within the row's
        // bound, and a zero point in 0 .. 1023: the word by integer arithmetic on the formats' fields (exponent bias
        // 127 -> 15, 7 -> 10 mantissa bits; 1024 + z is 0x6400 + z).  Else by conversions.
        const int bias = (15 - 127 - e) * 1024;
        uint32_t* out = a.meta + (int64_t)(g0 + warp * GW + gs) * a.Rp + v0 + rr;
        for (int g = warp * GW + gs; g < g1 - g0; g += kPrepThreads / ROWS, out += (int64_t)(kPrepThreads / ROWS) * a.Rp) {
            const uint32_t raw = s_raw[rr][g];
            const int h = (int)((raw & 0xFFFFu) << 3) + bias;
            uint32_t word = (uint32_t)h + (raw & 0xFFFF0000u) + 0x64000000u;
            if (h < 0x400 || h >= 0x6800 || (raw & 0x8000u) || raw >= (1024u << 16)) {
                const int z = (int)raw >> 16;
                const float s = scale2(bf16_bits_to_float((uint16_t)raw), -e);
                word = z != 0x7FFF ? (uint32_t)__half_as_ushort(__float2half_rn(s)) |
                                         ((uint32_t)__half_as_ushort(__int2half_rn(1024 + z)) << 16)
                                   : ((uint32_t)e & 0xFFFFu) | 0x7FFF0000u;
                // above the row's bound: a group of zeros (codes of 0 .. 15 alone can all be the zero point)
                if ((uint32_t)z < 16u && fabsf(s) >= 2048.f && (raw & 0x7F80u) != 0x7F80u) word = 0u;
            }
            *out = v0 + rr < a.R ? word : 0u;
        }
    }
}

// The largest exponent over the block, of per-thread values.
__device__ __forceinline__ int block_max(int v) {
    __shared__ int s_max[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if (lane == 0) s_max[warp] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? s_max[lane] : kNothing;
    return __reduce_max_sync(0xFFFFFFFFu, v);
}

// Row exponent a from the largest exponent E (|x| < 2^(E + 1)): x 2^-a < 2^15.
__device__ __forceinline__ int row_exp(int E) { return E == kNothing ? 0 : E + 1 - kTopExp; }

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

struct TokenArgs {
    const uint16_t* X;
    const float* xscale;
    __half* Xh;  // [M][K], 8-blocks in MMA order, scaled by 2^-a
    int* texp;   // [M] a
    int M, K;
};

// Forward preparation: the first M blocks take a token each, the others the weights' meta words.
template <int ROWS>
__global__ void __launch_bounds__(kPrepThreads) prep_forward_kernel(const MetaArgs ma, const TokenArgs t) {
    pdl_launch_dependents();
    pdl_wait_primary();  // X of an earlier kernel; the workspace's earlier readers
    const int m = blockIdx.x;
    if (m >= t.M) {
        meta_block<ROWS, false>(ma, m - t.M);
        return;
    }
    const uint4* x = reinterpret_cast<const uint4*>(t.X + (int64_t)m * t.K);
    uint4* out = reinterpret_cast<uint4*>(t.Xh + (int64_t)m * t.K);
    const int n8 = t.K / 8;
    auto load = [&](int i) {
        uint4 v = x[i];
        if (t.xscale) {
            const float4* r = reinterpret_cast<const float4*>(t.xscale) + 2 * i;
            const float4 r0 = __ldg(r), r1 = __ldg(r + 1);
            v = make_uint4(bf16x2_scaled(v.x, r0.x, r0.y), bf16x2_scaled(v.y, r0.z, r0.w),
                           bf16x2_scaled(v.z, r1.x, r1.y), bf16x2_scaled(v.w, r1.z, r1.w));
        }
        return v;
    };
    constexpr int U = 4;  // loads in flight per thread
    uint32_t top = 0;     // largest magnitude as BF16 bits
    for (int i0 = threadIdx.x; i0 < n8; i0 += U * kPrepThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = i0 + u * kPrepThreads < n8 ? load(i0 + u * kPrepThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        }
    }
    const int a = row_exp(block_max(top ? bf16_exponent(top) : kNothing));
    const int h = -a >> 1;
    const float f1 = pow2f(h), f2 = pow2f(-a - h);  // |a| <= 150: both factors are FP32 powers of two
    if (threadIdx.x == 0) t.texp[m] = a;
#pragma unroll 4
    for (int i = threadIdx.x; i < n8; i += kPrepThreads) {
        const uint4 v = load(i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16) * f1 * f2;
            f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * f1 * f2;
        }
        out[i] = make_uint4(half2_bits(f[0], f[4]), half2_bits(f[1], f[5]), half2_bits(f[2], f[6]),
                            half2_bits(f[3], f[7]));
    }
}

template <int ROWS>
__global__ void __launch_bounds__(kPrepThreads) prep_meta_kernel(const MetaArgs ma) {
    pdl_launch_dependents();
    pdl_wait_primary();
    meta_block<ROWS, true>(ma, blockIdx.x);
}

// Backward preparation, one block per token: the FP16 operand D'[m][n] = dY[m][n] 2^(e_n - a_m), row stride Np.
// dY is read, or (GATED) formed as [dG | dU] from dH and GU = [G | U] and also stored as BF16:
//   dG = dH U act'(G),  dU = dH act(G).
// The first pass over the row (from memory) finds an upper bound of its largest |dY 2^e| -- exact without GATED,
// |dH| max(2 |U|, |G|) with it, which needs no activation (|act'| <= 1.13, |act(G)| <= |G|) -- and the second (from
// L2) forms and stores the values.  Where a gated row turns out 2^-24 or more below its bound (every gate shut), its
// operand is stored again with its true exponent, from the BF16 gradients just stored: dGU may be GU itself (a thread
// reads its elements of GU before it writes them), which is then gone.
// The scaling is a product by 2^e and one by 2^-a in FP32 where both and the row's bound are far from the ends of
// its range, else in integer exponents.
struct GradArgs {
    const uint16_t* dY;
    const uint16_t* dH;
    const uint16_t* GU;
    uint16_t* dGU;
    const int16_t* exps;  // [>= N] e_n, kZeroRow for a row of zeros
    const uint8_t* pows;  // [>= N] exponent field of 2^e_n: 0 for a row of zeros, 255 where 2^e_n is no normal number
    __half* Dh;
    int* texp;
    int N, I, act;
    int64_t Np;
    int blocks;           // per token: a cluster of 1, 2, 4 or 8
};
// Eight elements of a row per thread and step: 8 consecutive ones, or pairs or single ones TH apart (W: what every
// row's alignment allows).
template <int W, int TH>
struct Lane8 {
    __device__ __forceinline__ static int first(int step) { return step * TH * 8 + (int)threadIdx.x * W; }
    __device__ __forceinline__ static int at(int i, int j) { return i + j / W * (W * TH) + j % W; }

    __device__ __forceinline__ static void load(const uint16_t* p, int i, int n, float (&f)[8]) {
        if constexpr (W == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else if constexpr (W == 2) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const uint32_t w = at(i, j) < n ? *reinterpret_cast<const uint32_t*>(p + at(i, j)) : 0u;
                f[j] = __uint_as_float(w << 16);
                f[j + 1] = __uint_as_float(w & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = at(i, j) < n ? bf16_bits_to_float(p[at(i, j)]) : 0.f;
        }
    }
    // powers of two from their exponent fields; 1 past the row
    __device__ __forceinline__ static void load_pows(const uint8_t* p, int i, int n, float (&f)[8]) {
        if constexpr (W == 8) {
            const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p + i));
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float((((j < 4 ? v.x : v.y) >> (8 * (j & 3))) & 0xFFu) << 23);
        } else if constexpr (W == 2) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const uint32_t w = at(i, j) < n ? __ldcg(reinterpret_cast<const uint16_t*>(p + at(i, j))) : 0x7F7Fu;
                f[j] = __uint_as_float((w & 0xFFu) << 23);
                f[j + 1] = __uint_as_float((w >> 8) << 23);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = at(i, j) < n ? __uint_as_float((uint32_t)__ldcg(p + at(i, j)) << 23) : 1.f;
        }
    }
    __device__ __forceinline__ static void load(const int16_t* p, int i, int n, int (&e)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = at(i, j) < n ? (int)__ldcg(p + at(i, j)) : 0;
    }
    __device__ __forceinline__ static void store_bf(uint16_t* p, int i, int n, const float (&f)[8]) {
        if constexpr (W == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(i, j) < n) p[at(i, j)] = to_bf16(f[j]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            store_words(p, i, n, w);
        }
    }
    __device__ __forceinline__ static void store_half(__half* p, int i, int n, const float (&f)[8]) {
        if constexpr (W == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(i, j) < n) p[at(i, j)] = __float2half_rn(f[j]);
        } else {
            const uint32_t w[4] = {half2_bits(f[0], f[1]), half2_bits(f[2], f[3]), half2_bits(f[4], f[5]),
                                   half2_bits(f[6], f[7])};
            store_words(p, i, n, w);
        }
    }
    __device__ __forceinline__ static void store_words(void* p, int i, int n, const uint32_t (&w)[4]) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
        if constexpr (W == 8) {
            *reinterpret_cast<uint4*>(q + i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                if (at(i, j) < n) *reinterpret_cast<uint32_t*>(q + at(i, j)) = w[j / 2];
        }
    }
};

// floor(log2 |x|) of an FP32 value, or above it for subnormals; zero counts as nothing
__device__ __forceinline__ int exp_of(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u == 0 ? kNothing : max((int)(u >> 23), 1) - 127;
}
// Bits a gated row may stay under its bound before it is stored again.  The bound is scaled to 2^14 .. 2^15 and FP16's
// half step is 2^-25 below 2^-14, so a row 24 bits under it is still off by at most 2^-15 of its largest value, where
// the BF16 gradients are off by 2^-8 of each.
constexpr int kFarBelow = 24;

// The largest of the token's values: over the block, and over the cluster's blocks through each other's shared memory
// (two places in turn: a block may still read the last maximum).
struct RowMax {
    int blocks, rank, turn = 0;
    __device__ __forceinline__ int operator()(int v) {
        __shared__ int s_all[2][8];
        v = block_max(v);
        if (blocks == 1) return v;
        if ((int)threadIdx.x < blocks) {
            uint32_t to;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&s_all[turn][rank])), "r"(threadIdx.x));
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
        }
        __syncwarp();
        cluster_sync();
        for (int i = 0; i < blocks; ++i) v = max(v, s_all[turn][i]);
        turn ^= 1;
        return v;
    }
};

template <int W, bool GATED, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) prep_grad_kernel(const GradArgs g) {
    using L = Lane8<W, TH>;
    pdl_launch_dependents();
    if (g.blocks > 1) cluster_sync();  // every block runs before another stores into its shared memory
    pdl_wait_primary();
    RowMax row_max{g.blocks, g.blocks == 1 ? 0 : (int)cluster_ctarank()};
    const int64_t m = blockIdx.x / g.blocks;
    const int n = GATED ? g.I : g.N;  // elements per sweep
    const int steps = (n + TH * 8 - 1) / (TH * 8);
    __half* out = g.Dh + m * g.Np;
    const uint16_t* d0 = GATED ? g.dH + m * g.I : g.dY + m * g.N;
    const uint16_t* gu = GATED ? g.GU + m * g.N : nullptr;
    uint16_t* dgu = GATED ? g.dGU + m * g.N : nullptr;

    float bound = 0.f, most_f = 1.f;  // a row of zeros (p = 0) adds nothing to the bound; most_f: the largest factor
#pragma unroll 2
    for (int s = row_max.rank; s < steps; s += g.blocks) {
        const int i = L::first(s);
        if (i >= n) break;
        float d[8], p[8];
        L::load(d0, i, n, d);
        L::load_pows(g.pows, i, n, p);
        if constexpr (GATED) {
            float gg[8], uu[8], q[8];
            L::load(gu, i, n, gg);
            L::load(gu + g.I, i, n, uu);
            L::load_pows(g.pows + g.I, i, n, q);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float b = fabsf(2.f * d[j] * uu[j]), c = fabsf(d[j] * gg[j]);
                bound = fmaxf(bound, fmaxf(b * p[j], c * q[j]));
                most_f = fmaxf(fmaxf(most_f, fmaxf(b, c)), fmaxf(p[j], q[j]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bound = fmaxf(bound, fabsf(d[j]) * p[j]);
                most_f = fmaxf(most_f, p[j]);
            }
        }
    }
    // fast: every 2^e a normal number (else p is infinite), dH U and dH G inside FP32's range (1000 stands for the bound
    // where one is not), and the bound so far inside it that neither 2^e nor the values that matter (down to 2^-40 of it)
    // can leave it
    constexpr float kInf = __builtin_huge_valf();
    const int E = row_max(most_f < kInf ? exp_of(bound) : 1000);
    const bool fast = E >= -70 && E < 100;

    // values of step s: dG, dU (or dY in v)
    auto values = [&](int i, float (&v)[8], float (&u)[8]) {
        float d[8];
        L::load(d0, i, n, d);
        if constexpr (GATED) {
            float gg[8], uu[8];
            L::load(gu, i, n, gg);
            L::load(gu + g.I, i, n, uu);
            act_grads<8>(gg, g.act, u, v);  // u = act, v = act'
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = d[j] * uu[j];
                // outside the range act' comes first, with half of U (|act'| <= 1.13), so that only dG itself overflows
                v[j] = fast || fabsf(t) < kInf ? v[j] * t : v[j] * (0.5f * uu[j]) * d[j] * 2.f;
                u[j] *= d[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = d[j];
        }
    };

    if (fast) {
        int a = row_exp(E);
        float fa = __uint_as_float((uint32_t)(127 - a) << 23);  // |a| <= 115
        float most = 0.f;  // largest scaled value
        for (int s = row_max.rank; s < steps; s += g.blocks) {
            const int i = L::first(s);
            if (i >= n) break;
            float v[8], u[8], p[8];
            values(i, v, u);
            if constexpr (GATED) L::store_bf(dgu, i, n, v);
            L::load_pows(g.pows, i, n, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = v[j] * p[j] * fa;
                most = fmaxf(most, fabsf(v[j]));
            }
            L::store_half(out, i, n, v);
            if constexpr (GATED) {
                L::store_bf(dgu + g.I, i, n, u);
                L::load_pows(g.pows + g.I, i, n, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = u[j] * p[j] * fa;
                    most = fmaxf(most, fabsf(u[j]));
                }
                L::store_half(out + g.I, i, n, u);
            }
        }
        if constexpr (!GATED) {
            if (threadIdx.x == 0 && row_max.rank == 0) g.texp[m] = a;
            return;
        }
        const int top = row_max(exp_of(most));  // 14 where the bound was tight
        if (top == kNothing || top >= kTopExp - 1 - kFarBelow) {
            if (threadIdx.x == 0 && row_max.rank == 0) g.texp[m] = a;
            return;
        }
    }
    if constexpr (GATED) {
        // rows far below their bound, and rows at the ends of the range.  GU may have been overwritten by dGU
        // (fast rows): those start from the BF16 gradients.
        int top = kNothing;
        auto each = [&](auto&& use) {
            for (int s = row_max.rank; s < steps; s += g.blocks) {
                const int i = L::first(s);
                if (i >= n) break;
                float v[8], u[8];
                if (fast) {
                    L::load(dgu, i, n, v);
                    L::load(dgu + g.I, i, n, u);
                } else {
                    values(i, v, u);
                }
                int ev[8], eu[8];
                L::load(g.exps, i, n, ev);
                L::load(g.exps + g.I, i, n, eu);
                use(i, v, u, ev, eu);
            }
        };
        each([&](int i, float (&v)[8], float (&u)[8], int (&ev)[8], int (&eu)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, max(exp_of(v[j]) + ev[j], exp_of(u[j]) + eu[j]));
        });
        top = row_max(top < kLeastExp ? kNothing : top);
        const int a = row_exp(top);
        if (threadIdx.x == 0 && row_max.rank == 0) g.texp[m] = a;
        each([&](int i, float (&v)[8], float (&u)[8], int (&ev)[8], int (&eu)[8]) {
            if (!fast) {
                L::store_bf(dgu, i, n, v);
                L::store_bf(dgu + g.I, i, n, u);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = ev[j] == kZeroRow ? 0.f : scale2(v[j], ev[j] - a);  // a gradient past the range too adds nothing
                u[j] = eu[j] == kZeroRow ? 0.f : scale2(u[j], eu[j] - a);
            }
            L::store_half(out, i, n, v);
            L::store_half(out + g.I, i, n, u);
        });
    } else {
        int top = kNothing;
        for (int s = row_max.rank; s < steps; s += g.blocks) {
            const int i = L::first(s);
            if (i >= n) break;
            float d[8];
            int e[8];
            L::load(d0, i, n, d);
            L::load(g.exps, i, n, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, exp_of(d[j]) + e[j]);
        }
        top = row_max(top < kLeastExp ? kNothing : top);
        const int a = row_exp(top);
        if (threadIdx.x == 0 && row_max.rank == 0) g.texp[m] = a;
        for (int s = row_max.rank; s < steps; s += g.blocks) {
            const int i = L::first(s);
            if (i >= n) break;
            float d[8];
            int e[8];
            L::load(d0, i, n, d);
            L::load(g.exps, i, n, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = scale2(d[j], e[j] - a);
            L::store_half(out, i, n, d);
        }
    }
}

// ------------------------------------------------------------------ the GEMM

struct HArgs {
    const uint32_t* meta;
    const int16_t* exps;  // forward: e of every output row
    const int* texp;      // a of every token
    const uint16_t* scales;
    const int32_t* zeros;
    const float* inv_s;   // backward: per output column, or null
    uint16_t* Y;          // Y, H or dX
    float* partial;       // [2 units][NT][256]
    int* fault;
    FusedEpilogue ep;
    int64_t I;            // gated: rows per half
    int M, R, C;          // tokens, output rows, contraction
    int GQ, group;        // groups per weight row, group size
    int NS;               // stages per tile
    int m_tiles, r_tiles;
    int whole_tiles;      // tiles 0 .. whole_tiles - 1 run whole: cluster b takes b, b + units, ...
    int units;            // clusters
    int base, rem, split_units;  // the other tiles' stages, dealt in equal ranges to the first split_units clusters
};

constexpr int kRaster = 4;
__device__ __forceinline__ void tile_coords(int t, const HArgs& a, int& rt, int& mt) {
    const int per_group = kRaster * a.r_tiles;
    const int grp = t / per_group, r = t - grp * per_group;
    const int gm = min(kRaster, a.m_tiles - grp * kRaster);
    rt = r / gm;
    mt = grp * kRaster + (r - rt * gm);
}

// Cluster b's segments: its whole tiles, then its range of the cut tiles' stages.
struct Segments {
    int tile, s0, s1;  // the current segment: stages s0 .. s1 - 1 of tile
    int next_whole;
    int64_t u, u_end;
    __device__ __forceinline__ Segments(int b, const HArgs& a) : tile(0), s0(0), s1(0), next_whole(b) {
        u = u_end = 0;
        if (b < a.split_units) {
            u = (int64_t)b * a.base + min(b, a.rem);
            u_end = u + a.base + (b < a.rem ? 1 : 0);
        }
    }
    __device__ __forceinline__ bool next(const HArgs& a) {
        if (next_whole < a.whole_tiles) {
            tile = next_whole;
            s0 = 0;
            s1 = a.NS;
            next_whole += a.units;
            return true;
        }
        if (u >= u_end) return false;
        const int r = (int)(u / a.NS);
        tile = a.whole_tiles + r;
        s0 = (int)(u - (int64_t)r * a.NS);
        s1 = (int)min((int64_t)a.NS, (int64_t)s0 + (u_end - u));
        u += s1 - s0;
        return true;
    }
};
// Position in the ring of S stages: stage s, whose barriers complete the phase of this parity on this round.
template <int S>
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == S) {
            s = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void prev() {
        if (s-- == 0) {
            s = S - 1;
            parity ^= 1u;
        }
    }
};
// Slot of cluster b's part of a cut tile that starts at stage s0: a cluster's range has at most one part that
// starts inside a tile (its first) and one that starts a tile and does not end it (its last).
__device__ __forceinline__ int slot_of(int b, int s0) { return 2 * b + (s0 == 0 ? 1 : 0); }

// The residual of T tokens of output row v from token m0 < M on, loaded ahead of the sums: without a branch per token
// (past the last one it is read again), since eight of them cost more than the rest of a batch's epilogue.
template <int MODE, int T>
__device__ __forceinline__ void load_residual(const HArgs& a, int m0, int v, uint16_t (&res)[MODE == kLinear ? T : 1]) {
    if constexpr (MODE == kLinear) {
        if (a.ep.residual == nullptr) return;
        const uint16_t* r = a.ep.residual + (int64_t)m0 * a.R + min(v, a.R - 1);
        const int last = a.M - 1 - m0;
#pragma unroll
        for (int j = 0; j < T; ++j) res[j] = __ldcg(r + (int64_t)min(j, last) * a.R);
    }
}
// A token's exponent a as the bits of 2^a where |a| <= kNear, else as a itself.
constexpr int kNear = 60, kNearBits = (127 - kNear) << 23;
__device__ __forceinline__ int scale_bits(int a) { return a >= -kNear && a <= kNear ? (a + 127) << 23 : a; }
__device__ __forceinline__ int scale_exp(int bits) { return bits >= kNearBits ? (bits >> 23) - 127 : bits; }
// T tokens' scales, 16-byte aligned.
template <int T>
__device__ __forceinline__ void load_scales(const int* te, int (&e)[T]) {
#pragma unroll
    for (int j = 0; j < T; j += 4) {
        const int4 t = *reinterpret_cast<const int4*>(te + j);
        e[j] = t.x;
        e[j + 1] = t.y;
        e[j + 2] = t.z;
        e[j + 3] = t.w;
    }
}

// What an output row brings to all of its tokens.
struct RowValues {
    float bias, col_s;
    int e;
    template <int MODE>
    __device__ __forceinline__ void load(const HArgs& a, int v) {
        bias = 0.f;
        col_s = 1.f;
        e = 0;
        if (v < a.R) {
            if (MODE != kDx) e = __ldcg(a.exps + v);
            if (MODE == kLinear && a.ep.bias) bias = load_bf16(a.ep.bias + v);
            if (MODE == kDx && a.inv_s) col_s = __ldg(a.inv_s + v);
        }
    }
};

// Finishes T tokens of one output row: y[j] (the raw sum) belongs to token m0 + j, of scale bits te[j], and output row v.
// All lanes of a warp call it together, with consecutive v from an even one (gated rows are exchanged between
// neighbours).  near: every token's and every row's exponent is within kNear of zero, so that no partial product of the
// scaling leaves FP32's normal range (sums are multiples of 2^-48 below 2^62).
template <int MODE, int T>
__device__ __forceinline__ void finish(const HArgs& a, float (&y)[T], const int (&te)[T],
                                       const uint16_t (&res)[MODE == kLinear ? T : 1], int m0, int v,
                                       const RowValues& r, bool near) {
    const bool row_ok = v < a.R;
    if (near) {  // scale, then row factor and bias, two tokens an instruction
        const float f = MODE == kDx ? r.col_s : __int_as_float(scale_bits(r.e));
        const uint64_t f2 = pack2(f, f), b2 = pack2(r.bias, r.bias);
#pragma unroll
        for (int j = 0; j < T; j += 2) {
            const uint64_t s = mul2(pack2(y[j], y[j + 1]), pack2(__int_as_float(te[j]), __int_as_float(te[j + 1])));
            unpack2(MODE == kLinear ? fma2(s, f2, b2) : mul2(s, f2), y[j], y[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j) {
            y[j] = scale2(y[j], r.e + scale_exp(te[j]), MODE == kDx ? r.col_s : 1.f);
            if (MODE == kLinear) y[j] += r.bias;
        }
    }
    // out[j stride] = f[j] for the tokens m + j that exist
    auto store = [&](uint16_t* out, int stride, int m, const auto& f) {
        constexpr int n = sizeof(f) / sizeof(float);
        if (!row_ok) return;
        uint32_t w[n / 2];
#pragma unroll
        for (int j = 0; j < n; j += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[j], f[j + 1]);
            w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int j = 0; j < n; ++j, out += stride)
            if (m + j < a.M) *out = (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
    };
    if constexpr (MODE != kGated) {
        if constexpr (MODE == kLinear) {
            act_all<T>(y, a.ep.act);
            if (a.ep.residual) {
#pragma unroll
                for (int j = 0; j < T; ++j) y[j] += bf16_bits_to_float(res[j]);
            }
        }
        store(a.Y + (int64_t)m0 * a.R + v, a.R, m0, y);
    } else {
        const int p = v & 1;
        const int64_t col = v >> 1;
        if (a.ep.GU) store(a.ep.GU + (int64_t)m0 * a.R + p * (int64_t)a.I + col, a.R, m0, y);
        // the even lane finishes the first half of the tokens, the odd lane the second
        float gate[T / 2], up[T / 2];
#pragma unroll
        for (int j = 0; j < T / 2; ++j) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, p ? y[j] : y[T / 2 + j], 1);
            gate[j] = p ? got : y[j];
            up[j] = p ? y[T / 2 + j] : got;
        }
        act_all<T / 2>(gate, a.ep.act);
#pragma unroll
        for (int j = 0; j < T / 2; ++j) gate[j] *= up[j];
        const int m = m0 + (p ? T / 2 : 0);
        store(a.Y + (int64_t)m * a.I + col, a.I, m, gate);
    }
}

// The 8 values of a code word whose zero point is beyond 1024, in binary64.
__device__ __noinline__ uint4 far_word(uint32_t w, float s, int z, int e) {
    const double f = __longlong_as_double((long long)(1023 - e) << 52) * s;  // s 2^-e, |e| < 400
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __half_as_ushort(__double2half((double)((long long)((w >> (4 * i)) & 15u) - z) * f));
        const uint32_t hi = __half_as_ushort(__double2half((double)((long long)((w >> (4 * i + 16)) & 15u) - z) * f));
        o[i] = lo | (hi << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int MODE, int NT>
__global__ void __launch_bounds__(Cfg<MODE, NT>::kThreads, 1) gemm_h_kernel(const __grid_constant__ CUtensorMap tx,
                                                             const __grid_constant__ CUtensorMap tq,
                                                             const __grid_constant__ CUtensorMap tm, const HArgs a) {
    using C = Cfg<MODE, NT>;
    constexpr int S = C::kStages, NS = C::kSlots;
    constexpr bool kBack = MODE == kDx;
    constexpr uint32_t kIdesc = idesc_f16(kTileRows, NT, kBack);
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[S], empty[S], afull[NS], mdone[2], dfree[2];
    __shared__ __align__(8) uint64_t drained;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) int s_te[2][NT];  // the tokens' exponents of the tile in each accumulator
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // same offset in both CTAs

    pdl_launch_dependents();
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    const int rank = (int)cluster_ctarank();
    const int b = blockIdx.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 2);  // two TMA warps
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < NS; ++s) mbar_init(&afull[s], 4 * 2);  // one dequantiser group in each CTA
        for (int i = 0; i < 2; ++i) {
            mbar_init(&mdone[i], 1);
            mbar_init(&dfree[i], C::kEpiWarps * 2);
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 0) tmem_alloc_pair(&s_tmem, C::kTmemCols);
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    Segments seg(b, a);

    // The issuing warps run their loops with all lanes, so that positions and descriptors stay in uniform
    // registers, and one elected lane issues: one thread's instruction latency per stage is what bounds them.
    if (warp >= C::kTmaWarp && warp < C::kMmaWarp) {  // -------------------------------------- TMA
        const bool leader = elect_one();
        const bool toks = ((warp - C::kTmaWarp) & 1) == 0;
        const int pair = (warp - C::kTmaWarp) >> 1;  // takes the ring's stages pair, pair + kTmaPairs, ...
        if (leader) {
            prefetch_tmap(toks ? &tx : &tq);
            if (!toks) prefetch_tmap(&tm);
        }
        Ring<S> r;
        int passed = 0;
        bool ok = true;
        const int lg = a.group >> 6;  // log2(group / 32): 0, 1, 2
        const int lines = kBack ? kBM / a.group : max((C::kStageK / 32) >> lg, 1);  // groups in the stage
        const uint32_t bytes = toks ? C::kXBytes : C::kCodeBytes + lines * (kBack ? kBK : kBM) * 4;
        pdl_wait_primary();  // operands and meta words come from the preparation kernels
        while (ok && seg.next(a)) {
            int rt, mt;
            tile_coords(seg.tile, a, rt, mt);
            const int row0 = rt * kTileRows + rank * kBM;  // this CTA's first output row
            const int tok0 = mt * NT + rank * (NT / 2);
            // backward: the first group of the CTA's columns (columns past K take any: they are never stored)
            const int gb = min(row0 >> (5 + lg), a.GQ - lines);
            for (int ks = seg.s0; ks < seg.s1; ++ks, r.next()) {
                ++passed;
                if (C::kTmaPairs > 1 && r.s % C::kTmaPairs != pair) continue;
                if (!mbar_wait(&empty[r.s], r.parity ^ 1u, a.fault, 171)) {
                    ok = false;
                    --passed;
                    break;
                }
                uint64_t* bar = &full[r.s];
                unsigned char* st = ring + r.s * C::kStageBytes;
                if (leader) {
                    mbar_arrive_expect_tx(bar, bytes);
                    if (toks) {
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_2d(st + h * C::kXHalf, &tx, ks * C::kStageK + h * kBK, tok0, bar);
                    } else {
                        unsigned char* codes = st + C::kCodeOff;
                        // codes, and one line of meta words per group: forward 128 rows, backward 64
                        if constexpr (kBack) {
                            tma_load_2d(codes, &tq, row0 / 8, ks * kBK, bar);
                            tma_load_2d(codes + C::kCodeBytes, &tm, ks * kBK, gb, bar);
                        } else {
                            if constexpr (MODE == kGated)
                                tma_load_3d(codes, &tq, ks * (C::kStageK / 8), 0, row0 / 2, bar);
                            else
                                tma_load_2d(codes, &tq, ks * (C::kStageK / 8), row0, bar);
                            tma_load_2d(codes + C::kCodeBytes, &tm, row0, ks * (C::kStageK / 32) >> lg, bar);
                        }
                    }
                }
            }
        }
        // this warp's copies in flight land before the CTA may exit: its stages among the last S
        for (int i = 0; i < min(passed, S); ++i) {
            r.prev();
            if (C::kTmaPairs == 1 || r.s % C::kTmaPairs == pair) mbar_wait(&full[r.s], r.parity, a.fault, 172);
        }
    } else if (warp == C::kMmaWarp) {  // ------------------------------------------------ MMA issue
        if (rank == 0) {
            const bool leader = elect_one();
            Ring<S> r;
            Ring<NS> q;  // the dequantised tiles
            int sc = 0;
            bool ok = true;
            const uint32_t x0 = smem_u32(ring), a0 = x0 + C::kXBytes;
            const uint64_t xdesc = sw128_kmajor_desc(x0), adesc = kBack ? sw128_mnmajor_desc(a0) : sw128_kmajor_desc(a0);
            constexpr uint64_t kAStep = (kBack ? 2048 : 32) >> 4, kXStep = 32 >> 4;  // descriptor units of 16 bytes
            while (ok && seg.next(a)) {
                const int buf = sc & 1;
                if (sc >= 2 && !mbar_wait(&dfree[buf], ((sc >> 1) - 1) & 1, a.fault, 173)) break;
                for (int ks = seg.s0; ks < seg.s1; ++ks, r.next(), q.next()) {
                    // the dequantisers of both CTAs waited on their copies first
                    if (!mbar_wait(&afull[q.s], q.parity, a.fault, 174)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)(r.s * (C::kStageBytes >> 4));
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < C::kStageK / 16; ++kk) {
                            if constexpr (C::kTs)  // 8 columns of the tile's slot
                                umma_ts_pair(tmem + buf * NT, tmem + 2 * NT + q.s * (C::kHalves * 32) + kk * 8,
                                             xdesc + off + (kk >> 2) * (C::kXHalf >> 4) + (kk & 3) * kXStep, kIdesc,
                                             ks > seg.s0 || kk > 0);
                            else
                                umma_ss_pair(tmem + buf * NT, adesc + off + kk * kAStep, xdesc + off + kk * kXStep, kIdesc,
                                             ks > seg.s0 || kk > 0);
                        }
                        umma_commit_pair(&empty[r.s], 0x3);
                    }
                }
                if (ok && leader) umma_commit_pair(&mdone[buf], 0x3);
                ++sc;
            }
            if (leader) umma_commit_pair(&drained, 0x1);  // every MMA issued completes before the teardown
            mbar_wait(&drained, 0, a.fault, 175);
        }
    } else if (warp < C::kEpiWarp) {  // ------------------------------------------------- dequantisers
        // Group dg takes the ring's stages dg, dg + kDqGroups, ..., a thread kHalves x 8 code words of each: forward, the
        // k of output row `row`; backward, 64 columns (half h of the CTA's) of contraction step `row`.
        const int dg = warp >> 2, tid = threadIdx.x & 127;
        const int row = kBack ? tid & 63 : tid, h = kBack ? tid >> 6 : 0;
        // The row's 16-byte code chunks: forward 2 or 4 in 32 or 64 bytes with the swizzle of that width, backward 4 in 64
        // bytes, this thread's 2 h and 2 h + 1.
        const int code_row = row * (kBack ? 64 : C::kStageK / 2);
        const int code_x = kBack || C::kTs ? (row >> 1) & 3 : (row >> 2) & 1;
        constexpr int kLine = kBack ? kBK : kBM;
        const int lg = a.group >> 6;             // log2(group / 32)
        const int a_off = h * 8192 + row * 128;  // operand row of 128 bytes, chunk j at j ^ (row % 8)
        Ring<S> r, freed;  // freed: the stage whose MMAs read this tile's slot last
        Ring<NS> slot;
        int turn = dg, before = NS;
        bool ok = true;
        while (ok && seg.next(a)) {
            int rt, mt;
            tile_coords(seg.tile, a, rt, mt);
            for (int ks = seg.s0; ks < seg.s1; ++ks, r.next(), slot.next()) {
                const bool first = before > 0;  // the slots' first round
                if (first) --before;
                if (turn-- == 0) {
                    turn = C::kDqGroups - 1;
                    if (!mbar_wait(&full[r.s], r.parity, a.fault, 176) ||
                        (C::kTs && !first && !mbar_wait(&empty[freed.s], freed.parity, a.fault, 178))) {
                        ok = false;
                        break;
                    }
                    unsigned char* st = ring + r.s * C::kStageBytes;
                    const unsigned char* codes = st + C::kCodeOff;
#pragma unroll
                    for (int half = 0; half < C::kHalves; ++half) {
                        uint32_t w[8], mw[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {  // 4 words, 32 values
                            const int chunk = 2 * (kBack ? h : half) + c;
                            const uint4 v = *reinterpret_cast<const uint4*>(codes + code_row + 16 * (chunk ^ code_x));
                            w[4 * c] = v.x;
                            w[4 * c + 1] = v.y;
                            w[4 * c + 2] = v.z;
                            w[4 * c + 3] = v.w;
                            mw[c] = *reinterpret_cast<const uint32_t*>(st + C::kMetaOff + ((chunk >> lg) * kLine + row) * 4);
                        }
                        uint32_t o[32];  // the words' values, four pairs each
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t m = mw[j >> 2], sp = __byte_perm(m, m, 0x1010), zp = __byte_perm(m, m, 0x3232);
                            const __half2 s2 = *reinterpret_cast<const __half2*>(&sp),
                                          z2 = *reinterpret_cast<const __half2*>(&zp);
                            const __half2 z64 = __hsub2(__float2half2_rn(960.f), z2);  // -(64 + z)
                            // q - z of codes e and e + 4, exact: 1024 + q less 1024 + z, or (1024 + 16 q) / 16 less 64 + z
                            const uint32_t w8 = w[j] >> 8;
                            uint32_t p[4];
                            asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(p[0]) : "r"(w[j]));
                            asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(p[1]) : "r"(w[j]));
                            asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(p[2]) : "r"(w8));
                            asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(p[3]) : "r"(w8));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 h2 = *reinterpret_cast<const __half2*>(&p[e]);
                                const __half2 d = e & 1 ? __hfma2(h2, __float2half2_rn(0.0625f), z64) : __hsub2(h2, z2);
                                const __half2 v = __hmul2(d, s2);
                                o[4 * j + e] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                        }
                        if ((mw[0] >> 16) == 0x7FFFu || (mw[1] >> 16) == 0x7FFFu) {  // rare: zero points beyond 1024
                            const int64_t vrow =
                                kBack ? (int64_t)ks * kBK + row : (int64_t)rt * kTileRows + rank * kBM + row;
                            const int64_t n = MODE == kGated ? gated_row(vrow, a.I) : vrow;
                            const int col = kBack ? rt * kTileRows + rank * kBM + h * 64 : ks * C::kStageK + half * 64;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t m = mw[j >> 2];
                                if ((m >> 16) != 0x7FFFu) continue;
                                const int64_t g = n * a.GQ + min((col + 32 * (j >> 2)) / a.group, a.GQ - 1);
                                const uint4 f = far_word(w[j], bf16_bits_to_float(__ldg(a.scales + g)), __ldg(a.zeros + g),
                                                         (int)(int16_t)(m & 0xFFFFu));
                                o[4 * j] = f.x;
                                o[4 * j + 1] = f.y;
                                o[4 * j + 2] = f.z;
                                o[4 * j + 3] = f.w;
                            }
                        }
                        if constexpr (C::kTs) {
                            __syncwarp();
                            tmem_st32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + 2 * NT + slot.s * (C::kHalves * 32) + half * 32,
                                      o);
                        } else {
                            unsigned char* arow = st + C::kXBytes + a_off;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<uint4*>(arow + 16 * (j ^ (row & 7))) =
                                    make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        }
                    }
                    if constexpr (C::kTs) {
                        tmem_wait_st();
                        tc_fence_before();
                    } else {
                        fence_proxy_async_shared();  // generic-proxy writes -> visible to the tensor core
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(&afull[slot.s], 0);
                }
                if (!first) freed.next();
            }
        }
    } else {  // ------------------------------------------------------------------------- epilogue
        pdl_wait_primary();  // exponents come from the preparation kernels, the residual from earlier ones
        const int quad = warp & 3, half = (warp - C::kEpiWarp) >> 2;
        const int lrow = quad * 32 + lane;  // TMEM lane
        // backward: position (0,1,..,7) of every 8-block holds column (0,4,1,5,2,6,3,7)
        const int orow = kBack ? (lrow & ~7) | ((lrow & 7) >> 1) | ((lrow & 1) << 2) : lrow;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        int sc = 0;
        bool ok = true;
        while (seg.next(a)) {
            int rt, mt;
            tile_coords(seg.tile, a, rt, mt);
            const int buf = sc & 1;
            const bool whole = seg.s0 == 0 && seg.s1 == a.NS;
            const int trow = rank * kBM + orow, v = rt * kTileRows + trow;
            constexpr int T = 8, kCols = NT / (C::kEpiWarps / 4);  // this warp's columns: kCols from half * kCols
            const int c0 = half * kCols, m0 = mt * NT + c0;
            // While the tile is multiplied: the row's values, the first residuals, and the tokens' exponents in shared
            // memory with whether they keep every sum's scale inside FP32's range.  (Loaded with each batch instead, their
            // latency made the epilogue as long as a tile of K = 4096: 1000 tokens with GELU 139 us instead of 133, 2048 gated
            // ones on 8192 x 57344 1448 instead of 1382.)
            RowValues rv;
            rv.load<MODE>(a, v);
            uint16_t res[MODE == kLinear ? T : 1] = {};
            bool near = false;
            if (whole) {
                if (m0 < a.M) load_residual<MODE, T>(a, m0, v, res);
                for (int i = threadIdx.x - C::kEpiWarp * 32; i < NT; i += C::kEpiWarps * 32)
                    s_te[buf][i] = scale_bits(mt * NT + i < a.M ? __ldcg(a.texp + mt * NT + i) : 0);
            }
            named_barrier_sync(1, C::kEpiWarps * 32);  // also: every warp is done with the exponents of two segments ago
            if (whole) {
                near = rv.e >= -kNear && rv.e <= kNear;
                for (int i = lane; i < NT; i += 32)
                    near = near && s_te[buf][i] >= kNearBits;
                near = __all_sync(0xFFFFFFFFu, near);
            }
            if (ok && !mbar_wait(&mdone[buf], (sc >> 1) & 1, a.fault, 177)) ok = false;
            ok = __all_sync(0xFFFFFFFFu, ok);
            ++sc;
            if (!ok) continue;
            tc_fence_after();
            float* part = a.partial + ((int64_t)slot_of(b, seg.s0) * NT + c0) * kTileRows + trow;
            uint32_t d[T];
            tmem_ld8(tl + buf * NT + c0, d);
#pragma unroll 1
            for (int cc = 0; cc < kCols; cc += T, part += T * kTileRows) {
                tmem_wait_ld();
                float y[T];
                uint16_t rc[MODE == kLinear ? T : 1];
#pragma unroll
                for (int j = 0; j < T; ++j) y[j] = __uint_as_float(d[j]);
#pragma unroll
                for (int j = 0; j < (MODE == kLinear ? T : 1); ++j) rc[j] = res[j];
                if (cc + T < kCols) {  // the next batch's loads
                    tmem_ld8(tl + buf * NT + c0 + cc + T, d);
                    if (whole && m0 + cc + T < a.M) load_residual<MODE, T>(a, m0 + cc + T, v, res);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(&dfree[buf], 0);
                }
                if (whole) {
                    if (m0 + cc < a.M) {
                        int te[T];
                        load_scales<T>(&s_te[buf][c0 + cc], te);
                        finish<MODE, T>(a, y, te, rc, m0 + cc, v, rv, near);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < T; ++j) part[j * kTileRows] = y[j];
                }
            }
        }
    }
    // teardown: every role done, every MMA complete (drained), no arrival still bound for the peer
    __syncwarp();
    cluster_sync();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

// The cut tiles: adds each tile's parts in cluster order and finishes the outputs.  One block per tile and 4 tokens, a
// thread per row of the tile; the loads of 4 parts are in flight together (this kernel is all latency).
constexpr int kJoinTokens = 4, kJoinParts = 4;
template <int MODE, int NT>
__global__ void __launch_bounds__(kTileRows) gemm_h_join_kernel(const HArgs a) {
    constexpr int T = kJoinTokens;
    pdl_launch_dependents();
    const int r = blockIdx.x / (NT / T), c0 = (blockIdx.x - r * (NT / T)) * T;
    int rt, mt;
    tile_coords(a.whole_tiles + r, a, rt, mt);
    const int64_t u0 = (int64_t)r * a.NS;  // the tile's first stage
    const int first = cta_of_unit(u0, a.base, a.rem), last = cta_of_unit(u0 + a.NS - 1, a.base, a.rem);
    const int m0 = mt * NT + c0, v = rt * kTileRows + threadIdx.x;
    pdl_wait_primary();
    if (m0 >= a.M || first == last) return;  // padding, or one cluster ran the tile whole
    auto part = [&](int b) {
        const int64_t u = (int64_t)b * a.base + min(b, a.rem);  // the cluster's first stage
        return a.partial + ((int64_t)slot_of(b, u > u0 ? 1 : 0) * NT + c0) * kTileRows + threadIdx.x;
    };
    float f[kJoinParts][T];
    auto load = [&](int b0) {
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i) {
            const float* p = part(min(b0 + i, last));
#pragma unroll
            for (int j = 0; j < T; ++j) f[i][j] = b0 + i <= last ? __ldcg(p + j * kTileRows) : 0.f;
        }
    };
    load(first);
    uint16_t res[MODE == kLinear ? T : 1] = {};
    load_residual<MODE, T>(a, m0, v, res);
    const int4 t4 = __ldcg(reinterpret_cast<const int4*>(a.texp + m0));
    const int te[T] = {scale_bits(t4.x), scale_bits(t4.y), scale_bits(t4.z), scale_bits(t4.w)};
    RowValues rv;
    rv.load<MODE>(a, v);
    float sum[T];
#pragma unroll
    for (int j = 0; j < T; ++j) sum[j] = 0.f;
    for (int b = first; b <= last; b += kJoinParts) {
        if (b > first) load(b);
#pragma unroll
        for (int i = 0; i < kJoinParts; ++i)
#pragma unroll
            for (int j = 0; j < T; ++j) sum[j] += f[i][j];
    }
    finish<MODE, T>(a, sum, te, res, m0, v, rv, false);
}

// ------------------------------------------------------------------ host

// Rows padded to 256 that 16 to a block leave SMs without a second block.
bool few_rows(int64_t Rp) { return Rp / 16 < 2 * (int64_t)num_sms_current(); }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens per tile.
int tile_tokens(int64_t M) { return M <= 64 ? 64 : M <= 128 ? 128 : 256; }

struct Layout {
    int64_t Rp, Cp, Mp;
    size_t meta, exps, pows, texp, op, partial, total;  // byte offsets
};

Layout layout_h(int64_t M, int64_t N, int64_t K, int group, bool back, int num_sms) {
    Layout l{};
    const int NT = tile_tokens(M);
    l.Rp = (N + 255) / 256 * 256;
    l.Cp = back ? (N + 63) / 64 * 64 : K;
    l.Mp = (M + 255) / 256 * 256;
    size_t o = kCounterBytes;
    l.meta = o;
    o += up256((size_t)(K / group) * l.Rp * 4);
    l.exps = o;
    o += up256((size_t)l.Rp * 2);
    l.pows = o;
    o += back ? up256((size_t)l.Rp) : 0;
    l.texp = o;
    o += up256((size_t)l.Mp * 4);
    l.op = o;
    o += up256((size_t)M * l.Cp * 2);
    l.partial = o;
    o += (size_t)(num_sms / 2) * 2 * NT * kTileRows * 4;  // two slots per CTA pair
    l.total = o;
    return l;
}

template <class Kern, class... Args>
int launch_clusters(Kern kernel, int64_t grid, int cluster, int block, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}
template <class Kern, class... Args>
int launch_pdl(Kern kernel, int64_t grid, int block, cudaStream_t stream, Args... args) {
    return launch_clusters(kernel, grid, 1, block, stream, args...);
}

template <int W, bool GATED, int TH>
int launch_grad_as(GradArgs g, int64_t M, cudaStream_t stream) {
    // few tokens of long rows: up to 8 blocks a token, doubled while there are no more blocks than SMs
    const int64_t steps = ceil_div(GATED ? g.I : g.N, TH * 8);
    g.blocks = 1;
    while (g.blocks < 8 && g.blocks < steps && M * g.blocks <= num_sms_current()) g.blocks *= 2;
    return launch_clusters(prep_grad_kernel<W, GATED, TH>, M * g.blocks, g.blocks, TH, stream, g);
}
// Threads per block: 128 for many tokens of short rows (a block's fixed cost is then most of it); else 512, or 256 for
// plain gradients of many tokens in 16-byte loads (4096 x 10240: 35.2 us against 41.3; 100 x 7680: 6.0 against 4.6; gated
// 2048 x 57344: 186-202 against 176).  us with 128 / 256 / 512 threads, rows of 2048: plain 160 tokens 3.5 / 2.7 / 2.9, 300
// 3.7 / 3.0 / 3.2, 600 4.0 / 3.4 / 4.9, 4096 11.4 / 12.2 / 19.6; gated 160 6.0 / 4.5 / 4.8, 300 6.5 / 5.5 / 7.5, 4096 28 /
// 32 / 49; rows of 4096: plain 600 tokens 6.3 / 5.1 / 5.8, 4096 18.9 / 19.4 / 23.8; gated 600 13.3 / 13.0 / 13.4, 4096 51 /
// 54 / 63.
template <int W, bool GATED>
int launch_grad_wide(const GradArgs& g, int64_t M, cudaStream_t stream) {
    const int64_t sms = num_sms_current(), n = GATED ? g.I : g.N;
    if (n <= 2048 && M > 2 * sms) return launch_grad_as<W, GATED, 128>(g, M, stream);
    if constexpr (!GATED && W == 8)
        if (M >= 4 * sms) return launch_grad_as<W, GATED, 256>(g, M, stream);
    return launch_grad_as<W, GATED, 512>(g, M, stream);
}
// 16-byte accesses where every row (gated: every half row) starts on 16 bytes, else 4-byte ones where on 4.
template <bool GATED>
int launch_grad(const GradArgs& g, int64_t M, cudaStream_t stream) {
    const int n = GATED ? g.I : g.N;
    return n % 8 == 0   ? launch_grad_wide<8, GATED>(g, M, stream)
           : n % 2 == 0 ? launch_grad_wide<2, GATED>(g, M, stream)
                        : launch_grad_wide<1, GATED>(g, M, stream);
}

template <int MODE, int NT>
int launch_tiles(HArgs a, const CUtensorMap& tx, const CUtensorMap& tq, const CUtensorMap& tm, cudaStream_t stream) {
    using C = Cfg<MODE, NT>;
    a.NS = (int)ceil_div(a.C, C::kStageK);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = 2;
    attrs[0].val.clusterDim.y = 1;
    attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    // clusters that are resident at once (a cluster needs two free SMs of one GPC)
    static PerContext<int> cache;
    const int units = cache.get([&]() -> int {
        if (cudaFuncSetAttribute(gemm_h_kernel<MODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) !=
            cudaSuccess)
            return 0;
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3((unsigned)(num_sms_current() / 2 * 2));
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, gemm_h_kernel<MODE, NT>, &q) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        return n < num_sms_current() / 2 ? n : num_sms_current() / 2;
    });
    if (units <= 0) return W4A16_ERR_CUDA;
    cfg.numAttrs = 2;
    const int tiles = a.m_tiles * a.r_tiles;
    // Whole waves run whole, and so does a last, partial one where cutting it saves less than it costs.  It saves the
    // idle clusters' share of a tile's stages, 0.32 us each (backward 0.27); it costs the parts' way through memory and
    // the join, 0.9 ns per tile and token place and 1 us (backward 2).  Measured, us cut / whole, with 256 tokens, K = 512,
    // 2048, 4096, 8192: 20 tiles 16.8 / 16.5, 22.5 / 23.8, 27.1 / 33.6, 34.7 / 58.3; 40 tiles 26.0 / 17.6, 31.2 / 25.7,
    // 38.0 / 38.0, 51.4 / 60.7; 60 tiles 32.9 / 18.6, 40.5 / 28.2, 50.3 / 40.7, 71.0 / 63.3; with 40 tokens and 40 tiles
    // 12.8 / 11.2, 15.7 / 15.6, 19.8 / 21.7, 27.3 / 34.3.
    int cut = tiles % units;
    const int64_t saves = (int64_t)(units - cut) * a.NS * (MODE == kDx ? 270 : 320) / units;
    const int64_t costs = (MODE == kDx ? 2000 : 1000) + (int64_t)cut * NT * 9 / 10;
    if (saves < costs) cut = 0;
    a.whole_tiles = tiles - cut;
    a.units = units;
    a.base = 1;
    a.rem = 0;
    a.split_units = 0;
    if (cut > 0) {
        const int64_t stages = (int64_t)cut * a.NS;
        int64_t parts = stages * C::kStageK / 256;  // at least four lines of 64 each
        if (parts > units) parts = units;
        if (parts < 1) parts = 1;
        a.split_units = (int)parts;
        a.base = (int)(stages / parts);
        a.rem = (int)(stages % parts);
    }
    const int busy = a.whole_tiles > 0 ? (a.whole_tiles < units ? a.whole_tiles : units) : 0;
    const int grid = busy > a.split_units ? busy : a.split_units;
    cfg.gridDim = dim3((unsigned)(grid * 2));
    if (cudaLaunchKernelEx(&cfg, gemm_h_kernel<MODE, NT>, tx, tq, tm, a) != cudaSuccess) return W4A16_ERR_CUDA;
    if (cut == 0) return W4A16_OK;
    return launch_pdl(gemm_h_join_kernel<MODE, NT>, (int64_t)cut * (NT / kJoinTokens), kTileRows, stream, a);
}

template <int MODE>
int launch_mode(int NT, const HArgs& a, const CUtensorMap& tx, const CUtensorMap& tq, const CUtensorMap& tm,
                cudaStream_t stream) {
    return NT == 64    ? launch_tiles<MODE, 64>(a, tx, tq, tm, stream)
           : NT == 128 ? launch_tiles<MODE, 128>(a, tx, tq, tm, stream)
                       : launch_tiles<MODE, 256>(a, tx, tq, tm, stream);
}

}  // namespace

size_t gemm_h_workspace_bytes(int64_t M, int64_t N, int64_t K, int group, bool backward, int num_sms) {
    return layout_h(M, N, K, group, backward, num_sms).total;
}

int launch_gemm_h(const uint16_t* X, const float* xscale, int64_t M, int64_t K, int group, const uint32_t* qweight,
                  const uint16_t* scales, const int32_t* zeros, int64_t N, const FusedEpilogue& e, uint16_t* Y,
                  void* workspace, cudaStream_t stream) {
    const Layout l = layout_h(M, N, K, group, false, num_sms_current());
    const int NT = tile_tokens(M);
    char* ws = reinterpret_cast<char*>(workspace);
    int* fault = fault_word();
    if (!fault) return W4A16_ERR_CUDA;
    const int64_t I = e.gated ? N / 2 : 0;
    HArgs a{};
    a.meta = reinterpret_cast<uint32_t*>(ws + l.meta);
    a.exps = reinterpret_cast<int16_t*>(ws + l.exps);
    a.texp = reinterpret_cast<int*>(ws + l.texp);
    a.scales = scales;
    a.zeros = zeros;
    a.Y = Y;
    a.partial = reinterpret_cast<float*>(ws + l.partial);
    a.fault = fault;
    a.ep = e;
    a.I = I;
    a.M = (int)M;
    a.R = (int)N;
    a.C = (int)K;
    a.GQ = (int)(K / group);
    a.group = group;
    a.m_tiles = (int)ceil_div(M, NT);
    a.r_tiles = (int)ceil_div(N, kTileRows);
    const uint32_t stage_k = NT == 256 ? Cfg<kLinear, 256>::kStageK : Cfg<kLinear, 64>::kStageK;
    // a stage's codes are stage_k / 2 bytes of a row
    const CUtensorMapSwizzle swizzle = stage_k == 64 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap tx, tq, tm;
    if (!encode_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws + l.op, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2, kBK,
                        (uint32_t)NT / 2, CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A16_ERR_CUDA;
    const bool ok = e.gated ? encode_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT32, qweight,
                                             {(uint64_t)K / 8, 2, (uint64_t)I}, {(uint64_t)I * K / 2, (uint64_t)K / 2},
                                             {stage_k / 8, 2, kBM / 2}, swizzle)
                            : encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT32, qweight, (uint64_t)K / 8, (uint64_t)N,
                                             (uint64_t)K / 2, stage_k / 8, kBM, swizzle);
    // the meta words of a stage: 128 rows x the groups of its k
    if (!ok || !encode_tmap_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, ws + l.meta, (uint64_t)l.Rp, (uint64_t)a.GQ,
                               (uint64_t)l.Rp * 4, kBM, stage_k > (uint32_t)group ? stage_k / (uint32_t)group : 1))
        return W4A16_ERR_CUDA;
    const MetaArgs ma{qweight, scales, zeros, reinterpret_cast<uint32_t*>(ws + l.meta),
                      reinterpret_cast<int16_t*>(ws + l.exps), nullptr, (int)N, (int)l.Rp, a.GQ, group / 8, I};
    const TokenArgs t{X, xscale, reinterpret_cast<__half*>(ws + l.op), reinterpret_cast<int*>(ws + l.texp), (int)M,
                      (int)K};
    const int st = few_rows(l.Rp) ? launch_pdl(prep_forward_kernel<8>, l.Rp / 8 + M, kPrepThreads, stream, ma, t)
                                  : launch_pdl(prep_forward_kernel<16>, l.Rp / 16 + M, kPrepThreads, stream, ma, t);
    if (st != W4A16_OK) return st;
    return e.gated ? launch_mode<kGated>(NT, a, tx, tq, tm, stream) : launch_mode<kLinear>(NT, a, tx, tq, tm, stream);
}

int launch_gemm_h_dx(const uint16_t* dY, const uint16_t* dH, const uint16_t* GU, int act, uint16_t* dGU, int64_t M,
                     int64_t N, int group, const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros,
                     int64_t K, const float* inv_s, uint16_t* dX, void* workspace, cudaStream_t stream) {
    const Layout l = layout_h(M, N, K, group, true, num_sms_current());
    const int NT = tile_tokens(M);
    char* ws = reinterpret_cast<char*>(workspace);
    int* fault = fault_word();
    if (!fault) return W4A16_ERR_CUDA;
    HArgs a{};
    a.meta = reinterpret_cast<uint32_t*>(ws + l.meta);
    a.exps = reinterpret_cast<int16_t*>(ws + l.exps);
    a.texp = reinterpret_cast<int*>(ws + l.texp);
    a.scales = scales;
    a.zeros = zeros;
    a.inv_s = inv_s;
    a.Y = dX;
    a.partial = reinterpret_cast<float*>(ws + l.partial);
    a.fault = fault;
    a.M = (int)M;
    a.R = (int)K;
    a.C = (int)N;
    a.GQ = (int)(K / group);
    a.group = group;
    a.m_tiles = (int)ceil_div(M, NT);
    a.r_tiles = (int)ceil_div(K, kTileRows);
    CUtensorMap tx, tq, tm;
    // rows of N values, Np apart: what lies past N is filled with zeros.  Codes: 64 rows x the columns; meta words: 64
    // rows x the columns' groups.
    if (!encode_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws + l.op, (uint64_t)N, (uint64_t)M, (uint64_t)l.Cp * 2,
                        kBK, (uint32_t)NT / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT32, qweight, (uint64_t)K / 8, (uint64_t)N, (uint64_t)K / 2,
                        kBM / 8, kBK, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_tmap_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, ws + l.meta, (uint64_t)l.Rp, (uint64_t)a.GQ,
                        (uint64_t)l.Rp * 4, kBK, (uint32_t)(kBM / group)))
        return W4A16_ERR_CUDA;
    const MetaArgs ma{qweight, scales, zeros, reinterpret_cast<uint32_t*>(ws + l.meta),
                      reinterpret_cast<int16_t*>(ws + l.exps), reinterpret_cast<uint8_t*>(ws + l.pows), (int)N, (int)l.Rp,
                      a.GQ, group / 8, 0};
    int st = few_rows(l.Rp) ? launch_pdl(prep_meta_kernel<8>, l.Rp / 8, kPrepThreads, stream, ma)
                            : launch_pdl(prep_meta_kernel<16>, l.Rp / 16, kPrepThreads, stream, ma);
    if (st != W4A16_OK) return st;
    GradArgs g{};
    g.dY = dY;
    g.dH = dH;
    g.GU = GU;
    g.dGU = dGU;
    g.exps = a.exps;
    g.pows = reinterpret_cast<uint8_t*>(ws + l.pows);
    g.Dh = reinterpret_cast<__half*>(ws + l.op);
    g.texp = reinterpret_cast<int*>(ws + l.texp);
    g.N = (int)N;
    g.I = (int)(N / 2);
    g.act = act;
    g.Np = l.Cp;
    st = dH ? launch_grad<true>(g, M, stream) : launch_grad<false>(g, M, stream);
    if (st != W4A16_OK) return st;
    return launch_mode<kDx>(NT, a, tx, tq, tm, stream);
}

}  // namespace w4a16
