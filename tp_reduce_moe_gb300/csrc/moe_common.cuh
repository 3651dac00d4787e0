// moe_common.cuh -- what the few-token weight-streaming kernels share
// (moe_experts.cu, matvec_w4.cu): parameters, the weight formats, the
// per-warp copy ring and the matrix instruction.
//
// Products of a few tokens with a large weight matrix read every weight once
// and use it a handful of times, so the time is the weights' bytes over the
// memory bandwidth.  One CTA per SM holds sixteen warps; each warp streams its
// own share of the weights through a private ring in shared memory (16-byte
// cp.async, six or seven stages of 16 rows x 64 bytes in flight per warp, about
// 100 KB per SM) and multiplies them with mma.sync m16n8k16, weight rows as
// the 16-row operand and up to eight tokens as the 8-column one.  The
// instruction does eight columns whatever the token count, which the tensor
// pipe has room for: 16 rows x 64 bytes are two bf16 or eight 4-bit
// instructions per warp, against the 44 cycles that the memory takes to
// deliver them to an SM.  A tcgen05 tile of 128 rows would need all its
// operands in shared memory (the 4-bit codes expanded there first) and pay in
// granularity: at one token an SM owns about 27 rows of the first product.
#pragma once

#include "arf_common.cuh"

namespace arf {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;  // routed + shared
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMaxTopK;
constexpr unsigned kErrExpertRange = 0x4u;

constexpr int kMvWarps = 16;
constexpr int kMvThreads = kMvWarps * 32;

struct RouteArgs {
    const uint16_t* x;     // bf16 [T, H]
    const uint16_t* gate;  // bf16 [E, H]
    const float* bias;     // [E] or nullptr
    int32_t* ids;          // [T, K + shared]
    float* weights;        // [T, K + shared]
    float2* logits;        // scratch [T, E], high and low part
    unsigned* count;       // scratch, one arrival counter per token group (zero between calls)
    int T, H, E, K, shared;
    int sigmoid, renorm, n_group, topk_group;
    float scale;
};

struct ExpertsArgs {
    const uint16_t* x;    // bf16 [T, H]
    const int32_t* ids;   // [T, K]
    const float* weights; // [T, K]
    const uint8_t* w13;   // rows of the first product: [E, 2I] rows of H values
    const uint8_t* w2;    // rows of the second: [E, H] rows of I values
    const uint16_t* s13;  // 4-bit: bf16 group scales [E, 2I, H / group]
    const uint16_t* s2;   // 4-bit: bf16 group scales [E, H, I / group]
    uint16_t* act;        // scratch bf16 [T * K, 2, I]: high and low part of the activations
    uint16_t* out;        // bf16 [T, H]
    unsigned* err;
    int T, K, E, H, I;
};

struct MatvecArgs {
    const uint16_t* x;  // bf16 [T, K]
    const uint8_t* q;   // [N, K / 2]
    const uint16_t* s;  // bf16 [N, K / group]
    void* out;          // [T, N] bf16 or fp32
    int T, N, K, out_f32;
};

cudaError_t moe_route_set_attributes();
cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t stream, bool pdl);
// group: 0 for bf16 weights, else 32, 64 or 128
cudaError_t launch_moe_experts(const ExpertsArgs& a, int group, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t moe_experts_set_attributes();
cudaError_t launch_matvec_w4(const MatvecArgs& a, int group, int num_sms, cudaStream_t stream);
cudaError_t matvec_w4_set_attributes();

// ------------------------------------------------------------ weight formats
// A step is 64 bytes of every row of a tile: 32 bf16 values or 128 4-bit
// codes.  GS: scale groups per step (0: bf16 weights).
template <int GS>
struct Fmt {
    static constexpr bool kW4 = GS > 0;
    static constexpr int kStepK = kW4 ? 128 : 32;
    static constexpr int kBlocks = kW4 ? 4 : 1;   // 16-byte activation loads per step and column
    static constexpr int kScaleRow = 16;          // bytes of one row's scale window in a stage
    static constexpr int kStageBytes = 1024 + (kW4 ? 16 * kScaleRow : 0);
    static constexpr int kStages = kW4 ? 7 : 8;  // ring slots per warp; one less in flight
    static constexpr int kRingBytes = kStages * kStageBytes;
    __host__ __device__ static int64_t row_bytes(int64_t k) { return kW4 ? k / 2 : k * 2; }
    __host__ __device__ static int steps(int k) { return (k + kStepK - 1) / kStepK; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c += A (16 x 16, row-major fragments) * B (16 x 8): bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two codes of a word (nibbles 0 and 4 of w) as a pair of bf16 values code - 8.
// 0x4300 is 128 in bf16, whose last place is 1, so or-ing a code into the
// mantissa adds it exactly, and so does taking 136 off.
__device__ __forceinline__ uint32_t dequant2(uint32_t w) {
    const uint32_t v = (w & 0x000f000fu) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// 16 bytes that this grid's predecessor wrote (not the read-only path).
__device__ __forceinline__ uint4 ld_coherent16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// One matrix of weights as the copies see it.
struct Rows {
    const uint8_t* q;       // packed rows
    const uint16_t* s;      // group scales (4-bit)
    const uint16_t* s_end;  // one past the last scale
    int64_t row_bytes;
    int row_scales;         // scales per row
};

// Copies step `step` of the 16-row tile (rows lo .. lo+7 and hi .. hi+7, of
// which n_lo and n_hi exist) into a ring stage.  Lane (g, t) = (lane / 4,
// lane % 4) brings the 16 bytes t of rows g and g + 8; bytes behind the row's
// end and rows that do not exist become zero.
//
// bf16: each lane reads back what it copied itself.  4-bit: the chunks of the
// eight rows are stored side by side, so that lane (g, t) reads word t of
// chunk b of row g without bank conflicts: one word then holds eight
// consecutive codes, and a pair of mma covers the 32 values of chunk b, all of
// one scale group.
template <int GS>
__device__ __forceinline__ void copy_stage(uint32_t stage, const Rows& m, int64_t lo, int n_lo, int64_t hi, int n_hi,
                                           int step, int lane) {
    using F = Fmt<GS>;
    const int g = lane >> 2, t = lane & 3;
    const int64_t at = (int64_t)step * 64 + t * 16;
    const bool in_row = at < m.row_bytes;
    const bool vl = in_row && g < n_lo, vh = in_row && g < n_hi;
    const uint32_t dst = stage + (F::kW4 ? (t * 8 + g) * 16 : lane * 16);
    cp_async16(dst, vl ? m.q + (lo + g) * m.row_bytes + at : m.q, vl);
    cp_async16(dst + 512, vh ? m.q + (hi + g) * m.row_bytes + at : m.q, vh);
    if (F::kW4) {
        // The row's scales of this step, as the aligned 4-byte words that hold
        // them (scales are 2-byte aligned; a step has at most four, so at most
        // three words), 16 bytes a row.  The last word is cut at the end of the
        // array.
        const int r = lane & 15;
        const bool ok = r < 8 ? r < n_lo : r - 8 < n_hi;
        const int64_t row = r < 8 ? lo + r : hi + r - 8;
        const int first = step * GS;
        const uint16_t* b = m.s + (ok ? row * m.row_scales + first : 0);
        const uint16_t* e = b + (ok ? min(GS, m.row_scales - first) : 0);
        const uintptr_t base = reinterpret_cast<uintptr_t>(b) & ~uintptr_t(3);
        const uint32_t sdst = stage + 1024 + r * F::kScaleRow;
#pragma unroll
        for (int w0 = 0; w0 < (GS == 4 ? 3 : 2); w0 += 2) {
            const int w = w0 + (lane >> 4);
            const uintptr_t p = base + 4 * w;
            if (p < reinterpret_cast<uintptr_t>(e)) {
                const int64_t left = (int64_t)(reinterpret_cast<uintptr_t>(m.s_end) - p);
                cp_async4(sdst + 4 * w, reinterpret_cast<const void*>(p), left >= 4 ? 4 : 2);
            }
        }
    }
}

// Activations of one step for one 8-column tile: lane (g, t) holds values
// 8t .. 8t+7 of every 32 of column g (p: the column's first value of the step;
// left: values from there to the end of the row; zeros beyond, and for a
// column that does not exist).
template <int GS, bool COHERENT>
__device__ __forceinline__ void load_columns(uint4 b[Fmt<GS>::kBlocks], const uint16_t* p, int left, bool ok, int t) {
#pragma unroll
    for (int i = 0; i < Fmt<GS>::kBlocks; ++i) {
        const int at = 32 * i + 8 * t;
        b[i] = make_uint4(0, 0, 0, 0);
        if (ok && at < left) b[i] = COHERENT ? ld_coherent16(p + at) : ld_early16(p + at);
    }
}

// The products of a stage: acc[nt] += tile (16 rows x one step) * columns.
// shift_lo, shift_hi: bytes from the scale window's start to the step's first
// scale, for the rows of each half.  groups: scale groups from the step's start
// to the end of the row; what lies behind them in a stage is not looked at (it
// may be the next row's, and zero columns times an infinite scale are not zero).
template <int GS, int NT>
__device__ __forceinline__ void multiply_stage(float (&acc)[NT][4], uint32_t stage, const uint4 (&b)[NT][Fmt<GS>::kBlocks],
                                               int shift_lo, int shift_hi, int groups, int lane) {
    using F = Fmt<GS>;
    if constexpr (!F::kW4) {
        const uint4 lo = lds128(stage + lane * 16), hi = lds128(stage + 512 + lane * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma_16816(acc[n], lo.x, hi.x, lo.y, hi.y, b[n][0].x, b[n][0].y);
            mma_16816(acc[n], lo.z, hi.z, lo.w, hi.w, b[n][0].z, b[n][0].w);
        }
    } else {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t at = stage + g * 16 + t * 4, sc = stage + 1024 + g * F::kScaleRow;
        constexpr int kPer = 4 / GS;  // 32-value blocks per scale group (within the step)
#pragma unroll
        for (int s = 0; s < GS; ++s) {
            if (s >= groups) break;
            float part[NT][4] = {};
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = s * kPer + j;
                const uint32_t lo = lds32(at + i * 128), hi = lds32(at + 512 + i * 128);
                const uint32_t l0 = dequant2(lo), l1 = dequant2(lo >> 4), l2 = dequant2(lo >> 8), l3 = dequant2(lo >> 12);
                const uint32_t h0 = dequant2(hi), h1 = dequant2(hi >> 4), h2 = dequant2(hi >> 8), h3 = dequant2(hi >> 12);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 v = b[n][i];  // values (0,1) (2,3) (4,5) (6,7); a code pair is (i, i + 4)
                    mma_16816(part[n], l0, h0, l1, h1, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
                    mma_16816(part[n], l2, h2, l3, h3, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                }
            }
            const float sl = lds_bf16(sc + shift_lo + 2 * s), sh = lds_bf16(sc + 8 * F::kScaleRow + shift_hi + 2 * s);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(sl, part[n][0], acc[n][0]);
                acc[n][1] = fmaf(sl, part[n][1], acc[n][1]);
                acc[n][2] = fmaf(sh, part[n][2], acc[n][2]);
                acc[n][3] = fmaf(sh, part[n][3], acc[n][3]);
            }
        }
    }
}

// Bytes from a row's aligned scale window to its first scale of the step.
template <int GS>
__device__ __forceinline__ int scale_shift(const Rows& m, int64_t row, int step) {
    if constexpr (GS == 0) return 0;
    return (int)(((unsigned)row * (unsigned)m.row_scales + (unsigned)(step * GS)) & 1u) * 2;
}

}  // namespace arf
