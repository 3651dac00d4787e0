// matvec_w4.cu -- products of a few tokens with a 4-bit weight matrix.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[t, k]
//
// Weight rows are dealt evenly over the SMs; a CTA takes its rows in blocks of
// up to 16 * MT, its sixteen warps split the columns of a block and add their
// parts through shared memory.  The codes are exact in bf16, so the inner sum
// is one of exact products in fp32, scaled once per group.
#include "moe_common.cuh"

namespace arf {
namespace {

template <int GS, int MT, int NT>
constexpr int smem_bytes() {
    return kMvWarps * Fmt<GS>::kRingBytes + 2 * kMvWarps * MT * NT * 512;
}

template <int GS, int MT, int NT>
__global__ void __launch_bounds__(kMvThreads, 1) matvec_w4_kernel(const __grid_constant__ MatvecArgs a) {
    using F = Fmt<GS>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + kMvWarps * F::kRingBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = (int)((int64_t)a.N * blockIdx.x / gridDim.x), r1 = (int)((int64_t)a.N * (blockIdx.x + 1) / gridDim.x);
    if (r0 >= r1) return;
    Rows m;
    m.q = a.q;
    m.s = a.s;
    m.row_bytes = F::row_bytes(a.K);
    m.row_scales = a.K / (128 / GS);
    m.s_end = a.s + (int64_t)a.N * m.row_scales;
    const int steps = F::steps(a.K);
    const int s0 = steps * warp / kMvWarps, s1 = steps * (warp + 1) / kMvWarps;
    const uint32_t ring = smem_addr(smem) + warp * F::kRingBytes;

    // Blocks in the order (rows, tokens): more tokens than columns read the same
    // rows again at once, from L2.
    int crow = r0, ctok = 0, cstep = s0, ctile = 0, cslot = 0;
    bool more = s0 < s1;
    auto copy_next = [&]() {
        if (more) {
            const int n = min(16 * MT, r1 - crow) - 16 * ctile;
            const int64_t lo = crow + 16 * ctile;
            copy_stage<GS>(ring + cslot * F::kStageBytes, m, lo, n, lo + 8, n - 8, cstep, lane);
            cslot = cslot + 1 == F::kStages ? 0 : cslot + 1;
            if (n <= 16 || ++ctile == MT) {
                ctile = 0;
                if (++cstep == s1) {
                    cstep = s0;
                    ctok += 8 * NT;
                    if (ctok >= a.T) {
                        ctok = 0;
                        crow += 16 * MT;
                        more = crow < r1;
                    }
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < F::kStages - 1; ++s) copy_next();

    int slot = 0, buf = 0;
    for (int row = r0; row < r1; row += 16 * MT)
        for (int tok = 0; tok < a.T; tok += 8 * NT) {
            const int rows = min(16 * MT, r1 - row), tiles = (rows + 15) >> 4;
            float acc[MT][NT][4] = {};
            uint4 col[NT][F::kBlocks], next[NT][F::kBlocks];
            auto columns = [&](uint4 (&c)[NT][F::kBlocks], int step) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int token = tok + 8 * n + g;
                    const bool ok = token < a.T && step < s1;
                    load_columns<GS, false>(c[n], a.x + (ok ? (int64_t)token * a.K + (int64_t)step * F::kStepK : 0),
                                            a.K - step * F::kStepK, ok, t);
                }
            };
            columns(next, s0);
            for (int step = s0; step < s1; ++step) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < F::kBlocks; ++i) col[n][i] = next[n][i];
                columns(next, step + 1);
#pragma unroll
                for (int tile = 0; tile < MT; ++tile)
                    if (tile < tiles) {
                        cp_async_wait<F::kStages - 2>();
                        __syncwarp();  // other lanes' copies; and all reads of the slot that is filled next
                        copy_next();
                        const int64_t lo = row + 16 * tile + g;
                        multiply_stage<GS, NT>(acc[tile], ring + slot * F::kStageBytes, col, scale_shift<GS>(m, lo, step),
                                               scale_shift<GS>(m, lo + 8, step), m.row_scales - step * GS, lane);
                        slot = slot + 1 == F::kStages ? 0 : slot + 1;
                    }
            }
            // add the warps' parts in warp order
            float* r = red + buf * kMvWarps * MT * NT * 128;
#pragma unroll
            for (int tile = 0; tile < MT; ++tile)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float4*>(r + ((warp * MT + tile) * NT + n) * 128 + lane * 4) =
                        make_float4(acc[tile][n][0], acc[tile][n][1], acc[tile][n][2], acc[tile][n][3]);
            __syncthreads();  // and the other buffer's readers are done before it is written again
            for (int i = threadIdx.x; i < MT * NT * 128; i += kMvThreads) {
                float y = 0.0f;
#pragma unroll
                for (int w = 0; w < kMvWarps; ++w) y += r[w * MT * NT * 128 + i];
                const int l = (i >> 2) & 31, n = (i >> 7) % NT, tile = (i >> 7) / NT;
                const int rr = 16 * tile + (l >> 2) + 8 * ((i >> 1) & 1), token = tok + 8 * n + 2 * (l & 3) + (i & 1);
                if (rr < rows && token < a.T) {
                    const int64_t o = (int64_t)token * a.N + row + rr;
                    if (a.out_f32)
                        reinterpret_cast<float*>(a.out)[o] = y;
                    else
                        reinterpret_cast<uint16_t*>(a.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
                }
            }
            buf ^= 1;
        }
    cp_async_wait<0>();
}

template <typename Kernel>
cudaError_t launch_kernel(Kernel kernel, const MatvecArgs& a, int grid, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int GS>
cudaError_t launch(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    const int grid = a.N < num_sms ? a.N : num_sms;
    if (a.T <= 8) return launch_kernel(matvec_w4_kernel<GS, 4, 1>, a, grid, smem_bytes<GS, 4, 1>(), stream);
    return launch_kernel(matvec_w4_kernel<GS, 2, 2>, a, grid, smem_bytes<GS, 2, 2>(), stream);
}

template <int GS>
cudaError_t set_attributes() {
    cudaError_t e = cudaFuncSetAttribute(matvec_w4_kernel<GS, 4, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<GS, 4, 1>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(matvec_w4_kernel<GS, 2, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<GS, 2, 2>());
    return e;
}

}  // namespace

cudaError_t launch_matvec_w4(const MatvecArgs& a, int group, int num_sms, cudaStream_t stream) {
    switch (group) {
        case 32: return launch<4>(a, num_sms, stream);
        case 64: return launch<2>(a, num_sms, stream);
        case 128: return launch<1>(a, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t matvec_w4_set_attributes() {
    cudaError_t e = set_attributes<1>();
    if (e == cudaSuccess) e = set_attributes<2>();
    if (e == cudaSuccess) e = set_attributes<4>();
    return e;
}

}  // namespace arf
