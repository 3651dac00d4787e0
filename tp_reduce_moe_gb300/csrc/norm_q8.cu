// norm_q8.cu -- all-reduce + residual + RMSNorm with an 8-bit output and its
// scales in one pass:
//
//   h = sum_r P_r + residual; y = h * rsqrt(mean(h^2) + eps) * (gamma + weight_bias)
//   s = max |y| / 448 over a group of columns (or the row), q = e4m3(y / s)
//
// One CTA per token row.  A thread holds CPT chunks of eight columns in fp32
// registers from the loads to the stores, so every byte is read and written
// once.  Chunks lie along the lanes, so a group of 32, 64 or 128 columns is 4,
// 8 or 16 neighbouring lanes and its maximum takes that many lanes' shuffles;
// the row's sum of squares and, for one scale a row, its largest |h * gamma|
// meet in shared memory behind one barrier.
#include "arf_host.h"

namespace arf {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr float kE4m3Max = 448.0f;

// A load of data that the kernel before may have written (coherent), read once.
__device__ __forceinline__ uint4 ld_once16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two values rounded to e4m3 (nearest even, NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// The scale of values up to `top`: 1 for a group of zeros, and never subnormal, so that its inverse is finite.
__device__ __forceinline__ float scale_of(float top) {
    return top == 0.0f ? 1.0f : max_nan(top * (1.0f / kE4m3Max), 0x1p-126f);
}

// GROUP_LANES: lanes of eight columns that share a scale; 0: the whole row.
template <int CPT, int GROUP_LANES, bool RES_F32>
__global__ void __launch_bounds__(kNormMaxThreads) norm_q8_kernel(const __grid_constant__ NormQ8Args a) {
    __shared__ float s_sum[32], s_top[32];
    pdl_trigger();
    pdl_wait();  // no global memory access before this point
    const int64_t t = blockIdx.x;
    const int chunks = a.H / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    uint4 gamma[CPT];
    float h[CPT][8];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
        gamma[c] = make_uint4(0, 0, 0, 0);
        if (chunk < chunks) gamma[c] = *reinterpret_cast<const uint4*>(a.gamma + chunk * 8);
    }
    // partials in rank order, then the residual, up to four rows of each chunk in flight
    for (int r0 = 0; r0 <= a.R; r0 += 4) {
        uint4 v[CPT][4];
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int chunk = threadIdx.x + c * blockDim.x;
                v[c][u] = make_uint4(0, 0, 0, 0);
                if (chunk < chunks && r0 + u <= a.R)
                    v[c][u] = ld_once16((r0 + u < a.R ? a.P[r0 + u] : a.residual) + t * a.H + chunk * 8);
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (r0 + u <= a.R)
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    float f[8];
                    bf16x8_to_f32(v[c][u], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[c][j] += f[j];
                }
    }

    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
        if (chunk < chunks) store_residual8<RES_F32>(a.residual_out, t * a.H + chunk * 8, h[c]);
        float g[8];
        bf16x8_to_f32(gamma[c], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = norm_input(h[c][j], a.norm_bf16_h);
            sum = fmaf(x, x, sum);
            h[c][j] = chunk < chunks ? x * (g[j] + a.weight_bias) : 0.0f;
            if (GROUP_LANES == 0) top = max_nan(top, fabsf(h[c][j]));
        }
    }
    sum = warp_sum(sum);
    if (GROUP_LANES == 0)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) {
        s_sum[warp] = sum;
        s_top[warp] = top;
    }
    __syncthreads();
    const int warps = blockDim.x >> 5;
    sum = warp_sum(lane < warps ? s_sum[lane] : 0.0f);
    const float rs = rsqrtf(sum / (float)a.H + a.eps);
    if (GROUP_LANES == 0) {
        top = lane < warps ? s_top[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        top *= rs;
    }
    const int per_row = GROUP_LANES == 0 ? 1 : (chunks + GROUP_LANES - 1) / GROUP_LANES;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
        float largest = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[c][j] *= rs;
            largest = max_nan(largest, fabsf(h[c][j]));
        }
        if (GROUP_LANES == 0) {
            largest = top;
        } else {
            if (chunk >= chunks) largest = 0.0f;  // (0 * rs is NaN where rs is not finite)
#pragma unroll
            for (int o = GROUP_LANES / 2; o > 0; o >>= 1) largest = max_nan(largest, __shfl_xor_sync(0xffffffffu, largest, o));
        }
        if (chunk >= chunks) continue;
        const float s = scale_of(largest), inv = 1.0f / s;
        if (a.out != nullptr) st_global16(a.out + t * a.H + chunk * 8, f32x8_to_bf16x8(h[c]));
        uint2 q;
        q.x = e4m3x2(h[c][0] * inv, h[c][1] * inv) | e4m3x2(h[c][2] * inv, h[c][3] * inv) << 16;
        q.y = e4m3x2(h[c][4] * inv, h[c][5] * inv) | e4m3x2(h[c][6] * inv, h[c][7] * inv) << 16;
        *reinterpret_cast<uint2*>(a.q + t * a.H + chunk * 8) = q;
        if (GROUP_LANES == 0 ? chunk == 0 : chunk % (GROUP_LANES > 0 ? GROUP_LANES : 1) == 0)
            a.scales[t * per_row + (GROUP_LANES > 0 ? chunk / (GROUP_LANES > 0 ? GROUP_LANES : 1) : 0)] = s;
    }
}

using Kernel = void (*)(NormQ8Args);

template <int CPT, bool RES_F32>
Kernel kernel_of(int group) {
    switch (group) {
        case 32: return norm_q8_kernel<CPT, 4, RES_F32>;
        case 64: return norm_q8_kernel<CPT, 8, RES_F32>;
        case 128: return norm_q8_kernel<CPT, 16, RES_F32>;
    }
    return norm_q8_kernel<CPT, 0, RES_F32>;
}

}  // namespace

cudaError_t launch_norm_q8(const NormQ8Args& a, int group, bool res_f32, cudaStream_t stream, bool pdl) {
    const int chunks = a.H / 8;
    const int cpt = chunks > kNormMaxThreads ? 2 : 1;
    const int threads = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
    if (a.T < 1 || a.T > 0x7fffffff || threads > kNormMaxThreads) return cudaErrorInvalidValue;
    const Kernel k = cpt == 1 ? (res_f32 ? kernel_of<1, true>(group) : kernel_of<1, false>(group))
                              : (res_f32 ? kernel_of<2, true>(group) : kernel_of<2, false>(group));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace arf
