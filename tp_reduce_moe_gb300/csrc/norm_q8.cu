// norm_q8.cu -- all-reduce + residual + RMSNorm with an 8-bit output and its
// scales in one pass:
//
//   h = sum_r P_r + residual; y = h * rsqrt(mean(h^2) + eps) * (gamma + weight_bias)
//   s = max |y| / 448 over a group of columns (or the row), q = e4m3(y / s)
//
// A thread holds CPT chunks of eight columns of a row in fp32 registers from the loads to
// the stores, so every byte is read and written once.  Chunks lie along the lanes, so a
// group of 32, 64 or 128 columns is 4, 8 or 16 neighbouring lanes and its maximum takes that
// many lanes' shuffles; the row's sum of squares and, for one scale a row, its largest
// |h * gamma| meet in shared memory behind one barrier.
//
// What bounds it: memory, for many rows (8192 of 8192 columns, two partials: 101 us, 6.1 TB/s of
// what is read and written, 0.90 of a copy's rate; 73 % of the issue slots are in use), and
// for few the launch and two trips to memory (one row 2.4 us).  The kernel of a CTA a row spills 32 bytes a thread where a thread has
// two chunks (rows of more than 8192 columns).
//
// Few rows: a CTA a row, partials loaded to registers, four in flight a chunk.  Many: CTAs
// stay and take every so many rows; the rows of partials come through a ring in shared
// memory by asynchronous copies, each thread copying what it reads itself, so that loads run
// ahead over the rows' barriers and nothing waits but for its own copies.
#include "arf_host.h"

namespace arf {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kPlaces = 6;        // of the ring
constexpr int kNormSmem = 220 * 1024;
static_assert(kPlaces * 2 * kNormMaxThreads * 16 <= kNormSmem, "shared memory of a CTA");
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

__device__ __forceinline__ float reciprocal(float x) {  // to a last place
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The scale of values up to `top`: 1 for a group of zeros, and never subnormal, so that its inverse is finite.
__device__ __forceinline__ float scale_of(float top) {
    return top == 0.0f ? 1.0f : max_nan(top * (1.0f / kE4m3Max), 0x1p-126f);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void add8(float h[8], uint4 v) {
    float f[8];
    bf16x8_to_f32(v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] += f[j];
}

// The largest |y| of a row, of the h that its norm reads, by all threads.
template <int CPT>
__device__ __forceinline__ float largest_of_row(const NormQ8Args& a, const float h[CPT][8], const uint4 gamma[CPT], float rs, float* s_top) {
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        float g[8];
        bf16x8_to_f32(gamma[c], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(h[c][j] * rs * (g[j] + a.weight_bias)));
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();  // what was in s_top has been read
    if (lane == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
    top = lane < (int)(blockDim.x >> 5) ? s_top[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}

// Everything behind the sum: h [CPT chunks of this thread], which is used up; of chunks behind the row it may be anything.
// s_sum and s_top are not written again before all threads have come through a barrier behind this.  GROUP_LANES: lanes of
// eight columns that share a scale; 0: the row.
template <int CPT, int GROUP_LANES, bool RES_F32>
__device__ __forceinline__ void finish_row(const NormQ8Args& a, int64_t t, float h[CPT][8], const uint4 gamma[CPT], float* s_sum, float* s_top) {
    const int chunks = a.H / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool full = chunks == CPT * (int)blockDim.x;  // every thread's chunks are columns
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
        if (full || chunk < chunks)
            store_residual8<RES_F32>(a.residual_out, t * a.H + chunk * 8, h[c]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[c][j] = norm_input(h[c][j], a.norm_bf16_h);
            sum = fmaf(h[c][j], h[c][j], sum);
        }
        if (GROUP_LANES == 0) {
            float g[8];
            bf16x8_to_f32(gamma[c], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(h[c][j] * (g[j] + a.weight_bias)));
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
    const float rs = rsqrtf(sum * reciprocal((float)a.H) + a.eps);
    if (GROUP_LANES == 0) {
        top = lane < warps ? s_top[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top == INFINITY)  // (all threads) products that pass the range, as y may not: again, of y itself
            top = largest_of_row<CPT>(a, h, gamma, rs, s_top);
        else
            top *= rs;
    }
    const int per_row = GROUP_LANES == 0 ? 1 : (chunks + GROUP_LANES - 1) / GROUP_LANES;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
        float largest = 0.0f, g[8];
        bf16x8_to_f32(gamma[c], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[c][j] *= rs;  // (first: with the weight it may pass the range)
            h[c][j] *= g[j] + a.weight_bias;
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
        const float s = scale_of(largest), inv = reciprocal(s);
        if (a.out != nullptr) st_global16(a.out + t * a.H + chunk * 8, f32x8_to_bf16x8(h[c]));
        uint2 q;
        q.x = e4m3x2(h[c][0] * inv, h[c][1] * inv) | e4m3x2(h[c][2] * inv, h[c][3] * inv) << 16;
        q.y = e4m3x2(h[c][4] * inv, h[c][5] * inv) | e4m3x2(h[c][6] * inv, h[c][7] * inv) << 16;
        *reinterpret_cast<uint2*>(a.q + t * a.H + chunk * 8) = q;
        if (GROUP_LANES == 0 ? chunk == 0 : chunk % (GROUP_LANES > 0 ? GROUP_LANES : 1) == 0)
            a.scales[t * per_row + (GROUP_LANES > 0 ? chunk / (GROUP_LANES > 0 ? GROUP_LANES : 1) : 0)] = s;
    }
}

template <int CPT, int GROUP_LANES, bool RES_F32>
__global__ void __launch_bounds__(kNormMaxThreads) norm_q8_kernel(const __grid_constant__ NormQ8Args a) {
    __shared__ float s_sum[32], s_top[32];
    pdl_trigger();
    pdl_wait();  // no global memory access before this point
    const int64_t t = blockIdx.x;
    const int chunks = a.H / 8;
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
                for (int c = 0; c < CPT; ++c) add8(h[c], v[c][u]);
    }
    finish_row<CPT, GROUP_LANES, RES_F32>(a, t, h, gamma, s_sum, s_top);
}

// Rows t, t + gridDim.x, ...: the ring's places hold CPT chunks of one partial (or the residual) for each thread.
template <int CPT, int GROUP_LANES, bool RES_F32>
__global__ void __launch_bounds__(kNormMaxThreads) norm_q8_stream_kernel(const __grid_constant__ NormQ8Args a) {
    extern __shared__ __align__(16) uint4 s_ring[];  // [kPlaces][CPT][threads]
    __shared__ float s_sum[2][32], s_top[2][32];
    pdl_trigger();
    pdl_wait();  // no global memory access before this point
    const int chunks = a.H / 8;
    const uint64_t policy = l2_evict_first_policy();
    uint4 gamma[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int chunk = threadIdx.x + c * blockDim.x;
        gamma[c] = chunk < chunks ? *reinterpret_cast<const uint4*>(a.gamma + chunk * 8) : make_uint4(0, 0, 0, 0);
    }
    int64_t ask_at = (int64_t)blockIdx.x * a.H + threadIdx.x * 8;  // in a partial, of the thread's first chunk
    const int64_t behind = a.T * a.H, further = (int64_t)gridDim.x * a.H;
    int ask_r = 0;
    uint4* const mine = s_ring + threadIdx.x;
    const uint32_t mine_at = smem_addr(mine);
    const bool any = (int)threadIdx.x < chunks, second = (int)(threadIdx.x + blockDim.x) < chunks;
    auto ask = [&](int place) {
        if (ask_at < behind) {
            const uint16_t* from = (ask_r < a.R ? a.P[ask_r] : a.residual) + ask_at;
            const uint32_t to = mine_at + place * CPT * blockDim.x * 16;
            if (any) copy16(to, from, policy);
            if (CPT == 2 && second) copy16(to + blockDim.x * 16, from + blockDim.x * 8, policy);
            if (++ask_r > a.R) {
                ask_r = 0;
                ask_at += further;
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int p = 0; p < kPlaces; ++p) ask(p);
    int place = 0;
    bool odd = false;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, odd = !odd) {
        float h[CPT][8];
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
        for (int r = 0; r <= a.R; ++r) {
            copy_wait<kPlaces - 1>();
            uint4 v[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) v[c] = mine[(place * CPT + c) * blockDim.x];
#pragma unroll
            for (int c = 0; c < CPT; ++c) add8(h[c], v[c]);  // (of chunks behind the row: anything, not used)
            ask(place);  // (a thread reads before it copies over)
            place = place + 1 == kPlaces ? 0 : place + 1;
        }
        // (a thread can be one row ahead of another: two places for the sums)
        finish_row<CPT, GROUP_LANES, RES_F32>(a, t, h, gamma, s_sum[odd], s_top[odd]);
    }
}

using Kernel = void (*)(NormQ8Args);

template <int CPT, bool RES_F32, bool STREAM>
Kernel kernel_of(int group) {
    switch (group) {
        case 32: return STREAM ? norm_q8_stream_kernel<CPT, 4, RES_F32> : norm_q8_kernel<CPT, 4, RES_F32>;
        case 64: return STREAM ? norm_q8_stream_kernel<CPT, 8, RES_F32> : norm_q8_kernel<CPT, 8, RES_F32>;
        case 128: return STREAM ? norm_q8_stream_kernel<CPT, 16, RES_F32> : norm_q8_kernel<CPT, 16, RES_F32>;
    }
    return STREAM ? norm_q8_stream_kernel<CPT, 0, RES_F32> : norm_q8_kernel<CPT, 0, RES_F32>;
}

template <bool STREAM>
Kernel kernel_for(int cpt, bool res_f32, int group) {
    return cpt == 1 ? (res_f32 ? kernel_of<1, true, STREAM>(group) : kernel_of<1, false, STREAM>(group))
                    : (res_f32 ? kernel_of<2, true, STREAM>(group) : kernel_of<2, false, STREAM>(group));
}

}  // namespace

cudaError_t launch_norm_q8(const NormQ8Args& a, int group, bool res_f32, int num_sms, std::atomic<unsigned>* ready, cudaStream_t stream) {
    const int chunks = a.H / 8;
    // CTAs that stay, once there are more rows than SMs.  (Two partials of 7168 columns, 896 threads a row: 152 rows 2.5 us, a CTA a
    // row; 153 4.1, a CTA a row 4.2; 200 4.2 and 4.3; 304 4.4 and 4.7; 400 7.9 and 7.1; 608 9.8 and 11.2; 4096 44 and 67.  Eight of
    // 6144: 153 rows 5.5 and 6.0, 200 5.9 and 7.2, 304 7.7 and 9.5, 4096 85 and 118.  Rows of 4096 columns, of which two CTAs fit an SM,
    // would rather have one each up to some 500 of them: 153 3.5 and 2.5, 256 4.4 and 2.6, 400 4.6 and 4.1, 608 4.8 and 4.9.)
    const bool stay = a.T > num_sms;
    const int cpt = chunks > (stay ? 256 : kNormMaxThreads) ? 2 : 1;
    const int threads = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
    if (a.T < 1 || a.T > 0x7fffffff || threads > kNormMaxThreads) return cudaErrorInvalidValue;
    const Kernel k = stay ? kernel_for<true>(cpt, res_f32, group) : kernel_for<false>(cpt, res_f32, group);
    int64_t grid = a.T;
    size_t smem = 0;
    if (stay) {
        const unsigned bit = 1u << ((cpt - 1) * 8 + res_f32 * 4 + (group == 0 ? 0 : group == 32 ? 1 : group == 64 ? 2 : 3));
        if (!(ready->load(std::memory_order_acquire) & bit)) {  // (two threads may both do this: it sets the same value)
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
            if (e != cudaSuccess) return e;
            ready->fetch_or(bit, std::memory_order_release);
        }
        smem = (size_t)kPlaces * cpt * threads * 16;
        // as many CTAs as an SM's threads (of up to 64 registers) and shared memory take
        int per_sm = 1024 / threads;
        if (per_sm > (int)(kNormSmem / smem)) per_sm = (int)(kNormSmem / smem);
        if (per_sm < 1) per_sm = 1;
        if (grid > (int64_t)per_sm * num_sms) grid = (int64_t)per_sm * num_sms;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // always: it only moves the launch under the end of the kernel before
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace arf
