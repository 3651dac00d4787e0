// moe_route.cu -- the router: gate product, choice of experts, weights.
//
//   l[t,e] = x[t] . gate[e];  s = softmax_e(l) or sigmoid(l)
//   c = l, or s + bias (with a bias or expert groups)
//   expert groups: only the topk_group groups with the largest sum of their two
//   best c stay; ids[t] = the top_k largest c, lowest index first among equals
//   weights[t] = s[ids], optionally over their sum, times scale
//
// One CTA per (expert, eight tokens) computes eight dot products; the last CTA
// of a token group to arrive chooses, one warp per token.  The choice must not
// depend on how a sum was split, so the sums carry a second word: bf16
// products are exact in fp32, and each addition's error is kept (two-sum), which
// leaves a relative error of about 2^-45 of the sum of magnitudes; scores are
// then formed and compared in 64 bits.
#include "moe_common.cuh"

namespace arf {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteTokens = 8;
constexpr int kPerLane = kMoeMaxExperts / 32;

struct Sum2 {
    float hi, lo;
};

// s + (hi, lo), the error of the leading addition kept
__device__ __forceinline__ Sum2 add2(Sum2 s, float hi, float lo) {
    const float r = __fadd_rn(s.hi, hi);
    const float b = __fsub_rn(r, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(r, b)), __fsub_rn(hi, b));
    return Sum2{r, __fadd_rn(s.lo, __fadd_rn(e, lo))};
}

// A double as an integer of the same order; NaN below everything.
__device__ __forceinline__ long long ordered(double v) {
    if (v != v) return (long long)0x8000000000000000ull;
    const long long b = __double_as_longlong(v + 0.0);  // -0 becomes +0
    return b >= 0 ? b : (long long)(0x8000000000000000ull - (unsigned long long)b);
}

struct Best {
    long long key;
    int index;
};
__device__ __forceinline__ Best better(Best a, Best b) { return b.key > a.key || (b.key == a.key && b.index < a.index) ? b : a; }
__device__ __forceinline__ Best warp_best(Best v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Best u;
        u.key = __shfl_xor_sync(0xffffffffu, v.key, o);
        u.index = __shfl_xor_sync(0xffffffffu, v.index, o);
        v = better(v, u);
    }
    return v;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp: the choice for one token.  Lane l holds experts l, l + 32, ...
__device__ void choose(const RouteArgs& a, int token, int lane, double* scores /* shared, [E] */,
                       long long* keys /* shared, [E] */) {
    constexpr long long kNone = (long long)0x8000000000000000ull;
    const float2* l = a.logits + (int64_t)token * a.E;
    double top = -INFINITY, total = 0.0;
    for (int e = lane; e < a.E; e += 32) {
        const float2 v = __ldcg(l + e);
        scores[e] = (double)v.x + (double)v.y;
        top = fmax(top, scores[e]);
    }
    const bool by_logit = a.bias == nullptr && a.n_group == 1;
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    for (int e = lane; e < a.E; e += 32) {
        const double z = scores[e];
        if (by_logit) keys[e] = ordered(z);
        scores[e] = a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - top);
        total += scores[e];
    }
    if (!a.sigmoid) {
        total = warp_sum_d(total);
        for (int e = lane; e < a.E; e += 32) scores[e] /= total;
    }
    if (!by_logit)
        for (int e = lane; e < a.E; e += 32) keys[e] = ordered(a.bias ? scores[e] + (double)a.bias[e] : scores[e]);
    __syncwarp();
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        // lane = group: the sum of its two best
        long long mine = kNone;
        if (lane < a.n_group) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double c = a.bias ? scores[e] + (double)a.bias[e] : scores[e];
                if (c > b0) {
                    b1 = b0;
                    b0 = c;
                } else if (c > b1) {
                    b1 = c;
                }
            }
            mine = ordered(b0 + b1);
        }
        unsigned kept = 0;
        bool out = lane >= a.n_group;
        for (int r = 0; r < a.topk_group; ++r) {
            const Best b = warp_best(Best{out ? kNone : mine, out ? 32 + lane : lane});
            kept |= 1u << b.index;
            out = out || lane == b.index;
        }
        for (int e = lane; e < a.E; e += 32)
            if (!(kept >> (e / size) & 1)) keys[e] = kNone;
        __syncwarp();
        // experts of dropped groups must lose to kept ones whose key is the lowest too (NaN, minus infinity)
        for (int e = lane; e < a.E; e += 32)
            if ((kept >> (e / size) & 1) && keys[e] == kNone) keys[e] = kNone + 1;
    }
    unsigned taken = 0;  // bit i: expert lane + 32 i
    double sum = 0.0, my_score = 0.0;
    int my_id = 0;
    for (int k = 0; k < a.K; ++k) {
        Best b{kNone, 0x7fffffff};
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !(taken >> i & 1)) b = better(b, Best{keys[e], e});
        }
        b = warp_best(b);
        if ((b.index & 31) == lane) taken |= 1u << (b.index >> 5);
        const double s = scores[b.index];
        sum += s;
        if (lane == k) {
            my_id = b.index;
            my_score = s;
        }
    }
    const int slots = a.K + a.shared;
    if (lane < a.K) {
        double w = my_score;
        if (a.renorm) w = sum > 0.0 || sum != sum ? w / sum : 0.0;
        a.ids[(int64_t)token * slots + lane] = my_id;
        a.weights[(int64_t)token * slots + lane] = (float)(w * (double)a.scale);
    } else if (lane < slots) {
        a.ids[(int64_t)token * slots + lane] = a.E + lane - a.K;
        a.weights[(int64_t)token * slots + lane] = 1.0f;
    }
}

__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];  // the choice: [warp][E] scores and keys
    __shared__ Sum2 part[kRouteWarps][kRouteTokens];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int expert = blockIdx.x, t0 = blockIdx.y * kRouteTokens, nt = min(kRouteTokens, a.T - t0);
    pdl_trigger();
    pdl_wait();  // no global memory access before this point

    Sum2 acc[kRouteTokens] = {};
    const uint16_t* w = a.gate + (int64_t)expert * a.H;
    for (int c = threadIdx.x; c < a.H / 8; c += kRouteThreads) {
        float f[8];
        bf16x8_to_f32(ld_early16(w + c * 8), f);
#pragma unroll
        for (int j = 0; j < kRouteTokens; ++j)
            if (j < nt) {
                float v[8];
                bf16x8_to_f32(ld_early16(a.x + (int64_t)(t0 + j) * a.H + c * 8), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j] = add2(acc[j], __fmul_rn(f[i], v[i]), 0.0f);
            }
    }
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) {
        if (j >= nt) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, acc[j].hi, o), lo = __shfl_xor_sync(0xffffffffu, acc[j].lo, o);
            acc[j] = add2(acc[j], hi, lo);
        }
        if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < nt) {
        Sum2 s = part[0][threadIdx.x];
        for (int u = 1; u < kRouteWarps; ++u) s = add2(s, part[u][threadIdx.x].hi, part[u][threadIdx.x].lo);
        // an infinite or undefined sum has no meaningful error word
        if (!isfinite(s.hi)) s.lo = 0.0f;
        a.logits[(int64_t)(t0 + threadIdx.x) * a.E + expert] = make_float2(s.hi, s.lo);
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.count + blockIdx.y, 1u) == (unsigned)a.E - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) a.count[blockIdx.y] = 0;  // for the next call
    double* scores = reinterpret_cast<double*>(smem) + warp * 2 * a.E;
    if (warp < nt) choose(a, t0 + warp, lane, scores, reinterpret_cast<long long*>(scores + a.E));
}

}  // namespace

cudaError_t moe_route_set_attributes() {
    return cudaFuncSetAttribute(moe_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteWarps * kMoeMaxExperts * 16);
}

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t stream, bool pdl) {
    const int smem = kRouteWarps * a.E * 16;  // at most 64 KB
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)a.E, (unsigned)((a.T + kRouteTokens - 1) / kRouteTokens));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_route_kernel, a);
}

}  // namespace arf
