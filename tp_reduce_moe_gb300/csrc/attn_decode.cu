// attn_decode.cu -- attention of one new token of each sequence over its paged
// keys and values:
//
//   s_j = scale q . k_j; out = sum_j softmax(s)_j v_j; lse = log sum_j exp(s_j)
//
// in one pass with a running maximum m, sum l and weighted sum of values: a token with
// score s turns them into m' = max(m, s), l 2^(m - m') + 2^(s - m'), o 2^(m - m') +
// 2^(s - m') v (scores times log2(e)).
//
// One CTA per sequence and query head; each warp takes every fourth token, the lanes
// share its columns, and the warps' results meet in shared memory.
#include "attn_common.cuh"

namespace arf {
namespace {

constexpr int kWarps = 4;

template <int PER>
__device__ __forceinline__ void load_values(const uint8_t* row, bool bytes, int lane, float f[PER]) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int d = lane * PER + j;
        if (bytes) {
            const uint32_t h = e4m3x2_to_f16x2(row[d]);
            f[j] = __half2float(__ushort_as_half((unsigned short)h));
        } else {
            f[j] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(row)[d] << 16);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attn_decode_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int PER = D / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    pdl_trigger();
    pdl_wait();  // no global memory access before this point
    const int head = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kv = head / (a.heads / a.kv);
    const bool bytes = a.k.scale != nullptr;
    const int length = checked_length(a, b, true);
    const int start = a.window > 0 && length > a.window ? length - a.window : 0;
    const float ks = bytes ? a.scale * a.k.scale[kv] : a.scale, vs = bytes ? a.v.scale[kv] : 1.0f;
    const uint16_t* q_row = a.q + ((int64_t)b * a.heads + head) * D;
    float q[PER], o[PER], m = -INFINITY, l = 0.0f;
    load_values<PER>(reinterpret_cast<const uint8_t*>(q_row), false, lane, q);
#pragma unroll
    for (int j = 0; j < PER; ++j) o[j] = 0.0f;
    for (int t = start + warp; t < length; t += kWarps) {
        const int index = t / a.page_size, page = a.table[b * a.table_stride + index];
        if ((unsigned)page >= (unsigned)a.pages) {
            atomicOr(a.err, kErrPageRange);
            continue;
        }
        const int64_t token = t - index * a.page_size;
        float f[PER], dot = 0.0f;
        load_values<PER>(a.k.data + page * a.k.page + token * a.k.token + kv * a.k.head, bytes, lane, f);
#pragma unroll
        for (int j = 0; j < PER; ++j) dot = fmaf(q[j], f[j], dot);
        const float s = warp_sum(dot) * ks, top = fmaxf(m, s), base = top == -INFINITY ? 0.0f : top;
        const float keep = exp2f(m - base), p = exp2f(s - base);
        load_values<PER>(a.v.data + page * a.v.page + token * a.v.token + kv * a.v.head, bytes, lane, f);
#pragma unroll
        for (int j = 0; j < PER; ++j) o[j] = fmaf(p, f[j], o[j] * keep);
        l = fmaf(l, keep, p);
        m = top;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) s_o[warp][lane * PER + j] = o[j];
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kWarps; ++w) total += s_l[w] * exp2f(s_m[w] - base);
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float sum = 0.0f;
        for (int w = 0; w < kWarps; ++w) sum += s_o[w][d] * exp2f(s_m[w] - base);
        const float v = total == 0.0f ? 0.0f : sum / total * vs;
        a.out[((int64_t)b * a.heads + head) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[(int64_t)b * a.heads + head] = total == 0.0f ? -INFINITY : (base + log2f(total)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attn_decode(const DecodeArgs& a, int head_dim, int, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)a.heads, (unsigned)a.B);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    switch (head_dim) {
        case 64: return cudaLaunchKernelEx(&cfg, attn_decode_kernel<64>, a);
        case 128: return cudaLaunchKernelEx(&cfg, attn_decode_kernel<128>, a);
        case 256: return cudaLaunchKernelEx(&cfg, attn_decode_kernel<256>, a);
    }
    return cudaErrorInvalidValue;
}

cudaError_t attn_decode_set_attributes() { return cudaSuccess; }
size_t attn_decode_counters(int) { return 64; }
size_t attn_decode_parts(int, int) { return 64; }

}  // namespace arf
