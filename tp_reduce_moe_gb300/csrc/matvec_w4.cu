// matvec_w4.cu -- products of a few tokens with a 4-bit weight matrix.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[t, k]
//
// Weight rows are dealt evenly over the SMs; the list of a CTA's tiles' segments
// is cut into sixteen equal ranges, one per warp.  More than eight tokens take the
// CTA's rows again for every eight, from L2 (sixteen columns at a time left no
// registers and, of long rows, a quarter of the activations staged at once: 60 us
// for 13 tokens with 18431 rows of 8192 instead of 49).
//
// One token: 36864 x 7168 in groups of 64 takes 25.9 us, 0.80 of the copy rate;
// 7168 x 2048 takes 4.2 us, launch and two trips to memory.  13 tokens: 49.5 us,
// 0.25, bound by the reads of the activations from shared memory, 512 bytes per
// eight columns of weights a lane, and by staging them four times.
#include "moe_common.cuh"

namespace arf {
namespace {

// Blocks of rows and tokens in the order (rows, tokens).
template <int GS>
struct Matvec {
    static constexpr bool kPairs = false;
    const MatvecArgs& a;
    int r0, r1;
    int block, chunk;  // rows and tokens per job, at most
    struct Job {
        int count;
        int row, rows, token, tokens;
    };
    struct Tile {
        int n, tokens, row, expert;
        int token;
    };
    __device__ void at(Job& j, int row, int token) const {
        j.row = row;
        j.rows = min(block, r1 - row);
        j.count = (j.rows + 15) >> 4;
        j.token = token;
        j.tokens = min(chunk, a.T - token);
    }
    __device__ Tile tile(const Job& j, int i) const {
        Tile t;
        t.n = max(0, min(16, j.rows - 16 * i));
        t.tokens = j.tokens;
        t.row = j.row + 16 * i;
        t.expert = 0;
        t.token = j.token;
        return t;
    }
    __device__ bool first(Job& j) const {
        if (r0 >= r1) return false;
        at(j, r0, 0);
        return true;
    }
    __device__ bool next(Job& j) const {
        if (j.token + j.tokens < a.T) {
            at(j, j.row, j.token + j.tokens);
            return true;
        }
        if (j.row + j.rows >= r1) return false;
        at(j, j.row + j.rows, 0);
        return true;
    }
    __device__ const uint16_t* scales(const Tile& t) const { return a.s + (int64_t)t.row * (a.K / (128 / GS)); }
    __device__ int second() const { return 8; }
    __device__ void lost() const {}
    __device__ const uint16_t* x(const Tile& t, int i) const { return a.x + (int64_t)(t.token + i) * a.K; }
    __device__ int staged_key(const Job& j) const { return j.token; }
    __device__ int staged(const Job& j) const { return j.tokens; }
    __device__ const uint16_t* staged_x(const Job& j, int i) const { return a.x + (int64_t)(j.token + i) * a.K; }
    __device__ int column(const Tile&, int i) const { return i; }
    __device__ void store(const Tile& t, int pair, int token, float first, float second) const {
        const int64_t o = (int64_t)(t.token + token) * a.N + t.row + pair;
        if (a.out_f32) {
            float* out = reinterpret_cast<float*>(a.out) + o;
            out[0] = first;
            if (pair + 8 < t.n) out[8] = second;
        } else {
            uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + o;
            out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(first));
            if (pair + 8 < t.n) out[8] = __bfloat16_as_ushort(__float2bfloat16_rn(second));
        }
    }
};

template <int GS>
__global__ void __launch_bounds__(kMvThreads, 1) matvec_w4_kernel(const __grid_constant__ MatvecArgs a, const __grid_constant__ Weights weights, const __grid_constant__ ProductPlan plan) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SlotRing::init(smem_addr(smem) + warp_index() * kMaxSlots * 8, kMaxSlots, Scales<GS>::arrivals(plan.piece), threadIdx.x & 31);
    if (threadIdx.x == 0) prefetch_maps(weights, plan.shape.row_bytes >= kSegment, plan.piece == 0);
    pdl_wait();  // no global memory access before this point
    pdl_trigger();
    const Share rows(a.N);
    Matvec<GS> jobs{a, rows.first, rows.last, 0, 8};
    jobs.block = 16 * kJobTiles<GS>;
    run_product<GS>(jobs, weights, smem, plan, a.K);
}

template <int GS>
cudaError_t launch(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    Weights weights{};
    const int grid = a.N < num_sms ? a.N : num_sms;
    const ProductPlan plan = plan_product<GS>(a.K, a.T < 8 ? a.T : 8, 8, ((a.N + grid - 1) / grid + 15) / 16, 0);
    const cudaError_t e = describe_weights(&weights, {a.q, a.s, a.N, Fmt<GS>::row_bytes(a.K), Fmt<GS>::scales(a.K), GS, 0, a.N / grid});
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = (size_t)plan.smem;
    cfg.stream = stream;
    // always: it only moves the launch and the barriers' initialisation under the end of the kernel before
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, matvec_w4_kernel<GS>, a, weights, plan);
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
    cudaError_t e = cudaFuncSetAttribute(matvec_w4_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(matvec_w4_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(matvec_w4_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    return e;
}

}  // namespace arf
