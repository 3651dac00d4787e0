// matvec_w4.cu -- products of a few tokens with a 4-bit weight matrix.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[t, k]
//
// Weight rows are dealt evenly over the SMs; the list of a CTA's tiles' segments
// is cut into sixteen equal ranges, one per warp.  More than eight tokens make
// groups of up to eight, each with its share of the SMs; neighbouring CTAs take
// the same rows for them, once from memory and else from L2.  (13 tokens with
// 18431 rows of 8192: 42 us; one CTA for one group after the other 49, staging the
// activations twice as often; sixteen columns at a time 60: no registers left.)
//
// One token: 36864 x 7168 in groups of 64 takes 26.5 us, 0.78 of the copy rate;
// 7168 x 2048 takes 4.3 us, launch and two trips to memory.  Of 18431 x 8192 two
// tokens take 19.6 us (0.64), eight 25.6 (0.49), sixteen 41, 32 91 and 64 178: each
// group of eight takes the codes out again, and from some sixteen tokens on the
// same matrix in bf16, read once in 44 us, is the better one.  The 13 tokens' 42 us
// are 0.30, bound by the reads of the activations from shared memory, 512 bytes
// per eight columns of weights a lane, twice the weights' own, and by staging them.
#include "moe_common.cuh"

namespace arf {
namespace {

// A range of rows for a group of tokens.
template <int GS>
struct Matvec {
    static constexpr bool kPairs = false;
    const MatvecArgs& a;
    int r0, r1;
    int token, tokens;
    struct Job {
        int count;
        int row, rows;
    };
    struct Tile {
        int n, tokens, row, expert;
    };
    __device__ void at(Job& j, int row) const {
        j.row = row;
        j.rows = min(16 * kJobTiles<GS>, r1 - row);
        j.count = (j.rows + 15) >> 4;
    }
    __device__ Tile tile(const Job& j, int i) const { return Tile{min(16, j.rows - 16 * i), tokens, j.row + 16 * i, 0}; }
    __device__ bool first(Job& j) const {
        if (r0 >= r1) return false;
        at(j, r0);
        return true;
    }
    __device__ bool next(Job& j) const {
        if (j.row + j.rows >= r1) return false;
        at(j, j.row + j.rows);
        return true;
    }
    __device__ const uint16_t* scales(const Tile& t) const { return a.s + (int64_t)t.row * (a.K / (128 / GS)); }
    __device__ int second() const { return 8; }
    __device__ void lost() const {}  // (there is no handle whose error word could say so)
    __device__ static constexpr unsigned long long stall() { return 0; }
    __device__ const uint16_t* x(const Tile&, int i) const { return a.x + (int64_t)(token + i) * a.K; }
    __device__ int staged_key(const Job&) const { return 0; }
    __device__ int staged(const Job&) const { return tokens; }
    __device__ const uint16_t* staged_x(const Job&, int i) const { return a.x + (int64_t)(token + i) * a.K; }
    __device__ int column(const Tile&, int i) const { return i; }
    __device__ void store(const Tile& t, int pair, int i, float first, float second) const {
        const int64_t o = (int64_t)(token + i) * a.N + t.row + pair;
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
__global__ void __launch_bounds__(kMvThreads, 1) matvec_w4_kernel(const __grid_constant__ MatvecArgs a, const __grid_constant__ Weights weights,
                                                                     const __grid_constant__ ProductPlan plan, int groups) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SlotRing::init(smem_addr(smem) + warp_index() * kMaxSlots * 8, Scales<GS>::arrivals(plan.piece), threadIdx.x & 31);
    if (threadIdx.x == 0) prefetch_maps(weights, plan.shape.row_bytes >= kSegment, plan.piece == 0);
    pdl_wait();  // no global memory access before this point
    pdl_trigger();
    // CTAs that follow each other take the same rows, for one group of tokens after the other.
    const int turn = blockIdx.x - quotient(blockIdx.x, groups) * groups;
    const Share rows(a.N, quotient(gridDim.x, groups), quotient(blockIdx.x, groups));
    const int each = quotient(a.T + groups - 1, groups);
    const Matvec<GS> jobs{a, rows.first, rows.last, turn * each, min(each, a.T - turn * each)};
    run_product<GS>(jobs, weights, smem, plan, a.K);
}

template <int GS>
cudaError_t launch(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    Weights weights{};
    const int groups = (a.T + 7) / 8, tokens = (a.T + groups - 1) / groups;
    const int most = num_sms > groups ? num_sms / groups : 1, parts = a.N < most ? a.N : most;  // of the rows
    const ProductPlan plan = plan_product<GS>(a.K, tokens, 8, ((a.N + parts - 1) / parts + 15) / 16, 0);
    const cudaError_t e = describe_weights(&weights, {a.q, a.s, a.N, Fmt<GS>::row_bytes(a.K), Fmt<GS>::scales(a.K), GS, 0, a.N / parts});
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(parts * groups));
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = (size_t)plan.smem;
    cfg.stream = stream;
    // always: it only moves the launch and the barriers' initialisation under the end of the kernel before
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, matvec_w4_kernel<GS>, a, weights, plan, groups);
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
