// moe_api.cu -- C entry points of the few-token MoE layer and the 4-bit
// product (declared in include/arfuse.h): argument checks, the handle, the
// launches.  Nothing here allocates or synchronises on the call path.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <new>

#include "arf_check.h"
#include "arfuse.h"
#include "moe_common.cuh"

static_assert(arf::kMoeMaxTokens == AR_MAX_MOE_TOKENS && arf::kMoeMaxGroups == AR_MAX_MOE_GROUPS &&
                  arf::kMaxTopK == AR_MAX_TOP_K && arf::kMoeMaxExperts == AR_MAX_MOE_EXPERTS &&
                  arf::kErrExpertRange == AR_DEVERR_EXPERT_RANGE,
              "the kernels' limits are the header's");

struct ar_moe {
    int device;
    int E, S, K, H, I;  // routed experts, shared experts, routed slots, hidden, intermediate
    int64_t max_tokens;
    unsigned flags;
    int num_sms;
    unsigned long long stall_ns[2];  // failure injection, first and second product
    uint8_t* d_mem;  // everything below
    unsigned* d_err;
    unsigned* d_count;  // [token groups], zero between calls
    float2* d_logits;   // [max_tokens, E]
    uint16_t* d_act;    // [max_tokens * slots, 2, I]
};

namespace {

using arf::aligned;
using arf::overlap;
using arf::Range;
using arf::range_of;

int slots(const ar_moe* m) { return m->K + m->S; }

// What every call on a handle checks first.
ar_status check_call(const ar_moe* m, int64_t T) {
    if (!m || T < 0) return AR_ERR_INVALID_ARG;
    if (T > m->max_tokens) return AR_ERR_CAPACITY;
    return AR_OK;
}

ar_status check_device(const ar_moe* m) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return AR_ERR_CUDA;
    return cur == m->device ? AR_OK : AR_ERR_INVALID_ARG;
}

ar_status launched(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    (void)cudaGetLastError();
    return AR_ERR_CUDA;
}

bool valid_group(int group) { return group == 32 || group == 64 || group == 128; }

ar_status experts(ar_moe* m, const void* x, const int32_t* ids, const float* weights, const void* w13, const void* s13,
                  const void* w2, const void* s2, int group, int64_t T, void* out, void* stream) {
    ar_status st = check_call(m, T);
    if (st != AR_OK) return st;
    if (m->I == 0) return AR_ERR_UNSUPPORTED;
    if (group != 0 && (!valid_group(group) || m->H % group != 0 || m->I % group != 0)) return AR_ERR_UNSUPPORTED;
    if (T == 0) return AR_OK;
    if (!x || !ids || !weights || !w13 || !w2 || !out || (group != 0 && (!s13 || !s2))) return AR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(out, 16) || !aligned(ids, 4) ||
        !aligned(weights, 4) || !aligned(s13, 16) || !aligned(s2, 16))
        return AR_ERR_ALIGNMENT;
    const int64_t E = m->E + m->S, values = E * m->H * m->I, n = T * slots(m);
    const Range r = range_of(out, T * m->H * 2);
    if (overlap(r, range_of(x, T * m->H * 2)) || overlap(r, range_of(ids, n * 4)) || overlap(r, range_of(weights, n * 4)) ||
        overlap(r, range_of(w13, group ? values : values * 4)) || overlap(r, range_of(w2, group ? values / 2 : values * 2)))
        return AR_ERR_INVALID_ARG;
    if (group && (overlap(r, range_of(s13, values / group * 4)) || overlap(r, range_of(s2, values / group * 2))))
        return AR_ERR_INVALID_ARG;
    if (m->flags & AR_WS_DRY_RUN) return AR_VALIDATED;
    st = check_device(m);
    if (st != AR_OK) return st;
    arf::ExpertsArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = static_cast<const uint16_t*>(x);
    a.ids = ids;
    a.weights = weights;
    a.w13 = static_cast<const uint8_t*>(w13);
    a.w2 = static_cast<const uint8_t*>(w2);
    a.s13 = static_cast<const uint16_t*>(s13);
    a.s2 = static_cast<const uint16_t*>(s2);
    a.act = m->d_act;
    a.out = static_cast<uint16_t*>(out);
    a.err = m->d_err;
    a.stall_ns[0] = m->stall_ns[0];
    a.stall_ns[1] = m->stall_ns[1];
    a.T = (int)T;
    a.K = slots(m);
    a.E = (int)E;
    a.H = m->H;
    a.I = m->I;
    return launched(arf::launch_moe_experts(a, group, m->num_sms, static_cast<cudaStream_t>(stream),
                                            (m->flags & AR_WS_PDL) != 0));
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// SMs per device, and whether the kernels' attributes are set there (0: not yet).
constexpr int kMaxDevices = 64;
std::atomic<int> g_matvec_sms[kMaxDevices];

}  // namespace

extern "C" {

ar_status ar_moe_create(int device, int experts, int shared, int top_k, int hidden, int inter, int64_t max_tokens,
                        unsigned flags, ar_moe** out) {
    if (!out) return AR_ERR_INVALID_ARG;
    *out = nullptr;
    if (max_tokens < 1 || experts < 1 || shared < 0 || top_k < 1 || top_k > experts || inter < 0) return AR_ERR_INVALID_ARG;
    if ((flags & ~(AR_WS_DRY_RUN | AR_WS_PDL)) != 0) return AR_ERR_INVALID_ARG;
    if (hidden < 8) return AR_ERR_UNSUPPORTED;
    if (hidden % 8 != 0 || inter % 8 != 0) return AR_ERR_ALIGNMENT;
    if (experts > AR_MAX_MOE_EXPERTS || shared > AR_MAX_MOE_EXPERTS - experts || top_k > AR_MAX_TOP_K ||
        shared > AR_MAX_TOP_K - top_k || hidden > AR_MAX_HIDDEN || inter > AR_MAX_HIDDEN || max_tokens > AR_MAX_MOE_TOKENS)
        return AR_ERR_UNSUPPORTED;
    ar_moe* m = new (std::nothrow) ar_moe();
    if (!m) return AR_ERR_CUDA;
    m->device = device;
    m->E = experts;
    m->S = shared;
    m->K = top_k;
    m->H = hidden;
    m->I = inter;
    m->max_tokens = max_tokens;
    m->flags = flags;
    if (flags & AR_WS_DRY_RUN) {
        *out = m;
        return AR_OK;
    }
    const size_t logits = round_up((size_t)max_tokens * experts * sizeof(float2));
    const size_t act = round_up((size_t)max_tokens * (top_k + shared) * 2 * inter * 2);
    int prev = -1, major = 0;
    ar_status st = AR_ERR_CUDA;
    if (cudaGetDevice(&prev) == cudaSuccess && cudaSetDevice(device) == cudaSuccess &&
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) == cudaSuccess &&
        cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess) {
        if (major < 10)
            st = AR_ERR_UNSUPPORTED;
        else if (arf::moe_route_set_attributes() == cudaSuccess && arf::moe_experts_set_attributes() == cudaSuccess &&
                 cudaMalloc(&m->d_mem, 512 + logits + act) == cudaSuccess && cudaMemset(m->d_mem, 0, 512) == cudaSuccess &&
                 cudaDeviceSynchronize() == cudaSuccess)
            st = AR_OK;
    }
    if (st != AR_OK) {
        (void)cudaGetLastError();
        if (m->d_mem) (void)cudaFree(m->d_mem);
        if (prev >= 0) (void)cudaSetDevice(prev);
        delete m;
        return st;
    }
    (void)cudaSetDevice(prev);
    m->d_err = reinterpret_cast<unsigned*>(m->d_mem);
    m->d_count = reinterpret_cast<unsigned*>(m->d_mem + 256);
    m->d_logits = reinterpret_cast<float2*>(m->d_mem + 512);
    m->d_act = reinterpret_cast<uint16_t*>(m->d_mem + 512 + logits);
    *out = m;
    return AR_OK;
}

ar_status ar_moe_destroy(ar_moe* m) {
    if (!m) return AR_OK;
    ar_status st = AR_OK;
    if (m->d_mem) {
        int prev = -1;
        (void)cudaGetDevice(&prev);
        if (cudaSetDevice(m->device) != cudaSuccess || cudaFree(m->d_mem) != cudaSuccess) {
            (void)cudaGetLastError();
            st = AR_ERR_CUDA;
        }
        if (prev >= 0) (void)cudaSetDevice(prev);
    }
    delete m;
    return st;
}

ar_status ar_moe_device_error(ar_moe* m, int* code) {
    if (!m || !code) return AR_ERR_INVALID_ARG;
    *code = 0;
    if (m->flags & AR_WS_DRY_RUN) return AR_OK;
    int prev = -1;
    (void)cudaGetDevice(&prev);
    unsigned v = 0;
    ar_status st = AR_OK;
    if (cudaSetDevice(m->device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&v, m->d_err, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(m->d_err, 0, sizeof v) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        (void)cudaGetLastError();
        st = AR_ERR_CUDA;
    }
    if (prev >= 0) (void)cudaSetDevice(prev);
    if (st != AR_OK) return st;
    *code = (int)v;
    return v ? AR_ERR_DEVICE_CHECK : AR_OK;
}

ar_status ar_moe_inject_wait_timeout(ar_moe* m, int product, int64_t limit_ns) {
    if (!m || product < 1 || product > 2) return AR_ERR_INVALID_ARG;
    if (limit_ns < 0 || limit_ns > (int64_t)arf::kWaitLimitNs) return AR_ERR_INVALID_ARG;
    m->stall_ns[product - 1] = (unsigned long long)limit_ns;
    return AR_OK;
}

ar_status ar_moe_route(ar_moe* m, const void* x, const void* gate, const float* bias, int scoring, int renorm, float scale,
                       int n_group, int topk_group, int64_t T, int32_t* ids, float* weights, void* stream) {
    ar_status st = check_call(m, T);
    if (st != AR_OK) return st;
    const int function = scoring & ~AR_MOE_GROUP_MAX;
    if ((function != AR_MOE_SOFTMAX && function != AR_MOE_SIGMOID) || (renorm != 0 && renorm != 1)) return AR_ERR_INVALID_ARG;
    if (n_group < 1 || n_group > AR_MAX_MOE_GROUPS || m->E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
        (n_group > 1 && m->E / n_group < 2) || topk_group * (m->E / n_group) < m->K)
        return AR_ERR_INVALID_ARG;
    if (T == 0) return AR_OK;
    if (!x || !gate || !ids || !weights) return AR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return AR_ERR_ALIGNMENT;
    const Range out[2] = {range_of(ids, T * slots(m) * 4), range_of(weights, T * slots(m) * 4)};
    if (overlap(out[0], out[1])) return AR_ERR_INVALID_ARG;
    for (const Range& r : out)
        if (overlap(r, range_of(x, T * m->H * 2)) || overlap(r, range_of(gate, (int64_t)m->E * m->H * 2)) ||
            (bias && overlap(r, range_of(bias, (int64_t)m->E * 4))))
            return AR_ERR_INVALID_ARG;
    if (m->flags & AR_WS_DRY_RUN) return AR_VALIDATED;
    st = check_device(m);
    if (st != AR_OK) return st;
    arf::RouteArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = static_cast<const uint16_t*>(x);
    a.gate = static_cast<const uint16_t*>(gate);
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.logits = m->d_logits;
    a.count = m->d_count;
    a.T = (int)T;
    a.H = m->H;
    a.E = m->E;
    a.K = m->K;
    a.shared = m->S;
    a.sigmoid = function == AR_MOE_SIGMOID;
    a.group_max = (scoring & AR_MOE_GROUP_MAX) != 0;
    a.renorm = renorm;
    a.n_group = n_group;
    a.topk_group = topk_group;
    a.scale = scale;
    return launched(arf::launch_moe_route(a, static_cast<cudaStream_t>(stream), (m->flags & AR_WS_PDL) != 0));
}

ar_status ar_moe_experts(ar_moe* m, const void* x, const int32_t* ids, const float* weights, const void* w13, const void* w2,
                         int64_t T, void* out, void* stream) {
    return experts(m, x, ids, weights, w13, nullptr, w2, nullptr, 0, T, out, stream);
}

ar_status ar_moe_experts_w4(ar_moe* m, const void* x, const int32_t* ids, const float* weights, const void* q13,
                            const void* s13, const void* q2, const void* s2, int group, int64_t T, void* out, void* stream) {
    if (!valid_group(group)) return m ? AR_ERR_UNSUPPORTED : AR_ERR_INVALID_ARG;
    return experts(m, x, ids, weights, q13, s13, q2, s2, group, T, out, stream);
}

ar_status ar_matvec_w4(const void* x, const void* q, const void* s, int group, int64_t T, int64_t N, int64_t K, void* out,
                       int out_is_fp32, void* stream) {
    if (T < 0 || N < 0 || K < 0 || (out_is_fp32 != 0 && out_is_fp32 != 1)) return AR_ERR_INVALID_ARG;
    if (!valid_group(group) || N < 1 || N > AR_MAX_MATVEC_ROWS || K < group || K > AR_MAX_MATVEC_COLS || K % group != 0)
        return AR_ERR_UNSUPPORTED;
    if (T > AR_MAX_MOE_TOKENS) return AR_ERR_CAPACITY;
    if (T == 0) return AR_OK;
    if (!x || !q || !s || !out) return AR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 16) || !aligned(out, 16)) return AR_ERR_ALIGNMENT;
    const Range r = range_of(out, T * N * (out_is_fp32 ? 4 : 2));
    if (overlap(r, range_of(x, T * K * 2)) || overlap(r, range_of(q, N * (K / 2))) || overlap(r, range_of(s, N * (K / group) * 2)))
        return AR_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return AR_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return AR_ERR_UNSUPPORTED;
    int sms = g_matvec_sms[dev].load(std::memory_order_acquire);
    if (sms == 0) {  // two threads may both do this: it sets the same values
        int major = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return launched(cudaErrorUnknown);
        if (major < 10) return AR_ERR_UNSUPPORTED;
        if (arf::matvec_w4_set_attributes() != cudaSuccess) return launched(cudaErrorUnknown);
        g_matvec_sms[dev].store(sms, std::memory_order_release);
    }
    arf::MatvecArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = static_cast<const uint16_t*>(x);
    a.q = static_cast<const uint8_t*>(q);
    a.s = static_cast<const uint16_t*>(s);
    a.out = out;
    a.T = (int)T;
    a.N = (int)N;
    a.K = (int)K;
    a.out_f32 = out_is_fp32;
    return launched(arf::launch_matvec_w4(a, group, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
