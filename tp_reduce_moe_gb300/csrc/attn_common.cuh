// attn_common.cuh -- what the attention entry points' host side and kernels
// share: the view of the cache, the kernels' arguments, 8-bit values.
#pragma once

#include "arf_common.cuh"

namespace arf {

constexpr unsigned kErrPageRange = 0x8u;
constexpr unsigned kErrSlotRange = 0x10u;
constexpr unsigned kErrLengthRange = 0x20u;

constexpr int kMaxHeadDim = 256;

// Keys or values of a paged cache: element (page, token, head, d) at
// data + (page * page_stride + token * token_stride + head * head_stride + d) * size.
struct CacheView {
    uint8_t* data;
    int64_t page, token, head;  // strides in bytes
    const float* scale;         // e4m3: [kv_heads]; bf16: nullptr
};

// A rotary table in device memory, written once.
struct RopeTable {
    uint64_t turns[kMaxHeadDim / 2];  // freq / (2 pi), turns a position, less the whole ones, in units of 2^-64
    int32_t axis[kMaxHeadDim / 2];
};

struct AppendArgs {
    const uint16_t* qkv;       // bf16 [T, (heads + 2 kv) D]
    const int32_t* positions;  // [axes, T]
    const int32_t* slots;      // [T]
    const RopeTable* rope;
    uint16_t* q;  // bf16 [T, heads D]
    CacheView k, v;
    unsigned* err;
    int64_t slot_count;  // pages * page_size
    int T, heads, kv, D, page_size;
    int rot, interleaved;
};

struct DecodeArgs {
    const uint16_t* q;  // bf16 [B, heads D]
    const int32_t* table;
    const int32_t* lengths;
    CacheView k, v;
    uint16_t* out;  // bf16 [B, heads D]
    float* lse;     // [B, heads] or nullptr
    unsigned* err;
    unsigned* count;  // arrival counters, zero between calls
    float* part;      // parts of rows split over several warps and CTAs
    int64_t table_stride;
    int64_t most;  // longest length that the page table holds
    int pages;
    int B, heads, kv, page_size;
    int shared, per_head, groups, rows_of_group;  // query heads of a key-value head, their groups, all groups, heads of one
    unsigned page_mul;  // token / page_size == token * page_mul >> (31 + page_shift) for tokens below 2^31
    int page_shift;
    int window;    // 0: none
    float scale;   // of the scores, times log2(e)
};

// Length of sequence b, clamped to what the page table holds.
__device__ __forceinline__ int checked_length(const DecodeArgs& a, int b, bool report) {
    const int n = a.lengths[b];
    if (n >= 0 && n <= a.most) return n;
    if (report) atomicOr(a.err, kErrLengthRange);
    return n < 0 ? 0 : (int)a.most;
}

// Two e4m3 values as two halves (exact), the low byte's in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// Two values rounded to e4m3 (nearest even, larger ones to 448, NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// Launches go out with programmatic dependent launch, always: it only moves the launch under the end of the kernel before.
cudaError_t launch_attn_append(const AppendArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_attn_decode(const DecodeArgs& a, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t attn_decode_set_attributes();
size_t attn_decode_counters(int num_sms);               // words
size_t attn_decode_parts(int num_sms, int head_dim);    // floats

}  // namespace arf
