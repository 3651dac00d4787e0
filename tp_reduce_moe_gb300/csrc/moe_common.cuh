// moe_common.cuh -- what the few-token weight-streaming kernels share
// (moe_experts.cu, matvec_w4.cu): parameters, the weight formats, the
// per-warp copy ring and the matrix instruction.
//
// Products of a few tokens with a large weight matrix read every weight once
// and use it a handful of times, so the time is the weights' bytes over the
// memory bandwidth.  One CTA per SM holds sixteen warps; each warp streams its
// own share of the weights through a private ring in shared memory, filled by
// tensor copies (TMA) of sixteen rows by 256 bytes, and multiplies them with
// mma.sync, weight rows as the 16-row operand and tokens as the 8-column one.
// (Tried before: cp.async from the same warps, 5.9 TB/s and ten instructions per
// KB, and plain loads issued behind it return behind it; bulk copies of single
// 256-byte row segments, 7 TB/s but issued lane by lane, 14 instructions each;
// tensor copies of eight rows by 128 bytes, four times as many to issue.)
// A kilobyte of weights takes the memory 44 cycles to deliver to an SM; the
// matrix instructions for it take 4 (bf16) to 16 (4-bit) on each of its four
// schedulers, and taking the codes out as long again.  bf16 weights come at the
// memory's rate, 4-bit ones at 50 to 80 % of it for up to eight tokens: no pipe is
// full then (issue slots 33 to 54 %, integer pipe 34 to 53), four warps a scheduler
// wait for their own dependent instructions, one of them ready on average.  So
// fewer instructions help, and more independent ones would.  More than eight tokens
// of one expert or matrix take the weights, and the codes out of them, once for
// every eight (four in the experts' second product): 30 % for 13 tokens, 7 % for
// 64.  A tcgen05 tile of
// 128 rows would need all its operands in shared memory, the 4-bit codes expanded
// there first, and pay in granularity: at one token an SM owns about 27 rows of
// the first product.
#pragma once

#include <cuda.h>

#include "arf_common.cuh"

namespace arf {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;  // routed + shared
constexpr int kMoeMaxGroups = 32;
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
    int sigmoid, renorm, n_group, topk_group, group_max;
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
    // Failure injection (0 = off): how long the warps of the first and of the second
    // product wait for a copy that is never made before they give up.
    unsigned long long stall_ns[2];
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
// A step is 64 bytes of a row: 32 bf16 values or 128 4-bit codes; a segment is
// four steps.  GS: scale groups per step (0: bf16 weights).
constexpr int kSegment = 256;
template <int GS>
struct Fmt {
    static constexpr bool kW4 = GS > 0;
    static constexpr int kStepK = kW4 ? 128 : 32;
    static constexpr int kSegK = 4 * kStepK;
    __host__ __device__ static int row_bytes(int k) { return kW4 ? k / 2 : k * 2; }
    __host__ __device__ static int scales(int k) { return kW4 ? k / (128 / (GS ? GS : 1)) : 0; }
};

// c += A (16 x 16, row-major fragments) * B (16 x 8): bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_bf16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = c + A * B
__device__ __forceinline__ void mma_bf16_from(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

template <int WORDS>
__device__ __forceinline__ void lds(uint32_t (&v)[WORDS], uint32_t a) {
    if constexpr (WORDS == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
    if constexpr (WORDS == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}
// 16 bytes that an earlier grid wrote, perhaps one that still ran when this one
// began: not the read-only path, which need not see that.
__device__ __forceinline__ uint4 ld_coherent16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_u16(const uint16_t* p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A value that is the same in all lanes, in a form that the compiler knows to
// be (branches and addresses made of it are the warp's, not the lanes').
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ int warp_index() { return uniform((int)(threadIdx.x >> 5)); }

// a / b for 0 <= a <= 2^24, 0 < b, a / b < 2^20: in floating point off by one at most.
__device__ __forceinline__ int quotient(int a, int b) {
    int q = (int)__fdividef((float)a, (float)b);
    q -= q * b > a;
    q += a - q * b >= b;
    return q;
}

// The pair of a tile that lane row g (of the eight) stands for: an order in which
// reads of a quarter (16 bytes a lane), half (8) or whole warp (4) meet every
// bank of the swizzled rows once.
template <int GS>
__host__ __device__ constexpr int pair_of_row(int g) {
    return GS == 1 ? (g >> 1 | (g & 1) << 2) : GS == 2 ? ((g & 3) << 1 | g >> 2) : g;
}

// --------------------------------------------------------------------- ring
// A tile is sixteen rows, two by two in a lane of the matrix instruction: rows i
// and i + 8 of a range of rows ("rows"), or a gate row and its up row, eight of
// each ("pairs").
//
// A ring slot holds a segment of a tile: of its first 128 bytes the eight first
// rows, then the eight second ones; then the same of the next 128 bytes; swizzled
// by the copy: the 16-byte chunk c of row g lies at place c ^ g of the row's
// eight.  All of it is one tensor copy (with four copies of eight rows by 128
// bytes 36864 rows of 7168 4-bit weights took 29.9 instead of 25.6 us).  What lies behind the end
// of the rows is zero in 128 bytes that begin before it; 128 bytes that begin
// behind it are not copied.  Rows that are not the tile's may be copied and are
// not used.  Every slot has its mbarrier; the warp that fills it is the one that
// reads it, and refills it at once.
constexpr int kBox = 128;
constexpr int kBoxBytes = 8 * kBox;
constexpr int kHalfAt = kBoxBytes;       // the second rows
constexpr int kNextAt = 2 * kBoxBytes;   // the next 128 bytes
constexpr int kSlotBytes = 4 * kBoxBytes;
constexpr int kMaxSlots = 2;

// A weight matrix for the copies.  A segment of 256 bytes of a whole tile takes
// `full`: rows of 128 bytes, one dimension the 128 bytes' index in the row.  The
// rest takes 128 bytes at a time: of 16, 8 or 4 rows ("rows"), or of a whole tile
// ("pairs", the first).  scales: of a segment of a tile, where rows have a multiple
// of eight.
struct Weights {
    CUtensorMap full, part[3], scales;
};
// What there is to describe.
struct WeightRows {
    const void* q;
    const void* s;  // 4-bit: group scales, row_scales per row
    int64_t rows;   // in all
    int row_bytes, row_scales, group_steps;
    int inter;      // pairs: rows come as [experts][2][inter]; 0: rows
    int each;       // rows: fewest rows of a CTA (the others have one more)
};
cudaError_t describe_weights(Weights* w, const WeightRows& rows);

struct RowShape {
    int row_bytes, segments;
    __host__ static RowShape of(int bytes) { return RowShape{bytes, (bytes + kSegment - 1) / kSegment}; }
    __device__ __forceinline__ int bytes(int segment) const { return min(kSegment, row_bytes - segment * kSegment); }
};

// The `index`-th of `parts` ranges of `total` things (up to 2^24, 2^20 a part), dealt evenly, whole ones to each.
struct Share {
    int first, last;
    __device__ __forceinline__ Share(unsigned total, unsigned parts, unsigned index) {
        const unsigned each = quotient(total, parts), rest = total - each * parts;
        first = index * each + min(index, rest);
        last = first + each + (index < rest);
    }
};

__device__ __forceinline__ void copy_tensor(uint32_t to, const CUtensorMap& map, uint32_t bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(to),
                 "l"(&map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void copy_tensor(uint32_t to, const CUtensorMap& map, uint32_t bar, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
                 "l"(&map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void copy_tensor(uint32_t to, const CUtensorMap& map, uint32_t bar, int x, int y, int z, int u) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
                 "l"(&map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void copy_tensor(uint32_t to, const CUtensorMap& map, uint32_t bar, int x, int y, int z, int u, int v) {
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(to),
                 "l"(&map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
                 : "memory");
}
// By one thread, ahead of the first copy: the maps come from memory otherwise.
__device__ __forceinline__ void prefetch_maps(const Weights& w, bool full, bool scales) {
    if (full) asm volatile("prefetch.tensormap [%0];" ::"l"(&w.full) : "memory");
    if (scales) asm volatile("prefetch.tensormap [%0];" ::"l"(&w.scales) : "memory");
}

// The thread's ordinary accesses to shared memory before it come before what
// asynchronous copies do to it that a barrier orders behind it: the barrier alone
// does not order the two kinds.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Multiples of 16 bytes at such addresses.
__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// A wait that sleeps in the instruction (the hint, in nanoseconds, is a limit)
// instead of polling: sixteen warps that poll take issue slots from those that
// have data.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(10000)
        : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t phase, unsigned long long limit_ns) {
    const unsigned long long t0 = global_timer_ns();
    for (unsigned it = 0; it < kWaitMaxIters; ++it) {
        if (mbar_sleep(bar, phase)) return true;
        if (global_timer_ns() - t0 > limit_ns) return false;
    }
    return false;
}

struct SlotRing {
    uint32_t slots, bars;  // shared addresses
    int two, step;         // whether there are two slots (else one), bytes between them
    uint32_t at;           // the next: counts fillings, later readings
    bool alive;            // the lane's waits have all ended in time

    __device__ __forceinline__ SlotRing(uint32_t slots, uint32_t bars, int n, int step)
        : slots(slots), bars(bars), two(n == 2), step(step), at(0), alive(true) {}
    __device__ __forceinline__ uint32_t slot() const { return slots + (at & two) * step; }
    __device__ __forceinline__ uint32_t bar() const { return bars + (at & two) * 8; }
    // The warp's barriers, before anything else; arrivals: of each, for each filling.
    __device__ static __forceinline__ void init(uint32_t bars, int arrivals, int lane) {
        if (lane < kMaxSlots) mbar_init(bars + lane * 8, arrivals);
        fence_mbar_init();
        __syncwarp();
    }
    // Copies `bytes` bytes of each row of a tile, from byte 256 * seg on, into the slot that was read last (or, at the start, one
    // after the other).  Rows: `n` of them from `row` on; pairs: from `row` of the expert's gate and up rows on.  more: bytes that
    // come with it.
    template <bool PAIRS>
    __device__ __forceinline__ void fill(const Weights& w, int row, int n, int expert, int seg, int bytes, int more) {
        const int x = seg * kSegment;
        const uint32_t slot = this->slot(), bar = this->bar();
        if (PAIRS || n > 8) {
            const bool wide = bytes > kBox;
            mbar_arrive_expect_tx(bar, (wide ? 4 * kBoxBytes : 2 * kBoxBytes) + more);
            if (bytes == kSegment) {
                if constexpr (PAIRS)
                    copy_tensor(slot, w.full, bar, 0, row, 0, 2 * seg, expert);
                else
                    copy_tensor(slot, w.full, bar, 0, row, 2 * seg);
            } else if constexpr (PAIRS) {
                copy_tensor(slot, w.part[0], bar, x, row, 0, expert);
                if (wide) copy_tensor(slot + kNextAt, w.part[0], bar, x + kBox, row, 0, expert);
            } else {
                copy_tensor(slot, w.part[0], bar, x, row);
                if (wide) copy_tensor(slot + kNextAt, w.part[0], bar, x + kBox, row);
            }
        } else {
            const bool wide = bytes > kBox, eight = n > 4;
            const CUtensorMap& map = w.part[eight ? 1 : 2];
            mbar_arrive_expect_tx(bar, (eight ? 8 : 4) * kBox * (wide ? 2 : 1) + more);
            copy_tensor(slot, map, bar, x, row);
            if (wide) copy_tensor(slot + kNextAt, map, bar, x + kBox, row);
        }
    }
    // Waits for the next slot.  A lane whose wait runs out (nothing but a lost copy
    // makes it) waits no more, and neither copies nor arrives any more: a barrier
    // whose phase has not ended takes no further arrivals, and the lost copy may
    // still land.  The warp learns of it at the end of a tile (ended).
    __device__ __forceinline__ void wait() {
        const uint32_t phase = at >> two & 1;
        if (!mbar_sleep(bar(), phase) && alive) alive = wait_long(bar(), phase, kWaitLimitNs);
    }
    // Whether any lane's wait has run out, for every lane the same: then all stop,
    // and what the warp has made of the slots is not a number.  (Asked at every wait
    // with a branch around the products it cost 2 to 5 %, behind them up to 4 %.)
    __device__ __forceinline__ bool ended(bool& more) {
        if (__all_sync(0xffffffffu, alive)) return false;
        alive = more = false;
        return true;
    }
    // Failure injection: instead of the first wait, one on the second slot's
    // barrier, before anything is copied there.
    __device__ __forceinline__ void lose(unsigned long long limit_ns, bool& more) {
        alive = wait_long(bars + 8, 0, limit_ns);
        ended(more);
    }
    // Where what comes with the slot lies, `bytes` bytes a slot.
    __device__ __forceinline__ uint32_t beside(uint32_t first, int bytes) const { return first + (at & two) * bytes; }
    __device__ __forceinline__ void next() { ++at; }
};

// ------------------------------------------------------------ products, bf16
// Of every box lane (g, t) = (lane / 4, lane % 4) takes the chunks 2t and 2t + 1
// of rows g (reads of eight lanes then meet every bank once), and so the values
// 16t .. 16t+15 of every 64 of column g, which come one segment ahead in
// registers.  A column that does not exist may repeat one that does.
//
// Part q of a segment: chunk 2t + q % 2 of box q / 2.
__device__ __forceinline__ uint4 load_column(const uint16_t* p, int left, int q, int t) {
    const int at = 64 * (q >> 1) + 16 * t + 8 * (q & 1);
    if (at >= left) return make_uint4(0, 0, 0, 0);
    return ld_coherent16(p + at);
}

// acc += (tile) * (columns), one segment of `bytes` bytes at `slot`.  load(q)
// replaces part q of the columns by a later segment's.
template <class Load>
__device__ __forceinline__ void multiply_bf16(float (&acc)[4], uint32_t slot, uint4 (&b)[4], int bytes, int lane, Load load) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t even = slot + g * kBox + ((2 * t) ^ g) * 16, odd = even ^ 16;
    float more[4] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (q < 2 || bytes > kBox) {
            uint32_t l[4], h[4];
            const uint32_t at = (q & 1 ? odd : even) + (q >> 1) * kNextAt;
            lds(l, at);
            lds(h, at + kHalfAt);
            mma_bf16(acc, l[0], h[0], l[1], h[1], b[q].x, b[q].y);
            mma_bf16(more, l[2], h[2], l[3], h[3], b[q].z, b[q].w);
        }
        load(q);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[u] += more[u];
}

// ----------------------------------------------------------- products, 4-bit
// 4-bit codes need no conversion.  A code in the low four bits of a bf16 is the
// subnormal number code * 2^-133, and one in bits 4-7 is code * 2^-129, since
// the smallest normal binade keeps the subnormals' spacing; the matrix
// instruction takes both exactly (measured: errors of 2^-23 of the sum of
// magnitudes, as for normal operands).  So one AND takes two codes out of a
// word, with one shift for half of them.  The activations are multiplied by a
// power of two that puts the largest of the step's 128 values of a token into
// [2^90, 2^91) (by 2^-4 of that where they meet codes in bits 4-7), so that all
// products are normal numbers; a factor per column brings a step's sum back.
// The columns' own sums times -8 are where the groups' sums start from.
// (Or-ing the codes into the mantissa of 128 and taking 136 off takes twice the
// instructions per code; e4m3 operands, which would take half the ANDs, are
// converted to half precision by the compiler first: 14 more per instruction.)
//
// A lane reads the codes that stand for 32 / GS consecutive values of every
// scale group of a step, in one word per eight, so that each matrix instruction
// stays within a group.
//
// In shared memory the values lie as the instructions take them: of every column
// the steps one after the other, 256 bytes each, in four parts (one per word of
// codes that a lane reads) of 16 bytes a lane: values (0, 4) (1, 5) (2, 6) (3,
// 7) of eight.  Columns are 64 bytes further apart than that, so that reads of
// two of them meet no bank twice.
// Behind the columns, for every column: of each segment the sums of its 4 * GS
// groups, then the factor (padded to 16 bytes).
template <int GS>
struct StagedView {
    static constexpr int kExtra = (4 * GS + 4) * 4;  // bytes per segment and column
    uint32_t values, extras;                         // shared addresses
    int stride, extra_stride;                        // between columns
    // `segments` of `columns` tokens: bytes in all
    __host__ __device__ static int bytes(int segments, int columns) { return columns * (segments * (1024 + kExtra) + 64); }
    __device__ __forceinline__ StagedView(uint32_t at, int segments, int columns) {
        values = at;
        stride = segments * 1024 + 64;
        extras = at + columns * stride;
        extra_stride = segments * kExtra;
    }
};

__device__ __forceinline__ void sts_f32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// One warp: a segment (512 bf16 values) of a token into column `col`; w[h]: of
// step 2 * h + lane / 16 the values 8 * (lane % 16) .. + 7 (zero behind the end of
// the row).
template <int GS>
__device__ __forceinline__ void stage_segment(const StagedView<GS>& v, int segment, int col, const uint4 (&w)[2], int lane) {
    // magnitudes as integers, two to a word: NaN is above everything
    constexpr unsigned kMagnitude = 0x7fff7fffu;
    unsigned big = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        big = __vmaxu2(__vmaxu2(__vmaxu2(w[h].x & kMagnitude, w[h].y & kMagnitude), __vmaxu2(w[h].z & kMagnitude, w[h].w & kMagnitude)), big);
    const unsigned top = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16)) >> 7;
    const bool bad = top > 227;  // infinite, undefined, or 2^101 and more: so is every sum it is in
    // 2^(up - 127) * 2^(top - 127) = 2^90, as far as bf16 goes and the factor does
    const unsigned up = bad ? 133u : max(min(344u - top, 254u), 133u);
    const uint32_t one = up << 7 | up << 23, sixteenth = (up - 4) << 7 | (up - 4) << 23;
    const int u = lane & 15;  // word of eight values: word i of lane t
    constexpr int kPer = 4 / GS, kLanes = 16 / GS;
    const int t = u / kPer % 4, i = u / (4 * kPer) * kPer + u % kPer;
    const uint32_t at = v.values + col * v.stride + segment * 1024 + (lane >> 4) * 256 + i * 64 + t * 16;
    const uint32_t extra = v.extras + col * v.extra_stride + segment * v.kExtra;
    const float minus8 = __uint_as_float((up - 130) << 23 | 0x80000000u);  // -8 * 2^(up - 127) * 2^-133
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 x = w[h];
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + h * 512), "r"(mul_bf16x2(__byte_perm(x.x, x.z, 0x5410), one)),
                     "r"(mul_bf16x2(__byte_perm(x.x, x.z, 0x7632), sixteenth)), "r"(mul_bf16x2(__byte_perm(x.y, x.w, 0x5410), one)),
                     "r"(mul_bf16x2(__byte_perm(x.y, x.w, 0x7632), sixteenth))
                     : "memory");
        // -8 * 2^-133 times the scaled values' sum, in each group
        float f[8];
        bf16x8_to_f32(x, f);
        float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (u % kLanes == 0) sts_f32(extra + ((2 * h + (lane >> 4)) * GS + u / kLanes) * 4, sum * minus8);
    }
    if (lane == 0)
        sts_f32(extra + 16 * GS,
                __uint_as_float(bad ? 0x7fc00000u : (387 - up) << 23));  // 2^(127 - up) * 2^133
}

// Where the products take their columns from: words(q, s, c, eight) gives the
// lane's values of scale group s of step q and what the group's sums start from,
// factor() what the sums are multiplied by.
//
// Staged in shared memory: a segment.
template <int GS>
struct StagedColumns {
    uint32_t values, extras[2];
    uint32_t sums[2][4];  // four of columns 2t and 2t + 1
    // column(i): the staged column of column i of the instructions
    template <class Column>
    __device__ __forceinline__ void set(const StagedView<GS>& v, int lane, Column column) {
        const int g = lane >> 2, t = lane & 3;
        values = v.values + column(g) * v.stride + t * 16;
#pragma unroll
        for (int u = 0; u < 2; ++u) extras[u] = v.extras + column(2 * t + u) * v.extra_stride;
    }
    __device__ __forceinline__ StagedColumns at(int segment) const {
        StagedColumns c;
        c.values = values + segment * 1024;
#pragma unroll
        for (int u = 0; u < 2; ++u) c.extras[u] = extras[u] + segment * StagedView<GS>::kExtra;
        return c;
    }
    // In order: q, s.
    __device__ __forceinline__ void words(int q, int s, uint32_t (&c)[4 / GS][4], float2& eight) {
#pragma unroll
        for (int j = 0; j < 4 / GS; ++j) lds(c[j], values + q * 256 + (s * (4 / GS) + j) * 64);
        const int i = q * GS + s;
        if (i % 4 == 0) {
            lds(sums[0], extras[0] + i * 4);
            lds(sums[1], extras[1] + i * 4);
        }
        eight = make_float2(__uint_as_float(sums[0][i % 4]), __uint_as_float(sums[1][i % 4]));
    }
    __device__ __forceinline__ float2 factor() const { return make_float2(lds_f32(extras[0] + 16 * GS), lds_f32(extras[1] + 16 * GS)); }
};

// Ready for the instruction in global memory, in the order of the staged values
// (ready_at), the power of two 2^64 whatever they are (ready_scale; sums keep 24
// bits while they are between 2^-56 and 2^63).  -8 times the sums comes from the
// matrix instruction with a constant operand.
template <int GS>
__device__ __forceinline__ int ready_at(int i) {
    constexpr int kPer = 4 / GS;
    const int u = i >> 3 & 15;
    return (i & ~127) + (u / (4 * kPer) * kPer + u % kPer) * 32 + u / kPer % 4 * 8 + (i & 3) * 2 + (i >> 2 & 1);
}
__device__ __forceinline__ float ready_scale(int i) { return i & 1 ? 0x1p60f : 0x1p64f; }
constexpr float kReadyFactor = 0x1p69f;
template <int GS>
__device__ __forceinline__ float2 minus8(const uint32_t (&c)[4 / GS][4]) {
    constexpr uint32_t kMinus8 = 0x80088008u, kMinus8x16 = 0x80808080u;
    float sum[4];
#pragma unroll
    for (int j = 0; j < 4 / GS; ++j) {
        if (j == 0)
            mma_bf16_from(sum, kMinus8, kMinus8, kMinus8x16, kMinus8x16, c[j][0], c[j][1], 0.f, 0.f, 0.f, 0.f);
        else
            mma_bf16(sum, kMinus8, kMinus8, kMinus8x16, kMinus8x16, c[j][0], c[j][1]);
        mma_bf16(sum, kMinus8, kMinus8, kMinus8x16, kMinus8x16, c[j][2], c[j][3]);
    }
    return make_float2(sum[0], sum[1]);
}
// .. in shared memory, a segment of the lane's column (its part of the first step).
template <int GS>
struct ReadyColumns {
    uint32_t values;
    __device__ __forceinline__ void words(int q, int s, uint32_t (&c)[4 / GS][4], float2& eight) const {
#pragma unroll
        for (int j = 0; j < 4 / GS; ++j) lds(c[j], values + q * 256 + (s * (4 / GS) + j) * 64);
        eight = minus8<GS>(c);
    }
};
// .. in registers, a step, ahead.
template <int GS>
struct DirectColumns {
    uint4 v[4];
    __device__ __forceinline__ void load(const uint16_t* p, int left, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = 32 * i + 8 * t;
            if (left >= Fmt<GS>::kStepK) {
                v[i] = ld_coherent16(p + at);
            } else {
                v[i] = make_uint4(0, 0, 0, 0);
                if (at < left) v[i] = ld_coherent16(p + at);
            }
        }
    }
    __device__ __forceinline__ void words(int, int s, uint32_t (&c)[4 / GS][4], float2& eight) const {
#pragma unroll
        for (int j = 0; j < 4 / GS; ++j) {
            const uint4 w = v[s * (4 / GS) + j];
            c[j][0] = w.x;
            c[j][1] = w.y;
            c[j][2] = w.z;
            c[j][3] = w.w;
        }
        eight = minus8<GS>(c);
    }
};

// ------------------------------------------------------------------- scales
// bf16 group scales of a segment's sixteen rows lie beside the slot, first rows
// then second rows, and come with it: a load that is waited for comes back behind
// all the copies in flight, which takes two to three microseconds, more than a
// segment's products.  Where rows have a multiple of eight they are a tensor copy
// (of at least 16 bytes of a row: two segments' with one group a step), else each
// lane copies half a row's in pieces of `piece` bytes (8 or 4), asynchronously, and
// arrives at the slot's barrier; rows of an odd number are copied by loads and
// stores.
template <int GS>
struct Scales {
    static constexpr int kHalf = 4 * GS;                     // bytes of a lane's half row
    static constexpr int kPitch = GS == 1 ? 16 : 2 * kHalf;  // between rows
    static constexpr int kSlot = 16 * kPitch;                // bytes beside a slot
    static constexpr int kWords = GS == 2 ? 1 : 2;           // of a row: all (one group a step), or a step's
    uint32_t raw[2][kWords];
    // 0: a tensor copy
    __host__ static int piece(int row_scales) { return row_scales % 8 == 0 ? 0 : GS == 2 && row_scales % 4 == 0 ? 8 : row_scales % 2 == 0 ? 4 : 2; }
    __host__ __device__ static int arrivals(int piece) { return piece == 0 ? 1 : 33; }
    // where a segment's begin in a row of the slot
    __device__ static __forceinline__ int skip(int seg) { return GS == 1 ? (seg & 1) * 8 : 0; }
    template <bool PAIRS>
    __device__ static __forceinline__ void copy(uint32_t to, uint32_t bar, const Weights& w, int row, int expert, int seg) {
        const int x = GS == 1 ? seg * 4 & ~7 : seg * 4 * GS;
        if constexpr (PAIRS)
            copy_tensor(to, w.scales, bar, x, row, 0, expert);
        else
            copy_tensor(to, w.scales, bar, x, row);
    }
    // base: the tile's first row's scales; n: its rows or pairs; second: rows from a pair's first to its second; column: the
    // segment's first
    template <bool PAIRS>
    __device__ static __forceinline__ void fill(uint32_t to, uint32_t bar, const uint16_t* base, int n, int second, int column,
                                                int row_scales, int piece, int lane) {
        const int row = lane & 15, mine = column + (lane >> 4) * (kHalf / 2);
        const int left = (row_scales - mine) * 2;  // bytes; none or less: zeros
        const uint16_t* from = base + (uint32_t)(PAIRS ? (row >= 8 ? second : 0) + min(row & 7, n - 1) : min(row, n - 1)) * row_scales;
        const uint32_t at = to + row * kPitch + (lane >> 4) * kHalf + skip(column / (4 * GS));
        if (GS == 2 && piece == 8) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at), "l"(left > 0 ? from + mine : from), "r"(left > 0 ? 8 : 0) : "memory");
        } else if (piece == 4) {
#pragma unroll 1
            for (int o = 0; o < kHalf; o += 4)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + o), "l"(left > o ? from + mine + o / 2 : from),
                             "r"(left > o ? 4 : 0)
                             : "memory");
        } else {
#pragma unroll 1
            for (int o = 0; o < kHalf; o += 2) {
                const uint32_t v = left > o ? ld_u16(from + mine + o / 2) : 0;
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + o), "h"((uint16_t)v) : "memory");
            }
            mbar_arrive(bar);
            return;
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
    // The lane's two rows, at `at`: of step q.
    __device__ __forceinline__ void read(uint32_t at, int q) {
        if (GS == 1 && q > 0) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) lds(raw[h], at + h * 8 * kPitch + (GS == 1 ? 0 : q * 2 * GS));
    }
    // Scale of group s of step q for the lane's row.
    __device__ __forceinline__ float get(int h, int q, int s) const {
        const int i = GS == 1 ? q : s;
        const uint32_t w = raw[h][i / 2];
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};

// sum += (tile) * (columns), step q of the segment at `slot`, its scales at
// `scales`.  Without the columns' factors.  In order: q.
template <int GS, class Columns>
__device__ __forceinline__ void multiply_w4(float (&sum)[4], uint32_t slot, uint32_t scales, Columns& columns, Scales<GS>& sc, int q, int lane) {
    const int g = lane >> 2, t = lane & 3;
    sc.read(scales + pair_of_row<GS>(g) * sc.kPitch, q);
    constexpr int kPer = 4 / GS;  // words of a lane per scale group
    // the lane's first chunk of the step's first group, and its bytes of it; other groups and the box's second step lie at an
    // exclusive or from there
    const int row = pair_of_row<GS>(g);
    const uint32_t base = slot + row * kBox + ((GS == 1 ? t : GS == 2 ? t >> 1 : 0) ^ row) * 16 + (GS == 1 ? 0 : GS == 2 ? (t & 1) * 8 : t * 4);
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
#pragma unroll
    for (int s = 0; s < GS; ++s) {
        const uint32_t at = (base ^ (s * (GS == 2 ? 32 : 16) + (q & 1) * 64)) + (q >> 1) * kNextAt;
        uint32_t c[kPer][4], l[kPer], h[kPer];
        float2 eight;
        lds(l, at);
        lds(h, at + kHalfAt);
        columns.words(q, s, c, eight);
        // two chains of matrix instructions where a group has eight
        constexpr bool kTwo = kPer == 4;
        float part[4], more[4];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t l8 = l[j] >> 8, h8 = h[j] >> 8;
            if (j == 0) {
                mma_bf16_from(part, l[j] & kLow, h[j] & kLow, l[j] & kHigh, h[j] & kHigh, c[j][0], c[j][1], eight.x, eight.y, eight.x, eight.y);
                if (kTwo)
                    mma_bf16_from(more, l8 & kLow, h8 & kLow, l8 & kHigh, h8 & kHigh, c[j][2], c[j][3], 0.f, 0.f, 0.f, 0.f);
                else
                    mma_bf16(part, l8 & kLow, h8 & kLow, l8 & kHigh, h8 & kHigh, c[j][2], c[j][3]);
            } else {
                mma_bf16(part, l[j] & kLow, h[j] & kLow, l[j] & kHigh, h[j] & kHigh, c[j][0], c[j][1]);
                mma_bf16(kTwo ? more : part, l8 & kLow, h8 & kLow, l8 & kHigh, h8 & kHigh, c[j][2], c[j][3]);
            }
        }
        const float sl = sc.get(0, q, s), sh = sc.get(1, q, s);
#pragma unroll
        for (int u = 0; u < 4; ++u) sum[u] = fmaf(u < 2 ? sl : sh, kTwo ? part[u] + more[u] : part[u], sum[u]);
    }
}
template <class Columns>
__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&sum)[4], const Columns& columns) {
    const float2 f = columns.factor();
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[u] = fmaf(u & 1 ? f.y : f.x, sum[u], acc[u]);
}

// ----------------------------------------------------------------- products
// How the sixteen warps of a CTA share tiles: a job's tiles, one after the other,
// are a list of segments, which is cut into sixteen ranges of equal length.  A
// warp adds up the segments that it has of a tile; the parts of a tile are added
// in the order of the warps, once a job.  (Tiles side by side and their segments
// dealt to powers of two of warps left a seventh of the warps idle, or took a
// round with two barriers for every few tiles, 1.8 us each.)
//
// 4-bit weights: as many tiles a job as a CTA has as a rule, since a job's end costs
// instructions.  bf16 weights: eight, and parts in two buffers, so that the memory
// does not wait at a job's end: 5 tokens with 10 of 32 experts of 3 x 1400 x 8192
// take 271 us, with 32 tiles and one buffer 284.
template <int GS>
constexpr int kJobTiles = GS ? 32 : 8;
template <int GS>
constexpr int kPartBuffers = GS ? 1 : 2;

// Shared memory of a product: barriers, parts of tiles (warp w's of tile i at i + w:
// ranges are in order), with several panels the sums over those done, staged
// activations, `extra` bytes, the rings, their scales.
constexpr int kSmemLimit = 227 * 1024;
struct ProductPlan {
    RowShape shape;
    uint8_t panel[9];  // segments whose activations are staged at a time, by the number of staged tokens
    int pairs;         // of columns that a tile has at most
    int tiles;         // of a job, at most
    int sums_at, staged_at, extra_at, ring_at, scales_at, smem;
    int piece;              // of the scales' copies
    int chunk = 8;          // tokens per item, at most
    bool together = false;  // all tokens are staged
};
// tokens: staged for a tile, at most; columns: staged at a time where whole rows of so many fit; tiles: of a CTA, at most
template <int GS>
inline ProductPlan plan_product(int K, int tokens, int columns, int tiles, int extra) {
    ProductPlan p;
    p.shape = RowShape::of(Fmt<GS>::row_bytes(K));
    const int segments = p.shape.segments;
    constexpr int kScales = GS ? Scales<GS ? GS : 1>::kSlot : 0, kSlot = kSlotBytes + kScales;
    p.piece = GS ? Scales<GS ? GS : 1>::piece(Fmt<GS>::scales(K)) : 0;
    tiles = tiles < kJobTiles<GS> ? tiles : kJobTiles<GS>;
    p.pairs = ((tokens < 8 ? tokens : 8) + 1) / 2;
    p.sums_at = kMvWarps * kMaxSlots * 8 + kPartBuffers<GS> * (tiles + kMvWarps) * p.pairs * 128;
    p.tiles = tiles;
    p.staged_at = p.sums_at;
    int fixed = p.staged_at + extra;
    using View = StagedView<GS ? GS : 1>;
    auto room = [&](int n) { return (kSmemLimit - fixed - kMaxSlots * kMvWarps * kSlot - 1024 - View::bytes(0, n)) / (View::bytes(1, n) - View::bytes(0, n)); };
    if (GS > 0 && room(tokens) < segments) {
        p.staged_at += tiles * p.pairs * 128;
        fixed += tiles * p.pairs * 128;
    }
    int staged = 0;
    for (int n = 0; n <= 8; ++n) {
        p.panel[n] = (uint8_t)segments;  // at most 128
        if (GS == 0 || n == 0) continue;
        const int most = room(n);
        if (n > tokens && (n > columns || most < segments)) {
            p.panel[n] = 0;
            continue;
        }
        const int panels = (segments + most - 1) / most;
        p.panel[n] = (uint8_t)((segments + panels - 1) / panels);
        const int bytes = (View::bytes(p.panel[n], n) + 15) / 16 * 16;
        staged = bytes > staged ? bytes : staged;
    }
    p.extra_at = p.staged_at + staged;
    p.ring_at = (p.extra_at + extra + 1023) / 1024 * 1024;
    p.scales_at = p.ring_at + kMaxSlots * kMvWarps * kSlotBytes;
    p.smem = p.scales_at + kMaxSlots * kMvWarps * kScales;
    return p;
}

// The products of tiles with up to 8 tokens each, up to kJobTiles tiles at a
// time ("job"), the copies running ahead across the jobs' borders.  Jobs is a
// class with
//   kPairs
//   struct Job { int count; .. }          tiles of the job
//   struct Tile { int n, tokens, row, expert; .. }  n: rows or pairs; row: the first, with pairs of the expert's
//   bool first(Job&), next(Job&)          the CTA's jobs in order
//   Tile tile(job, i)
//   scales(tile), second()                its first row's; rows from a pair's first to its second
//   x(tile, i)                            activations of the tile's token i
//   staged_key(job), staged(job), staged_x(job, i), column(tile, i): with 4-bit weights the job's tokens that are staged
//       (equal keys: the same ones), and which of them is the tile's token i
//   store(tile, pair, token, first, second)  results of a pair's two rows
//   lost()                                a wait ran out: what needed the warp's copies from there on is NaN
//   stall()                               failure injection: SlotRing::lose's limit, 0: off
// Deterministic: a tile's sums are added in the order of the warps.
template <int GS, class Jobs>
__device__ __forceinline__ void run_product(const Jobs& jobs, const Weights& weights, uint8_t* smem, const ProductPlan& plan, int K) {
    using F = Fmt<GS>;
    using Job = typename Jobs::Job;
    using Tile = typename Jobs::Tile;
    constexpr int kGS = GS ? GS : 1;
    float* parts = reinterpret_cast<float*>(smem + kMvWarps * kMaxSlots * 8);
    float* sums = reinterpret_cast<float*>(smem + plan.sums_at);
    const int lane = threadIdx.x & 31, warp = warp_index(), g = lane >> 2, t = lane & 3;
    const RowShape& shape = plan.shape;
    const int row_scales = F::scales(K), segments = shape.segments;
    const int part_size = plan.pairs * 32, in_part = (g * plan.pairs + t) * 4;  // floats
    const bool in_use = t < plan.pairs;
    SlotRing ring(smem_addr(smem) + plan.ring_at + warp * kMaxSlots * kSlotBytes, smem_addr(smem) + warp * kMaxSlots * 8, kMaxSlots, kSlotBytes);
    const uint32_t ring_scales = smem_addr(smem) + plan.scales_at + warp * kMaxSlots * Scales<kGS>::kSlot;
    auto scales_slot = [&]() { return ring.beside(ring_scales, Scales<kGS>::kSlot); };

    auto panel_of = [&](const Job& j) { return uniform(F::kW4 ? (int)plan.panel[jobs.staged(j)] : segments); };
    auto tile_of = [&](const Job& j, int i) {
        Tile t = jobs.tile(j, i);
        t.n = uniform(t.n);
        t.tokens = uniform(t.tokens);
        t.row = uniform(t.row);
        t.expert = uniform(t.expert);
        return t;
    };
    // The warp's range of a job's panel of `len` segments: from segment `seg` of tile `tile` on, `left` of them.
    struct Range {
        int tile, seg, left;
        __device__ __forceinline__ Range(int count, int len, int warp) {
            const unsigned total = count * len;
            const int f0 = (int)(total * warp / kMvWarps);
            left = (int)(total * (warp + 1) / kMvWarps) - f0;
            tile = quotient(f0, len);
            seg = f0 - tile * len;
        }
    };

    // Copies: the next (job, panel, range).
    Job cj;
    bool more = jobs.first(cj);
    if (!more) return;
    int cp = 0, cpanel = panel_of(cj), clen = min(cpanel, segments);
    Range c(cj.count, clen, warp);
    Tile ct;
    auto settle = [&]() {  // to the next panel, while nothing is left
        while (more && c.left == 0) {
            cp += clen;
            if (cp >= segments) {
                cp = 0;
                more = jobs.next(cj);
                if (more) cpanel = panel_of(cj);
            }
            if (more) {
                clen = min(cpanel, segments - cp);
                c = Range(cj.count, clen, warp);
            }
        }
        if (more) ct = tile_of(cj, c.tile);
    };
    auto fill = [&]() {
        if (!more) return;
        const bool scales = F::kW4 && plan.piece == 0;
        const int seg = cp + c.seg;
        if (lane == 0 && ring.alive) {
            ring.template fill<Jobs::kPairs>(weights, ct.row, ct.n, ct.expert, seg, shape.bytes(seg), scales ? Scales<kGS>::kSlot : 0);
            if constexpr (F::kW4)
                if (scales) Scales<kGS>::template copy<Jobs::kPairs>(scales_slot(), ring.bar(), weights, ct.row, ct.expert, seg);
        }
        if constexpr (F::kW4)
            if (!scales && ring.alive)
                Scales<kGS>::template fill<Jobs::kPairs>(scales_slot(), ring.bar(), jobs.scales(ct), ct.n, jobs.second(), seg * 4 * kGS, row_scales,
                                                         plan.piece, lane);
        if (--c.left == 0) {
            settle();
        } else if (++c.seg == clen) {
            c.seg = 0;
            ct = tile_of(cj, ++c.tile);
        }
    };
    settle();
    const unsigned long long stall = jobs.stall();
    auto fill_all = [&]() {
        for (int s = 0; s < (stall ? 1 : kMaxSlots); ++s) {
            fill();
            ring.next();
        }
        ring.at = 0;
    };

    // The columns, with bf16 weights asked for one segment ahead.
    uint4 col[4];
    StagedColumns<kGS> columns;
    const uint16_t* x = nullptr;
    auto load_part = [&](int segment, int q) { col[q] = load_column(x + segment * F::kSegK, K - segment * F::kSegK, q, t); };
    auto view = [&](const Job& j, int panel) { return StagedView<kGS>(smem_addr(smem) + plan.staged_at, panel, jobs.staged(j)); };
    auto enter = [&](const Job& j, int i, int panel) {
        const Tile tile = tile_of(j, i);
        if constexpr (F::kW4)
            // a column that does not exist repeats one of its parity: neighbours meet other banks
            columns.set(view(j, panel), lane, [&](int i) { return jobs.column(tile, i < tile.tokens ? i : min(i & 1, tile.tokens - 1)); });
        else
            x = jobs.x(tile, g < tile.tokens ? g : 0);
    };
    auto stage = [&](const Job& j, int p, int panel, bool start) {
        const int tokens = jobs.staged(j), units = min(panel, segments - p) * tokens;  // (segment, token)
        const StagedView<kGS> staged = view(j, panel);
        if (!start) __syncthreads();  // the panel before it is done with
        // four at a time, asked for together (and, at the start, before the first copies: an answer comes back behind them)
        constexpr int kAhead = 4;
#pragma unroll 1
        for (int i0 = warp; i0 < units || (start && i0 == warp); i0 += kAhead * kMvWarps) {
            uint4 w[kAhead][2];
            int s[kAhead], token[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kMvWarps;
                if (i >= units) break;
                s[u] = quotient(i, tokens);
                token[u] = i - s[u] * tokens;
                const uint16_t* from = jobs.staged_x(j, token[u]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = (p + s[u]) * F::kSegK + h * 256 + lane * 8;
                    w[u][h] = make_uint4(0, 0, 0, 0);
                    if (k < K) w[u][h] = ld_coherent16(from + k);
                }
            }
            if (start && i0 == warp) fill_all();
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i0 + u * kMvWarps >= units) break;
                stage_segment<kGS>(staged, s[u], token[u], w[u], lane);
            }
        }
        __syncthreads();
    };
    Job job;
    jobs.first(job);
    int panel = panel_of(job);
    Range range(job.count, min(panel, segments), warp);
    auto begin = [&]() {  // bf16: the first columns of a range
        if (range.left == 0) return;
        enter(job, range.tile, panel);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_part(range.seg, q);
    };
    if constexpr (F::kW4) {
        stage(job, 0, panel, true);
    } else {
        begin();
        fill_all();
    }
    if (stall) ring.lose(stall, more);
    int key = F::kW4 ? jobs.staged_key(job) : 0;
    for (int p = 0, buffer = 0;;) {
        const int len = min(panel, segments - p);
        float* part = parts + (buffer + warp) * part_size + in_part;
        if (F::kW4 && range.left > 0) enter(job, range.tile, panel);
        float acc[4] = {};
        while (range.left > 0) {
            const bool last = range.seg + 1 == len, final = range.left == 1;
            const int bytes = shape.bytes(p + range.seg), after = last ? 0 : range.seg + 1;
            if (!F::kW4 && last && !final) enter(job, range.tile + 1, panel);
            ring.wait();
            if constexpr (F::kW4) {
                Scales<kGS> now;
                const uint32_t scales = scales_slot() + Scales<kGS>::skip(p + range.seg);
                StagedColumns<kGS> here = columns.at(range.seg);
                float sum[4] = {};
                // of what is behind the end of the rows activations and scales are zero, codes whatever they are
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < 2 || bytes > kBox) multiply_w4<kGS>(sum, ring.slot(), scales, here, now, q, lane);
                add_scaled(acc, sum, here);
            } else {
                multiply_bf16(acc, ring.slot(), col, bytes, lane, [&](int q) {
                    if (!final) load_part(after, q);
                });
            }
            __syncwarp();  // all lanes have read the slot
            fill();
            ring.next();
            if (last || final) {
                if (ring.ended(more)) acc[0] = acc[1] = acc[2] = acc[3] = __uint_as_float(0x7fc00000u);
                if (in_use) *reinterpret_cast<float4*>(part + range.tile * part_size) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
                range.tile += last;
                if (F::kW4 && !final) enter(job, range.tile, panel);
            }
            range.seg = after;
            --range.left;
        }
        const Job done = job;
        const unsigned total = job.count * len;
        const int p0 = p;
        const bool whole = p + len >= segments;  // the sums are complete
        bool end = false;
        p += len;
        if (whole) {
            p = 0;
            end = !jobs.next(job);
        }
        if (!end) {
            panel = panel_of(job);
            range = Range(job.count, min(panel, segments - p), warp);
            if constexpr (!F::kW4) begin();
        }
        __syncthreads();
        // add the parts in the order of the warps, a tile per warp
#pragma unroll 1
        for (int at = warp; at < done.count; at += kMvWarps) {
            const unsigned lo = at * len, hi = lo + len;
            float4* sum = reinterpret_cast<float4*>(sums + at * part_size + in_part);
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!in_use) continue;
            if (p0 > 0) s = *sum;
#pragma unroll 1
            for (int w0 = quotient(at * kMvWarps, done.count); w0 < kMvWarps && total * w0 / kMvWarps < hi; w0 += 4) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const unsigned w = w0 + u, f0 = total * w / kMvWarps, f1 = total * (w + 1) / kMvWarps;
                    if (f0 < hi && f1 > lo && f1 > f0 && w < kMvWarps) {
                        const float4 v = *reinterpret_cast<const float4*>(parts + (buffer + w + at) * part_size + in_part);
                        s.x += v.x;
                        s.y += v.y;
                        s.z += v.z;
                        s.w += v.w;
                    }
                }
            }
            if (whole) {
                const Tile of = jobs.tile(done, at);
                const int pair = pair_of_row<GS>(g), token = 2 * t;
#pragma unroll 1
                for (int u = 0; u < 2; ++u)
                    if (pair < of.n && token + u < of.tokens) jobs.store(of, pair, token + u, u ? s.y : s.x, u ? s.w : s.z);
            } else {
                *sum = s;
            }
        }
        if (end) break;
        if (F::kW4 && (panel < segments || jobs.staged_key(job) != key)) {
            key = jobs.staged_key(job);
            stage(job, p, panel, false);  // with a barrier before
        } else if (F::kW4) {
            __syncthreads();
        }
        if (!F::kW4) buffer = buffer ? 0 : plan.tiles + kMvWarps;  // (the other one has been read before the barrier above)
    }
    if (ring.ended(more)) {
        jobs.lost();
        grace_period(10000000ull);  // copies that may still land
    }
}

}  // namespace arf
