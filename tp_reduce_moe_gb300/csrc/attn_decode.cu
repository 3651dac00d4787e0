// attn_decode.cu -- attention of one new token of each sequence over its paged
// keys and values:
//
//   s_j = scale q . k_j; out = sum_j softmax(s)_j v_j; lse = log sum_j exp(s_j)
//
// in one pass with a running maximum m, sum l and weighted sum of values o: tokens with
// scores s (times log2(e)) turn them into m' = max(m, s), l 2^(m - m') + sum 2^(s - m'),
// o 2^(m - m') + sum 2^(s - m') v.
//
// Work.  Eight (or sixteen) query heads of a key-value head share what is read: they are
// the columns of matrix instructions (m16n8k16) whose rows are tokens (scores) or columns of
// the values (o).  Such a group of heads of one sequence is an item; its tokens come in units
// of TOK.  The units of all items in a row are cut into equal ranges, one a warp, by the
// lengths on the device: lengths of any mixture keep every SM equally busy, and a captured
// launch serves any.  Where a CTA an item is nearly as fast, each item has one.
//
// A warp streams its units through a ring of its own in shared memory, keys and values in
// turn, by 16-byte asynchronous copies that run ahead across items, so that no barrier stands
// in the stream.  Items within a warp's range are finished from its registers; what is cut is
// added up once, at the end of the CTA, in the order of the warps, and over CTAs by the last of
// them to arrive, in the order of the CTAs.  No CTA waits for another.
//
// What bounds it.  Memory, where there is much: 64 sequences of 256 to 8192 tokens (eight
// key-value heads of 128 columns, 610 MB) take 100 to 104 us, 6 TB/s.  Else the way there and back,
// some 13 us: lengths and plan 2, the page's number and the first keys 2 to 3, the spread of
// the SMs' ends up to 3, a CTA's sums 2.5, joins 3 for each level.  A sequence of 500 tokens
// takes 9.5 us, of which the one SM reads for 3; one of 131071 (134 MB) 32.5.
//
// Roundings: scores, maxima, sums and o are fp32.  Weights go to the matrix instruction as
// two bf16 (their rounding and its remainder: 2^-17, where one bf16 would add 0.7 times the
// output's own rounding); with 8-bit values as halves (2^-11), whose products are exact, q
// then scaled by a power of two a row to the upper end of the halves' range: columns down to
// 2^-29 of the row's largest keep all their bits, smaller ones are off by 2^-40 of it.
#include "attn_common.cuh"

#include <cuda_fp16.h>

namespace arf {
namespace {

constexpr int kMaxGrid = 256;
constexpr int kScratchRows = 192;  // rows of sums that a CTA's warps leave in memory, eight or sixteen of each
constexpr int kFew = 24;          // parts that are joined at once
constexpr float kLazy = 8.0f;     // scores (log2) may pass the reference by so much before it moves
constexpr float kLn2 = 0.6931471805599453f;

// NT: groups of eight query heads.
template <int D, bool EIGHT, int NT>
struct Shape {
    // Sixteen warps of 128 registers hide each other's latencies; more sums need twelve of 168, or eight of 255.  (Sixteen heads
    // of 64 columns, 315 MB: twelve warps 64 us, eight 76, sixteen, whose registers spill, 70.)  Two groups of more columns spill
    // even so: of 128 columns 32 bytes a thread (228 over 8 bits), of 256 156 (148).
    static constexpr int kWarps = D == 256 ? 8 : NT == 1 ? 16 : 12;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * NT;
    static constexpr int kRing = 196608 / kWarps;                      // bytes of a warp's ring
    static constexpr int kTok = D == 64 || (D == 128 && EIGHT) ? 32 : 16;  // tokens of a unit: 4 KB of keys as a rule
    static constexpr int kRow = D * (EIGHT ? 1 : 2);                   // bytes of a key
    static constexpr int kChunks = kRow / 16;
    static constexpr int kHalf = kTok * kRow;  // bytes of a unit's keys (or values)
    static constexpr int kAhead = (kRing / kHalf - 1) / 2 < 4 ? (kRing / kHalf - 1) / 2 : 4;  // units that are asked for ahead
    static constexpr int kHalves = 2 * kAhead + 1;
    // Units that an item counts for besides its own: to begin and end one takes a warp 2 us.  (700 sequences of up to 89 tokens,
    // heads of 64 columns: none 37.6 us, two 31.4, four 29.9, six 32.6; five of 1 to 20001 tokens, 256 columns: one 24.5, four
    // 23.1.)
    static constexpr int kCost = 4;
    static constexpr int kMany = (1 << 27) / kHalf;  // units that are too many for all SMs (256 MB)
    // Units by which a CTA that keeps an item may pass an equal share: 2.6 a warp.  (One sequence, eight heads of 128 columns: 500
    // tokens 9.6 us by one CTA, 10.4 cut; 600 10.2 and 10.4; 700 10.9 and 10.3.  8-bit ones of 64 columns: 1000 7.8 and 9.0, 2000
    // 10.4 and 9.3.)
    static constexpr int kAlone = kWarps * 21 / 8;
    static constexpr int kPitch = D + 4;       // floats from a row of sums to the next in shared memory, free of bank conflicts
    // In memory nothing is between the rows: sectors that are not written whole would have to be read before they are merged.
    static constexpr int kSums = kRows * D;
    static constexpr int kPart = kSums + 2 * kRows;  // a CTA's part: sums, maxima, sums of weights
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kSmem + 26624 <= 232448, "shared memory of a CTA");
    static_assert(kWarps * kRows <= kScratchRows, "the handle's scratch");
    static_assert(kRows * kPitch * 4 <= kRing, "a warp's sums, in its ring");
    static_assert(kAhead >= 1 && kAhead + 2 <= 8, "units that are asked for and not used, of the eight masks and segments that are kept");
    static_assert(kPart % 4 == 0 && 2 * kFew * (kPart / 16 + 2 * kRows) * 4 <= kSmem && 16 * 16 >= kMaxGrid && kFew >= 16,
                  "sixteenths of the columns of all parts that two joins take");
    // where chunk c of row r lies, so that eight rows' chunks c are in eight different groups of banks
    __device__ static int place(int r, int c) {
        return r * kRow + ((kChunks >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & (kChunks - 1))) << 4);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
// Or zeros: nothing is read where bytes is 0.
__device__ __forceinline__ void copy16_or_zeros(uint32_t dst, const void* src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {  // of eight by eight 16-bit values
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <bool EIGHT>
__device__ __forceinline__ void mma(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (EIGHT)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^(m - top), 0 for a part without tokens.
__device__ __forceinline__ float share_of(float m, float top) { return ex2(m - (top == -INFINITY ? 0.0f : top)); }

// A warp's share of an item: units [u0, u1) of its n.
struct Segment {
    int64_t item;    // where the item's first unit is among all
    int u0, u1, n;
    int kv_head;
    int row, rows;   // first row of the output [B * heads], and how many
    bool last;       // of the warp
};

// Tokens that are looked at, and where they begin.
__device__ __forceinline__ int tokens_of(const DecodeArgs& a, int b, bool report, int* start) {
    const int len = checked_length(a, b, report);
    *start = a.window > 0 && len > a.window ? len - a.window : 0;
    return len;
}

template <int TOK>
__device__ __forceinline__ int units_of(int start, int len) {
    return (int)(((int64_t)len - start + TOK - 1) / TOK);
}

// Quotients of numbers that are small as a rule.
__device__ __noinline__ int64_t quotient64(int64_t n, int64_t d) {
    return ((n | d) >> 31) == 0 ? (int64_t)((unsigned)n / (unsigned)d) : n / d;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// A part of an item that the warps or CTAs share.
struct Part {
    int64_t item;  // first unit of the item, -1: no part
    int n, kv_head, row, rows;
};

// An item that CTAs share, `parts` of them from `first` on: every `step`-th has a sum, of which this CTA may add up `count`
// from `leader` on, each `fan` of them.
struct Join {
    int first, parts, fan, step, leader, count;
};

__device__ __forceinline__ float lse_of(float top, float weight) { return weight == 0.0f ? -INFINITY : (top + lg2(weight)) * kLn2; }

// Four columns of a row of the output, and with the first of them its lse.
__device__ __forceinline__ void finish_row(const DecodeArgs& a, int row, int d, int D, float4 sum, float weight, float vs, float top) {
    const float f = weight == 0.0f ? 0.0f : __fdividef(vs, weight);
    *reinterpret_cast<uint2*>(a.out + (int64_t)row * D + d) = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
    if (d == 0 && a.lse != nullptr) a.lse[row] = lse_of(top, weight);
}

// One more on a counter, seen by all behind what is written before it, and before what is read after it.
__device__ __forceinline__ unsigned arrive(unsigned* counter) {
    unsigned before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}

__device__ __forceinline__ void add(float4& sum, float f, float4 v) {
    sum.x += f * v.x;
    sum.y += f * v.y;
    sum.z += f * v.z;
    sum.w += f * v.w;
}

template <int D, bool EIGHT, int NT>
__global__ void __launch_bounds__(Shape<D, EIGHT, NT>::kThreads, 1)
    attn_decode_kernel(const __grid_constant__ DecodeArgs a) {
    using S = Shape<D, EIGHT, NT>;
    constexpr int TOK = S::kTok, MT = TOK / 16, kSteps = D / 16, kWarps = S::kWarps, kThreads = S::kThreads, kRows = S::kRows;
    constexpr float kOffset = EIGHT ? 7.0f : 0.0f;  // halves: weights up to 2^(8 + 7), so that small ones keep their bits
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[2 * kWarps][kRows], s_l[2 * kWarps][kRows], s_share[2 * kWarps][kRows], s_top[2 * kWarps][kRows],
        s_weight[2 * kWarps][kRows];
    __shared__ Part s_part[2 * kWarps];  // of each warp: what it began with, if it went on; what it ended with
    __shared__ int s_run[2 * kWarps];
    __shared__ int64_t s_scan[kWarps];
    __shared__ int s_most[kWarps];
    __shared__ int64_t s_before[kThreads];  // units before a thread's sequences
    __shared__ Join s_join[2];
    __shared__ unsigned s_mask[kWarps][8];
    __shared__ Segment s_seg[kWarps][8];
    __shared__ const uint8_t* s_row[kWarps][2][32];  // where the keys and values of a unit's tokens are
    pdl_wait();  // no global memory access before this point
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;

    // ---- what this CTA's warps take
    int64_t total, each = 0;   // units, and units of a warp where all are dealt out
    int64_t begin, end;        // units of this CTA
    // The walk over this warp's items (clamped where lengths that change during the call could lead it astray).  One counts for
    // kCost units more, before its first, for what it costs to begin and end it; these are walked over.
    int w_b = 0, w_group = 0, w_u = 0, w_start = 0, w_len = 0, w_n = 0;  // sequence, group, next unit of kCost + w_n, tokens
    int64_t w_item = 0;  // where the item's first unit (behind what it costs) is among all
    int64_t w_left = 0;  // units of the range that are not handed out; 0 once no real one is among them
    auto sequence = [&]() {
        w_len = tokens_of(a, w_b, false, &w_start);
        w_n = units_of<TOK>(w_start, w_len);
    };
    {
        auto units = [&](int b) {  // of one item, with what it costs
            int start;
            const int len = tokens_of(a, b, blockIdx.x == 0, &start), n = units_of<TOK>(start, len);
            return n > 0 ? n + S::kCost : 0;
        };
        // a thread's sequences, and before them the units of the threads before; few sequences: each warp sums by itself (4096
        // single tokens, whose lengths a thread reads one after the other: 14.8 us; 256 columns, half the threads, 31.6)
        const bool few = a.B <= 32;
        const int per_thread = few ? 1 : (a.B + kThreads - 1) / kThreads;
        const int b0 = (few ? lane : tid) * per_thread, b1 = min(a.B, b0 + per_thread);
        int64_t mine = 0;
        int most = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int n = units(b);
            mine += (int64_t)n * a.groups;
            most = max(most, n);
        }
        int64_t before = warp_scan(mine, lane);
        most = __reduce_max_sync(0xffffffffu, most);
        total = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
        if (!few) {
            if (lane == 0) {
                s_scan[warp] = total;
                s_most[warp] = most;
            }
            __syncthreads();
            const int64_t sum = warp_scan(lane < kWarps ? s_scan[lane] : 0, lane);
            most = __reduce_max_sync(0xffffffffu, lane < kWarps ? s_most[lane] : 0);
            total = __shfl_sync(0xffffffffu, sum, 31);
            before += __shfl_sync(0xffffffffu, sum, (warp + 31) & 31) * (warp > 0);
        }
        // Three quarters of the SMs draw what the memory gives, with fewer streams in each other's way.  128 columns: 610 MB 102 us
        // from 114 SMs, 108 from 152; 1.05 GB 168 and 180; 1.2 GB 191 and 202.  256: 525 MB 94 and 96, 1.3 GB 215 and 220.  134 MB,
        // where each SM's latencies count, take 35 and 33.4.  Where an SM has more work with a byte all are needed: 64 columns 540 MB
        // 109 us from 114 SMs, 103 from 152, 890 MB 173 and 164, 1.07 GB 210 and 196; sixteen heads a key 630 MB 141 and 112; 8-bit
        // caches too.
        const int fewer = max(1, (int)gridDim.x * 3 / 4);
        if ((int64_t)a.B * a.groups <= gridDim.x && (int64_t)(most - S::kAlone) * fewer <= total) {
            // One CTA an item: nothing to join over CTAs, and none has much more to do than with equal shares of those.
            // (128 equal items of 8 bits, 655 MB: 104 us, with equal shares of 152 SMs 114.)
            w_b = blockIdx.x / a.groups;
            w_group = blockIdx.x - w_b * a.groups;
            if (w_b < a.B) sequence();
            const int share = (w_n + kWarps - 1) / kWarps;
            w_u = min(w_n, warp * share);
            w_left = min(share, w_n - w_u);
            w_u += S::kCost;
            begin = 0;
            end = w_n;
        } else {
            // Equal ranges of all units; the last ones may be short or empty.
            const int warps = (D > 64 && !EIGHT && NT == 1 && a.per_head == 1 && total >= S::kMany ? fewer : (int)gridDim.x) * kWarps;
            each = max((int64_t)1, quotient64(total + warps - 1, warps));
            begin = each * (blockIdx.x * kWarps);
            end = min(total, begin + each * kWarps);
            const int64_t from = begin + each * warp;
            w_left = max((int64_t)0, min(each, total - from));
            int64_t skip = 0;
            if (few) {
                const unsigned at = __ballot_sync(0xffffffffu, before <= from && from < before + mine);
                w_b = at ? __ffs(at) - 1 : 0;
                skip = from - __shfl_sync(0xffffffffu, before, w_b);
            } else {
                // the last thread whose sequences begin at or before this warp's first unit: of each so many, then among them
                constexpr int kEach = kThreads / 32;
                s_before[tid] = before;
                __syncthreads();
                const int block = __popc(__ballot_sync(0xffffffffu, s_before[lane * kEach] <= from)) - 1;
                const unsigned upto = __ballot_sync(0xffffffffu, lane < kEach && s_before[block * kEach + lane % kEach] <= from);
                const int thread = block * kEach + __popc(upto) - 1;
                w_b = thread * per_thread;
                skip = from - s_before[thread];
                if (per_thread > 1 && w_left > 0)
#pragma unroll 1
                    for (int64_t n; w_b + 1 < a.B && (n = (int64_t)units(w_b) * a.groups) <= skip; ++w_b) skip -= n;
            }
            if (w_left > 0) {
                sequence();
                w_n = max(w_n, 1);
                w_group = (int)min(quotient64(skip, w_n + S::kCost), (int64_t)(a.groups - 1));
                w_u = (int)min(skip - (int64_t)w_group * (w_n + S::kCost), (int64_t)(w_n + S::kCost - 1));
                w_item = from - w_u + S::kCost;
                if (w_left <= S::kCost - w_u) w_left = 0;
            }
        }
    }

    // ---- the stream of this warp's units
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    bool asking = w_left > 0, live = false;  // there are units left; the one that is being asked for is one
    int ask_u = 0, ask_u1 = 0, ask_last = 0;  // of the segment that is asked for: next unit, end, last page of the sequence
    const uint8_t *k_head = nullptr, *v_head = nullptr;  // and its keys and values
    unsigned asked = 0, found = 0;  // units asked for, segments found
    // Copies are issued without a pause where latencies count (500 tokens 10.3 us with pauses, 9.4 without), and one behind its
    // place in the table where memory has all it can do (610 MB 103.5 us without pauses, 100.3 with; 1 GB 170.9 and 164.9).
    const bool quick = EIGHT || NT > 1 || total < S::kMany;
    constexpr unsigned kAll = 0xffffffffu >> (32 - TOK);
    unsigned present = 0;           // tokens of the unit that was looked up
    uint32_t fill = 0;              // place in the ring that is filled next
    // the page table's entries from table_at on: this lane's of the first 32 and of the next 32
    int table_at = 0, entry = 0, entry_next = 0;
    const uint64_t policy = a.per_head == 1 ? l2_evict_first_policy() : l2_evict_normal_policy();
    auto page_of = [&](int64_t token) { return (int)((uint64_t)token * a.page_mul >> (31 + a.page_shift)); };
    auto table_entry = [&](int index) {  // -1 behind the sequence's last
        return index <= ask_last ? a.table[w_b * a.table_stride + index] : -1;
    };
    auto advance = [&]() {  // to the next segment, once this one's units have been asked for
        if (!asking || ask_u != ask_u1) return;
        asking = w_left > 0;
        if (!asking) return;
        if (w_u == w_n + S::kCost) {  // the item is done: the next one that has units (there is one, for some are left)
            w_u = 0;
            w_item += w_n + S::kCost;
            if (++w_group == a.groups) {
                w_group = 0;
#pragma unroll 1
                while (w_b + 1 < a.B) {
                    ++w_b;
                    sequence();
                    if (w_n > 0) break;
                }
                w_n = max(w_n, 1);
            }
        }
        const int take = (int)(w_left < w_n + S::kCost - w_u ? w_left : w_n + S::kCost - w_u);
        const int head = a.per_head == 1 ? w_group : w_group / a.per_head, row = (w_group - head * a.per_head) * a.rows_of_group;
        ask_u = max(w_u - S::kCost, 0);
        w_u += take;
        ask_u1 = w_u - S::kCost;
        w_left -= take;
        if (w_left <= S::kCost) w_left = 0;
        if (lane == 0)
            s_seg[warp][found & 7] = Segment{w_item, ask_u, ask_u1, w_n, head, w_b * a.heads + head * a.shared + row,
                                             min(a.rows_of_group, a.shared - row), w_left == 0};
        ++found;
        ask_last = page_of(max(w_len, 1) - 1);
        table_at = page_of(w_start + (int64_t)ask_u * TOK);
        entry = table_entry(table_at + lane);
        entry_next = table_entry(table_at + 32 + lane);
        k_head = a.k.data + head * a.k.head;
        v_head = a.v.data + head * a.v.head;
    };
    auto copy_half = [&](int which) {  // keys (0) or values (1) of the unit that was looked up
        if (live) {
            const uint8_t* const* rows = s_row[warp][which] + lane / S::kChunks;
            const int c = lane % S::kChunks;
            if (present == kAll && quick) {
                // (places first, some at a time: one that is read behind a copy waits for it to be issued)
                constexpr int kCopies = TOK * S::kChunks / 32, kBatch = kCopies < 4 ? kCopies : 4;
#pragma unroll
                for (int i0 = 0; i0 < kCopies; i0 += kBatch) {
                    const uint8_t* from[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) from[i] = rows[(i0 + i) * 32 / S::kChunks] + c * 16;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) copy16(ring + fill + S::place(((i0 + i) * 32 + lane) / S::kChunks, c), from[i], policy);
                }
            } else {
                // (zeros that are read would all come from one place: 1184 single tokens take 21 us with them)
#pragma unroll 4
                for (int i = 0; i < TOK * S::kChunks; i += 32) {
                    const int row = (i + lane) / S::kChunks;
                    copy16_or_zeros(ring + fill + S::place(row, c), rows[i / S::kChunks] + c * 16, present >> row & 1 ? 16 : 0, policy);
                }
            }
        }
        copy_commit();
        fill = fill + S::kHalf == S::kHalves * S::kHalf ? 0 : fill + S::kHalf;
    };
    auto ask_keys = [&]() {
        live = asking;
        if (live) {
            const int64_t first = w_start + (int64_t)ask_u * TOK, token = first + lane;
            if (page_of(first) - table_at >= 32) {  // (a unit has 32 tokens at most)
                table_at += 32;
                entry = entry_next;
                entry_next = table_entry(table_at + 32 + lane);
            }
            const int index = page_of(token), in_page = (int)token - index * a.page_size, at = index - table_at;
            const int here = __shfl_sync(0xffffffffu, entry, at & 31), next = __shfl_sync(0xffffffffu, entry_next, at & 31);
            const int page = at < 32 ? here : next;
            const bool wanted = lane < TOK && token < w_len, there = wanted && (unsigned)page < (unsigned)a.pages;
            if (wanted && !there) atomicOr(a.err, kErrPageRange);
            present = __ballot_sync(0xffffffffu, there);
            __syncwarp();  // all lanes have read the places before
            if (lane == 0) s_mask[warp][asked & 7] = present;
            if (lane < TOK) {  // (what is not there is not read)
                s_row[warp][0][lane] = there ? k_head + (page * a.k.page + in_page * a.k.token) : k_head;
                s_row[warp][1][lane] = there ? v_head + (page * a.v.page + in_page * a.v.token) : v_head;
            }
            __syncwarp();
            ++asked;
            ++ask_u;
        }
        copy_half(0);
    };
    auto empty_rows = [&]() {  // rows without tokens: zeros, dealt to the warps
#pragma unroll 1
        for (int64_t b = blockIdx.x + (int64_t)gridDim.x * warp; b < a.B; b += gridDim.x * kWarps)
            if (checked_length(a, (int)b, false) == 0) {
#pragma unroll 1
                for (int j = lane; j < a.heads * D / 8; j += 32) st_global16(a.out + b * a.heads * D + j * 8, make_uint4(0, 0, 0, 0));
                if (a.lse != nullptr)
#pragma unroll 1
                    for (int j = lane; j < a.heads; j += 32) a.lse[b * a.heads + j] = -INFINITY;
            }
    };
    if (begin >= end) {
        empty_rows();
        return;
    }

    auto place_of = [&](int w) {  // of the sums that a warp leaves in mid-stream
        return a.part + (int64_t)gridDim.x * 2 * S::kPart + ((int64_t)blockIdx.x * kWarps + w) * S::kSums;
    };

    // ---- the units.  A turn asks for one and works on the one that was asked for kAhead turns before; the turn before the
    // first looks up where the first are.
    uint32_t take = 0;   // place in the ring that is used next
    unsigned taken = 0, begun = 0;  // units used, segments begun
    bool more = asking;
    if (lane < 2) s_part[2 * warp + lane].item = -1;
    auto wait_half = [&]() {
        copy_wait<2 * S::kAhead>();
        __syncwarp();
        const uint32_t slot = ring + take;
        take = take + S::kHalf == S::kHalves * S::kHalf ? 0 : take + S::kHalf;
        return slot;
    };
    uint32_t q[kSteps][NT][2];
    float q_scale[NT][2];  // of the scores of heads 8 i + 2 t4 (+1): log2(e), scale, scale of the keys, power of two of the row
    // o: of heads 8 n + 2 t4 (+1) the columns 16 i + g (+8), with bytes 16 i + 2 g (+1)
    float o[kSteps][NT][4], m[NT][2], l[NT][2];
    uint32_t p[MT][NT][2], rest[MT][NT][2];  // weights of a unit
    int u = 0, u1 = 0;  // of the segment that is worked on: the next unit, the end
    auto begin_segment = [&]() {
        const Segment& seg = s_seg[warp][begun & 7];
        u = seg.u0;
        u1 = seg.u1;
        // Query heads 8 i + g.  Columns of a step: 2 t4 (+1) and 2 t4 + 8 (+1); with bytes 4 t4 .. 4 t4 + 3, the order that
        // their keys come in.  (Rows that the item does not have are read as its last: what becomes of them is not used.)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint16_t* src = a.q + (int64_t)(seg.row + min(8 * n + g, seg.rows - 1)) * D;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                if (EIGHT) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src + i * 16 + t4 * 4);
                    q[i][n][0] = v.x;
                    q[i][n][1] = v.y;
                } else {
                    q[i][n][0] = *reinterpret_cast<const uint32_t*>(src + i * 16 + t4 * 2);
                    q[i][n][1] = *reinterpret_cast<const uint32_t*>(src + i * 16 + t4 * 2 + 8);
                }
            q_scale[n][0] = q_scale[n][1] = a.scale;
        }
        if constexpr (EIGHT) {
            const float ks = a.scale * a.k.scale[seg.kv_head];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[i][n][c] << 16)), fabsf(__uint_as_float(q[i][n][c] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the power of two that brings the row's largest value to [2^15, 2^16), less for rows below 2^-111 (65280 at most; a
                // sum of 256 products with 448 stays below 2^33)
                int e = (int)(__float_as_uint(top) >> 23) - 127 - 15;
                e = e < -126 ? -126 : e > 112 ? 112 : e;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = ks * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        q[i][n][c] = pack_f16x2(__uint_as_float(q[i][n][c] << 16) * down, __uint_as_float(q[i][n][c] & 0xffff0000u) * down);
                q_scale[n][0] = __shfl_sync(0xffffffffu, up, 8 * t4);
                q_scale[n][1] = __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][n][j] = 0.0f;
        }
    };
    // this lane's row of a matrix of 16 by 16: eights of rows before or behind eights of columns
    const int row8 = ((lane >> 3) & 1) * 8 + (lane & 7), odd8 = (lane >> 4) * 8 + (lane & 7);
    // scores of a unit's tokens, and their weights
    auto scores = [&]() {
        // of heads 8 n + 2 t4 (+1) the tokens 16 i + g (+8)
        const uint32_t slot = wait_half();
        float s[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] = 0.0f;
        if (EIGHT) {
            // a matrix is 8 tokens by 16 bytes: one step of the columns
#pragma unroll
            for (int c = 0; c < kSteps; c += 2)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t r[4];
                    ldmatrix4(r, slot + S::place(i * 16 + row8, c + (lane >> 4)));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)r[2 * j]), a1 = e4m3x2_to_f16x2((uint16_t)r[2 * j + 1]);
                        const uint32_t a2 = e4m3x2_to_f16x2((uint16_t)(r[2 * j] >> 16)), a3 = e4m3x2_to_f16x2((uint16_t)(r[2 * j + 1] >> 16));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma<true>(s[i][n], a0, a1, a2, a3, q[c + j][n][0], q[c + j][n][1]);
                    }
                }
        } else {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t r[4];
                    ldmatrix4(r, slot + S::place(i * 16 + row8, c * 2 + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma<false>(s[i][n], r[0], r[1], r[2], r[3], q[c][n][0], q[c][n][1]);
                }
        }
        const unsigned mask = s_mask[warp][taken++ & 7];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] *= q_scale[n][j & 1];
        if (mask != kAll) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                if (!(mask >> (8 * i + g) & 1))
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[i >> 1][n][2 * (i & 1)] = s[i >> 1][n][2 * (i & 1) + 1] = -INFINITY;
        }
        float keep[NT][2];
        bool moved = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = fmaxf(s[0][n][h], s[0][n][h + 2]);
                if (MT == 2) top = fmaxf(top, fmaxf(s[MT - 1][n][h], s[MT - 1][n][h + 2]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                keep[n][h] = 1.0f;
                if (top > m[n][h] + kLazy) {  // (the first finite score passes minus infinity)
                    keep[n][h] = ex2(m[n][h] - top);
                    m[n][h] = top;
                    l[n][h] *= keep[n][h];
                    moved = true;
                }
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][n][j] *= keep[n][j & 1];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) base[h] = m[n][h] == -INFINITY ? 0.0f : m[n][h] - kOffset;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float x = ex2(s[i][n][2 * r] - base[0]), y = ex2(s[i][n][2 * r + 1] - base[1]);
                    l[n][0] += x;
                    l[n][1] += y;
                    if (EIGHT) {
                        p[i][n][r] = transposed(pack_f16x2(x, y));
                    } else {
                        const uint32_t w = pack_bf16x2(x, y);
                        p[i][n][r] = transposed(w);
                        rest[i][n][r] = transposed(pack_bf16x2(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xffff0000u)));
                    }
                }
        }
    };
    auto values = [&]() {
        const uint32_t slot = wait_half();
        if (EIGHT) {
            // transposed by pairs of bytes: a register holds two columns of two tokens; even columns make rows 0 .. 7 of
            // an operand, odd ones rows 8 .. 15
#pragma unroll
            for (int c = 0; c < kSteps; c += 2)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t r[4];
                    ldmatrix4_trans(r, slot + S::place(i * 16 + row8, c + (lane >> 4)));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t x = __byte_perm(r[2 * j], 0, 0x3120), y = __byte_perm(r[2 * j + 1], 0, 0x3120);
                        const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)x), a1 = e4m3x2_to_f16x2((uint16_t)(x >> 16));
                        const uint32_t a2 = e4m3x2_to_f16x2((uint16_t)y), a3 = e4m3x2_to_f16x2((uint16_t)(y >> 16));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma<true>(o[c + j][n], a0, a1, a2, a3, p[i][n][0], p[i][n][1]);
                    }
                }
        } else {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t r[4];
                    ldmatrix4_trans(r, slot + S::place(i * 16 + odd8, c * 2 + ((lane >> 3) & 1)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<false>(o[c][n], r[0], r[1], r[2], r[3], p[i][n][0], p[i][n][1]);
                        mma<false>(o[c][n], r[0], r[1], r[2], r[3], rest[i][n][0], rest[i][n][1]);
                    }
                }
        }
    };
    // the item, or this warp's part of it
    auto end_segment = [&]() {
        const Segment& seg = s_seg[warp][begun++ & 7];
        more = !seg.last;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], x);
        if (seg.u0 > 0 || seg.u1 < seg.n) {  // a part
            __syncwarp();  // all lanes have read the ring
            // (when the last sums are written the stream has ended, and the ring is free)
            const int which = 2 * warp + (more ? 0 : 1), pitch = more ? D : S::kPitch;
            float* const to = more ? place_of(warp) : reinterpret_cast<float*>(smem + warp * S::kRing);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 8 * n + 2 * t4 + h;
                    if (g == 0) {
                        s_m[which][row] = m[n][h];
                        s_l[which][row] = l[n][h];
                    }
                    float* const line = to + row * pitch + (EIGHT ? 2 * g : g);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        if (EIGHT) {
                            *reinterpret_cast<float2*>(line + i * 16) = make_float2(o[i][n][h], o[i][n][h + 2]);
                        } else {
                            line[i * 16] = o[i][n][h];
                            line[i * 16 + 8] = o[i][n][h + 2];
                        }
                }
            if (lane == 0) s_part[which] = Part{seg.item, seg.n, seg.kv_head, seg.row, seg.rows};
            return;
        }
        // the whole: straight to the output
        const float vs = EIGHT ? a.v.scale[seg.kv_head] : 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * n + 2 * t4 + h;
                f[h] = l[n][h] == 0.0f ? 0.0f : __fdividef(vs, l[n][h]);
                if (g == 0 && a.lse != nullptr && row < seg.rows) a.lse[seg.row + row] = lse_of(m[n][h] - kOffset, l[n][h]);
            }
            if (EIGHT) {  // (neighbouring columns)
                uint16_t* const to = a.out + (int64_t)(seg.row + 8 * n + 2 * t4) * D + 2 * g;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (8 * n + 2 * t4 + h < seg.rows)
                            *reinterpret_cast<uint32_t*>(to + h * D + i * 16) = pack_bf16x2(o[i][n][h] * f[h], o[i][n][h + 2] * f[h]);
            } else {
                // with the lane next to this one two columns of one head each, with the one behind that four: whole sectors
                const bool second = g & 1, behind = g & 2;
                const int row = 8 * n + 2 * t4 + second;
                uint16_t* const to = a.out + (int64_t)(seg.row + row) * D + (behind ? 8 : 0) + (g & 4);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t two[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = o[i][n][2 * j] * f[0], y = o[i][n][2 * j + 1] * f[1];
                        const float next = __shfl_xor_sync(0xffffffffu, second ? x : y, 4);
                        two[j] = second ? pack_bf16x2(next, y) : pack_bf16x2(x, next);
                    }
                    const uint32_t next = __shfl_xor_sync(0xffffffffu, behind ? two[0] : two[1], 8);
                    if (row < seg.rows) *reinterpret_cast<uint2*>(to + i * 16) = behind ? make_uint2(next, two[1]) : make_uint2(two[0], next);
                }
            }
        }
    };
#pragma unroll 1
    for (int turn = -1; more; ++turn) {
        __syncwarp();  // the place that is filled now has been read by all lanes
        if (turn >= 0) ask_keys();
        const bool work = turn >= S::kAhead;
        if (work) {
            if (u == u1) begin_segment();
            scores();
        }
        __syncwarp();
        if (turn >= 0) copy_half(1);
        advance();
        if (work) {
            values();
            if (++u == u1) end_segment();
        }
    }
    pdl_trigger();
    empty_rows();

    // ---- what the warps share: runs of parts of one item
    __syncthreads();
    Part mine{-1, 0, 0, 0, 0};
    if (lane < 2 * kWarps) mine = s_part[lane];
    const unsigned there = __ballot_sync(0xffffffffu, mine.item >= 0), below = there & ((1u << lane) - 1);
    const int64_t previous = __shfl_sync(0xffffffffu, mine.item, below ? 31 - __clz(below) : lane);
    const bool starts = mine.item >= 0 && (below == 0 || previous != mine.item);
    const unsigned start_mask = __ballot_sync(0xffffffffu, starts);
    const int runs = __popc(start_mask);
    if (runs == 0) return;
    if (warp == 0 && starts) s_run[__popc(below & start_mask)] = lane;

    auto finish = [&](const Part& p, int row, int d, float4 sum, float top, float weight) {
        finish_row(a, p.row + row, d, D, sum, weight, EIGHT ? a.v.scale[p.kv_head] : 1.0f, top - kOffset);
    };
    // a CTA's part of an item: one for an item that began in a range before, one for an item that begins in this one
    auto part_of = [&](int cta, bool begins) { return a.part + ((int64_t)cta * 2 + (begins ? 1 : 0)) * S::kPart; };

    // items that this CTA shares with others: perhaps its first with those before it, and its last with those behind it
    auto owner = [&](int64_t unit) { return (int)min(quotient64(unit, each * kWarps), (int64_t)(gridDim.x - 1)); };
    if (tid >= kThreads - 2) {  // (of the last warp, the others have more to do)
        const int which = tid - (kThreads - 2);
        const Part p = s_part[which == 0 ? __ffs(start_mask) - 1 : 31 - __clz(start_mask)];
        Join j{0, 0, 0, 0, 0, 0};
        if ((which == 0 || runs > 1) && !(p.item >= begin && p.item + p.n <= end)) {
            j.first = owner(p.item);
            j.parts = owner(p.item + p.n - 1) - j.first + 1;
            j.fan = j.parts;
            if (j.parts > kFew)
                for (j.fan = 5; j.fan * j.fan < j.parts;) ++j.fan;
            j.step = 1;
        }
        s_join[which] = j;
    }

    // what each part counts, and the runs' maxima and weights: a lane a part, a warp a row
    {
        const int first = start_mask & ((2u << lane) - 1) ? 31 - __clz(start_mask & ((2u << lane) - 1)) : 0;  // of this lane's run
        const unsigned behind = start_mask & ~((2u << lane) - 1);
        const int last = behind ? __ffs(behind) - 2 : 31;
#pragma unroll 1
        for (int row = warp; row < kRows; row += kWarps) {
            const float m = there >> lane & 1 ? s_m[lane][row] : -INFINITY;
            float top = m;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {  // to the run's end, then back to its beginning
                const float v = __shfl_down_sync(0xffffffffu, top, x);
                if (lane + x <= last) top = fmaxf(top, v);
            }
            top = __shfl_sync(0xffffffffu, top, first);
            const float share = share_of(m, top);
            float weight = there >> lane & 1 ? share * s_l[lane][row] : 0.0f;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, weight, x);
                if (lane + x <= last) weight += v;
            }
            if (lane < 2 * kWarps) {
                s_share[lane][row] = share;
                s_top[lane][row] = top;
                s_weight[lane][row] = weight;  // (of the run, where it begins)
            }
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < runs * kRows * (D / 4); i += kThreads) {
        const int row = i / (D / 4) % kRows, d = i % (D / 4) * 4, j0 = s_run[i / (kRows * (D / 4))];
        const Part p = s_part[j0];
        const bool inside = p.item >= begin && p.item + p.n <= end;
        if (!inside && d == 0) {  // (of all rows, for whole sectors)
            float* to = part_of(blockIdx.x, p.item >= begin) + S::kSums + row;
            to[0] = s_top[j0][row];
            to[kRows] = s_weight[j0][row];
        }
        if (row >= p.rows) continue;
        const unsigned behind = start_mask & ~((2u << j0) - 1);
        const unsigned of_run = there & ~((1u << j0) - 1) & (behind ? (1u << (__ffs(behind) - 1)) - 1 : ~0u);
        // what warps in a row ended with, in their rings, and then perhaps what the next warp began with
        const unsigned ended = of_run & 0xaaaaaaaau, began = of_run & 0x55555555u;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int w0 = ended ? (__ffs(ended) - 1) >> 1 : 0, w1 = w0 + __popc(ended);
        const uint8_t* at = smem + w0 * S::kRing + (row * S::kPitch + d) * 4;
#pragma unroll 4
        for (int w = w0; w < w1; ++w, at += S::kRing) add(sum, s_share[2 * w + 1][row], *reinterpret_cast<const float4*>(at));
        if (began) {
            const int j = __ffs(began) - 1;
            add(sum, s_share[j][row], *reinterpret_cast<const float4*>(place_of(j >> 1) + row * D + d));
        }
        if (inside) finish(p, row, d, sum, s_top[j0][row], s_weight[j0][row]);
        else *reinterpret_cast<float4*>(part_of(blockIdx.x, p.item >= begin) + row * D + d) = sum;
    }

    // ---- what CTAs share: the last of them to arrive adds up their parts; of many parts the last of each few, and the last
    // of those.  (One SM reads some 60 GB/s: 76 parts of 4 KB take it 5 us, nine and nine of their sums 1.2.)
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        __syncthreads();
        if (tid < 2) {
            Join& j = s_join[tid];
            j.count = 0;
            if (j.step > 0) {
                const int reach = j.step * j.fan;
                j.leader = j.first + ((int)blockIdx.x - j.first) / reach * reach;
                const int count = min(j.fan, (j.first + j.parts - 1 - j.leader) / j.step + 1);
                // this level's counter, of the leader's part
                unsigned* counter = a.count + (j.leader * 2 + (j.leader == j.first ? 1 : 0)) * 2 + level;
                if (arrive(counter) == (unsigned)count - 1) {
                    *counter = 0;
                    j.count = count;
                }
            }
        }
        __syncthreads();
        const Join left = s_join[0], right = s_join[1];
        const int n = left.count + right.count;
        if (n == 0) return;
        const Part part_left = s_part[s_run[0]], part_right = s_part[s_run[runs - 1]];
        float* const head_left = part_of(left.leader, left.leader == left.first);
        float* const head_right = part_of(right.leader, right.leader == right.first);
        // both items' parts come to shared memory at once, in slices of their columns where they do not fit whole
        int log_w = D == 64 ? 4 : D == 128 ? 5 : 6;  // of fours of columns
#pragma unroll 1
        while (n * (kRows * 16 << log_w) + n * kRows * 8 > S::kSmem) --log_w;
        const int w = 1 << log_w, sums_of_all = n * (kRows * 4 << log_w);  // floats
        float* const parts = reinterpret_cast<float*>(smem);
        const float* const tops = parts + sums_of_all;  // of each part, and its weights behind them
#pragma unroll 1
        for (int d0 = 0; d0 < D; d0 += 4 * w) {
            if (d0 > 0) __syncthreads();  // the slice before has been read
            auto source = [&](int j) {
                const bool l = j < left.count;
                const int k = l ? j : j - left.count;
                if (k == 0) return l ? head_left : head_right;
                return part_of(l ? left.leader + k * left.step : right.leader + k * right.step, false);
            };
#pragma unroll 4
            for (int i = tid; i < n * (kRows << log_w); i += kThreads) {
                const int j = i / kRows >> log_w, row = i >> log_w & (kRows - 1);
                if (row < (j < left.count ? part_left : part_right).rows)
                    copy16(smem_addr(smem) + i * 16, source(j) + row * D + d0 + (i & (w - 1)) * 4, policy);
            }
            for (int i = tid; i < n * (kRows / 2); i += kThreads)
                copy16(smem_addr(tops + i * 4), source(i / (kRows / 2)) + S::kSums + i % (kRows / 2) * 4, policy);
            copy_commit();
            copy_wait<0>();
            __syncthreads();
            const int of_left = left.count > 0 ? part_left.rows : 0, of_right = right.count > 0 ? part_right.rows : 0;
#pragma unroll 1
            for (int e = tid; e < (of_left + of_right) << log_w; e += kThreads) {
                const bool l = e >> log_w < of_left;
                const Part& p = l ? part_left : part_right;
                const Join& join = l ? left : right;
                const int row = (e >> log_w) - (l ? 0 : of_left), d = (e & (w - 1)) * 4, j0 = l ? 0 : left.count;
                const float* const top_at = tops + j0 * 2 * kRows + row;
                const float* const sum_at = parts + (j0 * (kRows * 4) << log_w) + (row * 4 << log_w) + d;
                float top = -INFINITY, weight = 0.0f;
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                for (int j = 0; j < join.count; ++j) top = fmaxf(top, top_at[j * 2 * kRows]);
#pragma unroll 4
                for (int j = 0; j < join.count; ++j) {
                    const float f = share_of(top_at[j * 2 * kRows], top);
                    weight += f * top_at[j * 2 * kRows + kRows];
                    add(sum, f, *reinterpret_cast<const float4*>(sum_at + (j * (kRows * 4) << log_w)));
                }
                if (join.step * join.fan >= join.parts) {
                    finish(p, row, d0 + d, sum, top, weight);
                } else {
                    *reinterpret_cast<float4*>((l ? head_left : head_right) + row * D + d0 + d) = sum;
                    // (the maxima and weights, still read for the next slice, are left for the end)
                    if (d0 + d == 0) s_top[l ? 0 : 1][row] = top, s_weight[l ? 0 : 1][row] = weight;
                }
            }
        }
        __syncthreads();
        if (tid < 2 * kRows) {  // (of all rows, for whole sectors)
            const int which = tid / kRows, row = tid % kRows;
            const Join& join = which == 0 ? left : right;
            if (join.count > 0 && join.step * join.fan < join.parts) {
                float* const head = which == 0 ? head_left : head_right;
                head[S::kSums + row] = s_top[which][row];
                head[S::kSums + kRows + row] = s_weight[which][row];
            }
        }
        // (those that did not arrive last have left an item to others)
        if (tid < 2) {
            Join& j = s_join[tid];
            j.step = j.count > 0 && j.step * j.fan < j.parts ? j.step * j.fan : 0;
        }
    }
}

template <int D, bool EIGHT, int NT>
cudaError_t launch(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
    using S = Shape<D, EIGHT, NT>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(num_sms < kMaxGrid ? num_sms : kMaxGrid));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, EIGHT, NT>, a);
}

template <int D>
cudaError_t launch_dim(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
    const bool wide = a.rows_of_group > 8;
    if (a.k.scale != nullptr) return wide ? launch<D, true, 2>(a, num_sms, stream) : launch<D, true, 1>(a, num_sms, stream);
    return wide ? launch<D, false, 2>(a, num_sms, stream) : launch<D, false, 1>(a, num_sms, stream);
}

template <int D, bool EIGHT, int NT>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(attn_decode_kernel<D, EIGHT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, EIGHT, NT>::kSmem);
}

template <int D>
cudaError_t set_smem_dim() {
    for (const cudaError_t e : {set_smem<D, false, 1>(), set_smem<D, false, 2>(), set_smem<D, true, 1>(), set_smem<D, true, 2>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attn_decode(const DecodeArgs& args, int head_dim, int num_sms, cudaStream_t stream) {
    // Groups of up to sixteen query heads of a key-value head, of equal size as far as that goes; of up to eight where their
    // keys and values, read again from L2 by every group, are 64 MB at most for sixteen heads, as far as the page table and the
    // window say (the lengths are on the device).  Groups of eight have half the sums to join and twice the warps: sixteen
    // heads of 128 columns, 8 MB 11.4 us (groups of sixteen: 14.4), 66 MB 23.6 (26.2), 131 MB 40.9 (36.4), 262 MB 85.7 (56.2);
    // of 256 columns, 33 MB 21.3 (30.4), 66 MB 29.3 (37.5), 131 MB 41.4 (40.9); of 64, 33 MB 12.9 (13.3), 66 MB 17.2 (16.3).
    // Short sequences under a wide table get groups of sixteen: 8 of 500 tokens, table of 8192 pages, 13.3 us (exact table: 9.4), of
    // 256 columns 18.1 (12.0), in 8 bits 11.2 (8.0); 8 of 2000 15.0 (11.6).
    // More than sixteen heads: the groups of a key-value head lie one behind the other, and caches beyond L2 are read from memory once
    // a group (13 of 6000 tokens, 20 heads on each of 8: 640 MB of reads for 320, 110 us).
    DecodeArgs a = args;
    a.shared = a.heads / a.kv;
    a.per_head = (a.shared + 15) / 16;
    const int64_t longest = a.window > 0 && a.window < a.most ? a.window : a.most;
    const double bytes = (double)a.B * longest * a.kv * a.per_head * head_dim * (a.k.scale != nullptr ? 2 : 4);
    if (bytes <= (double)(1 << 26)) a.per_head = (a.shared + 7) / 8;
    a.groups = a.kv * a.per_head;
    a.rows_of_group = (a.shared + a.per_head - 1) / a.per_head;
    switch (head_dim) {
        case 64: return launch_dim<64>(a, num_sms, stream);
        case 128: return launch_dim<128>(a, num_sms, stream);
        case 256: return launch_dim<256>(a, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t attn_decode_set_attributes() {
    for (const cudaError_t e : {set_smem_dim<64>(), set_smem_dim<128>(), set_smem_dim<256>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

size_t attn_decode_counters(int num_sms) { return (size_t)(num_sms < kMaxGrid ? num_sms : kMaxGrid) * 4; }
size_t attn_decode_parts(int num_sms, int head_dim) {
    // two parts a CTA of up to sixteen rows, and its warps' sums
    return (size_t)(num_sms < kMaxGrid ? num_sms : kMaxGrid) * (2 * (16 * head_dim + 32) + kScratchRows * head_dim);
}

}  // namespace arf
