// attn_decode.cu -- attention of one new token of each sequence over its paged
// keys and values:
//
//   s_j = scale q . k_j; out = sum_j softmax(s)_j v_j; lse = log sum_j exp(s_j)
//
// in one pass with a running maximum m, sum l and weighted sum of values o: tokens with
// scores s (times log2(e)) turn them into m' = max(m, s), l 2^(m - m') + sum 2^(s - m'),
// o 2^(m - m') + sum 2^(s - m') v.
//
// Work.  Up to sixteen query heads of a key-value head are the rows of a matrix
// instruction (m16n8k16) and share what is read.  Such a group of one sequence is an item,
// its tokens come in units of TOK; the units of all items in a row are cut into one range
// per SM, by the lengths on the device, so lengths of any mixture keep every SM equally
// busy and a captured launch serves any.  An item that a range's end cuts is joined from
// its parts: the last CTA of each sixteen parts to arrive adds them up, the last of those
// the sums, always in the order of the parts.  No CTA waits for another.
//
// A CTA's range is cut into eight for its warps.  A warp streams its units through a ring
// of its own in shared memory, keys and values in turn, by 16-byte asynchronous copies that
// run ahead across items, so that no barrier stands in the stream; the places of a unit's
// tokens are looked up a unit earlier still.  Items that lie within a warp's share are
// finished from its registers; what is cut is added up once, at the end of the CTA, in the
// order of the warps.
//
// Roundings: scores, maxima, sums and o are fp32.  Weights go to the matrix instruction as
// two bf16 (their rounding and its remainder: 2^-17, where one bf16 would add 0.7 times the
// output's own rounding); with 8-bit values as halves (2^-11), whose products are
// exact, q then scaled by a power of two a row to the halves' range.
#include "attn_common.cuh"

#include <cuda_fp16.h>

namespace arf {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;          // query heads of an item
constexpr int kRing = 24576;       // bytes of a warp's ring
constexpr int kMaxGrid = 256;
constexpr int kFan = 16;           // parts that are joined at a time
constexpr int kMinUnits = 4;       // of a warp, while there are SMs left
constexpr float kLazy = 8.0f;      // scores (log2) may pass the reference by so much before it moves
constexpr float kLn2 = 0.6931471805599453f;

// Tokens of a unit: rows of 128 bytes and less come by 32, longer ones by 16.
constexpr int unit_tokens(int D, bool eight) { return D * (eight ? 1 : 2) <= 128 ? 32 : 16; }

template <int D, bool EIGHT>
struct Shape {
    static constexpr int kTok = unit_tokens(D, EIGHT);
    static constexpr int kRow = D * (EIGHT ? 1 : 2);  // bytes of a key
    static constexpr int kChunks = kRow / 16;
    static constexpr int kHalf = kTok * kRow;  // bytes of a unit's keys (or values)
    static constexpr int kHalves = kRing / kHalf;
    static constexpr int kLead = kHalves - 1;  // halves that are asked for ahead
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kSmem + 4096 <= 232448, "shared memory of a CTA");
    static_assert(kRows * D * 4 <= kRing, "a warp's part of an item, in its ring");
    // where chunk c of row r lies, so that eight rows' chunks c are in eight different groups of banks
    __device__ static int place(int r, int c) {
        return r * kRow + ((kChunks >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & (kChunks - 1))) << 4);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    const int bytes = there ? 16 : 0;  // the rest is zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

template <bool EIGHT>
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if (EIGHT)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Two maxima's share: 2^(m - top), 0 for a part without tokens.
__device__ __forceinline__ float share_of(float m, float top) { return ex2(m - (top == -INFINITY ? 0.0f : top)); }

// A warp's share of an item: units [u0, u1) of its n.
struct Segment {
    int b, group;    // sequence; group of query heads
    int start, len;  // tokens looked at
    int u0, u1, n;
};

// Walks the segments of a range of units.
template <int TOK>
struct Walk {
    int b, group, u;
    int start, len, n;
    int64_t left;  // units of the range that are not handed out

    __device__ void sequence(const DecodeArgs& a) {
        len = checked_length(a, b, false);
        start = a.window > 0 && len > a.window ? len - a.window : 0;
        n = (int)(((int64_t)len - start + TOK - 1) / TOK);
    }
    __device__ bool next(const DecodeArgs& a, int groups, Segment* s) {
        if (left <= 0) return false;
        if (u == n) {  // the item is done: the next one that has units (there is one, for some are left)
            u = 0;
            if (++group == groups) {
                group = 0;
                do {
                    ++b;
                    sequence(a);
                } while (n == 0);
            }
        }
        const int take = (int)(left < n - u ? left : n - u);
        *s = Segment{b, group, start, len, u, u + take, n};
        u += take;
        left -= take;
        return true;
    }
};

// Quotients of numbers that are small as a rule.
__device__ __forceinline__ int64_t quotient64(int64_t n, int64_t d) {
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
    int b, group, n;
};

// A CTA's part in memory holds [kRows, D] sums, then kRows maxima and kRows sums of weights; behind the parts, two a CTA,
// lie the sums that its warps leave in mid-stream.
template <int D>
constexpr int kPart = kRows * D + 2 * kRows;

template <int D, bool EIGHT>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const __grid_constant__ DecodeArgs a, int groups, int rows_of_group) {
    using S = Shape<D, EIGHT>;
    constexpr int TOK = S::kTok, kTiles = TOK / 8, kSteps = D / 16;
    constexpr float kOffset = EIGHT ? 7.0f : 0.0f;  // halves: weights up to 2^(8 + 7), so that small ones keep their bits
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[2 * kWarps][kRows], s_l[2 * kWarps][kRows], s_fm[kRows], s_fl[kRows];
    __shared__ float s_share[2 * kWarps][kRows], s_top[2 * kWarps][kRows], s_weight[2 * kWarps][kRows];
    __shared__ Part s_part[2 * kWarps];  // of each warp: what it began with, if it went on; what it ended with
    __shared__ int s_run[2 * kWarps + 1];
    __shared__ int64_t s_scan[kWarps];
    __shared__ int64_t s_first[kWarps];  // units of the found sequence before the warp's first
    __shared__ int s_b[kWarps], s_last;
    __shared__ unsigned s_mask[kWarps][8];
    pdl_wait();  // no global memory access before this point
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const int shared_heads = a.heads / a.kv, per_head = groups / a.kv;

    // ---- the ranges of this CTA's warps: equal ones, so that the last may be short or empty
    int64_t total, each;
    {
        const int per_thread = (a.B + kThreads - 1) / kThreads, b0 = tid * per_thread, b1 = min(a.B, b0 + per_thread);
        auto units = [&](int b) {
            const int len = checked_length(a, b, blockIdx.x == 0);
            const int n = a.window > 0 && len > a.window ? a.window : len;
            return ((int64_t)n + TOK - 1) / TOK * groups;
        };
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += units(b);
        const int64_t upto = warp_scan(mine, lane);
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        int64_t before = upto - mine;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        each = max((int64_t)kMinUnits, quotient64(total + gridDim.x * kWarps - 1, gridDim.x * kWarps));
        for (int w = 0; w < kWarps; ++w) {  // whose first unit is here?
            const int64_t from = each * (blockIdx.x * kWarps + w);
            if (before <= from && from < before + mine) {
                int b = b0;
                int64_t skip = from - before;
                if (per_thread > 1)
                    for (int64_t n; (n = units(b)) <= skip; ++b) skip -= n;
                s_b[w] = b;
                s_first[w] = skip;
            }
        }
        __syncthreads();
    }
    const int64_t from = each * (blockIdx.x * kWarps + warp);
    const int64_t begin = each * (blockIdx.x * kWarps), end = begin + each * kWarps;  // the CTA's
    Walk<TOK> walk;
    walk.left = min(each, total - from);
    if (walk.left > 0) {
        walk.b = s_b[warp];
        walk.sequence(a);
        walk.group = (int)quotient64(s_first[warp], walk.n);
        walk.u = (int)(s_first[warp] - (int64_t)walk.group * walk.n);
    }

    // ---- the stream of this warp's units: looked up, then asked for
    const uint32_t ring = smem_addr(smem) + warp * kRing;
    Walk<TOK> ahead = walk;
    Segment ask;
    int ask_u = 0;             // unit that is asked for next
    int ask_last = 0;          // last page of its sequence
    bool asking = ahead.next(a, groups, &ask);
    int64_t k_at = -1, v_at = -1;  // places of this lane's token of the unit that is being asked for
    bool live = false;             // there is such a unit
    unsigned asked = 0;            // units asked for
    int fill = 0;                  // slot of the ring that is filled next
    // the page table's entries from table_at on: this lane's of the first 32 and of the next 32
    int table_at = 0, entry = 0, entry_next = 0;
    auto page_of = [&](int64_t token) { return (int)((uint64_t)token * a.page_mul >> (31 + a.page_shift)); };
    auto table_entry = [&](int index) {  // -1 behind the sequence's last
        return index <= ask_last ? a.table[ask.b * a.table_stride + index] : -1;
    };
    auto look_up = [&]() {  // a new segment
        ask_u = ask.u0;
        ask_last = page_of(ask.len - 1);
        table_at = page_of(ask.start + (int64_t)ask_u * TOK);
        entry = table_entry(table_at + lane);
        entry_next = table_entry(table_at + 32 + lane);
    };
    if (asking) look_up();

    auto issue = [&](bool keys) {
        if (keys) {
            k_at = v_at = -1;
            live = asking;
            if (asking) {
                const int head = ask.group / per_head;
                const int64_t first = ask.start + (int64_t)ask_u * TOK, token = first + lane;
                while (page_of(first) - table_at >= 32) {
                    table_at += 32;
                    entry = entry_next;
                    entry_next = table_entry(table_at + 32 + lane);
                }
                const int index = page_of(token), in_page = (int)token - index * a.page_size, at = index - table_at;
                const int here = __shfl_sync(0xffffffffu, entry, at & 31), next = __shfl_sync(0xffffffffu, entry_next, at & 31);
                const int page = at < 32 ? here : next;
                const bool wanted = lane < TOK && token < ask.len, there = wanted && (unsigned)page < (unsigned)a.pages;
                if (wanted && !there) atomicOr(a.err, kErrPageRange);
                if (there) {
                    k_at = page * a.k.page + in_page * a.k.token + head * a.k.head;
                    v_at = page * a.v.page + in_page * a.v.token + head * a.v.head;
                }
                const unsigned mask = __ballot_sync(0xffffffffu, there);
                if (lane == 0) s_mask[warp][asked & 7] = mask;
                ++asked;
                if (++ask_u == ask.u1) {
                    asking = ahead.next(a, groups, &ask);
                    if (asking) look_up();
                }
            }
        }
        const int64_t at = keys ? k_at : v_at;
        const uint8_t* base = keys ? a.k.data : a.v.data;
        const uint32_t slot = ring + fill * S::kHalf;
        if (__any_sync(0xffffffffu, at >= 0)) {
#pragma unroll
            for (int i = 0; i < TOK * S::kChunks / 32; ++i) {
                const int r = (i * 32 + lane) / S::kChunks, c = (i * 32 + lane) % S::kChunks;
                const int64_t row = __shfl_sync(0xffffffffu, at, r);
                copy16(slot + S::place(r, c), base + (row < 0 ? 0 : row + c * 16), row >= 0);
            }
        } else if (live) {  // no token on a page of the cache: zeros
            for (int i = 0; i < S::kHalf / 512; ++i)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(slot + (i * 32 + lane) * 16), "r"(0) : "memory");
        }
        copy_commit();
        fill = fill + 1 == S::kHalves ? 0 : fill + 1;
    };
#pragma unroll 1
    for (int i = 0; i < S::kLead; ++i) issue(i % 2 == 0);

    // rows without tokens: zeros, dealt to the warps
    for (int64_t b = blockIdx.x + (int64_t)gridDim.x * warp; b < a.B; b += gridDim.x * kWarps)
        if (checked_length(a, (int)b, false) == 0) {
            for (int j = lane; j < a.heads * D / 8; j += 32) st_global16(a.out + b * a.heads * D + j * 8, make_uint4(0, 0, 0, 0));
            if (a.lse != nullptr)
                for (int j = lane; j < a.heads; j += 32) a.lse[b * a.heads + j] = -INFINITY;
        }
    if (begin >= total) return;

    auto mid_stream = [&](int w) { return a.part + (int64_t)gridDim.x * 2 * kPart<D> + ((int64_t)blockIdx.x * kWarps + w) * kRows * D; };
    auto lse_of = [&](float top, float weight) { return weight == 0.0f ? -INFINITY : (top - kOffset + log2f(weight)) * kLn2; };

    // ---- segments
    uint32_t q[kSteps][4];
    float q_scale[2];  // of the scores, rows g and g + 8: log2(e) * scale * scale of the keys * power of two of the row
    auto load_q = [&](const Segment& s) {
        const int head = s.group / per_head, part = s.group - head * per_head;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = part * rows_of_group + g + 8 * r;
            const bool there = g + 8 * r < rows_of_group && row < shared_heads;
            const uint16_t* src = a.q + ((int64_t)s.b * a.heads + head * shared_heads + (there ? row : 0)) * D;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                // columns of a step: 2 t4 (+1) and 2 t4 + 8 (+1); with bytes 4 t4 .. 4 t4 + 3, the order that their keys come in
                uint2 v;
                if (EIGHT) {
                    v = *reinterpret_cast<const uint2*>(src + i * 16 + t4 * 4);
                } else {
                    v.x = *reinterpret_cast<const uint32_t*>(src + i * 16 + t4 * 2);
                    v.y = *reinterpret_cast<const uint32_t*>(src + i * 16 + t4 * 2 + 8);
                }
                q[i][r] = there ? v.x : 0;
                q[i][r + 2] = there ? v.y : 0;
            }
            q_scale[r] = EIGHT ? a.scale * a.k.scale[head] : a.scale;
        }
    };
    auto prepare_q = [&]() {
        if constexpr (EIGHT) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int c = r; c < 4; c += 2)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[i][c] << 16)), fabsf(__uint_as_float(q[i][c] & 0xffff0000u))));
                top = quad_max(top);
                // the power of two that brings the row's largest value to [1, 2) (or next to it, at the ends of the range)
                int e = (int)(__float_as_uint(top) >> 23) - 127;
                e = e < -126 ? -126 : e > 126 ? 126 : e;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int c = r; c < 4; c += 2)
                        q[i][c] = pack_f16x2(__uint_as_float(q[i][c] << 16) * down, __uint_as_float(q[i][c] & 0xffff0000u) * down);
                q_scale[r] *= up;
            }
        }
    };

    int take = 0;        // slot of the ring that is used next
    unsigned taken = 0;  // units used
    int64_t position = from;
    Segment seg;
    bool more = walk.next(a, groups, &seg);
    if (lane < 2) s_part[2 * warp + lane].item = -1;
    __syncwarp();
    if (more) load_q(seg);
    while (more) {
        prepare_q();
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;

        for (int u = seg.u0; u < seg.u1; ++u) {
            // scores of TOK tokens
            __syncwarp();  // the slot that is filled now has been read by all lanes
            issue(S::kLead % 2 == 0);
            copy_wait<S::kLead>();
            __syncwarp();
            float s[kTiles][4];
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
            uint32_t slot = ring + take * S::kHalf;
            take = take + 1 == S::kHalves ? 0 : take + 1;
            if (EIGHT) {
                // a matrix is 8 tokens by 16 bytes: one step of the columns
#pragma unroll
                for (int i = 0; i < kSteps; i += 2)
#pragma unroll
                    for (int h = 0; h < TOK / 16; ++h) {
                        uint32_t r[4];
                        ldmatrix4(r, slot + S::place(h * 16 + (lane >> 4) * 8 + (lane & 7), i + ((lane >> 3) & 1)));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma<true>(s[h * 2 + (j >> 1)], q[i + (j & 1)], e4m3x2_to_f16x2((uint16_t)r[j]), e4m3x2_to_f16x2((uint16_t)(r[j] >> 16)));
                    }
            } else {
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int h = 0; h < TOK / 16; ++h) {
                        uint32_t r[4];
                        ldmatrix4(r, slot + S::place(h * 16 + (lane >> 4) * 8 + (lane & 7), i * 2 + ((lane >> 3) & 1)));
                        mma<false>(s[h * 2], q[i], r[0], r[1]);
                        mma<false>(s[h * 2 + 1], q[i], r[2], r[3]);
                    }
            }
            // their weights
            const unsigned mask = s_mask[warp][taken++ & 7] >> (2 * t4);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = mask >> (i * 8 + (j & 1)) & 1 ? s[i][j] * q_scale[j >> 1] : -INFINITY;
                    top[j >> 1] = fmaxf(top[j >> 1], s[i][j]);
                }
            float keep[2];
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = quad_max(top[r]);
                keep[r] = 1.0f;
                if (top[r] > m[r] + kLazy) {  // (the first finite score passes minus infinity)
                    keep[r] = ex2(m[r] - top[r]);
                    m[r] = top[r];
                    l[r] *= keep[r];
                    moved = true;
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= keep[j >> 1];
            }
            const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0] - kOffset, m[1] == -INFINITY ? 0.0f : m[1] - kOffset};
            uint32_t p[TOK / 16][4], rest[TOK / 16][4];
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float x = ex2(s[i][2 * r] - base[r]), y = ex2(s[i][2 * r + 1] - base[r]);
                    l[r] += x + y;
                    const int c = r + 2 * (i & 1);
                    if (EIGHT) {
                        p[i / 2][c] = pack_f16x2(x, y);
                    } else {
                        const uint32_t w = pack_bf16x2(x, y);
                        p[i / 2][c] = w;
                        rest[i / 2][c] = pack_bf16x2(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xffff0000u));
                    }
                }
            // and values
            __syncwarp();
            issue(S::kLead % 2 == 1);
            copy_wait<S::kLead>();
            __syncwarp();
            slot = ring + take * S::kHalf;
            take = take + 1 == S::kHalves ? 0 : take + 1;
            if (EIGHT) {
                // transposed by pairs of bytes: a register holds two columns of two tokens, even columns make one tile, odd
                // ones another
#pragma unroll
                for (int c = 0; c < kSteps; c += 2)
#pragma unroll
                    for (int h = 0; h < TOK / 16; ++h) {
                        uint32_t r[4];
                        ldmatrix4_trans(r, slot + S::place(h * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c + (lane >> 4)));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t x = __byte_perm(r[2 * j], 0, 0x3120), y = __byte_perm(r[2 * j + 1], 0, 0x3120);
                            mma<true>(o[2 * (c + j)], p[h], e4m3x2_to_f16x2((uint16_t)x), e4m3x2_to_f16x2((uint16_t)y));
                            mma<true>(o[2 * (c + j) + 1], p[h], e4m3x2_to_f16x2((uint16_t)(x >> 16)), e4m3x2_to_f16x2((uint16_t)(y >> 16)));
                        }
                    }
            } else {
#pragma unroll
                for (int c = 0; c < kSteps; ++c)
#pragma unroll
                    for (int h = 0; h < TOK / 16; ++h) {
                        uint32_t r[4];
                        ldmatrix4_trans(r, slot + S::place(h * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c * 2 + (lane >> 4)));
                        mma<false>(o[2 * c], p[h], r[0], r[1]);
                        mma<false>(o[2 * c + 1], p[h], r[2], r[3]);
                        mma<false>(o[2 * c], rest[h], r[0], r[1]);
                        mma<false>(o[2 * c + 1], rest[h], r[2], r[3]);
                    }
            }
        }

        // ---- the item, or this warp's part of it
        const Segment done = seg;
        more = walk.next(a, groups, &seg);
        if (more) load_q(seg);
        const int64_t item = position - done.u0;
        position += done.u1 - done.u0;
        const bool whole = done.u0 == 0 && done.u1 == done.n;
        const int kv_head = done.group / per_head, first_row = (done.group - kv_head * per_head) * rows_of_group;
        const int rows = min(rows_of_group, shared_heads - first_row);
        const int which = 2 * warp + (more ? 0 : 1);
        const int64_t out_row = (int64_t)done.b * a.heads + kv_head * shared_heads + first_row;
        l[0] = quad_sum(l[0]);
        l[1] = quad_sum(l[1]);
        __syncwarp();  // all lanes have read the ring
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            if (row >= rows) continue;
            if (whole) {
                const float f = l[r] == 0.0f ? 0.0f : (EIGHT ? a.v.scale[kv_head] : 1.0f) / l[r];
                uint16_t* to = a.out + (out_row + row) * D;
#pragma unroll
                for (int i = 0; i < D / 8; i += 2) {
                    if (EIGHT) {
                        *reinterpret_cast<uint2*>(to + i * 8 + t4 * 4) =
                            make_uint2(pack_bf16x2(o[i][2 * r] * f, o[i + 1][2 * r] * f), pack_bf16x2(o[i][2 * r + 1] * f, o[i + 1][2 * r + 1] * f));
                    } else {
                        *reinterpret_cast<uint32_t*>(to + i * 8 + t4 * 2) = pack_bf16x2(o[i][2 * r] * f, o[i][2 * r + 1] * f);
                        *reinterpret_cast<uint32_t*>(to + i * 8 + 8 + t4 * 2) = pack_bf16x2(o[i + 1][2 * r] * f, o[i + 1][2 * r + 1] * f);
                    }
                }
                if (a.lse != nullptr && t4 == 0) a.lse[out_row + row] = lse_of(m[r], l[r]);
                continue;
            }
            // (the stream has ended when the last part is written: its ring is free)
            float* to = (more ? mid_stream(warp) : reinterpret_cast<float*>(smem + warp * kRing)) + row * D;
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                if (EIGHT) {
                    *reinterpret_cast<float4*>(to + i * 8 + t4 * 4) = make_float4(o[i][2 * r], o[i + 1][2 * r], o[i][2 * r + 1], o[i + 1][2 * r + 1]);
                } else {
                    *reinterpret_cast<float2*>(to + i * 8 + t4 * 2) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                    *reinterpret_cast<float2*>(to + i * 8 + 8 + t4 * 2) = make_float2(o[i + 1][2 * r], o[i + 1][2 * r + 1]);
                }
            }
            if (t4 == 0) {
                s_m[which][row] = m[r];
                s_l[which][row] = l[r];
            }
        }
        if (!whole && lane == 0) s_part[which] = Part{item, done.b, done.group, done.n};
    }
    pdl_trigger();

    // ---- what the warps share: runs of parts of one item
    __syncthreads();
    Part mine{-1, 0, 0, 0};
    if (lane < 2 * kWarps) mine = s_part[lane];
    const unsigned there = __ballot_sync(0xffffffffu, mine.item >= 0), below = there & ((1u << lane) - 1);
    const int64_t previous = __shfl_sync(0xffffffffu, mine.item, below ? 31 - __clz(below) : lane);
    const bool starts = mine.item >= 0 && (below == 0 || previous != mine.item);
    const unsigned start_mask = __ballot_sync(0xffffffffu, starts);
    const int runs = __popc(start_mask);
    if (runs == 0) return;
    if (warp == 0 && starts) s_run[__popc(start_mask & ((1u << lane) - 1))] = lane;
    if (tid == 0) s_run[runs] = 2 * kWarps;
    __syncthreads();

    // a row's output from its sums
    auto finish = [&](const Part& p, int row, int d, float4 sum, float top, float weight) {
        const int kv_head = p.group / per_head;
        const int64_t out_row = (int64_t)p.b * a.heads + kv_head * shared_heads + (p.group - kv_head * per_head) * rows_of_group + row;
        const float f = weight == 0.0f ? 0.0f : (EIGHT ? a.v.scale[kv_head] : 1.0f) / weight;
        *reinterpret_cast<uint2*>(a.out + out_row * D + d) = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
        if (a.lse != nullptr && d == 0) a.lse[out_row] = lse_of(top, weight);
    };
    auto rows_of = [&](const Part& p) { return min(rows_of_group, shared_heads - p.group % per_head * rows_of_group); };
    // a CTA's part of an item: one for an item that began in a range before, one for an item that begins in this one
    auto part_of = [&](int cta, bool begins) { return a.part + ((int64_t)cta * 2 + (begins ? 1 : 0)) * kPart<D>; };

    // what each part counts, and the runs' maxima and weights
    {
        static_assert(kThreads == 2 * kWarps * kRows, "a thread for each part and row");
        const int j = tid / kRows, row = tid % kRows;
        const int first = 31 - __clz(start_mask & ((2u << j) - 1));  // (the run of part j begins here)
        if (there >> j & 1) {
            const unsigned behind = start_mask & ~((2u << first) - 1);
            const unsigned of_run = there & ~((1u << first) - 1) & (behind ? (1u << (__ffs(behind) - 1)) - 1 : ~0u);
            float top = -INFINITY, weight = 0.0f;
            for (unsigned i = of_run; i; i &= i - 1) top = fmaxf(top, s_m[__ffs(i) - 1][row]);
            for (unsigned i = of_run; i; i &= i - 1) weight += share_of(s_m[__ffs(i) - 1][row], top) * s_l[__ffs(i) - 1][row];
            s_share[j][row] = share_of(s_m[j][row], top);
            s_top[j][row] = top;
            s_weight[j][row] = weight;
        }
    }
    __syncthreads();
    for (int i = tid; i < runs * kRows * (D / 4); i += kThreads) {
        const int run = i / (kRows * (D / 4)), row = i / (D / 4) % kRows, d = i % (D / 4) * 4;
        const int j0 = s_run[run], j1 = s_run[run + 1];
        const Part p = s_part[j0];
        if (row >= rows_of(p)) continue;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = j0; j < j1; ++j)
            if (there >> j & 1) {
                const float* from_part = j & 1 ? reinterpret_cast<const float*>(smem + (j >> 1) * kRing) : mid_stream(j >> 1);
                const float4 v = *reinterpret_cast<const float4*>(from_part + row * D + d);
                const float f = s_share[j][row];
                sum.x += f * v.x;
                sum.y += f * v.y;
                sum.z += f * v.z;
                sum.w += f * v.w;
            }
        if (p.item >= begin && p.item + p.n <= end) {
            finish(p, row, d, sum, s_top[j0][row], s_weight[j0][row]);
        } else {
            float* to = part_of(blockIdx.x, p.item >= begin);
            *reinterpret_cast<float4*>(to + row * D + d) = sum;
            if (d == 0) {
                to[kRows * D + row] = s_top[j0][row];
                to[kRows * D + kRows + row] = s_weight[j0][row];
            }
        }
    }

    // ---- what CTAs share: sixteen parts at a time, then the sixteens
    auto owner = [&](int64_t unit) { return (int)quotient64(unit, each * kWarps); };
    for (int run = 0; run < runs; run += max(1, runs - 1)) {  // the first and the last
        const Part p = s_part[s_run[run]];
        if (p.item >= begin && p.item + p.n <= end) continue;
        const int first = owner(p.item), last = owner(p.item + p.n - 1);
        const int fans = (last - first + kFan) / kFan, rows = rows_of(p);
        for (int level = 0; level < 2; ++level) {
            const int fan = ((int)blockIdx.x - first) / kFan;
            const int leader = level == 0 ? first + fan * kFan : first, step = level == 0 ? 1 : kFan;
            const int count = level == 0 ? min(kFan, last - leader + 1) : fans;
            // this level's counter, of the leader's part
            unsigned* counter = a.count + (leader * 2 + (leader == first ? 1 : 0)) * 2 + level;
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                const unsigned before = atomicAdd(counter, 1);
                s_last = before == (unsigned)count - 1;
                if (s_last) {
                    *counter = 0;
                    __threadfence();
                }
            }
            __syncthreads();
            if (!s_last) break;
            auto part_at = [&](int i) { return part_of(leader + i * step, leader + i * step == first); };
            const bool end_here = level == 1 || fans == 1;
            for (int i = tid; i < rows * (D / 4); i += kThreads) {
                const int r = i / (D / 4), d = i % (D / 4) * 4;
                // everything is asked for before anything is used
                float top = -INFINITY, weight = 0.0f, pm[kFan], pl[kFan];
                float4 v[kFan], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < kFan; ++j) {
                    const float* from_part = part_at(j < count ? j : 0);
                    pm[j] = __ldcg(from_part + kRows * D + r);
                    pl[j] = __ldcg(from_part + kRows * D + kRows + r);
                    v[j] = __ldcg(reinterpret_cast<const float4*>(from_part + r * D + d));
                }
#pragma unroll
                for (int j = 0; j < kFan; ++j)
                    if (j < count) top = fmaxf(top, pm[j]);
#pragma unroll
                for (int j = 0; j < kFan; ++j)
                    if (j < count) {
                        const float f = share_of(pm[j], top);
                        weight += f * pl[j];
                        sum.x += f * v[j].x;
                        sum.y += f * v[j].y;
                        sum.z += f * v[j].z;
                        sum.w += f * v[j].w;
                    }
                if (end_here) {
                    finish(p, r, d, sum, top, weight);
                } else {
                    *reinterpret_cast<float4*>(part_at(0) + r * D + d) = sum;  // (no other thread reads these)
                    if (d == 0) {
                        s_fm[r] = top;
                        s_fl[r] = weight;
                    }
                }
            }
            if (end_here) break;
            __syncthreads();  // all have read the maxima and sums
            if (tid < rows) {
                part_at(0)[kRows * D + tid] = s_fm[tid];
                part_at(0)[kRows * D + kRows + tid] = s_fl[tid];
            }
        }
    }
}

template <int D, bool EIGHT>
cudaError_t launch(const DecodeArgs& a, int num_sms, cudaStream_t stream, bool pdl) {
    // groups of up to sixteen query heads of a key-value head, of equal size as far as that goes
    const int shared_heads = a.heads / a.kv, per = (shared_heads + kRows - 1) / kRows;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(num_sms < kMaxGrid ? num_sms : kMaxGrid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<D, EIGHT>::kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, EIGHT>, a, per * a.kv, (shared_heads + per - 1) / per);
}

template <int D, bool EIGHT>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(attn_decode_kernel<D, EIGHT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, EIGHT>::kSmem);
}

}  // namespace

cudaError_t launch_attn_decode(const DecodeArgs& a, int head_dim, int num_sms, cudaStream_t stream, bool pdl) {
    const bool eight = a.k.scale != nullptr;
    switch (head_dim) {
        case 64: return eight ? launch<64, true>(a, num_sms, stream, pdl) : launch<64, false>(a, num_sms, stream, pdl);
        case 128: return eight ? launch<128, true>(a, num_sms, stream, pdl) : launch<128, false>(a, num_sms, stream, pdl);
        case 256: return eight ? launch<256, true>(a, num_sms, stream, pdl) : launch<256, false>(a, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

cudaError_t attn_decode_set_attributes() {
    for (const cudaError_t e : {set_smem<64, false>(), set_smem<64, true>(), set_smem<128, false>(), set_smem<128, true>(),
                                set_smem<256, false>(), set_smem<256, true>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

size_t attn_decode_counters(int num_sms) { return (size_t)(num_sms < kMaxGrid ? num_sms : kMaxGrid) * 4; }
size_t attn_decode_parts(int num_sms, int head_dim) {
    return (size_t)(num_sms < kMaxGrid ? num_sms : kMaxGrid) * (2 * (kRows * head_dim + 2 * kRows) + kWarps * kRows * head_dim);
}

}  // namespace arf
