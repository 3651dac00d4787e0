// moe_experts.cu -- the experts' products of a few tokens.
//
//   h = W13_e x[t];  a = silu(h[0:I]) * h[I:2I];  y[t] += w[t,k] * W2_e a,   e = ids[t,k]
//
// Two kernels: the first writes the activations a of every (token, expert)
// slot, the second the sums y; both wait on memory with bf16 weights (64 tokens
// with 8 of 256 experts of 3 x 256 x 7168: 367 us, 0.98 of the copy rate; one token
// 18.6 us, 0.70: start, end and the way from one kernel to the other take 6 us).
// Both read each chosen expert's weights from memory once, whichever tokens chose
// it (from L2 again for every item of its tokens: 64 tokens with 2 of 8 experts
// reach 0.44), and deal weight rows evenly over the SMs: the first kernel flattens (chosen expert, row pair), the second gives every CTA
// its share of the H output rows for all chosen experts, so that the sum over
// a token's experts never leaves the CTA: no atomics, one rounding.
//
// The activations travel as a bf16 high part and a bf16 low part (16 bits of
// mantissa together), columns 0-3 and 4-7 of the matrix instruction's eight:
// rounding them to one bf16 would make the result's error 1.4 times that of its
// own rounding, and up to four tokens per expert the second part costs nothing.
#include <atomic>

#include "moe_common.cuh"

namespace arf {
namespace {

// Tokens per item of the first kernel (a power of two), and of the second.  The
// activations of the items that a CTA meets stay in shared memory if they are few
// (four of 7168 values); an expert's tokens beyond an item's take its rows out of
// L2 again.  So: small items where experts have few tokens on average.  (16 tokens
// with 8 of 256 experts of 2 x 256 x 7168 in 4 bits: with items of up to eight the
// last CTA of the first kernel ended 15 us after the others, which had not to
// stage activations twice, with four 10 us and with two 1 us.)
int chunk_first(int T, int K, int E) { return T * K > 4 * E ? 8 : T * K > E ? 4 : 2; }
constexpr int kChunk2 = 4;

// The chosen experts, in order, each with the tokens that chose it, in order,
// cut into items of up to `chunk` tokens.  In shared memory, for `slots` = T * K
// entries.
struct Items {
    float* w;          // entries: routing weight
    uint16_t* slot;    // entries: token * K + k
    uint16_t* expert;  // items
    uint16_t* off;     // items: first entry
    uint16_t* at;      // experts: first entry
    int* part;         // sums over the warps, then the number of items
    uint8_t* token;    // entries
    uint8_t* n;        // items: entries
    __host__ __device__ static int bytes(int slots, int experts) { return (slots * 12 + experts * 2 + (2 * kMvWarps + 1) * 4 + 15) / 16 * 16; }
    __device__ Items(uint8_t* p, int slots, int experts) {
        w = reinterpret_cast<float*>(p);
        part = reinterpret_cast<int*>(w + slots);
        slot = reinterpret_cast<uint16_t*>(part + 2 * kMvWarps + 1);
        expert = slot + slots;
        off = expert + slots;
        at = off + slots;
        token = reinterpret_cast<uint8_t*>(at + experts);
        n = token + slots;
    }
    __device__ int count() const { return uniform(part[2 * kMvWarps]); }
};

// Called by all threads of a CTA.  A token that names an expert twice gets one
// entry with the sum of its weights (a single token: an item each).  -1 names no expert; other values outside
// [0, E) are skipped too and flagged.  mask: scratch, two words per expert (the
// tokens that chose it), free again afterwards: it may be the ring's memory, since
// each thread's accesses to it are ordered before copies that follow the barrier.
__device__ void build_items(const Items& it, uint32_t (*mask)[2], const ExpertsArgs& a, int chunk) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.T == 1) {  // every slot an item: one warp does it
        if (warp == 0) {
            const int e = lane < a.K ? a.ids[lane] : -1;
            const float w = lane < a.K ? a.weights[lane] : 0.0f;
            const bool ok = (unsigned)e < (unsigned)a.E;
            const unsigned all = __ballot_sync(0xffffffffu, ok);
            const int i = __popc(all & ((1u << lane) - 1));
            if (ok) {
                it.expert[i] = e;
                it.off[i] = i;
                it.slot[i] = lane;
                it.n[i] = 1;
                it.token[i] = 0;
                it.w[i] = w;
            } else if (e != -1) {
                atomicOr(a.err, kErrExpertRange);
            }
            if (lane == 0) it.part[2 * kMvWarps] = __popc(all);
        }
        __syncthreads();
        return;
    }
    // a thread's slots, and their weights, asked for together
    constexpr int kMine = (kMoeMaxSlots + kMvThreads - 1) / kMvThreads;
    const int slots = a.T * a.K;
    int mine[kMine];
    float weight[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int s = tid + i * kMvThreads;
        mine[i] = s < slots ? a.ids[s] : -1;
        weight[i] = s < slots ? a.weights[s] : 0.0f;
    }
    int* twice = it.part + 2 * kMvWarps;  // some token names an expert twice; later the number of items
    if (tid == 0) *twice = 0;
    for (int e = tid; e < a.E; e += kMvThreads) mask[e][0] = mask[e][1] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int e = mine[i], t = quotient(tid + i * kMvThreads, a.K);
        if ((unsigned)e < (unsigned)a.E) {
            if (atomicOr(&mask[e][t >> 5], 1u << (t & 31)) >> (t & 31) & 1) *twice = 1;
        } else if (e != -1) {
            atomicOr(a.err, kErrExpertRange);
        }
    }
    __syncthreads();
    const bool dedupe = *twice != 0;
    static_assert(kMoeMaxExperts <= kMvThreads, "one expert per thread");
    const int n = tid < a.E ? __popc(mask[tid][0]) + __popc(mask[tid][1]) : 0;
    const int m = (n + chunk - 1) >> (chunk == 8 ? 3 : chunk == 4 ? 2 : 1);
    int ni = m, ne = n;  // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, ni, o), v = __shfl_up_sync(0xffffffffu, ne, o);
        if (lane >= o) {
            ni += u;
            ne += v;
        }
    }
    if (lane == 31) {
        it.part[warp] = ni;
        it.part[kMvWarps + warp] = ne;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ni += it.part[w];
        ne += it.part[kMvWarps + w];
    }
    if (tid == kMvThreads - 1) it.part[2 * kMvWarps] = ni;
    if (n > 0) {
        it.at[tid] = ne - n;
        for (int j = 0; j < m; ++j) {
            it.expert[ni - m + j] = tid;
            it.off[ni - m + j] = ne - n + j * chunk;
            it.n[ni - m + j] = min(chunk, n - j * chunk);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int s = tid + i * kMvThreads, e = mine[i];
        if ((unsigned)e >= (unsigned)a.E) continue;
        const int t = quotient(s, a.K);
        float w = weight[i];
        if (dedupe) {
            const int k = s - t * a.K;
            bool first = true;
            for (int j = 0; j < k; ++j) first = first && a.ids[t * a.K + j] != e;
            if (!first) continue;
            for (int j = k + 1; j < a.K; ++j)
                if (a.ids[t * a.K + j] == e) w += a.weights[t * a.K + j];
        }
        const uint32_t low = mask[e][0], high = mask[e][1];
        const int before = t < 32 ? __popc(low & ((1u << t) - 1)) : __popc(low) + __popc(high & ((1u << (t - 32)) - 1));
        it.slot[it.at[e] + before] = s;
        it.token[it.at[e] + before] = t;
        it.w[it.at[e] + before] = w;
    }
    fence_proxy_async();  // ordinary accesses to the masks, then copies over them
    __syncthreads();
}

// ------------------------------------------------------------- first product
// The CTA's share of the (item, row pair) list, a pair being gate row i and up
// row I + i of the item's expert: whole eights of the list (I is a multiple of 8,
// so that each is one item's and a tile), or, where there is less than one for
// every CTA, up to eight pairs, cut where the item ends.
//
// Staged activations (4-bit): all tokens if there are no more than eight and
// whole rows of them fit, else those of as many items as fit, and a job's tiles are
// of these.  (8 tokens with 8 of 256 experts of 2 x 256 x 7168: 53.5 instead of 62.8
// us with all staged in three pieces.)
template <int GS>
struct GateUp {
    static constexpr bool kPairs = true;
    const ExpertsArgs& a;
    const Items& it;
    const ProductPlan& plan;
    int q0, q1;      // pairs
    int eights;      // per item; 0: up to eight pairs, from this item on:
    int item0;
    int t0, t1;      // tiles
    bool together;   // all tokens are staged
    struct Job {
        int count;
        int tile;                // first
        int last, base, tokens;  // last item of those staged, first entry, entries
    };
    struct Tile {
        int n, tokens, row, expert;
        int entry, column;
    };
    __device__ GateUp(const ExpertsArgs& a, const Items& it, const ProductPlan& plan) : a(a), it(it), plan(plan) {
        const int pairs = it.count() * a.I;  // at most 2^24
        const bool whole = pairs >= 8 * (int)gridDim.x;
        const Share share(whole ? pairs >> 3 : pairs, gridDim.x, blockIdx.x);
        eights = whole ? a.I >> 3 : 0;
        q0 = share.first;
        q1 = share.last;
        t0 = whole ? q0 : 0;
        item0 = whole ? 0 : quotient(q0, a.I);
        t1 = whole ? q1 : (q0 < q1) + (q1 > (item0 + 1) * a.I);
        together = GS == 0 || plan.together;
    }
    __device__ int item_of(int tile) const { return eights ? quotient(tile, eights) : item0 + tile; }
    __device__ void at(Job& j, int tile, bool fresh) const {
        j.tile = tile;
        j.count = min(kJobTiles<GS>, t1 - tile);
        if (together) {
            j.last = 0;
            j.base = 0;
            j.tokens = a.T;
            return;
        }
        if (fresh || item_of(tile) > j.last) {
            const int item = item_of(tile), end = item_of(t1 - 1);
            j.base = it.off[item];
            j.tokens = it.n[item];
            for (j.last = item; j.last < end; ++j.last) {
                const int n = j.tokens + it.n[j.last + 1];
                if (n > 8 || plan.panel[n] < plan.shape.segments) break;
                j.tokens = n;
            }
        }
        j.count = min(j.count, (eights ? (j.last + 1) * eights : j.last + 1 - item0) - tile);
    }
    __device__ Tile tile(const Job& j, int i) const {
        Tile t;
        const int item = item_of(j.tile + i);
        if (eights) {
            t.n = 8;
            t.row = (j.tile + i - item * eights) * 8;
        } else {
            const int begin = max(q0, item * a.I);
            t.n = min(q1, (item + 1) * a.I) - begin;
            t.row = begin - item * a.I;
        }
        t.expert = it.expert[item];
        t.tokens = it.n[item];
        t.entry = it.off[item];
        t.column = t.entry - j.base;
        return t;
    }
    __device__ bool first(Job& j) const {
        if (t0 >= t1) return false;
        at(j, t0, true);
        return true;
    }
    __device__ bool next(Job& j) const {
        if (j.tile + j.count >= t1) return false;
        at(j, j.tile + j.count, false);
        return true;
    }
    __device__ const uint16_t* scales(const Tile& t) const { return a.s13 + ((int64_t)t.expert * 2 * a.I + t.row) * Fmt<GS>::scales(a.H); }
    __device__ int second() const { return a.I; }
    __device__ void lost() const { atomicOr(a.err, kErrTimeout); }
    __device__ unsigned long long stall() const { return a.stall_ns[0]; }
    __device__ const uint16_t* x(const Tile& t, int i) const { return a.x + (int64_t)it.token[t.entry + i] * a.H; }
    __device__ int staged_key(const Job& j) const { return j.base; }
    __device__ int staged(const Job& j) const { return j.tokens; }
    __device__ const uint16_t* staged_x(const Job& j, int i) const {
        return a.x + (int64_t)(together ? i : it.token[j.base + i]) * a.H;
    }
    __device__ int column(const Tile& t, int i) const { return together ? it.token[t.entry + i] : t.column + i; }
    __device__ void store(const Tile& t, int pair, int token, float gate, float up) const {
        const int i = t.row + pair;
        const float v = gate / (1.0f + expf(-gate)) * up * (GS ? ready_scale(i) : 1.0f);
        const __nv_bfloat16 high = __float2bfloat16_rn(v);
        const float rest = v - __bfloat162float(high);  // an infinite value has no rest
        uint16_t* o = a.act + (int64_t)it.slot[t.entry + token] * 2 * a.I + (GS ? ready_at<GS ? GS : 1>(i) : i);
        o[0] = __bfloat16_as_ushort(high);
        o[a.I] = __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(rest) ? rest : 0.0f));
    }
};

// (With 512 threads there are 128 registers for each; groups of 64 and 32 spill 8
// and 72 bytes.)
template <int GS>
__global__ void __launch_bounds__(kMvThreads, 1) moe_gate_up_kernel(const __grid_constant__ ExpertsArgs a, const __grid_constant__ Weights weights,
                                                                       const __grid_constant__ ProductPlan plan) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const Items it(smem + plan.extra_at, a.T * a.K, a.E);
    SlotRing::init(smem_addr(smem) + warp_index() * kMaxSlots * 8, GS > 0 ? Scales<GS ? GS : 1>::arrivals(plan.piece) : 1, threadIdx.x & 31);
    if (threadIdx.x == 0) prefetch_maps(weights, plan.shape.row_bytes >= kSegment, GS > 0 && plan.piece == 0);
    pdl_wait();     // no global memory access before this point
    pdl_trigger();  // after it: what the second kernel reads before its own wait is complete
    build_items(it, reinterpret_cast<uint32_t(*)[2]>(smem + plan.ring_at), a, plan.chunk);
    // (Cutting tiles to deal 13.5 pairs to each CTA instead of one or two tiles took 23.7 us instead of 18.5 for one token and 8
    // experts of 2 x 256 x 7168.)
    GateUp<GS> jobs(a, it, plan);
    run_product<GS>(jobs, weights, smem, plan, a.H);
}

// ------------------------------------------------------------ second product
// The CTA's output rows in tiles of 16; a tile's work is the concatenation of
// all items' columns (item, segment), cut into sixteen equal ranges.  Each warp
// adds its items' results, weighted, to its own sums [T][16] in shared memory;
// the sixteen sums are added in warp order.
//
// 4-bit weights: the activations are copied to shared memory once, every warp's
// by itself, if there is room for all.  Loads of them come back behind the
// copies in flight, two to three microseconds later.  What is left takes twice the
// matrix instructions of the first product, since the codes' offset is taken off by
// them, again for every tile (one token, 8 experts of 7168 x 2048: 16 us, 0.55 of
// the copy rate, with the issue slots a third busy and the tensor pipe too: chains
// of instructions that wait for each other).
struct DownPlan {
    RowShape shape;
    int round, items_at, ring_at, scales_at, slots, step, smem, piece;
    int act_at, act_entry, act_part;  // staged activations: at, bytes of an entry and of its high parts (0: not staged)
};
template <int GS>
DownPlan plan_down(int T, int K, int E, int I, int tiles) {  // tiles: of a CTA, at most
    DownPlan p;
    constexpr int kScales = GS ? Scales<GS ? GS : 1>::kSlot : 0;
    p.shape = RowShape::of(Fmt<GS>::row_bytes(I));
    p.piece = GS ? Scales<GS ? GS : 1>::piece(Fmt<GS>::scales(I)) : 0;
    p.step = p.shape.row_bytes <= kBox ? kSlotBytes / 2 : kSlotBytes;
    p.act_part = (2 * I + 511) / 512 * 512;
    // The first that fits of: activations staged, entries 64 bytes off a multiple of 128 (no bank conflicts); the same with one
    // tile a round; one tile a round, entries side by side; activations not staged.
    for (int option = GS ? 0 : 3;; ++option) {
        // sums of a round of tiles: all of them (one barrier in all) where that takes up to 48 KB, else as many as fit there
        const int most = 48 * 1024 / (kMvWarps * T * 64);
        p.round = option == 1 || option == 2 || most < 1 ? 1 : tiles < most ? tiles : most;
        p.act_entry = option == 3 ? 0 : 2 * p.act_part + (option < 2 ? 64 : 0);
        p.items_at = (kMaxSlots + 1) * kMvWarps * 8 + p.round * kMvWarps * T * 64;
        p.ring_at = (p.items_at + Items::bytes(T * K, E) + 1023) / 1024 * 1024;
        const int slots = (kSmemLimit - p.ring_at - T * K * p.act_entry) / (kMvWarps * (p.step + kScales));
        p.slots = slots < kMaxSlots ? slots : kMaxSlots;
        p.scales_at = p.ring_at + p.slots * kMvWarps * p.step;
        p.act_at = p.scales_at + p.slots * kMvWarps * kScales;
        p.smem = p.act_at + T * K * p.act_entry;
        if (p.act_entry == 0 || p.slots == kMaxSlots) return p;
    }
}

template <int GS, bool STAGED>
__global__ void __launch_bounds__(kMvThreads, 1) moe_down_kernel(const __grid_constant__ ExpertsArgs a, const __grid_constant__ Weights weights,
                                                                    const __grid_constant__ DownPlan plan) {
    using F = Fmt<GS>;
    constexpr int kGS = GS ? GS : 1;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem + kMvWarps * (kMaxSlots + 1) * 8);  // [tile of the round][warp][T][16]
    const Items it(smem + plan.items_at, a.T * a.K, a.E);
    const int lane = threadIdx.x & 31, warp = warp_index(), g = lane >> 2, t = lane & 3;
    pdl_trigger();
    const uint32_t act_bar = smem_addr(smem) + (kMvWarps * kMaxSlots + warp) * 8;
    if constexpr (STAGED) {
        if (lane == 0) mbar_init(act_bar, 1);
        // zeros behind the values, to the end of two steps
        const int pad = (plan.act_part - 2 * a.I) >> 4;
        for (int i = threadIdx.x; i < a.T * a.K * 2 * pad; i += kMvThreads) {
            const int row = i / pad, at = plan.act_at + (row >> 1) * plan.act_entry + (row & 1) * plan.act_part + 2 * a.I + (i - row * pad) * 16;
            *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
        }
    }
    SlotRing::init(smem_addr(smem) + warp * kMaxSlots * 8, F::kW4 ? Scales<kGS>::arrivals(plan.piece) : 1, lane);
    if (threadIdx.x == 0) prefetch_maps(weights, plan.shape.row_bytes >= kSegment, GS > 0 && plan.piece == 0);
    // Before the wait: ids, weights and expert weights.  The first kernel starts
    // nothing before its own wait, so everything ahead of it has completed; it
    // writes the activations alone.
    build_items(it, reinterpret_cast<uint32_t(*)[2]>(smem + plan.ring_at), a, kChunk2);

    const Share share(a.H, gridDim.x, blockIdx.x);
    const int r0 = share.first, r1 = share.last;
    const RowShape& shape = plan.shape;
    const int row_scales = F::scales(a.I), segments = shape.segments;
    const int total = it.count() * segments;
    const int f0 = total * warp / kMvWarps, f1 = total * (warp + 1) / kMvWarps;  // total <= 2^18
    const int item0 = quotient(f0, segments), seg0 = f0 - item0 * segments;
    SlotRing ring(smem_addr(smem) + plan.ring_at + warp * plan.slots * plan.step, smem_addr(smem) + warp * kMaxSlots * 8, plan.slots, plan.step);
    const uint32_t ring_scales = smem_addr(smem) + plan.scales_at + warp * plan.slots * Scales<kGS>::kSlot;
    auto scales_slot = [&]() { return ring.beside(ring_scales, Scales<kGS>::kSlot); };

    // Copies: the next (tile, item, segment).
    int crow = r0, cf = f0, citem = item0, cseg = seg0;
    bool more = f0 < f1 && r0 < r1;
    int cfirst = 0;
    auto aim = [&]() { cfirst = uniform(it.expert[citem]) * a.H + crow; };  // at most 2^23
    auto fill = [&]() {
        if (!more) return;
        const int rows = min(16, r1 - crow);
        const bool scales = F::kW4 && plan.piece == 0;
        if (lane == 0 && ring.alive) {
            ring.fill<false>(weights, cfirst, rows, 0, cseg, shape.bytes(cseg), scales ? Scales<kGS>::kSlot : 0);
            if constexpr (F::kW4)
                if (scales) Scales<kGS>::template copy<false>(scales_slot(), ring.bar(), weights, cfirst, 0, cseg);
        }
        if constexpr (F::kW4)
            if (!scales && ring.alive)
                Scales<kGS>::template fill<false>(scales_slot(), ring.bar(), a.s2 + (int64_t)cfirst * row_scales, rows, 8, cseg * 4 * kGS, row_scales,
                                                  plan.piece, lane);
        if (++cf == f1) {
            cf = f0;
            citem = item0;
            cseg = seg0;
            crow += 16;
            more = crow < r1;
            if (more) aim();
        } else if (++cseg == segments) {
            cseg = 0;
            ++citem;
            aim();
        }
    };
    if (more) aim();
    const unsigned long long stall = a.stall_ns[1];
    for (int s = 0; s < (stall ? 1 : plan.slots); ++s) {
        fill();
        ring.next();
    }
    ring.at = 0;
    pdl_wait();  // the activations
    if constexpr (STAGED) {
        // the warp's: of every item a range of its columns, lane = (entry, part)
        uint32_t bytes = 0;
        for (int f = f0, item = item0, seg = seg0; f < f1; ++item, seg = 0) {
            const int n = it.n[item], to = min(segments, seg + f1 - f), size = min(to * F::kSegK, a.I) * 2 - seg * F::kSegK * 2;
            const int entry = it.off[item] + (lane >> 1), part = lane & 1;
            if (lane < 2 * n)
                bulk_copy(smem_addr(smem) + plan.act_at + entry * plan.act_entry + part * plan.act_part + seg * F::kSegK * 2,
                          a.act + ((int64_t)it.slot[entry] * 2 + part) * a.I + seg * F::kSegK, size, act_bar);
            bytes += 2 * n * size;
            f += to - seg;
        }
        if (lane == 0) mbar_arrive_expect_tx(act_bar, bytes);
        if (!mbar_sleep(act_bar, 0)) ring.alive = wait_long(act_bar, 0, kWaitLimitNs);
    }
    if (stall) ring.lose(stall, more);

    for (int row = r0, in_round = 0; row < r1; row += 16) {
        const int rows = min(16, r1 - row);
        const int round_sums = kMvWarps * a.T * 16;
        float* mine = sums + in_round * round_sums + warp * a.T * 16;
        for (int i = lane; i < a.T * 16; i += 32) mine[i] = 0.0f;
        __syncwarp();
        // the next segment's operands
        uint4 col[4];
        DirectColumns<kGS> direct[2];  // a box's two steps
        const uint16_t* act = nullptr;
        uint32_t staged = 0;
        const int pair = pair_of_row<GS>(g);
        auto enter = [&](int item) {
            const int e = (g & 3) < it.n[item] ? g & 3 : min(g & 1, it.n[item] - 1);
            if constexpr (STAGED)
                staged = smem_addr(smem) + plan.act_at + (it.off[item] + e) * plan.act_entry + (g >> 2) * plan.act_part + t * 16;
            else
                act = a.act + ((int64_t)it.slot[it.off[item] + e] * 2 + (g >> 2)) * a.I;
        };
        auto load_part = [&](int segment, int q) {  // a step (4-bit) or a quarter of the lane's values
            const int at = segment * F::kSegK;
            if constexpr (F::kW4)
                direct[q & 1].load(act + at + q * F::kStepK, a.I - at - q * F::kStepK, t);
            else
                col[q] = load_column(act + at, a.I - at, q, t);
        };
        int item = item0, seg = seg0;
        if (f0 < f1) {
            enter(item);
            if constexpr (F::kW4 && !STAGED) {
                load_part(seg, 0);
                load_part(seg, 1);
            } else if constexpr (!STAGED) {
#pragma unroll
                for (int q = 0; q < 4; ++q) load_part(seg, q);
            }
        }
        float acc[1][4] = {};
        for (int f = f0; f < f1; ++f) {
            const bool last = seg + 1 == segments, final = f + 1 == f1;
            const int after = last ? 0 : seg + 1, bytes = shape.bytes(seg);
            ring.wait();
            if constexpr (STAGED) {
                Scales<kGS> now;
                const uint32_t scales = scales_slot() + Scales<kGS>::skip(seg);
                ReadyColumns<kGS> columns{staged + seg * (F::kSegK * 2)};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < 2 || bytes > kBox) multiply_w4<kGS>(acc[0], ring.slot(), scales, columns, now, q, lane);
                if (last && !final) enter(item + 1);
            } else if constexpr (F::kW4) {
                Scales<kGS> now;
                const uint32_t scales = scales_slot() + Scales<kGS>::skip(seg);
                // boxes of two steps; of what is behind the end of the rows codes and activations are zero
#pragma unroll
                for (int box = 0; box < 2; ++box)
                    if (box * kBox < bytes) {
                        const bool end = box == 1 || bytes <= kBox;
                        if (end && !final && last) enter(item + 1);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            multiply_w4<kGS>(acc[0], ring.slot(), scales, direct[q], now, 2 * box + q, lane);
                            if (!end)
                                load_part(seg, 2 + q);
                            else if (!final)
                                load_part(after, q);
                        }
                    }
            } else {
                if (last && !final) enter(item + 1);
                multiply_bf16(acc[0], ring.slot(), col, bytes, lane, [&](int q) {
                    if (!final) load_part(after, q);
                });
            }
            __syncwarp();  // all lanes have read the slot
            fill();
            ring.next();
            if (last || final) {
                // high part + low part, times the routing weight, to the token's sums
                const int n = it.n[item], at = it.off[item];
                if (F::kW4)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[0][u] *= kReadyFactor;
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[0][u] += __shfl_xor_sync(0xffffffffu, acc[0][u], 2);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int column = 2 * t + c;
                    if (t < 2 && column < n) {
                        const float w = it.w[at + column];
                        float* y = mine + it.token[at + column] * 16 + pair;
                        y[0] = fmaf(w, acc[0][c], y[0]);
                        y[8] = fmaf(w, acc[0][c + 2], y[8]);
                    }
                }
                acc[0][0] = acc[0][1] = acc[0][2] = acc[0][3] = 0.0f;
                __syncwarp();  // the next item's columns may be other lanes' tokens
            }
            seg = after;
            item += last;
        }
        if (ring.ended(more)) {
            atomicOr(a.err, kErrTimeout);
            for (int i = lane; i < a.T * 16; i += 32) mine[i] = __uint_as_float(0x7fc00000u);
        }
        if (++in_round < plan.round && row + 16 < r1) continue;
        __syncthreads();
        const int from = row - 16 * (in_round - 1);  // the round's rows, in the order (tile, token, row)
        for (int i = threadIdx.x; i < in_round * a.T * 16; i += kMvThreads) {
            const int tile = quotient(i >> 4, a.T), token = (i >> 4) - tile * a.T, at = from + 16 * tile + (i & 15);
            if (at >= r1) continue;
            const float* all = sums + tile * round_sums + token * 16 + (i & 15);
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < kMvWarps; ++w) y += all[w * a.T * 16];
            a.out[(int64_t)token * a.H + at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        }
        in_round = 0;
        if (row + 16 < r1) __syncthreads();  // the sums are added
    }
    if (!ring.alive) grace_period(10000000ull);  // copies that may still land
}

template <typename Kernel, typename Plan>
cudaError_t launch(Kernel kernel, const ExpertsArgs& a, const Weights& weights, const Plan& plan, int grid, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = (size_t)plan.smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, weights, plan);
}

template <int GS>
cudaError_t launch_both(const ExpertsArgs& a, int num_sms, cudaStream_t stream, bool pdl) {
    const int64_t pairs = (int64_t)a.T * a.K * a.I;
    const int most = (int)((pairs / 8 + num_sms - 1) / num_sms), tiles = most > 2 ? most : 2;
    Weights w13{}, w2{};
    cudaError_t e = describe_weights(&w13, {a.w13, a.s13, (int64_t)a.E * 2 * a.I, Fmt<GS>::row_bytes(a.H), Fmt<GS>::scales(a.H), GS, a.I, 0});
    if (e == cudaSuccess)
        e = describe_weights(&w2, {a.w2, a.s2, (int64_t)a.E * a.H, Fmt<GS>::row_bytes(a.I), Fmt<GS>::scales(a.I), GS, 0, a.H / num_sms});
    if (e != cudaSuccess) return e;
    // Up to eight tokens are all staged, if whole rows of them fit.
    const int items = Items::bytes(a.T * a.K, a.E);
    ProductPlan first = plan_product<GS>(a.H, a.T < 8 ? a.T : 8, 8, tiles, items);
    first.together = a.T <= 8 && first.panel[a.T] == first.shape.segments;
    if (GS > 0 && !first.together) {
        const int chunk = chunk_first(a.T, a.K, a.E);
        first = plan_product<GS>(a.H, a.T < chunk ? a.T : chunk, 8, tiles, items);
        first.chunk = chunk;
    }
    e = launch(moe_gate_up_kernel<GS>, a, w13, first, num_sms, stream, pdl);
    if (e != cudaSuccess) return e;
    const DownPlan plan = plan_down<GS>(a.T, a.K, a.E, a.I, ((a.H + num_sms - 1) / num_sms + 15) / 16);
    if (GS > 0 && plan.act_entry > 0) return launch(moe_down_kernel<GS, (GS > 0)>, a, w2, plan, num_sms, stream, true);
    return launch(moe_down_kernel<GS, false>, a, w2, plan, num_sms, stream, true);
}

template <int GS>
cudaError_t set_attributes() {
    cudaError_t e = cudaFuncSetAttribute(moe_gate_up_kernel<GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<GS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<GS, (GS > 0)>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    return e;
}

}  // namespace

cudaError_t describe_weights(Weights* w, const WeightRows& m) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> cached{nullptr};  // the same in every thread
    Encode encode = cached.load(std::memory_order_acquire);
    if (!encode) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
        encode = reinterpret_cast<Encode>(f);
        cached.store(encode, std::memory_order_release);
    }
    bool ok = true;
    auto map = [&](CUtensorMap* to, bool codes, int rank, const cuuint64_t* dim, const cuuint64_t* pitch, const cuuint32_t* box) {
        const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
        ok = ok && encode(to, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, (cuuint32_t)rank,
                          const_cast<void*>(codes ? m.q : m.s), dim, pitch, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          codes ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t bytes = (cuuint64_t)m.row_bytes, rows = (cuuint64_t)m.rows, whole = bytes / kBox;
    const bool ragged = bytes % kSegment != 0;
    const cuuint32_t scales = m.group_steps == 1 ? 8 : 4 * m.group_steps;
    const cuuint64_t scale_bytes = (cuuint64_t)m.row_scales * 2;
    const bool tensor_scales = m.group_steps > 0 && m.row_scales % 8 == 0;
    if (m.inter > 0) {
        const cuuint64_t inter = (cuuint64_t)m.inter, experts = rows / (2 * inter);
        if (bytes >= kSegment) {
            const cuuint64_t dim[5] = {kBox, inter, 2, whole, experts}, pitch[4] = {bytes, inter * bytes, kBox, 2 * inter * bytes};
            const cuuint32_t box[5] = {kBox, 8, 2, 2, 1};
            map(&w->full, true, 5, dim, pitch, box);
        }
        if (ragged) {
            const cuuint64_t dim[4] = {bytes, inter, 2, experts}, pitch[3] = {bytes, inter * bytes, 2 * inter * bytes};
            const cuuint32_t box[4] = {kBox, 8, 2, 1};
            map(&w->part[0], true, 4, dim, pitch, box);
        }
        if (tensor_scales) {
            const cuuint64_t dim[4] = {(cuuint64_t)m.row_scales, inter, 2, experts},
                             pitch[3] = {scale_bytes, inter * scale_bytes, 2 * inter * scale_bytes};
            const cuuint32_t box[4] = {scales, 8, 2, 1};
            map(&w->scales, false, 4, dim, pitch, box);
        }
    } else {
        // heights of the CTAs' last tiles
        const int last = m.each % 16, one_more = (m.each + 1) % 16;
        auto ends = [&](int from, int to) { return (last >= from && last <= to) || (one_more >= from && one_more <= to); };
        if (bytes >= kSegment) {
            const cuuint64_t dim[3] = {kBox, rows, whole}, pitch[2] = {bytes, kBox};
            const cuuint32_t box[3] = {kBox, 16, 2};
            map(&w->full, true, 3, dim, pitch, box);
        }
        const cuuint64_t dim[2] = {bytes, rows}, pitch[1] = {bytes};
        for (int i = 0; i < 3; ++i)
            if (i == 0 ? ragged : i == 1 ? ends(5, 8) : ends(1, 4)) {
                const cuuint32_t box[2] = {kBox, 16u >> i};
                map(&w->part[i], true, 2, dim, pitch, box);
            }
        if (tensor_scales) {
            const cuuint64_t dims[2] = {(cuuint64_t)m.row_scales, rows}, pitches[1] = {scale_bytes};
            const cuuint32_t box[2] = {scales, 16};
            map(&w->scales, false, 2, dims, pitches, box);
        }
    }
    return ok ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_moe_experts(const ExpertsArgs& a, int group, int num_sms, cudaStream_t stream, bool pdl) {
    switch (group) {
        case 0: return launch_both<0>(a, num_sms, stream, pdl);
        case 32: return launch_both<4>(a, num_sms, stream, pdl);
        case 64: return launch_both<2>(a, num_sms, stream, pdl);
        case 128: return launch_both<1>(a, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

cudaError_t moe_experts_set_attributes() {
    cudaError_t e = set_attributes<0>();
    if (e == cudaSuccess) e = set_attributes<1>();
    if (e == cudaSuccess) e = set_attributes<2>();
    if (e == cudaSuccess) e = set_attributes<4>();
    return e;
}

}  // namespace arf
