// moe_route.cu -- the router: gate product, choice of experts, weights.
//
//   l[t,e] = x[t] . gate[e];  s = softmax_e(l) or sigmoid(l)
//   c = l, or s + bias (with a bias or expert groups)
//   expert groups: only the topk_group groups with the largest sum of their two
//   best c (or the largest best c) stay; ids[t] = the top_k largest c, lowest index first among equals
//   weights[t] = s[ids], optionally over their sum, times scale
//
// One CTA per (expert, four tokens) computes four dot products; the last CTA of
// a token group to arrive chooses.  The choice must not
// depend on how a sum was split, so the sums carry a second word: bf16
// products are exact in fp32 (between 2^-126 and 2^128), and each addition's error
// is kept (two-sum), which leaves a relative error of about 2^-45 of the sum of
// magnitudes.  Scores are
// formed and compared in 32 bits where the gaps between the chosen are wider than
// what 32 bits can get wrong, else (one token in some thousands) in 64 bits,
// whose rate on this GPU is 1/64 of that; the weights of the chosen always are.
//
// Bound by latency: the gate is read in 1.5 us, the arrivals take 1.2, the choice
// 3.9 (a chain of top_k + 1 reductions at its end) and the weights 2.  One token of
// 256 experts in groups takes 9.4 us, 16 tokens of 160 experts 15.1, 64 tokens of 128
// 20.5: there the two-sums take about 10, seven operations for every product,
// although only near ties and the chosen experts need them.
#include "moe_common.cuh"

namespace arf {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteTokens = 4;
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

// Two such sums side by side, in packed instructions (twice the rate).
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pack(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 unpack(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair sub(Pair a, Pair b) {  // exact product by -1, one rounding
    Pair r;
    const Pair m = pack(-1.0f, -1.0f);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(b.v), "l"(m.v), "l"(a.v));
    return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
struct Sum2x2 {
    Pair hi, lo;
    // A two-sum of hi and the product, which is exact and needs no instruction of its own.
    __device__ __forceinline__ void add_product(Pair x, Pair w) {
        const Pair r = fma(x, w, hi), minus = sub(hi, r);  // -(r - hi)
        lo = add(lo, add(sub(hi, add(r, minus)), fma(x, w, minus)));
        hi = r;
    }
};

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

// A float as an unsigned integer of the same order, above 0 (NaN aside).
__device__ __forceinline__ unsigned ordered32(float v) {
    const unsigned b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered32(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A sigmoid, or a softmax's exponential.
__device__ __noinline__ double score64(const RouteArgs& a, double z, double top) {
    const double x = exp(a.sigmoid ? -z : z - top);
    return a.sigmoid ? 1.0 / (1.0 + x) : x;
}

// A token's choice, in order, before its weights: logits, and what a softmax needs.
struct Chosen {
    double z[kMaxTopK], total;
    float top;
    int id[kMaxTopK];
    bool done;  // and its weights
};

// One warp: the weights of the chosen ids (lane k holds the k-th), in 64 bits.
__device__ __noinline__ void store_choice(const RouteArgs& a, int token, int lane, int id, double score, double sum) {
    const int slots = a.K + a.shared;
    if (lane < a.K) {
        double w = score;
        if (a.renorm) w = sum > 0.0 || sum != sum ? w / sum : 0.0;
        a.ids[(int64_t)token * slots + lane] = id;
        a.weights[(int64_t)token * slots + lane] = (float)(w * (double)a.scale);
    } else if (lane < slots) {
        a.ids[(int64_t)token * slots + lane] = a.E + lane - a.K;
        a.weights[(int64_t)token * slots + lane] = 1.0f;
    }
}

// The choice in 32 bits, for every token of the CTA at once, the
// CTA's warps dealt to them evenly, warp `part` of a token's first.  What the
// tokens' warps tell each other goes through Part; False in `good` if some gap
// that decides is too narrow, or something is not a number: nothing is chosen then.
//
// What the difference of two choice values c = s + b may be off by, relative to
// |c| + 2 max|b| (no less than either score): a sigmoid's logit is rounded to 32
// bits, 2^-24 |l| of s; expf and the division are good to 2^-21.4 of it, the sum
// with b to 2^-24: for |l| <= 8 and two values 2^-19.  A softmax's exponent
// carries three such roundings and the difference's own, and the sum of the
// exponentials 2^-19.6: 2^-17.2.  Twice that is taken, and more for larger |l|.
// All of it holds for normal numbers: a score below e^-80 (over 512 experts, in a
// softmax, still above 2^-126) is for 64 bits, since in 32 it is coarse or zero.
//
// Loops, not unrolled code: one SM runs this once, and an instruction that has to
// be fetched costs it more than the instruction (unrolled over sixteen registers
// it took 20 us for one token).  One warp per token took 6.5 us for 256 experts in
// groups, all warps of the CTA take 3.9.
struct Part {
    unsigned top, big, bias;  // largest logit, magnitudes (ordered; bits)
    float total;
    int fine;
};
struct Group {
    unsigned key;
    float reach;
};
template <int TOKENS>
__device__ void choose32(const RouteArgs& a, int token, bool live, int part, int lane, unsigned* keys /* shared, [E] */,
                         float* biases /* the same */, Part* parts /* shared, one per warp of the token */, Group* groups /* shared */,
                         unsigned* kept_groups /* shared */, Chosen& chosen, int* good /* shared */) {
    constexpr int kParts = kRouteWarps / TOKENS, kStep = kParts * 32;
    const float2* l = a.logits + (int64_t)token * a.E;
    const bool by_logit = a.bias == nullptr && a.n_group == 1;
    const int e0 = part * 32 + lane, E = live ? a.E : 0;
    Part mine{0u, 0u, 0u, 0.0f, 1};
#pragma unroll 4
    for (int e = e0; e < E; e += kStep) {
        const float v = __ldcg(l + e).x;
        biases[e] = a.bias ? a.bias[e] : 0.0f;
        mine.fine = mine.fine && fabsf(v) < INFINITY;
        mine.top = max(mine.top, ordered32(v));
        mine.big = max(mine.big, __float_as_uint(fabsf(v)));
        keys[e] = by_logit ? ordered32(v) : __float_as_uint(v);
    }
    mine.top = __reduce_max_sync(0xffffffffu, mine.top);
    mine.big = __reduce_max_sync(0xffffffffu, mine.big);
    float top = 0.0f;
    if (!a.sigmoid && !by_logit) {  // exponentials are of differences from the largest logit
        if (lane == 0) parts[part] = mine;
        __syncthreads();
        unsigned all = 0u;
        for (int w = 0; w < kParts; ++w) all = max(all, parts[w].top);
        top = from_ordered32(all);
        __syncthreads();
    }
    if (!by_logit) {
#pragma unroll 1
        for (int e = e0; e < E; e += kStep) {
            const float v = __uint_as_float(keys[e]), x = expf(a.sigmoid ? -v : v - top), s = a.sigmoid ? 1.0f / (1.0f + x) : x, b = biases[e];
            mine.total += s;
            mine.fine = mine.fine && b == b && b < INFINITY && (a.sigmoid ? v : v - top) > -80.0f;
            if (fabsf(b) < INFINITY) mine.bias = max(mine.bias, __float_as_uint(fabsf(b)));
            keys[e] = a.sigmoid ? ordered32(s + b) : __float_as_uint(s);
        }
        mine.bias = __reduce_max_sync(0xffffffffu, mine.bias);
        mine.total = warp_sum(mine.total);
    }
    mine.fine = __all_sync(0xffffffffu, mine.fine);
    if (lane == 0) parts[part] = mine;
    __syncthreads();
    Part all = parts[0];
    for (int w = 1; w < kParts; ++w) {
        const Part p = parts[w];
        all.top = max(all.top, p.top);
        all.big = max(all.big, p.big);
        all.bias = max(all.bias, p.bias);
        all.total += p.total;
        all.fine = all.fine && p.fine;
    }
    const float bias = __uint_as_float(all.bias);
    const float wide = by_logit ? 0x1p-22f : (a.sigmoid ? 0x1p-18f : 0x1p-16f) * fmaxf(1.0f, __uint_as_float(all.big) * 0.125f);
    if (!a.sigmoid && !by_logit) {
        const float scale = 1.0f / all.total;
#pragma unroll 1
        for (int e = e0; e < E; e += kStep) keys[e] = ordered32(__uint_as_float(keys[e]) * scale + biases[e]);
        __syncthreads();
    }
    if (a.n_group > 1) {
        // a group's two best (or the best), a group per warp
        const int size = quotient(a.E, a.n_group);
#pragma unroll 1
        for (int j = part; live && j < a.n_group; j += kParts) {
            unsigned b0 = 0u, b1 = 0u;
#pragma unroll 1
            for (int e = lane; e < size; e += 32) {
                const unsigned k = keys[j * size + e];
                b1 = max(b1, min(b0, k));
                b0 = max(b0, k);
            }
            const unsigned first = __reduce_max_sync(0xffffffffu, b0);
            const int holder = __ffs(__ballot_sync(0xffffffffu, b0 == first)) - 1;
            const unsigned second = __reduce_max_sync(0xffffffffu, lane == holder ? b1 : b0);
            const float c0 = from_ordered32(first), c1 = a.group_max ? 0.0f : from_ordered32(second);
            if (lane == 0) groups[j] = Group{ordered32(c0 + c1), fabsf(c0) < INFINITY && fabsf(c1) < INFINITY ? fabsf(c0) + fabsf(c1) : 0.0f};
        }
        __syncthreads();
        if (part == 0) {
            unsigned mine = 0u, kept = 0u, last = 0u;
            float reach = 0.0f;
            if (live && lane < a.n_group) {
                mine = groups[lane].key;
                reach = groups[lane].reach;
            }
            reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(reach)));
#pragma unroll 1
            for (int r = 0; r <= a.topk_group && r < a.n_group; ++r) {
                const unsigned best = __reduce_max_sync(0xffffffffu, mine);
                const int holder = __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1;
                if (r == a.topk_group) {
                    if (!(from_ordered32(last) - from_ordered32(best) > 2.0f * wide * (reach + 4.0f * bias))) kept = 0u;
                    break;
                }
                kept |= 1u << holder;
                last = best;
                if (lane == holder) mine = 0u;
            }
            if (lane == 0) *kept_groups = kept;  // 0: too close
        }
        __syncthreads();
        const unsigned kept = *kept_groups;
        all.fine = all.fine && kept != 0u;
#pragma unroll 1
        for (int e = e0; e < E; e += kStep)
            if (!(kept >> quotient(e, size) & 1u)) keys[e] = 0u;
        __syncthreads();
    }
    if (part > 0 || !live) return;
    bool ok = all.fine;
    // the top_k largest, and the one behind them
    unsigned first = 0u, second = 0u, last = 0u;  // the lane's best two
    int first_at = 0, second_at = 0, my_id = 0;
    int known = 0;  // of those two
#pragma unroll 1
    for (int k = 0; ok && k <= a.K; ++k) {
        if (known == 0) {
            first = second = 0u;
#pragma unroll 4
            for (int e = lane; e < a.E; e += 32) {
                const unsigned v = keys[e];
                if (v > first) {
                    second = first;
                    second_at = first_at;
                    first = v;
                    first_at = e;
                } else if (v > second) {
                    second = v;
                    second_at = e;
                }
            }
            known = 2;
        }
        __syncwarp();
        const unsigned best = __reduce_max_sync(0xffffffffu, first);
        const int holder = __ffs(__ballot_sync(0xffffffffu, first == best)) - 1;
        const int id = __shfl_sync(0xffffffffu, first_at, holder);
        if (k > 0 && best != 0u) {  // (equal ones are for 64 bits too, lowest index first)
            const float c0 = from_ordered32(last), c1 = from_ordered32(best);
            if (!(c0 - c1 > wide * (fabsf(c0) + (by_logit ? 0.0f : 2.0f * bias)))) ok = false;
        }
        if (k == a.K) break;
        if (best == 0u) ok = false;
        if (lane == k) my_id = id;
        last = best;
        if (lane == holder) {
            keys[first_at] = 0u;
            first = second;
            first_at = second_at;
            --known;
        }
    }
    if (lane == 0) *good = ok;
    if (!ok) return;
    if (lane < a.K) {
        const float2 v = __ldcg(l + my_id);
        chosen.id[lane] = my_id;
        chosen.z[lane] = (double)v.x + (double)v.y;
    }
    if (lane == 0) chosen.top = from_ordered32(all.top);
    if (!a.sigmoid && !a.renorm) {
        double sum = 0.0;
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
            const float2 u = __ldcg(l + e);
            sum += score64(a, (double)u.x + (double)u.y, (double)from_ordered32(all.top));
        }
        sum = warp_sum_d(sum);
        if (lane == 0) chosen.total = sum;
    }
}

// One warp: the choice for one token in 64 bits, for every input.  Lane l holds
// experts l, l + 32, ...
__device__ __noinline__ void choose(const RouteArgs& a, int token, int lane, double* scores /* shared, [E] */,
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
        scores[e] = score64(a, z, top);
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
        // lane = group: the sum of its two best, or the best
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
            mine = ordered(a.group_max ? b0 : b0 + b1);
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
#pragma unroll 1
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
    store_choice(a, token, lane, my_id, my_score, sum);
}

// TOKENS per CTA.  One token: four of a thread's chunks of the expert's row at a
// time, all asked for before the first is used; more: a chunk of all tokens.
template <int TOKENS>
__global__ void __launch_bounds__(kRouteThreads, 4) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];  // the choice: [warp][E] scores and keys
    __shared__ Sum2 part[kRouteWarps][TOKENS];
    __shared__ Chosen chosen[TOKENS];
    __shared__ Part parts[kRouteWarps];
    __shared__ Group groups[TOKENS][kMoeMaxGroups];
    __shared__ unsigned kept[TOKENS];
    __shared__ int good[TOKENS];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int expert = blockIdx.x, t0 = blockIdx.y * TOKENS, nt = min(TOKENS, a.T - t0);
    pdl_trigger();
    pdl_wait();  // no global memory access before this point

    Sum2x2 sums[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) sums[j].hi = sums[j].lo = pack(0.0f, 0.0f);
    const int chunks = a.H / 8;
    const uint16_t* row = a.gate + (int64_t)expert * a.H;
    constexpr int kAhead = TOKENS == 1 ? 4 : 1;
    for (int c0 = threadIdx.x; c0 < chunks; c0 += kAhead * kRouteThreads) {
        uint4 wv[kAhead], xv[kAhead][TOKENS];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u * kRouteThreads;
            wv[u] = make_uint4(0, 0, 0, 0);
            if (c < chunks) wv[u] = ld_coherent16(row + c * 8);
#pragma unroll
            for (int j = 0; j < TOKENS; ++j) {
                xv[u][j] = make_uint4(0, 0, 0, 0);
                if (c < chunks && j < nt) xv[u][j] = ld_coherent16(a.x + (int64_t)(t0 + j) * a.H + c * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            float f[8], v[8];
            bf16x8_to_f32(wv[u], f);
#pragma unroll
            for (int j = 0; j < TOKENS; ++j)
                if (j < nt) {
                    bf16x8_to_f32(xv[u][j], v);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) sums[j].add_product(pack(v[i], v[i + 1]), pack(f[i], f[i + 1]));
                }
        }
    }
    // over the lanes, halving the tokens that a lane is left with
    Sum2 acc[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
        const float2 h = unpack(sums[j].hi), l = unpack(sums[j].lo);
        acc[j] = add2(Sum2{h.x, l.x}, h.y, l.y);
    }
    int o = 16;
#pragma unroll
    for (int n = TOKENS / 2; n > 0; n >>= 1, o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const Sum2 keep = upper ? acc[j + n] : acc[j], give = upper ? acc[j] : acc[j + n];
            const float hi = __shfl_xor_sync(0xffffffffu, give.hi, o), lo = __shfl_xor_sync(0xffffffffu, give.lo, o);
            acc[j] = add2(keep, hi, lo);
        }
    }
#pragma unroll
    for (; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, acc[0].hi, o), lo = __shfl_xor_sync(0xffffffffu, acc[0].lo, o);
        acc[0] = add2(acc[0], hi, lo);
    }
    if (lane % (32 / TOKENS) == 0) part[warp][lane / (32 / TOKENS)] = acc[0];
    __syncthreads();
    if (threadIdx.x < 32) {  // one warp writes, then arrives for all
        if (lane < nt) {
            Sum2 s = part[0][lane];
#pragma unroll
            for (int u = 1; u < kRouteWarps; ++u) s = add2(s, part[u][lane].hi, part[u][lane].lo);
            // the sum rounded, and the rest; an infinite or undefined sum has none
            const float hi = s.hi + s.lo;
            a.logits[(int64_t)(t0 + lane) * a.E + expert] =
                isfinite(hi) ? make_float2(hi, __fsub_rn(s.lo, __fsub_rn(hi, s.hi))) : make_float2(isfinite(s.hi) ? hi : s.hi, 0.0f);
            __threadfence();
        }
        __syncwarp();
        if (lane == 0) last = atomicAdd(a.count + blockIdx.y, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) a.count[blockIdx.y] = 0;  // for the next call
    {
        constexpr int kParts = kRouteWarps / TOKENS;
        const int j = warp / kParts, part = warp % kParts;
        double* scores = reinterpret_cast<double*>(smem) + j * 2 * a.E;
        choose32<TOKENS>(a, t0 + j, j < nt, part, lane, reinterpret_cast<unsigned*>(scores), reinterpret_cast<float*>(scores + a.E),
                         parts + j * kParts, groups[j], kept + j, chosen[j], good + j);
        __syncwarp();
        if (part == 0 && j < nt) {
            const bool done = !good[j];
            if (done) choose(a, t0 + j, lane, scores, reinterpret_cast<long long*>(scores + a.E));
            if (lane == 0) chosen[j].done = done;
        }
    }
    __syncthreads();
    // the weights in 64 bits, all tokens' chosen side by side: a warp's instruction takes that unit as long for one as for 32
    const int slots = a.K + a.shared;
    for (int i = threadIdx.x; i < nt * slots; i += kRouteThreads) {
        const int token = quotient(i, slots), k = i - token * slots;
        Chosen& c = chosen[token];
        if (!c.done && k < a.K) c.z[k] = score64(a, c.z[k], (double)c.top);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * slots; i += kRouteThreads) {
        const int token = quotient(i, slots), k = i - token * slots;
        const Chosen& c = chosen[token];
        if (c.done) continue;
        double w = 1.0;
        if (k < a.K) {
            w = c.z[k];
            if (a.renorm) {
                double sum = 0.0;
#pragma unroll 1
                for (int j = 0; j < a.K; ++j) sum += c.z[j];
                w = sum > 0.0 ? w / sum : 0.0;
            } else if (!a.sigmoid) {
                w /= c.total;
            }
            w *= (double)a.scale;
        }
        a.ids[(int64_t)(t0 + token) * slots + k] = k < a.K ? c.id[k] : a.E + k - a.K;
        a.weights[(int64_t)(t0 + token) * slots + k] = (float)w;
    }
}

template <int TOKENS>
cudaError_t launch(const RouteArgs& a, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)a.E, (unsigned)((a.T + TOKENS - 1) / TOKENS));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = (size_t)TOKENS * a.E * 16;  // at most 32 KB
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<TOKENS>, a);
}

}  // namespace

cudaError_t moe_route_set_attributes() {
    return cudaFuncSetAttribute(moe_route_kernel<kRouteTokens>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteTokens * kMoeMaxExperts * 16);
}

// 16 tokens took 16.9 us with four tokens per CTA and 19.5 with eight, 64 tokens
// 23.4 and 26.3; two experts per CTA gain nothing.  (Four CTAs to an SM, 64
// registers: 20.3 us for 64 tokens, 21.7 with 70.)
cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t stream, bool pdl) {
    return a.T <= 2 ? launch<1>(a, stream, pdl) : launch<kRouteTokens>(a, stream, pdl);
}

}  // namespace arf
