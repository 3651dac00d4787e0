// moe_experts.cu -- the experts' products of a few tokens.
//
//   h = W13_e x[t];  a = silu(h[0:I]) * h[I:2I];  y[t] += w[t,k] * W2_e a,   e = ids[t,k]
//
// Two kernels: the first writes the activations a of every (token, expert)
// slot, the second the sums y.  Both read each chosen expert's weights once,
// whichever tokens chose it, and deal weight rows evenly over the SMs: the
// first kernel flattens (chosen expert, row pair), the second gives every CTA
// its share of the H output rows for all chosen experts, so that the sum over
// a token's experts never leaves the CTA: no atomics, one rounding.
//
// The activations travel as a bf16 high part and a bf16 low part (16 bits of
// mantissa together), columns 0-3 and 4-7 of the matrix instruction's eight:
// rounding them to one bf16 would double the result's error against 32-bit
// arithmetic, and up to four tokens per expert the second part costs nothing.
#include "moe_common.cuh"

namespace arf {
namespace {

constexpr int kPairTiles = 2;      // 16-row tiles (8 gate rows, 8 up rows) per block of the first kernel
constexpr int kChunk1 = 8;         // tokens per item of the first kernel
constexpr int kChunk2 = 4;         // and of the second (high and low part)

// The chosen experts, in order, each with the tokens that chose it, in order,
// cut into items of up to `chunk` tokens.
struct Items {
    uint16_t expert[kMoeMaxSlots];
    uint16_t off[kMoeMaxSlots];     // first entry
    uint8_t n[kMoeMaxSlots];
    uint16_t slot[kMoeMaxSlots];    // entries: token * K + k
    float w[kMoeMaxSlots];          // entries: routing weight
    uint16_t at[kMoeMaxExperts];    // an expert's first entry
    uint32_t mask[kMoeMaxExperts][2];  // tokens that chose it
    int warp_items[kMvWarps], warp_entries[kMvWarps];
    int count;
};

// Called by all threads of a CTA.  A token that names an expert twice gets one
// entry with the sum of its weights.  -1 names no expert; other values outside
// [0, E) are skipped too and flagged.
__device__ void build_items(Items& it, const ExpertsArgs& a, int chunk) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slots = a.T * a.K;
    for (int e = tid; e < a.E; e += kMvThreads) it.mask[e][0] = it.mask[e][1] = 0;
    __syncthreads();
    for (int s = tid; s < slots; s += kMvThreads) {
        const int e = a.ids[s], t = s / a.K;
        if ((unsigned)e < (unsigned)a.E)
            atomicOr(&it.mask[e][t >> 5], 1u << (t & 31));
        else if (e != -1)
            atomicOr(a.err, kErrExpertRange);
    }
    __syncthreads();
    static_assert(kMoeMaxExperts <= kMvThreads, "one expert per thread");
    const int n = tid < a.E ? __popc(it.mask[tid][0]) + __popc(it.mask[tid][1]) : 0;
    const int m = (n + chunk - 1) / chunk;
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
        it.warp_items[warp] = ni;
        it.warp_entries[warp] = ne;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ni += it.warp_items[w];
        ne += it.warp_entries[w];
    }
    if (tid == kMvThreads - 1) it.count = ni;
    if (n > 0) {
        it.at[tid] = ne - n;
        for (int j = 0; j < m; ++j) {
            it.expert[ni - m + j] = tid;
            it.off[ni - m + j] = ne - n + j * chunk;
            it.n[ni - m + j] = min(chunk, n - j * chunk);
        }
    }
    __syncthreads();
    for (int s = tid; s < slots; s += kMvThreads) {
        const int e = a.ids[s], t = s / a.K, k = s % a.K;
        if ((unsigned)e >= (unsigned)a.E) continue;
        bool first = true;
        for (int j = 0; j < k; ++j) first = first && a.ids[t * a.K + j] != e;
        if (!first) continue;
        float w = a.weights[s];
        for (int j = k + 1; j < a.K; ++j)
            if (a.ids[t * a.K + j] == e) w += a.weights[t * a.K + j];
        const uint32_t low = it.mask[e][0], high = it.mask[e][1];
        const int before = t < 32 ? __popc(low & ((1u << t) - 1)) : __popc(low) + __popc(high & ((1u << (t - 32)) - 1));
        it.slot[it.at[e] + before] = s;
        it.w[it.at[e] + before] = w;
    }
    __syncthreads();
}

template <int GS>
constexpr int smem1() {
    return kMvWarps * Fmt<GS>::kRingBytes + 2 * kMvWarps * kPairTiles * 512 + (int)sizeof(Items);
}
// MT tiles of 16 rows at a time and up to 64 / MT tokens
template <int GS>
constexpr int smem2() {
    return kMvWarps * Fmt<GS>::kRingBytes + kMvWarps * 64 * 64 + (int)sizeof(Items);
}

// ------------------------------------------------------------- first product
// The CTA's row pairs (gate row i, up row I + i of an item's expert) in blocks
// of up to 16; the sixteen warps split a block's columns and add their parts
// through shared memory.
template <int GS>
__global__ void __launch_bounds__(kMvThreads, 1) moe_gate_up_kernel(const __grid_constant__ ExpertsArgs a) {
    using F = Fmt<GS>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + kMvWarps * F::kRingBytes);
    Items& it = *reinterpret_cast<Items*>(smem + kMvWarps * F::kRingBytes + 2 * kMvWarps * kPairTiles * 512);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    pdl_wait();     // no global memory access before this point
    pdl_trigger();  // after it: what the second kernel reads before its own wait is complete
    build_items(it, a, kChunk1);

    const int64_t pairs = (int64_t)it.count * a.I;
    const int64_t q0 = pairs * blockIdx.x / gridDim.x, q1 = pairs * (blockIdx.x + 1) / gridDim.x;
    if (q0 >= q1) return;
    Rows m;
    m.q = a.w13;
    m.s = a.s13;
    m.row_bytes = F::row_bytes(a.H);
    m.row_scales = F::kW4 ? a.H / (128 / (GS ? GS : 1)) : 0;
    m.s_end = a.s13 + (int64_t)a.E * 2 * a.I * m.row_scales;
    const int steps = F::steps(a.H);
    const int s0 = steps * warp / kMvWarps, s1 = steps * (warp + 1) / kMvWarps;
    const uint32_t ring = smem_addr(smem) + warp * F::kRingBytes;

    // A block of pairs, for the copies and (seven stages later) the products.
    struct Block {
        int64_t q;
        int item, i0, n;
    };
    auto block_at = [&](int64_t q) {
        Block b;
        b.q = q;
        b.item = (int)(q / a.I);
        b.i0 = (int)(q - (int64_t)b.item * a.I);
        b.n = (int)min((int64_t)min(8 * kPairTiles, a.I - b.i0), q1 - q);
        return b;
    };
    Block cb = block_at(q0);
    int cstep = s0, ctile = 0, cslot = 0;
    bool more = s0 < s1;
    auto copy_next = [&]() {
        if (more) {
            const int64_t lo = (int64_t)it.expert[cb.item] * 2 * a.I + cb.i0 + 8 * ctile;
            const int n = cb.n - 8 * ctile;
            copy_stage<GS>(ring + cslot * F::kStageBytes, m, lo, n, lo + a.I, n, cstep, lane);
            cslot = cslot + 1 == F::kStages ? 0 : cslot + 1;
            if (++ctile * 8 >= cb.n) {
                ctile = 0;
                if (++cstep == s1) {
                    cstep = s0;
                    if (cb.q + cb.n < q1)
                        cb = block_at(cb.q + cb.n);
                    else
                        more = false;
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < F::kStages - 1; ++s) copy_next();

    int slot = 0, buf = 0;
    for (int64_t q = q0; q < q1;) {
        const Block b = block_at(q);
        const int tiles = (b.n + 7) >> 3, tokens = it.n[b.item];
        const uint16_t* x = a.x + (g < tokens ? (int64_t)(it.slot[it.off[b.item] + g] / a.K) * a.H : 0);
        float acc[kPairTiles][1][4] = {};
        uint4 col[1][F::kBlocks], next[1][F::kBlocks];
        auto columns = [&](uint4 (&c)[1][F::kBlocks], int step) {
            load_columns<GS, false>(c[0], x + (int64_t)step * F::kStepK, a.H - step * F::kStepK, g < tokens && step < s1, t);
        };
        columns(next, s0);
        for (int step = s0; step < s1; ++step) {
#pragma unroll
            for (int i = 0; i < F::kBlocks; ++i) col[0][i] = next[0][i];
            columns(next, step + 1);
#pragma unroll
            for (int tile = 0; tile < kPairTiles; ++tile)
                if (tile < tiles) {
                    cp_async_wait<F::kStages - 2>();
                    if (F::kW4) __syncwarp();  // other lanes' copies; and all reads of the slot that is filled next
                    copy_next();
                    const int64_t lo = (int64_t)it.expert[b.item] * 2 * a.I + b.i0 + 8 * tile + g;
                    multiply_stage<GS, 1>(acc[tile], ring + slot * F::kStageBytes, col, scale_shift<GS>(m, lo, step),
                                          scale_shift<GS>(m, lo + a.I, step), m.row_scales - step * GS, lane);
                    slot = slot + 1 == F::kStages ? 0 : slot + 1;
                }
        }
        // add the warps' parts in warp order
        float* r = red + buf * kMvWarps * kPairTiles * 128;
#pragma unroll
        for (int tile = 0; tile < kPairTiles; ++tile)
            *reinterpret_cast<float4*>(r + (warp * kPairTiles + tile) * 128 + lane * 4) =
                make_float4(acc[tile][0][0], acc[tile][0][1], acc[tile][0][2], acc[tile][0][3]);
        __syncthreads();  // and the other buffer's readers are done before it is written again
        if (threadIdx.x < kPairTiles * 64) {
            const int tile = threadIdx.x >> 6, l = (threadIdx.x & 63) >> 1, c = threadIdx.x & 1;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kMvWarps; ++w) {
                gate += r[(w * kPairTiles + tile) * 128 + l * 4 + c];
                up += r[(w * kPairTiles + tile) * 128 + l * 4 + c + 2];
            }
            const int pair = 8 * tile + (l >> 2), column = 2 * (l & 3) + c;
            if (pair < b.n && column < tokens) {
                const float v = gate / (1.0f + expf(-gate)) * up;
                const __nv_bfloat16 high = __float2bfloat16_rn(v);
                const float rest = v - __bfloat162float(high);  // an infinite value has no rest
                const __nv_bfloat16 low = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
                uint16_t* p = a.act + (int64_t)it.slot[it.off[b.item] + column] * 2 * a.I + b.i0 + pair;
                p[0] = __bfloat16_as_ushort(high);
                p[a.I] = __bfloat16_as_ushort(low);
            }
        }
        buf ^= 1;
        q += b.n;
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------ second product
// The CTA's output rows in blocks of up to 16 * MT; a block's work is the
// concatenation of all items' columns (item, step), cut into sixteen equal
// ranges.  Each warp adds its items' results, weighted, to its own sums [T][16
// * MT] in shared memory; the sixteen sums are added in warp order.
template <int GS, int MT>
__global__ void __launch_bounds__(kMvThreads, 1) moe_down_kernel(const __grid_constant__ ExpertsArgs a) {
    using F = Fmt<GS>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem + kMvWarps * F::kRingBytes);  // [warp][T][16 * MT]
    Items& it = *reinterpret_cast<Items*>(smem + kMvWarps * F::kRingBytes + kMvWarps * 64 * 64);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    pdl_trigger();
    // Before the wait: ids, weights and expert weights.  The first kernel starts
    // nothing before its own wait, so everything ahead of it has completed; it
    // writes the activations alone.
    build_items(it, a, kChunk2);

    const int r0 = (int)((int64_t)a.H * blockIdx.x / gridDim.x), r1 = (int)((int64_t)a.H * (blockIdx.x + 1) / gridDim.x);
    Rows m;
    m.q = a.w2;
    m.s = a.s2;
    m.row_bytes = F::row_bytes(a.I);
    m.row_scales = F::kW4 ? a.I / (128 / (GS ? GS : 1)) : 0;
    m.s_end = a.s2 + (int64_t)a.E * a.H * m.row_scales;
    const int steps = F::steps(a.I);
    const int total = it.count * steps;
    const int f0 = (int)((int64_t)total * warp / kMvWarps), f1 = (int)((int64_t)total * (warp + 1) / kMvWarps);
    const uint32_t ring = smem_addr(smem) + warp * F::kRingBytes;

    int crow = r0, cf = f0, ctile = 0, cslot = 0;
    int citem = f0 / steps, cstep = f0 - citem * steps;
    bool more = f0 < f1 && r0 < r1;
    auto copy_next = [&]() {
        if (more) {
            const int n = min(16 * MT, r1 - crow) - 16 * ctile;
            const int64_t lo = (int64_t)it.expert[citem] * a.H + crow + 16 * ctile;
            copy_stage<GS>(ring + cslot * F::kStageBytes, m, lo, n, lo + 8, n - 8, cstep, lane);
            cslot = cslot + 1 == F::kStages ? 0 : cslot + 1;
            if (n <= 16 || ++ctile == MT) {
                ctile = 0;
                if (++cstep == steps) {
                    cstep = 0;
                    ++citem;
                }
                if (++cf == f1) {
                    cf = f0;
                    citem = f0 / steps;
                    cstep = f0 - citem * steps;
                    crow += 16 * MT;
                    more = crow < r1;
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < F::kStages - 1; ++s) copy_next();
    pdl_wait();  // the activations

    float* mine = sums + warp * a.T * 16 * MT;
    int slot = 0;
    for (int row = r0; row < r1; row += 16 * MT) {
        const int rows = min(16 * MT, r1 - row), tiles = (rows + 15) >> 4;
        for (int i = threadIdx.x; i < kMvWarps * a.T * 16 * MT; i += kMvThreads) sums[i] = 0.0f;
        __syncthreads();
        int item = f0 / steps, step = f0 - item * steps;
        uint4 col[1][F::kBlocks], next[1][F::kBlocks];
        auto columns = [&](uint4 (&c)[1][F::kBlocks], int item, int step, bool ok) {
            const int e = g & 3;
            ok = ok && e < it.n[item];
            const uint16_t* p = a.act;
            if (ok) p += ((int64_t)it.slot[it.off[item] + e] * 2 + (g >> 2)) * a.I + (int64_t)step * F::kStepK;
            load_columns<GS, true>(c[0], p, a.I - step * F::kStepK, ok, t);
        };
        if (f0 < f1) columns(next, item, step, true);
        float acc[MT][1][4] = {};
        for (int f = f0; f < f1; ++f) {
#pragma unroll
            for (int i = 0; i < F::kBlocks; ++i) col[0][i] = next[0][i];
            const bool last = step + 1 == steps;
            if (f + 1 < f1) columns(next, last ? item + 1 : item, last ? 0 : step + 1, true);
#pragma unroll
            for (int tile = 0; tile < MT; ++tile)
                if (tile < tiles) {
                    cp_async_wait<F::kStages - 2>();
                    if (F::kW4) __syncwarp();
                    copy_next();
                    const int64_t lo = (int64_t)it.expert[item] * a.H + row + 16 * tile + g;
                    multiply_stage<GS, 1>(acc[tile], ring + slot * F::kStageBytes, col, scale_shift<GS>(m, lo, step),
                                          scale_shift<GS>(m, lo + 8, step), m.row_scales - step * GS, lane);
                    slot = slot + 1 == F::kStages ? 0 : slot + 1;
                }
            if (last || f + 1 == f1) {
                // high part + low part, times the routing weight, to the token's sums
                const int n = it.n[item], off = it.off[item];
#pragma unroll
                for (int tile = 0; tile < MT; ++tile)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = acc[tile][0][j] + __shfl_xor_sync(0xffffffffu, acc[tile][0][j], 2);
                        const int column = 2 * t + (j & 1);
                        if (t < 2 && column < n) {
                            float* y = mine + (it.slot[off + column] / a.K) * 16 * MT + 16 * tile + g + 8 * (j >> 1);
                            *y = fmaf(it.w[off + column], v, *y);
                        }
                        acc[tile][0][j] = 0.0f;
                    }
                __syncwarp();  // the next item's columns may be other lanes' tokens
            }
            if (last) {
                step = 0;
                ++item;
            } else {
                ++step;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.T * 16 * MT; i += kMvThreads) {
            const int r = i % (16 * MT), token = i / (16 * MT);
            if (r < rows) {
                float y = 0.0f;
#pragma unroll
                for (int w = 0; w < kMvWarps; ++w) y += sums[w * a.T * 16 * MT + i];
                a.out[(int64_t)token * a.H + row + r] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, const ExpertsArgs& a, int grid, int smem, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int GS>
cudaError_t launch_both(const ExpertsArgs& a, int num_sms, cudaStream_t stream, bool pdl) {
    cudaError_t e = launch(moe_gate_up_kernel<GS>, a, num_sms, smem1<GS>(), stream, pdl);
    if (e != cudaSuccess) return e;
    // the more tokens, the fewer rows' sums fit
    if (a.T <= 16) return launch(moe_down_kernel<GS, 4>, a, num_sms, smem2<GS>(), stream, true);
    if (a.T <= 32) return launch(moe_down_kernel<GS, 2>, a, num_sms, smem2<GS>(), stream, true);
    return launch(moe_down_kernel<GS, 1>, a, num_sms, smem2<GS>(), stream, true);
}

template <int GS>
cudaError_t set_attributes() {
    cudaError_t e = cudaFuncSetAttribute(moe_gate_up_kernel<GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem1<GS>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<GS, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem2<GS>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<GS, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem2<GS>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<GS, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem2<GS>());
    return e;
}

}  // namespace

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
