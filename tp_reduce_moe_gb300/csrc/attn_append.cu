// attn_append.cu -- rotary positions and the write into the paged cache.
//
// Pair i of the first `rot` columns of a q or k head is turned by the angle
// freq[i] * position[axis[i]]; q goes out, k and v go to their slots of the cache.
//
// A piece is sixteen values of a head, of which a thread loads, turns and stores two
// groups of eight: both halves of eight pairs, so no value is exchanged between threads.
// A token's cosines and sines are formed once a CTA, in shared memory: the angle as a
// fraction of a turn in 64-bit integers, whose overflow takes the whole turns off, so that
// far positions lose nothing, then sincospi in fp32 of its upper half.
//
// What bounds it: memory, for many tokens (8192 of 64 + 2 x 8 heads of 128 columns: 55.6 us, 6 TB/s
// of what is read and written), and for few the launch, the slots and the positions (2.8 us).
//
// Of tokens with one slot the last one wins whatever order the CTAs run in: each CTA
// looks through the slots behind its own tokens and leaves out what is written again.
// A bitmap of its own slots (hashed by their low bits) answers for nearly all of them.  (With
// looks, angles and places 8192 tokens of 8 + 2 heads take 17.4 us, 6.2 of memory; 65536 121 and 50, of 32 + 16 heads 292 and 238.)
#include "attn_common.cuh"

namespace arf {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;  // of a CTA
constexpr int kTableTokens = 4; // whose angles are in shared memory at a time
constexpr int kHashBits = 14;
constexpr int kAhead = 4;       // pieces that a thread has asked for
constexpr int kScan = 8;        // slots that a thread has asked for
constexpr int kCtas = 5;        // that an SM has room for

// Sixteen bytes of what the kernel before may have written, to a place that only this thread reads.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Chunks (of eight columns) of piece p of a head: one of each half of the rotated columns, or of those behind, so that
// neighbouring threads' are neighbours (and sectors of memory are asked for once).
__device__ __forceinline__ void chunks_of(int p, int rot, int all, int* lo, int* hi) {
    const int turned = rot / 16;
    *lo = p < turned ? p : p + turned;
    *hi = *lo + (p < turned ? turned : all - turned);
}

__device__ __forceinline__ void store8(const CacheView& c, int head, int64_t token, int chunk, const float f[8]) {
    uint8_t* row = c.data + token + head * c.head;
    if (c.scale == nullptr) {
        *reinterpret_cast<uint4*>(row + chunk * 16) = f32x8_to_bf16x8(f);
        return;
    }
    const float s = c.scale[head];
    uint2 v;
    v.x = e4m3x2(f[0] / s, f[1] / s) | e4m3x2(f[2] / s, f[3] / s) << 16;
    v.y = e4m3x2(f[4] / s, f[5] / s) | e4m3x2(f[6] / s, f[7] / s) << 16;
    *reinterpret_cast<uint2*>(row + chunk * 8) = v;
}

__global__ void __launch_bounds__(kThreads, kCtas) attn_append_kernel(const __grid_constant__ AppendArgs a, int tokens_per_cta) {
    __shared__ int s_slot[kMaxTokens];
    __shared__ int s_dead[kMaxTokens];
    __shared__ int64_t s_k[kMaxTokens], s_v[kMaxTokens];  // byte offsets of the tokens' places, -1: none
    __shared__ unsigned s_hash[1 << (kHashBits - 5)];
    // Cosine and sine of a token's pairs, two beside each other, so that neighbouring pieces' are in neighbouring banks:
    // 8 p + 2 j and the next at 32 j + 2 p; of neighbouring columns 4 c + 2 k and the next, those of chunk c, at 64 k + 2 c.
    __shared__ __align__(16) float2 s_turn[kTableTokens][kMaxHeadDim / 2];
    __shared__ uint4 s_piece[kAhead][2][kThreads];
    pdl_trigger();
    pdl_wait();  // no global memory access before this point
    const int t0 = blockIdx.x * tokens_per_cta, count = min(tokens_per_cta, a.T - t0);
    const int shift = 31 - __clz(a.D / 16), per_head = 1 << shift, all_heads = a.heads + 2 * a.kv;
    // this CTA's pieces of a token
    const int pieces = all_heads * per_head;
    const int first = (int)((int64_t)pieces * blockIdx.y / gridDim.y);
    const int own = (int)((int64_t)pieces * (blockIdx.y + 1) / gridDim.y) - first;

    // a thread's pieces, every kThreads-th of all tokens' one after the other, are asked for ahead of anything else; one comes
    // from the one before without a division
    const int on_t = kThreads / own, on_r = kThreads - on_t * own;
    struct Place {
        int t, r;  // token, piece of it
    };
    auto follow = [&](Place& x) {
        x.t += on_t;
        x.r += on_r;
        if (x.r >= own) {
            x.r -= own;
            ++x.t;
        }
    };
    Place use;
    use.t = threadIdx.x / own;
    use.r = threadIdx.x - use.t * own;
    Place next = use;
    int slot = 0;
    const uint16_t* const rows = a.qkv + (int64_t)t0 * all_heads * a.D;
    auto ask = [&](int into) {
        if (next.t < count) {
            const int r = first + next.r, head = r >> shift;
            int lo, hi;
            chunks_of(r - (head << shift), head < a.heads + a.kv ? a.rot : 0, per_head, &lo, &hi);
            const uint16_t* row = rows + (next.t * all_heads + head) * a.D;
            copy16(smem_addr(&s_piece[into][0][threadIdx.x]), row + lo * 8);
            copy16(smem_addr(&s_piece[into][1][threadIdx.x]), row + hi * 8);
            follow(next);
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) ask(i);

    // places in the cache
    if (first + own > a.heads * per_head) {
        for (int i = threadIdx.x; i < 1 << (kHashBits - 5); i += kThreads) s_hash[i] = 0;
        if ((int)threadIdx.x < count) {
            int slot = a.slots[t0 + threadIdx.x];
            if (slot < -1 || slot >= a.slot_count) {
                atomicOr(a.err, kErrSlotRange);
                slot = -1;
            }
            s_slot[threadIdx.x] = slot;
            s_dead[threadIdx.x] = slot < 0;
        }
        __syncthreads();
        if ((int)threadIdx.x < count && s_slot[threadIdx.x] >= 0) {
            const unsigned h = (unsigned)s_slot[threadIdx.x] & ((1u << kHashBits) - 1);
            atomicOr(&s_hash[h >> 5], 1u << (h & 31));
        }
        __syncthreads();
        // eight loads in flight: one after the other they would take longer than the copies
#pragma unroll 1
        for (int t = t0 + 1 + threadIdx.x; t < a.T; t += kScan * kThreads) {
            int later[kScan];
#pragma unroll
            for (int k = 0; k < kScan; ++k) later[k] = t + k * kThreads < a.T ? a.slots[t + k * kThreads] : -1;
#pragma unroll
            for (int k = 0; k < kScan; ++k) {
                const unsigned h = (unsigned)later[k] & ((1u << kHashBits) - 1);
                if (later[k] < 0 || !(s_hash[h >> 5] >> (h & 31) & 1)) continue;
#pragma unroll 1
                for (int i = 0; i < count && t0 + i < t + k * kThreads; ++i)
                    if (s_slot[i] == later[k]) s_dead[i] = 1;
            }
        }
        __syncthreads();
        if ((int)threadIdx.x < count) {
            const int slot = s_slot[threadIdx.x];
            const int page = slot / a.page_size, token = slot - page * a.page_size;
            const bool dead = s_dead[threadIdx.x] != 0;
            s_k[threadIdx.x] = dead ? -1 : page * a.k.page + token * a.k.token;
            s_v[threadIdx.x] = dead ? -1 : page * a.v.page + token * a.v.token;
        }
    }

    const int pairs = a.rot / 2;
    uint16_t* const out = a.q + (int64_t)t0 * a.heads * a.D;
    for (int b = 0; b < count; b += kTableTokens) {
        const int n = min(kTableTokens, count - b);
        for (int j = threadIdx.x; j < n * pairs; j += kThreads) {
            const int t = j / pairs, pair = j - t * pairs;
            const uint64_t turns = (int64_t)a.positions[(int64_t)a.rope->axis[pair] * a.T + t0 + b + t] * a.rope->turns[pair];
            float s, c;
            sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
            s_turn[t][a.interleaved ? (pair & 2) * 32 + (pair >> 2) * 2 + (pair & 1) : (pair & 6) * 16 + (pair >> 3) * 2 + (pair & 1)] = make_float2(c, s);
        }
        __syncthreads();
        for (; use.t < b + n; follow(use)) {
            copy_wait<kAhead - 1>();
            const uint4 x_lo = s_piece[slot][0][threadIdx.x], x_hi = s_piece[slot][1][threadIdx.x];
            ask(slot);
            slot = slot + 1 == kAhead ? 0 : slot + 1;
            const int t = use.t, r = first + use.r, head = r >> shift, p = r - (head << shift);
            const bool turned = head < a.heads + a.kv && p < a.rot / 16;
            int lo, hi;
            chunks_of(p, head < a.heads + a.kv ? a.rot : 0, per_head, &lo, &hi);
            float u[8], v[8];
            bf16x8_to_f32(x_lo, u);
            bf16x8_to_f32(x_hi, v);
            if (turned) {
                float2 table[8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float4*>(table + 2 * j) =
                        *reinterpret_cast<const float4*>(&s_turn[t - b][a.interleaved ? (j & 1) * 64 + (j < 2 ? lo : hi) * 2 : j * 32 + p * 2]);
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = table[j], g = table[j + 4];
                        const float ua = u[2 * j], ub = u[2 * j + 1], va = v[2 * j], vb = v[2 * j + 1];
                        u[2 * j] = ua * f.x - ub * f.y;
                        u[2 * j + 1] = ub * f.x + ua * f.y;
                        v[2 * j] = va * g.x - vb * g.y;
                        v[2 * j + 1] = vb * g.x + va * g.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = table[j];
                        const float x0 = u[j], x1 = v[j];
                        u[j] = x0 * f.x - x1 * f.y;
                        v[j] = x1 * f.x + x0 * f.y;
                    }
                }
            }
            if (head < a.heads) {
                uint16_t* row = out + (t * a.heads + head) * a.D;
                st_global16(row + lo * 8, f32x8_to_bf16x8(u));
                st_global16(row + hi * 8, f32x8_to_bf16x8(v));
                continue;
            }
            const bool key = head < a.heads + a.kv;
            const int64_t place = key ? s_k[t] : s_v[t];
            if (place < 0) continue;
            const int h = key ? head - a.heads : head - a.heads - a.kv;
            store8(key ? a.k : a.v, h, place, lo, u);
            store8(key ? a.k : a.v, h, place, hi, v);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_attn_append(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    const int pieces = (a.heads + 2 * a.kv) * (a.D / 16);
    // Few tokens: a token's pieces over several CTAs; many: several tokens a CTA, so that all CTAs have room at once.  (1024
    // tokens of 32 + 2 x 8 heads of 128 columns: 7.4 us; with eight CTAs to an SM in two waves, 10.0; 8192 of them 38.1 and 41.3.)
    const int target = kCtas * num_sms;
    int tokens = (a.T + target - 1) / target;
    if (tokens > kMaxTokens) tokens = kMaxTokens;
    const int blocks = (a.T + tokens - 1) / tokens;
    int parts = (pieces + kThreads - 1) / kThreads;
    if (parts > (target + blocks - 1) / blocks) parts = (target + blocks - 1) / blocks;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)parts);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_append_kernel, a, tokens);
}

}  // namespace arf
