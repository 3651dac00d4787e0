// attn_api.cu -- C entry points of the attention of a decode layer (declared in
// include/arfuse.h): argument checks, the handle, the launches.  Nothing here
// allocates or synchronises on the call path.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "arf_check.h"
#include "arfuse.h"
#include "attn_common.cuh"

static_assert(arf::kErrPageRange == AR_DEVERR_PAGE_RANGE && arf::kErrSlotRange == AR_DEVERR_SLOT_RANGE &&
                  arf::kErrLengthRange == AR_DEVERR_LENGTH_RANGE,
              "the kernels' error bits are the header's");

namespace {

// Rotary tables that a handle has had, on the device and (to find one that is set again) here.  One is never written again:
// calls in flight and captured ones hold its address.
constexpr int kChunkTables = 64;
struct RopeChunk {
    RopeChunk* next;
    arf::RopeTable* d_tables;
    int used;
    arf::RopeTable tables[kChunkTables];
};

}  // namespace

struct ar_attn {
    int device;
    int heads, kv, D, page_size;
    int64_t max_seqs;
    unsigned flags;
    int num_sms;
    int rot, interleaved, axes;  // rotary positions (rot 0: none)
    uint8_t* d_mem;              // everything below
    unsigned* d_err;
    unsigned* d_count;  // zero between calls
    float* d_part;
    RopeChunk* ropes;                // latest first
    const arf::RopeTable* d_rope;    // the table in force
};

namespace {

using arf::aligned;
using arf::overlap;
using arf::Range;
using arf::range_of;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMostTokens = 0x7fffffff;  // of a cache, and of a sequence

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

ar_status check_device(const ar_attn* m) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return AR_ERR_CUDA;
    return cur == m->device ? AR_OK : AR_ERR_INVALID_ARG;
}

ar_status launched(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    (void)cudaGetLastError();
    return AR_ERR_CUDA;
}

// A table's place on the device, nullptr if there is none to be had.  A new one is complete there before this returns.
const arf::RopeTable* place_of_rope(ar_attn* m, const arf::RopeTable& t) {
    for (RopeChunk* c = m->ropes; c; c = c->next)
        for (int i = 0; i < c->used; ++i)
            if (std::memcmp(&c->tables[i], &t, sizeof t) == 0) return c->d_tables + i;
    RopeChunk* c = m->ropes;
    if (!c || c->used == kChunkTables) {
        c = new (std::nothrow) RopeChunk();
        if (!c) return nullptr;
        if (cudaMalloc(&c->d_tables, sizeof c->tables) != cudaSuccess) {
            delete c;
            return nullptr;
        }
        c->next = m->ropes;
        m->ropes = c;
    }
    if (cudaMemcpy(c->d_tables + c->used, &t, sizeof t, cudaMemcpyHostToDevice) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
        return nullptr;
    c->tables[c->used] = t;
    return c->d_tables + c->used++;
}

struct Dim {
    int64_t n, stride;
};

// Bytes from the first to behind the last element of keys or values; 0 if two elements would share a place or the
// strides are out of range.
int64_t extent(Dim page, Dim token, Dim head, int D, int size) {
    Dim d[3] = {page, token, head};
    int64_t most = (int64_t)1 << 47;  // more than any device holds
    for (const Dim& x : d)
        if (x.n > 1 && (x.stride < D || x.stride > most)) return 0;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].n <= 1 || (d[j + 1].n > 1 && d[j].stride > d[j + 1].stride)) {
                const Dim x = d[j];
                d[j] = d[j + 1];
                d[j + 1] = x;
            }
    // by stride, the single ones last: each has to step over all that is inside it
    int64_t inside = D;
    for (const Dim& x : d) {
        if (x.n <= 1) continue;
        if (x.stride < inside || x.n > most / x.stride) return 0;
        inside = (x.n - 1) * x.stride + inside;
    }
    return inside > most ? 0 : inside * size;
}

struct Cache {
    arf::CacheView k, v;
    Range k_range, v_range;
};

ar_status check_cache(const ar_attn* m, const ar_kv_cache* c, Cache* out) {
    if (!c || !c->k || !c->v || c->pages < 1 || !c->k_scale != !c->v_scale) return AR_ERR_INVALID_ARG;
    if (c->pages > kMostTokens / m->page_size) return AR_ERR_UNSUPPORTED;
    const int size = c->k_scale ? 1 : 2, step = 16 / size;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return AR_ERR_ALIGNMENT;
    const int64_t strides[6] = {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head};
    const int64_t counts[3] = {c->pages, m->page_size, m->kv};
    for (int i = 0; i < 6; ++i)
        if (counts[i % 3] > 1 && strides[i] % step != 0) return AR_ERR_ALIGNMENT;
    const int64_t kb = extent({c->pages, c->k_page}, {m->page_size, c->k_token}, {m->kv, c->k_head}, m->D, size);
    const int64_t vb = extent({c->pages, c->v_page}, {m->page_size, c->v_token}, {m->kv, c->v_head}, m->D, size);
    if (kb == 0 || vb == 0) return AR_ERR_INVALID_ARG;
    out->k = {static_cast<uint8_t*>(c->k), c->k_page * size, c->k_token * size, c->k_head * size, c->k_scale};
    out->v = {static_cast<uint8_t*>(c->v), c->v_page * size, c->v_token * size, c->v_head * size, c->v_scale};
    if (c->pages <= 1) out->k.page = out->v.page = 0;
    if (m->page_size <= 1) out->k.token = out->v.token = 0;
    if (m->kv <= 1) out->k.head = out->v.head = 0;
    out->k_range = range_of(c->k, kb);
    out->v_range = range_of(c->v, vb);
    return AR_OK;
}

}  // namespace

extern "C" {

ar_status ar_attn_create(int device, int heads, int kv_heads, int head_dim, int page_size, int64_t max_seqs, unsigned flags,
                         ar_attn** out) {
    if (!out) return AR_ERR_INVALID_ARG;
    *out = nullptr;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || page_size < 1 || max_seqs < 1) return AR_ERR_INVALID_ARG;
    if ((flags & ~(AR_WS_DRY_RUN | AR_WS_PDL)) != 0) return AR_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || heads > AR_MAX_ATTN_HEADS || page_size > AR_MAX_PAGE_SIZE ||
        max_seqs > AR_MAX_ATTN_SEQS)
        return AR_ERR_UNSUPPORTED;
    ar_attn* m = new (std::nothrow) ar_attn();
    if (!m) return AR_ERR_CUDA;
    m->device = device;
    m->heads = heads;
    m->kv = kv_heads;
    m->D = head_dim;
    m->page_size = page_size;
    m->max_seqs = max_seqs;
    m->flags = flags;
    if (flags & AR_WS_DRY_RUN) {
        *out = m;
        return AR_OK;
    }
    int prev = -1, major = 0;
    size_t count = 0;
    ar_status st = AR_ERR_CUDA;
    if (cudaGetDevice(&prev) == cudaSuccess && cudaSetDevice(device) == cudaSuccess &&
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) == cudaSuccess &&
        cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess) {
        count = round_up(arf::attn_decode_counters(m->num_sms) * sizeof(unsigned));
        const size_t part = arf::attn_decode_parts(m->num_sms, head_dim) * sizeof(float);
        if (major < 10)
            st = AR_ERR_UNSUPPORTED;
        else if (arf::attn_decode_set_attributes() == cudaSuccess &&
                 cudaMalloc(&m->d_mem, 256 + count + part) == cudaSuccess &&
                 cudaMemset(m->d_mem, 0, 256 + count) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess)
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
    m->d_part = reinterpret_cast<float*>(m->d_mem + 256 + count);
    *out = m;
    return AR_OK;
}

ar_status ar_attn_destroy(ar_attn* m) {
    if (!m) return AR_OK;
    ar_status st = AR_OK;
    if (m->d_mem) {
        int prev = -1;
        (void)cudaGetDevice(&prev);
        bool ok = cudaSetDevice(m->device) == cudaSuccess;
        ok = ok && cudaFree(m->d_mem) == cudaSuccess;
        while (RopeChunk* c = m->ropes) {
            ok = ok && cudaFree(c->d_tables) == cudaSuccess;
            m->ropes = c->next;
            delete c;
        }
        if (!ok) {
            (void)cudaGetLastError();
            st = AR_ERR_CUDA;
        }
        if (prev >= 0) (void)cudaSetDevice(prev);
    }
    delete m;
    return st;
}

ar_status ar_attn_device_error(ar_attn* m, int* code) {
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

ar_status ar_attn_set_rope(ar_attn* m, int rot, int interleaved, int axes, const double* freq, const int32_t* axis) {
    if (!m || rot < 0 || rot > m->D || (interleaved != 0 && interleaved != 1)) return AR_ERR_INVALID_ARG;
    if (rot % 16 != 0) return AR_ERR_UNSUPPORTED;
    if (rot > 0 && (axes < 1 || axes > AR_MAX_ROPE_AXES || !freq)) return AR_ERR_INVALID_ARG;
    arf::RopeTable t;
    std::memset(&t, 0, sizeof t);
    for (int i = 0; i < rot / 2; ++i) {
        if (!std::isfinite(freq[i]) || (axis && (axis[i] < 0 || axis[i] >= axes))) return AR_ERR_INVALID_ARG;
        const double turns = std::fabs(freq[i]) / 6.283185307179586476925286766559;
        t.turns[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
        if (freq[i] < 0) t.turns[i] = 0 - t.turns[i];
        t.axis[i] = axis ? axis[i] : 0;
    }
    if (rot > 0 && !(m->flags & AR_WS_DRY_RUN)) {
        int prev = -1;
        (void)cudaGetDevice(&prev);
        const arf::RopeTable* d = cudaSetDevice(m->device) == cudaSuccess ? place_of_rope(m, t) : nullptr;
        if (!d) (void)cudaGetLastError();
        if (prev >= 0) (void)cudaSetDevice(prev);
        if (!d) return AR_ERR_CUDA;
        m->d_rope = d;
    }
    m->rot = rot;
    m->interleaved = interleaved;
    m->axes = rot > 0 ? axes : 0;
    return AR_OK;
}

ar_status ar_attn_append(ar_attn* m, const ar_kv_cache* cache, const void* qkv, const int32_t* positions, const int32_t* slots,
                         int64_t T, void* q, void* stream) {
    if (!m || T < 0) return AR_ERR_INVALID_ARG;
    if (T > AR_MAX_ATTN_TOKENS) return AR_ERR_CAPACITY;
    Cache c;
    const ar_status st = check_cache(m, cache, &c);
    if (st != AR_OK) return st;
    if (cache->k == cache->v) return AR_ERR_INVALID_ARG;
    if (T == 0) return AR_OK;
    if (!qkv || !slots || !q || (m->rot > 0 && !positions)) return AR_ERR_INVALID_ARG;
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(slots, 4) || !aligned(positions, 4)) return AR_ERR_ALIGNMENT;
    const Range in[5] = {range_of(qkv, T * (m->heads + 2 * m->kv) * m->D * 2), range_of(slots, T * 4),
                         range_of(positions, positions ? T * m->axes * 4 : 0), range_of(cache->k_scale, cache->k_scale ? m->kv * 4 : 0),
                         range_of(cache->v_scale, cache->v_scale ? m->kv * 4 : 0)};
    const Range r_q = range_of(q, T * m->heads * m->D * 2);
    if (overlap(r_q, c.k_range) || overlap(r_q, c.v_range)) return AR_ERR_INVALID_ARG;
    for (const Range& r : in)
        if (overlap(r, r_q) || overlap(r, c.k_range) || overlap(r, c.v_range)) return AR_ERR_INVALID_ARG;
    if (m->flags & AR_WS_DRY_RUN) return AR_VALIDATED;
    const ar_status dev = check_device(m);
    if (dev != AR_OK) return dev;
    arf::AppendArgs a;
    std::memset(&a, 0, sizeof a);
    a.qkv = static_cast<const uint16_t*>(qkv);
    a.positions = positions;
    a.slots = slots;
    a.rope = m->d_rope;
    a.q = static_cast<uint16_t*>(q);
    a.k = c.k;
    a.v = c.v;
    a.err = m->d_err;
    a.slot_count = cache->pages * m->page_size;
    a.T = (int)T;
    a.heads = m->heads;
    a.kv = m->kv;
    a.D = m->D;
    a.page_size = m->page_size;
    a.rot = m->rot;
    a.interleaved = m->interleaved;
    return launched(arf::launch_attn_append(a, m->num_sms, static_cast<cudaStream_t>(stream)));
}

ar_status ar_attn_decode(ar_attn* m, const ar_kv_cache* cache, const void* q, const int32_t* page_table, int64_t table_width,
                         int64_t table_stride, const int32_t* lengths, int64_t B, int64_t window, float scale, void* out,
                         float* lse, void* stream) {
    if (!m || B < 0 || table_width < 0 || window < 0 || !std::isfinite(scale * kLog2e)) return AR_ERR_INVALID_ARG;
    if (B > m->max_seqs) return AR_ERR_CAPACITY;
    Cache c;
    const ar_status st = check_cache(m, cache, &c);
    if (st != AR_OK) return st;
    if (B == 0) return AR_OK;
    if (table_stride < table_width && B > 1) return AR_ERR_INVALID_ARG;
    if (table_stride > INT64_MAX / 4 / AR_MAX_ATTN_SEQS || table_width > kMostTokens) return AR_ERR_UNSUPPORTED;
    if (!q || (!page_table && table_width > 0) || !lengths || !out) return AR_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return AR_ERR_ALIGNMENT;
    const int64_t row = (int64_t)m->heads * m->D * 2;
    const Range outs[2] = {range_of(out, B * row), range_of(lse, lse ? B * m->heads * 4 : 0)};
    const Range in[7] = {range_of(q, B * row), range_of(lengths, B * 4),
                         range_of(page_table, table_width > 0 ? ((B - 1) * table_stride + table_width) * 4 : 0), c.k_range, c.v_range,
                         range_of(cache->k_scale, cache->k_scale ? m->kv * 4 : 0),
                         range_of(cache->v_scale, cache->v_scale ? m->kv * 4 : 0)};
    if (overlap(outs[0], outs[1])) return AR_ERR_INVALID_ARG;
    for (const Range& o : outs)
        for (const Range& r : in)
            if (overlap(o, r)) return AR_ERR_INVALID_ARG;
    if (m->flags & AR_WS_DRY_RUN) return AR_VALIDATED;
    const ar_status dev = check_device(m);
    if (dev != AR_OK) return dev;
    arf::DecodeArgs a;
    std::memset(&a, 0, sizeof a);
    a.q = static_cast<const uint16_t*>(q);
    a.table = page_table;
    a.lengths = lengths;
    a.k = c.k;
    a.v = c.v;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.err = m->d_err;
    a.count = m->d_count;
    a.part = m->d_part;
    a.table_stride = table_stride;
    const int64_t most = table_width * m->page_size;
    a.most = most < kMostTokens ? most : kMostTokens;
    a.pages = (int)cache->pages;
    a.B = (int)B;
    a.heads = m->heads;
    a.kv = m->kv;
    a.page_size = m->page_size;
    // 2^(s - 1) < page_size <= 2^s: m = ceil(2^(31 + s) / page_size) < 2^32, and m page_size passes 2^(31 + s) by less than
    // 2^s, too little for the quotient of a number below 2^31 to change
    while ((1 << a.page_shift) < m->page_size) ++a.page_shift;
    a.page_mul = (unsigned)((((uint64_t)1 << (31 + a.page_shift)) + m->page_size - 1) / m->page_size);
    a.window = (int)(window < kMostTokens ? window : 0);
    a.scale = scale * kLog2e;
    return launched(arf::launch_attn_decode(a, m->D, m->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
