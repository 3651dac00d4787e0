// Host check of the shared-memory plans of the weight-streaming kernels, over their sizes.
#include <cstdio>

#include "moe_experts.cu"

using namespace arf;

static long plans = 0, bad = 0;
#define CHECK(c)                                                                             \
    do {                                                                                     \
        if (!(c)) {                                                                          \
            if (bad++ < 10) printf("line %d: %s (GS %d, sizes %d %d %d %d)\n", __LINE__, #c, GS, a, b, c1, d); \
        }                                                                                    \
    } while (0)

template <int GS>
void product(int K, int tokens, int columns, int tiles, int extra) {
    using View = StagedView<GS ? GS : 1>;
    const int a = K, b = tokens, c1 = columns, d = tiles;
    const ProductPlan p = plan_product<GS>(K, tokens, columns, tiles, extra);
    ++plans;
    const int segments = p.shape.segments, job = tiles < kJobTiles<GS> ? tiles : kJobTiles<GS>;
    CHECK(p.tiles == job && p.pairs * 2 >= (tokens < 8 ? tokens : 8));
    // barriers, parts (warp 15 of the last tile is at tiles + 14), sums, staged, extra, rings, scales: one behind the other
    CHECK(p.sums_at >= kMvWarps * kMaxSlots * 8 + kPartBuffers<GS> * (job + kMvWarps) * p.pairs * 128);
    CHECK(p.staged_at >= p.sums_at && p.staged_at % 16 == 0 && p.extra_at % 16 == 0);
    CHECK(p.ring_at >= p.extra_at + extra && p.ring_at % 1024 == 0);
    CHECK(p.scales_at == p.ring_at + kMaxSlots * kMvWarps * kSlotBytes);
    CHECK(p.smem == p.scales_at + (GS ? kMaxSlots * kMvWarps * Scales<GS ? GS : 1>::kSlot : 0) && p.smem <= kSmemLimit);
    CHECK(kMoeMaxExperts * 8 <= kMaxSlots * kMvWarps * kSlotBytes);  // the items' masks
    for (int n = 1; GS && n <= 8; ++n) {
        const int panel = p.panel[n];
        CHECK(n > tokens || (panel >= 1 && panel <= segments));
        CHECK(n <= tokens || panel == 0 || panel == segments);
        CHECK(p.staged_at + View::bytes(panel, n) <= p.extra_at || panel == 0);
        CHECK(n > tokens || panel == segments || p.staged_at >= p.sums_at + job * p.pairs * 128);
    }
}

template <int GS>
void down(int T, int K, int E, int I, int tiles) {
    const int a = T, b = K, c1 = E, d = I;
    const DownPlan p = plan_down<GS>(T, K, E, I, tiles);
    ++plans;
    constexpr int kScales = GS ? Scales<GS ? GS : 1>::kSlot : 0;
    CHECK(p.slots >= 1 && p.slots <= kMaxSlots && p.round >= 1 && p.round <= tiles);
    CHECK(p.items_at >= (kMaxSlots + 1) * kMvWarps * 8 + p.round * kMvWarps * T * 64 && p.items_at % 16 == 0);
    CHECK(p.ring_at >= p.items_at + Items::bytes(T * K, E) && p.ring_at % 1024 == 0);
    CHECK(p.step == kSlotBytes || (p.step == kSlotBytes / 2 && p.shape.row_bytes <= kBox));
    CHECK(p.scales_at == p.ring_at + p.slots * kMvWarps * p.step && p.act_at == p.scales_at + p.slots * kMvWarps * kScales);
    CHECK(p.act_at % 128 == 0 && p.act_entry % 16 == 0 && p.smem >= p.act_at + T * K * p.act_entry && p.smem <= kSmemLimit);
    CHECK(p.act_entry == 0 || (GS && p.act_entry >= 2 * p.act_part && p.act_part >= (2 * I + 511) / 512 * 512));
    CHECK(E * 8 <= p.slots * kMvWarps * p.step);  // the items' masks
}

template <int GS>
void all() {
    const int step = GS ? 128 / GS : 8, most = GS ? 65536 : 16384;
    const int tiles[] = {1, 2, 3, 7, 8, 16, 27, 31, 32, 33, 400};
    for (int K = step; K <= most; K += step * (K < 2048 ? 1 : 13))
        for (int t : tiles)
            for (int tokens = 1; tokens <= 8; ++tokens) {
                product<GS>(K, tokens, 8, t, 0);
                if (K <= 16384)
                    for (int slots : {1, 8, 128, 1024}) product<GS>(K, tokens, tokens, t, Items::bytes(slots, 512));
                if (K <= 16384 && tokens <= 4) product<GS>(K, tokens, 8, t, Items::bytes(1024, 512));
            }
    for (int T = 1; T <= 64; ++T)
        for (int K = 1; K <= 16; ++K)
            for (int I = step; I <= 16384; I = I < 8 * step ? I + step : I * 5 / 4 / step * step)
                for (int tiles : {1, 3, 4, 7}) {
                    down<GS>(T, K, 512, I, tiles);
                    down<GS>(T, K, 1, I, tiles);
                }
}

int main() {
    all<0>();
    all<1>();
    all<2>();
    all<4>();
    printf("%ld plans, %ld bad\n", plans, bad);
    return bad != 0;
}
