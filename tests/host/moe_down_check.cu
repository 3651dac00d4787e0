// Host check of the pieces that group scales are copied in, and of which plan the experts' second product takes: the first that fits, of padded entries with a round's tiles,
// padded entries with one tile, entries without padding with one tile, and activations that are not staged.
#include <cstdio>

#include "moe_experts.cu"

using namespace arf;

static long plans[4], bad = 0;

template <int GS>
static bool fits(int T, int K, int E, int round, int step, int entry) {
    const int items_at = (kMaxSlots + 1) * kMvWarps * 8 + round * kMvWarps * T * 64;
    const int ring_at = (items_at + Items::bytes(T * K, E) + 1023) / 1024 * 1024;
    return ring_at + kMaxSlots * kMvWarps * (step + Scales<GS>::kSlot) + T * K * entry <= kSmemLimit;
}

template <int GS>
static void check(int T, int K, int E, int I, int tiles) {
    const DownPlan p = plan_down<GS>(T, K, E, I, tiles);
    const int most = 48 * 1024 / (kMvWarps * T * 64), many = most < 1 ? 1 : tiles < most ? tiles : most;
    const int part = (I * 2 + 511) / 512 * 512, step = I / 2 <= kBox ? kSlotBytes / 2 : kSlotBytes;
    const bool first = fits<GS>(T, K, E, many, step, 2 * part + 64), second = fits<GS>(T, K, E, 1, step, 2 * part + 64),
               third = fits<GS>(T, K, E, 1, step, 2 * part);
    const int entry = first || second ? 2 * part + 64 : third ? 2 * part : 0, round = first || !(second || third) ? many : 1;
    ++plans[first ? 0 : second ? 1 : third ? 2 : 3];
    if (p.act_entry != entry || p.round != round) {
        if (bad++ < 10)
            printf("GS %d, %d tokens, %d slots, %d experts of %d, %d tiles: entries of %d, rounds of %d; %d and %d would fit\n", GS, T, K, E, I, tiles,
                   p.act_entry, p.round, entry, round);
    }
}

// Rows of a multiple of eight scales take a tensor copy (0); so no piece is larger than 8 bytes, and 8 are a lane's half row
// with two groups a step alone.
template <int GS>
static void pieces() {
    bool met[9] = {};
    for (int n = 1; n <= 4096; ++n) {
        const int p = Scales<GS>::piece(n);
        const bool right = p == 0 ? n % 8 == 0 : n % 8 != 0 && n * 2 % p == 0 && (p == 8 ? GS == 2 : p == 4 ? GS != 2 || n % 4 != 0 : p == 2 && n % 2 == 1);
        if (!right && bad++ < 10) printf("GS %d, %d scales a row: pieces of %d\n", GS, n, p);
        if (p >= 0 && p <= 8) met[p] = true;
    }
    if (!(met[0] && met[2] && met[4]) || met[8] != (GS == 2)) ++bad;
}

int main() {
    pieces<1>();
    pieces<2>();
    pieces<4>();
    for (int T = 1; T <= 64; ++T)
        for (int K = 1; K <= 16; ++K)
            for (int I = 128; I <= 16384; I += I < 2048 ? 128 : 1024)
                for (int tiles : {1, 2, 3, 4, 7})
                    for (int E : {8, 256, 512}) {
                        check<1>(T, K, E, I, tiles);
                        check<2>(T, K, E, I, tiles);
                        check<4>(T, K, E, I, tiles);
                    }
    printf("%ld %ld %ld %ld plans, %ld bad\n", plans[0], plans[1], plans[2], plans[3], bad);
    return bad != 0 || !plans[0] || !plans[1] || !plans[2] || !plans[3];
}
