// How the 4-bit GEMV divides its work, on the host: every plan covers all tiles and
// groups of K with blocks that fit an SM, and the form whose sums take the
// activations' place is used where it saves a round of blocks, nowhere else.
#include <cstdio>

#include "w4.cu"

using namespace tts;

#define CHECK(x)                                                                                             \
    do {                                                                                                     \
        if (!(x)) return std::printf("%s: M %d epi %d N %d K %d, %d SMs\n", #x, M, epi, N, K, sms), false;   \
    } while (0)

static long plans = 0, taken = 0;

static bool check(int M, int epi, int N, int K, int sms) {
    W4Params p{};
    p.M = M, p.N = N, p.K = K, p.epi = epi;
    const int mv = M, parts = epi == 2 ? 2 : 1, at_once[4] = {sms, sms > 1 ? sms / 2 : 0, std::max(0, sms / 4 - 2), std::max(0, sms / 8 - 4)};
    const int groups = K / kW4Group, ntiles = (N + 15) / 16;
    W4Launch own{};
    for (int in_act = 0; in_act <= (int)has_in_act(mv, parts); ++in_act) {
        const W4Launch c = plan_gemv_w4(p, mv, parts, in_act, at_once);
        if (!c.warps && sms == 1) continue;  // K that wants a cluster, on a device without room for one
        ++plans;
        CHECK(c.warps >= 1 && c.warps <= c.share && c.warps <= max_warps(mv) && c.tiles >= 1);
        CHECK(c.tiles <= (in_act ? kMaxTiles / 2 : kMaxTiles) && c.smem <= kBlockSmem);
        CHECK((long)c.grid * c.tiles >= ntiles && c.grid <= ntiles && (long)(c.tiles - 1) * c.grid < ntiles);
        const int split = 1 << c.log_split;
        for (int r = 0; r < split; ++r) {
            const int kg = (groups * (r + 1) >> c.log_split) - (groups * r >> c.log_split);
            CHECK(kg >= 1 && kg <= c.share && (int)(kg * c.magic >> 32) == kg / c.warps);
        }
        const W4Smem o = smem_of(mv, parts, in_act, c.tiles, c.share, c.warps);
        CHECK(o.act % 16 == 0 && o.par % 16 == 0 && o.scales % 16 == 0 && o.sums % 16 == 0 && o.sq % 4 == 0);
        if (!in_act) own = c;
        if (in_act && saves_a_round(c, own, at_once)) {
            ++taken;
            CHECK(!own.warps || rounds_of(c, at_once) < rounds_of(own, at_once));
        }
        // gate/up rows of four vectors that fit both ways, and only one way
        if (in_act && sms == 152 && N == 6144 && K == 2560) CHECK(!saves_a_round(c, own, at_once));
        if (in_act && sms == 152 && N == 9728 && K == 2560) CHECK(saves_a_round(c, own, at_once));
    }
    return true;
}

int main() {
    for (int sms : {1, 76, 132, 152})
        for (int M : {1, 2, 4, 8})
            for (int epi : {0, 2})
                for (int K = 128; K <= 12288; K += 128)
                    for (int N : {1, 15, 16, 17, 500, 2560, 4096, 6144, 8208, 9728, 16384, 200000, 16777216})
                        if (!check(M, epi, N, K, sms)) return 1;
    std::printf("%ld plans, %ld with the sums in the activations' place\n", plans, taken);
    return taken > 0 ? 0 : 1;
}
