// How the code scoring shares a long row among warps and blocks, on the host: every
// plan is one the kernel takes, and it follows the number of SMs that it is given.
#include <cstdio>

#include "logprobs.cu"

int main() {
    using namespace tts;
    long n = 0;
    for (int sms : {1, 16, 76, 132, 152, 304})
        for (int V = kRun + 1; V <= 1 << 20; V += V / 7 + 1)
            for (int items = 1; items < 200000; items += items / 3 + 1) {
                const LongPlan p = plan_long(items, V, sms);
                const int runs = (V + kRun - 1) / kRun;
                const bool power = p.blocks == 1 || p.blocks == 2 || p.blocks == 4 || p.blocks == 8;
                if (p.warps < 1 || p.warps > kLongWarps || p.warps > runs || !power) return std::printf("shape %d %d\n", V, items), 1;
                if (p.blocks > 1 && (p.blocks / 2 * p.warps >= runs || (long long)items * p.blocks / 2 >= sms))
                    return std::printf("more blocks than wanted: %d SMs %d x %d\n", sms, items, V), 1;
                if (p.blocks < 8 && p.blocks * p.warps < runs && (long long)items * p.blocks < sms)
                    return std::printf("SMs left: %d SMs %d x %d\n", sms, items, V), 1;
                ++n;
            }
    // rows enough for one device are a cluster's on one of twice the SMs
    const int a = plan_long(152, 1 << 20, 152).blocks, b = plan_long(152, 1 << 20, 304).blocks;
    std::printf("%ld plans; 152 rows of 2^20: %d block on 152 SMs, %d on 304\n", n, a, b);
    return a == 1 && b == 2 ? 0 : 1;
}
