// A barrier that is completed 1.3 s after the wait began, past one wait's limit:
// mbar_wait gives up, mbar_arrived does not.  Every loop here is bounded.
#include <cstdio>

#include "fourbit.cuh"

__global__ void check(int* got) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        tts::mbar_init(&bar, 1);
        tts::fence_mbar_init();
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) got[0] = tts::mbar_wait(&bar, 0);
    if (threadIdx.x == 32) got[1] = tts::mbar_arrived(&bar);
    if (threadIdx.x == 64) {
        const uint64_t t0 = tts::globaltimer_ns();
        for (int i = 0; i < 4000000 && tts::globaltimer_ns() - t0 < 1300000000ull; ++i) __nanosleep(1000);
        tts::mbar_arrive_expect_tx(&bar, 0);
    }
    __syncwarp();
    if (warp == 3) got[2] = 1;
}

int main() {
    int *d = nullptr, h[3] = {-1, -1, -1};
    if (cudaMalloc(&d, sizeof(h)) != cudaSuccess) return 2;
    check<<<1, 128>>>(d);
    if (cudaMemcpy(h, d, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
    std::printf("one wait %d, two %d\n", h[0], h[1]);
    return h[0] == 0 && h[1] == 1 && h[2] == 1 ? 0 : 1;
}
