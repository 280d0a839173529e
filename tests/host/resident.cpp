// s4::Resident from four host threads (run under the thread sanitizer): the
// number of blocks per SM is the one of its block size, whoever asked first.
#include <cstdio>
#include <thread>

#include <cuda_runtime.h>

template <typename K>
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *blocks, K *, int block, size_t smem) {
    *blocks = 2048 / block + (smem ? 0 : 1);
    return cudaSuccess;
}
template <typename K>
cudaError_t cudaFuncSetAttribute(K *, cudaFuncAttribute, int) {
    return cudaSuccess;
}
extern "C" cudaError_t cudaGetDevice(int *d) {
    *d = 0;
    return cudaSuccess;
}

#include "launch.h"

static void kernel() {}

int main() {
    s4::Resident resident;
    int bad[4] = {};
    std::thread threads[4];
    for (int t = 0; t < 4; ++t)
        threads[t] = std::thread([&resident, &bad, t] {
            for (int k = 0; k < 1000; ++k)
                for (int block = 32; block <= 1024; block += 32) bad[t] |= resident.of(kernel, block, 1) != 2048 / block;
        });
    for (auto &t : threads) t.join();
    if (bad[0] | bad[1] | bad[2] | bad[3]) std::puts("a wrong number of blocks");
    return bad[0] | bad[1] | bad[2] | bad[3];
}
