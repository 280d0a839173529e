// s4::SmemLimit from two host threads, against a model of the runtime's
// attribute. The model holds one thread inside the call until the other has
// been through, for 0.3 s at most: the orders of events that lose a limit.
// Prints nothing and returns 0, or says what went wrong.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include <cuda_runtime.h>

template <typename K>   // nvcc's own overload for a typed kernel
cudaError_t cudaFuncSetAttribute(K *kernel, cudaFuncAttribute attr, int value) {
    return cudaFuncSetAttribute((const void *)kernel, attr, value);
}

#include "launch.h"

namespace {

constexpr int kSmall = 145000, kLarge = 161000;
std::atomic<int> attribute[2], calls_small, calls_large;
std::atomic<bool> inside;          // a held call has begun
int hold_before = 0, hold_after = 0;   // the size whose call waits before, or after, it takes effect
thread_local int device = 0;

void wait_for(const std::atomic<int> &calls) {
    for (int i = 0; i < 300 && calls.load() == 0; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

void kernel_a() {}

}  // namespace

extern "C" cudaError_t cudaGetDevice(int *d) {
    *d = device;
    return cudaSuccess;
}

extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
    const std::atomic<int> &other = bytes == kSmall ? calls_large : calls_small;
    if (bytes == hold_before) {
        inside = true;
        wait_for(other);
    }
    attribute[device] = bytes;
    (bytes == kSmall ? calls_small : calls_large)++;
    if (bytes == hold_after) {
        inside = true;
        wait_for(other);
    }
    return cudaSuccess;
}

namespace {

// `first` runs into the held call, then `second` comes
int together(const char *what, int first, int second, int before, int after) {
    s4::SmemLimit limit;
    hold_before = before, hold_after = after;
    attribute[0] = 48 * 1024;
    calls_small = calls_large = 0;
    inside = false;
    std::thread a([&] { limit.raise(kernel_a, first); });
    while (!inside) std::this_thread::yield();
    std::thread b([&] { limit.raise(kernel_a, second); });
    a.join();
    b.join();
    hold_before = hold_after = 0;
    const bool now = attribute[0] >= kLarge;   // what a raise that returned asked for
    limit.raise(kernel_a, kLarge);             // and a later call with the large size
    if (now && attribute[0] >= kLarge) return 0;
    std::printf("%s: a launch with %d bytes meets a lower limit%s\n", what, kLarge,
                attribute[0] < kLarge ? ", for good" : "");
    return 1;
}

int devices() {
    s4::SmemLimit limit;
    attribute[0] = attribute[1] = 0;
    limit.raise(kernel_a, kLarge);
    std::thread([&] {
        device = 1;
        limit.raise(kernel_a, kSmall);
    }).join();
    limit.raise(kernel_a, kSmall);
    if (attribute[0] == kLarge && attribute[1] == kSmall) return 0;
    std::printf("two devices: %d and %d\n", attribute[0].load(), attribute[1].load());
    return 1;
}

}  // namespace

int main() {
    int bad = 0;
    bad |= together("the smaller call takes effect last", kSmall, kLarge, kSmall, 0);
    bad |= together("the larger call is recorded last", kLarge, kSmall, 0, kLarge);
    bad |= devices();
    return bad;
}
