// Host-only check of ensure_smem (qmm_internal.h) under threads, run by
// test_smem_limit.py on a machine without a GPU: a thread that asks for little is
// held inside the attribute call until another has asked for much (or 0.3 s are
// over); the limit must end at the larger of the two.
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

namespace {

constexpr int kSmall = 40000, kLarge = 200000;
std::atomic<int> applied{0}, calls{0};
std::atomic<bool> small_inside{false}, large_done{false};

template <typename T>
cudaError_t fake_set_attribute(T *, cudaFuncAttribute attribute, int value) {
    if (attribute != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    ++calls;
    if (value == kSmall) {
        small_inside = true;
        const auto until = std::chrono::steady_clock::now() + std::chrono::milliseconds(300);
        while (!large_done && std::chrono::steady_clock::now() < until) std::this_thread::yield();
    }
    applied = value;
    return cudaSuccess;
}

}  // namespace

#define cudaFuncSetAttribute fake_set_attribute
#include "qmm_internal.h"

namespace qmm {
int current_device() { return 0; }
}  // namespace qmm

namespace {
__global__ void kernel() {}
int limits[qmm::kMaxDevices];
}  // namespace

int main() {
    std::thread first([] { qmm::ensure_smem(kernel, kSmall, false, limits); });
    while (!small_inside) std::this_thread::yield();
    std::thread second([] {
        qmm::ensure_smem(kernel, kLarge, false, limits);
        large_done = true;
    });
    first.join();
    second.join();
    const int after = calls;
    qmm::ensure_smem(kernel, kSmall, false, limits);
    qmm::ensure_smem(kernel, kLarge, false, limits);
    std::printf("applied %d cached %d further calls %d\n", applied.load(), limits[0], calls.load() - after);
    return applied == kLarge && limits[0] == kLarge && calls == after ? 0 : 1;
}
