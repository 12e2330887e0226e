// Two threads whose first calls of pkv::tma_encode_fn overlap: both have to get the driver's
// function.  The runtime's lookup is a stand-in here that takes a while.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include "tma_host.cuh"

static std::atomic<int> lookups{0};

static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}

extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned int,
                                                        unsigned long long,
                                                        cudaDriverEntryPointQueryResult* q) {
    ++lookups;
    std::this_thread::sleep_for(std::chrono::milliseconds(500));
    *fn = (void*)&encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

int main() {
    std::atomic<int> missing{0};
    auto call = [&] {
        if (pkv::tma_encode_fn() != (PFN_cuTensorMapEncodeTiled_v12000)&encode) ++missing;
    };
    std::thread first(call);
    while (lookups == 0) std::this_thread::yield();       // it is looking up
    std::thread second(call);
    first.join();
    second.join();
    std::printf("%d without the function, %d lookups\n", missing.load(), lookups.load());
    return missing == 0 && lookups == 1 ? 0 : 1;
}
