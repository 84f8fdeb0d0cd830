// What the paged KV4 attention kernels share: their arguments, and a
// request's rows and tokens from the device-side lengths.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

// A request's rows of q and out, and its cached tokens, clamped to what the
// buffers hold whatever the device arrays say.
struct PagedRequest {
    int row0, n, kv;
};

__device__ __forceinline__ PagedRequest paged_request(const PagedAttnParams &p, int b) {
    PagedRequest r;
    r.row0 = min(max(p.q_start[b], 0), (int)p.N);
    r.n = max(min(p.q_start[b + 1], (int)p.N) - r.row0, 0);
    r.kv = (int)min((int64_t)max(p.kv_lens[b], 0), (int64_t)p.max_pages << p.page_shift);
    return r;
}

__device__ __forceinline__ void paged_bad_request(const PagedAttnParams &p, int b) {
    if (atomicCAS(p.status, 0, QOQ_ERR_INVALID_ARG) == 0) p.status[1] = b;
}

// Pairs of FP32 values, for the operations that take two at once.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    return pair_of(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 of_pair(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Opts a kernel in to more than 48 KB of dynamic shared memory, once per device.
struct SmemOptIn {
    std::atomic<uint64_t> done{0};   // devices 0 .. 63, a bit each
    template <typename Kernel>
    cudaError_t set(Kernel kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

}  // namespace qoq
