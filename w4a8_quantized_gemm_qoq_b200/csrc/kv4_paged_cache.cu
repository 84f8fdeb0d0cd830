// Write and read of the paged KV4 cache: per-vector asymmetric 4-bit
// quantisation of ragged new tokens into their slots, and the gather of slots
// back to FP16.
//
// For each vector x of D values (a token's key or value of one head):
//   lo = min(0, min x), hi = max(0, max x), s = FP16((hi - lo) / 15),
//   z = RNE(-lo / s), q = clamp(RNE(x / s) + z, 0, 15); s == 0: q = z = 0,
// each FP32 step one correctly rounded operation, so the bytes equal those of
// the contiguous cache's write.
//
// Both kernels move 2 D + D/2 + 4 bytes per vector and are bound by HBM when
// there are many vectors. D / 8 lanes own a vector (16 bytes of FP16 and 4
// bytes of codes each), so a warp moves two vectors of 128 or four of 64 with
// full-width accesses. The quotients x / s come from the correctly rounded
// reciprocal and one residual FMA pair (Markstein's correction, as in the fused
// producers: the correctly rounded quotient for every FP16 numerator and
// scale), three operations in place of a division's sequence.
#include <cuda_fp16.h>
#include <stdint.h>

#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kPcThreads = 256;

struct PagedCacheParams {
    const __half *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *slots;
    uint8_t *k_codes, *v_codes;
    __half2 *k_params, *v_params;
    __half *k_out, *v_out;
    int64_t N;
    int Hkv, page_shift, n_slots;
};

__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// a / b correctly rounded, given y = RN(1/b) (Markstein's correction).
__device__ __forceinline__ float quotient(float a, float b, float y) {
    const float q0 = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-q0, b, a), y, q0);
}

// Vector index -> (tensor, row, head); returns the slot's place in the cache
// ((page * Hkv + head) * page_size + offset), or -1 for a row without a slot.
__device__ __forceinline__ int64_t vector_of(const PagedCacheParams &p, int64_t vec, int &row, int &h) {
    row = (int)(vec / p.Hkv);
    h = (int)(vec - (int64_t)row * p.Hkv);
    const int slot = __ldg(p.slots + row);
    if ((uint32_t)slot >= (uint32_t)p.n_slots) return -1;
    const int64_t page = slot >> p.page_shift;
    return ((page * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

template <int D>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_write_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8;   // lanes per vector
    const int64_t vec = ((int64_t)blockIdx.x * kPcThreads + threadIdx.x) / LPV;
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    int row = 0, h = 0;
    const bool in = vec < p.N * p.Hkv;
    const int64_t at = in ? vector_of(p, vec, row, h) : -1;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (at >= 0)
        u = __ldg(reinterpret_cast<const uint4 *>((is_v ? p.v + row * p.v_stride : p.k + row * p.k_stride) + h * D) + l);
    float x[8];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_half2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) {   // within the vector's lanes; the whole warp takes part
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (at < 0) return;
    const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __half2float(sh);
    float zf = 0.0f;
    uint32_t codes = 0u;
    if (s != 0.0f) {
        const float y = __frcp_rn(s);
        zf = rintf(quotient(-lo, s, y));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            codes |= (uint32_t)fminf(fmaxf(rintf(quotient(x[i], s, y)) + zf, 0.0f), 15.0f) << (4 * i);
    }
    reinterpret_cast<uint32_t *>(is_v ? p.v_codes : p.k_codes)[at * LPV + l] = codes;
    if (l == 0) (is_v ? p.v_params : p.k_params)[at] = __halves2half2(sh, __int2half_rn((int)zf));
}

template <int D>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_read_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8;
    const int64_t vec = ((int64_t)blockIdx.x * kPcThreads + threadIdx.x) / LPV;
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    if (vec >= p.N * p.Hkv) return;
    int row, h;
    const int64_t at = vector_of(p, vec, row, h);
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (at >= 0) {
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t *>(is_v ? p.v_codes : p.k_codes) + at * LPV + l);
        const float2 sz = __half22float2((is_v ? p.v_params : p.k_params)[at]);
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (q - z) * s is exact in FP32 (5 by 11 bits); one rounding to FP16.
            const float a = ((float)((c >> (8 * i)) & 15u) - sz.y) * sz.x;
            const float b = ((float)((c >> (8 * i + 4)) & 15u) - sz.y) * sz.x;
            const __half2 hh = __floats2half2_rn(a, b);
            r[i] = *reinterpret_cast<const uint32_t *>(&hh);
        }
        o = make_uint4(r[0], r[1], r[2], r[3]);
    }
    reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out)[vec * LPV + l] = o;
}

template <int D>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    constexpr int VPC = kPcThreads / (D / 8);   // vectors per CTA
    const dim3 grid((unsigned)((p.N * p.Hkv + VPC - 1) / VPC), 2);
    if (write)
        kv4_paged_write_kernel<D><<<grid, kPcThreads, 0, stream>>>(p);
    else
        kv4_paged_read_kernel<D><<<grid, kPcThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *slots,
                               int64_t N, int64_t Hkv, int64_t D, int64_t n_pages, int page_shift, uint8_t *k_codes,
                               void *k_params, uint8_t *v_codes, void *v_params, cudaStream_t stream) {
    PagedCacheParams p = {};
    p.k = static_cast<const __half *>(k);
    p.v = static_cast<const __half *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.k_codes = k_codes;
    p.v_codes = v_codes;
    p.k_params = static_cast<__half2 *>(k_params);
    p.v_params = static_cast<__half2 *>(v_params);
    p.N = N;
    p.Hkv = (int)Hkv;
    p.page_shift = page_shift;
    p.n_slots = (int)(n_pages << page_shift);
    return D == 128 ? launch<128>(p, true, stream) : launch<64>(p, true, stream);
}

cudaError_t launch_paged_read(const int32_t *slots, int64_t N, int64_t Hkv, int64_t D, int64_t n_pages, int page_shift,
                              const uint8_t *k_codes, const void *k_params, const uint8_t *v_codes,
                              const void *v_params, void *k_out, void *v_out, cudaStream_t stream) {
    PagedCacheParams p = {};
    p.slots = slots;
    p.k_codes = const_cast<uint8_t *>(k_codes);
    p.v_codes = const_cast<uint8_t *>(v_codes);
    p.k_params = static_cast<__half2 *>(const_cast<void *>(k_params));
    p.v_params = static_cast<__half2 *>(const_cast<void *>(v_params));
    p.k_out = static_cast<__half *>(k_out);
    p.v_out = static_cast<__half *>(v_out);
    p.N = N;
    p.Hkv = (int)Hkv;
    p.page_shift = page_shift;
    p.n_slots = (int)(n_pages << page_shift);
    return D == 128 ? launch<128>(p, false, stream) : launch<64>(p, false, stream);
}

}  // namespace qoq
