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
// there are many vectors: FIGURES.
// D / 8 lanes own a vector (16 bytes of FP16 and 4 bytes of codes each), so a warp
// moves two vectors of 128 or four of 64 with full-width accesses. Where there
// are enough vectors to fill the GPU all the same, a thread takes four, whose
// loads are in flight together (one each: FIGURES1).
//
// Issue slots bound them next, so operations per element are few:
//  - the extremes are found in FP16 pairs, then reduced over the lanes as (-lo, hi) pairs;
//  - the quotients x / s come from the correctly rounded reciprocal and one
//    residual FMA pair (Markstein's correction, as in the fused producers:
//    the correctly rounded quotient for every FP16 numerator and scale);
//  - they are rounded to integers by adding 1.5 * 2^23 (|x / s| <= 30: FP16's
//    rounding of s at most doubles the quotient), which leaves the code in the sum's low bits;
//  - a read's codes become FP16 integers 1024 + q by inserting them into a
//    mantissa, and (1024 + q) - (1024 + z) and its product with s are one
//    exact and one correctly rounded FP16 operation.
#include <cuda_fp16.h>
#include <stdint.h>

#include "kv4_mma.cuh"
#include "kv4_paged.cuh"
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

constexpr float kRoundInt = 12582912.0f;   // 1.5 * 2^23: added, it rounds to an integer

// a / b correctly rounded, given y = RN(1/b) (Markstein's correction).
__device__ __forceinline__ float quotient(float a, float b, float y) {
    const float q0 = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-q0, b, a), y, q0);
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

// Vector index -> row and head; returns the slot's place in the cache ((page
// * Hkv + head) * page_size + offset), or -1 for a row without a slot.
__device__ __forceinline__ int64_t vector_of(const PagedCacheParams &p, uint32_t vec, uint32_t &row, uint32_t &h) {
    row = vec / (uint32_t)p.Hkv;
    h = vec - row * (uint32_t)p.Hkv;
    const int slot = __ldg(p.slots + row);
    if ((uint32_t)slot >= (uint32_t)p.n_slots) return -1;
    const int64_t page = slot >> p.page_shift;
    return ((page * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

// PER: vectors per thread, PER spans of a CTA's width apart.
template <int D, int PER>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_write_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8, VPC = kPcThreads / LPV;   // lanes per vector, vectors per CTA and span
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    const __half *from = is_v ? p.v : p.k;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const uint32_t n = (uint32_t)(p.N * p.Hkv), vec0 = blockIdx.x * (PER * VPC) + threadIdx.x / LPV;
    int64_t at[PER];
    uint4 u[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t vec = vec0 + i * VPC;
        uint32_t row, h;
        at[i] = -1;
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        if (vec < n) {
            at[i] = vector_of(p, vec, row, h);
            u[i] = __ldg(reinterpret_cast<const uint4 *>(from + row * stride + h * D) + l);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        // (-lo, hi) of the lane's 8 values, then of the vector's lanes; a NaN counts for neither.
        const __half2 mn = __hmin2(__hmin2(as_half2(w[0]), as_half2(w[1])), __hmin2(as_half2(w[2]), as_half2(w[3])));
        const __half2 mx = __hmax2(__hmax2(as_half2(w[0]), as_half2(w[1])), __hmax2(as_half2(w[2]), as_half2(w[3])));
        const __half2 nm = __hneg2(mn);
        __half2 ext = __hmax2(__hmax2(__lows2half2(nm, mx), __highs2half2(nm, mx)), __floats2half2_rn(0.0f, 0.0f));
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1)   // the whole warp takes part
            ext = __hmax2(ext, as_half2(__shfl_xor_sync(0xffffffffu, half2_bits(ext), o)));
        if (at[i] < 0) continue;
        const float neg_lo = __low2float(ext);
        const __half sh = __float2half_rn(__fdiv_rn(__fadd_rn(__high2float(ext), neg_lo), 15.0f));
        const float s = __half2float(sh);
        float zf = 0.0f;
        uint32_t codes = 0u;
        if (s != 0.0f) {
            const float y = __frcp_rn(s);
            zf = rintf(quotient(neg_lo, s, y));
            // The sum's bits are those of 1.5 * 2^23 plus the code: the former's share of the shifted sum goes last.
            constexpr uint32_t base = 0x4B400000u;
            uint32_t shares = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = e % 2 ? __high2float(as_half2(w[e / 2])) : __low2float(as_half2(w[e / 2]));
                const float r = __fadd_rn(__fadd_rn(quotient(x, s, y), kRoundInt), zf);
                codes += __float_as_uint(fminf(fmaxf(r, kRoundInt), kRoundInt + 15.0f)) << (4 * e);   // NaN: 0
                shares += base << (4 * e);
            }
            codes -= shares;
        }
        reinterpret_cast<uint32_t *>(is_v ? p.v_codes : p.k_codes)[at[i] * LPV + l] = codes;
        if (l == 0) (is_v ? p.v_params : p.k_params)[at[i]] = __halves2half2(sh, __int2half_rn((int)zf));
    }
}

template <int D, int PER>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_read_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8, VPC = kPcThreads / LPV;
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(is_v ? p.v_codes : p.k_codes);
    const uint32_t *params = reinterpret_cast<const uint32_t *>(is_v ? p.v_params : p.k_params);
    const uint32_t n = (uint32_t)(p.N * p.Hkv), vec0 = blockIdx.x * (PER * VPC) + threadIdx.x / LPV;
    int64_t at[PER];
    uint32_t c[PER], sz[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        uint32_t row, h;
        at[i] = vec0 + i * VPC < n ? vector_of(p, vec0 + i * VPC, row, h) : -1;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = at[i] >= 0 ? __ldg(codes + at[i] * LPV + l) : 0u;
        sz[i] = at[i] >= 0 ? __ldg(params + at[i]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (vec0 + i * VPC >= n) continue;
        const __half2 s = __half2half2(__low2half(as_half2(sz[i])));
        const __half2 z = __hadd2(__half2half2(__high2half(as_half2(sz[i]))), __floats2half2_rn(1024.0f, 1024.0f));
        uint32_t r[4];   // codes e and e + 4 in r[e]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = (c[i] >> (4 * e) & 0x000F000Fu) | 0x64006400u;
            r[e] = half2_bits(__hmul2(__hsub2(as_half2(q), z), s));
        }
        reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out)[(int64_t)(vec0 + i * VPC) * LPV + l] =
            make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                       __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
}

template <int D, int PER>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    constexpr int VPC = PER * (kPcThreads / (D / 8));   // vectors per CTA
    const dim3 grid((unsigned)((p.N * p.Hkv + VPC - 1) / VPC), 2);
    if (write)
        kv4_paged_write_kernel<D, PER><<<grid, kPcThreads, 0, stream>>>(p);
    else
        kv4_paged_read_kernel<D, PER><<<grid, kPcThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// Four vectors per thread where that still makes a CTA for every SM.
template <int D>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    return p.N * p.Hkv * 2 * (D / 8) >= (int64_t)4 * kPcThreads * 148 ? launch<D, 4>(p, write, stream)
                                                                      : launch<D, 1>(p, write, stream);
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
