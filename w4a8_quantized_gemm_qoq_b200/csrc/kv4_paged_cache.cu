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
// there are many vectors, by a launch's latency where there are few. D / 16 lanes
// own a vector, two chunks of 8 values each, so that a load or store of theirs is
// 128 or 32 bytes in a row. Measured, a write and a read of 8192 tokens with 8
// heads of 128 (85 MB): 22.6 us, 3.8 TB/s (with one chunk per lane 25); of 1200
// tokens 5.6 us, of 64 tokens 3.7. Two vectors per thread take 5.9 us for 1200 tokens, 21.9
// for 8192: not worth a second form.
//
// With one chunk per lane four fifths of the write's issue slots were taken, so
// operations per element are few:
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

constexpr int kPcThreads = 128;

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

// A CTA takes one head of kPcThreads / LPV rows, so that the codes and parameters
// of neighbouring tokens, neighbours in a page, are stored together.
template <int LPV>
__device__ __forceinline__ void vector_of(const PagedCacheParams &p, int64_t &row, int &h) {
    const uint32_t block = blockIdx.x / (uint32_t)p.Hkv;
    h = (int)(blockIdx.x - block * (uint32_t)p.Hkv);
    row = (int64_t)block * (kPcThreads / LPV) + threadIdx.x / LPV;
}

// The place of a slot's vector of head h in the cache, (page * Hkv + head) *
// page_size + offset, or -1 for a row that has none.
__device__ __forceinline__ int64_t place_of(const PagedCacheParams &p, int64_t row, int h) {
    if (row >= p.N) return -1;
    const int slot = __ldg(p.slots + row);
    if ((uint32_t)slot >= (uint32_t)p.n_slots) return -1;
    return (((int64_t)(slot >> p.page_shift) * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

template <int D>
__global__ void __launch_bounds__(kPcThreads, 16) kv4_paged_write_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 16;   // lanes per vector
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    int64_t row;
    int h;
    vector_of<LPV>(p, row, h);
    const uint4 *from = reinterpret_cast<const uint4 *>((is_v ? p.v + row * p.v_stride : p.k + row * p.k_stride) + h * D) + l;
    uint4 u[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};   // chunks l and l + LPV of the vector
    if (row < p.N) {
        u[0] = __ldg(from);
        u[1] = __ldg(from + LPV);
    }
    const int64_t at = place_of(p, row, h);
    // (-lo, hi) of the lane's 16 values, then of the vector's lanes; a NaN counts for neither.
    __half2 mn[2], mx[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const __half2 x = as_half2(u[c].x), y = as_half2(u[c].y), z = as_half2(u[c].z), w = as_half2(u[c].w);
        mn[c] = __hmin2(__hmin2(x, y), __hmin2(z, w));
        mx[c] = __hmax2(__hmax2(x, y), __hmax2(z, w));
    }
    const __half2 nm = __hneg2(__hmin2(mn[0], mn[1])), m = __hmax2(mx[0], mx[1]);
    __half2 ext = __hmax2(__hmax2(__lows2half2(nm, m), __highs2half2(nm, m)), __floats2half2_rn(0.0f, 0.0f));
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1)   // the whole warp takes part
        ext = __hmax2(ext, as_half2(__shfl_xor_sync(0xffffffffu, half2_bits(ext), o)));
    if (at < 0) return;
    const float neg_lo = __low2float(ext);
    const __half sh = __float2half_rn(__fdiv_rn(__fadd_rn(__high2float(ext), neg_lo), 15.0f));
    const float s = __half2float(sh);
    float zf = 0.0f;
    uint32_t codes[2] = {0u, 0u};
    if (s != 0.0f) {
        const float y = __frcp_rn(s);
        zf = rintf(quotient(neg_lo, s, y));
        const uint64_t y2 = pair_of(y, y), s2 = pair_of(-s, -s), z2 = pair_of(zf, zf);
        const uint64_t round2 = pair_of(kRoundInt, kRoundInt);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
            // A sum's bits are those of 1.5 * 2^23 plus the code: the former's share of the shifted sum goes last.
            uint32_t shares = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = __half22float2(as_half2(w[e]));
                const uint64_t x2 = pair_of(x.x, x.y), q = mul2(x2, y2);
                const float2 r = of_pair(add2(add2(fma2(fma2(q, s2, x2), y2, q), round2), z2));   // Markstein's, as above
                codes[c] += __float_as_uint(fminf(fmaxf(r.x, kRoundInt), kRoundInt + 15.0f)) << (8 * e);   // NaN: 0
                codes[c] += __float_as_uint(fminf(fmaxf(r.y, kRoundInt), kRoundInt + 15.0f)) << (8 * e + 4);
                shares += 0x4B400000u * 17u << (8 * e);
            }
            codes[c] -= shares;
        }
    }
    uint32_t *to = reinterpret_cast<uint32_t *>(is_v ? p.v_codes : p.k_codes) + at * (D / 8) + l;
    to[0] = codes[0];
    to[LPV] = codes[1];
    if (l == 0) (is_v ? p.v_params : p.k_params)[at] = __halves2half2(sh, __int2half_rn((int)zf));
}

template <int D>
__global__ void __launch_bounds__(kPcThreads, 16) kv4_paged_read_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 16;
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    int64_t row;
    int h;
    vector_of<LPV>(p, row, h);
    if (row >= p.N) return;
    const int64_t at = place_of(p, row, h);
    uint32_t c[2] = {0u, 0u}, sz = 0u;
    if (at >= 0) {
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(is_v ? p.v_codes : p.k_codes) + at * (D / 8) + l;
        c[0] = __ldg(codes);
        c[1] = __ldg(codes + LPV);
        sz = __ldg(reinterpret_cast<const uint32_t *>(is_v ? p.v_params : p.k_params) + at);
    }
    const __half2 s = __low2half2(as_half2(sz));
    const __half2 z = __hadd2(__high2half2(as_half2(sz)), __floats2half2_rn(1024.0f, 1024.0f));
    uint4 *to = reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out) + (row * p.Hkv + h) * (D / 8) + l;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        uint32_t r[4];   // codes e and e + 4 in r[e]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = (c[x] >> (4 * e) & 0x000F000Fu) | 0x64006400u;
            r[e] = half2_bits(__hmul2(__hsub2(as_half2(q), z), s));
        }
        to[x * LPV] = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                                 __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
}

template <int D>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    constexpr int rows = kPcThreads / (D / 16);   // per CTA
    const dim3 grid((unsigned)((p.N + rows - 1) / rows * p.Hkv), 2);
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
