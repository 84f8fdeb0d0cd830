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
// there are many vectors, by a launch's latency where there are few. D / 8 lanes
// own a vector (16 bytes of FP16 and 4 bytes of codes each), so a warp moves
// two vectors of 128 or four of 64 with full-width accesses. Measured, a write and a
// read of 8192 tokens with 8 heads of 128 (85 MB): 25 us, 3.4 TB/s, the write
// 15 of them; of 64 tokens 3.6 us.
//
// The write's issue slots (157 instructions per 16-byte load, four fifths of the
// slots taken) bound it before HBM does, so operations per element are few:
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

// A CTA takes one head of PER x VPC rows (so that the codes and parameters of
// neighbouring tokens, neighbours in a page, are stored together), a thread of
// the rows `row`, row + VPC, ...
template <int VPC, int PER>
__device__ __forceinline__ void vectors_of(const PagedCacheParams &p, int64_t &row, int &h) {
    const uint32_t block = blockIdx.x / (uint32_t)p.Hkv;
    h = (int)(blockIdx.x - block * (uint32_t)p.Hkv);
    row = (int64_t)block * (PER * VPC) + threadIdx.x / (kPcThreads / VPC);
}

// The place of a slot's vector of head h in the cache, (page * Hkv + head) *
// page_size + offset, or -1 for a row that has none.
__device__ __forceinline__ int64_t place_of(const PagedCacheParams &p, int64_t row, int h) {
    if (row >= p.N) return -1;
    const int slot = __ldg(p.slots + row);
    if ((uint32_t)slot >= (uint32_t)p.n_slots) return -1;
    return (((int64_t)(slot >> p.page_shift) * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

template <int D, int PER>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_write_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8, VPC = kPcThreads / LPV;   // lanes per vector, vectors per CTA and turn
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    int64_t row;
    int h;
    vectors_of<VPC, PER>(p, row, h);
    const uint4 *from = reinterpret_cast<const uint4 *>((is_v ? p.v : p.k) + row * stride + h * D) + l;
    int64_t at[PER];
    uint4 u[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row + i * VPC < p.N) u[i] = __ldg(from + i * (VPC * stride / 8));
        at[i] = place_of(p, row + i * VPC, h);
    }
    __half2 mine;   // (-lo, hi) of the vector l % PER
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const __half2 a = as_half2(u[i].x), b = as_half2(u[i].y), c = as_half2(u[i].z), d = as_half2(u[i].w);
        // Of the lane's 8 values, then of the vector's lanes; a NaN counts for neither.
        const __half2 nm = __hneg2(__hmin2(__hmin2(a, b), __hmin2(c, d))), mx = __hmax2(__hmax2(a, b), __hmax2(c, d));
        __half2 ext = __hmax2(__hmax2(__lows2half2(nm, mx), __highs2half2(nm, mx)), __floats2half2_rn(0.0f, 0.0f));
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1)   // the whole warp takes part
            ext = __hmax2(ext, as_half2(__shfl_xor_sync(0xffffffffu, half2_bits(ext), o)));
        if (i == 0 || l % PER == i) mine = ext;
    }
    // A lane works out one vector's scale, its reciprocal and the zero.
    const float neg_lo = __low2float(mine);
    const __half sh = __float2half_rn(__fdiv_rn(__fadd_rn(__high2float(mine), neg_lo), 15.0f));
    const float scale = __half2float(sh), rcp = __frcp_rn(scale);
    const __half zh = __int2half_rn(scale != 0.0f ? (int)rintf(quotient(neg_lo, scale, rcp)) : 0);
    const uint32_t param = half2_bits(__halves2half2(sh, zh));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t sz = __shfl_sync(0xffffffffu, param, i, LPV);
        const float y = __shfl_sync(0xffffffffu, rcp, i, LPV);
        if (at[i] < 0) continue;
        const float s = half_lo(sz), zf = __half2float(half_hi(sz));
        uint32_t codes = 0u;
        if (s != 0.0f) {
            const uint64_t y2 = pair_of(y, y), s2 = pair_of(-s, -s), z2 = pair_of(zf, zf);
            const uint64_t round2 = pair_of(kRoundInt, kRoundInt);
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            // A sum's bits are those of 1.5 * 2^23 plus the code: the former's share of the shifted sum goes last.
            uint32_t shares = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = __half22float2(as_half2(w[e]));
                const uint64_t x2 = pair_of(x.x, x.y), q = mul2(x2, y2);
                const float2 r = of_pair(add2(add2(fma2(fma2(q, s2, x2), y2, q), round2), z2));   // Markstein's, as above
                codes += __float_as_uint(fminf(fmaxf(r.x, kRoundInt), kRoundInt + 15.0f)) << (8 * e);   // NaN: 0
                codes += __float_as_uint(fminf(fmaxf(r.y, kRoundInt), kRoundInt + 15.0f)) << (8 * e + 4);
                shares += 0x4B400000u * 17u << (8 * e);
            }
            codes -= shares;
        }
        reinterpret_cast<uint32_t *>(is_v ? p.v_codes : p.k_codes)[at[i] * LPV + l] = codes;
        if (l == i) (is_v ? p.v_params : p.k_params)[at[i]] = as_half2(sz);
    }
}

template <int D, int PER>
__global__ void __launch_bounds__(kPcThreads) kv4_paged_read_kernel(const __grid_constant__ PagedCacheParams p) {
    constexpr int LPV = D / 8, VPC = kPcThreads / LPV;
    const int l = threadIdx.x % LPV;
    const bool is_v = blockIdx.y != 0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(is_v ? p.v_codes : p.k_codes) + l;
    const uint32_t *params = reinterpret_cast<const uint32_t *>(is_v ? p.v_params : p.k_params);
    int64_t row;
    int h;
    vectors_of<VPC, PER>(p, row, h);
    uint4 *to = reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out) + (row * p.Hkv + h) * LPV + l;
    int64_t at[PER];
    uint32_t c[PER], sz[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) at[i] = place_of(p, row + i * VPC, h);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = sz[i] = 0u;
        if (at[i] >= 0) {
            c[i] = __ldg(codes + at[i] * LPV);
            sz[i] = __ldg(params + at[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (row + i * VPC >= p.N) break;
        const __half2 s = __low2half2(as_half2(sz[i]));
        const __half2 z = __hadd2(__high2half2(as_half2(sz[i])), __floats2half2_rn(1024.0f, 1024.0f));
        uint32_t r[4];   // codes e and e + 4 in r[e]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = (c[i] >> (4 * e) & 0x000F000Fu) | 0x64006400u;
            r[e] = half2_bits(__hmul2(__hsub2(as_half2(q), z), s));
        }
        to[(int64_t)i * VPC * p.Hkv * LPV] =
            make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                       __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
}

template <int D, int PER>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    constexpr int rows = PER * kPcThreads / (D / 8);   // per CTA
    const dim3 grid((unsigned)((p.N + rows - 1) / rows * p.Hkv), 2);
    if (write)
        kv4_paged_write_kernel<D, PER><<<grid, kPcThreads, 0, stream>>>(p);
    else
        kv4_paged_read_kernel<D, PER><<<grid, kPcThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// Four vectors per thread, whose loads are in flight together, where that still
// makes three CTAs for every SM (8 heads of 128, write and read: 1200 tokens 8.2 us,
// one vector each 7.1; 2400 tokens 10.7 and 11.4; 8192 tokens 25.5 and 28.6).
template <int D>
cudaError_t launch(const PagedCacheParams &p, bool write, cudaStream_t stream) {
    return p.N * p.Hkv * 2 * (D / 8) >= (int64_t)4 * kPcThreads * 3 * 148 ? launch<D, 4>(p, write, stream)
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
