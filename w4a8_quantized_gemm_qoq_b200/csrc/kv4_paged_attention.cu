// Attention of new tokens over the paged KV4 cache (grouped-query, causal,
// optional sliding window with sinks): the plain form of the kernel.
//
// One warp owns a (row, query head): 32 tokens at a time, each lane scores one
// token, the warp updates the running maximum and sum, then each lane adds the
// 32 weighted values of its D / 32 dims. Everything is FP32.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kv4_paged.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) kv4_paged_plain_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int DB = D / 2, VPL = D / 32;
    __shared__ float qs[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    if (item >= p.N * p.Hq) return;
    const int row = (int)(item / p.Hq), hq = (int)(item % p.Hq), h = hq / p.G;
    // The row's request: the last one whose start is at or before the row.
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.q_start[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    const int b = lo;
    const PagedRequest r = paged_request(p, b);
    if (row < r.row0 || row >= r.row0 + r.n || r.n > p.max_new || r.n * p.G <= kRowsMax) return;
    const int pos = r.kv - r.n + (row - r.row0);
    for (int d = lane; d < D; d += 32) qs[warp][d] = __half2float(p.q[row * p.q_stride + hq * D + d]);
    __syncwarp();
    const int first = p.window ? max(0, pos - p.window + 1) : 0;   // of the window
    const int sinks = p.window ? min(p.sinks, first) : 0;
    float m = -INFINITY, l = 0.0f, o[VPL] = {};
    const int P = 1 << p.page_shift;
    for (int i0 = 0; i0 < sinks + pos + 1 - first; i0 += 32) {
        const int i = i0 + lane;
        const int t = i < sinks ? i : first + i - sinks;
        const bool in = t <= pos;
        const int page = in ? p.block_table[(int64_t)b * p.max_pages + (t >> p.page_shift)] : 0;
        const bool bad = (uint32_t)page >= (uint32_t)p.n_pages;
        if (bad) paged_bad_request(p, b);
        const int64_t at = (((int64_t)page * p.Hkv + h) << p.page_shift) + (t & (P - 1));
        float s = -INFINITY, vs = 0.0f, vz = 0.0f;
        if (in && bad) s = 0.0f;
        if (in && !bad) {
            const float2 kp = __half22float2(p.k_params[at]);
            const float2 vp = __half22float2(p.v_params[at]);
            float acc = 0.0f;
            const uint32_t *c = reinterpret_cast<const uint32_t *>(p.k_codes + at * DB);
            for (int j = 0; j < D / 8; ++j)
                for (int e = 0; e < 8; ++e) acc += ((float)((c[j] >> (4 * e)) & 15u) - kp.y) * qs[warp][8 * j + e];
            s = acc * kp.x * p.qscale;
            vs = vp.x, vz = vp.y;
        }
        float mx = s;
        for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        mx = fmaxf(mx, m);
        const float al = m == -INFINITY ? 0.0f : exp2f(m - mx);
        const float w = s == -INFINITY ? 0.0f : exp2f(s - mx);
        m = mx;
        float sum = w;
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        l = l * al + sum;
        for (int e = 0; e < VPL; ++e) o[e] *= al;
        const float ws = w == 0.0f ? 0.0f : w * vs;
        const int64_t mine = in && !bad ? at : 0;
        for (int k = 0; k < 32; ++k) {
            const float wk = __shfl_sync(0xffffffffu, ws, k), zk = __shfl_sync(0xffffffffu, vz, k);
            const int64_t ak = __shfl_sync(0xffffffffu, mine, k);
            if (wk == 0.0f) continue;
            for (int e = 0; e < VPL; e += 2) {
                const uint8_t c = p.v_codes[ak * DB + lane * (VPL / 2) + e / 2];
                o[e] += wk * ((float)(c & 15) - zk);
                o[e + 1] += wk * ((float)(c >> 4) - zk);
            }
        }
    }
    for (int e = 0; e < VPL; ++e)
        p.out[row * p.out_stride + hq * D + lane * VPL + e] = __float2half_rn(l > 0.0f ? o[e] / l : 0.0f);
}

}  // namespace

// Bytes [0, 256) are the status words; the few-rows kernel's part follows.
size_t kv4_paged_workspace_bytes(int64_t B, int64_t, int64_t, int64_t, int64_t D, int64_t) {
    return 256 + rows_workspace_bytes(B, D);
}

cudaError_t launch_paged_attention(const PagedAttnParams &p, int64_t D, void *ws, cudaStream_t stream) {
    const cudaError_t e = launch_paged_rows(p, D, static_cast<uint8_t *>(ws) + 256, stream);
    if (e != cudaSuccess || (int64_t)p.max_new * p.G <= kRowsMax) return e;
    const unsigned blocks = (unsigned)((p.N * p.Hq + kWarps - 1) / kWarps);
    if (D == 128)
        kv4_paged_plain_kernel<128><<<blocks, 32 * kWarps, 0, stream>>>(p);
    else
        kv4_paged_plain_kernel<64><<<blocks, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace qoq
