// Paged KV4 attention for requests with few rows: n new tokens x G query
// heads per KV head <= 32 (decode steps, short drafts).
//
// The work is one pass over the request's K and V codes (D + 8 bytes per
// token and KV head), so it is bound by HBM where sequences are long, and by
// a launch's latency where they are short. Eight of a KV head's n x G (row,
// head) pairs are the columns of the tensor-core products, so K and V are read
// once for all of them; more pairs are columns of further pieces, which read
// the same cache again (from L2, as they run side by side). That costs 8
// columns x 64 tokens about 410 cycles of an SM; the many-rows kernel costs up to
// 128 pairs x 128 tokens about 5000, so up to 32 pairs come here (32 sequences
// x 5 rows x 4 heads: FIG us here, 127 there).
//
// Pieces. The lengths are known on the device only, so every CTA works out the
// same division: a request's visible tokens are 64-token tiles (those of the
// sinks, then those of the window), four tiles are a round, and each (request,
// KV head) is cut into ceil(rounds / S) even pieces, S the least of a few
// candidates that gives at most one piece per resident CTA (four per SM), so
// that all SMs end together whatever the mix of lengths. Pieces of one
// (request, KV head) leave FP32 partial sums, which the last to arrive
// combines in a fixed order.
//
// Within a piece, each warp walks every fourth tile. Its K and V code tiles
// pass through a ring of three buffers (16-byte asynchronous copies, one
// group per tile and tensor, so that two are in flight while one is computed); scales
// and zeros are loaded one tile ahead, page numbers two. The copies go through
// the load path and not as bulk copies because a small page makes those many
// (each costs the copy engine about 50 ns; a tile of 16-token pages would be eight
// of them every 200 ns). What limits the walk is instruction issue (unpacking
// codes), so that is kept to 5 operations per 4 operand
// registers: the codes enter the products as exact FP16 subnormals (c * 2^-24
// in a half's low nibble, c * 2^-20 in the next one, one AND per two codes and
// one shift per four), transposed loads of 16-bit units pair the value codes
// of neighbouring tokens without byte permutes, the queries that meet high
// nibbles are divided by 16 beforehand so that one accumulator takes both,
// and the zero points are subtracted afterwards: s (q.c) - s z sum(q) per
// score in FP32, and for the values as one more product row, sum_t P_t z_t.
// Token factors are converted once per token and read back by broadcast.
//
// The online softmax is FP32 with base-2 exponentials. Its maximum is raised
// only when a score exceeds it by 2^kRwSlack, so that most tiles need no
// rescaling of the output. The one rounding before the output is that of the
// weights P = p * s_V to FP16. They are kept scaled by 2^(8 - E), E the
// exponent of the largest value scale so far (a running maximum too), so that
// P stays below 2^(9 + kRwSlack) and keeps 11 bits down to 2^-22 of the
// largest weight.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kv4_mma.cuh"
#include "kv4_paged.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kRwWarps = 4;
constexpr int kRwThreads = 32 * kRwWarps;
constexpr int kRwTile = 64;                   // tokens per warp tile
constexpr int kRwResident = 4 * 148;          // CTAs that run at once
constexpr int kRwSplitSlots = 2 * kRwResident;   // pieces of divided items: see the bound at rows_candidate
constexpr int kRwWarpBatch = 128;             // requests whose division each warp works out itself
constexpr float kRwSlack = 6.0f;              // log2 by which scores may exceed the running maximum

struct RowsParams {
    PagedAttnParams a;
    int g_inv;               // ceil(2^16 / G): c / G = c g_inv >> 16 for c < 32
    int32_t *counters;       // [kRwSplitSlots], zero between calls
    float *part;             // [kRwSplitSlots][kRowsCols * D + 2 * kRowsCols]
    const int32_t *division; // [2][B + 1] from the division kernel where B > kRwWarpBatch, else null
};

// A request's tiles: [0, sink_tiles) and [first, end) in units of 64 tokens.
struct RowsTiles {
    int sink_tiles, first, count;
};

__device__ __forceinline__ RowsTiles rows_tiles(const PagedAttnParams &p, const PagedRequest &r) {
    RowsTiles t;
    const int w0 = p.window ? max(0, r.kv - r.n - p.window + 1) : 0;   // the first row's window
    t.first = w0 / kRwTile;
    const int sk = min(p.sinks, w0);
    t.sink_tiles = p.window ? min((sk + kRwTile - 1) / kRwTile, t.first) : 0;
    t.count = t.sink_tiles + max(0, (r.kv + kRwTile - 1) / kRwTile - t.first);
    return t;
}

// Groups of 8 (row, head) pairs of a request.
__device__ __forceinline__ int rows_groups(const PagedAttnParams &p, int b) {
    return (paged_request(p, b).n * p.G + kRowsCols - 1) / kRowsCols;
}

// Rounds (four tiles) of request b for this kernel: 0 if it has no rows or
// too many; one where it has rows but no token (zeros are written).
__device__ __forceinline__ int rows_rounds(const PagedAttnParams &p, int b) {
    const PagedRequest r = paged_request(p, b);
    if (r.n == 0 || r.n > p.max_new || r.n * p.G > kRowsMax) return 0;
    return max(1, (rows_tiles(p, r).count + kRwWarps - 1) / kRwWarps);
}

// Rounds per piece, from the batch's rounds (all heads) and the sums over the
// batch of ceil(rounds / S) for the candidates S.
//
// S >= total / C (C resident CTAs) bounds the divided pieces: a request is
// divided when x = rounds / S > 1, into ceil(x) <= 2 x pieces per head, so
// there are at most 2 total / S <= 2 C of them.
__device__ __forceinline__ int64_t rows_candidate(int64_t s0, int c) {
    return s0 + (c == 0 ? 0 : c == 1 ? (s0 + 3) / 4 : c == 2 ? (s0 + 1) / 2 : s0);
}

// Where a piece lies: its column group comes first, so that those which read the
// same tokens run side by side.
struct RowsPiece {
    int b, split, nsplit, h, group;
    int slot;   // the first slot of its item among the divided ones
};

__device__ __forceinline__ RowsPiece rows_piece(const PagedAttnParams &p, int b, int rest, int nsplit, int slot) {
    const int groups = rows_groups(p, b), hs = rest / groups;
    RowsPiece r;
    r.b = b;
    r.nsplit = nsplit;
    r.group = rest - hs * groups;
    r.h = hs / nsplit;
    r.split = hs - r.h * nsplit;
    r.slot = slot + (r.h * groups + r.group) * nsplit;
    return r;
}

// ceil(a / x) for 0 <= a < 2^23, 0 < x: `inv` = 1 / x rounded; the estimate is
// within one of the quotient, and the products are exact.
__device__ __forceinline__ int ceil_div(int a, int x, float inv) {
    int q = (int)((float)a * inv);
    q -= q * x >= a + x ? 1 : 0;
    q += q * x < a ? 1 : 0;
    return q + (q * x < a ? 1 : 0);
}

// The division by one warp: lane l holds the requests l, l + 32, ...
struct RowsDivision {
    int ns[kRwWarpBatch / 32], items[kRwWarpBatch / 32];      // pieces per item, items (heads x column groups)
    int start[kRwWarpBatch / 32], slot[kRwWarpBatch / 32];    // pieces and divided pieces before it
    int pieces;

    __device__ __forceinline__ void make(const PagedAttnParams &p) {
        constexpr int N = kRwWarpBatch / 32;
        const int lane = threadIdx.x & 31;
        int r[N], sum = 0, all = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r[i] = lane + 32 * i < p.B ? rows_rounds(p, lane + 32 * i) : 0;   // at most 2^23 each: the sum fits
            items[i] = r[i] ? rows_groups(p, lane + 32 * i) : 0;              // of one head for now
            sum += r[i] * items[i];
            all += items[i];
        }
        const int64_t total = (((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)sum >> 16) << 16) +
                               __reduce_add_sync(0xffffffffu, (uint32_t)sum & 0xffffu)) * p.Hkv;
        const int64_t s0 = max((int64_t)1, (total + kRwResident - 1) / kRwResident);
        int S = (int)min(s0, (int64_t)1 << 22);
        if ((int)__reduce_add_sync(0xffffffffu, (uint32_t)all) * p.Hkv <= kRwResident) {
            S = (int)rows_candidate(s0, 3);
#pragma unroll
            for (int c = 2; c >= 0; --c) {
                const int x = (int)rows_candidate(s0, c);
                const float inv = __frcp_rn((float)x);
                int n = 0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (32 * i < p.B) n += ceil_div(r[i], x, inv) * items[i];
                if ((int)__reduce_add_sync(0xffffffffu, (uint32_t)n) * p.Hkv <= kRwResident) S = x;
            }
        }
        const float inv = __frcp_rn((float)S);
        int base0 = 0, base1 = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ns[i] = start[i] = slot[i] = 0;
            if (32 * i >= p.B) continue;
            ns[i] = ceil_div(r[i], S, inv);
            items[i] *= p.Hkv;
            const int v0 = ns[i] * items[i], v1 = ns[i] > 1 ? v0 : 0;
            int i0 = v0, i1 = v1;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int u0 = __shfl_up_sync(0xffffffffu, i0, k), u1 = __shfl_up_sync(0xffffffffu, i1, k);
                if (lane >= k) i0 += u0, i1 += u1;
            }
            start[i] = base0 + i0 - v0;
            slot[i] = base1 + i1 - v1;
            base0 += __shfl_sync(0xffffffffu, i0, 31);
            base1 += __shfl_sync(0xffffffffu, i1, 31);
        }
        pieces = base0;
    }

    __device__ __forceinline__ RowsPiece find(const PagedAttnParams &p, int piece) const {
        int b = -1, rest = 0, n = 1, sl = 0;
#pragma unroll
        for (int i = 0; i < kRwWarpBatch / 32; ++i)
            if (piece >= start[i] && piece < start[i] + ns[i] * items[i])
                b = (int)(threadIdx.x & 31) + 32 * i, rest = piece - start[i], n = ns[i], sl = slot[i];
        const int owner = __ffs((int)__ballot_sync(0xffffffffu, b >= 0)) - 1;
        return rows_piece(p, __shfl_sync(0xffffffffu, b, owner), __shfl_sync(0xffffffffu, rest, owner),
                          __shfl_sync(0xffffffffu, n, owner), __shfl_sync(0xffffffffu, sl, owner));
    }
};

// The same division of a large batch, by one CTA into start[B + 1] (first
// piece of each request) and slot[B + 1] (first slot of each divided one).
constexpr int kDivThreads = 1024;

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *red) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = red[threadIdx.x & 31];
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
    return t;
}

__global__ void __launch_bounds__(kDivThreads) kv4_rows_division_kernel(const __grid_constant__ PagedAttnParams p,
                                                                        int32_t *start) {
    __shared__ int64_t red[32];
    __shared__ int red0[32], red1[32];
    int32_t *slot = start + p.B + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t rounds = 0, items = 0;
    for (int b = threadIdx.x; b < p.B; b += kDivThreads) {
        const int r = rows_rounds(p, b), g = r ? rows_groups(p, b) : 0;
        rounds += (int64_t)r * g;
        items += g;
    }
    const int64_t total = block_sum(rounds, red) * p.Hkv;
    const int64_t s0 = max((int64_t)1, (total + kRwResident - 1) / kRwResident);
    int64_t S = s0;
    if (block_sum(items, red) * p.Hkv <= kRwResident) {
        S = rows_candidate(s0, 3);
        for (int c = 2; c >= 0; --c) {
            const int64_t x = rows_candidate(s0, c);
            int64_t n = 0;
            for (int b = threadIdx.x; b < p.B; b += kDivThreads) {
                const int r = rows_rounds(p, b);
                if (r) n += (r + x - 1) / x * rows_groups(p, b);
            }
            if (block_sum(n, red) * p.Hkv <= kRwResident) S = x;
        }
    }
    int base0 = 0, base1 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kDivThreads) {
        const int b = b0 + threadIdx.x;
        const int ns = b < p.B ? (int)((rows_rounds(p, b) + S - 1) / S) : 0;
        const int v0 = ns ? ns * p.Hkv * rows_groups(p, b) : 0, v1 = ns > 1 ? v0 : 0;
        int i0 = v0, i1 = v1;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int u0 = __shfl_up_sync(0xffffffffu, i0, k), u1 = __shfl_up_sync(0xffffffffu, i1, k);
            if (lane >= k) i0 += u0, i1 += u1;
        }
        __syncthreads();
        if (lane == 31) red0[warp] = i0, red1[warp] = i1;
        __syncthreads();
        int o0 = base0, o1 = base1;
        for (int x = 0; x < kDivThreads / 32; ++x) {
            if (x < warp) o0 += red0[x], o1 += red1[x];
            base0 += red0[x], base1 += red1[x];
        }
        if (b < p.B) {
            start[b] = o0 + i0 - v0;
            slot[b] = o1 + i1 - v1;
        }
    }
    if (threadIdx.x == 0) start[p.B] = base0, slot[p.B] = base1;
}

__device__ __forceinline__ RowsPiece find_piece(const PagedAttnParams &p, const int32_t *start, int piece) {
    int lo = 0, hi = p.B - 1;   // the last request that starts at or before the piece
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= piece) lo = mid;
        else hi = mid - 1;
    }
    const int items = p.Hkv * rows_groups(p, lo);
    return rows_piece(p, lo, piece - start[lo], (start[lo + 1] - start[lo]) / items, start[p.B + 1 + lo]);
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// 16 bytes global -> shared, asynchronously; groups complete in order.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A 16x8 product without an accumulator to add to.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// NSUB: pages per 64-token tile (pages of 64 tokens or more: 1).
template <int D, int NSUB>
__global__ void __launch_bounds__(kRwThreads, 4) kv4_rows_kernel(const __grid_constant__ RowsParams w) {
    constexpr int DB = D / 2;         // code bytes per vector
    constexpr int KW = DB / 16;       // K words a lane reads per token (bytes 4 KW tig .. 4 KW tig + 4 KW - 1)
    constexpr int UB = DB / 16;       // 16-byte blocks (8 units of 4 dims) per vector
    constexpr int KS = D / 16;        // k-steps of the score product
    constexpr int MT = D / 16;        // m-tiles (16 dims) of the output product
    constexpr int TB = kRwTile * DB;  // bytes of one tensor's tile
    constexpr int PSZ = kRowsCols * D + 2 * kRowsCols;
    constexpr float kNone = -1e30f;   // below every score: a running maximum that has seen nothing
    constexpr int CPT = DB / 16;      // 16-byte chunks per vector
    constexpr int CPL = TB / 16 / 32; // chunks a lane copies per tile
    static_assert(kRowsCols * D * 4 <= 3 * TB, "the merge slots fit the code buffers");
    const PagedAttnParams &p = w.a;
    extern __shared__ __align__(128) uint8_t rw_smem[];
    __shared__ float mw[kRwWarps][kRowsCols], lw[kRwWarps][kRowsCols];
    __shared__ float mc[kRowsCols], lc[kRowsCols];
    __shared__ __align__(16) float2 kf_s[kRwWarps][kRwTile];   // per token: 2^24 s c, -z s c (c = log2(e) / sqrt(D))
    __shared__ float vf_s[kRwWarps][kRwTile];                  // value scale * 2^(8 - E)
    __shared__ __align__(16) __half vz_s[kRwWarps][kRwTile];   // value zero
    __shared__ int last_s;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    uint8_t *ring = rw_smem + (size_t)warp * 3 * TB;   // this warp's three tiles of codes, [64][DB] each
    const uint32_t ring_a = smem_u32(ring);
    __half *pt = reinterpret_cast<__half *>(rw_smem + (size_t)kRwWarps * 3 * TB) + warp * (kRwTile * 8);
    // A lane copies the chunks lane + 32 i of a tile: chunk ck of token tk + (32 / CPT) i.
    // Values are stored with a token's chunks permuted, so that the
    // transposed loads of 8 tokens' same chunk touch every bank once.
    const int tk = lane / CPT, ck = lane % CPT;
    const uint32_t k_dst = (uint32_t)(lane * 16);
    const uint32_t v_dst = (uint32_t)(tk * DB + ((ck ^ ((tk * CPT / 8) & (CPT - 1))) * 16));
    // Every request with more rows than the caller promised is named.
    if (blockIdx.x == gridDim.x - 1)
        for (int b = tid; b < p.B; b += kRwThreads)
            if (paged_request(p, b).n > p.max_new) paged_bad_request(p, b);
    const int page_mask = (1 << p.page_shift) - 1;
    const uint32_t page_vecs = (uint32_t)p.Hkv << p.page_shift;   // vectors of one tensor per page
    const int64_t v_minus_k = p.v_codes - p.k_codes;              // bytes
    const int64_t vp_minus_kp = reinterpret_cast<const uint8_t *>(p.v_params) - reinterpret_cast<const uint8_t *>(p.k_params);

    for (int piece = blockIdx.x, pieces;; piece += gridDim.x) {
        RowsPiece pc;
        if (w.division == nullptr) {
            RowsDivision dv;   // again for every piece: few CTAs take two, and it costs no registers meanwhile
            dv.make(p);
            pieces = dv.pieces;
            if (piece < pieces) pc = dv.find(p, piece);
        } else {
            pieces = w.division[p.B];
            if (piece < pieces) pc = find_piece(p, w.division, piece);
        }
        if (piece >= pieces) return;
        const int b = pc.b, h = pc.h, split = pc.split, nsplit = pc.nsplit;
        const PagedRequest r = paged_request(p, b);
        const RowsTiles tl = rows_tiles(p, r);
        const int rounds = max(1, (tl.count + kRwWarps - 1) / kRwWarps);
        const int each = rounds / nsplit, extra = rounds - each * nsplit;   // the first `extra` pieces take one more
        const int k_begin = (split * each + min(split, extra)) * kRwWarps;
        const int k_end = min(k_begin + (each + (split < extra ? 1 : 0)) * kRwWarps, tl.count);
        const int col0 = pc.group * kRowsCols, cols = min(r.n * p.G - col0, kRowsCols);   // the piece's columns
        const int pos0 = r.kv - r.n;   // position of the first row

        auto tile_t0 = [&](int k) {
            return (k < tl.sink_tiles ? k : tl.first + (k - tl.sink_tiles)) * kRwTile;
        };
        // The pages of tile k's parts: their numbers, or -1 past the
        // sequence's end and for numbers outside the cache.
        const int32_t *table = p.block_table + (int64_t)b * p.max_pages;
        auto load_pages = [&](int k, int (&pg)[NSUB]) {
            const int t = tile_t0(k);
#pragma unroll
            for (int i = 0; i < NSUB; ++i) {
                pg[i] = -1;
                if (k < k_end && t + i * (kRwTile / NSUB) < r.kv) {
                    pg[i] = __ldg(table + ((t + i * (kRwTile / NSUB)) >> p.page_shift));
                    if ((uint32_t)pg[i] >= (uint32_t)p.n_pages) {
                        paged_bad_request(p, b);
                        pg[i] = -1;
                    }
                }
            }
        };
        // Tile k's codes into the ring at `dst` as one copy group (empty past
        // the last tile). A part without a page copies page 0's codes, which
        // scales of 0 make nothing of; a page's tail past the sequence's end is in bounds.
        auto issue = [&](int k, bool value, const int (&pg)[NSUB], uint32_t dst) {
            if (k < k_end) {
                const int in_page = tile_t0(k) & page_mask;
                const uint8_t *base = p.k_codes + ((int64_t)h << p.page_shift) * DB + in_page * DB + lane * 16;
                if (value) base += v_minus_k;
#pragma unroll
                for (int i = 0; i < CPL; ++i) {
                    constexpr int per = CPL / NSUB;   // a lane's copies per page
                    const uint8_t *src = base + (uint64_t)(uint32_t)max(pg[i / per], 0) * (page_vecs * DB) + (i % per) * 512;
                    copy16(ring_a + dst + (uint32_t)(i * 512) + (value ? v_dst : k_dst), src);
                }
            }
            copy_commit();
        };
        // The tile's scales and zeros: token lane + 32 i in word i, as
        // (scale | zero << 16); 0 past the sequence's end and on bad pages.
        auto load_sz = [&](int k, const int (&pg)[NSUB], uint32_t (&kw)[2], uint32_t (&vw)[2]) {
            const int t = tile_t0(k) + lane, in_page = (NSUB == 1 ? t - lane : 0) & page_mask;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                constexpr int part = kRwTile / NSUB;   // tokens per page of the tile (64, 32 or 16)
                int page = pg[i * (NSUB / 2)];
                int off = in_page + lane + 32 * i;
                if (NSUB == 2) off = lane;
                if (NSUB == 4) {
                    page = lane < 16 ? pg[(2 * i) % NSUB] : pg[(2 * i + 1) % NSUB];
                    off = lane & (part - 1);
                }
                kw[i] = vw[i] = 0u;
                if (page >= 0 && t + 32 * i < r.kv) {
                    const uint8_t *at = reinterpret_cast<const uint8_t *>(p.k_params) +
                                        (((uint64_t)(uint32_t)page * page_vecs + ((uint32_t)h << p.page_shift) + off) << 2);
                    kw[i] = __ldg(reinterpret_cast<const uint32_t *>(at));
                    vw[i] = __ldg(reinterpret_cast<const uint32_t *>(at + vp_minus_kp));
                }
            }
        };

        int k = k_begin + warp;
        uint32_t s0 = 0, s1 = TB, s2 = 2 * TB;   // ring places of this tile's keys and values and the next tile's keys
        int pgn[NSUB];
        uint32_t kw[2] = {0u, 0u}, vw[2] = {0u, 0u};
        {
            int pg[NSUB];
            load_pages(k, pg);
            load_pages(k + kRwWarps, pgn);
            issue(k, false, pg, s0);
            issue(k, true, pg, s1);
            if (k < k_end) load_sz(k, pg, kw, vw);
            issue(k + kRwWarps, false, pgn, s2);
        }

        // The columns' queries as the B fragments of the score product
        // (columns >= cols zero). The product's k index is a permutation of
        // the dims, fixed by how a lane unpacks its code words: for the
        // lane's word i (dims d = (D/4) tig + 8 i .. d + 7; byte b holds dims
        // d + 2b, d + 2b + 1), k-step 2 i takes the low nibbles, pairing dims
        // (d, d+4) and (d+2, d+6), k-step 2 i + 1 the high nibbles, pairing
        // (d+1, d+5) and (d+3, d+7).
        uint32_t qf[KS][2];
        float sq2[2];
        {
            const int col = col0 + gid, i0 = (col * w.g_inv) >> 16;   // i0 = col / G
            const __half *qrow = p.q + (int64_t)(r.row0 + i0) * p.q_stride +
                                 (int64_t)(h * p.G + col - i0 * p.G) * D + tig * (D / 4);
            const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (gid < cols) u = __ldg(reinterpret_cast<const uint4 *>(qrow + 8 * i));
                qf[2 * i][0] = __byte_perm(u.x, u.z, 0x5410);
                qf[2 * i][1] = __byte_perm(u.y, u.w, 0x5410);
                // High nibbles enter 16 times too large.
                const uint32_t h0 = __byte_perm(u.x, u.z, 0x7632), h1 = __byte_perm(u.y, u.w, 0x7632);
                qf[2 * i + 1][0] = half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&h0), sixteenth));
                qf[2 * i + 1][1] = half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&h1), sixteenth));
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&uw[e]));
                    sq += f.x + f.y;
                }
            }
            sq += __shfl_xor_sync(0xffffffffu, sq, 1);
            sq += __shfl_xor_sync(0xffffffffu, sq, 2);            // column gid's sum of dims, for the zero points
            sq2[0] = __shfl_sync(0xffffffffu, sq, 8 * tig);       // column 2 tig
            sq2[1] = __shfl_sync(0xffffffffu, sq, 8 * tig + 4);   // column 2 tig + 1
        }
        // Positions of the lane's two columns; columns >= cols see every token.
        int cpos[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) cpos[c] = 2 * tig + c < cols ? pos0 + (((col0 + 2 * tig + c) * w.g_inv) >> 16) : r.kv - 1;

        float m2[2] = {kNone, kNone};    // running maximum of columns 2 tig, 2 tig + 1
        float l2[2] = {0.0f, 0.0f};      // running sum of the same columns
        int eb = 103;                    // 127 + the largest value scale's exponent so far (scales >= 2^-24)
        // The output, transposed (dims x columns), in units of 2^(E - 32) (the
        // codes enter the products as FP16 subnormals c * 2^-24). m-tile
        // 2 u + e holds dims 4 (8 u + gid) + 2 e in row gid and the next dim, in
        // units of 2^(E - 28), in row gid + 8; columns 2 tig, 2 tig + 1,
        // those of the lane's scores. oz: sum of z P in every row, units of 2^(E - 8).
        float o[MT][4], oz[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        const uint32_t pt_st = smem_u32(pt) + (uint32_t)(gid * 16 + tig * 4);
        const uint32_t pt_ld = smem_u32(pt) + (uint32_t)((lane & 15) * 16);
        // Transposed loads of value codes: matrices (tokens 0-7, chunk 2 x),
        // (tokens 8-15, chunk 2 x), then the same of chunk 2 x + 1. The lane's
        // token and its chunk's place, for x = 0; x = 1 flips bit 1 of the place.
        const uint32_t v_ld = (uint32_t)((lane & 15) * DB +
                                         (((lane >> 4) ^ (((lane & 7) * CPT / 8) & (CPT - 1))) * 16));

        for (; k < k_end; k += kRwWarps) {
            const int t0 = tile_t0(k);
            int pgnn[NSUB];
            load_pages(k + 2 * kRwWarps, pgnn);
            uint32_t kwn[2] = {0u, 0u}, vwn[2] = {0u, 0u};
            if (k + kRwWarps < k_end) load_sz(k + kRwWarps, pgn, kwn, vwn);   // in flight while this tile is computed
            // Whether every column sees every token of the tile.
            const bool whole = t0 + kRwTile - 1 <= pos0 &&
                               (p.window == 0 || pos0 + r.n - 1 - t0 < p.window || t0 + kRwTile <= p.sinks);
            // The largest value scale (FP16 bits of values >= 0 are ordered),
            // and the tokens' factors for everyone. A written scale is finite
            // and a zero at most 15; the bounds make the values' both so for
            // whatever a hidden token may hold, so that its weight 0 stays 0.
#pragma unroll
            for (int i = 0; i < 2; ++i) vw[i] = min(vw[i] & 0xFFFFu, 0x7BFFu) | (min(vw[i] >> 16, 0x4B80u) << 16);
            const uint32_t sv = __reduce_max_sync(0xffffffffu, max(vw[0] & 0xFFFFu, vw[1] & 0xFFFFu));
            const int ebn = max(eb, (int)(__float_as_uint(half_lo(sv)) >> 23));
            const float ef = __int_as_float((262 - ebn) << 23);   // 2^(8 - E)
            __syncwarp();   // every lane is done with the last tile's factors
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float s = half_lo(kw[i]) * p.qscale;
                kf_s[warp][lane + 32 * i] = make_float2(s * 0x1p24f, -__half2float(half_hi(kw[i])) * s);
                vf_s[warp][lane + 32 * i] = half_lo(vw[i]) * ef;
                vz_s[warp][lane + 32 * i] = half_hi(vw[i]);
            }
            copy_wait<2>();   // this tile's keys have landed
            __syncwarp();
            // 1. Scores (tokens x columns) of the tile's four 16-token steps:
            // s c (2^24 acc - z sum(q)).
            float sc[4][4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {   // two steps' chains of products side by side
                uint32_t wa[2][KW], wb[2][KW];
                float acc[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint8_t *ka = ring + s0 + (16 * (j + e) + gid) * DB + tig * (4 * KW);
                    if constexpr (KW == 4) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(ka);
                        const uint4 y = *reinterpret_cast<const uint4 *>(ka + 8 * DB);
                        wa[e][0] = x.x, wa[e][1] = x.y, wa[e][2] = x.z, wa[e][3] = x.w;
                        wb[e][0] = y.x, wb[e][1] = y.y, wb[e][2] = y.z, wb[e][3] = y.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(ka);
                        const uint2 y = *reinterpret_cast<const uint2 *>(ka + 8 * DB);
                        wa[e][0] = x.x, wa[e][1] = x.y;
                        wb[e][0] = y.x, wb[e][1] = y.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    uint32_t a[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[0] = wa[e][i] & 0x000F000Fu;
                        a[1] = wb[e][i] & 0x000F000Fu;
                        a[2] = (wa[e][i] >> 8) & 0x000F000Fu;
                        a[3] = (wb[e][i] >> 8) & 0x000F000Fu;
                        if (i == 0) mma_16816_first(acc[e], a, qf[0][0], qf[0][1]);
                        else mma_16816(acc[e], a, qf[2 * i][0], qf[2 * i][1]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[0] = wa[e][i] & 0x00F000F0u;
                        a[1] = wb[e][i] & 0x00F000F0u;
                        a[2] = (wa[e][i] >> 8) & 0x00F000F0u;
                        a[3] = (wb[e][i] >> 8) & 0x00F000F0u;
                        mma_16816(acc[e], a, qf[2 * i + 1][0], qf[2 * i + 1][1]);
                    }
                }
                // acc[0], acc[1]: token gid, columns 2 tig, 2 tig + 1; acc[2], acc[3]: token gid + 8.
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 fA = kf_s[warp][16 * (j + e) + gid], fB = kf_s[warp][16 * (j + e) + gid + 8];
                    sc[j + e][0] = fmaf(acc[e][0], fA.x, fA.y * sq2[0]);
                    sc[j + e][1] = fmaf(acc[e][1], fA.x, fA.y * sq2[1]);
                    sc[j + e][2] = fmaf(acc[e][2], fB.x, fB.y * sq2[0]);
                    sc[j + e][3] = fmaf(acc[e][3], fB.x, fB.y * sq2[1]);
                }
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int t = t0 + 16 * j + gid + (c >> 1) * 8, d = cpos[c & 1] - t;
                        if (!(d >= 0 && (p.window == 0 || d < p.window || t < p.sinks))) sc[j][c] = -INFINITY;
                    }
            }
            __syncwarp();   // every lane is done with the keys: the next tile's values take their place
            issue(k + kRwWarps, true, pgn, s0);
            // 2. Online softmax over the whole tile. The running maximum
            // starts at a finite value below every score, so a column that
            // sees nothing keeps p = 2^-inf = 0.
            float mx[2] = {m2[0], m2[1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mx[0] = fmaxf(mx[0], fmaxf(sc[j][0], sc[j][2]));
                mx[1] = fmaxf(mx[1], fmaxf(sc[j][1], sc[j][3]));
            }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], s));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], s));
            }
            const bool raise = mx[0] > m2[0] + kRwSlack || mx[1] > m2[1] + kRwSlack;
            if (__any_sync(0xffffffffu, raise || ebn != eb)) {
                const float es = __int_as_float((127 + eb - ebn) << 23);   // 2^(E_old - E_new)
                eb = ebn;
                float al[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mn = mx[c] > m2[c] + kRwSlack ? mx[c] : m2[c];
                    al[c] = ex2_approx(m2[c] - mn);
                    m2[c] = mn;
                    l2[c] *= al[c];
                    al[c] *= es;
                    oz[c] *= al[c];
                }
#pragma unroll
                for (int jj = 0; jj < MT; ++jj) {
                    o[jj][0] *= al[0];
                    o[jj][2] *= al[0];
                    o[jj][1] *= al[1];
                    o[jj][3] *= al[1];
                }
            }
            // P = p * s_V * 2^(8 - E), FP16, into the P tile.
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float svA = vf_s[warp][16 * j + gid], svB = vf_s[warp][16 * j + gid + 8];
                float pr[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    pr[c] = ex2_approx(sc[j][c] - m2[c & 1]);
                    l2[c & 1] += pr[c];   // this lane's tokens; summed over the lanes at the end
                }
                sts32(pt_st + (uint32_t)(16 * j * 16), half2_bits(__floats2half2_rn(pr[0] * svA, pr[1] * svA)));
                sts32(pt_st + (uint32_t)((16 * j + 8) * 16), half2_bits(__floats2half2_rn(pr[2] * svB, pr[3] * svB)));
            }
            copy_wait<2>();   // this tile's values have landed
            __syncwarp();     // and the P tile is written
            // 3. out^T (dims x columns) += c_V^T (dims x tokens) . P^T, 16
            // tokens at a time. A register of a transposed load holds the same
            // 4 dims of tokens 2 tig and 2 tig + 1 (or 2 tig + 8, 2 tig + 9).
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t pb0, pb1;   // P^T as the column-major B operand: tokens 2 tig.., column gid
                ldsm_x2_trans(pt_ld + (uint32_t)(16 * j * 16), pb0, pb1);
#pragma unroll
                for (int u = 0; u < UB; u += 2) {
                    uint32_t x[4];
                    ldsm_x4_trans(ring_a + s1 + (v_ld ^ (uint32_t)(u * 16)) + (uint32_t)(16 * j * DB), x);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t lo = x[2 * e], hi = x[2 * e + 1], lo8 = lo >> 8, hi8 = hi >> 8;
                        uint32_t a[4];
                        a[0] = lo & 0x000F000Fu;
                        a[1] = lo & 0x00F000F0u;
                        a[2] = hi & 0x000F000Fu;
                        a[3] = hi & 0x00F000F0u;
                        mma_16816(o[2 * (u + e)], a, pb0, pb1);
                        a[0] = lo8 & 0x000F000Fu;
                        a[1] = lo8 & 0x00F000F0u;
                        a[2] = hi8 & 0x000F000Fu;
                        a[3] = hi8 & 0x00F000F0u;
                        mma_16816(o[2 * (u + e) + 1], a, pb0, pb1);
                    }
                }
                const uint32_t z0 = *reinterpret_cast<const uint32_t *>(&vz_s[warp][16 * j + 2 * tig]);
                const uint32_t z8 = *reinterpret_cast<const uint32_t *>(&vz_s[warp][16 * j + 2 * tig + 8]);
                const uint32_t az[4] = {z0, z0, z8, z8};
                mma_16816(oz, az, pb0, pb1);
            }
            __syncwarp();   // every lane is done with the values: the keys after the next take their place
            issue(k + 2 * kRwWarps, false, pgnn, s1);
            const uint32_t s = s0;
            s0 = s2, s2 = s1, s1 = s;
            kw[0] = kwn[0], kw[1] = kwn[1], vw[0] = vwn[0], vw[1] = vwn[1];
#pragma unroll
            for (int i = 0; i < NSUB; ++i) pgn[i] = pgnn[i];
        }
        copy_wait<0>();

        // Merge the warps: maxima and sums per column, then the outputs in
        // real units rescaled to the CTA's maxima, each warp's into its own
        // FP32 slot over the (now idle) code buffers, summed in a fixed order.
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
            l2[0] += __shfl_xor_sync(0xffffffffu, l2[0], s);
            l2[1] += __shfl_xor_sync(0xffffffffu, l2[1], s);
        }
        if (gid == 0) {
            mw[warp][2 * tig] = m2[0];
            mw[warp][2 * tig + 1] = m2[1];
            lw[warp][2 * tig] = l2[0];
            lw[warp][2 * tig + 1] = l2[1];
        }
        __syncthreads();
        float *ow = reinterpret_cast<float *>(rw_smem);   // [kRwWarps][kRowsCols][D]
        if (tid < kRowsCols) {
            float M = kNone;
            for (int x = 0; x < kRwWarps; ++x) M = fmaxf(M, mw[x][tid]);
            float L = 0.0f;
            for (int x = 0; x < kRwWarps; ++x) L += exp2f(mw[x][tid] - M) * lw[x][tid];
            mc[tid] = M;
            lc[tid] = L;
        }
        __syncthreads();
        const float unit = __int_as_float((eb - 8) << 23);   // 2^(E - 8)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int g = 2 * tig + c;
            if (g < cols) {
                const float f = exp2f(m2[c] - mc[g]) * unit;
                float *dst = ow + (warp * kRowsCols + g) * D;
#pragma unroll
                for (int u = 0; u < UB; ++u)
                    *reinterpret_cast<float4 *>(dst + 4 * (8 * u + gid)) =
                        make_float4(fmaf(o[2 * u][c], 0x1p24f, -oz[c]) * f, fmaf(o[2 * u][2 + c], 0x1p20f, -oz[c]) * f,
                                    fmaf(o[2 * u + 1][c], 0x1p24f, -oz[c]) * f,
                                    fmaf(o[2 * u + 1][2 + c], 0x1p20f, -oz[c]) * f);
            }
        }
        __syncthreads();
        auto out_at = [&](int i) {   // element i of [columns][D]
            const int c = col0 + i / D, i0 = (c * w.g_inv) >> 16;   // i0 = c / G
            return p.out + (int64_t)(r.row0 + i0) * p.out_stride + (int64_t)(h * p.G + c - i0 * p.G) * D + (i % D);
        };
        if (nsplit == 1) {
            for (int i = tid; i < cols * D; i += kRwThreads) {
                float sum = ow[i];
                for (int x = 1; x < kRwWarps; ++x) sum += ow[x * kRowsCols * D + i];
                const float L = lc[i / D];
                *out_at(i) = __float2half_rn(L > 0.0f ? sum / L : 0.0f);
            }
        } else {
            // Several pieces of this (request, head): store this one's
            // unnormalised sums with its maxima and weights, arrive, and let
            // the last arriver combine.
            const int s0 = pc.slot;
            float *part = w.part + (int64_t)(s0 + split) * PSZ;
            for (int i = tid; i < cols * D; i += kRwThreads) {
                float sum = ow[i];
                for (int x = 1; x < kRwWarps; ++x) sum += ow[x * kRowsCols * D + i];
                part[i] = sum;
            }
            if (tid < kRowsCols) {
                part[kRowsCols * D + tid] = mc[tid];
                part[kRowsCols * D + kRowsCols + tid] = lc[tid];
            }
            __syncthreads();   // every store of the CTA precedes the arrival (cumulative release)
            if (tid == 0) last_s = atom_add_acq_rel_gpu(w.counters + s0, 1) == nsplit - 1;
            __syncthreads();
            if (last_s) {
                const float *base = w.part + (int64_t)s0 * PSZ;
                if (tid < kRowsCols) {
                    float M = kNone;
                    for (int c = 0; c < nsplit; ++c) M = fmaxf(M, __ldcg(base + c * PSZ + kRowsCols * D + tid));
                    float L = 0.0f;
                    for (int c = 0; c < nsplit; ++c)
                        L += exp2f(__ldcg(base + c * PSZ + kRowsCols * D + tid) - M) *
                             __ldcg(base + c * PSZ + kRowsCols * D + kRowsCols + tid);
                    mc[tid] = M;
                    lc[tid] = L;
                }
                __syncthreads();
                for (int i = tid; i < cols * D; i += kRwThreads) {
                    const int g = i / D;
                    float O = 0.0f;
                    for (int c = 0; c < nsplit; ++c)
                        O += exp2f(__ldcg(base + c * PSZ + kRowsCols * D + g) - mc[g]) * __ldcg(base + c * PSZ + i);
                    *out_at(i) = __float2half_rn(lc[g] > 0.0f ? O / lc[g] : 0.0f);
                }
                if (tid == 0) w.counters[s0] = 0;   // nobody arrives on it again in this call
            }
        }
        if (piece + (int)gridDim.x >= pieces) return;
        __syncthreads();   // the next piece's copies land where the merge wrote
    }
}

template <int D, int NSUB>
cudaError_t launch(const RowsParams &w, cudaStream_t stream) {
    // Per warp, three 64-token tiles of codes, then the P tiles (1 KB per
    // warp): 52 KB at D = 128, four CTAs per SM.
    constexpr int smem = kRwWarps * 3 * kRwTile * D / 2 + kRwWarps * kRwTile * 8 * 2;
    if (smem > 40 * 1024) {
        static SmemOptIn opt_in;
        const cudaError_t e = opt_in.set(kv4_rows_kernel<D, NSUB>, smem);
        if (e != cudaSuccess) return e;
    }
    kv4_rows_kernel<D, NSUB><<<kRwResident, kRwThreads, smem, stream>>>(w);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const RowsParams &w, cudaStream_t stream) {
    return w.a.page_shift >= 6 ? launch<D, 1>(w, stream)
                               : (w.a.page_shift == 5 ? launch<D, 2>(w, stream) : launch<D, 4>(w, stream));
}

}  // namespace

// Workspace: counters, partial results, the division of large batches.
size_t rows_workspace_bytes(int64_t B, int64_t D) {
    return (size_t)align256(4 * kRwSplitSlots) +
           (size_t)align256(4 * (int64_t)kRwSplitSlots * (kRowsCols * D + 2 * kRowsCols)) +
           (B > kRwWarpBatch ? (size_t)align256(8 * (B + 1)) : 0);
}

cudaError_t launch_paged_rows(const PagedAttnParams &p, int64_t D, void *ws, cudaStream_t stream) {
    RowsParams w;
    w.a = p;
    w.g_inv = (65536 + p.G - 1) / p.G;
    uint8_t *at = static_cast<uint8_t *>(ws);
    w.counters = reinterpret_cast<int32_t *>(at);
    at += align256(4 * kRwSplitSlots);
    w.part = reinterpret_cast<float *>(at);
    at += align256(4 * (int64_t)kRwSplitSlots * (kRowsCols * D + 2 * kRowsCols));
    w.division = nullptr;
    if (p.B > kRwWarpBatch) {
        w.division = reinterpret_cast<int32_t *>(at);
        kv4_rows_division_kernel<<<1, kDivThreads, 0, stream>>>(p, reinterpret_cast<int32_t *>(at));
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return D == 128 ? launch<128>(w, stream) : launch<64>(w, stream);
}

}  // namespace qoq
