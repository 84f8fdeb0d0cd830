// Paged KV4 attention for requests with few rows: n new tokens x G query
// heads per KV head <= 48 (decode steps, short drafts).
//
// The work is one pass over the request's K and V codes (D + 8 bytes per
// token and KV head), so it is bound by HBM where sequences are long, and by
// a launch's latency where they are short. Eight of a KV head's n x G (row,
// head) pairs are the columns of the tensor-core products, so K and V are read
// once for all of them; more pairs are the columns of further items, which read
// the same cache again (from L2, as they run side by side).
//
// Measured (8 KV heads of 128, 4 query heads each, GPU time of a call): 64
// sequences of 1024 tokens in 23.1 us (3.1 TB/s), of 4096 in 62 us (4.6 TB/s),
// 74 of 4096, which fill the GPU evenly, in 63 us (5.2 TB/s of 6.6 that a copy
// reaches); one of 64 tokens in 5.8 us. At length the issue slots are 55% taken, the
// ALU pipe, which unpacks, 55%, the tensor pipe 31% and the memory 60%: none at its
// limit, and four warps per scheduler (of 128 registers each) wait for their own chains.
//
// The division. The lengths are known on the device only, so every CTA works out
// the same division: a request's visible tokens are 64-token tiles (those of
// the sinks, then those of the window), four tiles are a round, and the rounds of
// all items, one after another, are cut into equal shares, one per resident CTA
// (four per SM), so that all SMs end together whatever the mix of lengths (24
// sequences of 100 to 32700 tokens in pages of 16 took 52 us when this was
// introduced, 56 in even pieces of each item; 46.4 now). An item that several
// CTAs share leaves FP32 partial sums, which the last to arrive combines in a
// fixed order.
//
// Within a share, each warp walks every fourth tile. Its K and V code tiles
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
// nibbles are divided by 16 beforehand, after a scaling that keeps their bits, so
// that one accumulator takes both, and the zero points are subtracted afterwards: s (q.c) - s z sum(q) per
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
constexpr int kRwStart = 2;                   // rounds that fit in the time in which an item starts and is merged (64
                                              // sequences of 100 to 9000 tokens: 53, 48, 47, 50 us with 0, 1, 2, 3)
constexpr int kRwWarpBatch = 128;             // requests whose division each warp works out itself (64 requests, 64 tokens
                                              // each: 8.4 us, with the division kernel 12.8)
constexpr float kRwSlack = 6.0f;              // log2 by which scores may exceed the running maximum

struct RowsParams {
    PagedAttnParams a;
    int g_inv;               // ceil(2^16 / G): c / G = c g_inv >> 16 for c < 64
    int reach;               // the window, or INT32_MAX: a row sees the tokens less than so far before it
    int32_t *counters;       // [kRwResident], zero between calls
    float *part;             // [2 kRwResident][kRowsCols * D + 2 * kRowsCols]
    const int64_t *first;    // [B + 2] from the division kernel where B > kRwWarpBatch, else null
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

__device__ __forceinline__ int rows_items(const PagedAttnParams &p, int b) { return p.Hkv * rows_groups(p, b); }

// Rounds (four tiles) of request b for this kernel: 0 if it has no rows or
// too many; one where it has rows but no token (zeros are written).
__device__ __forceinline__ int rows_rounds(const PagedAttnParams &p, int b) {
    const PagedRequest r = paged_request(p, b);
    if (r.n == 0 || r.n > p.max_new || r.n * p.G > kRowsMax) return 0;
    return max(1, (rows_tiles(p, r).count + kRwWarps - 1) / kRwWarps);
}

// The division. A (request, KV head, column group) is an item of so many
// rounds, and of kRwStart rounds' time before the first. The items follow one
// another by request, head, group; CTA c takes [c S, (c + 1) S) of that
// sequence, S = ceil(total / resident CTAs): as much for each whatever the
// lengths. Its first segment may be the end or a part of an item, its last a
// beginning; those between are whole. Where one item per CTA ends about as
// soon (the longest is hardly above S, and a second segment costs a start),
// every item counts as long as the longest and none is divided.
struct RowsWork {
    int S;            // rounds per CTA
    int same;         // the length that every item counts as, or 0: its own
    int remaining, done;   // rounds of this CTA, and those of them that are done
    int b, item, offset;   // where the next begins: item of request b, round of the item
};

// What the end of a segment needs of it.
struct RowsSegment {
    int count;             // rounds, the start's included
    int before, nsplit;    // CTAs before this one and CTAs that the item's rounds are divided over
    int row0, h, col0, cols;
    bool last_item;        // of its request
};

// Length of request b's items: 0 without rows for this kernel.
__device__ __forceinline__ int rows_length(const PagedAttnParams &p, int b, int same) {
    const int rounds = rows_rounds(p, b);
    return rounds == 0 ? 0 : same ? same : rounds + kRwStart;
}

// From the batch's items, the sum of their lengths and the longest: S, same
// and the sum that results.
__device__ __forceinline__ int64_t rows_shares(RowsWork &w, int64_t items, int64_t total, int longest) {
    w.S = total <= kRwResident ? 1 : (int)((uint64_t)(total + kRwResident - 1) / kRwResident);
    w.same = 0;
    if (items <= kRwResident && longest <= w.S + kRwStart) {
        w.S = w.same = longest;
        return items * longest;
    }
    return total;
}

// Where x of the sequence lies, in_request behind the first of request b's.
__device__ __forceinline__ void rows_begin(const PagedAttnParams &p, RowsWork &w, int64_t total, int64_t x, int b,
                                           int64_t in_request) {
    const int length = rows_length(p, b, w.same);
    w.remaining = (int)min((int64_t)w.S, total - x);
    w.done = 0;
    w.b = b;
    w.item = (int)((uint64_t)in_request / (uint32_t)max(length, 1));
    w.offset = (int)(in_request - (int64_t)w.item * length);
}

// floor(a / x) for 0 <= a < 2^24, 0 < x < 2^27: `inv` = 1 / x rounded; the
// estimate is within one of the quotient, and the products fit.
__device__ __forceinline__ int floor_div(int a, int x, float inv) {
    int q = (int)((float)a * inv);
    q -= q * x > a ? 1 : 0;
    return q + ((q + 1) * x <= a ? 1 : 0);
}

// A batch of up to kRwWarpBatch requests, by each warp: lane l holds the
// requests l per, l per + 1, ... false: nothing is left for this CTA.
__device__ __forceinline__ bool rows_divide(const PagedAttnParams &p, RowsWork &w) {
    const int lane = threadIdx.x & 31, per = (p.B + 31) >> 5;
    int64_t sum = 0;
    int items = 0, longest = 0;
    for (int i = 0; i < per; ++i) {
        const int b = lane * per + i, n = b < p.B ? rows_length(p, b, 0) : 0;
        if (n == 0) continue;
        const int k = rows_items(p, b);
        sum += (int64_t)n * k;
        items += k;
        longest = max(longest, n);
    }
    int64_t upto = sum;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, upto, k);
        if (lane >= k) upto += u;
    }
    const int64_t total = rows_shares(w, __reduce_add_sync(0xffffffffu, (uint32_t)items),
                                      __shfl_sync(0xffffffffu, upto, 31),
                                      (int)__reduce_max_sync(0xffffffffu, (uint32_t)longest));
    const int64_t x = (int64_t)blockIdx.x * w.S;
    if (x >= total) return false;
    if (w.same) {
        upto = (int64_t)items * w.same;
        sum = upto;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, upto, k);
            if (lane >= k) upto += u;
        }
    }
    const int owner = __ffs((int)__ballot_sync(0xffffffffu, upto > x)) - 1;
    int64_t rest = x - __shfl_sync(0xffffffffu, upto - sum, owner);
    int b = owner * per;
    for (; b + 1 < p.B; ++b) {
        const int64_t n = (int64_t)rows_length(p, b, w.same) * rows_items(p, b);
        if (rest < n) break;
        rest -= n;
    }
    rows_begin(p, w, total, x, b, rest);
    return true;
}

// The same of a large batch, by one CTA: what precedes each request, the sum,
// and `S`, `same`.
constexpr int kDivThreads = 1024;

__global__ void __launch_bounds__(kDivThreads) kv4_rows_division_kernel(const __grid_constant__ PagedAttnParams p,
                                                                        int64_t *first) {
    __shared__ int64_t red[32], red_items[32];
    __shared__ int red_longest[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t total = 0, items = 0;
    int longest = 0;
    for (int b = threadIdx.x; b < p.B; b += kDivThreads) {
        const int n = rows_length(p, b, 0), k = n ? rows_items(p, b) : 0;
        total += (int64_t)n * k;
        items += k;
        longest = max(longest, n);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, k);
        items += __shfl_xor_sync(0xffffffffu, items, k);
    }
    longest = (int)__reduce_max_sync(0xffffffffu, (uint32_t)longest);
    if (lane == 0) red[warp] = total, red_items[warp] = items, red_longest[warp] = longest;
    __syncthreads();
    total = 0, items = 0, longest = 0;
    for (int x = 0; x < kDivThreads / 32; ++x) {
        total += red[x], items += red_items[x];
        longest = max(longest, red_longest[x]);
    }
    RowsWork w;
    total = rows_shares(w, items, total, longest);
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kDivThreads) {
        const int b = b0 + threadIdx.x;
        const int n = b < p.B ? rows_length(p, b, w.same) : 0;
        const int64_t v = n ? (int64_t)n * rows_items(p, b) : 0;
        int64_t upto = v;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, upto, k);
            if (lane >= k) upto += u;
        }
        __syncthreads();
        if (lane == 31) red[warp] = upto;
        __syncthreads();
        int64_t before = base;
        for (int x = 0; x < kDivThreads / 32; ++x) {
            if (x < warp) before += red[x];
            base += red[x];
        }
        if (b < p.B) first[b] = before + upto - v;
    }
    if (threadIdx.x == 0) first[p.B] = total, first[p.B + 1] = (int64_t)w.S << 32 | (uint32_t)w.same;
}

__device__ __forceinline__ bool rows_find(const PagedAttnParams &p, RowsWork &w, const int64_t *first) {
    const int64_t total = first[p.B], shares = first[p.B + 1];
    w.S = (int)(shares >> 32);
    w.same = (int)(uint32_t)shares;
    const int64_t x = (int64_t)blockIdx.x * w.S;
    if (x >= total) return false;
    int lo = 0, hi = p.B - 1;   // the last request that begins at or before x: it has rounds
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    rows_begin(p, w, total, x, lo, x - first[lo]);
    return true;
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

// SMALL: pages below 64 tokens, so that a tile has several.
template <int D, bool SMALL>
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
    static_assert(kRwResident * kRowsCols * 4 <= kRwWarps * (3 * TB + kRwTile * 16), "and the segments' factors");
    const PagedAttnParams &p = w.a;
    extern __shared__ __align__(128) uint8_t rw_smem[];
    __shared__ float mw[kRwWarps][kRowsCols], lw[kRwWarps][kRowsCols];
    __shared__ float mc[kRowsCols], lc[kRowsCols];
    __shared__ __align__(16) float2 kf_s[kRwWarps][kRwTile];   // per token: 2^24 s c, -z s c (c = log2(e) / sqrt(D))
    __shared__ __align__(16) float vf_s[kRwWarps][kRwTile];                  // value scale * 2^(8 - E)
    __shared__ __align__(16) __half vz_s[kRwWarps][kRwTile];   // value zero
    __shared__ int last_s;
    __shared__ RowsWork work_s;       // kept here and not in registers while the tiles are walked
    __shared__ RowsSegment seg_s;

    griddep_launch_dependents();   // the many-rows kernel's division
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    uint8_t *ring = rw_smem + (size_t)warp * 3 * TB;   // this warp's three tiles of codes, [64][DB] each
    const uint32_t ring_a = smem_u32(ring);
    __half *pt = reinterpret_cast<__half *>(rw_smem + (size_t)kRwWarps * 3 * TB) + warp * (kRwTile * 8);
    // In small pages eight lanes copy the codes of 16 tokens, which lie in one
    // page whatever its size: lane l the 16-byte chunks l % 8 + 8 i of the
    // tile's tokens 16 (l / 8) .. + 15. Else a lane copies chunks l + 32 i:
    // 512 bytes in a row per copy (the former would cost 3% there; it saves 5%
    // where four lookups and addresses per tile and lane are the alternative).
    // Values are stored with a token's chunks permuted, so that the transposed
    // loads of 8 tokens' same chunk touch every bank once: chunk c of token t is
    // at c ^ (t / (8 / CPT)) % CPT, which is c ^ i % CPT in small pages and the same for every i else.
    const int part = SMALL ? (lane >> 3) * 16 : 0;   // first token of the lane's page in a tile
    // The two tokens whose factors it reads: neighbours, which share a small page, in one load; else two loads of a run.
    const int tok0 = SMALL ? 2 * lane : lane, tok1 = SMALL ? 2 * lane + 1 : lane + 32;
    const uint32_t src0 = (uint32_t)((SMALL ? lane & 7 : lane) * 16);
    const uint32_t dst0 = (uint32_t)(part * DB) + src0;
    const uint32_t swap = SMALL ? 0u : (uint32_t)((lane / 8) % CPT * 16);
    constexpr int STEP = SMALL ? 128 : 512;
    // Every request with more rows than the caller promised is named.
    if (blockIdx.x == gridDim.x - 1)
        for (int b = tid; b < p.B; b += kRwThreads)
            if (paged_request(p, b).n > p.max_new) paged_bad_request(p, b);
    const int page_mask = (1 << p.page_shift) - 1;
    const uint32_t page_vecs = (uint32_t)p.Hkv << p.page_shift;   // vectors of one tensor per page
    const int64_t v_minus_k = p.v_codes - p.k_codes;              // bytes
    const int64_t vp_minus_kp = reinterpret_cast<const uint8_t *>(p.v_params) - reinterpret_cast<const uint8_t *>(p.k_params);

    {
        RowsWork wk;
        if (!(w.first == nullptr ? rows_divide(p, wk) : rows_find(p, wk, w.first))) return;
        if (tid == 0) work_s = wk;
    }
    for (;;) {
        __syncthreads();   // work_s is written, and the last segment's merge done with the buffers
        const int b = work_s.b;
        const PagedRequest r = paged_request(p, b);
        const RowsTiles tl = rows_tiles(p, r);
        const int rounds = max(1, (tl.count + kRwWarps - 1) / kRwWarps);
        const int groups = max(1, (r.n * p.G + kRowsCols - 1) / kRowsCols);
        const int h = min(work_s.item / groups, p.Hkv - 1), group = work_s.item - h * groups;
        const int length = work_s.same ? work_s.same : rounds + kRwStart;
        const int count = min(length - work_s.offset, work_s.remaining - work_s.done);   // of this segment
        const int round0 = max(work_s.offset - kRwStart, 0), round1 = min(work_s.offset + count - kRwStart, rounds);
        const int k_begin = round0 * kRwWarps, k_end = min(round1 * kRwWarps, tl.count);
        const int col0 = group * kRowsCols, cols = min(r.n * p.G - col0, kRowsCols);   // the item's columns
        if (tid == 0) {
            // The item's rounds lie with the CTAs blockIdx.x - before ... of
            // which there are nsplit: `ahead` of its rounds precede this CTA's first.
            const int S = work_s.S;
            const float inv = __frcp_rn((float)S);
            const int ahead = round0 ? round0 : -(work_s.done + kRwStart - work_s.offset);
            seg_s.before = ahead > 0 ? floor_div(ahead + S - 1, S, inv) : 0;
            seg_s.nsplit = round0 < round1 ? seg_s.before + floor_div(rounds - 1 - ahead, S, inv) + 1 : 0;
            seg_s.row0 = r.row0;
            seg_s.h = h;
            seg_s.col0 = col0;
            seg_s.cols = cols;
            seg_s.count = count;
            seg_s.last_item = work_s.item + 1 == p.Hkv * groups;
        }
        const int pos0 = r.kv - r.n;   // position of the first row

        auto tile_t0 = [&](int k) {
            return (k < tl.sink_tiles ? k : tl.first + (k - tl.sink_tiles)) * kRwTile;
        };
        // The page of the lane's tokens of tile k, as the table has it (-1 past the
        // sequence's end). It is looked at a tile later, when it has arrived:
        // `checked` makes -1 of a number outside the cache, and names the request if
        // some row sees a token of that page in the tile: entries of pages
        // behind the sinks and before the window may have been taken back. (In
        // large pages a tile is walked only if a row sees some of it.)
        const int32_t *table = p.block_table + (int64_t)b * p.max_pages;
        auto load_page = [&](int k) {
            const int t = tile_t0(k) + part;
            return k < k_end && t < r.kv ? __ldg(table + (t >> p.page_shift)) : -1;
        };
        auto checked = [&](int k, int pg) {
            if ((uint32_t)pg < (uint32_t)p.n_pages) return pg;
            const int t = tile_t0(k) + part;
            if (k < k_end && t < r.kv && (!SMALL || pos0 - (t + 15) < w.reach || t < p.sinks)) paged_bad_request(p, b);
            return -1;
        };
        // Tile k's codes into the ring at `dst` as one copy group (empty past
        // the last tile). Tokens without a page copy page 0's codes, which
        // scales of 0 make nothing of; a page's tail past the sequence's end is in bounds.
        auto issue = [&](int k, bool value, int pg, uint32_t dst) {
            if (k < k_end) {
                const uint32_t vec = ((uint32_t)h << p.page_shift) + (uint32_t)((tile_t0(k) + part) & page_mask);
                const uint8_t *src = p.k_codes + ((uint64_t)(uint32_t)max(pg, 0) * page_vecs + vec) * DB + src0;
                if (value) src += v_minus_k;
                const uint32_t to = ring_a + dst + (value ? dst0 ^ swap : dst0);
#pragma unroll
                for (int i = 0; i < CPL; ++i)
                    copy16((value && SMALL ? to ^ (uint32_t)((i % CPT) * 16) : to) + (uint32_t)(i * STEP), src + i * STEP);
            }
            copy_commit();
        };
        // Whether some row sees token t. What the others hold must not matter: in
        // a tile that is walked for its neighbours they count as zero vectors. They
        // are the `hidden` tokens from p.sinks to the first row's window. A branch
        // skips their loads (loaded and then dropped they cost 3%).
        const uint32_t hidden = (uint32_t)(p.window ? max(max(pos0 - p.window + 1, 0) - p.sinks, 0) : 0);
        auto seen = [&](int t) { return t < r.kv && (uint32_t)(t - p.sinks) >= hidden; };
        // The scales and zeros of the lane's two tokens, (scale | zero << 16)
        // each; 0 where no row sees them and on bad pages.
        auto load_sz = [&](int k, int pg, uint32_t (&kw)[2], uint32_t (&vw)[2]) {
            const int t = tile_t0(k);
            kw[0] = kw[1] = vw[0] = vw[1] = 0u;
            if (pg < 0) return;
            const bool in0 = seen(t + tok0), in1 = seen(t + tok1);
            const uint32_t vec = ((uint32_t)h << p.page_shift) + (SMALL ? (uint32_t)((t + tok0) & page_mask) : (uint32_t)((t & page_mask) + tok0));
            const uint8_t *at = reinterpret_cast<const uint8_t *>(p.k_params) +
                                (((uint64_t)(uint32_t)pg * page_vecs + vec) << 2);
            if (SMALL) {
                const uint2 kk = __ldg(reinterpret_cast<const uint2 *>(at));
                const uint2 vv = __ldg(reinterpret_cast<const uint2 *>(at + vp_minus_kp));
                if (in0) kw[0] = kk.x, vw[0] = vv.x;
                if (in1) kw[1] = kk.y, vw[1] = vv.y;
            } else {
                if (in0) {
                    kw[0] = __ldg(reinterpret_cast<const uint32_t *>(at));
                    vw[0] = __ldg(reinterpret_cast<const uint32_t *>(at + vp_minus_kp));
                }
                if (in1) {
                    kw[1] = __ldg(reinterpret_cast<const uint32_t *>(at + 128));
                    vw[1] = __ldg(reinterpret_cast<const uint32_t *>(at + 128 + vp_minus_kp));
                }
            }
        };

        int k = k_begin + warp;
        uint32_t s0 = 0, s1 = TB, s2 = 2 * TB;   // ring places of this tile's keys and values and the next tile's keys
        int pgn;
        uint32_t kw[2] = {0u, 0u}, vw[2] = {0u, 0u};
        {
            int pg = load_page(k);
            pgn = load_page(k + kRwWarps);
            pg = checked(k, pg);
            pgn = checked(k + kRwWarps, pgn);
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
        //
        // The queries that meet high nibbles are divided by 16 as FP16. So that
        // small ones lose nothing by it, every column is first multiplied by a power of two
        // that brings its largest component to 2^15 or more (a subnormal one
        // to 2^5 times its units): what the division then rounds is below 2^-36 of
        // that component. The scores' exponentials take the power back.
        uint32_t qf[KS][2];
        float sq2[2], cs[2];   // sum of dims, for the zero points, and 2^-k, of columns 2 tig, 2 tig + 1
        {
            const int col = col0 + gid, i0 = (col * w.g_inv) >> 16;   // i0 = col / G
            const __half *qrow = p.q + (int64_t)(r.row0 + i0) * p.q_stride +
                                 (int64_t)(h * p.G + col - i0 * p.G) * D + tig * (D / 4);
            uint4 u[KW];
            __half2 top = __floats2half2_rn(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                u[i] = make_uint4(0u, 0u, 0u, 0u);
                if (gid < cols) u[i] = __ldg(reinterpret_cast<const uint4 *>(qrow + 8 * i));
                const uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&uw[e])));
            }
            uint32_t tb = half2_bits(top);
            tb = max(tb & 0xFFFFu, tb >> 16);   // FP16 bits of values >= 0 are ordered
            tb = max(tb, __shfl_xor_sync(0xffffffffu, tb, 1));
            tb = max(tb, __shfl_xor_sync(0xffffffffu, tb, 2));
            const int k2 = tb >= 0x7C00u ? 0 : 30 - max((int)(tb >> 10), 1);   // 2^k2 in two factors that FP16 holds
            const __half2 up0 = __float2half2_rn(__int_as_float((127 + min(k2, 15)) << 23));
            const __half2 up1 = __float2half2_rn(__int_as_float((127 + max(k2 - 15, 0)) << 23));
            const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 q2 = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&uw[e]), up0), up1);
                    uw[e] = half2_bits(q2);
                    const float2 f = __half22float2(q2);
                    sq += f.x + f.y;
                }
                qf[2 * i][0] = __byte_perm(uw[0], uw[2], 0x5410);
                qf[2 * i][1] = __byte_perm(uw[1], uw[3], 0x5410);
                // High nibbles enter 16 times too large.
                const uint32_t h0 = __byte_perm(uw[0], uw[2], 0x7632), h1 = __byte_perm(uw[1], uw[3], 0x7632);
                qf[2 * i + 1][0] = half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&h0), sixteenth));
                qf[2 * i + 1][1] = half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&h1), sixteenth));
            }
            sq += __shfl_xor_sync(0xffffffffu, sq, 1);
            sq += __shfl_xor_sync(0xffffffffu, sq, 2);            // column gid's
            const float down = __int_as_float((127 - k2) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sq2[c] = __shfl_sync(0xffffffffu, sq, 8 * tig + 4 * c);
                cs[c] = __shfl_sync(0xffffffffu, down, 8 * tig + 4 * c);
            }
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
            int pgnn = load_page(k + 2 * kRwWarps);
            uint32_t kwn[2] = {0u, 0u}, vwn[2] = {0u, 0u};
            if (k + kRwWarps < k_end) load_sz(k + kRwWarps, pgn, kwn, vwn);   // in flight while this tile is computed
            // Whether every column sees every token of the tile.
            const bool whole = t0 + kRwTile - 1 <= pos0 &&
                               (pos0 + r.n - 1 - t0 < w.reach || t0 + kRwTile <= p.sinks);
            // A written scale is finite, but for vectors that hold infinities. Such a
            // token makes the outputs of the rows that see it NaN: its score is NaN,
            // and its value's scale and zero finite, so that the weight 0 of the other rows
            // stays 0.
            const uint32_t sk = max(kw[0] & 0x7FFFu, kw[1] & 0x7FFFu);
            uint32_t sv = max(vw[0] & 0x7FFFu, vw[1] & 0x7FFFu);   // FP16 bits of values >= 0 are ordered
            const uint32_t zv = max(vw[0] & 0x7FFFFFFFu, vw[1] & 0x7FFFFFFFu);
            if (__any_sync(0xffffffffu, max(sk, sv) >= 0x7C00u || zv >= 0x7C000000u)) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (max(kw[i] & 0x7FFFu, vw[i] & 0x7FFFu) >= 0x7C00u || (vw[i] & 0x7FFFFFFFu) >= 0x7C000000u)
                        kw[i] = 0x7E00u, vw[i] = 0u;
                sv = max(vw[0] & 0x7FFFu, vw[1] & 0x7FFFu);
            }
            // The tile's largest value scale, and the tokens' factors for everyone.
            sv = __reduce_max_sync(0xffffffffu, sv);
            const int ebn = max(eb, (int)(__float_as_uint(half_lo(sv)) >> 23));
            const float ef = __int_as_float((262 - ebn) << 23);   // 2^(8 - E)
            __syncwarp();   // every lane is done with the last tile's factors
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = i ? tok1 : tok0;
                const float s = half_lo(kw[i]) * p.qscale;
                kf_s[warp][t] = make_float2(s * 0x1p24f, -__half2float(half_hi(kw[i])) * s);
                vf_s[warp][t] = half_lo(vw[i]) * ef;
                vz_s[warp][t] = half_hi(vw[i]);
            }
            copy_wait<2>();   // this tile's keys have landed
            __syncwarp();
            // 1. Scores (tokens x columns) of the tile's four 16-token steps:
            // s c (2^24 acc - z sum(q)), times the column's 2^k.
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
                        if (!(d >= 0 && (d < w.reach || t < p.sinks))) sc[j][c] = -INFINITY;
                    }
            }
            __syncwarp();   // every lane is done with the keys: the next tile's values take their place
            issue(k + kRwWarps, true, pgn, s0);
            // 2. Online softmax over the whole tile. The running maximum
            // starts at a finite value below every score, so a column that
            // sees nothing keeps p = 2^-inf = 0.
            float mx[2] = {-INFINITY, -INFINITY};
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
            mx[0] *= cs[0];
            mx[1] *= cs[1];
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
                    pr[c] = ex2_approx(fmaf(sc[j][c], cs[c & 1], -m2[c & 1]));
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
            pgnn = checked(k + 2 * kRwWarps, pgnn);
            issue(k + 2 * kRwWarps, false, pgnn, s1);
            const uint32_t s = s0;
            s0 = s2, s2 = s1, s1 = s;
            kw[0] = kwn[0], kw[1] = kwn[1], vw[0] = vwn[0], vw[1] = vwn[1];
            pgn = pgnn;
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
        __syncthreads();   // (and seg_s is written)
        const RowsSegment seg = seg_s;
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
            if (g < seg.cols) {
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
        // Four neighbouring dims per thread, the warps in order.
        auto warps_sum = [&](int i) {
            float4 sum = *reinterpret_cast<const float4 *>(ow + 4 * i);
#pragma unroll
            for (int x = 1; x < kRwWarps; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(ow + x * kRowsCols * D + 4 * i);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            return sum;
        };
        // A sum of 0 is that of a row which sees nothing; one that is no number (a
        // query or a visible key was none) makes the outputs none.
        auto store_out = [&](int i, const float4 &v, float L) {
            const int c = seg.col0 + 4 * i / D, i0 = (c * w.g_inv) >> 16;   // i0 = c / G
            const float x[4] = {v.x, v.y, v.z, v.w};
            uint32_t h2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                h2[e] = half2_bits(L == 0.0f ? __floats2half2_rn(0.0f, 0.0f) : __floats2half2_rn(x[2 * e] / L, x[2 * e + 1] / L));
            *reinterpret_cast<uint2 *>(p.out + (int64_t)(seg.row0 + i0) * p.out_stride +
                                       (int64_t)(seg.h * p.G + c - i0 * p.G) * D + 4 * i % D) = make_uint2(h2[0], h2[1]);
        };
        if (seg.nsplit == 0) {   // the start of an item whose rounds lie behind this CTA's
        } else if (seg.nsplit == 1) {
            for (int i = tid; i < seg.cols * (D / 4); i += kRwThreads) store_out(i, warps_sum(i), lc[4 * i / D]);
        } else {
            // Store this segment's unnormalised sums with its maxima and
            // weights, arrive, and let the last arriver combine. A CTA has
            // two slots: for an item that began before it, and for one that ends behind it.
            const int c0 = (int)blockIdx.x - seg.before;
            float *part = w.part + (int64_t)(2 * blockIdx.x + (seg.before ? 0 : 1)) * PSZ;
            for (int i = tid; i < seg.cols * (D / 4); i += kRwThreads) reinterpret_cast<float4 *>(part)[i] = warps_sum(i);
            if (tid < kRowsCols) {
                part[kRowsCols * D + tid] = mc[tid];
                part[kRowsCols * D + kRowsCols + tid] = lc[tid];
            }
            __syncthreads();   // every store of the CTA precedes the arrival (cumulative release)
            if (tid == 0) last_s = atom_add_acq_rel_gpu(w.counters + c0, 1) == seg.nsplit - 1;
            __syncthreads();
            if (last_s) {
                auto base = [&](int c) { return w.part + (int64_t)(2 * (c0 + c) + (c == 0 ? 1 : 0)) * PSZ; };
                // Each segment's factor per column, 2^(its maximum - the
                // greatest), over the idle buffers.
                float *fs = reinterpret_cast<float *>(rw_smem);   // [seg.nsplit][kRowsCols]
                constexpr int per = kRwThreads / kRowsCols;
                const int g = tid % kRowsCols;
                float M = kNone;
#pragma unroll 4
                for (int c = tid / kRowsCols; c < seg.nsplit; c += per) {
                    const float m = __ldcg(base(c) + kRowsCols * D + g);
                    fs[c * kRowsCols + g] = m;
                    M = fmaxf(M, m);
                }
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
                if (lane < kRowsCols) mw[warp][lane] = M;
                __syncthreads();
                M = fmaxf(fmaxf(mw[0][g], mw[1][g]), fmaxf(mw[2][g], mw[3][g]));
                float L = 0.0f;
#pragma unroll 4
                for (int c = tid / kRowsCols; c < seg.nsplit; c += per) {
                    const float f = exp2f(fs[c * kRowsCols + g] - M);
                    fs[c * kRowsCols + g] = f;
                    L = fmaf(f, __ldcg(base(c) + kRowsCols * D + kRowsCols + g), L);
                }
                L += __shfl_xor_sync(0xffffffffu, L, 8);
                L += __shfl_xor_sync(0xffffffffu, L, 16);
                if (lane < kRowsCols) lw[warp][lane] = L;
                __syncthreads();
                for (int i = tid; i < seg.cols * (D / 4); i += kRwThreads) {
                    const int col = 4 * i / D;
                    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int c = 0; c < seg.nsplit; ++c) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(base(c)) + i);
                        const float f = fs[c * kRowsCols + col];
                        O.x = fmaf(f, v.x, O.x), O.y = fmaf(f, v.y, O.y), O.z = fmaf(f, v.z, O.z), O.w = fmaf(f, v.w, O.w);
                    }
                    store_out(i, O, (lw[0][col] + lw[1][col]) + (lw[2][col] + lw[3][col]));
                }
                if (tid == 0) w.counters[c0] = 0;   // nobody arrives on it again in this call
            }
        }
        __syncthreads();   // nobody reads the segment any more
        if (tid == 0) {
            RowsWork &wk = work_s;
            wk.done += seg.count;
            if (wk.done < wk.remaining) {   // a request that has rounds follows, if this one's items end
                wk.offset = 0;
                if (seg.last_item) {
                    wk.item = 0;
                    do ++wk.b;
                    while (wk.b + 1 < p.B && rows_rounds(p, wk.b) == 0);
                } else {
                    ++wk.item;
                }
            }
        }
        __syncthreads();
        if (work_s.done == work_s.remaining) return;
    }
}

template <int D, bool SMALL>
cudaError_t launch(const RowsParams &w, cudaStream_t stream) {
    // Per warp, three 64-token tiles of codes, then the P tiles (1 KB per
    // warp): 52 KB at D = 128, four CTAs per SM.
    constexpr int smem = kRwWarps * 3 * kRwTile * D / 2 + kRwWarps * kRwTile * 8 * 2;
    if (smem > 40 * 1024) {
        static SmemOptIn opt_in;
        const cudaError_t e = opt_in.set(kv4_rows_kernel<D, SMALL>, smem);
        if (e != cudaSuccess) return e;
    }
    kv4_rows_kernel<D, SMALL><<<kRwResident, kRwThreads, smem, stream>>>(w);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const RowsParams &w, cudaStream_t stream) {
    return w.a.page_shift >= 6 ? launch<D, false>(w, stream) : launch<D, true>(w, stream);
}

}  // namespace

// Workspace: counters, partial results, the division of large batches.
size_t rows_workspace_bytes(int64_t B, int64_t D) {
    return (size_t)align256(4 * kRwResident) +
           (size_t)align256(8 * (int64_t)kRwResident * (kRowsCols * D + 2 * kRowsCols)) +
           (B > kRwWarpBatch ? (size_t)align256(8 * (B + 2)) : 0);
}

cudaError_t launch_paged_rows(const PagedAttnParams &p, int64_t D, void *ws, cudaStream_t stream) {
    RowsParams w;
    w.a = p;
    w.g_inv = (65536 + p.G - 1) / p.G;
    w.reach = p.window ? p.window : INT32_MAX;
    uint8_t *at = static_cast<uint8_t *>(ws);
    w.counters = reinterpret_cast<int32_t *>(at);
    at += align256(4 * kRwResident);
    w.part = reinterpret_cast<float *>(at);
    at += align256(8 * (int64_t)kRwResident * (kRowsCols * D + 2 * kRowsCols));
    w.first = nullptr;
    if (p.B > kRwWarpBatch) {
        w.first = reinterpret_cast<int64_t *>(at);
        kv4_rows_division_kernel<<<1, kDivThreads, 0, stream>>>(p, reinterpret_cast<int64_t *>(at));
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return D == 128 ? launch<128>(w, stream) : launch<64>(w, stream);
}

}  // namespace qoq
