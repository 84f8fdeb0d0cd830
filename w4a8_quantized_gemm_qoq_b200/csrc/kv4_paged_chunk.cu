// Paged KV4 attention for requests with many rows (prompts, chunks of them,
// long drafts) on the 5th-generation tensor cores.
//
// The work is 4 D flops per (query head, visible key). A CTA takes up to 256
// (row, head) pairs of one request and KV head, as two tiles of 128 rows, and
// walks the request's visible keys 128 at a time:
//   S = Q . C_K^T      tcgen05.mma, both operands in shared memory, FP32 in TMEM
//   x = S s_K c, online softmax in FP32 (one thread per row), P = p s_V as FP16
//   O += P . C_V       tcgen05.mma, P in TMEM, FP32 accumulator in TMEM
// C = q - z are the zero-subtracted codes, small integers that FP16 holds
// exactly, so the only rounding before the output is that of P. Scales are per
// token: s_K multiplies columns of S, s_V columns of P.
//
// One warpgroup unpacks codes for both row tiles (each code is unpacked once
// per 256 rows; c | 0x6400 is the half 1024 + c and c << 4 | 0x5400 is 64 + c,
// so an AND-OR and a subtraction of 1024 + z or 64 + z give two codes), one
// thread issues the products, two warpgroups do the softmaxes, in turn with
// one another: while one row tile's softmax runs, the tensor core works on the
// other's. K and V tiles are written in one layout, [token][dim] rows of 128
// bytes with the 128-byte swizzle: K is read from it dims-major, V
// tokens-major, so neither is transposed. Within each group of 8 the dims are in the
// order that unpacking yields, 0 4 1 5 2 6 3 7; Q is stored in the same order and
// the output is put back when it is written.
//
// Per 128 keys and 256 rows the tensor core needs 2048 cycles and so does
// the exponential unit (16 a cycle and SM): the two bound the kernel together.
//
// Pieces: (request, KV head, 256-row tile) items, long ones first, each cut
// along the keys into equal parts when there are too few of them to fill the
// SMs; the parts leave FP32 partial results, which a second kernel joins.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kv4_mma.cuh"
#include "kv4_paged.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kChCtas = 148;         // one per SM
constexpr int kChKeys = 128;         // keys per step
constexpr int kChRows = 256;         // rows per item: two tiles of 128
constexpr int kChThreads = 512;      // softmax 0, softmax 1, unpack, issue (one warp of four)
constexpr int kChSlots = 2 * kChCtas;   // pieces of divided items
constexpr int kChOverhead = 3;       // cost of a piece beside its steps, in steps
constexpr float kChSlack = 6.0f;     // log2 by which scores may exceed the running maximum
constexpr int kDvThreads = 1024;

struct ChunkParams {
    PagedAttnParams a;
    int rows_limit;      // requests with at most so many (row, head) pairs per KV head belong to the few-rows kernel
    int slot_rows;       // rows of a partial result
    int32_t *division;   // start[B + 1], slot[B + 1], parts[B]: pieces before, divided pieces before, parts per item
    int32_t *slots;      // [kChSlots][4]: request, head, tile, parts of the item whose part 0 the slot holds (else parts 0)
    float *part;         // [kChSlots][slot_rows][D] outputs, then [kChSlots][slot_rows][2] (maximum, sum)
};

// The steps of a 256-row tile: sink steps [0, sinks), then [first, first + count - sinks).
struct ChunkSteps {
    int sinks, first, count;
};

struct ChunkPiece {
    int b, h, tile, part, parts;   // request, KV head, row tile, which of its parts
    int rows;                      // (row, head) pairs of the item
    int k0, k1;                    // its steps
    int slot;                      // of the partial result, or -1
    PagedRequest r;
    ChunkSteps st;
};

__device__ __forceinline__ int chunk_rows(const ChunkParams &w, const PagedRequest &r) {
    const int rows = r.n * w.a.G;
    return r.n > w.a.max_new || rows <= w.rows_limit ? 0 : rows;
}

__device__ __forceinline__ ChunkSteps chunk_steps(const PagedAttnParams &p, const PagedRequest &r, int tile) {
    const int last = min((tile + 1) * kChRows, r.n * p.G) - 1;
    const int p0 = r.kv - r.n + tile * kChRows / p.G, p1 = r.kv - r.n + last / p.G;   // first and last position
    const int w0 = p.window ? max(0, p0 - p.window + 1) : 0;
    ChunkSteps s;
    s.first = w0 / kChKeys;
    s.sinks = p.window ? min((min(p.sinks, w0) + kChKeys - 1) / kChKeys, s.first) : 0;
    s.count = p1 < 0 ? 0 : s.sinks + p1 / kChKeys + 1 - s.first;
    if (s.count == 0) s.sinks = 0;
    return s;
}

// The longest item of a request, in steps (its last tile sees the most keys,
// or with a window as many as any), and its items.
__device__ __forceinline__ void chunk_request(const ChunkParams &w, int b, int &items, int &longest, int &shortest) {
    const PagedRequest r = paged_request(w.a, b);
    const int rows = chunk_rows(w, r);
    const int tiles = (rows + kChRows - 1) / kChRows;
    items = tiles * w.a.Hkv;
    longest = shortest = 0;
    if (tiles) {
        longest = max(1, chunk_steps(w.a, r, tiles - 1).count);
        shortest = max(1, min(longest, chunk_steps(w.a, r, 0).count));
    }
}

__device__ __forceinline__ int64_t block_sum64(int64_t v, int64_t *red) {
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

// How the batch is divided, by one CTA. Undivided, the items run in
// ceil(items / SMs) rounds of their average length; cut into parts of at most S
// steps they run in more rounds of shorter parts. The cheapest of a few S is
// taken, among those whose divided pieces fit the slots.
__global__ void __launch_bounds__(kDvThreads) kv4_chunk_division_kernel(const __grid_constant__ ChunkParams w) {
    __shared__ int64_t red[32];
    __shared__ int red0[32], red1[32];
    const PagedAttnParams &p = w.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t items = 0, steps = 0;
    for (int b = threadIdx.x; b < p.B; b += kDvThreads) {
        int n, hi, lo;
        chunk_request(w, b, n, hi, lo);
        items += n;
        steps += (int64_t)n * (hi + lo) / 2;
        if (paged_request(p, b).n > p.max_new) paged_bad_request(p, b);
    }
    items = block_sum64(items, red);
    steps = block_sum64(steps, red);
    int64_t S = INT32_MAX;
    if (items > 0 && items <= 4 * kChCtas) {
        int64_t best = (items + kChCtas - 1) / kChCtas * (steps + items * kChOverhead) / items;
        for (int c = 0; c < 6; ++c) {
            // Parts of 1 / m of an SM's share, and a little more.
            const int64_t m = 1 + c / 2, x = (steps + kChCtas * m - 1) / (kChCtas * m) * (c % 2 ? 9 : 8) / 8 + (c % 2);
            if (x < 1) continue;
            int64_t n = 0, cut = 0;
            for (int b = threadIdx.x; b < p.B; b += kDvThreads) {
                int k, hi, lo;
                chunk_request(w, b, k, hi, lo);
                const int64_t parts = (hi + x - 1) / x;
                n += parts * k;
                cut += parts > 1 ? parts * k : 0;
            }
            n = block_sum64(n, red);
            cut = block_sum64(cut, red);
            // A cut piece also writes its rows as FP32 and has them read again.
            const int64_t cost = (n + kChCtas - 1) / kChCtas * (steps + n * kChOverhead + cut) / n;
            if (cut <= kChSlots && cost < best) best = cost, S = x;
        }
    }
    int base0 = 0, base1 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kDvThreads) {
        const int b = b0 + threadIdx.x;
        int k = 0, hi = 0, lo = 0;
        if (b < p.B) chunk_request(w, b, k, hi, lo);
        const int parts = max(1, (int)((hi + S - 1) / S));
        const int v0 = k * parts, v1 = parts > 1 ? v0 : 0;
        int i0 = v0, i1 = v1;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int u0 = __shfl_up_sync(0xffffffffu, i0, s), u1 = __shfl_up_sync(0xffffffffu, i1, s);
            if (lane >= s) i0 += u0, i1 += u1;
        }
        __syncthreads();
        if (lane == 31) red0[warp] = i0, red1[warp] = i1;
        __syncthreads();
        int o0 = base0, o1 = base1;
        for (int x = 0; x < kDvThreads / 32; ++x) {
            if (x < warp) o0 += red0[x], o1 += red1[x];
            base0 += red0[x], base1 += red1[x];
        }
        if (b < p.B) {
            w.division[b] = o0 + i0 - v0;
            w.division[p.B + 1 + b] = o1 + i1 - v1;
            w.division[2 * p.B + 2 + b] = parts;
        }
    }
    if (threadIdx.x == 0) w.division[p.B] = base0, w.division[2 * p.B + 1] = base1;
}

// ------------------------------------------------------------ tensor cores

// kind::f16: FP16 operands, FP32 accumulator; b_mn: B is stored with its N
// index contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Shared-memory descriptor of an operand whose M or N index is contiguous:
// 128-byte swizzle, blocks of 64 (contiguous) x 8 elements; `panel` bytes to the
// next 64 along the contiguous index, 1024 to the next 8 along the other.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t panel) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(panel >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    __syncwarp();   // warp-collective (.sync.aligned)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return half2_bits(r);
}

// ------------------------------------------------------------ shared memory

template <int D>
struct ChunkSmem {
    static constexpr int DB = D / 2;
    static constexpr int kPanel = kChKeys * 128;            // 64 dims of 128 tokens (or rows), FP16
    static constexpr int kTile = (D / 64) * kPanel;         // one Q, K or V tile
    static constexpr int kCodes = kChKeys * DB;             // one tile's codes
    static constexpr int kRing = 3;                         // code tiles in flight
    static constexpr int kQ = 0;                            // two tiles
    static constexpr int kK = kQ + 2 * kTile;               // two stages
    static constexpr int kV = kK + 2 * kTile;               // two stages
    static constexpr int kC = kV + 2 * kTile;               // code ring
    static constexpr int kF = kC + kRing * kCodes;          // token factors: 4 x (128 K, 128 V) floats
    static constexpr int kZ = kF + 4 * 2 * kChKeys * 4;     // zeros of the tile in work: 128 K, 128 V words
    static constexpr int kEnd = kZ + 2 * kChKeys * 4;
    static constexpr int kBytes = kEnd + 1024;              // the base is rounded up to 1024
};

struct ChunkBars {
    uint64_t q, k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], drain;
};

enum ChunkSite : int {
    kSiteChunkQ = 20,       // issuer waiting for the queries
    kSiteChunkK = 21,       // issuer waiting for keys
    kSiteChunkV = 22,       // issuer waiting for values
    kSiteChunkP = 23,       // issuer waiting for weights
    kSiteChunkS = 24,       // softmax waiting for scores
    kSiteChunkO = 25,       // softmax waiting for the output
    kSiteChunkFree = 26,    // unpacking, waiting for a free stage
};

// wait_bounded with one answer for the warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Watchdog &wd, int site, int detail) {
    const bool ok = wait_bounded(bar, parity, wd, site, detail);
    return __all_sync(0xffffffffu, ok);
}

template <int D>
__global__ void __launch_bounds__(kChThreads, 1) kv4_chunk_kernel(const __grid_constant__ ChunkParams w) {
    using L = ChunkSmem<D>;
    constexpr int DB = D / 2;
    constexpr int CPT = DB / 16;                 // 16-byte code chunks per token
    constexpr int CPL = kChKeys * CPT / 128;     // chunks per unpacking thread and tile
    constexpr uint32_t kColS = 0, kColO = 256;   // TMEM: S0, S1 (P in their first halves), O0, O1
    constexpr float kNone = -1e30f;
    const PagedAttnParams &p = w.a;
    extern __shared__ uint8_t ch_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ch_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ ChunkBars bars;
    __shared__ uint32_t tmem_s;
    __shared__ volatile int abort_s;
    __shared__ float es_s[4], unit_s[4];   // per step (mod 4): 2^(E_old - E_new), 2^(E_new - 8)
    __shared__ uint32_t emax_s[2][4];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;
    const Watchdog wd{&abort_s, p.status};
    if (tid == 0) {
        abort_s = 0;
        mbar_init(&bars.q, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], 128);
            mbar_init(&bars.k_free[i], 1);
            mbar_init(&bars.v_full[i], 128);
            mbar_init(&bars.v_free[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 128);
            mbar_init(&bars.o_full[i], 1);
        }
        mbar_init(&bars.drain, 1);
        mbar_fence_init();
    }
    if (warp == 12) {
        tmem_alloc(&tmem_s, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    const uint32_t base = smem_u32(smem);
    float *factors = reinterpret_cast<float *>(smem + L::kF);

    const int pieces = w.division[p.B];
    // What this CTA's earlier pieces used of each barrier: steps, steps with a
    // second row tile, pieces, pieces with steps, those with a second row tile.
    uint32_t step_at = 0, step1_at = 0, piece_at = 0, out_at = 0, out1_at = 0;

    auto run_piece = [&](int piece, auto role) {
        int lo = 0, hi = p.B - 1;   // the last request that starts at or before the piece
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (w.division[mid] <= piece) lo = mid;
            else hi = mid - 1;
        }
        ChunkPiece c;
        c.b = lo;
        c.parts = w.division[2 * p.B + 2 + lo];
        c.r = paged_request(p, lo);
        const int rest = piece - w.division[lo], tiles = (c.r.n * p.G + kChRows - 1) / kChRows;
        // Long items first: the last tile's parts of every head, then the tile before.
        const int per_tile = c.parts * p.Hkv;
        c.tile = tiles - 1 - rest / per_tile;
        const int in_tile = rest % per_tile;
        c.h = in_tile / c.parts;
        c.part = in_tile - c.h * c.parts;
        c.rows = min(c.r.n * p.G - c.tile * kChRows, kChRows);
        c.st = chunk_steps(p, c.r, c.tile);
        const int each = c.st.count / c.parts, extra = c.st.count - each * c.parts;
        c.k0 = c.part * each + min(c.part, extra);
        c.k1 = c.k0 + each + (c.part < extra ? 1 : 0);
        c.slot = c.parts > 1 ? w.division[p.B + 1 + lo] + rest : -1;
        role(c);
        const uint32_t steps = (uint32_t)(c.k1 - c.k0), two = c.rows > 128 ? 1 : 0;
        step_at += steps;
        step1_at += two * steps;
        ++piece_at;
        out_at += steps > 0;
        out1_at += two & (steps > 0);
    };
    // Pieces in turn, forth and back over the CTAs: the lengths fall along the list.
    auto walk = [&](auto role) {
        for (int round = 0;; ++round) {
            const int piece = round * (int)gridDim.x + (round & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
            if (round * (int)gridDim.x >= pieces) break;
            if (piece < pieces) run_piece(piece, role);
            __syncthreads();   // every role is done with the piece
            if (abort_s) break;
        }
    };
    auto key_of = [&](const ChunkSteps &st, int k) {
        return (k < st.sinks ? k : st.first + (k - st.sinks)) * kChKeys;
    };

    if (wg < 2) {
        // ---------------------------------------------------------- softmax
        regs_inc<192>();
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's TMEM lanes
        const uint32_t ts = tmem + kColS + 128u * wg + lanes, to = tmem + kColO + (uint32_t)(D * wg) + lanes;
        const int row = tid & 127;
        walk([&](const ChunkPiece &c) {
            const PagedRequest &r = c.r;
            const int h = c.h, tile = c.tile, rows = c.rows, k0 = c.k0, k1 = c.k1, slot = c.slot;
            const bool active = wg * 128 < rows;
            const int pair = tile * kChRows + wg * 128 + row;            // (token, head) pair of the request
            const bool in = wg * 128 + row < rows;
            const int token = pair / p.G, head = h * p.G + (pair - token * p.G);
            // The queries, dims in unpacking order, 128-byte swizzle.
            {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(r.row0 + token) * p.q_stride +
                                                                   (int64_t)head * D);
                const uint32_t dst = base + L::kQ + (uint32_t)(wg * L::kTile + row * 128);
                if (active) {
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        uint4 u = make_uint4(0u, 0u, 0u, 0u);
                        if (in) u = __ldg(src + x);
                        sts128(dst + (uint32_t)((x >> 3) * L::kPanel + (((x & 7) ^ (row & 7)) << 4)),
                               __byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                               __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars.q);
            }
            if (!active) return;
            const int pos = r.kv - r.n + token;
            const int pos_lo = r.kv - r.n + (tile * kChRows + wg * 128) / p.G;
            const int pos_hi = r.kv - r.n + (tile * kChRows + min(wg * 128 + 128, rows) - 1) / p.G;
            float m = kNone, l = 0.0f, unit = 0.0f;
            for (int k = k0; k < k1; ++k) {
                const uint32_t s = step_at + (uint32_t)(k - k0);
                const uint32_t si = wg ? step1_at + (uint32_t)(k - k0) : s;
                const int t0 = key_of(c.st, k);
                if (!warp_wait(&bars.s_full[wg], si & 1, wd, kSiteChunkS, (int)s)) return;
                tc_fence_after();
                const float *kf = factors + (s & 3) * 2 * kChKeys, *vf = kf + kChKeys;
                float x[kChKeys];
                float mx = m;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t raw[32];
                    tmem_ld32_wait(ts + 32u * q, raw);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(kf + 32 * q + i);
                        x[32 * q + i] = __uint_as_float(raw[i]) * f.x;
                        x[32 * q + i + 1] = __uint_as_float(raw[i + 1]) * f.y;
                        x[32 * q + i + 2] = __uint_as_float(raw[i + 2]) * f.z;
                        x[32 * q + i + 3] = __uint_as_float(raw[i + 3]) * f.w;
                    }
                }
                const bool whole = t0 + kChKeys - 1 <= pos_lo &&
                                   (p.window == 0 || pos_hi - t0 < p.window || t0 + kChKeys <= p.sinks);
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < kChKeys; ++i) {
                        const int d = pos - t0 - i;
                        if (!(d >= 0 && (p.window == 0 || d < p.window || t0 + i < p.sinks))) x[i] = -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < kChKeys; i += 2) mx = fmaxf(mx, fmaxf(x[i], x[i + 1]));
                // A maximum that grew by much, or larger value scales:
                // the output accumulated so far changes its unit.
                const float es = es_s[s & 3];
                unit = unit_s[s & 3];
                const bool raise = mx > m + kChSlack;
                if (__any_sync(0xffffffffu, raise) || es != 1.0f) {
                    const float mn = raise ? mx : m, al = ex2_approx(m - mn);
                    m = mn;
                    l *= al;
                    if (k > k0) {
                        const float f = al * es;
#pragma unroll
                        for (int q = 0; q < D; q += 32) {
                            uint32_t o[32];
                            tmem_ld32_wait(to + q, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32_wait(to + q, o);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(vf + 32 * q + i);
                        const float a0 = ex2_approx(x[32 * q + i] - m), a1 = ex2_approx(x[32 * q + i + 1] - m);
                        const float a2 = ex2_approx(x[32 * q + i + 2] - m), a3 = ex2_approx(x[32 * q + i + 3] - m);
                        l += (a0 + a1) + (a2 + a3);
                        pk[i / 2] = half2_bits(__floats2half2_rn(a0 * f.x, a1 * f.y));
                        pk[i / 2 + 1] = half2_bits(__floats2half2_rn(a2 * f.z, a3 * f.w));
                    }
                    tmem_st16(ts + 16u * q, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars.p_full[wg]);
            }
            if (k1 > k0) {
                if (!warp_wait(&bars.o_full[wg], (wg ? out1_at : out_at) & 1, wd, kSiteChunkO, (int)piece_at)) return;
                tc_fence_after();
            }
            const float f = slot >= 0 ? unit : l > 0.0f ? unit / l : 0.0f;
            __half *out = p.out + (int64_t)(r.row0 + token) * p.out_stride + (int64_t)head * D;
            float *part_o = w.part + ((int64_t)slot * w.slot_rows + wg * 128 + row) * D;
#pragma unroll
            for (int q = 0; q < D; q += 32) {
                uint32_t o[32];
                if (k1 > k0) tmem_ld32_wait(to + q, o);
                else
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                if (!in) continue;
#pragma unroll
                for (int g = 0; g < 32; g += 8) {   // dims 0 4 1 5 2 6 3 7
                    const float d0 = __uint_as_float(o[g]) * f, d4 = __uint_as_float(o[g + 1]) * f;
                    const float d1 = __uint_as_float(o[g + 2]) * f, d5 = __uint_as_float(o[g + 3]) * f;
                    const float d2 = __uint_as_float(o[g + 4]) * f, d6 = __uint_as_float(o[g + 5]) * f;
                    const float d3 = __uint_as_float(o[g + 6]) * f, d7 = __uint_as_float(o[g + 7]) * f;
                    if (slot >= 0) {
                        reinterpret_cast<float4 *>(part_o + q + g)[0] = make_float4(d0, d1, d2, d3);
                        reinterpret_cast<float4 *>(part_o + q + g)[1] = make_float4(d4, d5, d6, d7);
                    } else {
                        *reinterpret_cast<uint4 *>(out + q + g) =
                            make_uint4(half2_bits(__floats2half2_rn(d0, d1)), half2_bits(__floats2half2_rn(d2, d3)),
                                       half2_bits(__floats2half2_rn(d4, d5)), half2_bits(__floats2half2_rn(d6, d7)));
                    }
                }
            }
            if (slot >= 0) {
                if (in) {
                    float2 *ml = reinterpret_cast<float2 *>(w.part + (int64_t)kChSlots * w.slot_rows * D);
                    ml[(int64_t)slot * w.slot_rows + wg * 128 + row] = make_float2(m, l);
                }
                if (wg == 0 && row == 0)
                    *reinterpret_cast<int4 *>(w.slots + 4 * slot) = make_int4(c.b, h, tile, c.part == 0 ? c.parts : 0);
            }
            tc_fence_before();   // the next piece's products come after these reads
        });
    } else if (wg == 2) {
        // ---------------------------------------------------------- unpack
        regs_dec<88>();
        const int t = tid & 127;
        const int tk = t / CPT, j = t % CPT;       // chunk j of tokens tk + (128 / CPT) i
        const int page_mask = (1 << p.page_shift) - 1;
        const uint32_t page_vecs = (uint32_t)p.Hkv << p.page_shift;
        float *zf = reinterpret_cast<float *>(smem + L::kZ);
        uint32_t *zeros = reinterpret_cast<uint32_t *>(zf);
        walk([&](const ChunkPiece &pc) {
            const PagedRequest &r = pc.r;
            const int b = pc.b, h = pc.h, k0 = pc.k0, k1 = pc.k1;
            const int32_t *table = p.block_table + (int64_t)b * p.max_pages;
            const uint8_t *kc = p.k_codes + ((int64_t)h << p.page_shift) * DB + j * 16;
            const uint8_t *vc = p.v_codes + ((int64_t)h << p.page_shift) * DB + j * 16;
            auto page_of = [&](int key) {   // -1 past the end and outside the cache
                int page = -1;
                if (key < r.kv) {
                    page = __ldg(table + (key >> p.page_shift));
                    if ((uint32_t)page >= (uint32_t)p.n_pages) {
                        paged_bad_request(p, b);
                        page = -1;
                    }
                }
                return page;
            };
            // One tile's codes of one tensor, each thread its own chunks to
            // its own places; parts without a page copy page 0's.
            uint32_t put = 0, get = 0;   // ring places
            auto fetch = [&](int half) {   // half steps: keys of step k0 + half / 2, then its values
                const int k = k0 + (half >> 1);
                if (k < k1) {
                    const int t0 = key_of(pc.st, k) + tk;
                    const uint8_t *c = half & 1 ? vc : kc;
                    const uint32_t dst = base + (uint32_t)(L::kC + t * 16) + put;
#pragma unroll
                    for (int i = 0; i < CPL; ++i) {
                        const int key = t0 + i * (128 / CPT);
                        const int page = max(page_of(key), 0);
                        copy16(dst + (uint32_t)(i * 2048), c + (uint64_t)(uint32_t)page * (page_vecs * DB) + (key & page_mask) * DB);
                    }
                }
                copy_commit();
                put = put + L::kCodes == L::kRing * L::kCodes ? 0 : put + L::kCodes;
            };
            auto load_sz = [&](int k, uint32_t &kw, uint32_t &vw) {   // token t's scale and zero
                kw = vw = 0u;
                if (k < k1) {
                    const int key = key_of(pc.st, k) + t;
                    const int page = page_of(key);
                    if (page >= 0) {
                        const uint64_t at = (uint64_t)(uint32_t)page * page_vecs + ((uint32_t)h << p.page_shift) + (key & page_mask);
                        kw = __ldg(reinterpret_cast<const uint32_t *>(p.k_params) + at);
                        vw = __ldg(reinterpret_cast<const uint32_t *>(p.v_params) + at);
                    }
                }
            };
            // Codes of the ring's next tile -> FP16 c - z in the stage at dst.
            auto unpack = [&](uint32_t dst, const uint32_t *z) {
                const uint32_t src = base + (uint32_t)(L::kC + t * 16) + get;
                get = get + L::kCodes == L::kRing * L::kCodes ? 0 : get + L::kCodes;
#pragma unroll
                for (int i = 0; i < CPL; ++i) {
                    const int token = tk + i * (128 / CPT);
                    const uint4 u = lds128(src + (uint32_t)(i * 2048));
                    const uint32_t zz = z[token];   // halves 1024 + z, 64 + z
                    const uint32_t z1 = __byte_perm(zz, zz, 0x1010), z2 = __byte_perm(zz, zz, 0x3232);
                    const uint32_t words[4] = {u.x, u.y, u.z, u.w};
                    const uint32_t row = dst + (uint32_t)(token * 128 + (j >> 1) * L::kPanel);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        // In an order in which 8 threads' stores touch every bank once.
                        const int e = x ^ (j & 2);
                        const uint32_t c = j & 2 ? words[x ^ 2] : words[x], c8 = c >> 8;
                        sts128(row + (uint32_t)(((4 * (j & 1) + e) ^ (token & 7)) << 4),
                               hsub2((c & 0x000F000Fu) | 0x64006400u, z1), hsub2((c & 0x00F000F0u) | 0x54005400u, z2),
                               hsub2((c8 & 0x000F000Fu) | 0x64006400u, z1), hsub2((c8 & 0x00F000F0u) | 0x54005400u, z2));
                    }
                }
            };
            uint32_t kw, vw;
            load_sz(k0, kw, vw);
            fetch(0);
            fetch(1);
            fetch(2);
            int eb = 103;   // 127 + the exponent of the largest value scale so far (scales >= 2^-24)
            for (int k = k0; k < k1; ++k) {
                const uint32_t s = step_at + (uint32_t)(k - k0), stage = s & 1;
                // The step's factors. A written scale is finite and a zero at
                // most 15; the bounds make a hidden token's values
                // so too, whatever it holds, so that its weight 0 stays 0.
                const uint32_t sv = min(vw & 0xFFFFu, 0x7BFFu);
                const float zk = fminf(fmaxf(__half2float(half_hi(kw)), 0.0f), 15.0f);
                const float zv = fminf(fmaxf(__half2float(half_hi(vw)), 0.0f), 15.0f);
                const uint32_t wmax = __reduce_max_sync(0xffffffffu, sv);
                if (lane == 0) emax_s[stage][warp & 3] = wmax;
                zeros[t] = half2_bits(__floats2half2_rn(1024.0f + zk, 64.0f + zk));
                zeros[kChKeys + t] = half2_bits(__floats2half2_rn(1024.0f + zv, 64.0f + zv));
                named_bar_sync(1, 128);
                const uint32_t top = max(max(emax_s[stage][0], emax_s[stage][1]), max(emax_s[stage][2], emax_s[stage][3]));
                const int ebn = max(eb, (int)(__float_as_uint(half_lo(top)) >> 23));
                float *kf = factors + (s & 3) * 2 * kChKeys;
                kf[t] = half_lo(kw) * p.qscale;
                kf[kChKeys + t] = half_lo(sv) * __int_as_float((262 - ebn) << 23);   // 2^(8 - E)
                if (t == 0) {
                    es_s[s & 3] = __int_as_float((127 + eb - ebn) << 23);
                    unit_s[s & 3] = __int_as_float((ebn - 8) << 23);
                }
                eb = ebn;
                load_sz(k + 1, kw, vw);
                const uint32_t freed = ((s >> 1) - 1) & 1;
                // Keys.
                bool ok = s < 2 || wait_bounded(&bars.k_free[stage], freed, wd, kSiteChunkFree, (int)s);
                copy_wait<2>();
                if (ok) {
                    unpack(base + L::kK + stage * L::kTile, zeros);
                    fence_proxy_async_smem();
                    mbar_arrive(&bars.k_full[stage]);
                }
                fetch(2 * (k - k0) + 3);
                // Values.
                ok = ok && (s < 2 || wait_bounded(&bars.v_free[stage], freed, wd, kSiteChunkFree, (int)s));
                copy_wait<2>();
                if (ok) {
                    unpack(base + L::kV + stage * L::kTile, zeros + kChKeys);
                    fence_proxy_async_smem();
                    mbar_arrive(&bars.v_full[stage]);
                }
                fetch(2 * (k - k0) + 4);
                if (named_bar_any(1, 128, !ok)) break;   // and the zeros are read
            }
            copy_wait<0>();
        });
    } else {
        // ---------------------------------------------------------- issue
        regs_dec<40>();
        walk([&](const ChunkPiece &c) {
            if (warp != 12) return;
            const int steps = c.k1 - c.k0;
            const bool two = c.rows > 128;
            constexpr uint32_t id_s = idesc_f16(128, kChKeys, false), id_o = idesc_f16(128, D, true);
            bool ok = warp_wait(&bars.q, piece_at & 1, wd, kSiteChunkQ, (int)piece_at);
            auto scores = [&](int i, uint32_t stage) {
                if (lane == 0) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t o = (uint32_t)((x >> 2) * L::kPanel + (x & 3) * 32);
                        mma_f16_ss(tmem + kColS + 128u * i, smem_desc_k_sw128(base + L::kQ + i * L::kTile + o),
                                   smem_desc_k_sw128(base + L::kK + stage * L::kTile + o), id_s, x > 0);
                    }
                    tc_commit(&bars.s_full[i]);
                }
            };
            auto values = [&](int i, uint32_t stage, bool first) {
                if (lane == 0) {
#pragma unroll
                    for (int x = 0; x < kChKeys / 16; ++x)
                        mma_f16_ts(tmem + kColO + (uint32_t)(D * i), tmem + kColS + 128u * i + 8u * x,
                                   smem_desc_mn_sw128(base + L::kV + stage * L::kTile + x * 2048, L::kPanel), id_o,
                                   !first || x > 0);
                }
            };
            auto commit = [&](uint64_t *bar) {
                if (lane == 0) tc_commit(bar);
            };
            if (ok && steps > 0) {
                const uint32_t s0 = step_at;
                ok = warp_wait(&bars.k_full[s0 & 1], (s0 >> 1) & 1, wd, kSiteChunkK, (int)s0);
                if (ok) {
                    tc_fence_after();
                    scores(0, s0 & 1);
                    if (two) scores(1, s0 & 1);
                    commit(&bars.k_free[s0 & 1]);
                }
                for (int k = 0; ok && k < steps; ++k) {
                    const uint32_t s = step_at + (uint32_t)k, stage = s & 1, next = stage ^ 1;
                    const bool more = k + 1 < steps;
                    if (!(ok = warp_wait(&bars.v_full[stage], (s >> 1) & 1, wd, kSiteChunkV, (int)s))) break;
                    if (!(ok = warp_wait(&bars.p_full[0], s & 1, wd, kSiteChunkP, (int)s))) break;
                    tc_fence_after();
                    values(0, stage, k == 0);
                    if (!more) commit(&bars.o_full[0]);
                    if (more) {
                        if (!(ok = warp_wait(&bars.k_full[next], ((s + 1) >> 1) & 1, wd, kSiteChunkK, (int)s + 1))) break;
                        tc_fence_after();
                        scores(0, next);
                    }
                    if (two) {
                        if (!(ok = warp_wait(&bars.p_full[1], (step1_at + (uint32_t)k) & 1, wd, kSiteChunkP, (int)s))) break;
                        tc_fence_after();
                        values(1, stage, k == 0);
                        if (!more) commit(&bars.o_full[1]);
                    }
                    commit(&bars.v_free[stage]);
                    if (more) {
                        if (two) scores(1, next);
                        commit(&bars.k_free[next]);
                    }
                }
            }
            if (!ok && lane == 0) {
                // Let the products in flight end before the memory is given back.
                tc_commit(&bars.drain);
                wait_drain(&bars.drain, 0, kWaitLimitNs);
            }
            __syncwarp();
        });
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

}  // namespace

namespace {

// Joins the parts of divided items: one warp per row, CTAs over (slot of a
// part 0, block of rows).
constexpr int kJoinRows = 16;

template <int D>
__global__ void __launch_bounds__(256) kv4_chunk_join_kernel(const __grid_constant__ ChunkParams w) {
    const PagedAttnParams &p = w.a;
    const int slot = blockIdx.x;
    if (slot >= w.division[2 * p.B + 1]) return;
    const int4 it = *reinterpret_cast<const int4 *>(w.slots + 4 * slot);   // request, head, tile, parts
    const int parts = it.w;
    if (parts == 0) return;
    const PagedRequest r = paged_request(p, it.x);
    const int rows = min(r.n * p.G - it.z * kChRows, kChRows);
    const int lane = threadIdx.x & 31;
    const float2 *ml = reinterpret_cast<const float2 *>(w.part + (int64_t)kChSlots * w.slot_rows * D);
    for (int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5); row < min(rows, (int)(blockIdx.y + 1) * kJoinRows); row += 8) {
        float m = -INFINITY, l = 0.0f, o[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = 0.0f;
        for (int i = 0; i < parts; ++i) m = fmaxf(m, ml[(int64_t)(slot + i) * w.slot_rows + row].x);
        for (int i = 0; i < parts; ++i) {
            const int64_t at = (int64_t)(slot + i) * w.slot_rows + row;
            const float2 x = ml[at];
            const float f = exp2f(x.x - m);
            l += f * x.y;
            const float *src = w.part + at * D + lane * (D / 32);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[e] = fmaf(f, src[e], o[e]);
        }
        const float f = l > 0.0f ? 1.0f / l : 0.0f;
        const int pair = it.z * kChRows + row, token = pair / p.G;
        __half2 *out = reinterpret_cast<__half2 *>(p.out + (int64_t)(r.row0 + token) * p.out_stride +
                                                   (int64_t)(it.y * p.G + pair - token * p.G) * D + lane * (D / 32));
#pragma unroll
        for (int e = 0; e < D / 32; e += 2) out[e / 2] = __floats2half2_rn(o[e] * f, o[e + 1] * f);
    }
}

int slot_rows(int64_t max_new, int64_t G) {
    const int64_t rows = max_new * G;
    return rows >= kChRows ? kChRows : (int)((rows + kJoinRows - 1) / kJoinRows * kJoinRows);
}

template <int D>
cudaError_t launch(const ChunkParams &w, cudaStream_t stream) {
    constexpr int smem = ChunkSmem<D>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kv4_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kv4_chunk_division_kernel<<<1, kDvThreads, 0, stream>>>(w);
    kv4_chunk_kernel<D><<<kChCtas, kChThreads, smem, stream>>>(w);
    kv4_chunk_join_kernel<D><<<dim3(kChSlots, (unsigned)(w.slot_rows / kJoinRows)), 256, 0, stream>>>(w);
    return cudaGetLastError();
}

}  // namespace

// Workspace: the division, the slots' items, the partial results.
size_t chunk_workspace_bytes(int64_t B, int64_t max_new, int64_t G, int64_t D) {
    return (size_t)align256(4 * (3 * B + 2)) + (size_t)align256(16 * kChSlots) +
           (size_t)align256((int64_t)4 * kChSlots * slot_rows(max_new, G) * (D + 2));
}

// Requests with more than rows_limit (row, head) pairs per KV head.
cudaError_t launch_paged_chunk(const PagedAttnParams &p, int64_t D, int rows_limit, int64_t max_new, void *ws,
                               cudaStream_t stream) {
    ChunkParams w;
    w.a = p;
    w.rows_limit = rows_limit;
    w.slot_rows = slot_rows(max_new, p.G);
    uint8_t *at = static_cast<uint8_t *>(ws);
    w.division = reinterpret_cast<int32_t *>(at);
    at += align256(4 * (3 * (int64_t)p.B + 2));
    w.slots = reinterpret_cast<int32_t *>(at);
    at += align256(16 * kChSlots);
    w.part = reinterpret_cast<float *>(at);
    return D == 128 ? launch<128>(w, stream) : launch<64>(w, stream);
}

}  // namespace qoq
