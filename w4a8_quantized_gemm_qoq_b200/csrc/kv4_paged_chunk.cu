// Paged KV4 attention for requests with many rows (prompts, chunks of them,
// long drafts) on the 5th-generation tensor cores.
//
// The work is 4 D flops per (query head, visible key). A CTA takes up to 256
// (row, head) pairs of one request and KV head, as two tiles of 128 rows, and
// walks the request's visible keys 128 at a time:
//   S = Q . C_K^T      tcgen05.mma, both operands in shared memory, FP32 in TMEM
//   x = S s_K c, online softmax in FP32 (a warp per 32 rows), P = p s_V as FP16
//   O += P . C_V       tcgen05.mma, P in TMEM, FP32 accumulator in TMEM
// C = q - z are the zero-subtracted codes, small integers that FP16 holds
// exactly, so the only rounding before the output is that of P. Scales are per
// token: s_K multiplies columns of S, s_V columns of P.
//
// One warpgroup unpacks the codes of K and V for both row tiles (each code is
// unpacked once per 256 rows; c | 0x6400 is the half 1024 + c and c << 4 | 0x5400 is 64 + c,
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
// the exponential unit (16 a cycle and SM): the two would bound the kernel
// together. Measured (32 query heads on 8, D 128): 2048 rows on 16384 tokens 727 us
// (709 TFLOP/s of 1614 that a large product reaches), a prompt of 4096 235 us
// (584). A step of 128 keys takes some 6800 cycles: a softmax 2400 alone and
// 4000 beside the other one, then about 1900 until the products of its row tile are
// through, since tensor memory holds two outputs and two score tiles and no third (P
// lies over S, so the next scores wait for this step's second product).
// Issue slots are 42% taken, the tensor core is busy 35% of the time:
// what bounds it is this chain. Slower than what is here, for the first of the
// two cases: steps of 64 keys (817 us), a block's scores computed ahead of the
// last block's weights (912, for want of registers), blocks of 16 keys (909) or
// votes on 64 (759), softmaxes made to take turns (836), weights handed over by
// halves of a step (778; by polling for whichever tile is ready 825), two unpacking
// warpgroups (771 when that was tried against 748); the others were tried against 723 to 728.
//
// Pieces: (request, KV head, 256-row tile) items, long ones first, each cut
// along the keys into equal parts when there are too few of them to fill the
// SMs; the parts leave FP32 partial results, which a second kernel joins.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kv4_mma.cuh"
#include "kv4_paged.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kChCtas = 148;         // one per SM
constexpr int kChKeys = 128;         // keys per step
constexpr int kChRows = 256;         // rows per item: two tiles of 128
constexpr int kChThreads = 512;      // warpgroups: softmax 0 and 1, unpack, issue (one of its warps)
constexpr int kChSlots = 2 * kChCtas;   // pieces of divided items
constexpr int kChOverhead = 3;       // cost of a piece beside its steps, in steps
// Registers per thread: the pool is 512 threads x 128, of which the roles take
// 256 x 176 + 128 x 104 + 128 x 56 = 65536 (184 / 104 / 40 spills in the issuing
// warp: 727 us for the first case above where this split took 723).
constexpr int kRegsSoftmax = 176, kRegsUnpack = 104, kRegsIssue = 56;
constexpr float kChSlack = 6.0f;     // log2 by which scores may exceed the running maximum
constexpr int kDvThreads = 1024;

struct ChunkParams {
    PagedAttnParams a;
    int slot_rows;       // rows of a partial result
    int32_t *division;   // by place in the order: start[B + 1], slot[B + 1] (pieces and divided pieces before),
                         // parts[B] (per item), request[B]
    int32_t *slots;      // [kChSlots][4]: request, head, tile, parts of the item whose part 0 the slot holds (else parts 0)
    float *part;         // [kChSlots][slot_rows][D] outputs, then [kChSlots][slot_rows][2] (maximum, sum)
};

// The steps of a 256-row tile: sink steps [0, sinks), then [first, first + count - sinks).
// Of their tokens some row sees those of [window, end) and the sinks before them.
struct ChunkSteps {
    int sinks, first, count;
    int window, end;
};

struct ChunkPiece {
    int b, h, tile, part, parts;   // request, KV head, row tile, which of its parts
    int rows;                      // (row, head) pairs of the item
    int k0, k1;                    // its steps
    int slot;                      // of the partial result, or -1
    PagedRequest r;
    ChunkSteps st;
};

// (row, head) pairs per KV head of a request for this kernel, else 0.
__device__ __forceinline__ int chunk_rows(const ChunkParams &w, const PagedRequest &r) {
    const int rows = r.n * w.a.G;
    return r.n > w.a.max_new || rows <= kRowsMax ? 0 : rows;
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
    s.window = w0;
    s.end = p1 + 1;
    return s;
}

// How the batch is divided, by one CTA. Undivided, the items run in
// ceil(items / SMs) rounds of their average length; cut into parts of at most S
// steps they run in more rounds of shorter parts. The cheapest of a few S is
// taken, among those whose divided pieces fit the slots. Requests are taken
// in the order of their longest items, so that the pieces' lengths fall along
// the list, which goes round the CTAs forth and back (32 requests of 1500 to 4500
// tokens, 20 rows each: 134 us, in the order given 178). The attention kernel
// waits for this one, so it is kept short: one reading of the lengths, one
// meeting for all sums (6 us for 16 requests; it runs beside the few-rows kernel).
constexpr int kSortBatch = 2048;   // largest batch that is ordered
constexpr int kCandidates = 6;

struct ChunkRequest {
    int items, longest, shortest;
};

__device__ __forceinline__ ChunkRequest chunk_request(const ChunkParams &w, int b) {
    const PagedRequest r = paged_request(w.a, b);
    if (r.n > w.a.max_new) paged_bad_request(w.a, b);
    const int rows = chunk_rows(w, r);
    const int tiles = (rows + kChRows - 1) / kChRows;
    ChunkRequest c = {tiles * w.a.Hkv, 0, 0};
    if (tiles) {
        c.longest = max(1, chunk_steps(w.a, r, tiles - 1).count);
        c.shortest = max(1, min(c.longest, chunk_steps(w.a, r, 0).count));
    }
    return c;
}

__global__ void __launch_bounds__(kDvThreads) kv4_chunk_division_kernel(const __grid_constant__ ChunkParams w) {
    __shared__ int order_s[kSortBatch], key_s[kSortBatch];
    __shared__ float items_s[32], steps_s[32];
    __shared__ float sums_s[2 * kCandidates][32];
    __shared__ int red0[32], red1[32];
    const PagedAttnParams &p = w.a;
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    auto warp_sum = [](float v) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        return v;
    };
    // The sums guide a choice and are kept in FP32; the slots' bound below holds
    // exactly, since whole numbers to 2^24 are exact.
    const bool sorted = p.B <= kSortBatch;
    const ChunkRequest mine = (int)threadIdx.x < p.B ? chunk_request(w, threadIdx.x) : ChunkRequest{0, 0, 0};
    float items = (float)mine.items, steps = 0.5f * (float)mine.items * (float)(mine.longest + mine.shortest);
    if (sorted && (int)threadIdx.x < p.B) key_s[threadIdx.x] = mine.longest;
    for (int b = threadIdx.x + blockDim.x; b < p.B; b += blockDim.x) {
        const ChunkRequest c = chunk_request(w, b);
        items += (float)c.items;
        steps += 0.5f * (float)c.items * (float)(c.longest + c.shortest);
        if (sorted) key_s[b] = c.longest;
    }
    items = warp_sum(items);
    steps = warp_sum(steps);
    if (lane == 0) items_s[warp] = items, steps_s[warp] = steps;
    __syncthreads();
    items = warp_sum(lane < warps ? items_s[lane] : 0.0f);
    steps = warp_sum(lane < warps ? steps_s[lane] : 0.0f);

    int S = INT32_MAX;
    if (items > 0.0f && items <= 4.0f * kChCtas) {
        // Parts of 1 / m of an SM's share, and of a little more.
        auto candidate = [&](int c) {
            return max(1, (int)(steps / (float)(kChCtas * (1 + c / 2)) * (c % 2 ? 1.125f : 1.0f)) + 1 + c % 2);
        };
        float n[2 * kCandidates];
#pragma unroll
        for (int c = 0; c < kCandidates; ++c) n[2 * c] = n[2 * c + 1] = 0.0f;
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const ChunkRequest r = b == (int)threadIdx.x ? mine : chunk_request(w, b);
#pragma unroll
            for (int c = 0; c < kCandidates; ++c) {
                const int x = candidate(c), parts = (r.longest + x - 1) / x;
                n[2 * c] += (float)parts * (float)r.items;
                n[2 * c + 1] += parts > 1 ? (float)parts * (float)r.items : 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < 2 * kCandidates; ++c) {
            const float v = warp_sum(n[c]);
            if (lane == 0) sums_s[c][warp] = v;
        }
        __syncthreads();
        float best = ceilf(items / kChCtas) * (steps / items + (float)kChOverhead);
#pragma unroll
        for (int c = 0; c < kCandidates; ++c) {
            const float all = warp_sum(lane < warps ? sums_s[2 * c][lane] : 0.0f);
            const float cut = warp_sum(lane < warps ? sums_s[2 * c + 1][lane] : 0.0f);
            // A cut piece also writes its rows as FP32 and has them read again, by
            // one more kernel: half a step on top of the estimate. Prompts of 300
            // and 500 tokens take 25 and 30 us uncut, as they then are, and 31 and 39
            // cut; with a whole step, 8 chunks of 200 to 500 tokens stay uncut
            // too, 112 us and not 105.
            const float cost = ceilf(all / kChCtas) * (steps + all * (float)kChOverhead + cut) / all + (cut > 0.0f ? 0.5f : 0.0f);
            if (cut <= (float)kChSlots && cost < best) best = cost, S = candidate(c);
        }
    }
    if (sorted) {
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const int key = key_s[b];
            int rank = 0;
            for (int x = 0; x < p.B; ++x) rank += key_s[x] > key || (key_s[x] == key && x < b);
            order_s[rank] = b;
        }
        __syncthreads();
    }
    int base0 = 0, base1 = 0;
    for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;   // place in the order
        const int request = b < p.B ? (sorted ? order_s[b] : b) : 0;
        const ChunkRequest r = b < p.B ? chunk_request(w, request) : ChunkRequest{0, 0, 0};
        const int parts = S == INT32_MAX ? 1 : max(1, (r.longest + S - 1) / S);
        const int v0 = r.items * parts, v1 = parts > 1 ? v0 : 0;
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
        for (int x = 0; x < warps; ++x) {
            if (x < warp) o0 += red0[x], o1 += red1[x];
            base0 += red0[x], base1 += red1[x];
        }
        if (b < p.B) {
            w.division[b] = o0 + i0 - v0;
            w.division[p.B + 1 + b] = o1 + i1 - v1;
            w.division[2 * p.B + 2 + b] = parts;
            w.division[3 * p.B + 2 + b] = request;
        }
    }
    if (threadIdx.x == 0) w.division[p.B] = base0, w.division[2 * p.B + 1] = base1;
    griddep_wait();   // the few-rows kernel: what waits for this one waits for both
}

// ------------------------------------------------------------ tensor cores

// kind::f16: FP16 operands, FP32 accumulator; b_mn: B is stored with its N
// index contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// Shared-memory operand descriptors with the 128-byte swizzle, as their low
// words (start address, and the stride between 64-element panels for operands
// whose M or N index is contiguous); the high word is the same for all: 1024
// bytes between groups of 8 rows, version 1, swizzle 2.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t panel) {
    return ((saddr & 0x3FFFFu) >> 4) | ((panel >> 4) << 16);
}

// D (+)= A . B over 64 of the inner index, both operands in shared memory with
// that index contiguous: four products of 16, 32 bytes apart in a swizzled row.
// The descriptors are put together inside, so that they are not all kept in
// registers across the loop.
__device__ __forceinline__ void mma4_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 u, v;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 u, {%1, %5};\n\tmov.b64 v, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, 1;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, 1;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, 1;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}

// D (+)= A . B over 64 keys: A in tensor memory (8 columns per 16 keys), B
// with its N index contiguous (2048 bytes per 16 keys).
__device__ __forceinline__ void mma4_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 v;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 v, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], v, %3, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, 1;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, 1;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 v, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, 1;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}

// The accesses below are warp-collective: the warp must be converged.
//
// Loads of 16 lanes x 32 columns in the layout of matrix fragments: lane t's
// registers 4 j .. 4 j + 3 are row t / 4, columns 8 j + 2 (t % 4) and the next
// one, and the same of row t / 4 + 8. Without the wait: tmem_wait16 must come
// before any use of r.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Waits for this thread's loads; the registers pass through it, so that no
// use of them is scheduled before.
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :);
}

// The store that matches tmem_ld_frag, without its wait.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// 16 lanes x 16 columns of FP16 pairs: register 2 j is row t / 4, column 4 j + t % 4,
// register 2 j + 1 the same of row t / 4 + 8. Without the wait.
__device__ __forceinline__ void tmem_st_half_frag(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// The load that matches tmem_st_half_frag, with its wait.
__device__ __forceinline__ void tmem_ld_half_frag_wait(uint32_t taddr, uint32_t (&r)[8]) {
    __syncwarp();   // warp-collective (.sync.aligned)
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint64_t lds64(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ void sts32f(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// sts128 at a constant offset.
template <int kOffset>
__device__ __forceinline__ void sts128_at(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0+%5], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w), "n"(kOffset)
                 : "memory");
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return half2_bits(r);
}

template <int N>
struct Index {
    static constexpr int value = N;
};

// ------------------------------------------------------------ shared memory

template <int D>
struct ChunkSmem {
    static constexpr int kPanel = kChKeys * 128;            // 64 dims of 128 tokens (or rows), FP16
    static constexpr int kTile = (D / 64) * kPanel;         // one Q, K or V tile
    static constexpr int kQ = 0;                            // two tiles
    static constexpr int kK = kQ + 2 * kTile;               // two stages
    static constexpr int kV = kK + 2 * kTile;               // two stages
    static constexpr int kF = kV + 2 * kTile;               // token factors: 4 x (128 K, 128 V) floats
    static constexpr int kZ = kF + 4 * 2 * kChKeys * 4;     // zeros: 2 x (128 K, 128 V) words
    static constexpr int kEnd = kZ + 2 * 2 * kChKeys * 4;
    static constexpr int kBytes = kEnd + 1024;              // the base is rounded up to 1024
};

struct ChunkBars {
    uint64_t q[2], k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], drain;
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

// wait_bounded for a role that waits for long beside busy warps: each try
// suspends the thread for up to 20 us instead of polling, which would take the
// others' issue slots.
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, const Watchdog &wd, int site, int detail) {
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(a), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if ((it & 31u) == 31u) {
            if (wd.aborted()) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                wd.fail(QOQ_ERR_TIMEOUT, site, detail);
                return false;
            }
        }
    }
}

// wait_bounded with one answer for the warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Watchdog &wd, int site, int detail) {
    const bool ok = wait_bounded(bar, parity, wd, site, detail);
    return __all_sync(0xffffffffu, ok);
}

// The softmax state of a warp's 32 rows. A thread holds four rows (8 i +
// lane / 4 of the warp's) and of each the keys 8 j + 2 (lane % 4) and the
// next one, so that a key's factors are read for 8 lanes and used for four
// rows each (reading them for one row per thread would take 2048 cycles of the
// shared memory per step).
struct RowState {
    float m[4];       // running maximum, in log2 units
    uint64_t l[4];    // two partial sums over this thread's keys
    float f[4];       // what the output so far has to be multiplied by in this step
    uint32_t fresh;   // rows that have seen no key yet, a bit each
};

// A block of 32 keys and 32 rows: the scores x = S s_K c - m, as pairs of keys
// [row half][4 groups of 8 keys x 2 rows], and the largest of each row's.
struct ScoreBlock {
    uint64_t x[2][8];
    float top[2][2];
};

// Scores of block q, whose first 16 rows' S is on its way in raw[0]; starts the
// load of the next block's. kf: shared-memory address of the lane's first factor.
__device__ __forceinline__ void block_scores(uint32_t ts, uint32_t kf, int q, const RowState &st, uint32_t (&raw)[2][16],
                                             ScoreBlock &b) {
    uint64_t f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = lds64(kf + 128 * q + 32 * j);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        uint32_t(&r)[16] = raw[hh];
        tmem_wait16(r);
        if (hh == 0) tmem_ld_frag(ts + (1u << 20) + 32u * q, raw[1]);
        else tmem_ld_frag(ts + 32u * ((q + 1) & 3), raw[0]);   // after the last block not used
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * hh + e;
            const uint64_t minus_m = pair_of(-st.m[i], -st.m[i]);
            float t = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                b.x[hh][2 * j + e] = fma2(pair_of(r[4 * j + 2 * e], r[4 * j + 2 * e + 1]), f[j], minus_m);
                const float2 y = of_pair(b.x[hh][2 * j + e]);
                t = fmaxf(t, fmaxf(y.x, y.y));
            }
            b.top[hh][e] = t;
        }
    }
}

// p = 2^x added to the sums, P = p s_V 2^(8 - E) as FP16 over the scores' place.
__device__ __forceinline__ void block_weights(uint32_t ts, uint32_t vf, int q, RowState &st, const ScoreBlock &b) {
    uint64_t g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = lds64(vf + 128 * q + 32 * j);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 y = of_pair(b.x[hh][2 * j + e]);
                const uint64_t p = pair_of(ex2_approx(y.x), ex2_approx(y.y));
                st.l[2 * hh + e] = add2(st.l[2 * hh + e], p);
                const float2 z = of_pair(mul2(p, g[j]));
                pk[2 * j + e] = half2_bits(__floats2half2_rn(z.x, z.y));
            }
        tmem_st_half_frag(ts + ((uint32_t)hh << 20) + 16u * q, pk);
    }
}

__device__ __forceinline__ bool block_raises(const RowState &st, const ScoreBlock &b) {
    return __any_sync(0xffffffffu, st.fresh != 0 || fmaxf(fmaxf(b.top[0][0], b.top[0][1]), fmaxf(b.top[1][0], b.top[1][1])) > kChSlack);
}

// A step's weights. Most steps are seen whole by every row and raise no
// maximum, and their loop is kept to what such steps need: with the rest inside,
// jumps over it left the instruction cache, which cost as much as the arithmetic
// (5000 cycles a step for what takes 2400 alone). The first block that raises a
// maximum, and a masked step, go to the loop below.
//
// A row's maximum is raised only when a score exceeds it by 2^kChSlack, by a
// whole number, so that what is already stored is rescaled exactly; a row takes
// its first maximum as it is. The step's keys stand at positions key0 .. key0 +
// 127; the key at c is hidden from row i where c > pos[i], or beyond the window
// (pos[i] - c >= reach) and the sinks (c >= sinks). pos_lo and pos_hi: the least
// and largest of the warp's rows.
__device__ __forceinline__ void softmax_rows(uint32_t ts, uint32_t kf, uint32_t vf, RowState &st, bool masked,
                                             const int (&pos)[4], int pos_lo, int pos_hi, int key0, int reach,
                                             int sinks) {
    uint32_t raw[2][16];
    ScoreBlock b;
    int q = 0;
    if (!masked) {
        tmem_ld_frag(ts, raw[0]);
#pragma unroll 1
        for (; q < 4; ++q) {
            block_scores(ts, kf, q, st, raw, b);
            if (block_raises(st, b)) break;
            block_weights(ts, vf, q, st, b);
        }
        tmem_wait16(raw[0]);
        if (q == 4) return;
    }
    tmem_ld_frag(ts + 32u * q, raw[0]);
#pragma unroll 1
    for (; q < 4; ++q) {
        // What of the block the warp's rows see: all of it, none, or some.
        const int c0 = key0 + 32 * q;
        const bool whole = c0 + 31 <= pos_lo && (pos_hi - c0 < reach || c0 + 32 <= sinks);
        if (c0 > pos_hi || (pos_lo - c0 - 31 >= reach && c0 >= sinks)) {
            const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            tmem_wait16(raw[0]);
            tmem_st_half_frag(ts + 16u * q, none);
            tmem_st_half_frag(ts + (1u << 20) + 16u * q, none);
            tmem_ld_frag(ts + 32u * ((q + 1) & 3), raw[0]);
            continue;
        }
        block_scores(ts, kf, q, st, raw, b);
        if (!whole) {
            const int first = c0 + 2 * ((int)threadIdx.x & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t = -INFINITY;
                const int d = pos[i] - first;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 y = of_pair(b.x[i >> 1][2 * j + (i & 1)]);
                    if (!(d >= 8 * j && (d - 8 * j < reach || first + 8 * j < sinks))) y.x = -INFINITY;
                    if (!(d >= 8 * j + 1 && (d - 8 * j - 1 < reach || first + 8 * j + 1 < sinks))) y.y = -INFINITY;
                    b.x[i >> 1][2 * j + (i & 1)] = pair_of(y.x, y.y);
                    t = fmaxf(t, fmaxf(y.x, y.y));
                }
                b.top[i >> 1][i & 1] = t;
            }
        }
        if (block_raises(st, b)) {
            float al[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t = b.top[i >> 1][i & 1];
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));   // of the row
                float up = 0.0f;
                al[i] = 1.0f;
                if (st.fresh >> i & 1u) {
                    if (t > -INFINITY) up = t, st.fresh &= ~(1u << i);
                } else if (t > kChSlack) {
                    up = ceilf(t);
                    al[i] = up < 126.0f ? __int_as_float((127 - (int)up) << 23) : 0.0f;
                    st.l[i] = mul2(st.l[i], pair_of(al[i], al[i]));
                    st.f[i] *= al[i];
                }
                st.m[i] += up;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b.x[i >> 1][2 * j + (i & 1)] = add2(b.x[i >> 1][2 * j + (i & 1)], pair_of(-up, -up));
            }
            __syncwarp();
            // The step's weights stored so far, times a power of two: exact, but for those
            // that become subnormal, which are rounded a second time, by at most 2^-25
            // beside a largest weight of some 2^8. A load of tensor memory is ordered
            // behind this warp's own stores of it by their wait alone.
            if (q > 0) tmem_st_wait();
#pragma unroll 1
            for (int o = 0; o < q; ++o)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const __half2 a0 = __float2half2_rn(al[2 * hh]), a1 = __float2half2_rn(al[2 * hh + 1]);
                    uint32_t pk[8];
                    tmem_ld_half_frag_wait(ts + ((uint32_t)hh << 20) + 16u * o, pk);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        pk[j] = half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&pk[j]), j & 1 ? a1 : a0));
                    tmem_st_half_frag(ts + ((uint32_t)hh << 20) + 16u * o, pk);
                }
        }
        block_weights(ts, vf, q, st, b);
    }
    tmem_wait16(raw[0]);
}

template <int D>
__global__ void __launch_bounds__(kChThreads, 1) kv4_chunk_kernel(const __grid_constant__ ChunkParams w) {
    using L = ChunkSmem<D>;
    constexpr int DB = D / 2;
    constexpr int CPT = DB / 16;                 // 16-byte code chunks per token
    constexpr int CPL = kChKeys * CPT / 128;     // chunks per unpacking thread and tile
    constexpr uint32_t kColS = 0, kColO = 256;   // TMEM: S0, S1 (P in their first halves), O0, O1
    const PagedAttnParams &p = w.a;
    extern __shared__ uint8_t ch_raw[];
    __shared__ ChunkBars bars;
    __shared__ uint32_t tmem_s;
    __shared__ volatile int abort_s;
    __shared__ float es_s[4], unit_s[4];   // per step (mod 4): 2^(E_old - E_new), 2^(E_new - 8)
    __shared__ uint32_t emax_s[2][4];
    __shared__ ChunkPiece piece_s[kChThreads / 32][2];   // each warp's piece, and the softmaxes' next
    __shared__ float2 stats_s[8][32];      // rows' maxima and sums at a piece's end

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;
    const Watchdog wd{&abort_s, p.status};
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q[i], 128);
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
    const uint32_t base = (smem_u32(ch_raw) + 1023u) & ~1023u;
    const uint32_t factors = base + (uint32_t)L::kF;

    griddep_wait();   // the division
    griddep_launch_dependents();
    const int pieces = w.division[p.B];
    // What this CTA's earlier pieces used of each barrier: steps, pieces and
    // pieces with steps, and of each those with a second row tile.
    uint32_t step_at = 0, step1_at = 0, piece_at = 0, out_at = 0, out1_at = 0;

    // The CTA's piece of a round, into *out (its warp's own place in shared
    // memory, where the roles read what they need of it); false after the
    // last. Pieces go round the CTAs forth and back: the lengths fall along the
    // list. Every role takes them by itself, in step with the others through the
    // barriers alone, so that the next piece's first keys are unpacked and its
    // queries loaded while the last one's output is written.
    auto locate = [&](int round, ChunkPiece *out) {
        const int piece = round * (int)gridDim.x + (round & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
        if (__any_sync(0xffffffffu, piece >= pieces || abort_s != 0)) return false;
        int lo = 0, hi = p.B - 1;   // the last place that starts at or before the piece
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (w.division[mid] <= piece) lo = mid;
            else hi = mid - 1;
        }
        ChunkPiece c;
        c.b = w.division[3 * p.B + 2 + lo];
        c.parts = w.division[2 * p.B + 2 + lo];
        c.r = paged_request(p, c.b);
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
        __syncwarp();
        if (lane == 0) *out = c;
        __syncwarp();
        return true;
    };
    auto advance = [&](const ChunkPiece &c) {
        const uint32_t steps = (uint32_t)(c.k1 - c.k0), two = c.rows > 128 ? 1 : 0;
        step_at += steps;
        step1_at += two * steps;
        ++piece_at;
        out_at += steps > 0;
        out1_at += two & (steps > 0);
        __syncwarp();
    };
    auto walk = [&](auto agree, auto role) {
        ChunkPiece *c = &piece_s[warp][0];
        for (int round = 0; agree(locate(round, c)); ++round) {
            role(*c);
            advance(*c);
        }
    };
    auto key_of = [&](const ChunkSteps &st, int k) {
        return (k < st.sinks ? k : st.first + (k - st.sinks)) * kChKeys;
    };

    if (wg < 2) {
        // ---------------------------------------------------------- softmax
        regs_inc<kRegsSoftmax>();
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's TMEM lanes
        const uint32_t ts = tmem + kColS + 128u * wg + lanes, to = tmem + kColO + (uint32_t)(D * wg) + lanes;
        const int row = tid & 127;
        // A piece's queries, a row per thread: dims in unpacking order, 128-byte swizzle.
        auto load_q = [&](const ChunkPiece &c) {
            if (wg * 128 >= c.rows || c.k0 == c.k1) return;
            const int pair = c.tile * kChRows + wg * 128 + row, token = pair / p.G;
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(c.r.row0 + token) * p.q_stride +
                                                               (int64_t)(c.h * p.G + pair - token * p.G) * D);
            const uint32_t dst = base + L::kQ + (uint32_t)(wg * L::kTile + row * 128);
            const bool in = wg * 128 + row < c.rows;
#pragma unroll
            for (int x0 = 0; x0 < D / 8; x0 += 8) {
                uint4 u[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    u[x] = make_uint4(0u, 0u, 0u, 0u);
                    if (in) u[x] = __ldg(src + x0 + x);
                }
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    sts128(dst + (uint32_t)((x0 >> 3) * L::kPanel + ((x ^ (row & 7)) << 4)),
                           __byte_perm(u[x].x, u[x].z, 0x5410), __byte_perm(u[x].x, u[x].z, 0x7632),
                           __byte_perm(u[x].y, u[x].w, 0x5410), __byte_perm(u[x].y, u[x].w, 0x7632));
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars.q[wg]);
        };
        bool have = locate(0, &piece_s[warp][0]);
        if (have) load_q(piece_s[warp][0]);
        for (int round = 0; have; ++round) {
            const ChunkPiece &c = piece_s[warp][round & 1];
            const PagedRequest &r = c.r;
            const int tile = c.tile, k0 = c.k0, k1 = c.k1;
            const bool active = wg * 128 < c.rows;
            bool ok = true;
            const int first_row = tile * kChRows + wg * 128 + 32 * (warp & 3);   // of the warp
            const int pos_lo = r.kv - r.n + first_row / p.G, pos_hi = r.kv - r.n + (first_row + 31) / p.G;
            // The thread's rows in the products' layout: 8 i + lane / 4 of the warp's.
            int pos[4];
            RowState rs;
            rs.fresh = 15u;
            float unit = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) rs.m[i] = 0.0f, rs.l[i] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pos[i] = r.kv - r.n + (first_row + 8 * i + (lane >> 2)) / p.G;
            for (int k = k0; active && k < k1; ++k) {
                const uint32_t s = step_at + (uint32_t)(k - k0);
                const uint32_t si = wg ? step1_at + (uint32_t)(k - k0) : s;
                const int t0 = key_of(c.st, k);
                if (!(ok = warp_wait(&bars.s_full[wg], si & 1, wd, kSiteChunkS, (int)s))) break;
                tc_fence_after();
                const uint32_t kf = factors + 4 * ((s & 3) * 2 * kChKeys + 2 * (lane & 3)), vf = kf + 4 * kChKeys;
                const bool whole = t0 + kChKeys - 1 <= pos_lo &&
                                   (p.window == 0 || pos_hi - t0 < p.window || t0 + kChKeys <= p.sinks);
                const float es = es_s[s & 3];
                unit = unit_s[s & 3];
#pragma unroll
                for (int i = 0; i < 4; ++i) rs.f[i] = es;
                softmax_rows(ts, kf, vf, rs, !whole, pos, pos_lo, pos_hi, t0, p.window ? p.window : INT32_MAX, p.sinks);
                const bool change = rs.f[0] != 1.0f || rs.f[1] != 1.0f || rs.f[2] != 1.0f || rs.f[3] != 1.0f;
                if (k > k0 && __any_sync(0xffffffffu, change)) {
#pragma unroll 1
                    for (int q = 0; q < D; q += 32)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t o[16];
                            tmem_ld_frag(to + ((uint32_t)hh << 20) + q, o);
                            tmem_wait16(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * rs.f[2 * hh + (i >> 1 & 1)]);
                            tmem_st_frag(to + ((uint32_t)hh << 20) + q, o);
                        }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars.p_full[wg]);
            }
            // The scores of the last step are in: the queries' place is free.
            have = ok && locate(round + 1, &piece_s[warp][(round + 1) & 1]);
            if (have) load_q(piece_s[warp][(round + 1) & 1]);
            if (active && k1 > k0)
                ok = ok && warp_wait(&bars.o_full[wg], (wg ? out1_at : out_at) & 1, wd, kSiteChunkO, (int)piece_at);
            if (!ok) break;
            advance(c);
            if (!active) continue;
            tc_fence_after();
            const int pair = tile * kChRows + wg * 128 + row;   // (token, head) pair of the request
            const bool in = wg * 128 + row < c.rows;
            const int token = pair / p.G, head = c.h * p.G + (pair - token * p.G), slot = c.slot;
            // Each row's maximum and sum, for the thread that writes the row.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = of_pair(rs.l[i]);
                float x = v.x + v.y;
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if ((lane & 3) == 0) stats_s[warp][8 * i + (lane >> 2)] = make_float2(rs.m[i], x);
            }
            __syncwarp();
            const float row_max = stats_s[warp][lane].x, row_sum = stats_s[warp][lane].y;
            __syncwarp();
            // A row before the sequence sees nothing and gives zeros. Every other one
            // sees itself: without a sum its scores were all -infinity, and 0 / 0 says so.
            const float f = slot >= 0 ? unit : r.kv - r.n + token < 0 ? 0.0f : unit / row_sum;
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
                    ml[(int64_t)slot * w.slot_rows + wg * 128 + row] = make_float2(row_sum > 0.0f ? row_max : -INFINITY, row_sum);
                }
                if (wg == 0 && row == 0)
                    *reinterpret_cast<int4 *>(w.slots + 4 * slot) = make_int4(c.b, c.h, tile, c.part == 0 ? c.parts : 0);
            }
            tc_fence_before();   // the next piece's products come after these reads
        }
    } else if (wg == 2) {
        // ---------------------------------------------------------- unpack
        // Codes to FP16, scales to factors of the scores and of the weights.
        regs_dec<kRegsUnpack>();
        const int t = tid & 127;
        // A thread unpacks chunk j (16 bytes, 32 dims) of the tokens
        // tk + 128 / CPT i: two lanes read a 32-byte half of a token's codes,
        // and the stores of 8 lanes touch every bank once.
        const int j = D == 128 ? 2 * (warp & 1) + (lane & 1) : lane & 1;
        const int tk = D == 128 ? 16 * ((warp >> 1) & 1) + (lane >> 1) : t >> 1;
        constexpr int kStride = 128 / CPT;
        const int page_mask = (1 << p.page_shift) - 1;
        const uint32_t page_vecs = (uint32_t)p.Hkv << p.page_shift, page_bytes = page_vecs * DB;
        const uint32_t last_page = (uint32_t)p.n_pages - 1u;
        const int64_t v_minus_k = p.v_codes - p.k_codes;
        const uint32_t zeros = base + (uint32_t)L::kZ;
        // Where the thread's four groups of 8 dims of its first token go, in K's
        // first stage.
        uint32_t to[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            to[x] = base + (uint32_t)(L::kK + tk * 128 + (j >> 1) * L::kPanel + (((4 * (j & 1) + x) ^ (tk & 7)) << 4));
        // Steps start at multiples of 128 tokens, so a token's place within
        // its page and its table entry relative to the step's first do not
        // change from step to step (pages of 256 tokens: but for 128).
        int part[CPL];   // table entries past the step's first: of the chunks
#pragma unroll
        for (int i = 0; i < CPL; ++i) part[i] = (tk + i * kStride) >> p.page_shift;
        const int part_t = t >> p.page_shift;   // of token t
        // The four warps meet in every step, so that they go on or stop (another
        // role may just have given up) as one.
        walk([](bool more) { return !named_bar_any(2, 128, !more); }, [&](const ChunkPiece &pc) {
            const int k0 = pc.k0, k1 = pc.k1, kv = pc.r.kv;
            if (k0 == k1) return;
            const int32_t *table = p.block_table + (int64_t)pc.b * p.max_pages;
            const int last_entry = (kv - 1) >> p.page_shift;   // there is a step only where kv > 0
            const uint32_t head_vec = (uint32_t)pc.h << p.page_shift;
            const uint8_t *from[CPL];   // the chunks' places in page 0 of K
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                from[i] = p.k_codes + ((uint64_t)head_vec + ((tk + i * kStride) & page_mask)) * DB + j * 16;
            const int64_t from_t = (int64_t)head_vec + (t & page_mask);
            // Table entries are loaded a step before anything depends on them.
            struct Pages {
                int chunk[CPL], token;
            };
            auto load_pages = [&](int k, Pages &g) {
                const int first = key_of(pc.st, min(k, k1 - 1)) >> p.page_shift;
#pragma unroll
                for (int i = 0; i < CPL; ++i) g.chunk[i] = __ldg(table + min(first + part[i], last_entry));
                g.token = __ldg(table + min(first + part_t, last_entry));
            };
            // Step k's codes of this thread. Numbers outside the cache read
            // its last page, which scales of 0 make nothing of.
            auto load_codes = [&](int k, const Pages &g, int64_t tensor, uint4 (&u)[CPL]) {
                const int64_t more = tensor + (p.page_shift == 8 ? (key_of(pc.st, min(k, k1 - 1)) & 128) * DB : 0);
#pragma unroll
                for (int i = 0; i < CPL; ++i)
                    u[i] = __ldg(reinterpret_cast<const uint4 *>(
                        from[i] + (uint64_t)min((uint32_t)g.chunk[i], last_page) * page_bytes + more));
            };
            uint32_t szk = 0u, szv = 0u;   // token t's scales and zeros
            // What a token holds that no row of the tile sees must not matter: it
            // counts as zero vectors, and its page may have been taken back.
            const int seen_from = pc.st.window, seen_to = pc.st.end;
            auto load_sz = [&](int k, int page) {
                szk = szv = 0u;
                const int key = key_of(pc.st, k) + t;
                if (k < k1 && key < seen_to && (key >= seen_from || key < p.sinks)) {
                    if ((uint32_t)page <= last_page) {
                        const int64_t at = from_t + (int64_t)page * page_vecs + (p.page_shift == 8 ? (key - t) & 128 : 0);
                        szk = __ldg(reinterpret_cast<const uint32_t *>(p.k_params) + at);
                        szv = __ldg(reinterpret_cast<const uint32_t *>(p.v_params) + at);
                    } else {
                        paged_bad_request(p, pc.b);
                    }
                }
            };
            uint4 uk[CPL], uv[CPL];   // this step's codes, then the next one's
            Pages g;                  // entries of the next step
            load_pages(k0, g);
            load_codes(k0, g, 0, uk);
            load_codes(k0, g, v_minus_k, uv);
            load_sz(k0, g.token);
            load_pages(k0 + 1, g);
            int eb = 103;   // 127 + the exponent of the largest value scale so far (scales >= 2^-24)
            bool ok = true;
            // A tensor's tile into its stage at `place` past K's first.
            auto unpack_tile = [&](const uint4 (&u)[CPL], uint32_t z, uint32_t place) {
                uint32_t dst[4], zz[CPL];
#pragma unroll
                for (int x = 0; x < 4; ++x) dst[x] = to[x] + place;
#pragma unroll
                for (int i = 0; i < CPL; ++i) zz[i] = lds32(z + 4 * (tk + i * kStride));   // halves 1024 + z, 64 + z
                auto unpack = [&](auto index) {
                    constexpr int i = decltype(index)::value;
                    const uint32_t z1 = __byte_perm(zz[i], zz[i], 0x1010), z2 = __byte_perm(zz[i], zz[i], 0x3232);
                    const uint32_t words[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t c = words[x], c8 = c >> 8;
                        sts128_at<i * kStride * 128>(
                            dst[x], hsub2((c & 0x000F000Fu) | 0x64006400u, z1), hsub2((c & 0x00F000F0u) | 0x54005400u, z2),
                            hsub2((c8 & 0x000F000Fu) | 0x64006400u, z1), hsub2((c8 & 0x00F000F0u) | 0x54005400u, z2));
                    }
                };
                unpack(Index<0>());
                unpack(Index<1>());
                if constexpr (CPL == 4) {
                    unpack(Index<2>());
                    unpack(Index<3>());
                }
                fence_proxy_async_smem();
            };
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                const uint32_t s = step_at + (uint32_t)(k - k0), stage = s & 1;
                const uint32_t z = zeros + 4 * stage * 2 * kChKeys;
                // The step's factors. A written scale is finite and a zero at
                // most 22 (15 times the 1.5 by which a subnormal scale may be
                // rounded down); up to 30 1024 + z, 64 + z and the codes' differences from them are
                // exact. Vectors that hold infinities have scales that are not
                // finite: such a token makes the outputs of the rows that see it NaN by
                // a NaN score, and has finite values, so that the weight 0 of the other rows stays 0.
                const bool finite = max(szk & 0x7FFFu, szv & 0x7FFFu) < 0x7C00u;
                const uint32_t sv = finite ? szv & 0x7FFFu : 0u;
                const float zk = fminf(fmaxf(__half2float(half_hi(szk)), 0.0f), 30.0f);
                const float zv = fminf(fmaxf(__half2float(half_hi(szv)), 0.0f), 30.0f);
                sts32(z + 4 * t, half2_bits(__floats2half2_rn(1024.0f + zk, 64.0f + zk)));
                sts32(z + 4 * (kChKeys + t), half2_bits(__floats2half2_rn(1024.0f + zv, 64.0f + zv)));
                const uint32_t wmax = __reduce_max_sync(0xffffffffu, sv);
                if (lane == 0) emax_s[stage][warp & 3] = wmax;
                // The only meeting of a step: zeros and maxima are double-buffered.
                if (named_bar_any(2, 128, !ok)) break;
                const uint32_t f = factors + 4 * ((s & 3) * 2 * kChKeys + t);
                const uint32_t top = max(max(emax_s[stage][0], emax_s[stage][1]), max(emax_s[stage][2], emax_s[stage][3]));
                const int ebn = max(eb, (int)(__float_as_uint(half_lo(top)) >> 23));
                sts32f(f, finite ? half_lo(szk) * p.qscale : __int_as_float(0x7FFFFFFF));
                sts32f(f + 4 * kChKeys, half_lo(sv) * __int_as_float((262 - ebn) << 23));   // 2^(8 - E)
                if (t == 0) {
                    es_s[s & 3] = __int_as_float((127 + eb - ebn) << 23);
                    unit_s[s & 3] = __int_as_float((ebn - 8) << 23);
                }
                eb = ebn;
                load_sz(k + 1, g.token);
                const uint32_t freed = ((s >> 1) - 1) & 1;
                ok = s < 2 || wait_long(&bars.k_free[stage], freed, wd, kSiteChunkFree, (int)s);
                if (ok) {
                    unpack_tile(uk, z, stage * (uint32_t)L::kTile);
                    mbar_arrive(&bars.k_full[stage]);
                }
                load_codes(k + 1, g, 0, uk);
                ok = ok && (s < 2 || wait_long(&bars.v_free[stage], freed, wd, kSiteChunkFree, (int)s));
                if (ok) {
                    unpack_tile(uv, z + 4 * kChKeys, (uint32_t)(L::kV - L::kK) + stage * (uint32_t)L::kTile);
                    mbar_arrive(&bars.v_full[stage]);
                }
                load_codes(k + 1, g, v_minus_k, uv);
                load_pages(k + 2, g);
            }
        });
    } else {
        // ---------------------------------------------------------- issue
        regs_dec<kRegsIssue>();
        if (warp == 12) walk([](bool more) { return more; }, [&](const ChunkPiece &c) {
            const int steps = c.k1 - c.k0;
            const bool two = c.rows > 128;
            constexpr uint32_t id_s = idesc_f16(128, kChKeys, false), id_o = idesc_f16(128, D, true);
            if (lane == 0 && steps > 0) {
                bool ok = wait_bounded(&bars.q[0], out_at & 1, wd, kSiteChunkQ, (int)piece_at);
                const uint32_t qd = desc_low(base + L::kQ, 16), kd = desc_low(base + L::kK, 16);
                const uint32_t vd = desc_low(base + L::kV, L::kPanel);
                auto scores = [&](int i, uint32_t stage) {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        mma4_f16_ss(tmem + kColS + 128u * i, qd + (uint32_t)((i * L::kTile + x * L::kPanel) >> 4),
                                    kd + (uint32_t)((stage * L::kTile + x * L::kPanel) >> 4), id_s, x > 0);
                    tc_commit(&bars.s_full[i]);
                };
                auto values = [&](int i, uint32_t stage, bool first) {
#pragma unroll
                    for (int x = 0; x < kChKeys / 64; ++x)
                        mma4_f16_ts(tmem + kColO + (uint32_t)(D * i), tmem + kColS + 128u * i + 32u * x,
                                    vd + (uint32_t)((stage * L::kTile + x * 64 * 128) >> 4), id_o, !first || x > 0);
                };
                if (ok) {
                    const uint32_t s0 = step_at;
                    ok = wait_bounded(&bars.k_full[s0 & 1], (s0 >> 1) & 1, wd, kSiteChunkK, (int)s0);
                    if (ok) {
                        tc_fence_after();
                        scores(0, s0 & 1);
                        // The second tile's queries come later, by as much as its softmax was behind in the last piece.
                        if (two && (ok = wait_bounded(&bars.q[1], out1_at & 1, wd, kSiteChunkQ, (int)piece_at))) {
                            tc_fence_after();
                            scores(1, s0 & 1);
                        }
                        tc_commit(&bars.k_free[s0 & 1]);
                    }
                    for (int k = 0; ok && k < steps; ++k) {
                        const uint32_t s = step_at + (uint32_t)k, stage = s & 1, next = stage ^ 1;
                        const bool more = k + 1 < steps;
                        if (!(ok = wait_bounded(&bars.v_full[stage], (s >> 1) & 1, wd, kSiteChunkV, (int)s))) break;
                        if (!(ok = wait_bounded(&bars.p_full[0], s & 1, wd, kSiteChunkP, (int)s))) break;
                        tc_fence_after();
                        values(0, stage, k == 0);
                        if (more) {
                            if (!(ok = wait_bounded(&bars.k_full[next], ((s + 1) >> 1) & 1, wd, kSiteChunkK, (int)s + 1))) break;
                            tc_fence_after();
                            scores(0, next);
                        } else {
                            tc_commit(&bars.o_full[0]);
                        }
                        if (two) {
                            if (!(ok = wait_bounded(&bars.p_full[1], (step1_at + (uint32_t)k) & 1, wd, kSiteChunkP, (int)s)))
                                break;
                            tc_fence_after();
                            values(1, stage, k == 0);
                            if (!more) tc_commit(&bars.o_full[1]);
                        }
                        tc_commit(&bars.v_free[stage]);
                        if (more) {
                            if (two) scores(1, next);
                            tc_commit(&bars.k_free[next]);
                        }
                    }
                }
                if (!ok) {
                    // Let the products in flight end before the memory is given back.
                    tc_commit(&bars.drain);
                    wait_drain(&bars.drain, 0, kWaitLimitNs);
                }
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

// Joins the parts of divided items, one warp per row.
constexpr int kJoinRows = 16;   // of an item, per turn of a CTA
constexpr int kJoinCtas = 8 * kChCtas;

template <int D>
__global__ void __launch_bounds__(256) kv4_chunk_join_kernel(const __grid_constant__ ChunkParams w) {
    const PagedAttnParams &p = w.a;
    griddep_wait();   // the parts
    const int slots = w.division[2 * p.B + 1], turns = w.slot_rows / kJoinRows;
    using Row = typename std::conditional<D == 128, float4, float2>::type;   // a lane's dims
    const int lane = threadIdx.x & 31;
    const float2 *ml = reinterpret_cast<const float2 *>(w.part + (int64_t)kChSlots * w.slot_rows * D);
#pragma unroll 1
    for (int turn = blockIdx.x; turn < slots * turns; turn += gridDim.x) {
        const int slot = turn / turns, row0 = (turn - slot * turns) * kJoinRows;
        const int4 it = *reinterpret_cast<const int4 *>(w.slots + 4 * slot);   // request, head, tile, parts
        const int parts = it.w;
        if (parts == 0) continue;   // not an item's first
        const PagedRequest r = paged_request(p, it.x);
        const int rows = min(min(r.n * p.G - it.z * kChRows, kChRows), row0 + kJoinRows);
#pragma unroll 1
        for (int row = row0 + (threadIdx.x >> 5); row < rows; row += 8) {
            // Lane i holds part i's maximum and weight (then i + 32's, ...).
            float m = -INFINITY, l = 0.0f, o[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[e] = 0.0f;
#pragma unroll 1
            for (int i = lane; i < parts; i += 32) m = fmaxf(m, ml[(int64_t)(slot + i) * w.slot_rows + row].x);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll 1
            for (int i0 = 0; i0 < parts; i0 += 32) {
                const float2 x = i0 + lane < parts ? ml[(int64_t)(slot + i0 + lane) * w.slot_rows + row] : make_float2(0.0f, 0.0f);
                const float mine = x.y > 0.0f ? exp2f(x.x - m) : 0.0f;
                l = fmaf(mine, x.y, l);
                const float *src = w.part + ((int64_t)(slot + i0) * w.slot_rows + row) * D + lane * (D / 32);
                const int n = min(parts - i0, 32);
#pragma unroll 4
                for (int i = 0; i < n; ++i) {
                    const float f = __shfl_sync(0xffffffffu, mine, i);
                    Row v = *reinterpret_cast<const Row *>(src + (int64_t)i * w.slot_rows * D);
                    const float *x4 = reinterpret_cast<const float *>(&v);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) o[e] = fmaf(f, x4[e], o[e]);
                }
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
            const int pair = it.z * kChRows + row, token = pair / p.G;
            const float f = r.kv - r.n + token < 0 ? 0.0f : 1.0f / l;   // as for undivided items
            __half2 *out = reinterpret_cast<__half2 *>(p.out + (int64_t)(r.row0 + token) * p.out_stride +
                                                       (int64_t)(it.y * p.G + pair - token * p.G) * D + lane * (D / 32));
#pragma unroll
            for (int e = 0; e < D / 32; e += 2) out[e / 2] = __floats2half2_rn(o[e] * f, o[e + 1] * f);
        }
    }
}

int slot_rows(int64_t max_new, int64_t G) {
    const int64_t rows = max_new * G;
    return rows >= kChRows ? kChRows : (int)((rows + kJoinRows - 1) / kJoinRows * kJoinRows);
}

// A launch that may begin before the kernel ahead of it has ended, whose results
// it waits for itself.
template <typename Kernel>
cudaError_t launch_dependent(Kernel kernel, int blocks, int threads, int smem, const ChunkParams &w, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, w);
}

template <int D>
cudaError_t launch(const ChunkParams &w, cudaStream_t stream) {
    constexpr int smem = ChunkSmem<D>::kBytes;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in.set(kv4_chunk_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    const int threads = w.a.B >= kDvThreads ? kDvThreads : (w.a.B + 31) / 32 * 32;
    // Beside the few-rows kernel: it reads nothing that one writes.
    e = launch_dependent(kv4_chunk_division_kernel, 1, threads, 0, w, stream);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kv4_chunk_kernel<D>, kChCtas, kChThreads, smem, w, stream);
    if (e != cudaSuccess) return e;
    return launch_dependent(kv4_chunk_join_kernel<D>, kJoinCtas, 256, 0, w, stream);
}

}  // namespace

// Workspace: the division, the slots' items, the partial results.
size_t chunk_workspace_bytes(int64_t B, int64_t max_new, int64_t G, int64_t D) {
    return (size_t)align256(4 * (4 * B + 2)) + (size_t)align256(16 * kChSlots) +
           (size_t)align256((int64_t)4 * kChSlots * slot_rows(max_new, G) * (D + 2));
}

// Requests with more than kRowsMax (row, head) pairs per KV head, behind launch_paged_rows.
cudaError_t launch_paged_chunk(const PagedAttnParams &p, int64_t D, int64_t max_new, void *ws, cudaStream_t stream) {
    ChunkParams w;
    w.a = p;
    w.slot_rows = slot_rows(max_new, p.G);
    uint8_t *at = static_cast<uint8_t *>(ws);
    w.division = reinterpret_cast<int32_t *>(at);
    at += align256(4 * (4 * (int64_t)p.B + 2));
    w.slots = reinterpret_cast<int32_t *>(at);
    at += align256(16 * kChSlots);
    w.part = reinterpret_cast<float *>(at);
    return D == 128 ? launch<128>(w, stream) : launch<64>(w, stream);
}

}  // namespace qoq
