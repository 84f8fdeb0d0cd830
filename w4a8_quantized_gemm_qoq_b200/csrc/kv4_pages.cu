// Page tables and slot maps of the paged KV4 cache, built on the GPU from the
// requests' lengths, and the release of ended requests' pages.
//
// One thread-block cluster does a whole step in one launch: every CTA scans
// all requests' lengths into its own shared memory (8 bytes read per request,
// from L2 after the first CTA), checks its share of the page numbers, and
// after one cluster barrier -- when everything the step reads of the state has
// been read, so that the state may be updated in place -- writes its share of
// the rows and pages. A row finds its request by a binary search of the
// scanned row starts in shared memory. Nothing is kept between calls and no
// workspace is needed. The work is a few microseconds of latency (two dependent
// loads, the scan, the barrier), not bytes: 64 requests with a token each 5.0 us, 256
// with 37000 tokens between them and the release of all of them 13.8 us together.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4_paged.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"

namespace qoq {

namespace {

constexpr int kPgThreads = 512;
constexpr int kPgWarps = kPgThreads / 32;

struct PagesParams {
    const int32_t *seq_lens, *new_lens;
    const int32_t *free_pages, *free_count;
    int32_t *block_table;
    int32_t *kv_lens, *q_start, *positions, *slots, *free_left;
    int32_t *status;
    int B, n_pages, max_pages, max_tokens, page_shift;
};

// Exclusive prefix sums over the CTA's threads of two values; `ta`, `tb` are
// the totals. `red` holds 2 * kPgWarps values and is free again on return.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t &ta, int64_t &tb, int64_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t a0 = a, b0 = b;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, a, s), ub = __shfl_up_sync(0xffffffffu, b, s);
        if (lane >= s) a += ua, b += ub;
    }
    if (lane == 31) red[warp] = a, red[kPgWarps + warp] = b;
    __syncthreads();
    int64_t oa = 0, ob = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) {
        const int64_t xa = red[w], xb = red[kPgWarps + w];
        if (w < warp) oa += xa, ob += xb;
        ta += xa, tb += xb;
    }
    a += oa - a0;
    b += ob - b0;
    __syncthreads();
}

// The last b with start[b] <= x (start[0] = 0 <= x): requests without rows or
// pages share their start with the next one, so the last one is the owner.
__device__ __forceinline__ int owner_of(const int32_t *start, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A cluster barrier in two halves: no CTA's shared memory is written from another
// before it runs and has initialised it.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Raise `err` (at offset of this CTA's own variable) in every CTA of the cluster.
__device__ __forceinline__ void cluster_raise(int32_t *err, int code, int ctas) {
    const uint32_t a = smem_u32(err);
    for (int r = 0; r < ctas; ++r) {
        uint32_t ra;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(r));
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(ra), "r"(code) : "memory");
    }
}

__device__ __forceinline__ void record(int32_t *status, int code, int request, int64_t rows, int64_t pages) {
    if (atomicCAS(status, 0, code) == 0) {
        status[1] = request;
        status[2] = (int32_t)(rows < INT32_MAX ? rows : INT32_MAX);
        status[3] = (int32_t)(pages < INT32_MAX ? pages : INT32_MAX);
    }
}

__global__ void __launch_bounds__(kPgThreads) kv4_assign_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ int32_t pg_smem[];
    int32_t *row0 = pg_smem, *page0 = row0 + p.B, *len = page0 + p.B;   // first row, first taken page, cached tokens
    __shared__ int64_t red[2 * kPgWarps];
    __shared__ int32_t bad_pages;   // raised by any CTA of the cluster
    __shared__ int32_t bad_request;
    const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
    const int P = 1 << p.page_shift;
    if (tid == 0) bad_pages = 0, bad_request = INT32_MAX;
    __syncthreads();
    if (ctas > 1) cluster_arrive();   // this CTA runs and may be told of bad pages: waited for before it is

    // 1. Every CTA: the rows and pages before each request.
    const int count = *p.free_count;
    int64_t rows = 0, pages = 0;
    int code = count < 0 || count > p.n_pages ? QOQ_ERR_INVALID_ARG : 0;
    bool bad_arg = false;
    for (int base = 0; base < p.B; base += kPgThreads) {
        const int b = base + tid;
        int64_t n = 0, take = 0;
        if (b < p.B) {
            const int s = p.seq_lens[b], m = p.new_lens[b];
            len[b] = s;
            if (s < 0 || m < 0) {
                bad_arg = true;
                atomicMin(&bad_request, b);
            } else if ((int64_t)s + m > ((int64_t)p.max_pages << p.page_shift)) {
                atomicMin(&bad_request, b);
                n = m;
                take = (((int64_t)s + m + P - 1) >> p.page_shift) - (((int64_t)s + P - 1) >> p.page_shift);
            } else {
                n = m;
                take = ((s + m + (int64_t)P - 1) >> p.page_shift) - ((s + (int64_t)P - 1) >> p.page_shift);
            }
        }
        int64_t rn, rt;
        block_scan2(n, take, rn, rt, red);
        if (b < p.B) {
            // Beyond INT32_MAX the step is refused below and these are not used.
            row0[b] = (int32_t)(rows + n);
            page0[b] = (int32_t)(pages + take);
        }
        rows += rn;
        pages += rt;
    }
    if (__syncthreads_or(bad_arg)) code = QOQ_ERR_INVALID_ARG;
    const int request = bad_request == INT32_MAX ? -1 : bad_request;
    if (code == 0 && (request >= 0 || rows > p.max_tokens || pages > count)) code = QOQ_ERR_WORKSPACE;

    // 2. This CTA's share of the page numbers that the step reads.
    if (ctas > 1) cluster_wait();
    if (code == 0) {
        bool bad = false;
        for (int b = rank * kPgThreads + tid; b < p.B; b += ctas * kPgThreads)
            if ((len[b] & (P - 1)) && p.new_lens[b] > 0)
                bad |= (uint32_t)p.block_table[(int64_t)b * p.max_pages + (len[b] >> p.page_shift)] >=
                       (uint32_t)p.n_pages;
        for (int g = rank * kPgThreads + tid; g < (int)pages; g += ctas * kPgThreads)
            bad |= (uint32_t)p.free_pages[count - 1 - g] >= (uint32_t)p.n_pages;
        if (bad) cluster_raise(&bad_pages, QOQ_ERR_INVALID_ARG, ctas);
    }
    __syncthreads();
    if (ctas > 1) cluster_sync_all();   // every CTA has read the state, and knows of every bad page
    if (code == 0) code = bad_pages;

    // 3. This CTA's share of the step.
    const int total = code ? 0 : (int)rows;
    for (int b = rank * kPgThreads + tid; b < p.B; b += ctas * kPgThreads) {
        p.q_start[b] = code ? 0 : row0[b];
        p.kv_lens[b] = code ? len[b] : len[b] + p.new_lens[b];
    }
    if (rank == 0 && tid == 0) {
        p.q_start[p.B] = total;
        *p.free_left = code ? count : count - (int)pages;
        if (code) record(p.status, code, request, rows, pages);
    }
    // A row per thread where that covers the step (its loads are independent);
    // else four in a row, with one search and one table or stack entry per page
    // (37000 rows of 256 requests: 11 us, 13 with a row per thread).
    const int per = total <= ctas * kPgThreads ? 1 : 4;
    const bool wide = per == 4 && ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
    for (int t = per * (rank * kPgThreads + tid); t < p.max_tokens; t += per * ctas * kPgThreads) {
        int pos[4], slot[4];
        int b = t < total ? owner_of(row0, p.B, t) : 0, entry = -1, page = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pos[e] = slot[e] = -1;
            if (e >= per || t + e >= total) continue;
            while (b + 1 < p.B && row0[b + 1] <= t + e) ++b, entry = -1;
            const int s = len[b];
            pos[e] = s + (t + e - row0[b]);
            const int i = pos[e] >> p.page_shift, have = (s + P - 1) >> p.page_shift;
            if (i != entry) {
                entry = i;
                page = i < have ? p.block_table[(int64_t)b * p.max_pages + i] : p.free_pages[count - 1 - page0[b] - (i - have)];
            }
            slot[e] = (page << p.page_shift) + (pos[e] & (P - 1));
        }
        if (wide && t + 4 <= p.max_tokens) {
            *reinterpret_cast<int4 *>(p.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(p.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < per && t + e < p.max_tokens) p.positions[t + e] = pos[e], p.slots[t + e] = slot[e];
        }
    }
    if (code == 0)
        for (int g = rank * kPgThreads + tid; g < (int)pages; g += ctas * kPgThreads) {
            const int b = owner_of(page0, p.B, g);
            const int have = (len[b] + P - 1) >> p.page_shift;
            p.block_table[(int64_t)b * p.max_pages + have + (g - page0[b])] = p.free_pages[count - 1 - g];
        }
}

struct ReleaseParams {
    const int32_t *leave;
    int32_t *seq_lens, *block_table, *free_pages, *free_count, *status;
    int B, n_pages, max_pages, page_shift;
};

__global__ void __launch_bounds__(kPgThreads) kv4_release_kernel(const __grid_constant__ ReleaseParams p) {
    extern __shared__ int32_t pg_smem[];
    int32_t *page0 = pg_smem;   // first page, among those given back, of each request
    __shared__ int64_t red[2 * kPgWarps];
    __shared__ int32_t bad_pages, bad_request;
    const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
    const int P = 1 << p.page_shift;
    if (tid == 0) bad_pages = 0, bad_request = INT32_MAX;
    __syncthreads();
    if (ctas > 1) cluster_arrive();   // this CTA runs and may be told of bad pages: waited for before it is
    const int count = *p.free_count;
    int64_t pages = 0;
    int code = count < 0 || count > p.n_pages ? QOQ_ERR_INVALID_ARG : 0;
    for (int base = 0; base < p.B; base += kPgThreads) {
        const int b = base + tid;
        int64_t n = 0, none = 0, rn, r0;
        if (b < p.B && p.leave[b] != 0) {
            const int64_t s = p.seq_lens[b];
            n = s < 0 ? 0 : (s + P - 1) >> p.page_shift;
            if (s < 0 || n > p.max_pages) {
                atomicMin(&bad_request, b);
                n = 0;
            }
        }
        block_scan2(n, none, rn, r0, red);
        if (b < p.B) page0[b] = (int32_t)(pages + n);
        pages += rn;
    }
    __syncthreads();
    const int request = bad_request == INT32_MAX ? -1 : bad_request;
    if (request >= 0) code = QOQ_ERR_INVALID_ARG;
    if (code == 0 && pages > p.n_pages - count) code = QOQ_ERR_WORKSPACE;
    if (ctas > 1) cluster_wait();
    if (code == 0) {
        bool bad = false;
        for (int g = rank * kPgThreads + tid; g < (int)pages; g += ctas * kPgThreads) {
            const int b = owner_of(page0, p.B, g);
            bad |= (uint32_t)p.block_table[(int64_t)b * p.max_pages + (g - page0[b])] >= (uint32_t)p.n_pages;
        }
        if (bad) cluster_raise(&bad_pages, QOQ_ERR_INVALID_ARG, ctas);
    }
    __syncthreads();
    if (ctas > 1) cluster_sync_all();   // every CTA has read the lengths and the count, and knows of every bad page
    if (code == 0) code = bad_pages;
    if (code) {
        if (rank == 0 && tid == 0) record(p.status, code, request, 0, pages);
        return;
    }
    for (int g = rank * kPgThreads + tid; g < (int)pages; g += ctas * kPgThreads) {
        const int b = owner_of(page0, p.B, g);
        int32_t *e = p.block_table + (int64_t)b * p.max_pages + (g - page0[b]);
        p.free_pages[count + (int)pages - 1 - g] = *e;
        *e = -1;
    }
    for (int b = rank * kPgThreads + tid; b < p.B; b += ctas * kPgThreads)
        if (p.leave[b] != 0) p.seq_lens[b] = 0;
    if (rank == 0 && tid == 0) *p.free_count = count + (int)pages;
}

// One CTA where its threads cover the rows in a few steps, else a cluster of
// eight (the portable size).
int page_ctas(int64_t B, int64_t work) { return B <= 1024 && work <= 4 * kPgThreads ? 1 : 8; }

// The kernel's shared-memory limit belongs to the process and not to a call:
// it is set once, to what the largest batch needs, since a call that set its
// own need would lower the limit between another thread's setting and launch.
template <typename Params>
cudaError_t launch_cluster(void (*kernel)(Params), SmemOptIn &opt_in, int words, const Params &p, int ctas,
                           cudaStream_t stream) {
    const size_t per = sizeof(int32_t) * (size_t)words, smem = per * (size_t)p.B;
    if (smem > 40 * 1024) {   // 48 KB are free to use, the kernels' static arrays among them
        const cudaError_t e = opt_in.set(kernel, (int)(per * kMaxPagedBatch));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_pages_assign(const int32_t *seq_lens, const int32_t *new_lens, int64_t B, int page_shift,
                                const int32_t *free_pages, const int32_t *free_count, int64_t n_pages,
                                int32_t *block_table, int64_t max_pages, int64_t max_tokens, int32_t *kv_lens,
                                int32_t *q_start, int32_t *positions, int32_t *slots, int32_t *free_left,
                                int32_t *status, cudaStream_t stream) {
    PagesParams p;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.q_start = q_start;
    p.positions = positions;
    p.slots = slots;
    p.free_left = free_left;
    p.status = status;
    p.B = (int)B;
    p.n_pages = (int)n_pages;
    p.max_pages = (int)max_pages;
    p.max_tokens = (int)max_tokens;
    p.page_shift = page_shift;
    static SmemOptIn opt_in;
    return launch_cluster(kv4_assign_kernel, opt_in, 3, p, page_ctas(B, max_tokens), stream);
}

cudaError_t launch_pages_release(const int32_t *leave, int64_t B, int page_shift, int32_t *seq_lens,
                                 int32_t *block_table, int64_t max_pages, int32_t *free_pages, int32_t *free_count,
                                 int64_t n_pages, int32_t *status, cudaStream_t stream) {
    ReleaseParams p;
    p.leave = leave;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.status = status;
    p.B = (int)B;
    p.n_pages = (int)n_pages;
    p.max_pages = (int)max_pages;
    p.page_shift = page_shift;
    static SmemOptIn opt_in;
    return launch_cluster(kv4_release_kernel, opt_in, 1, p, page_ctas(B, n_pages), stream);
}

}  // namespace qoq
