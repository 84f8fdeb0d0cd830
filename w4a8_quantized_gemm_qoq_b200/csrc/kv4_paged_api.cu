// C-ABI entry points of the paged KV4 cache (declared in include/qoq.h):
// argument validation, size queries and dispatch. Nothing here allocates,
// frees or synchronises; every launch goes to the caller's stream.
#include <cmath>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qoq_internal.h"

using namespace qoq;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

qoq_status status_of(cudaError_t e) { return e == cudaSuccess ? QOQ_OK : QOQ_ERR_CUDA; }

// Page size (a power of two from 16 to 256) and page count; *shift = log2(page size).
qoq_status check_pages(int64_t page_size, int64_t n_pages, int *shift) {
    if (page_size <= 0 || n_pages <= 0) return QOQ_ERR_INVALID_ARG;
    int s = 4;
    while (s < 8 && ((int64_t)1 << s) != page_size) ++s;
    if (((int64_t)1 << s) != page_size || n_pages > INT32_MAX / page_size) return QOQ_ERR_UNSUPPORTED;
    *shift = s;
    return QOQ_OK;
}

qoq_status check_table(int64_t B, int64_t page_size, int64_t max_pages) {
    if (B < 0 || max_pages <= 0) return QOQ_ERR_INVALID_ARG;
    if (B > kMaxPagedBatch || max_pages > INT32_MAX / 2 / page_size) return QOQ_ERR_UNSUPPORTED;
    return QOQ_OK;
}

qoq_status check_heads(int64_t Hkv, int64_t D) {
    if (Hkv <= 0 || D <= 0) return QOQ_ERR_INVALID_ARG;
    if (Hkv > 65535 || (D != 64 && D != 128)) return QOQ_ERR_UNSUPPORTED;
    return QOQ_OK;
}

}  // namespace

extern "C" {

qoq_status qoq_kv4_pages_assign(const int32_t *seq_lens, const int32_t *new_lens, int64_t B, int64_t page_size,
                                const int32_t *free_pages, const int32_t *free_count, int64_t n_pages,
                                int32_t *block_table, int64_t max_pages, int64_t max_tokens, int32_t *kv_lens,
                                int32_t *q_start, int32_t *positions, int32_t *slots, int32_t *free_left,
                                int32_t *status, void *stream) {
    int shift = 0;
    qoq_status st = check_pages(page_size, n_pages, &shift);
    if (st != QOQ_OK) return st;
    if ((st = check_table(B, page_size, max_pages)) != QOQ_OK) return st;
    if (max_tokens < 0) return QOQ_ERR_INVALID_ARG;
    if (max_tokens > INT32_MAX / 2) return QOQ_ERR_UNSUPPORTED;
    if (free_pages == nullptr || free_count == nullptr || q_start == nullptr || free_left == nullptr ||
        status == nullptr || (max_tokens > 0 && (positions == nullptr || slots == nullptr)) ||
        (B > 0 && (seq_lens == nullptr || new_lens == nullptr || block_table == nullptr || kv_lens == nullptr)))
        return QOQ_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_start, 4) || !aligned(positions, 4) ||
        !aligned(slots, 4) || !aligned(free_left, 4) || !aligned(status, 4))
        return QOQ_ERR_ALIGNMENT;
    return status_of(launch_pages_assign(seq_lens, new_lens, B, shift, free_pages, free_count, n_pages, block_table,
                                         max_pages, max_tokens, kv_lens, q_start, positions, slots, free_left, status,
                                         static_cast<cudaStream_t>(stream)));
}

qoq_status qoq_kv4_pages_release(const int32_t *leave, int64_t B, int64_t page_size, int32_t *seq_lens,
                                 int32_t *block_table, int64_t max_pages, int32_t *free_pages, int32_t *free_count,
                                 int64_t n_pages, int32_t *status, void *stream) {
    int shift = 0;
    qoq_status st = check_pages(page_size, n_pages, &shift);
    if (st != QOQ_OK) return st;
    if ((st = check_table(B, page_size, max_pages)) != QOQ_OK) return st;
    if (B == 0) return QOQ_OK;
    if (leave == nullptr || seq_lens == nullptr || block_table == nullptr || free_pages == nullptr ||
        free_count == nullptr || status == nullptr)
        return QOQ_ERR_INVALID_ARG;
    if (!aligned(leave, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
        !aligned(free_count, 4) || !aligned(status, 4))
        return QOQ_ERR_ALIGNMENT;
    return status_of(launch_pages_release(leave, B, shift, seq_lens, block_table, max_pages, free_pages, free_count,
                                          n_pages, status, static_cast<cudaStream_t>(stream)));
}

qoq_status qoq_kv4_paged_write(const void *k_fp16, int64_t k_stride, const void *v_fp16, int64_t v_stride,
                               const int32_t *slots, int64_t N, int64_t Hkv, int64_t D, int64_t n_pages,
                               int64_t page_size, uint8_t *k_codes, void *k_params, uint8_t *v_codes,
                               void *v_params, void *stream) {
    int shift = 0;
    qoq_status st = check_heads(Hkv, D);
    if (st != QOQ_OK) return st;
    if ((st = check_pages(page_size, n_pages, &shift)) != QOQ_OK) return st;
    if (N < 0 || k_stride < Hkv * D || v_stride < Hkv * D) return QOQ_ERR_INVALID_ARG;
    if (N > INT32_MAX || N * Hkv > ((int64_t)1 << 31)) return QOQ_ERR_UNSUPPORTED;
    if (N == 0) return QOQ_OK;
    if (k_fp16 == nullptr || v_fp16 == nullptr || slots == nullptr || k_codes == nullptr || k_params == nullptr ||
        v_codes == nullptr || v_params == nullptr)
        return QOQ_ERR_INVALID_ARG;
    if (!aligned(k_fp16, 16) || !aligned(v_fp16, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_params, 8) || !aligned(v_params, 8) ||
        !aligned(slots, 4))
        return QOQ_ERR_ALIGNMENT;
    return status_of(launch_paged_write(k_fp16, k_stride, v_fp16, v_stride, slots, N, Hkv, D, n_pages, shift, k_codes,
                                        k_params, v_codes, v_params, static_cast<cudaStream_t>(stream)));
}

qoq_status qoq_kv4_paged_read(const int32_t *slots, int64_t N, int64_t Hkv, int64_t D, int64_t n_pages,
                              int64_t page_size, const uint8_t *k_codes, const void *k_params,
                              const uint8_t *v_codes, const void *v_params, void *k_out_fp16, void *v_out_fp16,
                              void *stream) {
    int shift = 0;
    qoq_status st = check_heads(Hkv, D);
    if (st != QOQ_OK) return st;
    if ((st = check_pages(page_size, n_pages, &shift)) != QOQ_OK) return st;
    if (N < 0) return QOQ_ERR_INVALID_ARG;
    if (N > INT32_MAX || N * Hkv > ((int64_t)1 << 31)) return QOQ_ERR_UNSUPPORTED;
    if (N == 0) return QOQ_OK;
    if (slots == nullptr || k_codes == nullptr || k_params == nullptr || v_codes == nullptr || v_params == nullptr ||
        k_out_fp16 == nullptr || v_out_fp16 == nullptr)
        return QOQ_ERR_INVALID_ARG;
    if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_params, 8) || !aligned(v_params, 8) ||
        !aligned(slots, 4) || !aligned(k_out_fp16, 16) || !aligned(v_out_fp16, 16))
        return QOQ_ERR_ALIGNMENT;
    return status_of(launch_paged_read(slots, N, Hkv, D, n_pages, shift, k_codes, k_params, v_codes, v_params,
                                       k_out_fp16, v_out_fp16, static_cast<cudaStream_t>(stream)));
}

qoq_status qoq_kv4_paged_attention(const void *q_fp16, int64_t q_stride, const uint8_t *k_codes,
                                   const void *k_params, const uint8_t *v_codes, const void *v_params,
                                   const int32_t *block_table, int64_t max_pages, const int32_t *q_start,
                                   const int32_t *kv_lens, int64_t B, int64_t N, int64_t max_new, int64_t Hq,
                                   int64_t Hkv, int64_t D, int64_t n_pages, int64_t page_size, int64_t window,
                                   int64_t sinks, void *out_fp16, int64_t out_stride, void *workspace,
                                   size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return QOQ_ERR_INVALID_ARG;
    qoq_status st = check_heads(Hkv, D);
    if (st != QOQ_OK) return st;
    if (Hq <= 0 || B < 0 || N < 0 || max_new < 1) return QOQ_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || Hq / Hkv > 8 || B > kMaxPagedBatch || N > INT32_MAX / 8) return QOQ_ERR_UNSUPPORTED;
    if (max_new > N) max_new = N > 0 ? N : 1;
    const size_t need = kv4_paged_workspace_bytes(B, N, Hq, Hkv, D, max_new);
    if (workspace == nullptr) {
        *workspace_bytes = need;
        return QOQ_OK;
    }
    if (*workspace_bytes < need) return QOQ_ERR_WORKSPACE;
    int shift = 0;
    if ((st = check_pages(page_size, n_pages, &shift)) != QOQ_OK) return st;
    if ((st = check_table(B, page_size, max_pages)) != QOQ_OK) return st;
    if (window < 0 || sinks < 0 || q_stride < Hq * D || out_stride < Hq * D) return QOQ_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return QOQ_OK;
    if (q_fp16 == nullptr || k_codes == nullptr || k_params == nullptr || v_codes == nullptr || v_params == nullptr ||
        block_table == nullptr || q_start == nullptr || kv_lens == nullptr || out_fp16 == nullptr)
        return QOQ_ERR_INVALID_ARG;
    if (!aligned(q_fp16, 16) || !aligned(out_fp16, 16) || q_stride % 8 != 0 || out_stride % 8 != 0 ||
        !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_params, 8) || !aligned(v_params, 8) ||
        !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 256))
        return QOQ_ERR_ALIGNMENT;
    PagedAttnParams p;
    p.q = static_cast<const __half *>(q_fp16);
    p.q_stride = q_stride;
    p.k_codes = k_codes;
    p.v_codes = v_codes;
    p.k_params = static_cast<const __half2 *>(k_params);
    p.v_params = static_cast<const __half2 *>(v_params);
    p.block_table = block_table;
    p.q_start = q_start;
    p.kv_lens = kv_lens;
    p.out = static_cast<__half *>(out_fp16);
    p.out_stride = out_stride;
    p.status = static_cast<int32_t *>(workspace);
    p.N = N;
    p.B = (int)B;
    p.max_pages = (int)max_pages;
    p.max_new = (int)max_new;
    p.Hq = (int)Hq;
    p.Hkv = (int)Hkv;
    p.G = (int)(Hq / Hkv);
    p.n_pages = (int)n_pages;
    p.page_shift = shift;
    // No two positions are further apart than the table holds tokens.
    const int64_t reach = max_pages << shift;
    p.window = window >= reach ? 0 : (int)window;
    p.sinks = (int)(sinks < reach ? sinks : reach);
    p.qscale = (float)(1.4426950408889634 / std::sqrt((double)D));
    return status_of(launch_paged_attention(p, D, max_new, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
