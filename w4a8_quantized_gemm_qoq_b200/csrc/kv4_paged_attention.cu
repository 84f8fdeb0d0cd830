// Attention of new tokens over the paged KV4 cache: which kernels a call runs.
#include "qoq_internal.h"

namespace qoq {

// Workspace: status words in bytes [0, 256), the few-rows kernel's part, the
// many-rows kernel's.
size_t kv4_paged_workspace_bytes(int64_t B, int64_t, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_new) {
    const int64_t G = Hq / Hkv;
    return 256 + rows_workspace_bytes(B, D) + (max_new * G > kRowsMax ? chunk_workspace_bytes(B, max_new, G, D) : 0);
}

// A request with at most 48 (row, head) pairs per KV head goes to the few-rows
// kernel, the others to the many-rows one. Measured on both sides of it, 32 sequences
// of 1500 to 4500 tokens, 8 KV heads of 128: with 8, 16, 24, 32, 40, 48 and 64
// pairs the former takes 34, 52, 70, 86, 104, 122 and 157 us, the latter
// 127 to 132 us with 16 to 64 of them. Where
// every request has max_new rows (as N says it may) and those are many, the
// few-rows kernel would find nothing, and the other takes whatever comes.
cudaError_t launch_paged_attention(const PagedAttnParams &p, int64_t D, int64_t max_new, void *ws,
                                   cudaStream_t stream) {
    uint8_t *at = static_cast<uint8_t *>(ws) + 256;
    const bool many = max_new * p.G > kRowsMax, all = many && p.N >= p.B * max_new;
    if (!all) {
        const cudaError_t e = launch_paged_rows(p, D, at, stream);
        if (e != cudaSuccess || !many) return e;
    }
    return launch_paged_chunk(p, D, all ? 0 : kRowsMax, max_new, at + rows_workspace_bytes(p.B, D), stream);
}

}  // namespace qoq
