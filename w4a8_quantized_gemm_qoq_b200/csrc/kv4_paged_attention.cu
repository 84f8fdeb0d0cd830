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
// 127 to 132 us with 16 to 64 of them. Which requests have few rows is known on the
// device only: N and max_new are what the buffers have room for. So where
// some may have many, both kernels run. Where all of them do, the few-rows kernel
// finds nothing, which costs 1 to 2 us (a prompt of 100 in 20.4 us, of 4096 in 234.2, without
// it 19.4 and 232.0); without it 32 decoding requests in a step with room for
// 16 rows each take 121 us, not 38.7, and 5 drafted tokens of each 126, not 76.
cudaError_t launch_paged_attention(const PagedAttnParams &p, int64_t D, int64_t max_new, void *ws,
                                   cudaStream_t stream) {
    uint8_t *at = static_cast<uint8_t *>(ws) + 256;
    const cudaError_t e = launch_paged_rows(p, D, at, stream);
    if (e != cudaSuccess || max_new * p.G <= kRowsMax) return e;
    return launch_paged_chunk(p, D, max_new, at + rows_workspace_bytes(p.B, D), stream);
}

}  // namespace qoq
