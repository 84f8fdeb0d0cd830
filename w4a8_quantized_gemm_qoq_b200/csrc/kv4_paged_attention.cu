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
// kernel, the others to the many-rows one. Both sides of it, in us with 16, 32, 48, 56 and 64
// pairs (8 KV heads), few-rows kernel / many-rows kernel:
//   32 sequences of 1500 to 4500 tokens, D 128   49/134  82/137  118/141  137/141  153/138
//   the same, D 64                               33/116  54/118   78/120   88/120  100/123
//   one of 16000 tokens, D 128                   20/46   26/47    32/48    35/49    38/50
//   4 of 2000 tokens, D 128                      15/31   19/32    23/33    23/33    26/34
// In the first, the heaviest, the sides meet at 56 pairs; in the others later.
//
// Which requests have few rows is known on the device only: N and max_new are
// what the buffers have room for. So where some may have many, both kernels run.
// Where all of them do, the few-rows kernel finds nothing, which costs 1 to 2 us (a
// prompt of 100 tokens in 20.3 us, of 4096 in 234.3; 19.2 and 232.0 without it).
// Where they do not, as in a captured step with room for 16 rows of each of 32 requests, a
// decode step takes 38.7 us and not 121, 5 drafted tokens of each 76 and not 126.
cudaError_t launch_paged_attention(const PagedAttnParams &p, int64_t D, int64_t max_new, void *ws,
                                   cudaStream_t stream) {
    uint8_t *at = static_cast<uint8_t *>(ws) + 256;
    const cudaError_t e = launch_paged_rows(p, D, at, stream);
    if (e != cudaSuccess || max_new * p.G <= kRowsMax) return e;
    return launch_paged_chunk(p, D, max_new, at + rows_workspace_bytes(p.B, D), stream);
}

}  // namespace qoq
