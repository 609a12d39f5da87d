// Tensor-core paths of attention over a paged cache (internal).
#pragma once

#include "paged.cuh"

namespace attn {

int sm_count();  // of the current device
// Widths, types, page size and alignment that the tensor-core paths take.
bool paged_pieces_ok(const PagedP& p);

// Few new tokens a sequence: 16 or 32 rows (tokens x query heads of a group) per
// K/V head at most, by a measured rule. Bytes of workspace after the status block, and the
// launch itself, which sets the status word (nothing needs clearing).
bool paged_decode_supported(const PagedP& p, int32_t max_q);
size_t paged_decode_workspace_bytes();
cudaError_t launch_paged_decode(const PagedP& p, int32_t max_q, void* ws, cudaStream_t st);

// Any number of new tokens: 256-row blocks on tcgen05. Its plan kernel clears
// the status word and everything else that must start at zero. Workspace
// bytes after the status block, for `rows` new tokens in `batch` sequences and
// `group` query heads per K/V head.
bool paged_chunk_supported(const PagedP& p);
size_t paged_chunk_workspace_bytes(int64_t rows, int batch, int group);
cudaError_t launch_paged_chunk(const PagedP& p, void* ws, cudaStream_t st);

}  // namespace attn
