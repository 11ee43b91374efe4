// kv4_launch.cuh -- launchers of the 4-bit paged cache's kernels (host side).
#pragma once

#include "kv4.cuh"

namespace pnmix {
namespace kv4 {

cudaError_t launch_norm_rope(const pnmix_rope& rope, int n_tokens, int nq, int nk, const pnmix_rows& q,
                             const pnmix_rows& k, const uint16_t* qw, const uint16_t* kw, const int32_t* positions,
                             const pnmix_rows& qo, const pnmix_rows& ko, cudaStream_t s);
cudaError_t launch_append(const Geo& g, const Batch& bt, const pnmix_rows& k, const pnmix_rows& v, cudaStream_t s);
cudaError_t launch_append_qkv(const Geo& g, const Batch& bt, const pnmix_rope& rope, const pnmix_rows& q,
                              const pnmix_rows& k, const pnmix_rows& v, const uint16_t* qw, const uint16_t* kw,
                              const int32_t* positions, const pnmix_rows& qo, cudaStream_t s);
cudaError_t launch_read(const Geo& g, const Batch& bt, const pnmix_rows& k, const pnmix_rows& v, cudaStream_t s);

size_t attention_workspace_bytes(const Geo& g, const Batch& bt);
cudaError_t launch_attention(const Geo& g, const Batch& bt, const pnmix_rows& q, const pnmix_rows& out, void* ws,
                             cudaStream_t s);

}  // namespace kv4
}  // namespace pnmix
