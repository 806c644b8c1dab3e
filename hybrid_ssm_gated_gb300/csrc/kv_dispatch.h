// kv_dispatch.h -- launches of the key/value-cache kernels (one translation unit a family).
#pragma once

#include <cuda_runtime.h>

#include "kv_common.cuh"

namespace gdn {

// Attention and accumulation on the FP32 pipe. vec: every row can be read 16 bytes at a time.
cudaError_t launch_kv_attn(KvArgs& a, bool vec, cudaStream_t stream);
cudaError_t launch_kv_weights(KvArgs& a, bool vec, cudaStream_t stream);
// Bytes of partials that launch_kv_attn may write.
cudaError_t kv_attn_workspace(KvArgs& a, int64_t& bytes);

// Attention and accumulation on the tensor cores: whether the cache's type and sizes fit, the launches (cudaErrorNotSupported
// where the rows' addresses have no tensor map: the caller takes the other kernel), and its partials.
bool kv_tc_fits(const KvArgs& a);
cudaError_t launch_kv_attn_tc(KvArgs& a, cudaStream_t stream);
cudaError_t kv_attn_tc_workspace(KvArgs& a, int64_t& bytes);
cudaError_t launch_kv_weights_tc(const KvArgs& a, cudaStream_t stream);

// Joins the partials of an attention kernel of `grid` CTAs, on the same stream.
cudaError_t launch_kv_join(const KvArgs& a, int grid, cudaStream_t stream);

// Attention of packed prompts: on the FP32 pipe, on the tensor cores (as above), the join of either, workspaces.
cudaError_t launch_kv_prompt(KvArgs& a, bool vec, cudaStream_t stream);
cudaError_t kv_prompt_workspace(KvArgs& a, int64_t& bytes);
bool kv_prompt_tc_fits(const KvArgs& a);
cudaError_t launch_kv_prompt_tc(KvArgs& a, cudaStream_t stream);
cudaError_t kv_prompt_tc_workspace(KvArgs& a, int64_t& bytes);
cudaError_t launch_kp_join(const KvArgs& a, int grid, cudaStream_t stream);

// Norm and rotation of rows; with `cache`, keys and values go to its pages. vec: rows 16 bytes at a time.
cudaError_t launch_kv_rotate(KvRotateArgs& r, const KvArgs* cache, bool vec, cudaStream_t stream);

cudaError_t launch_kv_fork(const KvArgs& a, const int32_t* src, const int32_t* dst, const int32_t* new_pages, bool vec,
                           cudaStream_t stream);
cudaError_t launch_kv_compact(const KvArgs& a, int32_t* ws, int32_t* used, bool vec, cudaStream_t stream);

cudaError_t launch_kv_commit(const KvArgs& a, bool vec, cudaStream_t stream);
cudaError_t launch_kv_evict(const KvArgs& a, int cap, bool vec, cudaStream_t stream);

}  // namespace gdn
