// Host-side helpers of the entry points (defined in sconv_kv.cu): launches
// with programmatic dependent launch, and the caches of device properties.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "common.cuh"
#include "sconv_kv.h"

namespace sconv {

// Checks of a step call's tensors and options; fills the kernel arguments
// except num_tokens, cu_seqlens, num_seqs, eps, state_indices and err.
int host_step_params(const void* k, const void* v, int64_t row_stride, const void* conv_w_k,
                     const void* conv_w_v, const float* gamma_k, const float* gamma_v, int W,
                     int num_kv_heads, int head_dim, void* conv_state, int64_t state_pool_size,
                     const int64_t* slot_mapping, void* k_cache, void* v_cache,
                     const sconv_kv_cache_layout_t* layout, uint8_t* k_scale, uint8_t* v_scale,
                     bool mx, const sconv_kv_options_t* options, StepParams* P);

// Enqueue `fn`; SCONV_KV_OK or SCONV_KV_ERR_CUDA (text kept for
// sconv_kv_last_cuda_error).
int host_launch(const void* fn, dim3 grid, dim3 block, void** args, size_t smem, void* stream);
// Opt `fn` into `smem` bytes of dynamic shared memory; false if refused.
bool host_smem(const void* fn, size_t smem);
// SMs of the current device, and the blocks of `fn` that fit on one.
int host_sm_count();
int host_resident(const void* fn, int threads, size_t smem, int fallback);

}  // namespace sconv
