// Launches of the 8-bit key/value cache (moe_kv8.cu, moe_kv8_attn.cu).  Apart from
// moe_internal.h, which is a source of moe_decode_kernel, too.
#pragma once

#include "moe_internal.h"

namespace moe {

int launch_kv8_append(const moe_kv8 &c, const moe_rows &k_new, const moe_rows &v_new, int M, const int32_t *pos,
                      const int32_t *counts, int *err, cudaStream_t stream);
int launch_kv8_read(const moe_kv8 &c, const int32_t *start, int n, const int32_t *lens, uint16_t *k_out, uint16_t *v_out,
                    cudaStream_t stream);
int launch_kv8_evict(const moe_kv8 &c, const moe_kv8 &d, const int32_t *lens, const float *acc, int budget, int sinks,
                     int recent, float *dacc, int32_t *idx, int32_t *lens_out, int *err, cudaStream_t stream);
size_t kv8_attn_workspace_bytes(const moe_kv8 &c, int M, bool weights);
int launch_kv8_attn(const moe_kv8 &c, const moe_rows &q, int M, const int32_t *pos, const int32_t *counts, float scale,
                    void *o, int o_type, const float *acc_in, float *acc, float decay, void *ws, int *err,
                    cudaStream_t stream);

}  // namespace moe
