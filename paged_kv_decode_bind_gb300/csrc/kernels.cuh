// Internal launch interface between the C-ABI layer (pkv_api.cu) and the
// kernel translation units.  Every launcher returns cudaGetLastError().
#pragma once

#include "common.cuh"

namespace pkv {

cudaError_t launch_bind_meta(const pkv_workspace &ws, int batch, int mode, cudaStream_t st);
cudaError_t launch_flat_index(const pkv_workspace &ws, int batch, cudaStream_t st);
cudaError_t launch_append(const pkv_workspace &ws, int batch, int layer_begin, int layer_count,
                          const void *k_new, const void *v_new, cudaStream_t st);
int meta_max_batch();

struct DecodeArgs {
  pkv_workspace ws;
  int batch;
  int layer;
  const void *q;
  float scale;
  int num_splits;
  int flags;
  const void *k_new;  // fused append source (bf16 [batch, Hkv, D]) or NULL
  const void *v_new;
  int fused_merge;    // 1: the last split of each (request, KV head) merges
  int apportion;      // tensor-core kernel: apportioned splits (set by its launcher)
};

// CUDA-core split-KV decode.  Returns cudaErrorNotSupported for shapes
// without an instantiation.
cudaError_t launch_decode_simt(const DecodeArgs &a, cudaStream_t st);
bool decode_simt_supported(int head_dim, int group);

// Tensor-core (warp mma) split-KV decode; same contract as the SIMT kernel,
// plus the fused append and merge.
cudaError_t launch_decode_mma(const DecodeArgs &a, cudaStream_t st);
// The step's split plan for the tensor-core kernel (pkv_plan_step) and the
// size of ws.work_plan it needs.
cudaError_t launch_plan(const DecodeArgs &a, cudaStream_t st);
size_t plan_bytes();
bool decode_mma_supported(int head_dim, int group);

// 8-bit cache (kv8_cache.cu, kv8_decode.cu).
struct Kv8Args;
// early: the next kernel on the stream may start before this one's predecessor
// has ended (it was launched to wait for this kernel where it must).  lens:
// requests without a usable length are passed over; NULL: every entry has a row.
cudaError_t launch_kv8_append(const pkv_workspace &ws, const pkv_kv8 &c, int batch,
                              int layer_begin, int layer_count, const void *k_new,
                              const void *v_new, bool early, const int *lens,
                              cudaStream_t st);
cudaError_t launch_kv8_extend_append(const pkv_workspace &ws, const pkv_kv8 &c, int batch,
                                     int layer, const int *qo_indptr, int max_qo_len,
                                     const void *k_new, const void *v_new, cudaStream_t st);
cudaError_t launch_kv8_read(const pkv_workspace &ws, const pkv_kv8 &c, int batch, int layer,
                            const int *starts, const int *dst_indptr, int n_rows, void *k_out,
                            void *v_out, int flags, cudaStream_t st);
cudaError_t launch_kv8_decode(const Kv8Args &a, cudaStream_t st);
bool kv8_decode_supported(int head_dim, int group);

// Norm and rotation of queries and keys (qk_norm_rope.cu).
cudaError_t launch_qk_norm_rope(const pkv_qk_norm_rope_args &p, int n_tokens, const void *q,
                                long long q_stride, const void *k, long long k_stride,
                                const int *positions, void *q_out, long long q_out_stride,
                                void *k_out, long long k_out_stride, cudaStream_t st);

cudaError_t launch_merge(const pkv_workspace &ws, int batch, int num_splits, int flags,
                         cudaStream_t st);

}  // namespace pkv
