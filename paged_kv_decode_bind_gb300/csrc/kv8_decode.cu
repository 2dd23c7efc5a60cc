// Decode attention over the 8-bit cache.
//
// One warp per (request, query head): lanes share the row of a token, one
// token at a time, with an online softmax in fp32.
#include "decode_plan.cuh"
#include "kernels.cuh"
#include "kv8.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;

template <int D, int DT>
__global__ void __launch_bounds__(kWarps * 32)
    kv8_decode_kernel(const __grid_constant__ Kv8Args a) {
  pdl_wait();
  pdl_trigger();
  const pkv_workspace &ws = a.ws;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (long long)a.batch * ws.n_q_heads) return;
  const int b = (int)(row / ws.n_q_heads), h = (int)(row - (long long)b * ws.n_q_heads);
  const int g = h / (ws.n_q_heads / ws.n_kv_heads);
  const int L = checked_len(ws, b, ws.err);
  const ReqIndex ri = req_index(ws, b);
  constexpr int E = D / 32;  // elements of a row per lane
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[row * D + lane * E + i]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  int bad = !ri.ok && L > 0 ? PKV_DEVERR_PAGE : 0;
  for (int t = 0; t < L && !bad; ++t) {
    const int slot = token_slot(ws, ri.base, t, &bad);
    if (slot < 0) break;
    const long long at = (((long long)a.layer * ws.pool_slots + slot) * ws.n_kv_heads + g) * D +
                         lane * E;
    const long long si = scale_index(ws, a.c.scale_block, a.layer, slot, g);
    uint32_t kw = 0, vw = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      kw |= (uint32_t)static_cast<const uint8_t *>(a.c.k_pool)[at + i] << (8 * i);
      vw |= (uint32_t)static_cast<const uint8_t *>(a.c.v_pool)[at + i] << (8 * i);
    }
    float k[4], v[4], s = 0.f;
    decode4<DT>(kw, k);
    decode4<DT>(vw, v);
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale * a.c.k_scale[si];
    const float mn = fmaxf(m, s), al = expf(m - mn), p = expf(s - mn);
    l = l * al + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * al + p * a.c.v_scale[si] * v[i];
  }
  if (bad && lane == 0) atomicOr(ws.err, bad);
  const bool empty = bad || L == 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float y = empty ? 0.f : o[i] / l;
    const long long at = row * D + lane * E + i;
    if (a.flags & PKV_FLAG_OUT_F32) static_cast<float *>(ws.out)[at] = y;
    else static_cast<uint16_t *>(ws.out)[at] = (uint16_t)f32_to_bf16_bits(y);
  }
  if ((a.flags & PKV_FLAG_WRITE_LSE) && lane == 0) ws.lse[row] = empty ? -INFINITY : m + logf(l);
}

template <int D, int DT>
cudaError_t launch_one(const Kv8Args &a, cudaStream_t st) {
  const long long rows = (long long)a.batch * a.ws.n_q_heads;
  return launch_pdl(kv8_decode_kernel<D, DT>, dim3((unsigned)((rows + kWarps - 1) / kWarps)),
                    dim3(kWarps * 32), 0, st, a);
}

}  // namespace

bool kv8_decode_supported(int head_dim, int group) {
  return (head_dim == 64 || head_dim == 128) &&
         (group == 1 || group == 2 || group == 4 || group == 8 || group == 16);
}

cudaError_t launch_kv8_decode(const Kv8Args &a, cudaStream_t st) {
  if (a.k_new) {
    const cudaError_t e =
        launch_kv8_append(a.ws, a.c, a.batch, a.layer, 1, a.k_new, a.v_new, st);
    if (e != cudaSuccess) return e;
  }
  const bool fp8 = a.c.dtype == PKV_KV8_E4M3;
  if (a.ws.head_dim == 128)
    return fp8 ? launch_one<128, PKV_KV8_E4M3>(a, st) : launch_one<128, PKV_KV8_INT8>(a, st);
  return fp8 ? launch_one<64, PKV_KV8_E4M3>(a, st) : launch_one<64, PKV_KV8_INT8>(a, st);
}

}  // namespace pkv
