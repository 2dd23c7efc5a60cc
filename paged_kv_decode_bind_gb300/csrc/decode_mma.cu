// Launches of the tensor-core decode kernel (decode_mma.cuh) and of the step's plan.
#include "decode_mma.cuh"

namespace pkv {

namespace {

// The step's plan (see pkv_plan_step): the compact plan every decode block
// would derive, and the TMA page ids of every block's first kPlanTiles tiles
// (one thread per (block, tile)).  Block 0 writes the header and the arrays.
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const __grid_constant__ pkv_workspace ws, int batch, int S, int grid,
                int apportion, int tma) {
  __shared__ int s_len[kMaxCompactBatch], s_base[kMaxCompactBatch], s_chunk[kMaxCompactBatch];
  __shared__ int s_pref[kMaxCompactBatch + 1];
  __shared__ int s_tmp[32];
  __shared__ int s_max;
  Plan pl;
  pl.set_pages(ws);
  pl.batch = batch;
  pl.hkv = ws.n_kv_heads;
  pl.S = S;
  const int budget = apportion ? grid : 0;
  const int pairs =
      batch_plan_compact(ws, batch, S, budget, s_len, s_base, s_pref, s_chunk, s_tmp, &s_max,
                         &pl.chunk);
  pl.pref = s_pref;
  pl.lens = s_len;
  pl.chunks = budget > 0 ? s_chunk : nullptr;
  pl.n_units = pairs * pl.hkv;
  int *P = ws.work_plan;
  const int tid = threadIdx.x;
  if (tma) {
    for (int item = blockIdx.x * blockDim.x + tid; item < grid * kPlanTiles;
         item += gridDim.x * blockDim.x) {
      const int blk = item / kPlanTiles, t = item - blk * kPlanTiles;
      Cursor<kMT> c;
      c.start(ws, pl, blk, grid);
      c.advance_by(ws, pl, t);
      int v[4] = {-1, -1, -1, -1};
      if (!c.done) {
        const Unit &u = c.it.un;
        const ReqIndex ri = req_index_cached(ws, s_base, u.b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = u.t0 + c.i * kMT + 16 * r;
          if (tok < u.t1 && ri.ok) v[r] = *index_src(ws, pl, ri, tok);
        }
      }
      *reinterpret_cast<int4 *>(P + kPlanFirst + item * 4) = make_int4(v[0], v[1], v[2], v[3]);
    }
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b < batch; b += blockDim.x) {
      P[kPlanPref + b] = s_pref[b];
      P[kPlanLen + b] = s_len[b];
      P[kPlanBase + b] = s_base[b];
      P[kPlanChunk + b] = budget > 0 ? s_chunk[b] : 0;
    }
    if (tid == 0) {
      P[kPlanPref + batch] = s_pref[batch];
      P[kHBatch] = batch;
      P[kHSplits] = S;
      P[kHGrid] = grid;
      P[kHUnits] = pl.n_units;
      P[kHChunk] = pl.chunk;
      P[kHMaxLen] = s_max;
      P[kHApportion] = budget > 0;
      P[kHTma] = tma;
      P[kHHkv] = pl.hkv;
      P[kHMagic] = kPlanMagic;
    }
  }
}

template <int D, int G>
cudaError_t launch_plan_one(const DecodeArgs &a, cudaStream_t st) {
  MmaShape sh;
  cudaError_t e = mma_shape<D, G, false>(a, &sh);
  if (e != cudaSuccess) return e;
  if (sh.grid <= 0 || sh.grid > kPlanMaxGrid || a.batch > kMaxCompactBatch) return cudaSuccess;
  const int items = sh.tma ? sh.grid * kPlanTiles : 1;
  const int blocks = (items + kPlanThreads - 1) / kPlanThreads;
  plan_kernel<<<blocks, kPlanThreads, 0, st>>>(a.ws, a.batch, a.num_splits, sh.grid,
                                                sh.apportion, sh.tma);
  return cudaGetLastError();
}

}  // namespace

bool decode_mma_supported(int head_dim, int group) {
  return (head_dim == 64 || head_dim == 128) &&
         (group == 1 || group == 2 || group == 4 || group == 8 || group == 16);
}

size_t plan_bytes() { return (size_t)kPlanInts * 4; }

cudaError_t launch_plan(const DecodeArgs &a, cudaStream_t st) {
  const int D = a.ws.head_dim, G = a.ws.n_q_heads / a.ws.n_kv_heads;
#define PKV_PLAN_CASE(DD, GG) \
  if (D == DD && G == GG) return launch_plan_one<DD, GG>(a, st);
  PKV_PLAN_CASE(128, 1) PKV_PLAN_CASE(128, 2) PKV_PLAN_CASE(128, 4) PKV_PLAN_CASE(128, 8)
  PKV_PLAN_CASE(128, 16) PKV_PLAN_CASE(64, 1) PKV_PLAN_CASE(64, 2) PKV_PLAN_CASE(64, 4)
  PKV_PLAN_CASE(64, 8) PKV_PLAN_CASE(64, 16)
#undef PKV_PLAN_CASE
  return cudaErrorNotSupported;
}

cudaError_t launch_decode_mma(const DecodeArgs &a, cudaStream_t st) {
  const int D = a.ws.head_dim, G = a.ws.n_q_heads / a.ws.n_kv_heads;
#define PKV_MMA_CASE(DD, GG) \
  if (D == DD && G == GG) return launch_mma_one<DD, GG, false>(a, st);
  PKV_MMA_CASE(128, 1) PKV_MMA_CASE(128, 2) PKV_MMA_CASE(128, 4) PKV_MMA_CASE(128, 8)
  PKV_MMA_CASE(128, 16) PKV_MMA_CASE(64, 1) PKV_MMA_CASE(64, 2) PKV_MMA_CASE(64, 4)
  PKV_MMA_CASE(64, 8) PKV_MMA_CASE(64, 16)
#undef PKV_MMA_CASE
  return cudaErrorNotSupported;
}

}  // namespace pkv
