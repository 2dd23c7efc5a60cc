// Eviction by the attention tally: for each request past the limit, layer and KV head,
// the `budget` tokens that rank first stay, and their rows move together in place.
//
// Choice.  A token's rank key is its weight as an ordered 32-bit integer (protected
// tokens above every weight, NaN below).  The key of the budget-th token comes from four
// passes of an 8-bit radix select over keys held in shared memory; tokens above it stay,
// and of those equal to it the first by index.
// Move.  Kept tokens past the budget fill, in order, the free indices below it.  Sources
// lie past the budget and destinations below, so no row that is read is written and the
// rows move in any order, each once; a compaction that kept all tokens' order would move
// every kept token behind the first gap (at 4096 -> 1024 tokens about twice the rows).
// Keys carry their rotation, so attention does not depend on a token's index.
//
// A (request, layer, head) unit is a cluster of C CTAs (1 to 8), each with a contiguous
// segment of the request's tokens; histograms, counts and the lists of movers and free
// indices are read from the other CTAs' shared memory.  The unit that finishes last of a
// request (a ticket on split_counters) writes its new length.
#include <algorithm>

#include "decode_plan.cuh"
#include "kernels.cuh"
#include "tally.cuh"

namespace pkv {

namespace {

constexpr int kEThreads = 512;
constexpr int kEWarps = kEThreads / 32;
constexpr int kEMaxCluster = 8;
constexpr int kESegMax = PKV_TALLY_MAX_LEN / kEMaxCluster;  // tokens of a CTA at most
constexpr int kECopies = 8;    // of a histogram: lanes of a warp often hit one bin
constexpr int kEPer = 4;       // keys of a thread per scan chunk

struct EvictArgs {
  pkv_workspace ws;
  pkv_tally t;
  int batch, max_len, limit, budget, sinks, recent;
  int seg;      // tokens a CTA has room for
  int cluster;  // CTAs per unit
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
}
// 32-bit word at this CTA's shared address `addr`, in CTA `rank` of the cluster
__device__ __forceinline__ int ld_cluster(uint32_t addr, int rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Larger weight, larger key; NaN lowest; a protected token above all.
__device__ __forceinline__ uint32_t rank_key(float w, bool safe) {
  if (safe) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Inclusive sum over the block of (x, y) in this thread's order; totals in *tx, *ty.
// s: 2 * kEWarps ints, free to reuse after the call's last barrier.
__device__ __forceinline__ void block_scan2(int &x, int &y, int *s, int &tx, int &ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x, d), b = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    s[warp] = x;
    s[kEWarps + warp] = y;
  }
  __syncthreads();
  int px = 0, py = 0;
  tx = ty = 0;
#pragma unroll
  for (int w = 0; w < kEWarps; ++w) {
    const int a = s[w], b = s[kEWarps + w];
    if (w < warp) {
      px += a;
      py += b;
    }
    tx += a;
    ty += b;
  }
  x += px;
  y += py;
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kEThreads, 2)
    tally_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t s_key[];  // [seg] keys, then the CTA's list
  __shared__ int s_hist[4][256];
  __shared__ int s_copy[kECopies][256];
  __shared__ int s_scan[2 * kEWarps];
  __shared__ int s_bin[2];     // the pass's digit, and how many of its keys are wanted
  __shared__ int s_info[4];    // for the cluster: bad page bits, ties, free indices, movers
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.cluster, rank = (int)cluster_rank();
  pdl_wait();
  pdl_trigger();
  const int unit = blockIdx.x / C;
  const int g = unit % ws.n_kv_heads, r0 = unit / ws.n_kv_heads;
  const int layer = r0 % ws.n_layers, b = r0 / ws.n_layers;
  const int L = ws.seq_lens[b];
  const bool first = g == 0 && layer == 0 && rank == 0 && tid == 0;
  // every exit before the first cluster barrier is the whole cluster's
  if (L < 0 || (long long)L > len_cap(ws) || L > a.max_len) {
    if (first) atomicOr(ws.err, PKV_DEVERR_LEN);
    return;
  }
  if (L <= a.limit) return;
  const int row = ws.req_pool_indices[b];
  if (row < 0 || row >= ws.max_reqs) {
    if (first) atomicOr(ws.err, PKV_DEVERR_PAGE);
    return;
  }
  const int gone = a.t.evicted[row];
  const int late = (int)min((long long)L + gone - a.recent, 0x7fffffffll);
  const int *table = ws.page_table + (long long)row * ws.max_pages_per_req;
  Plan pl;
  pl.set_pages(ws);
  const int per = (((L + C - 1) / C) + kEPer - 1) / kEPer * kEPer;  // <= a.seg
  const int t0 = min(L, rank * per), n = min(L, t0 + per) - t0;

  for (int i = tid; i < 4 * 256; i += kEThreads) (&s_hist[0][0])[i] = 0;
  for (int i = tid; i < kECopies * 256; i += kEThreads) (&s_copy[0][0])[i] = 0;
  __syncthreads();
  // ---- keys of the segment, and the histogram of their first digit ----
  int bad = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kEThreads) {
    const int t = t0 + i;
    const int page = table[pl.page_of(t)];
    uint32_t key = 0;
    if (page >= 0 && page < pl.n_pages) {
      const long long at = tally_at(ws, pl.n_pages, layer, page, g, pl.in_page(t));
      const int o = a.t.origin[at];
      key = rank_key(a.t.weight[at], o < a.sinks || o >= late);
    } else {
      bad = 1;
    }
    s_key[i] = key;
    atomicAdd(&s_copy[lane & (kECopies - 1)][key >> 24], 1);
  }
  bad = __syncthreads_or(bad);
  if (tid < 256) {
    int sum = 0;
#pragma unroll
    for (int c = 0; c < kECopies; ++c) sum += s_copy[c][tid];
    s_hist[0][tid] = sum;
  }
  if (tid == 0) s_info[0] = bad;
  // ---- radix select of the budget-th key ----
  uint32_t prefix = 0;
  int want = a.budget;  // of the keys that share the prefix, how many stay
  int equal = 0;        // keys of the cluster equal to the one found
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    if (pass > 0) {
      for (int i = tid; i < n; i += kEThreads) {
        const uint32_t key = s_key[i];
        if ((key >> (shift + 8)) == prefix) atomicAdd(&s_hist[pass][(key >> shift) & 255], 1);
      }
    }
    cluster_sync();  // every CTA's histogram of the pass (each pass has its own)
    if (pass == 0) {
      for (int c = 0; c < C; ++c) bad |= ld_cluster(smem_addr(&s_info[0]), c);
    }
    if (warp == 0) {
      // lane l: the eight bins from the top, 255 - 8 l ... 248 - 8 l
      int cnt[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cnt[j] = 0;
        for (int c = 0; c < C; ++c)
          cnt[j] += ld_cluster(smem_addr(&s_hist[pass][255 - 8 * lane - j]), c);
        sum += cnt[j];
      }
      int above = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, above, d);
        if (lane >= d) above += v;
      }
      above -= sum;  // keys in bins above this lane's
      if (above < want && want <= above + sum) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < want && want <= above + cnt[j]) {
            s_bin[0] = 255 - 8 * lane - j;
            s_bin[1] = want - above;
            s_scan[0] = cnt[j];
          }
          above += cnt[j];
        }
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_bin[0];
    want = s_bin[1];
    equal = s_scan[0];
    __syncthreads();
  }
  // every CTA of the cluster agrees on `bad`, and a request's units read the same table
  if (bad) {
    if (first) atomicOr(ws.err, PKV_DEVERR_PAGE);
    cluster_sync();  // no shared memory leaves while a neighbour may read it
    return;
  }
  // ---- ties: those of lower index stay, so each CTA needs the count before it ----
  int tie_left = 0x7fffffff;  // of this CTA's ties, how many stay (in index order)
  if (want < equal) {         // the same in the whole cluster
    int mine = 0;
    for (int i = tid; i < n; i += kEThreads) mine += s_key[i] == prefix;
    int zero = 0, tot, z;
    block_scan2(mine, zero, s_scan, tot, z);
    if (tid == 0) s_info[1] = tot;
    cluster_sync();
    tie_left = want;
    for (int c = 0; c < rank; ++c) tie_left -= ld_cluster(smem_addr(&s_info[1]), c);
  }
  // ---- the CTA's list: free indices below the budget, then movers past it, in order,
  // over the keys (an entry's place is never behind its token's) ----
  int ties = 0, listed = 0, freed = 0;
  for (int c0 = 0; c0 < n; c0 += kEThreads * kEPer) {
    const int i0 = c0 + tid * kEPer;
    uint32_t key[kEPer];
    int eq = 0;
#pragma unroll
    for (int j = 0; j < kEPer; ++j) {
      key[j] = i0 + j < n ? s_key[i0 + j] : 0u;
      eq += i0 + j < n && key[j] == prefix;
    }
    int tie = eq, dummy = 0, ttot, dtot;
    if (want < equal) {
      block_scan2(tie, dummy, s_scan, ttot, dtot);
      tie = ties + tie - eq;  // ties of this CTA before this thread's
      ties += ttot;
    } else {
      tie = -0x40000000;  // all of them stay
    }
    unsigned in_list = 0;
    int cnt = 0, fr = 0;
#pragma unroll
    for (int j = 0; j < kEPer; ++j) {
      if (i0 + j >= n) continue;
      bool kept = key[j] > prefix;
      if (key[j] == prefix) kept = tie++ < tie_left;
      const bool below = t0 + i0 + j < a.budget;
      if (below != kept) {  // free below the budget, or kept past it
        in_list |= 1u << j;
        ++cnt;
        fr += below;
      }
    }
    int x = cnt, y = fr, tx, ty;
    block_scan2(x, y, s_scan, tx, ty);  // its barriers: every key of the chunk is read
    int at = listed + x - cnt;
#pragma unroll
    for (int j = 0; j < kEPer; ++j)
      if (in_list >> j & 1) s_key[at++] = (uint32_t)(t0 + i0 + j);
    listed += tx;
    freed += ty;
  }
  if (tid == 0) {
    s_info[2] = freed;
    s_info[3] = listed - freed;
  }
  cluster_sync();
  // ---- the rows move: mover j of the unit to free index j, shared out evenly ----
  int fbase[kEMaxCluster + 1], mbase[kEMaxCluster + 1], fcnt[kEMaxCluster];
  fbase[0] = mbase[0] = 0;
#pragma unroll
  for (int c = 0; c < kEMaxCluster; ++c) {
    const int f = c < C ? ld_cluster(smem_addr(&s_info[2]), c) : 0;
    const int m = c < C ? ld_cluster(smem_addr(&s_info[3]), c) : 0;
    fcnt[c] = f;
    fbase[c + 1] = fbase[c] + f;
    mbase[c + 1] = mbase[c] + m;
  }
  const int M = min(mbase[kEMaxCluster], fbase[kEMaxCluster]);  // equal
  constexpr int LPR = D / 8;     // lanes of a row, 16 bytes each
  constexpr int RPW = 32 / LPR;  // rows a warp instruction
  constexpr int UN = 4;          // warp instructions in flight (K and V each)
  const int sub = lane / LPR, ch = lane % LPR;
  const long long head0 = ((long long)layer * ws.pool_slots * ws.n_kv_heads + g) * LPR + ch;
  uint4 *kp = static_cast<uint4 *>(ws.k_pool) + head0;
  uint4 *vp = static_cast<uint4 *>(ws.v_pool) + head0;
  const long long slot_vecs = (long long)ws.n_kv_heads * LPR;
  for (int j0 = (rank * kEWarps + warp) * 32; j0 < M; j0 += C * kEThreads) {
    const int j = j0 + lane;
    int src = 0, dst = 0;  // slots of this lane's mover
    if (j < M) {
      int cf = 0, cm = 0;
#pragma unroll
      for (int c = 1; c < kEMaxCluster; ++c) {
        cf += j >= fbase[c];
        cm += j >= mbase[c];
      }
      int fb = 0, mb = 0, fn = 0;
#pragma unroll
      for (int c = 0; c < kEMaxCluster; ++c) {
        if (c == cf) fb = fbase[c];
        if (c == cm) {
          mb = mbase[c];
          fn = fcnt[c];
        }
      }
      const uint32_t list = smem_addr(s_key);
      const int to = ld_cluster(list + 4 * (j - fb), cf);
      const int from = ld_cluster(list + 4 * (fn + j - mb), cm);
      const int ps = table[pl.page_of(from)], pd = table[pl.page_of(to)];
      src = ps * pl.P + pl.in_page(from);
      dst = pd * pl.P + pl.in_page(to);
      const long long as = tally_at(ws, pl.n_pages, layer, ps, g, pl.in_page(from));
      const long long ad = tally_at(ws, pl.n_pages, layer, pd, g, pl.in_page(to));
      a.t.weight[ad] = a.t.weight[as];
      a.t.origin[ad] = a.t.origin[as];
    }
    const int m = min(32, M - j0);
    for (int k0 = 0; k0 < m; k0 += UN * RPW) {
      uint4 kx[UN], vx[UN];
      int to[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int k = k0 + u * RPW + sub;
        const int from = __shfl_sync(0xffffffffu, src, k & 31);
        to[u] = __shfl_sync(0xffffffffu, dst, k & 31);
        if (k >= m) to[u] = -1;
        if (to[u] >= 0) {
          kx[u] = kp[from * slot_vecs];
          vx[u] = vp[from * slot_vecs];
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        if (to[u] >= 0) {
          kp[to[u] * slot_vecs] = kx[u];
          vp[to[u] * slot_vecs] = vx[u];
        }
      }
    }
  }
  cluster_sync();  // the lists stay until every CTA has read them
  if (rank == 0 && tid == 0) {
    // every unit of the request has read its length before its ticket
    int *ctr = ws.split_counters + b;
    if (atomic_add_acq_rel_gpu(ctr, 1) == ws.n_layers * ws.n_kv_heads - 1) {
      *ctr = 0;
      ws.seq_lens[b] = a.budget;
      a.t.evicted[row] = gone + L - a.budget;
    }
  }
}

template <int D>
cudaError_t launch_one(EvictArgs a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const long long units = (long long)a.batch * a.ws.n_layers * a.ws.n_kv_heads;
  // CTAs per unit: segments of 8192 tokens at most while the cluster can grow, and more
  // CTAs while the units leave SMs idle and segments stay at 1024 tokens or more
  int C = 1;
  while (C < kEMaxCluster &&
         (a.max_len > 8192 * C || (units * C * 2 <= sms && a.max_len >= 2048 * C)))
    C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.cluster = C;
  a.seg = ((a.max_len + C - 1) / C + kEPer - 1) / kEPer * kEPer;
  const size_t smem = (size_t)a.seg * 4;
  auto kern = tally_evict_kernel<D>;
  static bool set[64] = {false};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (!set[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kESegMax * 4);
    if (e != cudaSuccess) return e;
    set[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kEThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_tally_evict(const pkv_workspace &ws, const pkv_tally &t, int batch, int max_len,
                               int limit, int budget, int sinks, int recent, cudaStream_t st) {
  const int cap = (int)std::min<long long>(max_len, len_cap(ws));  // longer ones are refused
  const EvictArgs a{ws, t, batch, cap, limit, budget, sinks, recent, 0, 1};
  if (ws.head_dim == 64) return launch_one<64>(a, st);
  if (ws.head_dim == 128) return launch_one<128>(a, st);
  return cudaErrorNotSupported;
}

}  // namespace pkv
