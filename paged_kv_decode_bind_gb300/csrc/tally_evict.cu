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
// A decode loop without slack is one token over at every step: the one that ranks last is
// then a minimum, and one row moves (bind and eviction of 16 requests at 2048 tokens, 8
// heads, 9.7 us; 15.3 with the select).
//
// A (request, layer, head) unit is a cluster of C CTAs (1 to 16), each with a contiguous
// segment of the request's tokens; histograms, counts and the lists of movers and free
// indices are read from the other CTAs' shared memory.  The unit that finishes last of a
// request (a ticket on split_counters) writes its new length.
//
// Measured (GB300): 64 requests of 1024-4096 tokens to 1024, 4 layers of 2 heads, 81 us, 4 x
// 65536 to 8192, 8 heads, 74 us; the choice alone 18 and 29 (launch 2, keys 7 and 9, four
// passes 6 and 14, lists 4), the rows then move at 5.1 and 5.4 TB/s.  That is what 256-byte
// rows at scattered places give: half as many rows in flight, or lookups a batch ahead, change
// nothing.  CTAs of 512 threads, two an SM: 111 and 91 us.
#include <algorithm>

#include "decode_plan.cuh"
#include "kernels.cuh"
#include "tally.cuh"

namespace pkv {

namespace {

constexpr int kEThreads = 256;
constexpr int kEWarps = kEThreads / 32;
constexpr int kEPerSM = 4;        // CTAs of an SM: some choose while others move rows
constexpr int kEMaxCluster = 16;  // (8 where the device has no room for 16)
constexpr int kESegMax = PKV_TALLY_MAX_LEN / 8;  // tokens of a CTA at most
constexpr int kEBatch = 16;       // rows that a warp moves at a time
constexpr int kECopies = 8;    // of a histogram: lanes of a warp often hit one bin
constexpr int kEPer = 8;       // keys of a thread per scan chunk

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
// 32-bit word at this CTA's shared address `addr`, in every CTA of the cluster: their sum
__device__ __forceinline__ int ld_cluster(uint32_t addr, int rank);
__device__ __forceinline__ int sum_cluster(uint32_t addr, int C) {
  int sum = 0;
  for (int c0 = 0; c0 < C; c0 += 4) {  // C is a power of two; four loads in flight
    int v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j < C) v[j] = ld_cluster(addr, c0 + j);
    sum += (v[0] + v[1]) + (v[2] + v[3]);
  }
  return sum;
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
__global__ void __launch_bounds__(kEThreads, kEPerSM)
    tally_evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t s_key[];  // [seg] keys, then the CTA's list
  __shared__ int s_hist[4][256];
  __shared__ int s_copy[kECopies][256];
  __shared__ int s_scan[2 * kEWarps];
  __shared__ unsigned long long s_last[kEWarps];
  __shared__ int s_bin[3];   // the pass's digit, how many of its keys are wanted, and all
  __shared__ int s_info[4];  // for the cluster: bad page bits, ties, free indices, movers
  // of each CTA of the cluster: free indices and movers before it, its free indices
  __shared__ int s_fbase[kEMaxCluster + 1], s_mbase[kEMaxCluster + 1], s_fcnt[kEMaxCluster];
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
  const bool one = L - a.budget == 1;
  // the token that ranks last: least key, highest index among equals
  unsigned long long last = ~0ull;
  int bad = 0;
  constexpr int KU = 8;  // keys whose loads a thread has in flight
  for (int i0 = tid; i0 < n; i0 += KU * kEThreads) {
    int page[KU], org[KU];
    float wgt[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int i = i0 + j * kEThreads;
      page[j] = i < n ? table[pl.page_of(t0 + i)] : 0;
    }
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int i = i0 + j * kEThreads;
      if (page[j] < 0 || page[j] >= pl.n_pages) {
        bad = 1;
        page[j] = 0;
      }
      if (i >= n) continue;
      const long long at = tally_at(ws, pl.n_pages, layer, page[j], g, pl.in_page(t0 + i));
      org[j] = a.t.origin[at];
      wgt[j] = a.t.weight[at];
    }
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int i = i0 + j * kEThreads;
      if (i >= n) continue;
      const uint32_t key = rank_key(wgt[j], org[j] < a.sinks || org[j] >= late);
      if (one) {
        last = min(last, ((unsigned long long)key << 32) | (uint32_t)~(t0 + i));
        continue;
      }
      s_key[i] = key;
      atomicAdd(&s_copy[lane & (kECopies - 1)][key >> 24], 1);
    }
  }
  bad = __syncthreads_or(bad);
  auto unit_sync = [&]() {
    if (C == 1) __syncthreads();
    else cluster_sync();
  };
  // every unit of the request has read its length before its ticket
  auto ticket = [&]() {
    if (rank != 0 || tid != 0) return;
    int *ctr = ws.split_counters + b;
    if (atomic_add_acq_rel_gpu(ctr, 1) == ws.n_layers * ws.n_kv_heads - 1) {
      *ctr = 0;
      ws.seq_lens[b] = a.budget;
      a.t.evicted[row] = gone + L - a.budget;
    }
  };
  constexpr int LPR = D / 8;  // lanes of a row, 16 bytes each
  if (one) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) last = min(last, __shfl_xor_sync(0xffffffffu, last, d));
    if (lane == 0) s_last[warp] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kEWarps; ++w) last = min(last, s_last[w]);
    if (tid == 0) {
      s_info[0] = bad;
      s_info[1] = (int)(uint32_t)last;
      s_info[2] = (int)(last >> 32);
    }
    unit_sync();
    if (rank == 0 && warp == 0) {
      for (int c = 0; c < C; ++c) {
        const uint32_t lo = (uint32_t)ld_cluster(smem_addr(&s_info[1]), c);
        const uint32_t hi = (uint32_t)ld_cluster(smem_addr(&s_info[2]), c);
        bad |= ld_cluster(smem_addr(&s_info[0]), c);
        last = min(last, ((unsigned long long)hi << 32) | lo);
      }
      const int to = (int)~(uint32_t)last, from = L - 1;
      if (bad) {
        if (first) atomicOr(ws.err, PKV_DEVERR_PAGE);
      } else if (to != from) {
        const int ps = table[pl.page_of(from)], pd = table[pl.page_of(to)];
        const long long sv = ((long long)ps * pl.P + pl.in_page(from)) * ws.n_kv_heads + g;
        const long long dv = ((long long)pd * pl.P + pl.in_page(to)) * ws.n_kv_heads + g;
        const long long l0 = (long long)layer * ws.pool_slots * ws.n_kv_heads;
        if (lane < 2 * LPR) {
          uint4 *pool = static_cast<uint4 *>(lane < LPR ? ws.k_pool : ws.v_pool);
          pool[(l0 + dv) * LPR + lane % LPR] = pool[(l0 + sv) * LPR + lane % LPR];
        }
        if (lane == 0) {
          const long long as = tally_at(ws, pl.n_pages, layer, ps, g, pl.in_page(from));
          const long long ad = tally_at(ws, pl.n_pages, layer, pd, g, pl.in_page(to));
          a.t.weight[ad] = a.t.weight[as];
          a.t.origin[ad] = a.t.origin[as];
        }
      }
      if (!bad) ticket();
    }
    unit_sync();  // no shared memory leaves while a neighbour may read it
    return;
  }
  {
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
    unit_sync();  // every CTA's histogram of the pass (each pass has its own)
    if (pass == 0) {
      bad = sum_cluster(smem_addr(&s_info[0]), C);
    }
    // a bin a thread, from the top
    const uint32_t bin = smem_addr(&s_hist[pass][255 - tid]);
    int cnt = 0;
    if (C == 1) cnt = s_hist[pass][255 - tid];
    else cnt = sum_cluster(bin, C);
    int above = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, above, d);
      if (lane >= d) above += v;
    }
    if (lane == 31) s_scan[warp] = above;
    __syncthreads();
    above -= cnt;
    for (int w = 0; w < warp; ++w) above += s_scan[w];
    if (above < want && want <= above + cnt) {
      s_bin[0] = 255 - tid;
      s_bin[1] = want - above;
      s_bin[2] = cnt;
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_bin[0];
    want = s_bin[1];
    equal = s_bin[2];
  }
  // every CTA of the cluster agrees on `bad`, and a request's units read the same table
  if (bad) {
    if (first) atomicOr(ws.err, PKV_DEVERR_PAGE);
    unit_sync();  // no shared memory leaves while a neighbour may read it
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
    unit_sync();
    tie_left = want;
    for (int c = 0; c < rank; ++c) tie_left -= ld_cluster(smem_addr(&s_info[1]), c);
  }
  // ---- the CTA's list: free indices below the budget, then movers past it, in order,
  // over the keys (an entry's place is never behind its token's) ----
  int ties = 0, listed = 0, freed = 0;
  for (int c0 = 0; c0 < n; c0 += kEThreads * kEPer) {
    const int i0 = c0 + tid * kEPer;
    uint32_t key[kEPer];
#pragma unroll
    for (int j = 0; j < kEPer; j += 4) {
      const uint4 k4 = i0 + j < n ? *reinterpret_cast<const uint4 *>(s_key + i0 + j)
                                  : make_uint4(0, 0, 0, 0);
      key[j] = k4.x;
      key[j + 1] = k4.y;
      key[j + 2] = k4.z;
      key[j + 3] = k4.w;
    }
    int eq = 0;
#pragma unroll
    for (int j = 0; j < kEPer; ++j) eq += i0 + j < n && key[j] == prefix;
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
  unit_sync();
  if (warp == 0) {
    const int f = lane < C ? ld_cluster(smem_addr(&s_info[2]), lane) : 0;
    const int m = lane < C ? ld_cluster(smem_addr(&s_info[3]), lane) : 0;
    int fs = f, ms = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, fs, d), y = __shfl_up_sync(0xffffffffu, ms, d);
      if (lane >= d) {
        fs += x;
        ms += y;
      }
    }
    if (lane <= kEMaxCluster) {  // those past C hold the totals
      s_fbase[lane] = fs - f;
      s_mbase[lane] = ms - m;
      if (lane < kEMaxCluster) s_fcnt[lane] = f;
    }
  }
  __syncthreads();
  // ---- the rows move: mover j of the unit to free index j, shared out evenly ----
  const int M = min(s_mbase[C], s_fbase[C]);  // equal
  constexpr int RPW = 32 / LPR;  // rows a warp instruction
  constexpr int UN = 2;          // warp instructions in flight (K and V each)
  const int sub = lane / LPR, ch = lane % LPR;
  const long long head0 = ((long long)layer * ws.pool_slots * ws.n_kv_heads + g) * LPR + ch;
  uint4 *kp = static_cast<uint4 *>(ws.k_pool) + head0;
  uint4 *vp = static_cast<uint4 *>(ws.v_pool) + head0;
  const long long slot_vecs = (long long)ws.n_kv_heads * LPR;
  for (int j0 = (rank * kEWarps + warp) * kEBatch; j0 < M; j0 += C * kEWarps * kEBatch) {
    const int j = j0 + lane, m = min(kEBatch, M - j0);
    int src = 0, dst = 0;  // slots of this lane's mover
    long long ad = 0;      // its tally entry's new place; stored behind the rows
    float w = 0.f;
    int o = 0;
    if (lane < m) {
      int cf = 0, cm = 0;
      for (int c = 1; c < C; ++c) {
        cf += j >= s_fbase[c];
        cm += j >= s_mbase[c];
      }
      const uint32_t list = smem_addr(s_key);
      const int to = ld_cluster(list + 4 * (j - s_fbase[cf]), cf);
      const int from = ld_cluster(list + 4 * (s_fcnt[cm] + j - s_mbase[cm]), cm);
      const int ps = table[pl.page_of(from)], pd = table[pl.page_of(to)];
      src = ps * pl.P + pl.in_page(from);
      dst = pd * pl.P + pl.in_page(to);
      const long long as = tally_at(ws, pl.n_pages, layer, ps, g, pl.in_page(from));
      ad = tally_at(ws, pl.n_pages, layer, pd, g, pl.in_page(to));
      w = a.t.weight[as];
      o = a.t.origin[as];
    }
#pragma unroll
    for (int k0 = 0; k0 < kEBatch; k0 += UN * RPW) {
      uint4 kx[UN], vx[UN];
      long long to[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int k = k0 + u * RPW + sub;
        const long long from = __shfl_sync(0xffffffffu, src, k) * slot_vecs;
        to[u] = __shfl_sync(0xffffffffu, dst, k) * slot_vecs;
        if (k >= m) to[u] = -1;
        if (to[u] >= 0) {
          kx[u] = kp[from];
          vx[u] = vp[from];
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        if (to[u] >= 0) {
          kp[to[u]] = kx[u];
          vp[to[u]] = vx[u];
        }
      }
    }
    if (lane < m) {
      a.t.weight[ad] = w;
      a.t.origin[ad] = o;
    }
  }
  unit_sync();  // the lists stay until every CTA has read them
  ticket();
}

template <int D>
cudaError_t launch_one(EvictArgs a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const long long units = (long long)a.batch * a.ws.n_layers * a.ws.n_kv_heads;
  auto kern = tally_evict_kernel<D>;
  static int most[64] = {0};  // CTAs of a cluster at most, by device
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int &top = most[dev & 63];
  if (top == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kESegMax * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kEMaxCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.gridDim = dim3(kEMaxCluster);
    c.blockDim = dim3(kEThreads);
    c.dynamicSmemBytes = PKV_TALLY_MAX_LEN / kEMaxCluster * 4;
    c.attrs = at;
    c.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &c) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    top = n > 0 ? kEMaxCluster : 8;
  }
  // CTAs per unit: segments of 4096 tokens at most while the cluster can grow, and more
  // CTAs while the units leave SMs idle and segments stay at 1024 tokens or more
  int C = 1;
  while (C < top && (a.max_len > 4096 * C || (units * C * 2 <= sms && a.max_len >= 2048 * C)))
    C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.cluster = C;
  a.seg = ((a.max_len + C - 1) / C + kEPer - 1) / kEPer * kEPer;
  const size_t smem = (size_t)a.seg * 4;
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
