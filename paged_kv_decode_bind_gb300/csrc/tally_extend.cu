// The weight that a chunk's observed queries give every token of their context
// (pkv_tally_extend), on the fifth-generation tensor cores.
//
//   weight[t, g] (+)= sum_{i, h} exp2(scale log2e q_ih . k_t - lse_ih log2e)
//
// The sum runs over queries, so keys are the rows: S^T = K Q^T with a tile of 128 keys
// as the A operand (M = 128, one TMEM lane a key) and 128 query rows (128 / G tokens x
// the group's G heads) as B.  A thread then owns a key and adds up its lane's columns;
// nothing is exchanged between threads until the two halves of the tiles meet at the
// end.  A CTA takes a unit (request, key tile, KV head): the key tile stays in shared
// memory while the query tiles that see it pass through a ring of tensor-map boxes, so
// an entry is written by one CTA, once, in an order that no launch shape changes.
//
// Warps: 0 loads query tiles (one box per 64-column half: all G heads of 128 / G
// tokens), 1 issues the products into two 128-column TMEM buffers, 2-5 take the even
// tiles and 6-9 the odd ones.  All ten copy the key tile (16-byte cp.async through the
// page table, any page size).  Two CTAs share an SM, so one's key tile loads while the
// other computes.  Every mbarrier wait is bounded (~1 s): one that runs out raises
// PKV_DEVERR_TIMEOUT, the CTA's warps then walk the remaining units without waiting,
// loading or writing, and the copies and products in flight are waited for before the
// TMEM is freed.
#include <algorithm>
#include <cstring>

#include "decode_plan.cuh"
#include "extend_common.cuh"
#include "kernels.cuh"
#include "tally.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr int kTM = 128;           // keys of a tile (TMEM lanes)
constexpr int kTN = 128;           // query rows of a tile (TMEM columns)
constexpr int kTStages = 2;        // query ring, and TMEM buffers
constexpr int kXThreads = 320;
constexpr int kXBatch = 1024;      // requests of a launch
constexpr uint32_t kXTmemCols = 256;

template <int D>
struct TCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int KSTEPS = D / 16;
  static constexpr int HALF = 128 * 128;  // one 64-column half of 128 rows
  static constexpr int BYTES = HALVES * HALF;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = BYTES;
  // two CTAs an SM and no third: each holds half of the SM's 512 TMEM columns
  static constexpr int USED = OFF_Q + kTStages * BYTES + 1024;
  static constexpr int SMEM = USED < 90 * 1024 ? 90 * 1024 : USED;
};

struct TallyXArgs {
  pkv_workspace ws;
  pkv_tally t;
  int b0, batch, total_batch, layer, max_qo_len, n_rows, window;
  const int *qo_indptr;
  const float *lse;
  float scale;
};

// Request b as a launch sees it: n new tokens from row q0, L cached with them.
struct TReq {
  int n, L, q0, row;
  int kind;  // error bits, 0 where it is served
};

__device__ __forceinline__ TReq treq(const TallyXArgs &a, int b) {
  const pkv_workspace &ws = a.ws;
  TReq x;
  x.q0 = a.qo_indptr[b];
  const long long n = (long long)a.qo_indptr[b + 1] - x.q0;
  x.n = (int)n;
  x.L = ws.seq_lens[b];
  x.row = ws.req_pool_indices[b];
  x.kind = 0;
  if (x.L < 0 || (long long)x.L > len_cap(ws) || n < 0 || n > x.L || n > a.max_qo_len ||
      x.q0 < 0 || x.q0 + n > a.n_rows || x.q0 + n > a.qo_indptr[a.total_batch]) {
    x.kind = PKV_DEVERR_LEN;
  } else if (n > 0 && (x.row < 0 || x.row >= ws.max_reqs)) {
    x.kind = PKV_DEVERR_PAGE;
  } else if (n > 0 && ws.index_mode == PKV_IDX_FLAT) {
    const int base = ws.kv_indptr[b];
    if (base < 0 || (long long)base + x.L > ws.max_total_tokens) x.kind = PKV_DEVERR_TOTAL;
  }
  return x;
}

__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

template <int D, int G>
__global__ void __launch_bounds__(kXThreads, 2)
    tally_extend_kernel(const __grid_constant__ TallyXArgs a,
                        const __grid_constant__ CUtensorMap tmq) {
  using C = TCfg<D>;
  constexpr int TQ = kTN / G;  // query tokens of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[kTStages], q_empty[kTStages];
  __shared__ __align__(8) uint64_t s_full[kTStages], s_free[kTStages], drain;
  __shared__ int s_pref[kXBatch + 1];
  __shared__ int s_warp[kXThreads / 32];
  // -lse log2e of a tile's columns: [half of the tiles][parity of its tile][column]
  __shared__ __align__(16) float s_lse[2][2][kTN];
  __shared__ float s_part[kTM];
  __shared__ int s_bad;  // serial number of the last unit that met a bad index
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hq = ws.n_q_heads, hkv = ws.n_kv_heads;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmq) : "memory");
    for (int i = 0; i < kTStages; ++i) {
      mbar_init(&q_full[i], 1);   // the loader's expect-tx arrival
      mbar_init(&q_empty[i], 1);  // commit after the tile's products
      mbar_init(&s_full[i], 1);   // the same commit
      mbar_init(&s_free[i], 4);   // the four warps that read the buffer
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    s_bad = -1;
    fence_barrier_init();
  }
  // TMEM is taken once the previous kernel is done (its CTAs may want all of it), and
  // the next one may start once this CTA has its own.
  pdl_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&s_tmem)),
                 "r"(kXTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ---- units: s_pref[i] = key tiles of the launch's requests before the i-th ----
  {
    constexpr int PER = (kXBatch + kXThreads - 1) / kXThreads;
    int cnt[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j;
      cnt[j] = 0;
      if (i < a.batch) {
        const TReq x = treq(a, a.b0 + i);
        if (x.kind && blockIdx.x == 0) atomicOr(ws.err, x.kind);
        cnt[j] = x.kind || x.n == 0 ? 0 : (x.L + kTM - 1) / kTM;
      }
      sum += cnt[j];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j;
      if (i <= a.batch) s_pref[i] = run;
      run += cnt[j];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = s_tmem;
  const long long units = (long long)s_pref[a.batch] * hkv;

  // A bounded wait; one that runs out stops the whole CTA.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (s_abort) return false;
    if (mbar_wait_sleep(bar, parity)) return true;
    s_abort = 1;
    atomicOr(ws.err, PKV_DEVERR_TIMEOUT);
    return false;
  };
  auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };

  Plan pl;
  pl.set_pages(ws);
  const float fs = a.scale * kLog2e;
  int k = 0;       // query tiles of the CTA so far (the same count in every warp)
  int issued = 0;  // loader: tiles whose boxes it issued
  int serial = 0;
  for (long long u = blockIdx.x; u < units; u += gridDim.x, ++serial) {
    const int w = (int)(u / hkv), g = (int)(u - (long long)w * hkv);
    int lo = 0, hi = a.batch - 1;  // last i with s_pref[i] <= w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= w) lo = mid;
      else hi = mid - 1;
    }
    const int b = a.b0 + lo;
    const TReq x = treq(a, b);
    const int t0 = (w - s_pref[lo]) * kTM;
    const int before = x.L - x.n;  // position of the first new token
    // observed queries that see some key of the tile: [i0, n)
    const int i0 = max(max(0, x.n - a.window), t0 - before);
    const int T = (x.n - i0 + TQ - 1) / TQ;  // >= 1: t0 < L
    const ReqIndex ri = req_index(ws, b);
    __syncthreads();  // the unit before is done with the key tile and s_part
    if (warp == 0) {
      // the first query tiles, while the keys come
      for (int t = 0; t < min(T, kTStages); ++t) {
        const int kk = k + t, s = kk % kTStages;
        if (kk >= kTStages && !wwait(&q_empty[s], ((kk / kTStages) - 1) & 1)) continue;
        if (__any_sync(0xffffffffu, s_abort)) continue;
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          tma_box(sbase + C::OFF_Q + s * C::BYTES + h * C::HALF, &tmq, h, g * G, x.q0 + i0 + t * TQ,
                  &q_full[s]);
        if (lane == 0) mbar_arrive_expect_tx(&q_full[s], C::BYTES);
        issued = kk + 1;
      }
    }
    // ---- the key tile, 16 bytes a thread, zeros past the request's end ----
    {
      constexpr int CH = D / 8;
      const long long head0 = ((long long)a.layer * ws.pool_slots * hkv + g) * D;
      const uint16_t *kb = static_cast<const uint16_t *>(ws.k_pool) + head0;
      int bad = 0;
      for (int e = tid; e < kTM * CH; e += kXThreads) {
        const int r = e / CH, c = e % CH, t = t0 + r;
        long long slot = -1;
        if (t < x.L) {
          int kind = 0;
          slot = slot_from_raw(ws, pl, *index_src(ws, pl, ri, t), t, kind);
          bad |= kind;
        }
        cp_async_16z(sbase + C::OFF_K + (c >> 3) * C::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     kb + (slot >= 0 ? slot * hkv * D + c * 8 : 0), slot >= 0 ? 16 : 0);
      }
      if (bad) {
        atomicOr(ws.err, bad);
        s_bad = serial;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    if (warp == 0) {
      for (int t = kTStages; t < T; ++t) {
        const int kk = k + t, s = kk % kTStages;
        if (!wwait(&q_empty[s], ((kk / kTStages) - 1) & 1) || __any_sync(0xffffffffu, s_abort))
          break;
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          tma_box(sbase + C::OFF_Q + s * C::BYTES + h * C::HALF, &tmq, h, g * G, x.q0 + i0 + t * TQ,
                  &q_full[s]);
        if (lane == 0) mbar_arrive_expect_tx(&q_full[s], C::BYTES);
        issued = kk + 1;
      }
    } else if (warp == 1) {
      constexpr uint32_t kId = umma_idesc(kTM, kTN, 0);
      const uint64_t dk = umma_desc(sbase + C::OFF_K, 16, 1024);
      const uint64_t dq = umma_desc(sbase + C::OFF_Q, 16, 1024);
      tc_fence_after();
      for (int t = 0; t < T; ++t) {
        const int kk = k + t, s = kk % kTStages;
        if (!wwait(&q_full[s], (kk / kTStages) & 1) ||
            (kk >= kTStages && !wwait(&s_free[s], ((kk / kTStages) - 1) & 1)))
          break;
        tc_fence_after();
        const uint64_t qs = dq + (uint64_t)((s * C::BYTES) >> 4);
#pragma unroll
        for (int ks = 0; ks < C::KSTEPS; ++ks) {
          const uint64_t off = (uint64_t)(((ks >> 2) * C::HALF + (ks & 3) * 32) >> 4);
          umma_ss(tmem + s * kTN, dk + off, qs + off, kId, ks > 0);
        }
        umma_commit(&s_full[s]);
        umma_commit(&q_empty[s]);
      }
    } else {
      // -------------------------------------------------- weights ----
      const int half = (warp - 2) >> 2, wq = warp & 3;
      const int r = 32 * wq + lane, col = r;
      const uint32_t trow = tmem + ((uint32_t)(32 * wq) << 16);
      const int t_key = t0 + r;
      const uint64_t fs2 = f2(fs, fs);
      // -lse log2e of this thread's column of tile t; -inf: the column weighs nothing
      auto lse_of = [&](int t) -> float {
        const int i = i0 + t * TQ + col / G;
        if (t >= T || i >= x.n) return -INFINITY;
        const float l = a.lse[(long long)(x.q0 + i) * Hq + g * G + col % G];
        return l > -INFINITY ? -l * kLog2e : -INFINITY;
      };
      float sum = 0.f;
      const int first = (k & 1) == half ? 0 : 1;  // tile kk belongs to half kk & 1
      float nl = lse_of(first);
      for (int t = first; t < T; t += 2) {
        const int kk = k + t, s = kk % kTStages, par = (kk >> 1) & 1;
        float *lt = s_lse[half][par];
        lt[col] = nl;
        named_sync(1 + half, 128);
        nl = lse_of(t + 2);
        const bool ok = wait(&s_full[s], (kk / kTStages) & 1);
        const bool alive = __all_sync(0xffffffffu, ok);
        const int it = i0 + t * TQ;  // the tile's first query token
        // columns [c_lo, c_hi) see this thread's key
        const int c_lo = max(0, (t_key - before - it) * G), c_hi = min(kTN, (x.n - it) * G);
        const bool whole = before + it >= t0 + kTM - 1 && it + TQ <= x.n;  // tile-uniform
        if (alive) {
          tc_fence_after();
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
          for (int c0 = 0; c0 < kTN; c0 += 32) {
            uint32_t sv[32];
            tmem_ld32(sv, trow + s * kTN + c0);
            tmem_wait_ld();
            if (c0 == kTN - 32) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_free[s]);
            }
            uint64_t part[2] = {0ull, 0ull};
            if (whole) {
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float4 l4 = *reinterpret_cast<const float4 *>(lt + c0 + c);
                const uint64_t x0 = f2_fma(f2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                           fs2, f2(l4.x, l4.y));
                const uint64_t x1 =
                    f2_fma(f2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), fs2,
                           f2(l4.z, l4.w));
                part[0] = f2_add(part[0], f2(ex2_approx(f2_lo(x0)), ex2_approx(f2_hi(x0))));
                part[1] = f2_add(part[1], f2(ex2_approx(f2_lo(x1)), ex2_approx(f2_hi(x1))));
              }
            }
            const uint64_t p2 = f2_add(part[0], part[1]);
            const float p = f2_lo(p2) + f2_hi(p2);
            if (!whole || p != p) {
              // masked columns, and weights that are NaN, one by one
              float clean = 0.f;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float e = ex2_approx(fmaf(__uint_as_float(sv[c]), fs, lt[c0 + c]));
                clean += c0 + c >= c_lo && c0 + c < c_hi ? tally_clean(e) : 0.f;
              }
              sum += clean;
            } else {
              acc[0] = f2_add(acc[0], p2);
            }
          }
          sum += f2_lo(acc[0]) + f2_hi(acc[0]);
        }
      }
      if (half == 1) s_part[r] = sum;
      named_sync(3, 256);
      if (half == 0 && t_key < x.L && s_bad != serial && !s_abort) {
        sum += s_part[r];
        int kind = 0;
        const long long slot = slot_from_raw(ws, pl, *index_src(ws, pl, ri, t_key), t_key, kind);
        if (slot >= 0) {
          const int page = pl.page_of((int)slot);
          const long long at =
              tally_at(ws, pl.n_pages, a.layer, page, g, (int)slot - page * pl.P);
          if (t_key >= before) {
            a.t.weight[at] = sum;
            a.t.origin[at] = t_key + a.t.evicted[x.row];
          } else {
            a.t.weight[at] += sum;
          }
        }
      }
    }
    k += T;
  }
  // copies and products in flight end before the CTA does
  if (warp == 0) {
    for (int kk = max(0, issued - kTStages); kk < issued; ++kk)
      mbar_wait_bounded(&q_full[kk % kTStages], (kk / kTStages) & 1);
  } else if (warp == 1) {
    umma_commit(&drain);
    mbar_wait_bounded(&drain, 0);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kXTmemCols)
                 : "memory");
  }
}

// q [n_rows, Hq, D] as (64 columns, 64-column half, head, row): a box of one half, the
// group's G heads and 128 / G rows lands as 128 swizzled rows, row = token * G + head.
bool encode_q_map(CUtensorMap *m, const void *q, const pkv_workspace &ws, int n_rows, int G) {
  static XTmapEncodeFn fn = nullptr;
  static bool tried = false;
  if (!tried) {
    tried = true;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<XTmapEncodeFn>(p);
  }
  if (!fn) return false;
  const cuuint64_t D = (cuuint64_t)ws.head_dim, H = (cuuint64_t)ws.n_q_heads;
  const cuuint64_t dims[4] = {64, D / 64, H, (cuuint64_t)n_rows};
  const cuuint64_t strides[3] = {128, D * 2, H * D * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)G, (cuuint32_t)(kTN / G)};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int G>
cudaError_t launch_one(TallyXArgs a, const void *q, int batch, cudaStream_t st) {
  using C = TCfg<D>;
  auto kern = tally_extend_kernel<D, G>;
  static bool set[64] = {false};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (e = device_sms(&sms)) != cudaSuccess) return e;
  if (!set[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev & 63] = true;
  }
  CUtensorMap tmq;
  memset(&tmq, 0, sizeof(tmq));
  if (!encode_q_map(&tmq, q, a.ws, a.n_rows, G)) return cudaErrorNotSupported;
  for (a.b0 = 0; a.b0 < batch; a.b0 += kXBatch) {
    a.batch = std::min(kXBatch, batch - a.b0);
    const long long tiles = (len_cap(a.ws) + kTM - 1) / kTM * a.batch * a.ws.n_kv_heads;
    const int grid = (int)std::min<long long>(2ll * sms, tiles);
    e = launch_pdl(kern, dim3(grid), dim3(kXThreads), C::SMEM, st, a, tmq);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_tally_extend(const pkv_workspace &ws, const pkv_tally &t, int batch, int layer,
                                const int *qo_indptr, int max_qo_len, int n_rows, int window,
                                const void *q, const float *lse, float scale, cudaStream_t st) {
  const TallyXArgs a{ws, t, 0, 0, batch, layer, max_qo_len, n_rows, window, qo_indptr, lse, scale};
  const int D = ws.head_dim, G = ws.n_q_heads / ws.n_kv_heads;
#define PKV_TX_CASE(DD, GG) \
  if (D == DD && G == GG) return launch_one<DD, GG>(a, q, batch, st);
  PKV_TX_CASE(128, 1) PKV_TX_CASE(128, 2) PKV_TX_CASE(128, 4) PKV_TX_CASE(128, 8)
  PKV_TX_CASE(128, 16) PKV_TX_CASE(64, 1) PKV_TX_CASE(64, 2) PKV_TX_CASE(64, 4)
  PKV_TX_CASE(64, 8) PKV_TX_CASE(64, 16)
#undef PKV_TX_CASE
  return cudaErrorNotSupported;
}

}  // namespace pkv
