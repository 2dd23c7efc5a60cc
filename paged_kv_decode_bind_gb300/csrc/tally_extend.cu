// The weight that a chunk's observed queries give every token of their context
// (pkv_tally_extend), on the fifth-generation tensor cores.
//
//   weight[t, g] (+)= sum_{i, h} exp2(scale log2e q_ih . k_t - lse_ih log2e)
//
// The sum runs over queries, so keys are the rows: S^T = K Q^T with a tile of 128 keys
// as the A operand (M = 128, one TMEM lane a key) and query rows as B.  A thread then
// owns a key and adds up its lane's columns; nothing is exchanged between threads until
// a unit's partial sums meet at its end, in an order that no launch shape changes.
// A product is 128 keys x 256 query rows (256 / G tokens x the group's G heads): issuing
// eight MMAs and the hand-offs around them cost ~1200 cycles, of which the tensor cores
// work 1024; with 128 query rows they worked 512 of those.
// The log-sum-exps enter through the tensor cores too, as a ninth step of 16 dims: a key
// has 1, 1, 1, 0 ... there, a query row -lse / scale in three bf16 parts (2^-24 of it).
// Read from shared memory a column at a time they came to every lane of every warp, as
// many bytes as the products' operands (a whole 8192-token prompt 266 us, 227 without the
// reads).
//
// One persistent CTA per SM.  Two shapes of unit, by how many query tiles a request has
// at most:
//   few (one or two)  the query tiles stay in shared memory over a CTA's consecutive keys
//               of the same request and head, and only keys stream, two tiles a unit (one
//               where there are two query tiles, and room for two key tiles): the last
//               chunk of a long prompt.
//   many        a unit is two key tiles; they stay while the query tiles that see them
//               pass, each used twice.
// Units are dealt out in snake order of their cost (many) or in even runs (few).
//
// Warps: 0 loads query tiles (one tensor-map box per 64-column half: all G heads of
// 256 / G tokens) and their log-sum-exps, 1 issues the products into two 256-column TMEM
// buffers, 2-3 write units out, 4-7 copy key tiles (16-byte cp.async through the page
// table, any page size) ahead, 8-23 are four groups of four warps: two take half the
// columns each of every other product.  Every mbarrier wait is bounded (~1 s): one that
// runs out raises PKV_DEVERR_TIMEOUT and stops the CTA, which writes no further entry and
// waits (again bounded) for its copies and products before the TMEM is freed.
//
// Measured (GB300, 32/8 heads, D = 128): a whole 8192-token prompt 220 us, 1250 TFLOP/s (65 %
// of the measured bf16 burst; the tensor pipe 67 % busy, the exponentials' 59 %): a product
// takes ~1500 cycles of the issuing warp, and the costliest CTA has 15 % above the mean; the
// last 64 queries on 32768 tokens 27.4 us (2.5 TB/s of keys): the hand-offs of a unit; four
// chunks of up to 256 tokens on 820-1845 26 us: launch, first tiles, and the costliest CTA's
// 14 products in a row, where the mean is 9.7.
// Not kept: two issuing warps, a buffer each (whole prompt 277 us: their MMAs alternate and
// both finish late), key tiles by tensor-map boxes (27 us where cp.async took 26), two
// groups of loader warps (no difference).
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
constexpr int kTN = 256;           // query rows of a tile (TMEM columns)
constexpr int kMaxK = 4;           // key tiles in shared memory at most
constexpr int kMaxQ = 2;           // query tiles in shared memory at most
constexpr int kBufs = 2;           // TMEM buffers
constexpr int kGroups = 4;         // groups of four warps: two a buffer, half its columns each
constexpr int kParts = 6;          // units whose partial sums may wait to be written out
constexpr int kBadRing = 64;       // key tiles whose bad index bits are kept
constexpr int kWriteWarp = 2, kLoadWarp = 4, kSumWarp = 8;
constexpr float kScaleMin = 1e-30f;  // smaller scales give scores that are 0 beside any lse
constexpr float kDead = 0x1p126f;    // -lse / scale of a row that weighs nothing
constexpr int kXThreads = (kSumWarp + 4 * kGroups) * 32;
constexpr int kXBatch = 128;       // requests of a launch
constexpr int kXRank = 256;        // (request, key block) pairs ordered by cost
constexpr uint32_t kXTmemCols = 512;

template <int D>
struct TCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int KSTEPS = D / 16;
  static constexpr int KHALF = kTM * 128, QHALF = kTN * 128;  // a 64-column half of a tile
  static constexpr int KBYTES = HALVES * KHALF, QBYTES = HALVES * QHALF;
  // the query ring from 0, the key ring behind it: 2 + 2 tiles, or 1 + 4
  static constexpr int RINGS = 2 * QBYTES + 2 * KBYTES;
  static_assert(RINGS == QBYTES + 4 * KBYTES, "both splits fill the rings");
  // Behind them the ninth step's operands.  A key's 16 dims are 1, 1, 1, 0 ... 0, its two
  // 16-byte halves in blocks of 8 rows; of a query row only the first half is stored: its
  // second is multiplied by zeros and read from the next 8 rows' block (finite values).
  static constexpr int OFF_ONE = RINGS, OFF_LSE = OFF_ONE + kTM * 32;
  static constexpr int USED = OFF_LSE + kMaxQ * kTN * 16 + 128 + 1024;
  // one CTA an SM (it holds all of the SM's TMEM)
  static constexpr int SMEM = USED < 120 * 1024 ? 120 * 1024 : USED;
  static_assert(SMEM + 21 * 1024 <= 227 * 1024, "shared memory of one CTA");
};

// Place in a ring of n stages and the parity of the current pass over it.  A consumer
// waits for `ph` on a stage's full barrier, a producer for `ph ^ 1` on its empty barrier
// (which a fresh barrier passes).
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      ph ^= 1;
    }
  }
};

struct TallyXArgs {
  pkv_workspace ws;
  pkv_tally t;
  int b0, batch, total_batch, layer, max_qo_len, n_rows, window;
  int few;     // 1: query tiles kept over a run of keys (see above)
  int block;   // keys of a unit
  int nk, nq;  // stages of the key and the query ring
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

// One unit: nk key tiles from token t0 of request b and KV head g, and the T query
// tiles from observed token i0 on that see some of them.
struct TUnit {
  int b, g, t0, nk, i0, T;
  int L, n, q0, before;  // before: position of the first new token
  bool same;             // same request, head and query tiles as the CTA's unit before
};

template <int D, int G>
__global__ void __launch_bounds__(kXThreads, 1)
    tally_extend_kernel(const __grid_constant__ TallyXArgs a,
                        const __grid_constant__ CUtensorMap tmq) {
  using C = TCfg<D>;
  constexpr int TQ = kTN / G;  // query tokens of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[kMaxK], k_empty[kMaxK];
  __shared__ __align__(8) uint64_t q_full[kMaxQ], q_empty[kMaxQ];
  __shared__ __align__(8) uint64_t s_full[kBufs], s_free[kBufs];
  __shared__ __align__(8) uint64_t p_full[kParts], p_empty[kParts], drain;
  __shared__ float s_part[kParts][kGroups][kTM];
  __shared__ int s_bad[kBadRing];  // bad index bits of the CTA's j-th key tile
  __shared__ int4 s_req[kXBatch];      // n, L, q0, row of a request (n = 0: not served)
  __shared__ long long s_base[kXBatch];  // its first index entry
  __shared__ int s_pref[kXBatch + 1];  // key blocks of the launch's requests before
  __shared__ int s_cost[kXRank], s_order[kXRank];
  __shared__ int s_warp[kXThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hq = ws.n_q_heads, hkv = ws.n_kv_heads;
  const int block = a.block;  // keys of a unit: one key tile, or two
  if (tid < kBadRing) s_bad[tid] = 0;
  // the ninth step of the keys, and finite values behind and in the query rows'
  if (tid < kTM * 2) {
    const uint32_t at =
        sbase + C::OFF_ONE + (tid >> 4) * 256 + ((tid >> 3) & 1) * 128 + (tid & 7) * 16;
    const bool first = ((tid >> 3) & 1) == 0;
    st_shared_v4(at, first ? 0x3f803f80u : 0u, first ? 0x3f80u : 0u, 0u, 0u);
  }
  for (int e = tid; e < kMaxQ * kTN + 8; e += kXThreads)
    st_shared_v4(sbase + C::OFF_LSE + e * 16, 0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmq) : "memory");
    for (int i = 0; i < kMaxK; ++i) {
      mbar_init(&k_full[i], 4);   // the four loader warps
      mbar_init(&k_empty[i], 1);  // commit after the tile's last product
    }
    for (int i = 0; i < kMaxQ; ++i) {
      mbar_init(&q_full[i], 1);   // the loader's expect-tx arrival
      mbar_init(&q_empty[i], 1);  // commit after the tile's last product
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);  // commit after the product
      mbar_init(&s_free[i], 8);  // the eight warps that read the buffer
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&p_full[i], 4 * kGroups);
      mbar_init(&p_empty[i], kLoadWarp - kWriteWarp);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
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
  // ---- requests, and the key blocks before each ----
  {
    int cnt = 0;
    if (tid < a.batch) {
      const TReq x = treq(a, a.b0 + tid);
      if (x.kind && blockIdx.x == 0) atomicOr(ws.err, x.kind);
      const int n = x.kind ? 0 : x.n;
      s_req[tid] = make_int4(n, x.L, x.q0, x.row);
      s_base[tid] = n == 0 ? 0 : req_index(ws, a.b0 + tid).base;
      cnt = n == 0 ? 0 : (x.L + block - 1) / block;
    }
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int run = incl - cnt;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
    if (tid <= a.batch && tid <= kXBatch) s_pref[tid] = run;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = s_tmem;
  const int blocks = s_pref[a.batch];
  const long long units = (long long)blocks * hkv;

  // block w of the launch: its request (index in the launch), first token and unit
  auto block_at = [&](int w, TUnit &x) {
    int lo = 0, hi = a.batch - 1;  // last i with s_pref[i] <= w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= w) lo = mid;
      else hi = mid - 1;
    }
    const int4 r = s_req[lo];
    x.b = lo;
    x.n = r.x;
    x.L = r.y;
    x.q0 = r.z;
    x.t0 = (w - s_pref[lo]) * block;
    x.nk = block == kTM || x.t0 + kTM >= x.L ? 1 : 2;
    x.before = x.L - x.n;
    x.i0 = max(max(0, x.n - a.window), x.t0 - x.before);  // < n, as t0 < L
    x.T = (x.n - x.i0 + TQ - 1) / TQ;
  };
  const bool ranked = !a.few && blocks <= kXRank;
  if (ranked) {
    for (int w = tid; w < blocks; w += kXThreads) {
      TUnit x;
      block_at(w, x);
      s_cost[w] = x.T * x.nk;
    }
    __syncthreads();
    for (int w = tid; w < blocks; w += kXThreads) {
      const int cw = s_cost[w];
      int rank = 0;
      for (int o = 0; o < blocks; ++o) rank += s_cost[o] > cw || (s_cost[o] == cw && o < w);
      s_order[rank] = w;
    }
    __syncthreads();
  }
  // The CTA's i-th unit, x being the one before; false past the last.  few: an even run of
  // (request, head, block); else snake order over (block by cost, head).
  const long long u_lo = units * blockIdx.x / gridDim.x;
  const long long u_hi = units * (blockIdx.x + 1) / gridDim.x;
  auto unit_at = [&](int i, TUnit &x) -> bool {
    if (a.few) {
      const long long u = u_lo + i;
      if (u >= u_hi) return false;
      if (i > 0 && x.t0 + block < x.L) {  // the next keys of the same request and head
        const int was = x.i0;
        x.t0 += block;
        if (x.t0 + kTM >= x.L) x.nk = 1;
        x.i0 = max(max(0, x.n - a.window), x.t0 - x.before);
        x.same = x.i0 == was;
        if (!x.same) x.T = (x.n - x.i0 + TQ - 1) / TQ;
        return true;
      }
      const int pb = x.b, pg = x.g, pi = x.i0;
      int lo = 0, hi = a.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)s_pref[mid] * hkv <= u) lo = mid;
        else hi = mid - 1;
      }
      const int tiles = s_pref[lo + 1] - s_pref[lo];
      const int at = (int)(u - (long long)s_pref[lo] * hkv);
      const int g = at / tiles;
      block_at(s_pref[lo] + at - g * tiles, x);
      x.g = g;
      x.same = i > 0 && x.b == pb && x.g == pg && x.i0 == pi;
      return true;
    }
    const long long pos = (i & 1) ? (long long)(i + 1) * gridDim.x - 1 - blockIdx.x
                                  : (long long)i * gridDim.x + blockIdx.x;
    if (pos >= units) return false;
    const int w = (int)(pos / hkv);
    block_at(ranked ? s_order[w] : w, x);
    x.g = (int)(pos - (long long)w * hkv);
    x.same = false;
    return true;
  };

  // A bounded wait; one that runs out stops the whole CTA.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (s_abort) return false;
    if (mbar_wait_sleep(bar, parity)) return true;
    s_abort = 1;
    atomicOr(ws.err, PKV_DEVERR_TIMEOUT);
    return false;
  };
  // the decision is the warp's
  auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const bool ok = wait(bar, parity);
    return __all_sync(0xffffffffu, ok);
  };

  const float scale = fabsf(a.scale) >= kScaleMin ? a.scale : copysignf(kScaleMin, a.scale);
  const float fs = scale * kLog2e;
  const uint32_t q_base = sbase, k_base = sbase + a.nq * C::QBYTES;
  TUnit x{};
  bool dead = false;
  if (warp == 0) {
    // --------------------------------------------- query tiles ----
    Ring q;
    int loaded = 0;
    constexpr int PER = kTN / 32;
    const float inv = -1.f / scale, none = scale > 0.f ? -kDead : kDead;
    for (int i = 0; !dead && unit_at(i, x); ++i) {
      if (x.same) continue;
      for (int t = 0; t < x.T; ++t) {
        // lane: rows lane + 32 j
        float y[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int col = lane + 32 * j, it = x.i0 + t * TQ + col / G;
          y[j] = -INFINITY;
          if (it < x.n) y[j] = a.lse[(long long)(x.q0 + it) * Hq + x.g * G + col % G];
        }
        if (!wwait(&q_empty[q.s], q.ph ^ 1)) {
          dead = true;
          break;
        }
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          tma_box(q_base + q.s * C::QBYTES + h * C::QHALF, &tmq, h, x.g * G, x.q0 + x.i0 + t * TQ,
                  &q_full[q.s]);
        // a row of the ninth step: -lse / scale in three parts, then zeros
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          // an lse of -inf, NaN or +inf weighs nothing
          const float f = fabsf(y[j]) < INFINITY ? fminf(fmaxf(y[j] * inv, -kDead), kDead) : none;
          const float hi = bf16lo(pack_bf16x2(f, 0.f)), r1 = f - hi;
          const float mid = bf16lo(pack_bf16x2(r1, 0.f)), lo = r1 - mid;
          const int row = lane + 32 * j;
          st_shared_v4(sbase + C::OFF_LSE + (q.s * kTN + row) * 16, pack_bf16x2(hi, mid),
                       pack_bf16x2(lo, 0.f), 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&q_full[q.s], C::QBYTES);
        q.next(a.nq);
        ++loaded;
      }
    }
    // the last tiles may still be landing
    for (int j = max(0, loaded - a.nq); j < loaded; ++j)
      mbar_wait_bounded(&q_full[j % a.nq], (j / a.nq) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------ products ----
    constexpr uint32_t kId = umma_idesc(kTM, kTN, 0);  // both operands K-major
    const uint64_t dk = umma_desc(k_base, 16, 1024), dq = umma_desc(q_base, 16, 1024);
    const uint64_t d1 = umma_desc_plain(sbase + C::OFF_ONE, 128, 256);
    const uint64_t dl = umma_desc_plain(sbase + C::OFF_LSE, 128, 128);
    Ring kr, qr, sb;  // this unit's first key tile and query tile, the next TMEM buffer
    bool more = unit_at(0, x);
    for (int i = 0; more && !dead; ++i) {
      TUnit y = x;  // the unit after
      more = unit_at(i + 1, y);
      const bool keep = more && y.same;  // its query tiles are this unit's
      Ring qt = qr, k1 = kr;
      k1.next(a.nk);  // the second key tile
      for (int t = 0; t < x.T && !dead; ++t) {
        if (!x.same && !wwait(&q_full[qt.s], qt.ph)) {
          dead = true;
          break;
        }
        const uint64_t qd = dq + (uint64_t)((qt.s * C::QBYTES) >> 4);
        for (int c = 0; c < x.nk; ++c) {
          const Ring &kc = c ? k1 : kr;
          if ((t == 0 && !wwait(&k_full[kc.s], kc.ph)) || !wwait(&s_free[sb.s], sb.ph ^ 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint64_t kd = dk + (uint64_t)((kc.s * C::KBYTES) >> 4);
          const uint32_t acc = tmem + sb.s * kTN;
#pragma unroll
          for (int ks = 0; ks < C::KSTEPS; ++ks) {
            constexpr uint64_t kh = C::KHALF >> 4, qh = C::QHALF >> 4;
            umma_ss(acc, kd + (ks >> 2) * kh + (ks & 3) * 2, qd + (ks >> 2) * qh + (ks & 3) * 2,
                    kId, ks > 0);
          }
          // last, so that the scores' sum is rounded with the log-sum-exp once
          umma_ss(acc, d1, dl + (uint64_t)(qt.s * kTN), kId, 1);
          umma_commit(&s_full[sb.s]);
          if (t == x.T - 1) umma_commit(&k_empty[kc.s]);
          sb.next(kBufs);
        }
        if (!dead && !keep) umma_commit(&q_empty[qt.s]);
        qt.next(a.nq);
      }
      kr = k1;
      if (x.nk == 2) kr.next(a.nk);
      if (!keep) qr = qt;
      x = y;
    }
    // every product issued is done before the TMEM is freed
    umma_commit(&drain);
    mbar_wait_bounded(&drain, 0);
    __syncwarp();
  } else if (warp < kLoadWarp) {
    // ------------------------------------------- units written out ----
    Plan pl;
    pl.set_pages(ws);
    Ring pr;
    int kv = 0, kk0 = 0;  // key tiles and products before the unit
    for (int i = 0; unit_at(i, x); ++i) {
      if (!wwait(&p_full[pr.s], pr.ph)) break;
      const int row = s_req[x.b].w;
      const long long base = s_base[x.b];
      for (int c = 0; c < x.nk; ++c) {
        // a buffer's two groups; of one key tile, both buffers' have a share
        const int b0 = (kk0 + c) & 1, bad = s_bad[(kv + c) % kBadRing];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = (warp - kWriteWarp) * 64 + j * 32 + lane, t = x.t0 + c * kTM + r;
          float sum = s_part[pr.s][b0][r] + s_part[pr.s][b0 + 2][r];
          if (x.nk == 1) sum += s_part[pr.s][b0 ^ 1][r] + s_part[pr.s][(b0 ^ 1) + 2][r];
          if (t >= x.L || bad || s_abort) continue;
          int kind = 0;
          const int slot =
              (int)slot_from_raw(ws, pl, *index_src(ws, pl, ReqIndex{base, true}, t), t, kind);
          if (slot < 0) continue;
          const int page = pl.page_of(slot);
          const long long at = tally_at(ws, pl.n_pages, a.layer, page, x.g, slot - page * pl.P);
          if (t >= x.before) {
            a.t.weight[at] = sum;
            a.t.origin[at] = t + a.t.evicted[row];
          } else {
            // one addition an entry and launch: a reduction that does not wait for the
            // old value
            asm volatile("red.global.add.f32 [%0], %1;" ::"l"(a.t.weight + at), "f"(sum)
                         : "memory");
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_empty[pr.s]);
      pr.next(kParts);
      kv += x.nk;
      kk0 += x.T * x.nk;
    }
  } else if (warp < kSumWarp) {
    // ----------------------------------------------- key tiles ----
    const int ltid = tid - kLoadWarp * 32;
    Plan pl;
    pl.set_pages(ws);
    constexpr int CH = D / 8;     // 16-byte chunks of a row
    constexpr int RPI = 32 / CH;  // rows a warp instruction
    int kt = 0;                   // key tiles issued
    Ring kr, kp;                  // the stage to fill, the oldest not yet published
    // the oldest copies have landed
    auto publish = [&](int tiles) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      for (; tiles > 0; --tiles) {
        if (lane == 0) mbar_arrive(&k_full[kp.s]);
        kp.next(a.nk);
      }
    };
    // index entry of this thread's row of key tile c of unit u
    auto raw_of = [&](const TUnit &u, int c) -> int {
      const int t = u.t0 + c * kTM + ltid;
      return t < u.L ? *index_src(ws, pl, ReqIndex{s_base[u.b], true}, t) : -1;
    };
    const int lw = warp - kLoadWarp, sub = lane / CH, ch = lane % CH;
    int c = 0, i = 0;
    bool have = unit_at(0, x);
    int raw = have ? raw_of(x, 0) : -1;
    while (have) {
      TUnit y = x;  // of the tile after, whose index entries come with this tile's copies
      int c2 = c + 1;
      bool have2 = true;
      if (c2 == x.nk) {
        c2 = 0;
        have2 = unit_at(++i, y);
      }
      const int raw2 = have2 ? raw_of(y, c2) : -1;
      if (!wwait(&k_empty[kr.s], kr.ph ^ 1)) {
        dead = true;
        break;
      }
      const int t1 = x.t0 + c * kTM;
      int slot = -1, bad = 0;
      if (t1 + ltid < x.L) slot = (int)slot_from_raw(ws, pl, raw, t1 + ltid, bad);
      const uint16_t *kb = static_cast<const uint16_t *>(ws.k_pool) +
                           ((long long)a.layer * ws.pool_slots * hkv + x.g) * D + ch * 8;
      const uint32_t dst = k_base + kr.s * C::KBYTES + (ch >> 3) * C::KHALF;
#pragma unroll
      for (int j = 0; j < 32 / RPI; ++j) {
        const int rl = j * RPI + sub, sl = __shfl_sync(0xffffffffu, slot, rl), rr = 32 * lw + rl;
        // zeros past the request's end and at a bad index
        cp_async_16z(dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                     kb + (sl >= 0 ? (long long)sl * hkv * D : 0), sl >= 0 ? 16 : 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      // The writers read these bits when the unit is written out, past the arrivals on
      // p_full that follow this tile's k_full.  A warp is at most kMaxK tiles ahead of
      // another and of the products, which are at most kParts units (12 tiles) ahead of
      // the writers: the bits of half a ring ago are read, those of half a ring ahead not
      // yet set.
      if (ltid == 0) s_bad[(kt + kBadRing / 2) % kBadRing] = 0;
      bad = __reduce_or_sync(0xffffffffu, bad);
      if (bad && lane == 0) {
        atomicOr(ws.err, bad);
        atomicOr(&s_bad[kt % kBadRing], bad);
      }
      // The copies of one tile may still be under way when the next is issued (few).  A
      // unit of two tiles that fills a ring of two (many): the stage of the next tile is
      // free only once this tile's products are done, so it is published first.
      if (a.few) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (kt >= a.few) publish(1);
      ++kt;
      kr.next(a.nk);
      x = y;
      c = c2;
      raw = raw2;
      have = have2;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!dead) publish(min(kt, a.few));
  } else if (warp >= kSumWarp) {
    // ------------------------------------------------- weights ----
    const int grp = (warp - kSumWarp) >> 2, wq = warp & 3;
    const int r = 32 * wq + lane;
    // products are dealt to the buffers in turn
    const int buf = grp & 1, col0 = (grp >> 1) * (kTN / 2);
    const uint32_t src = tmem + ((uint32_t)(32 * wq) << 16) + buf * kTN + col0;
    const uint64_t fs2 = f2(fs, fs);
    int kk0 = 0;       // products before this unit
    uint32_t sph = 0;  // parity of the buffer's next product
    Ring pr;
    for (int i = 0; !dead && unit_at(i, x); ++i) {
      const int P = x.T * x.nk;
      float sum = 0.f;
      for (int p = (buf - kk0) & 1; p < P; p += kBufs) {
        const int c = x.nk == 2 ? p & 1 : 0, t = x.nk == 2 ? p >> 1 : p;
        if (!wwait(&s_full[buf], sph)) {
          dead = true;
          break;
        }
        sph ^= 1;
        tc_fence_after();
        const int it = x.i0 + t * TQ, tk = x.t0 + c * kTM;  // first query token, first key
        // columns [lo, hi) see this thread's key; those past hi weigh nothing by their
        // lse, so only lo is looked at, and only where some key of the tile is not seen
        // by all
        const int lo = (tk + r - x.before - it) * G - col0, hi = (x.n - it) * G - col0;
        const bool whole = x.before + it >= tk + kTM - 1;
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        auto add16 = [&](const uint32_t (&sv)[16], int c0, bool masked) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const uint64_t x2 =
                f2_mul(f2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), fs2);
            float w0 = ex2_approx(f2_lo(x2)), w1 = ex2_approx(f2_hi(x2));
            if (masked) {
              w0 = c0 + e >= lo ? w0 : 0.f;
              w1 = c0 + e + 1 >= lo ? w1 : 0.f;
            }
            acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2(w0, w1));
          }
        };
        uint32_t u[16], v[16];
        if (whole) {
          // the next 16 columns come while these are summed
          tmem_ld16(u, src);
#pragma unroll
          for (int c0 = 0; c0 < kTN / 2; c0 += 32) {
            tmem_wait_ld16(u);
            tmem_ld16(v, src + c0 + 16);
            add16(u, c0, false);
            tmem_wait_ld16(v);
            if (c0 + 32 < kTN / 2) tmem_ld16(u, src + c0 + 32);
            add16(v, c0 + 16, false);
          }
        } else {
#pragma unroll 1
          for (int c0 = 0; c0 < kTN / 2; c0 += 16) {
            tmem_ld16(u, src + c0);
            tmem_wait_ld16(u);
            add16(u, c0, true);
          }
        }
        const uint64_t s2 = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
        const float s1 = f2_lo(s2) + f2_hi(s2);
        if (__all_sync(0xffffffffu, s1 < INFINITY)) {
          sum += s1;
        } else {
          // A lane whose sum is not finite takes its weights one by one, those that are NaN
          // or infinite as nothing, and looks up the columns that weigh nothing by their
          // lse.  The others keep their sum: a key's weight is its own.
          float rest = 0.f;
#pragma unroll 1
          for (int c0 = 0; c0 < kTN / 2; c0 += 16) {
            tmem_ld16(u, src + c0);
            tmem_wait_ld16(u);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int col = c0 + e;
              if (col < lo || col >= hi) continue;
              const float w = ex2_approx(__uint_as_float(u[e]) * fs);
              const int i = it + (col0 + col) / G;
              const float l = a.lse[(long long)(x.q0 + i) * Hq + x.g * G + (col0 + col) % G];
              if (fabsf(l) < INFINITY) rest += tally_clean(w);
            }
          }
          sum += s1 < INFINITY ? s1 : rest;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[buf]);
      }
      if (dead || !wwait(&p_empty[pr.s], pr.ph ^ 1)) break;
      s_part[pr.s][grp][r] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[pr.s]);
      pr.next(kParts);
      kk0 += P;
    }
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
// group's G heads and 256 / G rows lands as 256 swizzled rows, row = token * G + head.
bool encode_q_map(CUtensorMap *m, const void *q, const pkv_workspace &ws, int n_rows, int G) {
  static const XTmapEncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r);
    return e == cudaSuccess && r == cudaDriverEntryPointSuccess
               ? reinterpret_cast<XTmapEncodeFn>(p)
               : nullptr;
  }();
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
    const int grid = (int)std::min<long long>(sms, tiles);
    e = launch_pdl(kern, dim3(grid), dim3(kXThreads), C::SMEM, st, a, tmq);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_tally_extend(const pkv_workspace &ws, const pkv_tally &t, int batch, int layer,
                                const int *qo_indptr, int max_qo_len, int n_rows, int window,
                                const void *q, const float *lse, float scale, cudaStream_t st) {
  const int D = ws.head_dim, G = ws.n_q_heads / ws.n_kv_heads;
  // query tiles of a request at most; rings: one query tile and four key tiles, or two
  // and two
  const long long most = ((long long)std::min(window, max_qo_len) * G + kTN - 1) / kTN;
  const int few = most <= kMaxQ, nq = most <= 1 ? 1 : 2, nk = nq == 1 ? 4 : 2;
  const int block = few && nq == 2 ? kTM : 2 * kTM;
  const TallyXArgs a{ws,  t,     0,  0,  batch,     layer, max_qo_len, n_rows, window,
                     few, block, nk, nq, qo_indptr, lse,   scale};
#define PKV_TX_CASE(DD, GG) \
  if (D == DD && G == GG) return launch_one<DD, GG>(a, q, batch, st);
  PKV_TX_CASE(128, 1) PKV_TX_CASE(128, 2) PKV_TX_CASE(128, 4) PKV_TX_CASE(128, 8)
  PKV_TX_CASE(128, 16) PKV_TX_CASE(64, 1) PKV_TX_CASE(64, 2) PKV_TX_CASE(64, 4)
  PKV_TX_CASE(64, 8) PKV_TX_CASE(64, 16)
#undef PKV_TX_CASE
  return cudaErrorNotSupported;
}

}  // namespace pkv
