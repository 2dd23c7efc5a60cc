// Split-KV GQA decode attention over the 8-bit cache, on warp-level fp16
// tensor-core products.
//
// Math.  For a unit (request b, KV head g, split c) both products keep the
// token (or head_dim) axis on the 16-row side of mma.m16n8k16 and the query
// group on the 8-wide side:  S^T = K Q_g^T (16 tokens x 8 heads) and
// O^T += V^T W^T (16 dims x 8 heads).  Codes become fp16 exactly (e4m3 and
// int8 both fit its 11-bit mantissa), Q is a bf16 row times a power of two
// that puts its largest element near 2^14, so it is exact too except for
// elements 2^-28 below that; products accumulate in fp32.
//
// The block scales stay out of the products.  A token's score is
//   x_t = (q . code_k,t) * k_scale_t * scale,  and its weight in O
//   w_t = exp(x_t - r) * v_scale_t,
// with a reference r that follows max(x_t + ln max(v_scale_t, 2^-80)): the
// largest w_t is then 2^8 .. 2^16, which fp16 holds whatever the value scales
// are, while the softmax sum  l = sum exp(x_t - r)  stays in fp32.  out = O / l.
// The floor of 2^-80 is for l: a block of zeros has v_scale = 2^-100, and terms
// of 2^116 each would pass fp32's range from 4096 such tokens on; no term is
// now above 2^96, so 2^31 tokens stay below 2^127.
//
// w goes into the product as two fp16 parts, what fp16 towards zero keeps and
// what that leaves, 2^-20 of w together (weights under 2^-12 of the largest: 2^-32
// of the largest; where all value scales that count lie below 2^-80, that is
// 2^-12, at 2^-100).  One part, 2^-11, put as many bf16 outputs on the other side
// of a rounding step as 0.0008 of their size, and showed in fp32 outputs.  Up to
// four heads a group leave half the columns of the product empty: the low parts
// go there for 11 instructions a piece, the queries standing in Q^T twice.  Eight
// and sixteen heads take a second product (4 x 65536 tokens, 4 heads a group 91.4 us,
// 91.1 with one part; 64 x 1024-4096, 8 heads 24.0 and 23.8, 16 heads 31.1 and 29.7).
// r moves only when a weight (at the floored scale) would pass fp16's range, so most
// tokens need one vote instead of a maximum over lanes and a rescaling of O.
//
// Data.  Each warp takes every W-th piece of 16 tokens of the unit and fills
// its own ring of stages, so no block barrier stands between a copy and its
// product.  A stage is the piece's K rows then its V rows, D bytes each, with
// the 16-byte chunks swizzled (TMA's 128- or 64-byte pattern).  Pages of whole
// pieces come as one TMA box for K and one for V, completing on the stage's
// mbarrier; other page sizes and flat indices as 16-byte cp.async copies of
// the rows (whole rows per 8 or 4 lanes), the index entries NS pieces ahead.
// Fragments are read with plain 16-byte loads: which token a row of S^T is, and which head_dim an index of
// the contraction is, is free as long as V and Q agree.  K: lane (r = lane / 4,
// c = lane % 4) takes 16 bytes of token perm(r); V: 16 (8 at D = 64) bytes of
// the tokens perm(2 c), perm(2 c + 1) (+ 8), whose bytes one byte permute per
// word interleaves into the (token, token) pairs of the A fragments of O^T.
// perm is chosen so that both reads touch every bank once.
//
// The warps' states meet in shared memory at the end of a unit, in the stage
// that the warp's last piece left free, while the next unit's pieces are on
// their way; the splits of a request meet in the block that finishes last (an
// atomic ticket).
//
// Measured (GB300, 2070 MHz; a pass in a graph): 4 x 65536 tokens, 32/8 heads, int8
// 91 us, 5.9 TB/s, 88 % of the copy rate; 64 x 1024-4096, 16/2 heads 24.0 us,
// 3.3 TB/s; 16 flat contexts of 1-8192, 19.6 us, 2.3 TB/s; 4 x 512-2048 9.5 us.
// The bound of the long case is the warps' own latency (364 instructions a piece for
// e4m3, 460 for int8 at four heads a group, four warps a scheduler, IPC 2.0 for int8;
// they waited for data in 8 of 86 us), that of the short ones the chain lengths -
// page ids - tile - meeting - ticket - merge.  Two stages beat three (94 against
// 96 us, flat 20.5 against 23.7 when that was measured): the first tile does not
// wait behind two more.
#include <cuda.h>

#include <cstring>

#include "decode_plan.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "merge.cuh"

namespace pkv {

namespace {

template <int D, int G>
struct KCfg {
  static constexpr int NH = (G + 7) / 8;           // 8-wide head tiles
  // the weights' low parts: in the columns G .. 2 G - 1 of the head tile, or in
  // products of their own
  static constexpr bool LOCOL = G <= 4;
  // warps (16 heads: twice the registers); one block of sixteen was no faster
  // (93.0 against 93.5 us at 4 x 65536, 25.4 against 23.6 at 64 x 1024-4096)
  static constexpr int W = NH == 1 ? 8 : 4;
  static constexpr int THREADS = W * 32;
  static constexpr int KB = 16 * D;                // K (or V) bytes of a piece
  static constexpr int STAGE = 2 * KB;
  static constexpr int NS = W == 8 ? (D == 128 ? 2 : 2) : (D == 128 ? 3 : 4);  // ring stages
  static constexpr int VB = D / 8;                 // V bytes of a row per lane
  static constexpr int SMEM = W * NS * STAGE + 1024;  // + alignment slack
  static_assert(STAGE == 8 * D * 4, "a stage holds a warp's O for 8 heads");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int c0, int c1,
                                            int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same, towards zero.
__device__ __forceinline__ uint32_t pack_f16x2_rz(float lo, float hi) {
  uint32_t d;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// x without its first 11 bits (those that fp16 towards zero keeps) where `mask` is
// kHighBits, x itself where it is 0.
constexpr uint32_t kHighBits = 0xffffe000u;
__device__ __forceinline__ float low_part(float x, uint32_t mask) {
  return x - __uint_as_float(__float_as_uint(x) & mask);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Token (of 8) that row r of S^T stands for, and the byte offset of a row's
// 16-byte chunk in a stage.
template <int D>
__device__ __forceinline__ int perm(int r) {
  return D == 128 ? (r & 6) ^ ((r & 1) * 5) : (((r >> 1) & 1) | (r & 4)) ^ ((r & 1) * 3);
}
template <int D>
__device__ __forceinline__ int swz(int row, int chunk) {
  return row * D + ((chunk ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

// Bytes 0, 1 and bytes 2, 3 of a word of codes as two pairs of fp16.
template <int DT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (DT == PKV_KV8_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 0x64uu is 1024 + u for u = code + 128; minus 1152 leaves the code
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const uint32_t k = 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(k));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(k));
  }
}

// A unit of work: tokens [t0, t1) of (request b, KV head g), split c of n.
struct KUnit {
  int b, g, c, n, t0, t1;
  int bad;         // error bits
  int fresh;       // first token of the block that this call appends to
  long long base;  // where the request's index entries start
  long long srow;  // scale index of (layer, page 0, head g)
  long long row0;  // byte of (layer, slot 0, head g) in a code pool
};

// A block's units in order.
//
// Shared out (S > 1): the requests, one after the other, make a line of 16-token
// pieces.  The blocks form groups of Hkv, one block per KV head, and each group
// takes a run of q pieces, so every block has the same number whatever the lengths
// are; a run that crosses the end of a request becomes two units.  The heads of a
// token lie side by side in the pool, so the blocks of a group read whole DRAM pages
// between them (with runs over one head after the other 4 x 65536 tokens took
// 138 us, not 96).  Each request counts kUnitCost pieces more than it has, in front:
// what a block spends on starting and finishing a unit (2 us against 0.2 us for a
// piece, D = 128 and up to 8 heads).  One number for all shapes: of 4, 8, 14, 20 and
// 28, 14 was within 6 % of the best for each and 20 within 3 (16 flat contexts 24.3 /
// 21.3 / 19.4 / 19.7 / 20.3 us, 4 x 512-2048 11.7 / 9.3 / 9.3 / 9.3 / 9.8, 64 x
// 1024-4096 24.5 / 24.1 / 23.8 / 23.0 / 22.5, with 16 heads a group 31.3 / 30.9 / 29.9
// / 29.2 / 29.6, with D = 64 20.2 / 19.8 / 19.2 / 19.1 / 18.6).
// q = ceil(line / groups), at least 8 (one piece per warp) and at least
// ceil(longest request / (S - 1)), so that none lies in more than S runs: two runs
// may cut a request anywhere.  Few splits then leave few shares (S = 2: one request
// whole), so where that bound is the larger one and fixed chunks, which start with
// the request, give a block less, those are taken (65536 tokens, 8 heads: S = 2
// 233 us, was 446, S = 3 161, was 228, S = 8 66, was 73; 64 x 8192, 2 heads, S = 2
// 52, was 84; the decision costs a short batch 0.1 us).
// A block keeps the line of up to kMaxCompactBatch requests in shared memory.
// Of more it keeps where each thread's few requests start, and walks on from
// there (300 requests of 100-900 tokens 29 us, against 49 with fixed chunks;
// tables for 1024 requests would cost the gathering form its L1: 16 flat
// contexts 20.6 us, against 19.0 then).
// Whole pairs (S == 1), or fixed chunks (as above, or fewer blocks than heads):
// unit u = (split, request, head), every gridDim.x-th one from blockIdx.x.
constexpr int kUnitCost = 14;

struct KUnits {
  int q;                   // pieces of a run; 0: whole pairs or fixed chunks
  int pos, end, b, chunk;  // pos, end: of the line, or unit numbers
  int at;                  // where request b starts (batches past the tables)
  int group, head;         // the block's, where shared out
};

// Pieces of a request in the line.
__device__ __forceinline__ int line_pieces(int len) {
  return len > 0 ? kUnitCost + ((len + 15) >> 4) : 0;
}

// PAGED: pages hold whole 16-token pieces, loaded as TMA boxes.
template <int D, int G, int DT, bool PAGED>
__global__ void __launch_bounds__(KCfg<D, G>::THREADS, 2)
    kv8_decode_kernel(const __grid_constant__ Kv8Args a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
  using C = KCfg<D, G>;
  constexpr int W = C::W, NS = C::NS, NH = C::NH;
  // log2 of the largest weight where r is placed, and the weight at which it moves
  constexpr float kPlace = 8.f, kMove = 65504.f;  // fp16's largest number
  constexpr float kScaleFloor = 8.271806125530277e-25f;  // 2^-80
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[PAGED ? W : 1][NS];
  __shared__ int s_pref[kMaxCompactBatch + 1];
  __shared__ int s_len[kMaxCompactBatch];
  __shared__ int s_base[kMaxCompactBatch];
  // scales of tokens t and t + 8 of a piece: (K, K, V, V) at [4 t]
  __shared__ __align__(16) float s_scale[W][NS][32];
  __shared__ int s_idx[PAGED ? 1 : W][PAGED ? 1 : 2 * NS][16];
  __shared__ float2 s_ml[W][16];
  __shared__ int s_slot[W];  // ring slot holding a warp's O, -1: it had no piece
  __shared__ int s_bad[W];
  __shared__ KUnits s_us;
  __shared__ KUnit s_unit[3];  // the current unit, the next, the one after
  __shared__ int s_plan;       // most pieces of a pair / longest length
  __shared__ int s_merge[2][3];  // splits to merge (0: not by this block), request, head
  __shared__ int s_seen[PAGED ? 1 : W][NS];  // index entries fetched by a stage's fill
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int Hq = ws.n_q_heads, H = ws.n_kv_heads;
  if constexpr (PAGED) {
    // a warp is the only user of its barriers
    if (lane < NS) mbar_init(&s_bar[warp][lane], 1);
    fence_barrier_init();
    __syncwarp();
  }
  bool waited = false;
  auto wait_previous = [&]() {
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
  };
  if (!(a.flags & PKV_FLAG_PLAN_EARLY)) wait_previous();

  // ---- the block's share ----
  Plan pl;
  pl.set_pages(ws);
  const bool compact = a.batch <= kMaxCompactBatch;
  // a block's run of a line of `run` pieces, the longest request having `most`
  auto share = [&](int run, int most) {
    const int groups = (int)gridDim.x / H, group = (int)blockIdx.x / H;
    KUnits us;
    us.group = group;
    us.head = (int)blockIdx.x - group * H;
    us.q = max((run + groups - 1) / groups, 8);
    const int least = (most - kUnitCost + a.num_splits - 2) / (a.num_splits - 1);
    if (least > us.q) {
      us.q = least;
      const int units = a.num_splits * a.batch * H;
      const int chunk = split_chunk(16 * (most - kUnitCost), a.num_splits, ws.page_size);
      const int each = (units + (int)gridDim.x - 1) / (int)gridDim.x;
      if ((long long)each * ((chunk + 15) / 16 + kUnitCost) < least) {
        us.q = us.b = 0;
        us.chunk = chunk;
        us.pos = blockIdx.x;
        us.end = units;
        return us;
      }
    }
    const long long first = group < groups ? (long long)group * us.q : run;
    us.pos = (int)min(first, (long long)run);
    us.end = (int)min(first + us.q, (long long)run);
    return us;
  };
  // the last of n entries of s_pref that is not past pos
  auto find = [&](int n, int pos) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= pos) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  if (compact) {
    if (warp == 0) {
      // lane i holds requests i, i + 32, ...: all loads in flight at once
      constexpr int PER = kMaxCompactBatch / 32;
      int len[PER], base[PER];
      const long long cap = len_cap(ws);
      const bool flat = ws.index_mode == PKV_IDX_FLAT;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = lane + 32 * i;
        len[i] = b < a.batch ? ws.seq_lens[b] : 0;
        base[i] = b < a.batch ? (flat ? ws.kv_indptr[b] : ws.req_pool_indices[b]) : 0;
      }
      int run = 0, most = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (32 * i >= a.batch) break;
        const int b = lane + 32 * i;
        int err = 0;
        if (len[i] < 0 || (long long)len[i] > cap) err = PKV_DEVERR_LEN;
        else if (flat && len[i] > 0 &&
                 (base[i] < 0 || (long long)base[i] + len[i] > ws.max_total_tokens))
          err = PKV_DEVERR_TOTAL;
        if (err) {
          if (blockIdx.x == 0) atomicOr(ws.err, err);
          len[i] = 0;
        }
        const int pcs = line_pieces(len[i]);
        most = max(most, pcs);
        int incl = pcs;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        if (b < a.batch) {
          s_pref[b] = run + incl - pcs;
          s_len[b] = len[i];
          s_base[b] = base[i];
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) s_pref[a.batch] = run;
      __syncwarp();
      if (lane == 0 && a.apportion) {
        KUnits us = share(run, most);
        if (us.q > 0) us.b = find(a.batch, us.pos);
        s_us = us;
      }
    }
  } else if (a.apportion) {
    // thread t adds up requests t per .. t per + per - 1
    const int per = (a.batch + C::THREADS - 1) / C::THREADS;
    int sum = 0, most = 0;
    for (int b = tid * per; b < min((tid + 1) * per, a.batch); ++b) {
      const int pcs = line_pieces(blockIdx.x == 0 ? checked_len(ws, b, ws.err) : usable_len(ws, b));
      sum += pcs;
      most = max(most, pcs);
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) s_slot[warp] = incl;
    if (lane == 0) s_bad[warp] = most;
    __syncthreads();
    int run = 0;
    for (int w = 0; w < W; ++w) {
      if (w == warp) s_pref[tid] = run + incl - sum;
      run += s_slot[w];
      most = max(most, s_bad[w]);
    }
    __syncthreads();
    if (tid == 0) {
      KUnits us = share(run, most);
      if (us.q > 0) {
        const int t = find(C::THREADS, us.pos);
        us.b = t * per;
        us.at = s_pref[t];
      }
      s_us = us;
    }
  }
  if (!a.apportion) {
    if (a.num_splits > 1) batch_max_len(ws, a.batch, &s_plan);
    if (tid == 0) {
      KUnits us;
      us.q = 0;
      us.chunk = a.num_splits == 1 ? 0x7ffffff0  // whole requests
                                   : split_chunk(s_plan, a.num_splits, ws.page_size);
      us.pos = blockIdx.x;
      us.end = a.num_splits * a.batch * H;
      us.b = 0;
      s_us = us;
    }
  }

  const int SB = a.c.scale_block, per_page = ws.page_size / SB;
  // The next unit into *dst by thread 0 (t0 == t1: past the last one).
  auto next_unit = [&](KUnit *dst) {
    KUnits us = s_us;
    KUnit u;
    u.b = u.g = u.c = u.n = u.t0 = u.t1 = u.bad = 0;
    u.base = u.srow = u.row0 = 0;
    u.fresh = 0x7fffffff;
    while (us.pos < us.end) {
      ReqIndex ri;
      int L;
      if (us.q > 0) {
        int start, last;  // the request's pieces in the line
        if (compact) {
          while (s_pref[us.b + 1] <= us.pos) ++us.b;
          start = s_pref[us.b], last = s_pref[us.b + 1];
          L = s_len[us.b];
        } else {
          for (;; ++us.b) {
            L = us.b < a.batch ? usable_len(ws, us.b) : 0;
            start = us.at, last = start + line_pieces(L);
            if (last > us.pos || us.b >= a.batch) break;
            us.at = last;
          }
          if (last <= us.pos) {  // lengths that changed since they were added up
            us.pos = us.end;
            continue;
          }
        }
        const int real = start + kUnitCost;
        const int from = max(us.pos, real), stop = min(us.end, last);
        us.pos = stop;
        if (from >= stop) continue;  // the run ends in what the request counts in front
        const int first = real / us.q;
        u.b = us.b;
        u.g = us.head;
        u.c = us.group - first;
        u.n = (last - 1) / us.q - first + 1;
        u.t0 = 16 * (from - real);
        u.t1 = min(16 * (stop - real), L);
        ri = compact ? req_index_cached(ws, s_base, us.b) : req_index(ws, us.b);
      } else {
        const int hb = a.batch * H;
        u.c = us.pos / hb;
        const int x = us.pos - u.c * hb;
        u.b = x / H;
        u.g = x - u.b * H;
        us.pos += gridDim.x;
        L = compact                  ? s_len[u.b]
            : u.c == 0 && u.g == 0 ? checked_len(ws, u.b, ws.err)
                                   : usable_len(ws, u.b);
        const bool whole = a.num_splits == 1;
        if (u.c * (long long)us.chunk >= L) continue;  // past the request's end
        u.t0 = whole ? 0 : u.c * us.chunk;
        u.t1 = whole ? L : min(u.t0 + us.chunk, L);
        u.n = whole ? 1 : (L + us.chunk - 1) / us.chunk;
        ri = compact ? req_index_cached(ws, s_base, u.b) : req_index(ws, u.b);
      }
      u.base = ri.base;
      u.bad = ri.ok ? 0 : PKV_DEVERR_PAGE;
      u.srow = ((long long)a.layer * pl.n_pages * H + u.g) * per_page;
      if (a.k_new) u.fresh = (L - 1) / SB * SB;
      u.row0 = ((long long)a.layer * ws.pool_slots * H + u.g) * D;
      s_us = us;
      *dst = u;
      return;
    }
    s_us = us;
    u.t0 = u.t1 = 0;
    *dst = u;
  };
  if (tid == 0) {  // in warp 0, which has the arrays
#pragma unroll 1  // one copy of the code: the second pass has it at hand
    for (int i = 0; i < 2; ++i) next_unit(&s_unit[i]);
  }
  __syncthreads();
  // Requests with no usable token have no unit: zero their outputs here.
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if ((compact ? s_len[b] : usable_len(ws, b)) > 0) continue;
    wait_previous();
    for (int i = tid; i < Hq * D; i += C::THREADS) {
      const long long o = (long long)b * Hq * D + i;
      if (a.flags & PKV_FLAG_OUT_F32) static_cast<float *>(ws.out)[o] = 0.f;
      else static_cast<uint16_t *>(ws.out)[o] = 0;
    }
    if (a.flags & PKV_FLAG_WRITE_LSE)
      for (int h = tid; h < Hq; h += C::THREADS) ws.lse[(long long)b * Hq + h] = -INFINITY;
  }

  uint8_t *const wring = smem + warp * (NS * C::STAGE);
  const uint32_t ring = smem_addr(wring);
  const int sshift = (SB & (SB - 1)) == 0 ? __ffs(SB) - 1 : -1;
  const int page_row = H * per_page;  // scales of a page
  const int rs = H * D;               // bytes between the rows of consecutive slots
  const int layer_slot = a.layer * ws.pool_slots;  // PAGED only: fits (checked by the host)
  // fragment offsets in a stage (rows + 8 are 8 D bytes on)
  const int tk = perm<D>(r);
  const int koff = swz<D>(tk, c);
  const int tv0 = perm<D>(2 * c), tv1 = perm<D>(2 * c + 1);
  const int voff0 = C::KB + (D == 128 ? swz<D>(tv0, r) : swz<D>(tv0, r >> 1) + (r & 1) * 8);
  const int voff1 = C::KB + (D == 128 ? swz<D>(tv1, r) : swz<D>(tv1, r >> 1) + (r & 1) * 8);
  // LOCOL: this lane's heads 2 c and 2 c + 1 are high or low parts
  const uint32_t lo0 = 2 * c >= G ? kHighBits : 0, lo1 = 2 * c + 1 >= G ? kHighBits : 0;
  int st_in = 0, st_out = 0, ph_out = 0;  // ring positions: next to fill, next to read
  bool dead = false;                      // a wait of this warp ran out

  int cu = 0;  // s_unit[cu]: the current unit, then (cu + 1) % 3 the next
  auto after = [](int i) { return i == 2 ? 0 : i + 1; };
  // pieces of a unit that are this warp's: every W-th from its own
  auto count = [&](const KUnit &u) {
    return dead ? 0 : (((u.t1 - u.t0 + 15) >> 4) - warp + W - 1) / W;
  };
  int np = count(s_unit[0]), nn = count(s_unit[1]);
  // Positions count this warp's pieces from the start of the current unit and
  // go on into the next unit.
  int done_idx = 0, done_kv = 0;  // next index entries / rows to copy
  int landed_idx = 0;             // index entries before this one have landed
  int base_pos = 0;               // position 0, counted from the block's first

  // PAGED: lane i holds, for piece 32 m + i of the unit, its page id and, from
  // the first of those pieces on, the row of its TMA box instead, and its offset
  // among the head's scales; *_unit the same for the first 32 of the next unit.
  auto load_pages = [&](const KUnit &u, int j0, int n) {
    const int j = j0 + lane;
    return PAGED && j < n && !(u.bad & PKV_DEVERR_PAGE)
               ? ws.page_table[u.base + pl.page_of(u.t0 + 16 * (warp + W * j))]
               : -1;
  };
  // A bad page id becomes page 0, an in-range stand-in: the unit is written empty.
  auto to_row = [&](KUnit &u, int j0, int n, int &row, unsigned &off) {
    const int j = j0 + lane, in0 = pl.in_page(u.t0 + 16 * (warp + W * j));
    int page = row;
    if (page < 0 || page >= pl.n_pages) {
      if (j < n) atomicOr(&u.bad, PKV_DEVERR_PAGE);
      page = 0;
    }
    row = layer_slot + page * pl.P + in0;
    off = (unsigned)page * page_row + (sshift >= 0 ? in0 >> sshift : in0 / SB);
  };
  int row = load_pages(s_unit[0], 0, np), row_unit = load_pages(s_unit[1], 0, nn);
  unsigned off = 0, off_unit = 0;

  // Else: the 16 index entries of position p into the index ring.
  auto copy_idx = [&](int p) {
    const bool in_next = p >= np;
    const KUnit &u = s_unit[in_next ? after(cu) : cu];
    if (lane < 16) {
      const int tok = u.t0 + 16 * (warp + W * (in_next ? p - np : p)) + lane;
      int *dst = &s_idx[warp][(base_pos + p) % (2 * NS)][lane];
      if (tok < u.t1 && !(u.bad & PKV_DEVERR_PAGE)) {
        const int *src = ws.index_mode == PKV_IDX_FLAT ? ws.kv_indices + u.base + tok
                                                       : ws.page_table + u.base + pl.page_of(tok);
        cp4(smem_addr(dst), src, 4);
      } else {
        *dst = -1;
      }
    }
  };
  // The copies of position p into the next stage.  Rows past the unit's end may
  // hold anything (TMA) or are zeros (cp.async).
  const int tt = lane & 15;  // lanes 0-15: K scale of token tt, 16-31: V scale
  const float *const scales = lane < 16 ? a.c.k_scale : a.c.v_scale;
  // block of token tt after the piece's first (PAGED: a piece is whole blocks,
  // or inside one)
  const unsigned tok_block = tt / SB;
  auto copy_kv = [&](int p) {
    const bool in_next = p >= np;
    const int j = in_next ? p - np : p;
    KUnit &u = s_unit[in_next ? after(cu) : cu];
    // the append's kernel is the one before this: its block waits for it
    if (u.t0 + 16 * (warp + W * j) + 16 > u.fresh) wait_previous();
    const int g = u.g;
    const float *sbase = scales + u.srow;
    const uint32_t dst = ring + st_in * C::STAGE;
    const uint32_t sd = smem_addr(&s_scale[warp][st_in][4 * (tt & 7) + 2 * (lane >> 4) + (tt >> 3)]);
    int bad = 0;
    if constexpr (PAGED) {
      if ((j & 31) == 0) {
        if (in_next) to_row(u, j, nn, row_unit, off_unit);
        else to_row(u, j, np, row, off);
      }
      const int at = __shfl_sync(0xffffffffu, in_next ? row_unit : row, j & 31);
      const unsigned so = __shfl_sync(0xffffffffu, in_next ? off_unit : off, j & 31);
      if (lane == 0) {
        uint64_t *bar = &s_bar[warp][st_in];
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_load_3d(dst, &tmk, 0, at, g, bar);
        tma_load_3d(dst + C::KB, &tmv, 0, at, g, bar);
      }
      cp4(sd, sbase + (so + tok_block), 4);
      if (!in_next && (j & 31) == 31) row = load_pages(u, j + 1, np);
    } else {
      constexpr int CH = D / 16, RPI = 32 / CH;  // chunks per row, rows per copy
      const int tok0 = u.t0 + 16 * (warp + W * j), nv = u.t1 - tok0;
      // lanes t and t + 16 resolve token t's slot (-1: none), the others ask them
      int s = -1;
      if (tt < nv) s = (int)slot_from_raw(ws, pl, s_idx[warp][(base_pos + p) % (2 * NS)][tt],
                                          tok0 + tt, bad);
      const uint8_t *kp = static_cast<const uint8_t *>(a.c.k_pool) + u.row0 + (lane % CH) * 16;
      const uint8_t *vp = static_cast<const uint8_t *>(a.c.v_pool) + u.row0 + (lane % CH) * 16;
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const int row = i * RPI + lane / CH, sr = __shfl_sync(0xffffffffu, s, row);
        const long long at = (long long)max(sr, 0) * rs;
        const uint32_t d = dst + swz<D>(row, lane % CH);
        cp16(d, kp + at, sr >= 0 ? 16 : 0);
        cp16(d + C::KB, vp + at, sr >= 0 ? 16 : 0);
      }
      long long si = 0;
      if (s >= 0) {
        const int page = pl.P == 1 ? s : s / pl.P;
        si = (long long)page * page_row + (pl.P == 1 ? 0 : (s - page * pl.P) / SB);
      }
      cp4(sd, sbase + si, s >= 0 ? 4 : 0);
    }
    if (bad) atomicOr(&u.bad, bad);
  };
  // Everything up to position p whose stage is free (p is at most NS past the
  // last piece read): rows, and index entries NS further.
  auto fill = [&](int p) {
    if (dead) return;
    const int most = min(p + 1, np + nn);
    while (done_kv < most) {
      if constexpr (!PAGED) {
        // Entries NS ahead land before their turn: the wait for the rows of
        // position p covers what was fetched with them.  The first pieces of
        // a block, and those of a unit that follows very short ones, are
        // known too late for that and wait here.
        const int to = min(done_kv + NS + 1, np + nn);
        for (; done_idx < to; ++done_idx) copy_idx(done_idx);
        if (landed_idx <= done_kv) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          landed_idx = done_idx;
        }
      }
      copy_kv(done_kv);
      if constexpr (!PAGED)
        if (lane == 0) s_seen[warp][st_in] = base_pos + done_idx;
      asm volatile("cp.async.commit_group;" ::: "memory");  // one group per position
      st_in = st_in + 1 == NS ? 0 : st_in + 1;
      ++done_kv;
    }
  };
  if (PAGED && (a.flags & PKV_FLAG_TEST_SKIP_FIRST_TILE)) {
    // test hook: the first stage is never armed, the wait for it runs out
    if (np + nn > 0) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      st_in = 1;
      done_kv = 1;
    }
  }
  fill(NS - 2);  // the last stage follows in the unit's first step

  // Q^T as the B operand: lane r is head r (+ 8), its 16 elements 64 x + 16 c ..
  // 64 x + 16 c + 15 of each half x match the K bytes the lane reads.  With LOCOL
  // columns G .. 2 G - 1 are the same heads again: scores and reference come out the
  // same, their weights go into the second product as low parts.
  uint4 qraw[NH][D / 32];
  auto load_q = [&](const KUnit &u) {
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const int h = r + 8 * n;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        qraw[n][i] = h < (C::LOCOL ? 2 * G : G)
                         ? reinterpret_cast<const uint4 *>(
                               a.q)[((long long)u.b * Hq + u.g * G + h % G) * (D / 8) +
                                    8 * (i >> 1) + 2 * c + (i & 1)]
                         : make_uint4(0, 0, 0, 0);
    }
  };
  wait_previous();  // q comes from the previous kernel
  if (s_unit[0].t0 < s_unit[0].t1) load_q(s_unit[0]);

  int n_part = 0;  // tickets taken and not looked at
  while (s_unit[cu].t0 < s_unit[cu].t1) {  // the same in every thread
    const int nv0 = s_unit[cu].t1 - s_unit[cu].t0 - 16 * warp;  // tokens from piece 0 on
    uint32_t qb[NH][D / 16][2];
    float qs[NH][2];  // scale of heads 2 c and 2 c + 1, log2 units
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float f[8];
        unpack8(qraw[n][i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^k brings m into [2^14, 2^15) (k <= 126: a smaller row keeps all it has)
      const int k = m > 0.f ? min(126, 141 - (__float_as_int(m) >> 23)) : 0;
      const float up = pow2i(k);
      const float down = a.scale * kLog2e * pow2i(-k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float f[8];
        unpack8(qraw[n][i], f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qb[n][2 * i + e][0] = pack_f16x2(f[4 * e] * up, f[4 * e + 1] * up);
          qb[n][2 * i + e][1] = pack_f16x2(f[4 * e + 2] * up, f[4 * e + 3] * up);
        }
      }
      qs[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);
      qs[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }
    // acc[n][j] = O of heads 8 n + 2 c + {0, 1} at dims VB r + 2 j (elements 0, 1)
    // and VB r + 2 j + 1 (elements 2, 3)
    float acc[NH][D / 16][4];
    float m_run[NH][2], l_run[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.f;
      m_run[n][0] = m_run[n][1] = -INFINITY;
      l_run[n][0] = l_run[n][1] = 0.f;
    }

    // Step j reads piece j and refills the ring behind it; step -1 only fills.
    // After the last piece its stage stays free: it takes the warp's O.
#pragma unroll 1
    for (int j = -1; j < np; ++j) {
      if (j >= 0) {
        // this position's group: the groups of the newer positions may pend
        const int newer = done_kv - 1 - j;
        if (newer >= NS - 1) asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (PAGED && __any_sync(0xffffffffu, !mbar_wait_bounded(&s_bar[warp][st_out], ph_out))) {
          // The copies still in flight (bounded too) end before anything else
          // uses their stages; the warp copies nothing from here on.
          for (int i = j; i < done_kv; ++i) {
            mbar_wait_bounded(&s_bar[warp][st_out], ph_out);
            if (++st_out == NS) {
              st_out = 0;
              ph_out ^= 1;
            }
          }
          dead = true;
          break;
        }
        __syncwarp();  // the other lanes' copies too
        if constexpr (!PAGED) landed_idx = max(landed_idx, s_seen[warp][st_out] - base_pos);
        const uint8_t *stage = wring + st_out * C::STAGE;
        const float *ss = s_scale[warp][st_out];
        const int nv = nv0 - 16 * W * j;
        // ---- S^T = K Q^T, in two chains ----
        float sc[NH][4], sc2[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[n][i] = sc2[n][i] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const uint4 lo = *reinterpret_cast<const uint4 *>(stage + (koff ^ (x * 64)));
          const uint4 hi = *reinterpret_cast<const uint4 *>(stage + (koff ^ (x * 64)) + 8 * D);
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            codes_f16<DT>(wl[w], a0, a2);
            codes_f16<DT>(wh[w], a1, a3);
#pragma unroll
            for (int n = 0; n < NH; ++n)
              mma_f16((w & 1) ? sc2[n] : sc[n], a0, a1, a2, a3, qb[n][4 * x + w][0],
                      qb[n][4 * x + w][1]);
          }
        }
        // ---- weights: tokens tk and tk + 8, heads 2 c and 2 c + 1 ----
        const float4 scl = *reinterpret_cast<const float4 *>(ss + 4 * tk);
        const float ks[2] = {scl.x, scl.y};
        float vs[2] = {scl.z, scl.w};
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[n][i] = (sc[n][i] + sc2[n][i]) * (ks[i >> 1] * qs[n][i & 1]);
        if (nv < 16) {  // rows past the end: any score and scale, no weight
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (tk + 8 * t >= nv) {
              vs[t] = 1.f;
#pragma unroll
              for (int n = 0; n < NH; ++n) sc[n][2 * t] = sc[n][2 * t + 1] = -INFINITY;
            }
        }
        const float vt[2] = {fmaxf(vs[0], kScaleFloor), fmaxf(vs[1], kScaleFloor)};
        float p[NH][4];  // exp(x - r); element 2 t + e
        auto weigh = [&]() {
          bool big = false;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[n][i] = fast_exp2(sc[n][i] - m_run[n][i & 1]);
              big |= p[n][i] * vt[i >> 1] > kMove;
            }
          return big;
        };
        if (__any_sync(0xffffffffu, weigh())) {
          const float lv[2] = {fast_log2(vt[0]), fast_log2(vt[1])};
#pragma unroll
          for (int n = 0; n < NH; ++n) {
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = fmaxf(sc[n][e] + lv[0], sc[n][2 + e] + lv[1]);
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              const float mn = fmaxf(m_run[n][e], t - kPlace);
              al[e] = mn == -INFINITY ? 1.f : fast_exp2(m_run[n][e] - mn);
              m_run[n][e] = mn;
              l_run[n][e] *= al[e];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[n][i][0] *= al[0];
              acc[n][i][1] *= al[1];
              acc[n][i][2] *= al[0];
              acc[n][i][3] *= al[1];
            }
          }
          weigh();
        }
        uint32_t wb[NH][2];  // W^T as B: tokens of rows 0-7 / 8-15
        uint32_t wl[C::LOCOL ? 1 : NH][2];  // its low parts
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            l_run[n][0] += p[n][2 * t];
            l_run[n][1] += p[n][2 * t + 1];
            const float w0 = p[n][2 * t] * vs[t], w1 = p[n][2 * t + 1] * vs[t];
            if constexpr (C::LOCOL) {
              wb[n][t] = movmatrix_t(pack_f16x2_rz(low_part(w0, lo0), low_part(w1, lo1)));
            } else {
              wb[n][t] = movmatrix_t(pack_f16x2_rz(w0, w1));
              wl[n][t] = movmatrix_t(
                  pack_f16x2_rz(low_part(w0, kHighBits), low_part(w1, kHighBits)));
            }
          }
        // ---- O^T += V^T W^T ----
        uint32_t v[4][C::VB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t *src = stage + ((i & 1) ? voff1 : voff0) + (i >> 1) * 8 * D;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src);
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(src);
            v[i][0] = x.x, v[i][1] = x.y;
          }
        }
        if (nv < 16) {  // what lies past the end may stand for NaN
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (((i & 1) ? tv1 : tv0) + (i >> 1) * 8 >= nv) {
#pragma unroll
              for (int w = 0; w < C::VB / 4; ++w) v[i][w] = 0;
            }
        }
#pragma unroll
        for (int w = 0; w < C::VB / 4; ++w) {
#pragma unroll
          for (int hlf = 0; hlf < 2; ++hlf) {
            const uint32_t sel = hlf ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            codes_f16<DT>(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
            codes_f16<DT>(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
#pragma unroll
            for (int n = 0; n < NH; ++n) {
              mma_f16(acc[n][2 * w + hlf], a0, a1, a2, a3, wb[n][0], wb[n][1]);
              if constexpr (!C::LOCOL)
                mma_f16(acc[n][2 * w + hlf], a0, a1, a2, a3, wl[n][0], wl[n][1]);
            }
          }
        }
        if (++st_out == NS) {
          st_out = 0;
          ph_out ^= 1;
        }
        __syncwarp();  // every lane is done with the stage
        if (j == np - 1) break;
      }
      fill(j + NS);
    }

    // ---- the warps' states meet ----
    const int at = np > 0 && !dead ? (st_out == 0 ? NS - 1 : st_out - 1) : -1;
    if (lane == 0) {
      s_slot[warp] = at;
      s_bad[warp] = dead ? PKV_DEVERR_TIMEOUT : 0;
    }
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[n][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (r == 0) s_ml[warp][8 * n + 2 * c + e] = make_float2(m_run[n][e], l);
      }
    const bool has_next = s_unit[after(cu)].t0 < s_unit[after(cu)].t1;
    if (has_next) load_q(s_unit[after(cu)]);  // on its way while the block meets
    const int split = s_unit[cu].c;
    const bool final_out = s_unit[cu].n == 1;
    const long long q0 = (long long)s_unit[cu].b * Hq + s_unit[cu].g * G;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      // 8 heads x D floats in the free stage; word d of row h sits at d ^ its
      // lanes' (r, c) bits, so the 8-byte stores of half a warp take every bank
      if (at >= 0) {
        float *o = reinterpret_cast<float *>(wring + at * C::STAGE);
        const int x = D == 128 ? (((r >> 1) & 1) << 1) | (c << 2) : c << 1;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2 *>(o + (2 * c + e) * D + ((C::VB * r + 2 * i) ^ x)) =
                make_float2(acc[n][i][e], acc[n][i][2 + e]);
      }
      __syncthreads();
      int unit_bad = s_unit[cu].bad;
#pragma unroll
      for (int w = 0; w < W; ++w) unit_bad |= s_bad[w];
      if (n == 0 && tid == C::THREADS - 1) {
        if (unit_bad) atomicOr(ws.err, unit_bad);
      }
      for (int i = tid * 4; i < min(8, G - 8 * n) * D; i += C::THREADS * 4) {
        const int h8 = i / D, h = h8 + 8 * n, d = i - h8 * D;
        float M = -INFINITY, L = 0.f;
        float2 ml[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          ml[w] = s_ml[w][h];
          M = fmaxf(M, ml[w].x);
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        // 4 floats of row hh, column d of a warp's O
        auto take = [&](const uint8_t *o, int hh) {
          const int sx = D == 128 ? (((d >> 5) & 1) << 1) | ((hh >> 1) << 2) : (hh >> 1) << 1;
          const float4 y = *reinterpret_cast<const float4 *>(o + (hh * D + (d ^ (sx & ~3))) * 4);
          return sx & 2 ? make_float4(y.z, y.w, y.x, y.y) : y;
        };
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int slot = s_slot[w];
          if (slot < 0) continue;
          // a warp whose scores are all NaN never placed its reference: it
          // passes its NaN on
          const float f = ml[w].x == -INFINITY ? 1.f : fast_exp2(ml[w].x - M);
          L += f * ml[w].y;
          const uint8_t *o = smem + (w * NS + slot) * C::STAGE;
          float4 y = take(o, h8);
          if constexpr (C::LOCOL) {
            const float4 z = take(o, h8 + G);
            y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
          }
          x.x = fmaf(f, y.x, x.x);
          x.y = fmaf(f, y.y, x.y);
          x.z = fmaf(f, y.z, x.z);
          x.w = fmaf(f, y.w, x.w);
        }
        const float inv = 1.f / L;
        x = unit_bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        const long long qrow = q0 + h;
        if (!final_out) {
          *reinterpret_cast<float4 *>(ws.o_part + (qrow * a.num_splits + split) * D + d) = x;
        } else if (a.flags & PKV_FLAG_OUT_F32) {
          *reinterpret_cast<float4 *>(static_cast<float *>(ws.out) + qrow * D + d) = x;
        } else {
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(ws.out) + qrow * D + d) =
              make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        }
        if (d == 0) {
          const float lse = unit_bad ? -INFINITY : M * kLn2 + logf(L);
          if (!final_out)
            *reinterpret_cast<float2 *>(ws.ml_part + (qrow * a.num_splits + split) * 2) =
                // NaN as an infinite weight: the merge's difference of infinities
                // makes the row NaN again
                make_float2(lse == lse ? lse : INFINITY, unit_bad ? 0.f : 1.f);
          else if (a.flags & PKV_FLAG_WRITE_LSE)
            ws.lse[qrow] = lse;
        }
      }
      // the unit after the next one, in the place of the one before this
      if (n == 0 && tid == 0) next_unit(&s_unit[after(after(cu))]);
      // the stages go back to copies of the async proxy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
    // Ticket: the block that completes a pair's partials merges them, after
    // its last unit.  The barrier above orders the block's partial before the
    // ticket; the last taker acquires every other block's.
    if (!final_out) {
      if (tid == 0) {
        const KUnit &u = s_unit[cu];
        int *ctr = ws.split_counters + (long long)u.b * H + u.g;
        const int last = atomic_add_acq_rel_gpu(ctr, 1) == u.n - 1;
        if (last) *ctr = 0;  // ready for the next launch
        s_merge[n_part][0] = last ? u.n : 0;
        s_merge[n_part][1] = u.b;
        s_merge[n_part][2] = u.g;
      }
      ++n_part;
    }

    // ---- on to the next unit ----
    done_idx -= np;
    done_kv -= np;
    landed_idx -= np;
    base_pos += np;
    cu = after(cu);
    np = dead ? 0 : nn;
    row = row_unit;
    off = off_unit;
    nn = count(s_unit[after(cu)]);
    row_unit = load_pages(s_unit[after(cu)], 0, nn);

    // A run has at most two partials (its first and its last unit); blocks of
    // fixed chunks (larger batches) merge as they go.
    if (n_part == 2 || (n_part > 0 && !has_next)) {
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < n_part; ++i) {
        const int n = s_merge[i][0];
        if (n > 0 && warp < G) {
          constexpr int RPW = G >= W ? G / W : 1;
          merge_rows_batched<D, RPW>(ws, (long long)s_merge[i][1] * Hq + s_merge[i][2] * G + warp, W,
                                     a.num_splits, n, a.flags, lane);
        }
      }
      __syncthreads();  // s_merge
      n_part = 0;
    }
  }
}

using TmapEncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// 3-D view of a code pool [NL * pool_slots, Hkv, D] as (byte, slot, head): a
// box of D x 16 x 1 is one 16-token piece of one head.
bool encode_codes_map(CUtensorMap *m, void *base, const pkv_workspace &ws) {
  static const TmapEncodeFn fn = [] {  // looked up once, whichever thread is first
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<TmapEncodeFn>(p) : nullptr;
  }();
  if (!fn) return false;
  const cuuint64_t D = (cuuint64_t)ws.head_dim, H = (cuuint64_t)ws.n_kv_heads;
  const cuuint64_t dims[3] = {D, (cuuint64_t)ws.n_layers * (cuuint64_t)ws.pool_slots, H};
  const cuuint64_t strides[2] = {H * D, D};
  const cuuint32_t box[3] = {(cuuint32_t)D, 16, 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int G, int DT, bool PAGED>
cudaError_t launch_one(Kv8Args a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
  using C = KCfg<D, G>;
  auto kern = kv8_decode_kernel<D, G, DT, PAGED>;
  static int occ_cache[64] = {0};
  static int sms_cache[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int di = dev & 63;
  if (occ_cache[di] == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    int occ = 0, sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, C::THREADS, C::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sms_cache[di] = sms;
    occ_cache[di] = occ > 0 ? occ : 1;
  }
  const pkv_workspace &ws = a.ws;
  const long long units = (long long)a.num_splits * a.batch * ws.n_kv_heads;
  const long long cap = (long long)sms_cache[di] * occ_cache[di];
  const int grid = (int)(units < cap ? units : cap);
  // sharing out by length needs a block per head and a line whose length fits
  // an int
  a.apportion = a.num_splits > 1 && grid >= ws.n_kv_heads &&
                (long long)a.batch * (len_cap(ws) / 16 + 1 + kUnitCost) < 0x7fffffffll;
  return launch_pdl(kern, dim3(grid), dim3(C::THREADS), (size_t)C::SMEM, st, a, tmk, tmv);
}

template <int D, int G>
cudaError_t launch_shape(const Kv8Args &a, cudaStream_t st) {
  CUtensorMap tmk, tmv;
  memset(&tmk, 0, sizeof(tmk));
  memset(&tmv, 0, sizeof(tmv));
  const bool paged = a.ws.index_mode == PKV_IDX_PAGE_TABLE && a.ws.page_size % 16 == 0 &&
                     (long long)a.ws.n_layers * a.ws.pool_slots < 0x7fffffffll &&
                     (16 % a.c.scale_block == 0 || a.c.scale_block % 16 == 0) &&
                     (long long)a.ws.pool_slots / a.c.scale_block * a.ws.n_kv_heads < 0xffffffffll &&
                     encode_codes_map(&tmk, a.c.k_pool, a.ws) &&
                     encode_codes_map(&tmv, a.c.v_pool, a.ws);
  if (a.c.dtype == PKV_KV8_E4M3)
    return paged ? launch_one<D, G, PKV_KV8_E4M3, true>(a, tmk, tmv, st)
                 : launch_one<D, G, PKV_KV8_E4M3, false>(a, tmk, tmv, st);
  return paged ? launch_one<D, G, PKV_KV8_INT8, true>(a, tmk, tmv, st)
               : launch_one<D, G, PKV_KV8_INT8, false>(a, tmk, tmv, st);
}

}  // namespace

bool kv8_decode_supported(int head_dim, int group) {
  return (head_dim == 64 || head_dim == 128) &&
         (group == 1 || group == 2 || group == 4 || group == 8 || group == 16);
}

cudaError_t launch_kv8_decode(const Kv8Args &args, cudaStream_t st) {
  Kv8Args a = args;
  if (a.k_new) {
    // With PKV_FLAG_PLAN_EARLY the append lets this kernel start while the one
    // before the append still runs: it plans and loads everything but the block
    // appended to, and waits for the append (which waits for the rest) there.
    const cudaError_t e = launch_kv8_append(a.ws, a.c, a.batch, a.layer, 1, a.k_new, a.v_new,
                                            (a.flags & PKV_FLAG_PLAN_EARLY) != 0, a.ws.seq_lens, st);
    if (e != cudaSuccess) return e;
  }
  const int D = a.ws.head_dim, G = a.ws.n_q_heads / a.ws.n_kv_heads;
#define PKV_KV8_CASE(DD, GG) \
  if (D == DD && G == GG) return launch_shape<DD, GG>(a, st);
  PKV_KV8_CASE(128, 1) PKV_KV8_CASE(128, 2) PKV_KV8_CASE(128, 4) PKV_KV8_CASE(128, 8)
  PKV_KV8_CASE(128, 16) PKV_KV8_CASE(64, 1) PKV_KV8_CASE(64, 2) PKV_KV8_CASE(64, 4)
  PKV_KV8_CASE(64, 8) PKV_KV8_CASE(64, 16)
#undef PKV_KV8_CASE
  return cudaErrorNotSupported;
}

}  // namespace pkv
