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
// with a reference r that follows max(x_t + ln v_scale_t): the largest w_t is
// then 2^7 .. 2^15, which fp16 holds whatever the value scales are, while the
// softmax sum  l = sum exp(x_t - r)  stays in fp32 (v_scale_t in [2^-100,
// 2^100] keeps exp(x_t - r) in its range).  out = O / l.  Rounding w to fp16
// costs 2^-11 of a weight, an eighth of what the bf16 output's own rounding
// may cost (weights under 2^-21 of the largest: 2^-32 of the largest).
// r moves only when a weight would pass 2^15, so most tokens need one vote
// instead of a maximum over lanes and a rescaling of O.
//
// Data.  Each warp takes every W-th piece of 16 tokens of the unit and fills
// its own ring of stages, so no block barrier stands between a copy and its
// product.  A stage is the piece's K rows then its V rows, D bytes each, with
// the 16-byte chunks swizzled (TMA's 128- or 64-byte pattern).  Pages of whole
// pieces come as one TMA box for K and one for V, completing on the stage's
// mbarrier; other page sizes and flat indices as 16-byte cp.async copies of
// the rows (whole rows per 8 or 4 lanes).  Fragments are read with plain
// 16-byte loads: which token a row of S^T is, and which head_dim an index of
// the contraction is, is free as long as V and Q agree.  K: lane (r = lane / 4,
// c = lane % 4) takes 16 bytes of token perm(r); V: 16 (8 at D = 64) bytes of
// the tokens perm(2 c), perm(2 c + 1) (+ 8), whose bytes one byte permute per
// word interleaves into the (token, token) pairs of the A fragments of O^T.
// perm is chosen so that both reads touch every bank once.
//
// The warps' states meet in shared memory at the end of a unit; the splits of
// a request meet in the block that finishes last (an atomic ticket).
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
  static constexpr int W = NH == 1 ? 8 : 4;        // warps (16 heads: twice the registers)
  static constexpr int THREADS = W * 32;
  static constexpr int KB = 16 * D;                // K (or V) bytes of a piece
  static constexpr int STAGE = 2 * KB;
  static constexpr int NS = W == 8 ? (D == 128 ? 3 : 4) : (D == 128 ? 6 : 8);  // ring stages
  static constexpr int VB = D / 8;                 // V bytes of a row per lane
  static constexpr int RS = D + 4;                 // row stride of a warp's O (floats)
  static constexpr int SMEM = W * NS * STAGE + 1024;  // + alignment slack
  static_assert(NS * STAGE >= G * RS * 4, "a warp's O fits its ring");
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// PAGED: pages hold whole 16-token pieces, loaded as TMA boxes.
template <int D, int G, int DT, bool PAGED>
__global__ void __launch_bounds__(KCfg<D, G>::THREADS, 2)
    kv8_decode_kernel(const __grid_constant__ Kv8Args a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
  using C = KCfg<D, G>;
  constexpr int W = C::W, NS = C::NS, NH = C::NH;
  // log2 of the largest weight where r is placed, and where it has to move
  constexpr float kPlace = 7.f, kMove = 15.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[PAGED ? W : 1][NS];
  __shared__ int s_pref[kMaxCompactBatch + 1];
  __shared__ int s_len[kMaxCompactBatch];
  __shared__ int s_base[kMaxCompactBatch];
  __shared__ int s_chunk[kMaxCompactBatch];
  __shared__ float s_scale[W][NS][32];  // K scales of a piece's tokens, then V scales
  __shared__ int s_idx[PAGED ? 1 : W][PAGED ? 1 : 2 * NS][16];
  __shared__ float s_ml[W][16][2];
  __shared__ float s_hml[16][2];
  __shared__ int s_bad[W];
  __shared__ int s_tmp[32];
  __shared__ int s_max_len, s_last;
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int Hq = ws.n_q_heads, H = ws.n_kv_heads;
  const bool early = (a.flags & PKV_FLAG_PLAN_EARLY) != 0;
  if (!early) {
    pdl_wait();
    pdl_trigger();
  }
  if constexpr (PAGED) {
    // a warp is the only user of its barriers
    if (lane < NS) mbar_init(&s_bar[warp][lane], 1);
    fence_barrier_init();
    __syncwarp();
  }

  Plan pl;
  pl.set_pages(ws);
  pl.batch = a.batch;
  pl.hkv = H;
  pl.S = a.num_splits;
  const bool direct = pl.S == 1;
  if (a.batch <= kMaxCompactBatch) {
    const int budget = a.apportion ? (int)gridDim.x : 0;
    const int pairs = batch_plan_compact(ws, a.batch, pl.S, budget, s_len, s_base, s_pref, s_chunk,
                                         s_tmp, &s_max_len, &pl.chunk);
    pl.pref = s_pref;
    pl.lens = s_len;
    pl.chunks = budget > 0 ? s_chunk : nullptr;
    pl.n_units = pairs * H;
  } else {
    pl.chunk = split_chunk(batch_max_len(ws, a.batch, &s_max_len), pl.S, ws.page_size);
    pl.n_units = pl.S * pl.batch * H;
  }

  uint8_t *const wring = smem + warp * (NS * C::STAGE);
  const uint32_t ring = smem_addr(wring);
  float *obuf = reinterpret_cast<float *>(wring);
  const int SB = a.c.scale_block, per_page = ws.page_size / SB;
  const int sshift = (SB & (SB - 1)) == 0 ? __ffs(SB) - 1 : -1;
  const long long layer_slot = (long long)a.layer * ws.pool_slots;
  // fragment offsets in a stage (rows + 8 are 8 D bytes on)
  const int tk = perm<D>(r);
  const int koff = swz<D>(tk, c);
  const int tv0 = perm<D>(2 * c), tv1 = perm<D>(2 * c + 1);
  const int voff0 = C::KB + (D == 128 ? swz<D>(tv0, r) : swz<D>(tv0, r >> 1) + (r & 1) * 8);
  const int voff1 = C::KB + (D == 128 ? swz<D>(tv1, r) : swz<D>(tv1, r >> 1) + (r & 1) * 8);
  int st_in = 0, st_out = 0, ph_out = 0;  // ring positions: next to fill, next to read
  bool dead = false;                      // a wait of this warp ran out

  bool waited = !early;
  auto wait_previous = [&]() {
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
  };
  if (pl.pref) {
    // Requests with no usable token have no unit: zero their outputs here.
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      if (s_pref[b + 1] != s_pref[b]) continue;
      wait_previous();
      for (int i = tid; i < Hq * D; i += C::THREADS) {
        const long long o = (long long)b * Hq * D + i;
        if (a.flags & PKV_FLAG_OUT_F32) static_cast<float *>(ws.out)[o] = 0.f;
        else static_cast<uint16_t *>(ws.out)[o] = 0;
      }
      if (a.flags & PKV_FLAG_WRITE_LSE)
        for (int h = tid; h < Hq; h += C::THREADS) ws.lse[(long long)b * Hq + h] = -INFINITY;
    }
  }

  UnitIter ui;
  for (ui.first(ws, pl); !ui.done; ui.next(ws, pl)) {
    const Unit un = ui.un;
    const int hq0 = un.g * G;
    if (un.t0 >= un.t1) {  // dense enumeration only: past the request's end
      if (un.c == 0) {
        wait_previous();
        for (int i = tid; i < G * D; i += C::THREADS) {
          const long long o = ((long long)un.b * Hq + hq0) * D + i;
          if (a.flags & PKV_FLAG_OUT_F32) static_cast<float *>(ws.out)[o] = 0.f;
          else static_cast<uint16_t *>(ws.out)[o] = 0;
        }
        if ((a.flags & PKV_FLAG_WRITE_LSE) && tid < G)
          ws.lse[(long long)un.b * Hq + hq0 + tid] = -INFINITY;
      }
      continue;
    }
    const int pieces = (un.t1 - un.t0 + 15) / 16;
    const int np = dead ? 0 : (pieces - warp + W - 1) / W;  // this warp's
    const ReqIndex ri = pl.pref ? req_index_cached(ws, s_base, un.b) : req_index(ws, un.b);
    int bad = (ri.ok ? 0 : PKV_DEVERR_PAGE) | (dead ? PKV_DEVERR_TIMEOUT : 0);
    auto piece_tok = [&](int j) { return un.t0 + 16 * (warp + W * j); };

    // Index entries.  PAGED: lane i holds the page of piece 32 m + i, the next
    // 32 follow in pg_next.  Else the 16 entries of a piece are copied, one
    // group ahead of its rows, into a ring of 2 NS pieces.
    int pg = -1, pg_next = -1;
    auto load_pages = [&](int j0) {
      const int j = j0 + lane;
      return PAGED && ri.ok && j < np ? *index_src(ws, pl, ri, piece_tok(j)) : -1;
    };
    auto fetch_idx = [&](int j) {
      if constexpr (!PAGED) {
        if (j < np && lane < 16) {
          const int tok = piece_tok(j) + lane;
          int *dst = &s_idx[warp][j % (2 * NS)][lane];
          if (ri.ok && tok < un.t1) cp4(smem_addr(dst), index_src(ws, pl, ri, tok), 4);
          else *dst = -1;
        }
      }
    };
    // The copies of piece j into the next stage; their small ones (scales and
    // index entries) are a commit group each piece.  Rows past the unit's end
    // may hold anything (TMA) or are zeros (cp.async).
    const long long srow = ((long long)a.layer * pl.n_pages * H + un.g) * per_page;
    const float *sbase = (lane < 16 ? a.c.k_scale : a.c.v_scale) + srow;
    const int tt = lane & 15;  // lanes 0-15: K scale of token tt, 16-31: V scale
    auto issue = [&](int j) {
      const int tok0 = piece_tok(j);
      const uint32_t dst = ring + st_in * C::STAGE;
      const uint32_t sd = smem_addr(&s_scale[warp][st_in][lane]);
      if constexpr (PAGED) {
        int page = __shfl_sync(0xffffffffu, pg, j & 31);
        if (page < 0 || page >= pl.n_pages) {
          bad |= PKV_DEVERR_PAGE;
          page = 0;  // an in-range stand-in: the unit is written empty
        }
        const int in0 = pl.in_page(tok0);
        if (lane == 0) {
          uint64_t *bar = &s_bar[warp][st_in];
          const int row = (int)layer_slot + page * pl.P + in0;
          mbar_arrive_expect_tx(bar, C::STAGE);
          tma_load_3d(dst, &tmk, 0, row, un.g, bar);
          tma_load_3d(dst + C::KB, &tmv, 0, row, un.g, bar);
        }
        const int sub = sshift >= 0 ? (in0 + tt) >> sshift : (in0 + tt) / SB;
        cp4(sd, sbase + ((long long)page * (H * per_page) + sub), 4);
        if ((j & 31) == 31) {
          pg = pg_next;
          pg_next = load_pages(j + 33);
        }
      } else {
        constexpr int CH = D / 16, RPI = 32 / CH;  // chunks per row, rows per copy
        const int nv = un.t1 - tok0;
        const int *raw = s_idx[warp][j % (2 * NS)];
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const int row = i * RPI + lane / CH, ch = lane % CH;
          int kind = 0;
          const int s = row < nv ? (int)slot_from_raw(ws, pl, raw[row], tok0 + row, kind) : -1;
          bad |= kind;
          const long long off =
              s >= 0 ? ((layer_slot + s) * H + un.g) * (long long)D + ch * 16 : 0;
          const uint32_t d = dst + swz<D>(row, ch);
          cp16(d, static_cast<const uint8_t *>(a.c.k_pool) + off, s >= 0 ? 16 : 0);
          cp16(d + C::KB, static_cast<const uint8_t *>(a.c.v_pool) + off, s >= 0 ? 16 : 0);
        }
        int kind = 0;
        const int s = tt < nv ? (int)slot_from_raw(ws, pl, raw[tt], tok0 + tt, kind) : -1;
        long long si = 0;
        if (s >= 0) {
          const int page = pl.P == 1 ? s : s / pl.P;
          si = (long long)page * (H * per_page) + (pl.P == 1 ? 0 : (s - page * pl.P) / SB);
        }
        cp4(sd, sbase + si, s >= 0 ? 4 : 0);
      }
      st_in = st_in + 1 == NS ? 0 : st_in + 1;
    };

    // Q^T as the B operand: lane r is head r (+ 8), its 16 elements 64 x + 16 c
    // .. 64 x + 16 c + 15 of each half x match the K bytes the lane reads.
    uint32_t qb[NH][D / 16][2];
    float qs[NH][2];  // scale of heads 2 c and 2 c + 1, log2 units
    auto load_q = [&]() {
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        const int h = r + 8 * n;
        uint4 raw[D / 32];
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            raw[2 * x + i] =
                h < G ? reinterpret_cast<const uint4 *>(a.q)[((long long)un.b * Hq + hq0 + h) *
                                                                 (D / 8) + 8 * x + 2 * c + i]
                      : make_uint4(0, 0, 0, 0);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float f[8];
          unpack8(raw[i], f);
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
          unpack8(raw[i], f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qb[n][2 * i + e][0] = pack_f16x2(f[4 * e] * up, f[4 * e + 1] * up);
            qb[n][2 * i + e][1] = pack_f16x2(f[4 * e + 2] * up, f[4 * e + 3] * up);
          }
        }
        qs[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);
        qs[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      }
    };

    if constexpr (PAGED) {
      pg = load_pages(0);
      pg_next = load_pages(32);
    } else {
      for (int j = 0; j < NS; ++j) fetch_idx(j);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
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

    // Iteration j: consume piece j (from 0 on), then fill its stage with piece
    // j + NS; the NS iterations before the first only fill.
#pragma unroll 1
    for (int j = -NS; j < np; ++j) {
      if (j >= 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        if constexpr (PAGED) {
          const bool ok = mbar_wait_bounded(&s_bar[warp][st_out], ph_out);
          if (__any_sync(0xffffffffu, !ok)) {
            // The copies still in flight (bounded too) end before anything
            // else uses their stages; the warp copies nothing from here on.
            for (int i = j; i < min(j + NS, np); ++i) {
              mbar_wait_bounded(&s_bar[warp][st_out], ph_out);
              if (++st_out == NS) {
                st_out = 0;
                ph_out ^= 1;
              }
            }
            dead = true;
            bad |= PKV_DEVERR_TIMEOUT;
            break;
          }
        }
        __syncwarp();  // the other lanes' copies too
        const uint8_t *stage = wring + st_out * C::STAGE;
        const float *ss = s_scale[warp][st_out];
        const int nv = un.t1 - piece_tok(j);
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
        const float ks[2] = {ss[tk], ss[tk + 8]};
        float vs[2] = {ss[16 + tk], ss[24 + tk]};
        if (nv < 16) {  // rows past the end: any scale, no weight
          if (tk >= nv) vs[0] = 1.f;
          if (tk + 8 >= nv) vs[1] = 1.f;
        }
        const float lv[2] = {fast_log2(vs[0]), fast_log2(vs[1])};
        bool move = false;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[n][i] = (sc[n][i] + sc2[n][i]) * ks[i >> 1] * qs[n][i & 1];
        if (nv < 16) {
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tk + 8 * (i >> 1) >= nv) sc[n][i] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) move |= sc[n][i] + lv[i >> 1] > m_run[n][i & 1] + kMove;
        if (__any_sync(0xffffffffu, move)) {
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
        }
        uint32_t wb[NH][2];  // W^T as B: tokens of rows 0-7 / 8-15
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float p0 = fast_exp2(sc[n][2 * t] - m_run[n][0]);
            const float p1 = fast_exp2(sc[n][2 * t + 1] - m_run[n][1]);
            l_run[n][0] += p0;
            l_run[n][1] += p1;
            wb[n][t] = movmatrix_t(pack_f16x2(p0 * vs[t], p1 * vs[t]));
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
            for (int n = 0; n < NH; ++n)
              mma_f16(acc[n][2 * w + hlf], a0, a1, a2, a3, wb[n][0], wb[n][1]);
          }
        }
        if (++st_out == NS) {
          st_out = 0;
          ph_out ^= 1;
        }
        __syncwarp();  // every lane is done with the stage
      }
      if (j + NS < np) {
        if (PAGED && j == -NS && (a.flags & PKV_FLAG_TEST_SKIP_FIRST_TILE)) {
          // test hook: the stage is never armed, its wait runs out
          st_in = st_in + 1 == NS ? 0 : st_in + 1;
        } else {
          issue(j + NS);
        }
      }
      fetch_idx(j + 2 * NS);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (j == -1) {
        wait_previous();  // q comes from the previous kernel
        load_q();
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    bad = __reduce_or_sync(0xffffffffu, (unsigned)bad);
    if (bad && lane == 0) atomicOr(ws.err, bad);

    // ---- the warps' states meet ----
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[n][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (r == 0) {
          s_ml[warp][8 * n + 2 * c + e][0] = m_run[n][e];
          s_ml[warp][8 * n + 2 * c + e][1] = l;
        }
      }
    if (lane == 0) s_bad[warp] = bad;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * c + e;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w][h][0]);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float mw = s_ml[w][h][0], lw = s_ml[w][h][1];
          // a warp without pieces has nothing; one whose scores are all NaN
          // never moved its reference and passes its NaN on
          L += mw == -INFINITY ? (lw == 0.f ? 0.f : lw) : fast_exp2(mw - M) * lw;
        }
        if (warp == 0 && r == 0 && h < G) {
          s_hml[h][0] = M;
          s_hml[h][1] = L;
        }
        const float f = m_run[n][e] == -INFINITY ? 1.f : fast_exp2(m_run[n][e] - M);
        if (h < G) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2 *>(obuf + h * C::RS + C::VB * r + 2 * i) =
                make_float2(acc[n][i][e] * f, acc[n][i][2 + e] * f);
        }
      }
    int unit_bad = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) unit_bad |= s_bad[w];
    __syncthreads();

    // ---- write: final row, or a partial (and maybe merge them all) ----
    const bool final_out = direct || un.n == 1;
    for (int i = tid * 4; i < G * D; i += C::THREADS * 4) {
      const int h = i / D, d = i - h * D;
      const float L = s_hml[h][1];
      const float inv = 1.f / L;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!unit_bad) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 y = *reinterpret_cast<const float4 *>(
              smem + w * (NS * C::STAGE) + (h * C::RS + d) * 4);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
      }
      const long long qrow = (long long)un.b * Hq + hq0 + h;
      if (!final_out) {
        *reinterpret_cast<float4 *>(ws.o_part + (qrow * pl.S + un.c) * D + d) = x;
      } else if (a.flags & PKV_FLAG_OUT_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(ws.out) + qrow * D + d) = x;
      } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(ws.out) + qrow * D + d) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      }
    }
    if (tid < G) {
      const float lse = unit_bad ? -INFINITY : s_hml[tid][0] * kLn2 + logf(s_hml[tid][1]);
      const long long qrow = (long long)un.b * Hq + hq0 + tid;
      if (final_out) {
        if (a.flags & PKV_FLAG_WRITE_LSE) ws.lse[qrow] = lse;
      } else {
        const long long o = (qrow * pl.S + un.c) * 2;
        ws.ml_part[o] = lse;
        ws.ml_part[o + 1] = unit_bad ? 0.f : 1.f;
      }
    }
    if (!final_out) {
      __syncthreads();
      if (tid == 0) {
        // the block's partial (ordered by the barrier) is released with the
        // ticket; the last taker acquires every other block's
        int *ctr = ws.split_counters + (long long)un.b * H + un.g;
        const int last = atomic_add_acq_rel_gpu(ctr, 1) == un.n - 1;
        if (last) *ctr = 0;  // ready for the next launch
        s_last = last;
      }
      __syncthreads();
      if (s_last && warp < G) {
        constexpr int RPW = G >= W ? G / W : 1;
        merge_rows_batched<D, RPW>(ws, (long long)un.b * Hq + hq0 + warp, W, pl.S, un.n, a.flags,
                                   lane);
      }
    }
    // the rings, s_ml and the ticket serve the next unit, the rings by copies of
    // the async proxy
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  wait_previous();
}

using TmapEncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// 3-D view of a code pool [NL * pool_slots, Hkv, D] as (byte, slot, head): a
// box of D x 16 x 1 is one 16-token piece of one head.
bool encode_codes_map(CUtensorMap *m, void *base, const pkv_workspace &ws) {
  static TmapEncodeFn fn = nullptr;
  static bool tried = false;
  if (!tried) {
    tried = true;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<TmapEncodeFn>(p);
  }
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
  // splits shared out by length need the compact plan and a sum that fits an int
  a.apportion = a.num_splits > 1 && a.batch <= kMaxCompactBatch &&
                (long long)a.batch * ws.max_pages_per_req * ws.page_size < 0x7fffffffll;
  return launch_pdl(kern, dim3(grid), dim3(C::THREADS), (size_t)C::SMEM, st, a, tmk, tmv);
}

template <int D, int G>
cudaError_t launch_shape(const Kv8Args &a, cudaStream_t st) {
  CUtensorMap tmk, tmv;
  memset(&tmk, 0, sizeof(tmk));
  memset(&tmv, 0, sizeof(tmv));
  const bool paged = a.ws.index_mode == PKV_IDX_PAGE_TABLE && a.ws.page_size % 16 == 0 &&
                     (long long)a.ws.n_layers * a.ws.pool_slots < 0x7fffffffll &&
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
    const cudaError_t e =
        launch_kv8_append(a.ws, a.c, a.batch, a.layer, 1, a.k_new, a.v_new, st);
    if (e != cudaSuccess) return e;
    a.flags &= ~PKV_FLAG_PLAN_EARLY;  // the append's rows are read
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
