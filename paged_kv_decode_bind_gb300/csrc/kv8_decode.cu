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
// Data.  Each warp takes every W-th piece of 16 tokens of the unit and has its
// own ring of stages in shared memory, filled by 16-byte cp.async copies whose
// destination a lane later reads itself: K rows as the A fragments of S^T
// (lane r = lane / 4, c = lane % 4 reads 16 bytes of rows r and r + 8; which
// head_dim a fragment's k index means is free, as long as Q agrees), V rows as
// 4 tokens x 16 bytes, whose bytes one byte permute per word interleaves into
// the (token, token + 1) pairs of the A fragments of O^T.  So no barrier and
// no transposition stand between a copy and its product; only the scales
// (one 4-byte copy per lane) and, without whole 16-token pages, the slots
// cross lanes.
//
// The warps' states meet in shared memory at the end of a unit; the splits of
// a request meet in the block that finishes last (an atomic ticket).
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
  static constexpr int SMEM = W * NS * STAGE;
  static_assert(NS * STAGE >= G * RS * 4, "a warp's O fits its ring");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// PAGED: pages hold whole 16-token pieces, so a piece has one page id.
template <int D, int G, int DT, bool PAGED>
__global__ void __launch_bounds__(KCfg<D, G>::THREADS, 2)
    kv8_decode_kernel(const __grid_constant__ Kv8Args a) {
  using C = KCfg<D, G>;
  constexpr int W = C::W, NS = C::NS, NH = C::NH;
  // log2 of the largest weight where r is placed, and where it has to move
  constexpr float kPlace = 7.f, kMove = 15.f;
  extern __shared__ __align__(128) uint8_t smem[];
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
  const pkv_workspace &ws = a.ws;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int Hq = ws.n_q_heads, H = ws.n_kv_heads;
  const bool early = (a.flags & PKV_FLAG_PLAN_EARLY) != 0;
  if (!early) {
    pdl_wait();
    pdl_trigger();
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

  const uint32_t ring = smem_addr(smem) + warp * (NS * C::STAGE);
  float *obuf = reinterpret_cast<float *>(smem + warp * (NS * C::STAGE));
  const int SB = a.c.scale_block, per_page = ws.page_size / SB;
  const int sshift = (SB & (SB - 1)) == 0 ? __ffs(SB) - 1 : -1;
  const uint8_t *kpool = static_cast<const uint8_t *>(a.c.k_pool);
  const uint8_t *vpool = static_cast<const uint8_t *>(a.c.v_pool);
  const int rs = H * D;  // bytes between the rows of consecutive slots
  const long long layer_slot = (long long)a.layer * ws.pool_slots;
  const long long layer_page = (long long)a.layer * pl.n_pages;

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
    const int np = (pieces - warp + W - 1) / W;  // this warp's (0 or less: none)
    const ReqIndex ri = pl.pref ? req_index_cached(ws, s_base, un.b) : req_index(ws, un.b);
    int bad = ri.ok ? 0 : PKV_DEVERR_PAGE;
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
    // The copies of piece j into its stage (one commit group each, possibly
    // empty); rows past the unit's end and rows without a slot become zeros.
    auto issue = [&](int j) {
      if (j < np) {
        const int st = j % NS;
        const uint32_t kd = ring + st * C::STAGE + lane * 16;
        const uint32_t vd = ring + st * C::STAGE + C::KB + lane * C::VB;
        const int tok0 = piece_tok(j), nv = min(16, un.t1 - tok0);
        const int tt = lane & 15;  // lanes 0-15: K scale of token tt, 16-31: V scale
        const float *sbase = lane < 16 ? a.c.k_scale : a.c.v_scale;
        const uint32_t sd = smem_addr(&s_scale[warp][st][lane]);
        if constexpr (PAGED) {
          const int page = __shfl_sync(0xffffffffu, pg, j & 31);
          const bool ok = page >= 0 && page < pl.n_pages;
          if (!ok) bad |= PKV_DEVERR_PAGE;
          const int in0 = pl.in_page(tok0);
          const long long row0 =
              ok ? ((layer_slot + (long long)page * pl.P + in0) * H + un.g) * D : 0;
          const int n = ok ? nv : 0;
          const uint8_t *kp = kpool + row0 + r * rs + 16 * c;
          const uint8_t *vp = vpool + row0 + 2 * c * rs + C::VB * r;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            cp16(kd + i * 512, kp + (i & 1) * 8 * rs + (i >> 1) * 64,
                 r + 8 * (i & 1) < n ? 16 : 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) cp16(vd + i * 512, vp + row * rs, 2 * c + row < n ? 16 : 0);
            else cp8(vd + i * 256, vp + row * rs, 2 * c + row < n ? 8 : 0);
          }
          const int sub = sshift >= 0 ? (in0 + tt) >> sshift : (in0 + tt) / SB;
          const long long si =
              ok ? ((layer_page + page) * H + un.g) * per_page + (tt < n ? sub : 0) : 0;
          cp4(sd, sbase + si, tt < n ? 4 : 0);
          if ((j & 31) == 31) {
            pg = pg_next;
            pg_next = load_pages(j + 33);
          }
        } else {
          const int *raw = s_idx[warp][j % (2 * NS)];
          // a slot, or -1 past the end or for a bad entry
          auto slot_of = [&](int row) {
            int kind = 0;
            const int s =
                row < nv ? (int)slot_from_raw(ws, pl, raw[row], tok0 + row, kind) : -1;
            bad |= kind;
            return s;
          };
#pragma unroll
          for (int hlf = 0; hlf < 2; ++hlf) {
            const int s = slot_of(r + 8 * hlf);
            const uint8_t *kp =
                kpool + (s >= 0 ? ((layer_slot + s) * H + un.g) * D + 16 * c : 0);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
              cp16(kd + (2 * i + hlf) * 512, kp + i * 64, s >= 0 ? 16 : 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int s = slot_of(2 * c + (i & 1) + 8 * (i >> 1));
            const uint8_t *vp =
                vpool + (s >= 0 ? ((layer_slot + s) * H + un.g) * D + C::VB * r : 0);
            if constexpr (D == 128) cp16(vd + i * 512, vp, s >= 0 ? 16 : 0);
            else cp8(vd + i * 256, vp, s >= 0 ? 8 : 0);
          }
          const int s = slot_of(tt);
          long long si = 0;
          if (s >= 0)
            si = pl.P == 1 ? (layer_slot + s) * H + un.g : scale_index(ws, SB, a.layer, s, un.g);
          cp4(sd, sbase + si, s >= 0 ? 4 : 0);
        }
      }
      fetch_idx(j + NS);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if constexpr (PAGED) {
      pg = load_pages(0);
      pg_next = load_pages(32);
    } else {
      for (int j = 0; j < NS; ++j) fetch_idx(j);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
    for (int j = 0; j < NS; ++j) issue(j);

    // Q^T as the B operand: lane r is head r (+ 8), its 16 elements 64 x + 16 c
    // .. 64 x + 16 c + 15 of each half x match the K bytes the lane reads.
    wait_previous();
    uint32_t qb[NH][D / 16][2];
    float qs[NH][2];  // scale of heads 2 c and 2 c + 1, log2 units
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

    for (int j = 0; j < np; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
      __syncwarp();  // the other lanes' scales and index entries too
      const int st = j % NS;
      const uint8_t *stage = smem + warp * (NS * C::STAGE) + st * C::STAGE;
      // ---- S^T = K Q^T ----
      float sc[NH][4], sc2[NH][4];
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = sc2[n][i] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(stage + (2 * x) * 512 + lane * 16);
        const uint4 hi = *reinterpret_cast<const uint4 *>(stage + (2 * x + 1) * 512 + lane * 16);
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
      // ---- weights: tokens r and r + 8, heads 2 c and 2 c + 1 ----
      const float *ss = s_scale[warp][st];
      const float ks[2] = {ss[r], ss[r + 8]}, vs[2] = {ss[16 + r], ss[24 + r]};
      const int nv = un.t1 - piece_tok(j);
      const bool live[2] = {r < nv, r + 8 < nv};
      const float lv[2] = {fast_log2(vs[0]), fast_log2(vs[1])};
      bool move = false;
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float s = (sc[n][2 * t + e] + sc2[n][2 * t + e]) * ks[t] * qs[n][e];
            sc[n][2 * t + e] = live[t] ? s : -INFINITY;
            move |= live[t] && s + lv[t] > m_run[n][e] + kMove;
          }
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = live[0] ? sc[n][e] + lv[0] : -INFINITY;
            t = fmaxf(t, live[1] ? sc[n][2 + e] + lv[1] : -INFINITY);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float mn = fmaxf(m_run[n][e], t - kPlace);
            al[e] = mn == -INFINITY ? 1.f : exp2f(m_run[n][e] - mn);
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
      uint32_t wb[NH][2];  // W^T as B: tokens 0-7 / 8-15
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = live[t] ? exp2f(sc[n][2 * t + e] - m_run[n][e]) : 0.f;
            l_run[n][e] += p;
            w[e] = p * vs[t];
          }
          wb[n][t] = movmatrix_t(pack_f16x2(w[0], w[1]));
        }
      // ---- O^T += V^T W^T ----
      uint32_t v[4][C::VB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t *src = stage + C::KB + i * (32 * C::VB) + lane * C::VB;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4 *>(src);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(src);
          v[i][0] = x.x, v[i][1] = x.y;
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
      __syncwarp();  // every lane is done with the stage
      issue(j + NS);
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
          L += mw == -INFINITY ? (lw == 0.f ? 0.f : lw) : exp2f(mw - M) * lw;
        }
        if (warp == 0 && r == 0 && h < G) {
          s_hml[h][0] = M;
          s_hml[h][1] = L;
        }
        const float f = m_run[n][e] == -INFINITY ? 1.f : exp2f(m_run[n][e] - M);
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
    __syncthreads();  // the rings, s_ml and the ticket serve the next unit
  }
  wait_previous();
}

template <int D, int G, int DT, bool PAGED>
cudaError_t launch_one(Kv8Args a, cudaStream_t st) {
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
  return launch_pdl(kern, dim3(grid), dim3(C::THREADS), (size_t)C::SMEM, st, a);
}

template <int D, int G>
cudaError_t launch_shape(const Kv8Args &a, cudaStream_t st) {
  const bool paged = a.ws.index_mode == PKV_IDX_PAGE_TABLE && a.ws.page_size % 16 == 0;
  if (a.c.dtype == PKV_KV8_E4M3)
    return paged ? launch_one<D, G, PKV_KV8_E4M3, true>(a, st)
                 : launch_one<D, G, PKV_KV8_E4M3, false>(a, st);
  return paged ? launch_one<D, G, PKV_KV8_INT8, true>(a, st)
               : launch_one<D, G, PKV_KV8_INT8, false>(a, st);
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
