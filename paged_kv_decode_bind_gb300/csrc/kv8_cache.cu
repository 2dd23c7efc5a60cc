// The 8-bit cache's writes and read-back: rows quantised as they are appended
// (one per request, or a chunk per request) and cached rows back as bf16.
//
// All three move each byte once and are bound by memory for long inputs and
// by the chain of dependent loads (slot, scale, rows) for short ones.  Codes
// and scales follow pkv.h; every scale written is a power of two, so the values
// compared and rounded are exact and the results do not depend on the order
// of any sum.  A block that keeps a scale that is none divides by it (kv8.cuh).
//
// Measured (GB300; a pass in a graph): 64 decode rows with the blocks they touch
// read back 5.9 us; 4 x 256 rows with their 6500-row contexts read back 14.6 us;
// 32832 tokens of 8 heads read back 34.9 us, 5.8 TB/s (87 % of the copy rate),
// the same from 1 KB rows at random slots 81 %.  An append of 64 rows of 2 heads
// takes 2.0 us; when every block's scale grows, its last row's append takes 7.8 us at
// blocks of 16, 20 at 64, 38 at 128 (e4m3; int8 9.0, 25, 48): the older rows are
// rounded one after the other.  A chunk of 32768 rows of 8 heads takes 40.5 us in
// blocks of 16 (floor 30), 120 in blocks of 4 and 440-457 with a token a block, pages
// or flat: a warp has a single row then, and half its lanes idle.
#include "kernels.cuh"
#include "kv8.cuh"

namespace pkv {

namespace {

// 8 bf16 values in fp32.
__device__ __forceinline__ float row_max(const uint4 &v) {
  float f[8];
  unpack8(v, f);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(f[i]));
  return m;
}

template <int DT>
__device__ __forceinline__ uint2 encode8(const uint4 &v, float inv) {
  float f[8];
  unpack8(v, f);
  return make_uint2(encode4<DT>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    encode4<DT>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// Codes of 8 elements under a new scale: ratio = old scale / new scale.
template <int DT>
__device__ __forceinline__ uint2 recode8(const uint2 &w, float ratio) {
  float a[4], b[4];
  decode4<DT>(w.x, a);
  decode4<DT>(w.y, b);
  return make_uint2(encode4<DT>(a[0] * ratio, a[1] * ratio, a[2] * ratio, a[3] * ratio),
                    encode4<DT>(b[0] * ratio, b[1] * ratio, b[2] * ratio, b[3] * ratio));
}

// The same for 8 elements of rows r0, r0 + by, ... < r1 where the scale, or the
// ratio, is no power of two.  Functions of their own: the usual rows keep their
// registers (with both forms in the loops a block of 16 that grew took 9.1 us
// instead of 7.7, a chunk 4 % longer).
template <int DT>
__device__ __noinline__ void encode_rows_odd(uint2 *dst, const uint4 *src, long long step, int r0,
                                             int r1, int by, float s) {
#pragma unroll 1
  for (int r = r0; r < r1; r += by) {
    float f[8];
    unpack8(src[r * step], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = div_odd(f[i], s);
    dst[r * step] =
        make_uint2(encode4<DT>(f[0], f[1], f[2], f[3]), encode4<DT>(f[4], f[5], f[6], f[7]));
  }
}
template <int DT>
__device__ __noinline__ void recode_rows_odd(uint2 *dst, long long step, int r0, int r1, int by,
                                             float ratio) {
#pragma unroll 1
  for (int r = r0; r < r1; r += by) {
    float a[4], b[4];
    decode4<DT>(dst[r * step].x, a);
    decode4<DT>(dst[r * step].y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = mul_odd(a[i], ratio);
      b[i] = mul_odd(b[i], ratio);
    }
    dst[r * step] =
        make_uint2(encode4<DT>(a[0], a[1], a[2], a[3]), encode4<DT>(b[0], b[1], b[2], b[3]));
  }
}

// Scale of a block for new rows with finite maximum amax; `held`: the block
// already has rows under `old`.  *inv = 1 / scale, or 0 where the scale kept is
// no power of two (the appends write none, a cache may come with one).
template <int DT>
__device__ __forceinline__ float block_scale(float amax, bool held, float old, float *inv,
                                             bool *grown) {
  const int e = need_exp<DT>(amax);
  const float need = pow2i(e);
  *grown = held && !(old >= need);
  if (held && !*grown) {
    *inv = is_pow2(old) ? 1.f / old : 0.f;
    return old;
  }
  *inv = pow2i(-e);
  return need;
}

constexpr int kKAThreads = 256;

// One CTA per (request, layer).  D / 8 lanes hold one head's new row of K or
// V; its maximum is a butterfly over them.  Only a block whose scale grows is
// read again (at most scale_block - 1 rows of D bytes).
template <int D, int DT>
__global__ void __launch_bounds__(kKAThreads)
    kv8_append_kernel(const __grid_constant__ pkv_workspace ws, const __grid_constant__ pkv_kv8 c,
                      int batch, int layer_begin, bool early, const int *__restrict__ lens,
                      const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new) {
  if (early) pdl_trigger();  // the next kernel itself waits for what it must
  pdl_wait();
  if (!early) pdl_trigger();
  constexpr int LPR = D / 8;
  const int b = blockIdx.x, rel = blockIdx.y, layer = layer_begin + rel;
  const int loc = ws.out_loc[b], L = lens ? lens[b] : 1;
  if (L <= 0 || (long long)L > len_cap(ws)) return;  // no newest token, as in attention
  if (loc < 0 || loc >= ws.pool_slots) {
    if (threadIdx.x == 0) atomicOr(ws.err, PKV_DEVERR_SLOT);
    return;
  }
  const int H = ws.n_kv_heads, inside = loc % ws.page_size % c.scale_block;
  const int j = threadIdx.x % LPR;
  for (int i0 = 0; i0 < 2 * H; i0 += kKAThreads / LPR) {
    const int item = i0 + threadIdx.x / LPR;
    const bool live = item < 2 * H;
    const int side = item >= H, g = item - side * H;
    const uint4 *src = (side ? v_new : k_new) + (((long long)rel * batch + b) * H + g) * LPR + j;
    uint4 x = make_uint4(0, 0, 0, 0);
    float *sp = nullptr;
    float old = 0.f;
    if (live) {
      x = *src;
      sp = (side ? c.v_scale : c.k_scale) + scale_index(ws, c.scale_block, layer, loc, g);
      if (inside > 0) old = *sp;
    }
    float amax = row_max(x);
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    __syncwarp();  // every lane has read the old scale
    if (!live) continue;
    float inv;
    bool grown;
    const float s = block_scale<DT>(amax, inside > 0, old, &inv, &grown);
    uint8_t *pool = static_cast<uint8_t *>(side ? c.v_pool : c.k_pool);
    const long long row = ((long long)layer * ws.pool_slots + loc) * H + g;
    uint2 *dst = reinterpret_cast<uint2 *>(pool + row * D) + j;
    const long long step = (long long)H * LPR;  // 8-byte words between slots
    if (grown) {
      const float ratio = old * inv;
      if (is_pow2(ratio))
        for (int r = 1; r <= inside; ++r) dst[-r * step] = recode8<DT>(dst[-r * step], ratio);
      else
        recode_rows_odd<DT>(dst, step, -inside, 0, 1, ratio);
    }
    if (inv > 0.f) *dst = encode8<DT>(x, inv);
    else encode_rows_odd<DT>(dst, src, 0, 0, 1, 1, s);
    if (j == 0 && (inside == 0 || grown)) *sp = s;
  }
}

constexpr int kKXWarps = 4;
constexpr int kKXRows = 8;  // rows a lane keeps between the maximum and the rounding

// One warp per (request, block that gets rows, head, K or V): 32 / (D / 8)
// rows side by side.  Blocks of up to kKXRows passes stay in registers between
// the maximum and the rounding; larger ones are read a second time.  Eight CTAs
// an SM, 64 registers: with 72, which it would take, 32768 rows of 16-token
// blocks took 42.8 us instead of 40.5.
template <int D, int DT>
__global__ void __launch_bounds__(kKXWarps * 32, 8)
    kv8_extend_append_kernel(const __grid_constant__ pkv_workspace ws,
                             const __grid_constant__ pkv_kv8 c, int batch, int layer,
                             const int *__restrict__ qo_indptr, int max_qo_len, int per_req,
                             const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new) {
  pdl_wait();
  pdl_trigger();
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const int b = blockIdx.x / per_req;
  const bool lead = blockIdx.x == b * per_req && threadIdx.x == 0;
  const int q0 = qo_indptr[b], n = qo_indptr[b + 1] - q0, L = ws.seq_lens[b];
  bool ok = n >= 0 && n <= L && n <= max_qo_len && q0 >= 0 && q0 + n <= qo_indptr[batch] &&
            (long long)L <= len_cap(ws);
  long long base = 0;
  if (ok && ws.index_mode == PKV_IDX_FLAT) {
    base = ws.kv_indptr[b];
    ok = base >= 0 && base + L <= ws.max_total_tokens;
  } else if (ok) {
    const int row = ws.req_pool_indices[b];
    ok = row >= 0 && row < ws.max_reqs;
    base = ok ? (long long)row * ws.max_pages_per_req : 0;
  }
  if (!ok) {
    if (lead) atomicOr(ws.err, PKV_DEVERR_LEN);
    return;
  }
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int H = ws.n_kv_heads, SB = c.scale_block, P = ws.page_size;
  const int item = (blockIdx.x - b * per_req) * kKXWarps + (threadIdx.x >> 5);
  const int blk = item / (2 * H), hs = item - blk * 2 * H;
  const int side = hs >= H, g = hs - side * H;
  const int first = L - n;  // position of the first new token
  // blocks lie inside pages: block number = page * (P / SB) + block in page
  const int p0 = first / P, in0 = first - p0 * P;
  const int nb = p0 * (P / SB) + in0 / SB + blk;
  const int pg = nb / (P / SB), tb = pg * P + (nb - pg * (P / SB)) * SB;  // first position
  if (n == 0 || tb >= L) return;  // warp-uniform
  const int lo = max(first - tb, 0), hi = min(SB, L - tb);
  int kind = 0;
  const int slot = token_slot(ws, base, tb, &kind);
  if (slot < 0) {
    if (lane == 0 && hs == 0) atomicOr(ws.err, kind);
    return;
  }
  const long long step = (long long)H * LPR;  // 16-byte bf16 words, or 8-byte code words
  const uint4 *src = (side ? v_new : k_new) + ((long long)q0 + tb - first) * step + g * LPR + j;
  uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(side ? c.v_pool : c.k_pool)) +
               ((long long)layer * ws.pool_slots + slot) * step + g * LPR + j;
  float *sp = (side ? c.v_scale : c.k_scale) + scale_index(ws, SB, layer, slot, g);
  const float old = lo > 0 ? *sp : 0.f;

  uint4 v[kKXRows];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kKXRows; ++i) {
      const int r = r0 + i * RPP + sub;
      v[i] = r < hi ? src[r * step] : make_uint4(0, 0, 0, 0);
    }
  };
  float amax = 0.f;
  for (int r0 = lo; r0 < hi; r0 += kKXRows * RPP) {
    load(r0);
#pragma unroll
    for (int i = 0; i < kKXRows; ++i) amax = fmaxf(amax, row_max(v[i]));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  float inv;
  bool grown;
  const float s = block_scale<DT>(amax, lo > 0, old, &inv, &grown);
  if (grown) {
    const float ratio = old * inv;
    if (is_pow2(ratio))
      for (int r = sub; r < lo; r += RPP) dst[r * step] = recode8<DT>(dst[r * step], ratio);
    else
      recode_rows_odd<DT>(dst, step, sub, lo, RPP, ratio);
  }
  if (inv == 0.f) {  // the scale stays as it is
    encode_rows_odd<DT>(dst, src, step, lo + sub, hi, RPP, s);
    return;
  }
  const bool kept = hi - lo <= kKXRows * RPP;
  for (int r0 = lo; r0 < hi; r0 += kKXRows * RPP) {
    if (!kept) load(r0);
#pragma unroll
    for (int i = 0; i < kKXRows; ++i) {
      const int r = r0 + i * RPP + sub;
      if (r < hi) dst[r * step] = encode8<DT>(v[i], inv);
    }
  }
  if (lane == 0 && (lo == 0 || grown)) *sp = s;
}

constexpr int kKRThreads = 256;
constexpr int kKRTokens = 16;  // tokens per tile
constexpr int kKRUnroll = 4;  // rows whose loads a thread has in flight

// 32 bytes: one store where the address allows it.
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// CTAs launched for each one that fits the GPU at once.  Two: 32832 tokens of 8
// heads 34.7 us (one 37.2, three 34.5, four 34.8), 16 flat contexts 28.8 (29.8, 29.2,
// 29.0).  The second one's lay-out of the requests is work again: 64 x 2000 tokens of
// 2 heads 47.6 (46.6, 49.0, 50.4), 600 x 300 84 (78, 88, 96).
constexpr int kKRWaves = 2;
constexpr int kKRBatch = 256;  // requests whose tiles are laid out at a time

// The tiles of kKRTokens tokens of all requests, one after the other, go round
// the CTAs (one request's tiles over a share of the CTAs each left a batch of 16
// requests of 1 to 8192 tokens waiting for its longest: 35 us, against 29).
// A tile's slots and scale rows are resolved while the tile before it is read;
// then 2^tshift threads share a row of K or V, 16 codes (32 or 64 bytes of
// values) at a time, with kKRUnroll rows' loads issued before any is used.
template <int D, int DT, bool F32>
__global__ void __launch_bounds__(kKRThreads)
    kv8_read_kernel(const __grid_constant__ pkv_workspace ws, const __grid_constant__ pkv_kv8 c,
                    int batch, int layer, int tshift, bool early, const int *__restrict__ starts,
                    const int *__restrict__ dst_indptr, int n_rows, uint8_t *k_out,
                    uint8_t *v_out) {
  __shared__ int s_pref[kKRBatch + 1], s_n[kKRBatch], s_start[kKRBatch], s_row[kKRBatch];
  __shared__ long long s_base[kKRBatch];  // its index entries; -1: no row of the table
  __shared__ int s_slot[2][kKRTokens];         // -1: a bad index entry
  __shared__ long long s_scale[2][kKRTokens];  // index of head 0's scale in the layer
  if (!early) {
    pdl_wait();
    pdl_trigger();
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const bool flat = ws.index_mode == PKV_IDX_FLAT;
  const int H = ws.n_kv_heads, W = H * (D / 16);  // 16-code words of a token's row
  const int P = ws.page_size, per_page = P / c.scale_block, n_pages = ws.pool_slots / P;
  const uint4 *kp = static_cast<const uint4 *>(c.k_pool) + (long long)layer * ws.pool_slots * W;
  const uint4 *vp = static_cast<const uint4 *>(c.v_pool) + (long long)layer * ws.pool_slots * W;
  const long long srow = (long long)layer * n_pages * H * per_page;
  const float *ks = c.k_scale + srow, *vs = c.v_scale + srow;
  constexpr int OB = F32 ? 64 : 32;  // bytes of 16 values
  const bool wide =
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  const int col = tid & ((1 << tshift) - 1), rr = tid >> tshift;
  const int rows = kKRThreads >> tshift;  // rows side by side

  for (int g0 = 0; g0 < batch; g0 += kKRBatch) {
    const int nb = min(kKRBatch, batch - g0);
    __syncthreads();  // the last group is done with
    if (tid < 32) {
      int run = 0;
      for (int i = lane; i < (nb + 31) / 32 * 32; i += 32) {
        const int b = g0 + i;
        int n = 0, kind = 0, start = 0, row0 = 0;
        long long base = 0;
        if (i < nb) {
          const int L = ws.seq_lens[b];
          start = starts ? starts[b] : 0;
          row0 = dst_indptr[b];
          base = flat ? ws.kv_indptr[b] : ws.req_pool_indices[b];
          if (L < 0 || (long long)L > len_cap(ws) || start < 0) kind = PKV_DEVERR_LEN;
          else n = max(L - start, 0);
          if (n > 0 && (row0 < 0 || (long long)row0 + n > n_rows)) kind = PKV_DEVERR_TOTAL;
          if (n > 0 && flat && (base < 0 || base + L > ws.max_total_tokens))
            kind = PKV_DEVERR_TOTAL;
          // no row of the table: every token is bad (written as zeros below)
          if (!flat) base = base >= 0 && base < ws.max_reqs ? base * ws.max_pages_per_req : -1;
          if (kind) {
            if (blockIdx.x == 0) atomicOr(ws.err, kind);
            n = 0;
          }
        }
        const int tiles = (n + kKRTokens - 1) / kKRTokens;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        if (i < nb) {
          s_pref[i] = run + incl - tiles;
          s_n[i] = n;
          s_start[i] = start;
          s_row[i] = row0;
          s_base[i] = base;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) s_pref[nb] = run;
    }
    __syncthreads();
    const int total = s_pref[nb];
    // request (in the group) of a tile
    auto find = [&](int tile) {
      int lo = 0, hi = nb - 1;  // last one with pref <= tile
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pref[mid] <= tile) lo = mid;
        else hi = mid - 1;
      }
      return lo;
    };
    // threads 0 .. 15 resolve a tile's tokens: the raw entry early, the slot late
    int raw = -1, tok = 0;
    auto fetch = [&](int tile) {
      raw = -1;
      if (tid < kKRTokens && tile < total) {
        const int q = find(tile), t = (tile - s_pref[q]) * kKRTokens + tid;
        if (t < s_n[q] && s_base[q] >= 0) {
          tok = s_start[q] + t;
          raw = flat ? ws.kv_indices[s_base[q] + tok] : ws.page_table[s_base[q] + tok / P];
        }
      }
    };
    auto resolve = [&](int tile, int buf) {
      if (tid < kKRTokens && tile < total) {
        const int q = find(tile), t = (tile - s_pref[q]) * kKRTokens + tid;
        if (t < s_n[q]) {
          int slot = -1, page = 0;
          if (raw >= 0 && raw < (flat ? ws.pool_slots : n_pages)) {
            page = flat ? raw / P : raw;
            slot = flat ? raw : raw * P + tok % P;
          } else {
            atomicOr(ws.err, flat ? PKV_DEVERR_SLOT : PKV_DEVERR_PAGE);
          }
          s_slot[buf][tid] = slot;
          s_scale[buf][tid] = (long long)page * H * per_page +
                              (slot >= 0 ? (slot - page * P) / c.scale_block : 0);
        }
      }
    };
    fetch(blockIdx.x);
    resolve(blockIdx.x, 0);
    if (early && g0 == 0) {  // codes, scales and the output's last readers
      pdl_wait();
      pdl_trigger();
    }
    int buf = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, buf ^= 1) {
      __syncthreads();  // this tile's slots; and the other buffer is free
      fetch(tile + gridDim.x);
      const int q = find(tile), t0 = (tile - s_pref[q]) * kKRTokens;
      const int m = min(kKRTokens, s_n[q] - t0);
      const long long row0 = (long long)s_row[q] + t0;
      for (int w = col; w < W; w += 1 << tshift) {
        const long long head = (long long)(w / (D / 16)) * per_page;
        // row i of the tile: K of token i, then V of token i - m
        for (int i0 = rr; i0 < 2 * m; i0 += kKRUnroll * rows) {
          uint4 code[kKRUnroll];
          float s[kKRUnroll];
#pragma unroll
          for (int k = 0; k < kKRUnroll; ++k) {
            const int i = i0 + k * rows;
            const bool isv = i >= m;
            const int t = isv ? i - m : i;
            code[k] = make_uint4(0, 0, 0, 0);
            s[k] = 0.f;
            if (i < 2 * m && s_slot[buf][t] >= 0) {
              code[k] = ldg_nc_v4((isv ? vp : kp) + (long long)s_slot[buf][t] * W + w);
              s[k] = (isv ? vs : ks)[s_scale[buf][t] + head];
            }
          }
#pragma unroll
          for (int k = 0; k < kKRUnroll; ++k) {
            const int i = i0 + k * rows;
            if (i >= 2 * m) break;
            const bool isv = i >= m;
            const int t = isv ? i - m : i;
            const uint32_t cw[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
            float f[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a[4];
              decode4<DT>(cw[e], a);
#pragma unroll
              for (int y = 0; y < 4; ++y) f[4 * e + y] = a[y] * s[k];
            }
            uint8_t *p = (isv ? v_out : k_out) + ((row0 + t) * W + w) * OB;
            if constexpr (F32) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(f[8 * h + e]);
                store32(p + 32 * h, o, wide);
              }
            } else {
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
              store32(p, o, wide);
            }
          }
        }
      }
      resolve(tile + gridDim.x, buf ^ 1);
    }
  }
}

template <typename F>
cudaError_t by_shape(const pkv_workspace &ws, const pkv_kv8 &c, F f) {
  if (ws.head_dim == 128)
    return c.dtype == PKV_KV8_E4M3 ? f.template operator()<128, PKV_KV8_E4M3>()
                                   : f.template operator()<128, PKV_KV8_INT8>();
  if (ws.head_dim == 64)
    return c.dtype == PKV_KV8_E4M3 ? f.template operator()<64, PKV_KV8_E4M3>()
                                   : f.template operator()<64, PKV_KV8_INT8>();
  return cudaErrorNotSupported;
}

struct AppendLaunch {
  const pkv_workspace &ws;
  const pkv_kv8 &c;
  int batch, layer_begin, layer_count;
  const void *k, *v;
  bool early;
  const int *lens;
  cudaStream_t st;
  template <int D, int DT>
  cudaError_t operator()() {
    return launch_pdl(kv8_append_kernel<D, DT>, dim3(batch, layer_count), dim3(kKAThreads), 0, st,
                      ws, c, batch, layer_begin, early, lens, static_cast<const uint4 *>(k),
                      static_cast<const uint4 *>(v));
  }
};

struct ExtendAppendLaunch {
  const pkv_workspace &ws;
  const pkv_kv8 &c;
  int batch, layer;
  const int *qo_indptr;
  int max_qo_len;
  const void *k, *v;
  cudaStream_t st;
  template <int D, int DT>
  cudaError_t operator()() {
    // a request's new rows touch at most this many blocks
    const long long blocks = ((long long)max_qo_len + c.scale_block - 1) / c.scale_block + 1;
    const long long per = (blocks * 2 * ws.n_kv_heads + kKXWarps - 1) / kKXWarps;
    if (per * batch > 0x7fffffffll || blocks * 2 * ws.n_kv_heads > 0x7fffffffll)
      return cudaErrorInvalidConfiguration;
    return launch_pdl(kv8_extend_append_kernel<D, DT>, dim3((unsigned)(per * batch)),
                      dim3(kKXWarps * 32), 0, st, ws, c, batch, layer, qo_indptr, max_qo_len,
                      (int)per, static_cast<const uint4 *>(k), static_cast<const uint4 *>(v));
  }
};

struct ReadLaunch {
  const pkv_workspace &ws;
  const pkv_kv8 &c;
  int batch, layer;
  const int *starts, *dst_indptr;
  int n_rows;
  void *k, *v;
  int flags;
  cudaStream_t st;
  template <int D, int DT, bool F32>
  cudaError_t launch() {
    auto kern = kv8_read_kernel<D, DT, F32>;
    static int resident[64] = {0};  // blocks that fit an SM, asked once per device
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = device_sms(&sms);
    int &occ = resident[dev & 63];
    if (e == cudaSuccess && occ == 0)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kKRThreads, 0);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)n_rows / kKRTokens + batch;  // at most
    const long long most = (long long)sms * (occ > 0 ? occ : 1) * kKRWaves;
    const unsigned grid = (unsigned)(tiles < most ? tiles : most);
    // threads per row: the power of two that covers its 16-code words, 256 at most
    int tshift = 0;
    while (tshift < 8 && (1 << tshift) < ws.n_kv_heads * (D / 16)) ++tshift;
    return launch_pdl(kern, dim3(grid), dim3(kKRThreads), 0, st, ws, c, batch, layer, tshift,
                      (flags & PKV_FLAG_PLAN_EARLY) != 0, starts, dst_indptr, n_rows,
                      static_cast<uint8_t *>(k), static_cast<uint8_t *>(v));
  }
  template <int D, int DT>
  cudaError_t operator()() {
    return flags & PKV_FLAG_OUT_F32 ? launch<D, DT, true>() : launch<D, DT, false>();
  }
};

}  // namespace

cudaError_t launch_kv8_append(const pkv_workspace &ws, const pkv_kv8 &c, int batch,
                              int layer_begin, int layer_count, const void *k_new,
                              const void *v_new, bool early, const int *lens,
                              cudaStream_t st) {
  return by_shape(ws, c, AppendLaunch{ws, c, batch, layer_begin, layer_count, k_new, v_new, early,
                                      lens, st});
}

cudaError_t launch_kv8_extend_append(const pkv_workspace &ws, const pkv_kv8 &c, int batch,
                                     int layer, const int *qo_indptr, int max_qo_len,
                                     const void *k_new, const void *v_new, cudaStream_t st) {
  return by_shape(
      ws, c, ExtendAppendLaunch{ws, c, batch, layer, qo_indptr, max_qo_len, k_new, v_new, st});
}

cudaError_t launch_kv8_read(const pkv_workspace &ws, const pkv_kv8 &c, int batch, int layer,
                            const int *starts, const int *dst_indptr, int n_rows, void *k_out,
                            void *v_out, int flags, cudaStream_t st) {
  return by_shape(ws, c, ReadLaunch{ws, c, batch, layer, starts, dst_indptr, n_rows, k_out, v_out,
                                    flags, st});
}

}  // namespace pkv
