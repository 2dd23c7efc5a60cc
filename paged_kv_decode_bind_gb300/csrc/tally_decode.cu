// Decode attention with the tally: the tensor-core kernel also stores every token's
// scores (decode_mma.cuh), and a second launch turns them into weights.
//
//   weight[t, g] += sum over the group's heads of 2^(score_t,h - lse_h log2 e)
//
// A weight needs the log-sum-exp of its whole request, which exists only once the last
// split is merged, so it cannot be added where the score is made.  The scores are 4 G
// bytes a token and head beside the 4 D of its K and V (3 % at G = 4, D = 128), stay in
// L2, and spare a second reading of K.
//
// Measured (GB300, us a layer in graphs of 24): 64 requests of 1024-4096 tokens, 16/2 heads
// 43.8 (33.9 without the tally), 16 of 2048, 32/8 heads, 32.7 (27.2), 4 of 512-2048 11.7
// (8.9), 16 flat of 200-4000 42.5 (33.3).  Of 4 x 65536 tokens (190 us, 161 without) the
// scores' stores take 13 us and the second launch 16.
#include <algorithm>

#include "decode_mma.cuh"
#include "tally.cuh"

namespace pkv {

namespace {

constexpr int kTThreads = 256;
template <int G>
constexpr int kAddBlocks = G == 4 ? 6 : G <= 8 ? 5 : 4;  // of an SM (G = 16: 64 registers)
// Whether the next items' indices come beside an item's loads.  24 layers' steps, us a layer,
// of 16 requests of 2048 tokens and 16 flat of 200-4000 (G = 8: 64 of 1024-4096), with them in
// five blocks, and without in six: G = 1 31.7 and 40.5, 31.5 and 40.6; G = 2 32.6 and 42.8,
// 33.1 and 43.8 (40 registers spill); G = 4 33.6 and 43.1, 32.8 and 42.4; G = 8 44.0, 44.2.
template <int G>
constexpr bool kAddAhead = G != 4;
// Items of a warp whose loads are in flight (the same loads: G = 8 44.9 with two in four
// blocks, G = 4 34.9 with one).
template <int G>
constexpr int kAddItems = G <= 4 ? 2 : 1;

struct TallyArgs {
  pkv_workspace ws;
  pkv_tally t;
  int batch, layer;
  int appended;  // the newest token's entry starts anew
  int tl_log, hl_log;  // a warp takes 2^tl tokens of 2^hl KV heads
};

// G consecutive values that the launch before has written.
template <int G>
__device__ __forceinline__ void load_group(float (&x)[G], const float *s) {
  if constexpr (G >= 4) {
#pragma unroll
    for (int h = 0; h < G; h += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + h));
      x[h] = v.x;
      x[h + 1] = v.y;
      x[h + 2] = v.z;
      x[h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int h = 0; h < G; ++h) x[h] = __ldcg(s + h);
  }
}

// One item of a warp: 2^tl_log tokens x 2^hl_log heads, a lane each.  Tokens run fastest
// over the lanes, so that a page's entries of a head, and a head's scores, are read in
// runs.  A warp has UN items' loads in flight, and may look the next ones' indices up beside
// them.
//
// The launch waits for the attention only where it reads what that writes, the scores and
// log-sum-exps: lengths, tables and the tally are older than the attention's own start,
// as this launch starts behind the attention's wait for its predecessor.
template <int G>
__global__ void __launch_bounds__(kTThreads, kAddBlocks<G>)
    tally_add_kernel(const __grid_constant__ TallyArgs a) {
  constexpr int UN = kAddItems<G>;
  const pkv_workspace &ws = a.ws;
  pdl_trigger();
  Plan pl;
  pl.set_pages(ws);
  const int lane = threadIdx.x & 31;
  const int ts = lane & ((1 << a.tl_log) - 1), hs = lane >> a.tl_log;
  const int hgroups = (ws.n_kv_heads + (1 << a.hl_log) - 1) >> a.hl_log;
  const int Hq = ws.n_q_heads;
  bool waited = false;
  for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
    const int L = usable_len(ws, b);
    const ReqIndex ri = req_index(ws, b);
    const int row = ws.req_pool_indices[b];
    const bool row_ok = row >= 0 && row < ws.max_reqs;
    // a warp keeps its head group and strides over the groups of tokens
    const int tgroups = row_ok && ri.ok ? (L + (1 << a.tl_log) - 1) >> a.tl_log : 0;
    const int wid = blockIdx.x * (kTThreads / 32) + (threadIdx.x >> 5);
    const int step = gridDim.x * (kTThreads / 32) / hgroups;  // >= 1
    const int tg0 = wid / hgroups, g = ((wid - tg0 * hgroups) << a.hl_log) + hs;
    const int first = g < ws.n_kv_heads && tg0 < step ? tg0 : tgroups;
    float l2[G];  // the heads' lse log2 e; +inf: the attention was written as empty
    int raw[UN];
    auto look_up = [&](int t0) {
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = ((t0 + u * step) << a.tl_log) + ts;
        raw[u] = t0 + u * step < tgroups && t < L ? *index_src(ws, pl, ri, t) : -1;
      }
    };
    if constexpr (kAddAhead<G>) look_up(first);
    for (int t0 = first; __any_sync(0xffffffffu, t0 < tgroups); t0 += UN * step) {
      if constexpr (!kAddAhead<G>) look_up(t0);
      long long at[UN];
      float was[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = ((t0 + u * step) << a.tl_log) + ts;
        int kind = 0;  // the attention has raised it
        const int slot = (int)slot_from_raw(ws, pl, raw[u], t, kind);
        at[u] = -1;
        was[u] = 0.f;
        if (slot < 0) continue;
        const int page = pl.page_of(slot);
        at[u] = tally_at(ws, pl.n_pages, a.layer, page, g, slot - page * pl.P);
        if (!(a.appended && t == L - 1)) was[u] = a.t.weight[at[u]];
      }
      if constexpr (kAddAhead<G>) look_up(t0 + UN * step);
      if (!waited) {
        pdl_wait();
        waited = true;
      }
      float x[UN][G];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = ((t0 + u * step) << a.tl_log) + ts;
        if (at[u] >= 0)
          load_group<G>(
              x[u], a.t.score + (((long long)b * ws.n_kv_heads + g) * a.t.score_tokens + t) * G);
      }
      if (t0 == first) {
        if (g < ws.n_kv_heads) load_group<G>(l2, ws.lse + (long long)b * Hq + g * G);
#pragma unroll
        for (int h = 0; h < G; ++h) l2[h] = l2[h] > -INFINITY ? l2[h] * kLog2e : INFINITY;
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int t = ((t0 + u * step) << a.tl_log) + ts;
        if (at[u] < 0) continue;
        float w = 0.f;
#pragma unroll
        for (int h = 0; h < G; ++h) w += tally_clean(exp2f(x[u][h] - l2[h]));
        a.t.weight[at[u]] = was[u] + w;
        if (a.appended && t == L - 1) a.t.origin[at[u]] = L - 1 + a.t.evicted[row];
      }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && L > 0 && !row_ok)
      atomicOr(ws.err, PKV_DEVERR_PAGE);
  }
  if (!waited) pdl_wait();
}

template <int G>
cudaError_t launch_add(const DecodeArgs &a, const pkv_tally &t, cudaStream_t st) {
  const pkv_workspace &ws = a.ws;
  TallyArgs g{ws, t, a.batch, a.layer, a.k_new != nullptr, 0, 0};
  // Pages of 32 tokens and more: a warp reads 32 of one head's.  Smaller ones: the same
  // page's next heads, whose entries follow, down to 4 tokens of 8 heads for flat
  // indices, where a slot's heads share a 32-byte sector.
  g.tl_log = 2;
  while (g.tl_log < 5 && (2 << g.tl_log) <= ws.page_size) ++g.tl_log;
  while (g.tl_log < 5 && (1 << (4 - g.tl_log)) >= ws.n_kv_heads) ++g.tl_log;
  g.hl_log = 5 - g.tl_log;
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  // about one wave of resident warps, shared by the requests, and no more than the longest
  // request that the table allows has items for
  const int by = a.batch < 65535 ? a.batch : 65535;
  const int hgroups = (ws.n_kv_heads + (1 << g.hl_log) - 1) >> g.hl_log;
  constexpr int per = kTThreads / 32;
  const long long items = ((len_cap(ws) + (1 << g.tl_log) - 1) >> g.tl_log) * hgroups;
  constexpr int each = kAddItems<G> * per;
  const long long need = (items + each - 1) / each;
  const int wave = (kAddBlocks<G> * sms + by - 1) / by, least = (hgroups + per - 1) / per;
  const int bx = std::max(least, (int)std::min<long long>(wave, need));
  return launch_pdl(tally_add_kernel<G>, dim3(bx, by), dim3(kTThreads), 0, st, g);
}

}  // namespace

cudaError_t launch_tally_decode(const DecodeArgs &a0, const pkv_tally &t, cudaStream_t st) {
  DecodeArgs a = a0;
  a.flags |= PKV_FLAG_WRITE_LSE;
  a.score = t.score;
  a.score_tokens = t.score_tokens;
  const int D = a.ws.head_dim, G = a.ws.n_q_heads / a.ws.n_kv_heads;
  cudaError_t e = cudaErrorNotSupported;
#define PKV_TALLY_CASE(DD, GG) \
  if (D == DD && G == GG) e = launch_mma_one<DD, GG, true>(a, st);
  PKV_TALLY_CASE(128, 1) PKV_TALLY_CASE(128, 2) PKV_TALLY_CASE(128, 4) PKV_TALLY_CASE(128, 8)
  PKV_TALLY_CASE(128, 16) PKV_TALLY_CASE(64, 1) PKV_TALLY_CASE(64, 2) PKV_TALLY_CASE(64, 4)
  PKV_TALLY_CASE(64, 8) PKV_TALLY_CASE(64, 16)
#undef PKV_TALLY_CASE
  if (e != cudaSuccess) return e;
  switch (G) {
    case 1: return launch_add<1>(a, t, st);
    case 2: return launch_add<2>(a, t, st);
    case 4: return launch_add<4>(a, t, st);
    case 8: return launch_add<8>(a, t, st);
    case 16: return launch_add<16>(a, t, st);
  }
  return cudaErrorNotSupported;
}

}  // namespace pkv
