// RMS norm of every query and key head with the position rotation, one pass.
//
// Each head is read once and written once; the bound is memory for long
// prompts and the launch for a decode step.  D / 16 lanes hold a head, two
// 16-byte chunks each, chosen so that both members of every rotated pair are
// in one lane: chunks (l, l + rot / 16) when the pairs are halves apart,
// adjacent chunks when they are adjacent elements.  The mean square is a sum
// of 16 products per lane and a butterfly over the head's lanes, in fp32.  The
// cosines and sines a lane needs do not depend on the head, so a warp loads
// them once for all the heads of its token that it handles.
//
// Measured (GB300; a pass in a graph): 32768 tokens of 32/8 heads 107.8 us, 6.4
// TB/s (96 % of the copy rate; 155 us when every group of heads read its token's
// row of the table again); 4 tokens 2.0 us, 1024 tokens of 16/2 heads 2.8 us.
#include <algorithm>

#include "kernels.cuh"

namespace pkv {

namespace {

constexpr int kRWarps = 4;

struct RopeArgs {
  pkv_qk_norm_rope_args p;
  int n_tokens, per_token;  // warps per token
  const uint16_t *q, *k;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  const int *positions;
  uint16_t *q_out, *k_out;
};

template <int D>
__global__ void __launch_bounds__(kRWarps * 32) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LG = D / 16;    // lanes per head
  constexpr int HPW = 32 / LG;  // heads side by side in a warp
  pdl_wait();
  pdl_trigger();
  const pkv_qk_norm_rope_args &p = a.p;
  const long long wid = (long long)blockIdx.x * kRWarps + (threadIdx.x >> 5);
  const long long tok = wid / a.per_token;
  if (tok >= a.n_tokens) return;
  const int part = (int)(wid - tok * a.per_token);
  const int lane = threadIdx.x & 31, l = lane % LG, sub = lane / LG;
  const int heads = p.n_q_heads + p.n_kv_heads, rot = p.rot_dim;
  // this lane's two chunks of 8 elements, and whether they rotate
  const bool turns = l < rot / 16;
  int c0, c1;
  if (p.interleaved) {
    c0 = 2 * l;
    c1 = c0 + 1;
  } else if (turns) {
    c0 = l;
    c1 = l + rot / 16;
  } else {
    c0 = rot / 8 + (l - rot / 16);
    c1 = c0 + (D - rot) / 16;
  }
  float cs[8], sn[8];
  bool bad = false;
  if (rot > 0) {
    const int pos = a.positions[tok];
    bad = pos < 0 || pos >= p.max_positions;
    // -1 is an empty request of a padded batch
    if (bad && pos != -1 && part == 0 && lane == 0) atomicOr(p.err, PKV_DEVERR_POSITION);
    if (turns && !bad) {
      const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (long long)pos * rot);
      *reinterpret_cast<float4 *>(cs) = row[2 * l];
      *reinterpret_cast<float4 *>(cs + 4) = row[2 * l + 1];
      *reinterpret_cast<float4 *>(sn) = row[rot / 8 + 2 * l];
      *reinterpret_cast<float4 *>(sn + 4) = row[rot / 8 + 2 * l + 1];
    }
  }
  const int groups = (heads + HPW - 1) / HPW;
  constexpr int UN = 2;  // groups whose loads are in flight together
  for (int i0 = part; i0 < groups; i0 += UN * a.per_token) {
    uint4 x[UN][2];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int hh = (i0 + k * a.per_token) * HPW + sub;
      x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
      if (i0 + k * a.per_token < groups && hh < heads) {
        const bool isk = hh >= p.n_q_heads;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            isk ? a.k + tok * a.k_stride + (long long)(hh - p.n_q_heads) * D
                : a.q + tok * a.q_stride + (long long)hh * D);
        x[k][0] = src[c0];
        x[k][1] = src[c1];
      }
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      if (i0 + k * a.per_token >= groups) break;  // warp-uniform
      const int hh = (i0 + k * a.per_token) * HPW + sub;
      const bool isk = hh >= p.n_q_heads;
      const int h = isk ? hh - p.n_q_heads : hh;
      float u[8], v[8];
      unpack8(x[k][0], u);
      unpack8(x[k][1], v);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
#pragma unroll
      for (int d = LG / 2; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if (hh >= heads) continue;
      const uint4 *w = static_cast<const uint4 *>(isk ? p.k_weight : p.q_weight);
      if (w) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        float wu[8], wv[8];
        unpack8(w[c0], wu);
        unpack8(w[c1], wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] *= r * wu[e];
          v[e] *= r * wv[e];
        }
      }
      if (turns) {
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = u[2 * e], b0 = u[2 * e + 1], a1 = v[2 * e], b1 = v[2 * e + 1];
            u[2 * e] = a0 * cs[e] - b0 * sn[e];
            u[2 * e + 1] = b0 * cs[e] + a0 * sn[e];
            v[2 * e] = a1 * cs[4 + e] - b1 * sn[4 + e];
            v[2 * e + 1] = b1 * cs[4 + e] + a1 * sn[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y0 = u[e], y1 = v[e];
            u[e] = y0 * cs[e] - y1 * sn[e];
            v[e] = y1 * cs[e] + y0 * sn[e];
          }
        }
      }
      uint4 *dst = reinterpret_cast<uint4 *>(isk ? a.k_out + tok * a.k_out_stride + (long long)h * D
                                                 : a.q_out + tok * a.q_out_stride + (long long)h * D);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      dst[c0] = bad ? zero
                    : make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                                 pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
      dst[c1] = bad ? zero
                    : make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
}

template <int D>
cudaError_t launch_one(RopeArgs a, cudaStream_t st) {
  const int per_warp = 32 / (D / 16);
  const int groups = (a.p.n_q_heads + a.p.n_kv_heads + per_warp - 1) / per_warp;
  // Warps per token: one per group of heads while that fits about one wave
  // (decode: latency counts), else as few as still give that many warps, so
  // that a token's cosines and sines are loaded once for many heads.
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const long long wave = 32ll * sms;
  a.per_token = (int)std::min<long long>(groups, std::max<long long>(1, wave / a.n_tokens));
  const long long blocks = ((long long)a.n_tokens * a.per_token + kRWarps - 1) / kRWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_pdl(qk_norm_rope_kernel<D>, dim3((unsigned)blocks), dim3(kRWarps * 32), 0, st, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const pkv_qk_norm_rope_args &p, int n_tokens, const void *q,
                                long long q_stride, const void *k, long long k_stride,
                                const int *positions, void *q_out, long long q_out_stride,
                                void *k_out, long long k_out_stride, cudaStream_t st) {
  const RopeArgs a{p, n_tokens, 1, static_cast<const uint16_t *>(q),
                   static_cast<const uint16_t *>(k), q_stride, k_stride, q_out_stride,
                   k_out_stride, positions, static_cast<uint16_t *>(q_out),
                   static_cast<uint16_t *>(k_out)};
  if (p.head_dim == 64) return launch_one<64>(a, st);
  if (p.head_dim == 128) return launch_one<128>(a, st);
  if (p.head_dim == 256) return launch_one<256>(a, st);
  return cudaErrorNotSupported;
}

}  // namespace pkv
