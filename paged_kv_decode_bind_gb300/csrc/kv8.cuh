// 8-bit KV cache: code types, block scales and slot arithmetic shared by its
// append, read-back and attention kernels (see pkv_kv8 in pkv.h).
//
// A scale is a power of two, so dividing a bf16 value by it, and reading
// code * scale back as bf16, are exact: the only rounding is the one to the
// code.  For e4m3 a power of two costs nothing (its own exponent takes up the
// difference); for int8 it costs less than one bit against amax / 127, and
// makes a block that grows lose at most its low bits once.  A cache may come with
// other scales, as a calibration leaves them: rows appended to a block that keeps
// such a scale divide by it, rounded to odd, so that the code is the one nearest
// to the exact quotient.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kKv8MaxBlock = 128;
constexpr int kKv8MinExp = -100, kKv8MaxExp = 100;

struct Kv8Args {
  pkv_workspace ws;
  pkv_kv8 c;
  int batch, layer;
  const void *q, *k_new, *v_new;
  float scale;
  int num_splits, flags;
  int apportion;  // set by the launcher: splits shared out by length
};

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Smallest e in [kKv8MinExp, kKv8MaxExp] with amax <= qmax * 2^e, for a finite
// amax >= 0, from its bits: amax = (1 + f / 2^23) 2^x against qmax = 1.75 * 2^8
// (e4m3) or 1.984375 * 2^6 (int8).
template <int DT>
__device__ __forceinline__ int need_exp(float amax) {
  constexpr int kShift = DT == PKV_KV8_E4M3 ? 8 : 6;
  constexpr int kTop = DT == PKV_KV8_E4M3 ? 0x600000 : 0x7e0000;
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - 127 - kShift + ((bits & 0x7fffff) > kTop ? 1 : 0);
  return amax > 0.f ? max(kKv8MinExp, min(kKv8MaxExp, e)) : kKv8MinExp;
}

__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_int(s) & 0x7fffff) == 0; }

// A value rounded towards zero, and what was cut off: rounded to odd.  A later
// rounding to at most 22 bits then gives what rounding the exact value gives.
// (NaN in `rest`, behind an infinity, leaves the value.)
__device__ __forceinline__ float to_odd(float value, float rest) {
  return rest < 0.f || rest > 0.f ? __int_as_float(__float_as_int(value) | 1) : value;
}

// x / s for s in [2^-100, 2^100] that is no power of two, rounded to odd.  A small s
// and its x are first brought 2^64 up, so that the remainder cannot underflow where
// the quotient is not far below every code.
__device__ __forceinline__ float div_odd(float x, float s) {
  const float up = s < 1.f ? 18446744073709551616.f : 1.f;
  x *= up;
  s *= up;
  const float q = __fdiv_rz(x, s);
  return to_odd(q, fmaf(-q, s, x));
}

// a * b rounded to odd.
__device__ __forceinline__ float mul_odd(float a, float b) {
  const float p = __fmul_rz(a, b);
  return to_odd(p, fmaf(a, b, -p));
}

// |x| for the maximum of a block: elements that are not finite do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // false for NaN and infinity
}

// Two values already divided by their scale -> two codes, lo in the low byte.
template <int DT>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if constexpr (DT == PKV_KV8_E4M3) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
  } else {
    const int a = lo == lo ? __float2int_rn(fminf(fmaxf(lo, -127.f), 127.f)) : 0;
    const int b = hi == hi ? __float2int_rn(fminf(fmaxf(hi, -127.f), 127.f)) : 0;
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
  }
}

template <int DT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return encode2<DT>(a, b) | (encode2<DT>(c, d) << 16);
}

// Four codes -> the values they stand for at scale 1.
template <int DT>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
  if constexpr (DT == PKV_KV8_E4M3) {
    uint32_t h0, h1;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f[0]), "=f"(f[1])
        : "r"(h0));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f[2]), "=f"(f[3])
        : "r"(h1));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// Index of the scale of (layer, slot, head g), slot = page * P + inside.
__device__ __forceinline__ long long scale_index(const pkv_workspace &ws, int scale_block,
                                                 int layer, int slot, int g) {
  const int P = ws.page_size, page = slot / P;
  const long long row = ((long long)layer * (ws.pool_slots / P) + page) * ws.n_kv_heads + g;
  return row * (P / scale_block) + (slot - page * P) / scale_block;
}

// Slot of token t of the request whose index entries start at `base` (the
// table row in page mode, the kv_indptr offset in flat mode), or -1 with the
// error bit in *kind.
__device__ __forceinline__ int token_slot(const pkv_workspace &ws, long long base, int t,
                                          int *kind) {
  if (ws.index_mode == PKV_IDX_FLAT) {
    const int s = ws.kv_indices[base + t];
    if (s >= 0 && s < ws.pool_slots) return s;
    *kind |= PKV_DEVERR_SLOT;
    return -1;
  }
  const int P = ws.page_size, p = t / P;
  const int page = ws.page_table[base + p];
  if (page >= 0 && page < ws.pool_slots / P) return page * P + (t - p * P);
  *kind |= PKV_DEVERR_PAGE;
  return -1;
}

}  // namespace pkv
