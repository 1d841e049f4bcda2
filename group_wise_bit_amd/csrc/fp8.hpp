// Device helpers of the block-scaled FP8 operators: typed 8-element loads and stores,
// the block scale and the e4m3 conversion.
//
// One block is 128 columns of one row (activations) or of 128 rows (weights); the last
// block of a row or column may be shorter. Its scale from a = min(max |v|, FLT_MAX), NaN
// ignored:
//   float32  s = max(fl32(a / 448), 2^-126)
//   E8M0     s = 2^e, e = max(ceil(log2(a / 448)), -126), stored as the byte e + 127
// and a code is the e4m3 value nearest fl32(v * r), ties to even, r = fl32(1 / s). The
// bound 2^-126 keeps r finite; |v r| is at most 448 (1 + 2^-22), well below 464 where
// e4m3 would stop rounding to 448; a NaN or infinite v gives a NaN code.
#pragma once

#include <float.h>

#include "device_common.hpp"
#include "kernels.hpp"

namespace gwb {

struct BlockScale {
  float s, r;
};
__device__ __forceinline__ BlockScale block_scale(float amax, bool e8m0) {
  const float a = fminf(amax, FLT_MAX);
  if (e8m0) {
    // 448 = 1.75 * 2^8: with a = m * 2^E the exponent is E - 8 up to m = 1.75, E - 7 beyond
    // (a subnormal a has the exponent field 0 and falls to the bound)
    const uint32_t b = __float_as_uint(a);
    const int e = max((int)(b >> 23) - 135 + (int)((b & 0x7FFFFFu) > 0x600000u), -126);
    return BlockScale{__uint_as_float((uint32_t)(e + 127) << 23), __uint_as_float((uint32_t)(127 - e) << 23)};
  }
  const float s = fmaxf(a / 448.0f, 0x1p-126f);
  return BlockScale{s, 1.0f / s};
}
__device__ __forceinline__ void store_scale(void* scales, int64_t i, float s, bool e8m0) {
  if (e8m0) static_cast<uint8_t*>(scales)[i] = (uint8_t)(__float_as_uint(s) >> 23);
  else static_cast<float*>(scales)[i] = s;
}

// Four values -> four e4m3 codes (round to nearest even), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// ---- typed elements: float, uint16_t (bf16 bits), _Float16
__device__ __forceinline__ float fp8_widen(float v) { return v; }
__device__ __forceinline__ float fp8_widen(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float fp8_widen(_Float16 v) { return (float)v; }
template <typename T> __device__ __forceinline__ T fp8_narrow(float v);
template <> __device__ __forceinline__ float fp8_narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ uint16_t fp8_narrow<uint16_t>(float v) { return (uint16_t)f32_to_bf16_rne(v); }
template <> __device__ __forceinline__ _Float16 fp8_narrow<_Float16>(float v) { return (_Float16)v; }

// 16 and 8 bytes at any address of an element (the target takes unaligned accesses whole).
// ONCE / once: not used again soon, non-temporal (aligned only).
template <bool ALIGNED, bool ONCE>
__device__ __forceinline__ U4 fp8_ld16(const void* p) {
  if constexpr (ALIGNED) {
    if constexpr (ONCE) return ld16_nt(p);
    else return ld16(p);
  } else {
    U4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
  }
}
template <bool ALIGNED>
__device__ __forceinline__ void fp8_st16(void* p, U4 v, bool once) {
  if constexpr (ALIGNED) {
    if (once) st16_nt(p, v);
    else st16(p, v);
  } else {
    __builtin_memcpy(p, &v, 16);
  }
}

// The 8 elements from p, n of them valid (the rest 0). ALIGNED: n is 0 or 8 and p is
// 16-byte aligned; otherwise n from 1 to 7 gives zeros (see fp8_load_rest).
typedef _Float16 fp8_f16x8_t __attribute__((ext_vector_type(8)));
template <bool ALIGNED, bool ONCE = true, typename T>
__device__ __forceinline__ void fp8_load8(const T* p, int n, float* v) {
  const bool whole = ALIGNED ? n > 0 : n == 8;
  const U4 zero{0, 0, 0, 0};
  if constexpr (sizeof(T) == 4) {
    U4 a = zero, b = zero;
    if (whole) {
      a = fp8_ld16<ALIGNED, ONCE>(p);
      b = fp8_ld16<ALIGNED, ONCE>(p + 4);
    }
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    const U4 w = whole ? fp8_ld16<ALIGNED, ONCE>(p) : zero;
    if constexpr (__is_same(T, uint16_t)) {
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    } else {
      const fp8_f16x8_t h = __builtin_bit_cast(fp8_f16x8_t, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    }
  }
}
// The row's last n < 8 elements, which fp8_load8 left at 0. Apart from it, so that no
// branch stands between the loads of a lane's units.
template <bool ALIGNED, typename T>
__device__ __forceinline__ void fp8_load_rest(const T* p, int n, float* v) {
  if (!ALIGNED && n > 0 && n < 8) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) v[i] = fp8_widen(p[i]);
  }
}

// 8 values to p in its type, n of them (ALIGNED: all 8, p 16-byte aligned).
template <bool ALIGNED, typename T>
__device__ __forceinline__ void fp8_store8(T* p, int n, const float* v, bool once = false) {
  if (ALIGNED ? n > 0 : n == 8) {
    if constexpr (sizeof(T) == 4) {
      fp8_st16<ALIGNED>(p, U4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, once);
      fp8_st16<ALIGNED>(p + 4, U4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])}, once);
    } else if constexpr (__is_same(T, uint16_t)) {
      fp8_st16<ALIGNED>(p, U4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])}, once);
    } else {
      fp8_f16x8_t h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
      fp8_st16<ALIGNED>(p, __builtin_bit_cast(U4, h), once);
    }
  } else if constexpr (!ALIGNED) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = fp8_narrow<T>(v[i]);
  }
}

// Codes of 8 values, n of them stored (ALIGNED: all 8, p 8-byte aligned).
template <bool ALIGNED>
__device__ __forceinline__ void fp8_store_codes8(uint8_t* p, int n, const float* v, float r) {
  const uint2 c{e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r)};
  if constexpr (ALIGNED) {
    if (n > 0) *reinterpret_cast<uint2*>(p) = c;
  } else if (n == 8) {
    __builtin_memcpy(p, &c, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// The largest magnitude, at least 0 (8 NaN must not leave a NaN).
__device__ __forceinline__ float absmax8(const float* v) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}

// g / (1 + exp(-g)) without expf and a division (which bound the gated activation by
// arithmetic: 42 us at 2048 x 17408 against 33). exp(-g) = 2^t * 2^lo with t = fl(-g log2 e)
// and lo its rounding error, log2 e in two parts; 2^lo = 1 + lo ln 2 to far below an ulp; one
// Newton step on the hardware reciprocal. Within 7 u, u = 2^-24: 2^t to 1 ulp (2 u), its
// correction, the product and the sum with 1 (u each), the reciprocal and the product with
// g (u each); measured over the gates from -87 to 88: 4.1 u with the quotient by 448 that
// makes it visible. Below g = -87 the result is taken as g * 0 (it is less than 2e-36
// there): NaN for -inf, as the formula gives.
__device__ __forceinline__ float silu(float g) {
  const float x = __builtin_amdgcn_fmed3f(-g, -104.0f, 87.0f);
  const float t = x * 0x1.715476p+0f;
  const float lo = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));
  const float d = 1.0f + __builtin_amdgcn_exp2f(t) * __builtin_fmaf(lo, 0x1.62e43p-1f, 1.0f);
  const float r = __builtin_amdgcn_rcpf(d);
  return g * (g < -87.0f ? 0.0f : __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r));
}

// Maximum and sum of a float over the wavefront, the same value in every lane; fixed
// order. (Call them where every lane is active: the lane reads see what each lane computed.)
__device__ __forceinline__ float wave_max_f32(float v) {
  v = lanes_max<16>(v);
  const auto at = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
  return fmaxf(fmaxf(at(0), at(16)), fmaxf(at(32), at(48)));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_read<kDppXor1>(v);
  v += dpp_read<kDppXor2>(v);
  v += dpp_read<kDppHalfMirror>(v);
  v += dpp_read<kDppMirror>(v);
  const auto at = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
  return ((at(0) + at(16)) + at(32)) + at(48);
}

}  // namespace gwb
