// Device-side helpers of the 8-bit linear layer and layer norm: the block
// scale of e4m3 values, conversions, unaligned 8-element accesses and
// reductions over lanes.  Internal; not part of the C ABI.
#pragma once

#include "muon_device.h"

namespace muon {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Magnitude bits of x, or 0 where x is an infinity or NaN: those have no
// part in a block's scale.  As unsigned numbers they order like |x|.
__device__ __forceinline__ unsigned finite_bits(float x) {
  const unsigned u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// The byte e + 127 of a block whose largest finite magnitude has the bits u:
// e is the smallest integer >= -117 with |x| <= 448 * 2^e = 1.75 * 2^(e + 8).
// With |x| = 1.f * 2^(E - 127) that is e = E - 135, one more where the
// fraction is above .75.  The lower limit keeps every value q * 2^e (q a
// multiple of 2^-9) a normal bf16 and fp32 number.
__device__ __forceinline__ int scale_byte(unsigned u) {
  const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (e < -117 ? -117 : e) + 127;
}
// The byte of a block with a value above 1.75 * 2^127, the largest there is.
constexpr int kTopScale = 247;
// 2^e and 2^-e of a scale byte 10 .. 247: both normal fp32 numbers.
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float((unsigned)byte << 23); }
__device__ __forceinline__ float inv_scale_of(int byte) {
  return __uint_as_float((unsigned)(254 - byte) << 23);
}

// An infinity divided by a scale stays one: it is replaced by NaN before the
// conversion, whose own result for it depends on the wave's overflow mode.
__device__ __forceinline__ float inf_to_nan(float x) {
  return (__float_as_uint(x) & 0x7fffffffu) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : x;
}
// Eight values divided by their block's scale.  In a block of the largest scale,
// 2^120, e4m3's 256 would stand for 2^128, which neither fp32 nor bf16 has: what
// would round to it (248 * 2^120 and above, both types' largest among them) takes
// 240, at most 2^-4 off, which is e4m3's half step too.
__device__ __forceinline__ void to_units(const float (&v)[8], int byte, float (&w)[8]) {
  const float inv = inv_scale_of(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = inf_to_nan(v[i]) * inv;
  if (byte == kTopScale) {
#pragma unroll
    for (int i = 0; i < 8; ++i)  // (a NaN stays)
      w[i] = w[i] > 240.f ? 240.f : w[i] < -240.f ? -240.f : w[i];
  }
}

// Eight values, already divided by their scale, as e4m3 bytes (rounded to
// nearest even).  The scaled magnitudes are at most 448, so nothing
// overflows; a NaN becomes e4m3's NaN.
__device__ __forceinline__ u32x2_t to_e4m3(const float (&v)[8]) {
  u32x2_t o;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    int p = 0;
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w], v[4 * w + 1], p, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w + 2], v[4 * w + 3], p, true);
    o[w] = (unsigned)p;
  }
  return o;
}

__device__ __forceinline__ void from_e4m3(u32x2_t q, float scale, float (&v)[8]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[w], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[w], true);
    v[4 * w] = lo[0] * scale;
    v[4 * w + 1] = lo[1] * scale;
    v[4 * w + 2] = hi[0] * scale;
    v[4 * w + 3] = hi[1] * scale;
  }
}

// Eight e4m3 values times their scale as bf16, exact.
__device__ __forceinline__ u32x4_t bf16_of_e4m3(unsigned lo, unsigned hi, float scale) {
  u32x4_t o = {0u, 0u, 0u, 0u};
#if defined(__HIP_DEVICE_COMPILE__)
  o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
#endif
  return o;
}

// Eight consecutive elements in one access (bf16: 16 bytes, fp32: 32) at an
// address aligned to one element only: rows of any stride go the same way
// (global memory takes unaligned vector accesses).
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  u32x4_t w;
  __builtin_memcpy(&w, p, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  f32x4_t a, b;
  __builtin_memcpy(&a, p, 16);
  __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const bf16x2_t p = {static_cast<bf16_t>(lo), static_cast<bf16_t>(hi)};
  return __builtin_bit_cast(unsigned, p);
}
template <bool STRM>
__device__ __forceinline__ void store16(void* p, u32x4_t v) {
  typedef u32x4_t __attribute__((aligned(2))) any_t;
  if constexpr (STRM)
    __builtin_nontemporal_store(v, static_cast<any_t*>(p));
  else
    *static_cast<any_t*>(p) = v;
}
template <bool STRM = false>
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  store16<STRM>(p, w);
}
template <bool STRM = false>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  store16<STRM>(p, __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}));
  store16<STRM>(p + 4, __builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}));
}
// The first `n` of eight elements (n <= 0: none); the others read as zero.
template <typename T>
__device__ __forceinline__ void load8_edge(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
// STRM: streamed past the caches.
template <bool STRM = false, typename T>
__device__ __forceinline__ void store8_edge(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    store8<STRM>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// 4 bytes per lane from global memory straight into LDS (see buffer_load_lds16).
__device__ __forceinline__ void buffer_load_lds4(__amdgpu_buffer_rsrc_t rsrc, unsigned voffset,
                                                 void* lds_wave_base) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (__attribute__((address_space(3))) void*)lds_wave_base, 4, (int)voffset, 0, 0, 0);
#endif
}

// Maximum over each row of 16 lanes, in all of them (DPP rotations).
__device__ __forceinline__ unsigned max16(unsigned u) {
  auto step = [&](auto ctrl) {
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(
        0, (int)u, decltype(ctrl)::value, 0xf, 0xf, false);
    u = u > o ? u : o;
  };
  step(std::integral_constant<int, 0x128>{});  // row_ror:8
  step(std::integral_constant<int, 0x124>{});
  step(std::integral_constant<int, 0x122>{});
  step(std::integral_constant<int, 0x121>{});
  return u;
}

// Sum over the wave, the same in all lanes and from run to run: DPP adds inside
// rows of 16 lanes, then across the rows; lane 63 ends up with the total.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
    v += __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(v), decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
  };
  using All = std::integral_constant<int, 0xf>;
  add(std::integral_constant<int, 0x111>{}, All{});  // row_shr:1
  add(std::integral_constant<int, 0x112>{}, All{});
  add(std::integral_constant<int, 0x114>{}, All{});
  add(std::integral_constant<int, 0x118>{}, All{});
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast:15
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast:31
  return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Eight consecutive elements as they lie in memory, so that a row can be on
// its way while another one is worked on.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const bf16_t* p, int n) {
    if (n >= 8) {
      __builtin_memcpy(&w, p, 16);
    } else {
      float v[8];
      load8_edge(p, n, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p, int n) { load8_edge(p, n, w); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i];
  }
};

// The four scale bytes of a wave whose rows of 16 lanes each hold one, as a
// word (the same in all lanes).
__device__ __forceinline__ unsigned pack_scales(int byte) {
  return (unsigned)__builtin_amdgcn_readlane(byte, 0) |
         (unsigned)__builtin_amdgcn_readlane(byte, 16) << 8 |
         (unsigned)__builtin_amdgcn_readlane(byte, 32) << 16 |
         (unsigned)__builtin_amdgcn_readlane(byte, 48) << 24;
}

}  // namespace muon
