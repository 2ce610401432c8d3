// fp8_common.h -- e4m3 codes with a power-of-two scale for each block of 128 (internal).
//
// A block holds 128 consecutive elements of a row (128 x 128 of a weight matrix) as e4m3
// codes q and one exponent byte b, the power of two 2^(b-127): the values are q * 2^(b-127).
// The scale is the least power of two with max |x| <= 448 * 2^e, at least 2^-117, so that
// codes never saturate and every value they stand for (down to 2^-9 * 2^-117) is a normal
// fp32. Powers of two cost no precision here (e4m3 is itself a floating type: the values'
// relative step is the same) and are what the matrix instructions apply for free.
#pragma once

#include "device_common.h"

namespace bgt {

constexpr uint32_t kF8MinByte = 10;                  // 2^-117
constexpr uint32_t kF8NanByte = 255;
constexpr float kF8Nan = __builtin_nanf("");

// exponent byte of a block from the largest |x| as float bits (integer order: an infinity
// or a NaN in the block wins, and gives the NaN byte). 448 = 1.75 * 2^8: a mantissa above
// 1.75 takes the next power.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return kF8NanByte;
  const int b = (int)((top + 0x1FFFFFu) >> 23) - 8;
  return b < (int)kF8MinByte ? kF8MinByte : (uint32_t)b;
}
// 2^(byte - 127) (byte 0 is a subnormal); NaN for the NaN byte
__device__ __forceinline__ float f8_scale(uint32_t byte) {
  return __uint_as_float(byte == kF8NanByte ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// the largest over a row of 16 lanes, in all of them: lane exchanges of the vector unit (pairs,
// quads, then the row's halves mirrored)
__device__ __forceinline__ uint32_t max16(uint32_t t) {
  t = umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0xB1, 0xF, 0xF, true));
  t = umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x4E, 0xF, 0xF, true));
  t = umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x141, 0xF, 0xF, true));
  return umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x140, 0xF, 0xF, true));
}

// four values over scale (a power of two) to four codes, rounded once to nearest even, first
// value in the low byte; whatever of a block whose scale is NaN
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float scale) {
  typedef short v2s __attribute__((ext_vector_type(2)));
  v2s w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2s{0, 0}, a, b, scale, false);
  return __builtin_bit_cast(uint32_t, (v2s)__builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true));
}
// the four codes of a word as values
__device__ __forceinline__ void f8_unpack4(uint32_t w, float* v) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// lanes of a wave exchange through LDS: what one wrote before this the others read after it. A
// wave's LDS accesses run in order, so this is for the compiler only.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// stores past the L2, of outputs that nobody reads soon or that would push out what is shared
__device__ __forceinline__ void store_once(void* p, uint4 v) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(__builtin_bit_cast(v4u, v), static_cast<v4u*>(p));
}
__device__ __forceinline__ void store_once(void* p, uint2 v) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(__builtin_bit_cast(v2u, v), static_cast<v2u*>(p));
}

// eight consecutive elements of type IT at element i, widened: one or two 16-byte loads
template <int IT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float* v) {
  if constexpr (IT == kF32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const float4 a = widen_x4<IT>(make_uint2(u.x, u.y)), b = widen_x4<IT>(make_uint2(u.z, u.w));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
// the same of a row of n elements from its element c on, element by element, zeros behind it
template <int IT>
__device__ __forceinline__ void load8_tail(const void* x, int64_t row, int c, int n, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = c + j < n ? load_x1<IT>(x, row + c + j) : 0.0f;
}
// eight values stored as type OT at element i: 16-byte stores, or one by one below n
template <int OT>
__device__ __forceinline__ void store8(void* y, int64_t i, const float* v) {
  if constexpr (OT == kF32) {
    float* p = static_cast<float*>(y) + i;
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + i) =
        make_uint4(narrow2<OT>(v[0], v[1]), narrow2<OT>(v[2], v[3]), narrow2<OT>(v[4], v[5]),
                   narrow2<OT>(v[6], v[7]));
  }
}
template <int OT>
__device__ __forceinline__ void store8_tail(void* y, int64_t row, int c, int n, const float* v) {
  const OutY o{y, OT};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < n) o.put(row + c + j, v[j]);
}

}  // namespace bgt
