// moe_rows.hip -- token rows to expert order and back (gfx950).
//
// pos[t][i] is the sorted slot of token t's i-th expert, or -1 (dropped).
//   gather            xs[pos[t][i]] = x[t];  slots past the last expert's are zero
//   combine           y[t] = sum_i w[t][i] ys[pos[t][i]]   (w = 1 without weights:
//                     the gradient of gather)
//   combine backward  dys[pos[t][i]] = w[t][i] dy[t],  dw[t][i] = <dy[t], ys[pos[t][i]]>
//
// All are bound by memory traffic. Each works by token: the token's row is read
// (or written) once, whatever k is, and no two tokens share a slot, so nothing
// is added across workgroups. Sums are in fp32, i ascending, rounded once.
#include "device_common.h"
#include "launch.h"

namespace bgt {

constexpr int kRowThreads = 256;
constexpr int kTailBlocks = 64;       // workgroups that zero the slots past the last one

// VEC consecutive elements of type IT as fp32, and back (rounded to nearest even)
template <int IT, int VEC> struct Chunk { using T = uint4; };
template <> struct Chunk<kF32, 1> { using T = float; };
template <> struct Chunk<kF16, 1> { using T = uint16_t; };
template <> struct Chunk<kBF16, 1> { using T = uint16_t; };

template <int IT> constexpr int kVec = IT == kF32 ? 4 : 8;      // elements of 16 bytes

template <int IT, int VEC>
__device__ __forceinline__ void widen(const typename Chunk<IT, VEC>::T& u, float* v) {
  if constexpr (VEC == 1) {
    v[0] = load_x1<IT>(&u, 0);
  } else if constexpr (IT == kF32) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  } else {
    const float4 a = widen_x4<IT>(make_uint2(u.x, u.y)), b = widen_x4<IT>(make_uint2(u.z, u.w));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <int IT, int VEC>
__device__ __forceinline__ typename Chunk<IT, VEC>::T narrow(const float* v) {
  if constexpr (VEC == 1) {
    if constexpr (IT == kF32) return v[0];
    else return (uint16_t)narrow2<IT>(v[0], 0.0f);
  } else if constexpr (IT == kF32) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  } else {
    return make_uint4(narrow2<IT>(v[0], v[1]), narrow2<IT>(v[2], v[3]), narrow2<IT>(v[4], v[5]),
                      narrow2<IT>(v[6], v[7]));
  }
}

// chunk h of row r of a matrix of `ld` chunks a row
template <typename C>
__device__ __forceinline__ const C& at(const void* p, int64_t r, int64_t ld, int h) {
  return static_cast<const C*>(p)[r * ld + h];
}
template <typename C>
__device__ __forceinline__ C& at(void* p, int64_t r, int64_t ld, int h) {
  return static_cast<C*>(p)[r * ld + h];
}

// zero the slots from the last expert's end to R (workgroup b of nb)
template <typename C>
__device__ __forceinline__ void zero_tail(const int32_t* offs, int E, int64_t R, int hc, void* out,
                                          int b, int nb) {
  for (int64_t r = clamp_route(offs[E], 0, (int)R) + b; r < R; r += nb)
    for (int h = threadIdx.x; h < hc; h += kRowThreads) at<C>(out, r, hc, h) = C{};
}

template <typename C>
__global__ __launch_bounds__(kRowThreads) void k_moe_gather(const void* __restrict__ x, int64_t ld,
                                                            const int32_t* __restrict__ offs,
                                                            const int32_t* __restrict__ pos,
                                                            int64_t T, int E, int k, int hc,
                                                            void* __restrict__ xs) {
  const int64_t R = T * k, t = blockIdx.x;
  if (t >= T) return zero_tail<C>(offs, E, R, hc, xs, (int)(t - T), kTailBlocks);
  for (int h = threadIdx.x; h < hc; h += kRowThreads) {
    const C v = at<C>(x, t, ld, h);
    for (int i = 0; i < k; ++i) {
      const int p = pos[t * k + i];
      if (p >= 0 && p < R) at<C>(xs, p, hc, h) = v;
    }
  }
}

template <int IT, int VEC>
__global__ __launch_bounds__(kRowThreads) void k_moe_combine(const void* __restrict__ ys,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w, int64_t T,
                                                             int k, int hc, void* __restrict__ y) {
  using C = typename Chunk<IT, VEC>::T;
  const int64_t R = T * k, t = blockIdx.x;
  for (int h = threadIdx.x; h < hc; h += kRowThreads) {
    float acc[VEC] = {};
    for (int i = 0; i < k; ++i) {
      const int p = pos[t * k + i];
      if (p < 0 || p >= R) continue;
      const float wi = w ? w[t * k + i] : 1.0f;
      float v[VEC];
      widen<IT, VEC>(at<C>(ys, p, hc, h), v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = __builtin_fmaf(wi, v[j], acc[j]);
    }
    at<C>(y, t, hc, h) = narrow<IT, VEC>(acc);
  }
}

template <int IT, int VEC>
__global__ __launch_bounds__(kRowThreads) void k_moe_combine_grad(
    const void* __restrict__ dy, int64_t ld, const void* __restrict__ ys,
    const int32_t* __restrict__ offs, const int32_t* __restrict__ pos, const float* __restrict__ w,
    int64_t T, int E, int k, int hc, void* __restrict__ dys, float* __restrict__ dw) {
  using C = typename Chunk<IT, VEC>::T;
  __shared__ float sums[kRowThreads / kWave];
  const int64_t R = T * k, t = blockIdx.x;
  if (t >= T) return zero_tail<C>(offs, E, R, hc, dys, (int)(t - T), kTailBlocks);
  for (int i = 0; i < k; ++i) {
    const int p = pos[t * k + i];
    const bool ok = p >= 0 && p < R;
    const float wi = w[t * k + i];
    float dot = 0.0f;
    if (ok)
      for (int h = threadIdx.x; h < hc; h += kRowThreads) {
        float g[VEC], v[VEC];
        widen<IT, VEC>(at<C>(dy, t, ld, h), g);
        widen<IT, VEC>(at<C>(ys, p, hc, h), v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          dot = __builtin_fmaf(g[j], v[j], dot);
          g[j] *= wi;
        }
        at<C>(dys, p, hc, h) = narrow<IT, VEC>(g);
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
    if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) dw[t * k + i] = ((sums[0] + sums[1]) + sums[2]) + sums[3];
    __syncthreads();
  }
}

// ----------------------------------------------------------------- launchers
namespace {

// rows of H elements of `size` bytes, `ld` apart, can be taken 16 bytes at a time
bool wide_rows(const void* p, int64_t ld, int64_t H, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * size % 16 == 0 && H * size % 16 == 0;
}
int size_of(int type) { return type == kF32 ? 4 : 2; }

template <typename F>
void with_type(int type, bool wide, F f) {
  if (type == kF32) wide ? f(IC<kF32>{}, IC<4>{}) : f(IC<kF32>{}, IC<1>{});
  else if (type == kF16) wide ? f(IC<kF16>{}, IC<8>{}) : f(IC<kF16>{}, IC<1>{});
  else wide ? f(IC<kBF16>{}, IC<8>{}) : f(IC<kBF16>{}, IC<1>{});
}

}  // namespace

hipError_t launch_moe_gather(const void* x, int type, int64_t ld, const int32_t* offs,
                             const int32_t* pos, int64_t T, int64_t E, int64_t k, int64_t H,
                             void* xs, hipStream_t stream) {
  const int size = size_of(type);
  const dim3 grid((unsigned)(T + kTailBlocks));
  if (wide_rows(x, ld, H, size) && wide_rows(xs, H, H, size))
    hipLaunchKernelGGL((k_moe_gather<uint4>), grid, dim3(kRowThreads), 0, stream, x,
                       ld * size / 16, offs, pos, T, (int)E, (int)k, (int)(H * size / 16), xs);
  else if (size == 4)
    hipLaunchKernelGGL((k_moe_gather<uint32_t>), grid, dim3(kRowThreads), 0, stream, x, ld, offs,
                       pos, T, (int)E, (int)k, (int)H, xs);
  else
    hipLaunchKernelGGL((k_moe_gather<uint16_t>), grid, dim3(kRowThreads), 0, stream, x, ld, offs,
                       pos, T, (int)E, (int)k, (int)H, xs);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* ys, int type, const int32_t* pos, const float* weights,
                              int64_t T, int64_t k, int64_t H, void* y, hipStream_t stream) {
  const int size = size_of(type);
  const bool wide = wide_rows(ys, H, H, size) && wide_rows(y, H, H, size);
  with_type(type, wide, [&](auto it, auto vec) {
    constexpr int IT = decltype(it)::value, VEC = decltype(vec)::value;
    hipLaunchKernelGGL((k_moe_combine<IT, VEC>), dim3((unsigned)T), dim3(kRowThreads), 0, stream,
                       ys, pos, weights, T, (int)k, (int)(H / VEC), y);
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* dy, int64_t ld, const void* ys, int type,
                                       const int32_t* offs, const int32_t* pos,
                                       const float* weights, int64_t T, int64_t E, int64_t k,
                                       int64_t H, void* dys, float* dweights, hipStream_t stream) {
  const int size = size_of(type);
  const bool wide =
      wide_rows(dy, ld, H, size) && wide_rows(ys, H, H, size) && wide_rows(dys, H, H, size);
  with_type(type, wide, [&](auto it, auto vec) {
    constexpr int IT = decltype(it)::value, VEC = decltype(vec)::value;
    hipLaunchKernelGGL((k_moe_combine_grad<IT, VEC>), dim3((unsigned)(T + kTailBlocks)),
                       dim3(kRowThreads), 0, stream, dy, ld / VEC, ys, offs, pos, weights, T,
                       (int)E, (int)k, (int)(H / VEC), dys, dweights);
  });
  return hipGetLastError();
}

}  // namespace bgt
