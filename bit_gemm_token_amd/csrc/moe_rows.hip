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
//
// A power of two of lanes shares a token, 16 bytes of a row each at a time, so
// short rows leave no lanes idle and a workgroup takes several tokens. Rows are
// read and written 16 bytes at a time at the alignment of their elements (odd
// lengths put rows at any of them).
#include "device_common.h"
#include "launch.h"

namespace bgt {

constexpr int kRowThreads = 256;
constexpr int kTailBlocks = 64;       // workgroups that zero the slots past the last one
constexpr int64_t kMostBlocks = 1 << 20;

typedef uint32_t u4e __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes, element-aligned

template <int IT> struct Elem { using T = uint16_t; static constexpr int VEC = 8; };
template <> struct Elem<kF32> { using T = uint32_t; static constexpr int VEC = 4; };

// elements [h, h + VEC) of a row of H as fp32 (past its end 0, where the piece
// is not WHOLE), and back (rounded to nearest even)
template <int IT, bool WHOLE>
__device__ __forceinline__ void load_piece(const void* m, int64_t row, int64_t ld, int h, int H,
                                           float (&v)[Elem<IT>::VEC]) {
  constexpr int VEC = Elem<IT>::VEC;
  const typename Elem<IT>::T* p = static_cast<const typename Elem<IT>::T*>(m) + row * ld + h;
  if constexpr (WHOLE) {
    const u4e u = *reinterpret_cast<const u4e*>(p);
    if constexpr (IT == kF32) {
      v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
      v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    } else {
      const float4 a = widen_x4<IT>(make_uint2(u.x, u.y)), b = widen_x4<IT>(make_uint2(u.z, u.w));
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = h + j < H ? load_x1<IT>(p, j) : 0.0f;
  }
}
template <int IT, bool WHOLE>
__device__ __forceinline__ void store_piece(void* m, int64_t row, int64_t ld, int h, int H,
                                            const float (&v)[Elem<IT>::VEC]) {
  constexpr int VEC = Elem<IT>::VEC;
  typename Elem<IT>::T* p = static_cast<typename Elem<IT>::T*>(m) + row * ld + h;
  if constexpr (WHOLE) {
    u4e u;
    if constexpr (IT == kF32)
      u = u4e{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
              __float_as_uint(v[3])};
    else
      u = u4e{narrow2<IT>(v[0], v[1]), narrow2<IT>(v[2], v[3]), narrow2<IT>(v[4], v[5]),
              narrow2<IT>(v[6], v[7])};
    *reinterpret_cast<u4e*>(p) = u;
  } else {
    const OutY out{p, IT};
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (h + j < H) out.put(j, v[j]);
  }
}

// f(whole, h, skip) for the pieces of a row of H that lane l of `lanes` takes. A
// last, partial piece is a whole one moved back to end with the row, whose first
// `skip` elements are the piece's before it: written twice with the same values,
// and not to be summed twice. Rows shorter than a piece go by element.
template <int VEC, typename F>
__device__ __forceinline__ void for_pieces(int l, int lanes, int H, F f) {
  if (H >= VEC) {
    for (int h = l * VEC; h < H; h += lanes * VEC) {
      const int at = min(h, H - VEC);
      f(IC<1>{}, at, h - at);
    }
  } else if (l == 0) {
    f(IC<0>{}, 0, 0);
  }
}

// f(whole, t, h) for all pieces that this thread takes: `blocks` workgroups of
// 256 >> sh tokens, 1 << sh lanes each, grid y splitting a token's row further.
// A launch has at most kMostBlocks of them (a grid's threads are counted in 32
// bits), hence the loop over tokens.
template <int VEC, typename F>
__device__ __forceinline__ void for_tokens(int blocks, int64_t tokens, int sh, int H, F f) {
  const int lanes = 1 << sh, l = threadIdx.x & (lanes - 1);
  const int64_t each = 256 >> sh;
  for (int64_t t = blockIdx.x * each + (threadIdx.x >> sh); t < tokens; t += blocks * each)
    for_pieces<VEC>(blockIdx.y * lanes + l, gridDim.y * lanes, H,
                    [&](auto whole, int h, int) { f(whole, t, h); });
}

// zero the slots from the last expert's end to R (workgroup b of kTailBlocks), which
// are contiguous, 16 bytes at a time; a last, partial piece is a whole one moved back
// to end with them. T is the element's type. (4096 x 4096 bf16, k = 2, seven eighths of
// the slots dropped: gather 21.0 us, with an element a lane 55.8; combine's gradient
// 24.1 and 69.9.)
template <typename T>
__device__ __forceinline__ void zero_tail(const int32_t* offs, int E, int64_t R, int H, T* out,
                                          int b) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t first = clamp_route(offs[E], 0, (int)R) * (int64_t)H, n = R * H - first;
  T* tail = out + first;
  const int64_t at = (int64_t)b * kRowThreads + threadIdx.x;
  if (n >= VEC) {
    for (int64_t o = at * VEC; o < n; o += (int64_t)kTailBlocks * kRowThreads * VEC)
      *reinterpret_cast<u4e*>(tail + min(o, n - VEC)) = u4e{};
  } else if (at < n) {
    tail[at] = 0;
  }
}

// The last kTailBlocks workgroups zero the tail.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void k_moe_gather(const T* __restrict__ x, int64_t ld,
                                                            const int32_t* __restrict__ offs,
                                                            const int32_t* __restrict__ pos,
                                                            int64_t tokens, int E, int k, int H,
                                                            int sh, T* __restrict__ xs) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t R = tokens * k;
  const int tail = (int)(blockIdx.x + kTailBlocks) - (int)gridDim.x;
  if (tail >= 0) {
    if (blockIdx.y == 0) zero_tail<T>(offs, E, R, H, xs, tail);
    return;
  }
  for_tokens<VEC>(gridDim.x - kTailBlocks, tokens, sh, H, [&](auto whole, int64_t t, int h) {
    const T* src = x + t * ld + h;
    u4e v{};
    if constexpr (decltype(whole)::value) v = *reinterpret_cast<const u4e*>(src);
    for (int i = 0; i < k; ++i) {
      const int p = pos[t * k + i];
      if (p < 0 || p >= R) continue;
      T* dst = xs + (int64_t)p * H + h;
      if constexpr (decltype(whole)::value) *reinterpret_cast<u4e*>(dst) = v;
      else
        for (int j = 0; j < H - h; ++j) dst[j] = src[j];
    }
  });
}

// AT: expert rows of a token in flight together. A dropped place reads row 0 and
// uses none of it, which costs less than a branch around the load. All three
// kernels run near the rate of a copy (5.2 TB/s) where the rows are many: 4096 x 4096
// bf16, k = 2, gather 16.1 us, combine 16.2 (100 MB each, partly from the Infinity
// Cache), combine's gradient 31.2 (168 MB). Smaller ones are bound by launch and
// ramp (8192 x 127 fp16, k = 4, 10 MB, combine 5.4 us).
template <int IT, int AT>
__global__ __launch_bounds__(kRowThreads) void k_moe_combine(const void* __restrict__ ys,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w,
                                                             int64_t tokens, int k, int H, int sh,
                                                             void* __restrict__ y) {
  constexpr int VEC = Elem<IT>::VEC;
  const int64_t R = tokens * k;
  for_tokens<VEC>(gridDim.x, tokens, sh, H, [&](auto whole, int64_t t, int h) {
    constexpr bool WHOLE = decltype(whole)::value;
    float acc[VEC] = {};
    for (int i0 = 0; i0 < k; i0 += AT) {
      float v[AT][VEC], wi[AT];
      bool ok[AT];
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        ok[j] = false;
        wi[j] = 1.0f;
        if (i0 + j < k) {                          // uniform
          const int64_t o = t * k + i0 + j;
          const int p = pos[o];
          ok[j] = p >= 0 && p < R;
          if (w) wi[j] = w[o];
          load_piece<IT, WHOLE>(ys, ok[j] ? p : 0, H, h, H, v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < AT; ++j)
        if (i0 + j < k)
#pragma unroll
          for (int c = 0; c < VEC; ++c)
            acc[c] = ok[j] ? __builtin_fmaf(wi[j], v[j][c], acc[c]) : acc[c];
    }
    store_piece<IT, WHOLE>(y, t, H, h, H, acc);
  });
}

// A token's lanes are part of one wave, or the whole workgroup (sh = 8), whose
// waves' sums then meet in LDS. Grid y deals a token's places out, AT at a time; a
// place's sum has the same order whichever workgroup takes it.
template <int IT, int AT>
__global__ __launch_bounds__(kRowThreads) void k_moe_combine_grad(
    const void* __restrict__ dy, int64_t ld, const void* __restrict__ ys,
    const int32_t* __restrict__ offs, const int32_t* __restrict__ pos, const float* __restrict__ w,
    int64_t tokens, int E, int k, int H, int sh, void* __restrict__ dys, float* __restrict__ dw) {
  constexpr int VEC = Elem<IT>::VEC, WAVES = kRowThreads / kWave;
  __shared__ float sums[WAVES][AT];
  const int64_t R = tokens * k;
  const int tail = (int)(blockIdx.x + kTailBlocks) - (int)gridDim.x;
  if (tail >= 0 && blockIdx.y > 0) return;
  if (tail >= 0)
    return zero_tail(offs, E, R, H, static_cast<typename Elem<IT>::T*>(dys), tail);
  const int lanes = 1 << sh, l = threadIdx.x & (lanes - 1);
  const int64_t each = 256 >> sh, stride = (gridDim.x - kTailBlocks) * each;
  // the same count of rounds for all threads (they meet at barriers)
  for (int64_t t0 = blockIdx.x * each; t0 < tokens; t0 += stride) {
    for (int i0 = AT * blockIdx.y; i0 < k; i0 += AT * gridDim.y) {
      const int64_t t = t0 + (threadIdx.x >> sh);
      const bool in = t < tokens;
      float wi[AT], dot[AT];
      int p[AT];
      bool ok[AT];
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        ok[j] = false;
        p[j] = 0;
        wi[j] = dot[j] = 0.0f;
        if (in && i0 + j < k) {
          p[j] = pos[t * k + i0 + j];
          ok[j] = p[j] >= 0 && p[j] < R;
          if (!ok[j]) p[j] = 0;
          wi[j] = w[t * k + i0 + j];
        }
      }
      if (in)
        for_pieces<VEC>(l, lanes, H, [&](auto whole, int h, int skip) {
          constexpr bool WHOLE = decltype(whole)::value;
          float g[VEC], v[AT][VEC];
          load_piece<IT, WHOLE>(dy, t, ld, h, H, g);
#pragma unroll
          for (int j = 0; j < AT; ++j)
            if (i0 + j < k) load_piece<IT, WHOLE>(ys, p[j], H, h, H, v[j]);       // uniform
#pragma unroll
          for (int j = 0; j < AT; ++j)
            if (i0 + j < k) {
#pragma unroll
              for (int c = 0; c < VEC; ++c) {
                if (ok[j] && c >= skip) dot[j] = __builtin_fmaf(g[c], v[j][c], dot[j]);
                v[j][c] = g[c] * wi[j];
              }
              if (ok[j]) store_piece<IT, WHOLE>(dys, p[j], H, h, H, v[j]);
            }
        });
      for (int o = 1; o < min(lanes, kWave); o <<= 1)
#pragma unroll
        for (int j = 0; j < AT; ++j) dot[j] += __shfl_xor(dot[j], o, kWave);
      if (sh == 8) {
        __syncthreads();                             // the last round's sums are read
#pragma unroll
        for (int j = 0; j < AT; ++j)
          if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave][j] = dot[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < AT; ++j)
          dot[j] = ((sums[0][j] + sums[1][j]) + sums[2][j]) + sums[3][j];
      }
      if (in && l == 0)
#pragma unroll
        for (int j = 0; j < AT; ++j)
          if (i0 + j < k) dw[t * k + i0 + j] = dot[j];
    }
  }
}

// ----------------------------------------------------------------- launchers
namespace {

// log2 of the lanes of a token: one piece of 16 bytes a lane, up to 2^most lanes
int lanes_log2(int64_t pieces, int most) {
  int sh = 0;
  while (sh < most && ((int64_t)1 << sh) < pieces) ++sh;
  return sh;
}
unsigned token_blocks(int64_t T, int sh) {
  const int64_t each = 256 >> sh;
  const int64_t blocks = (T + each - 1) / each;
  return (unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks);
}
// workgroups along a row: rows longer than one workgroup's pieces are split
// where there are fewer workgroups than CUs
unsigned row_blocks(int64_t pieces, unsigned blocks) {
  const int64_t parts = (pieces + kRowThreads - 1) / kRowThreads;
  const int64_t room = device_cus() / blocks;
  return (unsigned)(parts < room ? parts : room > 1 ? room : 1);
}

template <typename F>
void with_type(int type, bool two, F f) {          // f(type, rows in flight together)
  const auto of_type = [&](auto it) { two ? f(it, IC<2>{}) : f(it, IC<4>{}); };
  if (type == kF32) of_type(IC<kF32>{});
  else if (type == kF16) of_type(IC<kF16>{});
  else of_type(IC<kBF16>{});
}
int64_t pieces_of(int type, int64_t H) { return type == kF32 ? (H + 3) / 4 : (H + 7) / 8; }

}  // namespace

hipError_t launch_moe_gather(const void* x, int type, int64_t ld, const int32_t* offs,
                             const int32_t* pos, int64_t T, int64_t E, int64_t k, int64_t H,
                             void* xs, hipStream_t stream) {
  const int64_t pieces = pieces_of(type, H);
  const int sh = lanes_log2(pieces, 8);
  const unsigned blocks = token_blocks(T, sh);
  const dim3 grid(blocks + kTailBlocks, row_blocks(pieces, blocks));
  if (type == kF32)
    hipLaunchKernelGGL((k_moe_gather<uint32_t>), grid, dim3(kRowThreads), 0, stream,
                       static_cast<const uint32_t*>(x), ld, offs, pos, T, (int)E, (int)k, (int)H,
                       sh, static_cast<uint32_t*>(xs));
  else
    hipLaunchKernelGGL((k_moe_gather<uint16_t>), grid, dim3(kRowThreads), 0, stream,
                       static_cast<const uint16_t*>(x), ld, offs, pos, T, (int)E, (int)k, (int)H,
                       sh, static_cast<uint16_t*>(xs));
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* ys, int type, const int32_t* pos, const float* weights,
                              int64_t T, int64_t k, int64_t H, void* y, hipStream_t stream) {
  const int64_t pieces = pieces_of(type, H);
  const int sh = lanes_log2(pieces, 8);
  const unsigned blocks = token_blocks(T, sh);
  with_type(type, k <= 2, [&](auto it, auto at) {
    hipLaunchKernelGGL((k_moe_combine<decltype(it)::value, decltype(at)::value>),
                       dim3(blocks, row_blocks(pieces, blocks)), dim3(kRowThreads), 0, stream, ys,
                       pos, weights, T, (int)k, (int)H, sh, y);
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* dy, int64_t ld, const void* ys, int type,
                                       const int32_t* offs, const int32_t* pos,
                                       const float* weights, int64_t T, int64_t E, int64_t k,
                                       int64_t H, void* dys, float* dweights, hipStream_t stream) {
  const int64_t pieces = pieces_of(type, H);
  // a wave a token at most, so that no barrier is met (4096 x 1001 bf16, k = 4:
  // 16 us, a workgroup a token 26), unless each lane of a workgroup has two
  // pieces or more (4096 x 4096 bf16, k = 2: 35.3 us, a workgroup a token 33.9; 1000 x
  // 8192 fp16, k = 4: 57.5 and 28.9)
  const int sh = pieces >= 2 * kRowThreads ? 8 : lanes_log2(pieces, 6);
  // rows in flight: 4 for more than 2 experts (2000 x 2048 fp32, k = 8: 63.0 us, with 2
  // 66.4; 1000 x 8192 fp16, k = 4: 28.9 and 30.9; 4096 x 1001 bf16, k = 4: 15.7 and 16.6;
  // against it 4096 x 4096 bf16, k = 4: 68.2 and 65.3), 2 where tokens leave half of the
  // CUs without a workgroup: a token's places then go to more of them (1 x 8192 fp32,
  // k = 8: 5.9 us, with 4 9.7, all places in one workgroup 18.2)
  const unsigned blocks = token_blocks(T, sh), cus = device_cus();
  with_type(type, k <= 2 || 2 * blocks <= cus, [&](auto it, auto at) {
    constexpr unsigned AT = decltype(at)::value;
    const unsigned parts = ((unsigned)k + AT - 1) / AT, room = cus / blocks;
    hipLaunchKernelGGL((k_moe_combine_grad<decltype(it)::value, decltype(at)::value>),
                       dim3(blocks + kTailBlocks, parts < room ? parts : room > 1 ? room : 1),
                       dim3(kRowThreads), 0, stream, dy, ld, ys, offs, pos, weights, T, (int)E,
                       (int)k, (int)H, sh, dys, dweights);
  });
  return hipGetLastError();
}

}  // namespace bgt
