// quant_fp8.hip -- rows and weights held in 8 bits (e4m3 with a power of two per block), the
// gated activation from and to that form, and its gradient (gfx950).
//
//   rows      q_ik = e4m3(x_ik / 2^e), e of (row i, block k/128): fp8_common.h
//   weights   the same with one e for 128 x 128 elements, written N x K' (the product over K)
//             and, if asked for, K x N' (the product over N, a gradient's)
//   gate      h = silu(g) * u, silu(g) = g / (1 + exp(-g)), stored as rows; g and u too, which
//             is all that the gradient needs:
//             dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = 1 / (1 + exp(-g))
//
// All are bound by memory. A row's block lies in 16 lanes of 8 elements (16-byte loads of
// 16-bit types, 8-byte stores of codes); its maximum takes four lane exchanges. A workgroup
// takes one block of R rows, so that the rows' exponent bytes, kept block by block, leave as
// one run.
#include "fp8_common.h"
#include "launch.h"

namespace bgt {

namespace {

constexpr int kRowLanes = 16, kRowsAtOnce = 16, kThreads = kRowLanes * kRowsAtOnce;

__device__ __forceinline__ uint32_t top_of(const float* v) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = umax(t, abs_bits(v[j]));
  return max16(t);
}
__device__ __forceinline__ uint2 codes_of(const float* v, float scale) {
  return make_uint2(f8_pack4(v[0], v[1], v[2], v[3], scale), f8_pack4(v[4], v[5], v[6], v[7], scale));
}
template <int IT, bool VEC>
__device__ __forceinline__ void load_piece(const void* x, int64_t row, int c, int K, float* v) {
  if constexpr (VEC) {                               // K % 8 == 0: a piece is whole or absent
    if (c < K) load8<IT>(x, row + c, v);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  } else {
    load8_tail<IT>(x, row, c, K, v);
  }
}

}  // namespace

// one block of STEPS * 16 rows per workgroup: rows m0 .., columns 128 b ..
template <int IT, bool VEC, int STEPS>
__global__ __launch_bounds__(kThreads) void k_f8_rows(const void* __restrict__ x, int64_t M, int K,
                                                      int64_t ld, uint8_t* __restrict__ q,
                                                      uint8_t* __restrict__ scale) {
  const int G = (K + kGroup - 1) / kGroup;
  const int b = blockIdx.x % G;
  const int64_t m0 = (int64_t)(blockIdx.x / G) * (STEPS * kRowsAtOnce) + threadIdx.x / kRowLanes;
  const int c = b * kGroup + 8 * (threadIdx.x % kRowLanes);
  float v[STEPS][8];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce;
    load_piece<IT, VEC>(x, (m < M ? m : M - 1) * ld, c, K, v[s]);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce;
    const uint32_t byte = f8_scale_byte(top_of(v[s]));
    if (m >= M) continue;
    *reinterpret_cast<uint2*>(q + m * ((int64_t)G * kGroup) + c) = codes_of(v[s], f8_scale(byte));
    if (threadIdx.x % kRowLanes == 0) scale[(int64_t)b * M + m] = (uint8_t)byte;
  }
}

template <int OT, bool VEC, int STEPS>
__global__ __launch_bounds__(kThreads) void k_f8_values(const uint8_t* __restrict__ q,
                                                        const uint8_t* __restrict__ scale,
                                                        int64_t M, int K, void* __restrict__ y) {
  const int G = (K + kGroup - 1) / kGroup;
  const int b = blockIdx.x % G;
  const int64_t m0 = (int64_t)(blockIdx.x / G) * (STEPS * kRowsAtOnce) + threadIdx.x / kRowLanes;
  const int c = b * kGroup + 8 * (threadIdx.x % kRowLanes);
  uint2 w[STEPS];
  float s[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t m = m0 + i * kRowsAtOnce < M ? m0 + i * kRowsAtOnce : M - 1;
    w[i] = *reinterpret_cast<const uint2*>(q + m * ((int64_t)G * kGroup) + c);
    s[i] = f8_scale(scale[(int64_t)b * M + m]);
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t m = m0 + i * kRowsAtOnce;
    if (m >= M) continue;
    float v[8];
    f8_unpack4(w[i].x, v);
    f8_unpack4(w[i].y, v + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s[i];
    if constexpr (VEC) {
      if (c < K) store8<OT>(y, m * K + c, v);
    } else {
      store8_tail<OT>(y, m * K, c, K, v);
    }
  }
}

// ------------------------------------------------------------------------ weights
// One workgroup per 128 x 128 block: thread (r, n8) holds rows 8r .. 8r+7 of columns 8 n8 ..,
// the block's maximum meets in LDS, codes go out turned (K x N') from the registers, and as
// N x K' through an LDS tile: eight codes of a column are one 8-byte LDS write after a byte
// transposition of 8 x 8 in registers.
constexpr int kTilePitch = 128 + 16;                 // 16-byte reads of a row stay aligned

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}
// 4 x 4 bytes: word i of out holds byte i of each input word
__device__ __forceinline__ void transpose4(const uint32_t* in, uint32_t* out) {
  const uint32_t a = perm(in[1], in[0], 0x05010400u), b = perm(in[3], in[2], 0x05010400u);
  const uint32_t c = perm(in[1], in[0], 0x07030602u), d = perm(in[3], in[2], 0x07030602u);
  out[0] = perm(b, a, 0x05040100u);
  out[1] = perm(b, a, 0x07060302u);
  out[2] = perm(d, c, 0x05040100u);
  out[3] = perm(d, c, 0x07060302u);
}

template <int IT, bool VEC>
__global__ __launch_bounds__(256) void k_f8_weights(const void* __restrict__ w, int K, int N,
                                                    uint8_t* __restrict__ qw,
                                                    uint8_t* __restrict__ sw,
                                                    uint8_t* __restrict__ qt,
                                                    uint8_t* __restrict__ st) {
  __shared__ __align__(16) uint8_t tile[128 * kTilePitch];
  __shared__ uint32_t tops[4];
  const int A = (K + kGroup - 1) / kGroup, B = (N + kGroup - 1) / kGroup;
  const int a = blockIdx.x / B, b = blockIdx.x % B;
  const int64_t e = blockIdx.y;
  const int t = threadIdx.x, r8 = 8 * (t / 16), n8 = 8 * (t % 16);
  const int k0 = a * kGroup + r8, n0 = b * kGroup + n8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k0 + i < K) {
      load_piece<IT, VEC>(w, (e * K + k0 + i) * N, n0, N, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, abs_bits(v[i][j]));
  top = max16(top);
#pragma unroll
  for (int o = kRowLanes; o < kWave; o <<= 1) top = umax(top, (uint32_t)__shfl_xor((int)top, o, kWave));
  if (t % kWave == 0) tops[t / kWave] = top;
  __syncthreads();
  top = umax(umax(tops[0], tops[1]), umax(tops[2], tops[3]));
  const uint32_t byte = f8_scale_byte(top);
  const float scale = f8_scale(byte);
  if (t == 0) {
    sw[(e * A + a) * B + b] = (uint8_t)byte;
    if (st != nullptr) st[(e * B + b) * A + a] = (uint8_t)byte;
  }
  uint32_t lo[8], hi[8];                             // row i: columns 0..3 and 4..7
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint2 c = codes_of(v[i], scale);
    lo[i] = c.x;
    hi[i] = c.y;
  }
  if (qt != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < K)
        *reinterpret_cast<uint2*>(qt + (e * K + k0 + i) * ((int64_t)B * kGroup) + n0) =
            make_uint2(lo[i], hi[i]);
  }
  uint32_t x[4], y[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    transpose4(h ? hi : lo, x);                      // rows 0..3 of columns 4h ..
    transpose4((h ? hi : lo) + 4, y);                // rows 4..7
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint2*>(tile + (n8 + 4 * h + j) * kTilePitch + r8) = make_uint2(x[j], y[j]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = 32 * i + t / 8, c = 16 * (t % 8);
    if (b * kGroup + n < N)
      *reinterpret_cast<uint4*>(qw + (e * N + b * kGroup + n) * ((int64_t)A * kGroup) + a * kGroup + c) =
          *reinterpret_cast<const uint4*>(tile + n * kTilePitch + c);
  }
}

// --------------------------------------------------------------------- gated activation
// 1 / (1 + exp(-g)) from t = exp(-|g|), which does not overflow: 1 / (1 + t), for g < 0 times t.
// t = 2^y (1 + r ln 2) with y + r = -|g| log2(e) to twice fp32's digits; 1 + t lies in [1, 2], where
// the reciprocal instruction is right to one unit. A NaN gives 1; every use multiplies by g too.
// (k_f8_gate, 8192 x 14336 bf16: 200 us with expf and a division, which instructions bound, 180 with
// this, 167 with sigmoid_fast and codes scaled by their conversion.)
__device__ __forceinline__ float sigmoid(float g) {
  const float a = -fminf(fabsf(g), 200.0f);           // t is 0 from 104 on
  const float y = a * 1.44269504f;
  const float r = __builtin_fmaf(a, 1.92596299e-8f, __builtin_fmaf(a, 1.44269504f, -y));
  const float e = __builtin_exp2f(y), t = __builtin_fmaf(e, r * 0.693147181f, e);
  const float s = __builtin_amdgcn_rcpf(1.0f + t);
  return g < 0.0f ? t * s : s;
}

// The same where the result goes to 8 bits: below 2^-126 (g < -87) it may be 0. 1 / (1 + t) with
// t = exp(-g), infinite where that overflows.
__device__ __forceinline__ float sigmoid_fast(float g) {
  const float a = __builtin_amdgcn_fmed3f(-g, -100.0f, 100.0f);
  const float y = a * 1.44269504f;
  const float r = __builtin_fmaf(a, 1.92596299e-8f, __builtin_fmaf(a, 1.44269504f, -y));
  const float t = __builtin_amdgcn_exp2f(y) * __builtin_fmaf(r, 0.693147181f, 1.0f);
  return __builtin_amdgcn_rcpf(1.0f + t);
}

template <int IT, bool VEC, int STEPS>
__global__ __launch_bounds__(kThreads) void k_f8_gate(
    const void* __restrict__ gate, int64_t ldg, const void* __restrict__ up, int64_t ldu, int64_t M,
    int K, uint8_t* __restrict__ hq, uint8_t* __restrict__ hs, uint8_t* __restrict__ gq,
    uint8_t* __restrict__ gs, uint8_t* __restrict__ uq, uint8_t* __restrict__ us) {
  const int G = (K + kGroup - 1) / kGroup;
  const int b = blockIdx.x % G;
  const int64_t m0 = (int64_t)(blockIdx.x / G) * (STEPS * kRowsAtOnce) + threadIdx.x / kRowLanes;
  const int c = b * kGroup + 8 * (threadIdx.x % kRowLanes);
  float g[STEPS][8], u[STEPS][8];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce < M ? m0 + s * kRowsAtOnce : M - 1;
    load_piece<IT, VEC>(gate, m * ldg, c, K, g[s]);
    load_piece<IT, VEC>(up, m * ldu, c, K, u[s]);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce;
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[s][j] * sigmoid_fast(g[s][j]) * u[s][j];
    const uint32_t bg = f8_scale_byte(top_of(g[s])), bu = f8_scale_byte(top_of(u[s]));
    float top = 0.0f;                                 // a NaN of h comes from one, or an infinity, of g or u
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[j]));
    uint32_t bh = f8_scale_byte(max16(__float_as_uint(top)));
    bh = umax(bh, umax(bg, bu) == kF8NanByte ? kF8NanByte : 0u);
    if (m >= M) continue;
    const int64_t o = m * ((int64_t)G * kGroup) + c;
    *reinterpret_cast<uint2*>(hq + o) = codes_of(h, f8_scale(bh));
    // g and u wait for the backward pass, h is read next (8192 x 14336 bf16 171 us without)
    store_once(gq + o, codes_of(g[s], f8_scale(bg)));
    store_once(uq + o, codes_of(u[s], f8_scale(bu)));
    if (threadIdx.x % kRowLanes == 0) {
      hs[(int64_t)b * M + m] = (uint8_t)bh;
      gs[(int64_t)b * M + m] = (uint8_t)bg;
      us[(int64_t)b * M + m] = (uint8_t)bu;
    }
  }
}

template <int IT, bool VEC, int STEPS>
__global__ __launch_bounds__(kThreads) void k_f8_gate_grad(
    const void* __restrict__ dh, int64_t ld, const uint8_t* __restrict__ gq,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uq, const uint8_t* __restrict__ us,
    int64_t M, int K, void* __restrict__ dg, void* __restrict__ du) {
  const int G = (K + kGroup - 1) / kGroup;
  const int b = blockIdx.x % G;
  const int64_t m0 = (int64_t)(blockIdx.x / G) * (STEPS * kRowsAtOnce) + threadIdx.x / kRowLanes;
  const int c = b * kGroup + 8 * (threadIdx.x % kRowLanes);
  float d[STEPS][8], sg[STEPS], su[STEPS];
  uint2 wg[STEPS], wu[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce < M ? m0 + s * kRowsAtOnce : M - 1;
    const int64_t o = m * ((int64_t)G * kGroup) + c;
    load_piece<IT, VEC>(dh, m * ld, c, K, d[s]);
    wg[s] = *reinterpret_cast<const uint2*>(gq + o);
    wu[s] = *reinterpret_cast<const uint2*>(uq + o);
    sg[s] = f8_scale(gs[(int64_t)b * M + m]);
    su[s] = f8_scale(us[(int64_t)b * M + m]);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t m = m0 + s * kRowsAtOnce;
    if (m >= M) continue;
    float g[8], u[8], a[8];
    f8_unpack4(wg[s].x, g);
    f8_unpack4(wg[s].y, g + 4);
    f8_unpack4(wu[s].x, u);
    f8_unpack4(wu[s].y, u + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g[j] * sg[s], uj = u[j] * su[s], sig = sigmoid(gj);
      // the larger of dh and u meets the small factor first: dh u alone may leave fp32's range
      const float f = sig * (1.0f + gj * (1.0f - sig)), dj = d[s][j];
      const bool up = fabsf(uj) > fabsf(dj);
      a[j] = (up ? uj : dj) * f * (up ? dj : uj);
      d[s][j] = dj * (gj * sig);
    }
    if constexpr (VEC) {
      if (c < K) {
        store8<IT>(dg, m * K + c, a);
        store8<IT>(du, m * K + c, d[s]);
      }
    } else {
      store8_tail<IT>(dg, m * K, c, K, a);
      store8_tail<IT>(du, m * K, c, K, d[s]);
    }
  }
}

// ------------------------------------------------------------------ launchers
namespace {

// 16 bytes at a time: pieces of 8 elements start on 16 bytes in every row and are whole
bool whole(const void* p, int type, int64_t ld, int64_t K) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && K % 8 == 0 && ld * (type == kF32 ? 4 : 2) % 16 == 0;
}
// four rows a thread once the launch still has a few workgroups for every CU
int steps_of(int64_t M, int64_t G) { return (M + 63) / 64 * G >= 4 * device_cus() ? 4 : 1; }

int64_t grid_of(int64_t M, int64_t G, int steps) {
  return (M + steps * kRowsAtOnce - 1) / (steps * kRowsAtOnce) * G;
}

}  // namespace

#define BGT_BY_TYPE(T, CALL)                \
  do {                                      \
    if ((T) == kF32) CALL(kF32);            \
    else if ((T) == kF16) CALL(kF16);       \
    else CALL(kBF16);                       \
  } while (0)

hipError_t launch_f8_rows(const void* x, int type, int64_t M, int64_t K, int64_t ld, uint8_t* q,
                          uint8_t* scale, hipStream_t stream) {
  const int64_t G = (K + kGroup - 1) / kGroup;
  const bool vec = whole(x, type, ld, K);
  const int steps = vec ? steps_of(M, G) : 1;
  const int64_t wgs = grid_of(M, G, steps);
  if (!grid_fits(wgs, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs), block(kThreads);
#define BGT_CALL(T)                                                                                \
  do {                                                                                             \
    if (!vec) hipLaunchKernelGGL((k_f8_rows<T, false, 1>), grid, block, 0, stream, x, M, (int)K, ld, q, scale); \
    else if (steps == 1) hipLaunchKernelGGL((k_f8_rows<T, true, 1>), grid, block, 0, stream, x, M, (int)K, ld, q, scale); \
    else hipLaunchKernelGGL((k_f8_rows<T, true, 4>), grid, block, 0, stream, x, M, (int)K, ld, q, scale); \
  } while (0)
  BGT_BY_TYPE(type, BGT_CALL);
#undef BGT_CALL
  return hipGetLastError();
}

hipError_t launch_f8_values(const uint8_t* q, const uint8_t* scale, int64_t M, int64_t K, void* y,
                            int type, hipStream_t stream) {
  const int64_t G = (K + kGroup - 1) / kGroup;
  const bool vec = whole(y, type, K, K);
  const int steps = vec ? steps_of(M, G) : 1;
  const int64_t wgs = grid_of(M, G, steps);
  if (!grid_fits(wgs, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs), block(kThreads);
#define BGT_CALL(T)                                                                                \
  do {                                                                                             \
    if (!vec) hipLaunchKernelGGL((k_f8_values<T, false, 1>), grid, block, 0, stream, q, scale, M, (int)K, y); \
    else if (steps == 1) hipLaunchKernelGGL((k_f8_values<T, true, 1>), grid, block, 0, stream, q, scale, M, (int)K, y); \
    else hipLaunchKernelGGL((k_f8_values<T, true, 4>), grid, block, 0, stream, q, scale, M, (int)K, y); \
  } while (0)
  BGT_BY_TYPE(type, BGT_CALL);
#undef BGT_CALL
  return hipGetLastError();
}

hipError_t launch_f8_weights(const void* w, int type, int64_t E, int64_t K, int64_t N, uint8_t* qw,
                             uint8_t* sw, uint8_t* qt, uint8_t* st, hipStream_t stream) {
  const int64_t A = (K + kGroup - 1) / kGroup, B = (N + kGroup - 1) / kGroup;
  const bool vec = whole(w, type, N, N);
  if (!grid_fits(A * B, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(A * B), (unsigned)E), block(256);
#define BGT_CALL(T)                                                                                \
  do {                                                                                             \
    if (vec) hipLaunchKernelGGL((k_f8_weights<T, true>), grid, block, 0, stream, w, (int)K, (int)N, qw, sw, qt, st); \
    else hipLaunchKernelGGL((k_f8_weights<T, false>), grid, block, 0, stream, w, (int)K, (int)N, qw, sw, qt, st); \
  } while (0)
  BGT_BY_TYPE(type, BGT_CALL);
#undef BGT_CALL
  return hipGetLastError();
}

hipError_t launch_f8_gate(const void* gate, int64_t ldg, const void* up, int64_t ldu, int type,
                          int64_t M, int64_t K, uint8_t* hq, uint8_t* hs, uint8_t* gq, uint8_t* gs,
                          uint8_t* uq, uint8_t* us, hipStream_t stream) {
  const int64_t G = (K + kGroup - 1) / kGroup;
  const bool vec = whole(gate, type, ldg, K) && whole(up, type, ldu, K);
  const int steps = vec && steps_of(M, G) == 4 ? 2 : 1;
  const int64_t wgs = grid_of(M, G, steps);
  if (!grid_fits(wgs, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs), block(kThreads);
#define BGT_CALL(T)                                                                                \
  do {                                                                                             \
    if (!vec) hipLaunchKernelGGL((k_f8_gate<T, false, 1>), grid, block, 0, stream, gate, ldg, up, ldu, M, (int)K, hq, hs, gq, gs, uq, us); \
    else if (steps == 1) hipLaunchKernelGGL((k_f8_gate<T, true, 1>), grid, block, 0, stream, gate, ldg, up, ldu, M, (int)K, hq, hs, gq, gs, uq, us); \
    else hipLaunchKernelGGL((k_f8_gate<T, true, 2>), grid, block, 0, stream, gate, ldg, up, ldu, M, (int)K, hq, hs, gq, gs, uq, us); \
  } while (0)
  BGT_BY_TYPE(type, BGT_CALL);
#undef BGT_CALL
  return hipGetLastError();
}

hipError_t launch_f8_gate_grad(const void* dh, int64_t ld, int type, const uint8_t* gq,
                               const uint8_t* gs, const uint8_t* uq, const uint8_t* us, int64_t M,
                               int64_t K, void* dg, void* du, hipStream_t stream) {
  const int64_t G = (K + kGroup - 1) / kGroup;
  const bool vec = whole(dh, type, ld, K) && whole(dg, type, K, K) && whole(du, type, K, K);
  const int steps = vec && steps_of(M, G) == 4 ? 2 : 1;
  const int64_t wgs = grid_of(M, G, steps);
  if (!grid_fits(wgs, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs), block(kThreads);
#define BGT_CALL(T)                                                                                \
  do {                                                                                             \
    if (!vec) hipLaunchKernelGGL((k_f8_gate_grad<T, false, 1>), grid, block, 0, stream, dh, ld, gq, gs, uq, us, M, (int)K, dg, du); \
    else if (steps == 1) hipLaunchKernelGGL((k_f8_gate_grad<T, true, 1>), grid, block, 0, stream, dh, ld, gq, gs, uq, us, M, (int)K, dg, du); \
    else hipLaunchKernelGGL((k_f8_gate_grad<T, true, 2>), grid, block, 0, stream, dh, ld, gq, gs, uq, us, M, (int)K, dg, du); \
  } while (0)
  BGT_BY_TYPE(type, BGT_CALL);
#undef BGT_CALL
  return hipGetLastError();
}

}  // namespace bgt
