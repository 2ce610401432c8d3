// wgrad_fp8.hip -- a weight's gradient from the rows kept in 8 bits (gfx950).
//
//     dW_kn = sum_m (2^a_{k/128,m} qx_mk) dy_mn
//
// for one matrix, or for every expert over its slots (rows of dy are slots, rows of qx their
// tokens). The kept values are exact in bf16 (a power of two times e4m3). A bf16 dy is one
// bf16 operand as it is; an fp16 one is the sum of two bf16 terms, an fp32 one of three (8
// significant bits each, by truncation, the least term added first), so every product is exact
// and the sum is fp32.
//
// Both operands lie with the summed index m outermost, while a matrix instruction wants eight
// consecutive m of one column in a lane. A lane therefore loads two columns of eight rows
// (whole rows are contiguous over the lanes, and a wave's rows and scales are uniform), pairs
// rows with byte permutes, and writes 16-byte pieces [m / 8][column][8] to LDS, which are the
// operands: reads and writes are 16 bytes a lane in lane order. Two LDS stages of 32 rows, the
// next rows in registers, one barrier a step.
#include <algorithm>

#include "fp8_common.h"
#include "launch.h"

namespace bgt {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr int kStepRows = 32;

// the high halves of two words, the first in the low half
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
// leading 8 significant bits of v as a bf16 in the high half (a NaN stays one), and the rest
__device__ __forceinline__ uint32_t lead(float v, float& rest) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t h = (u & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : u & 0xFFFF0000u;
  rest = (u & 0x7F800000u) == 0x7F800000u ? 0.0f : v - __uint_as_float(h);
  return h;
}
constexpr int terms_of(int type) { return type == kBF16 ? 1 : type == kF16 ? 2 : 3; }

}  // namespace

// S x S outputs of dW a workgroup (S / 32 waves); GR: blockIdx.y is the expert. parts > 1:
// blockIdx.y is a part of the rows, whose fp32 sums go to part[y] (K x N).
template <int S, int DT, bool VEC, bool GR>
__global__ __launch_bounds__(S * 2) __attribute__((amdgpu_waves_per_eu(2))) void k_f8_wgrad(
    const uint8_t* __restrict__ qx, const uint8_t* __restrict__ sx, const void* __restrict__ dy,
    int64_t ld, int M, int K, int N, Route rt, OutY dw, int parts, float* __restrict__ part) {
  constexpr int NW = S / 32, TERMS = terms_of(DT);
  constexpr int WN = NW / 2;                          // 2 x WN waves
  constexpr int FK = S / 2 / 32, FN = S / WN / 32;    // 32 x 32 blocks of a wave
  constexpr int PANEL = 4 * S * 16;                   // 32 rows of S columns
  __shared__ __align__(16) uint8_t X0[PANEL];
  __shared__ __align__(16) uint8_t X1[PANEL];
  __shared__ __align__(16) uint8_t Y0[TERMS * PANEL];
  __shared__ __align__(16) uint8_t Y1[TERMS * PANEL];
  const int Kp = (K + kGroup - 1) / kGroup * kGroup;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = tid % kWave;
  const int ntk = (K + S - 1) / S, ntn = (N + S - 1) / S;
  int tk, tn, from = 0, to = M;
  tile_of(blockIdx.x, ntk, ntn, tk, tn);
  const int64_t Ms = GR ? rt.T : M;
  int64_t out0 = 0;
  if constexpr (GR) {
    from = clamp_route(rt.offs[blockIdx.y], 0, rt.R);
    to = clamp_route(rt.offs[blockIdx.y + 1], from, rt.R);
    out0 = (int64_t)blockIdx.y * K * N;
  } else if (parts > 1) {                             // whole steps to each part
    const int steps = (M + kStepRows - 1) / kStepRows;
    from = (int)((int64_t)blockIdx.y * steps / parts) * kStepRows;
    to = std::min(M, (int)((int64_t)(blockIdx.y + 1) * steps / parts) * kStepRows);
  }
  const int k0 = tk * S, n0 = tn * S;

  // this lane's columns 2 cp, 2 cp + 1 of the tile, rows 8 oct .. of a step; columns past the
  // end read the last ones (their outputs are never stored)
  const int oct = wave % 4, cp = wave / 4 * kWave + lane;
  int kc = k0 + 2 * cp, nc = n0 + 2 * cp;
  kc = kc < Kp ? kc : Kp - 2;
  const int kb = (k0 + wave / 4 * kGroup < Kp ? k0 + wave / 4 * kGroup : Kp - kGroup) / kGroup;
  if constexpr (VEC) nc = nc < N ? nc : N - 2;        // N even
  const int na = nc < N ? nc : N - 1, nb = nc + 1 < N ? nc + 1 : N - 1;

  constexpr int DW = DT == kF32 ? 2 : 1;              // words of two elements
  uint32_t xr[8], dr[8][DW], sr = 0;                  // rows as loaded; lane i < 8: scale of row i
  int tok = 0;                                        // lane i < 8: token of row i, a step ahead
  auto load_tok = [&](int m) {
    if constexpr (GR) {
      const int r = m + 8 * oct + (lane & 7);
      tok = clamp_route(rt.tok[r < to ? r : to - 1], 0, rt.T - 1);
    }
  };
  auto load = [&](int m) {                            // rows m + 8 oct ..; past the end: the last
    const int r = m + 8 * oct + (lane & 7);
    const int64_t mine = GR ? tok : (r < to ? r : to - 1);
    sr = sx[(int64_t)kb * Ms + mine];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ri = m + 8 * oct + i < to ? m + 8 * oct + i : to - 1;
      const int64_t src = GR ? __builtin_amdgcn_readlane(tok, i) : ri;
      xr[i] = *reinterpret_cast<const uint16_t*>(qx + src * Kp + kc);
      if constexpr (DT == kF32) {
        const float* p = static_cast<const float*>(dy) + (int64_t)ri * ld;
        if constexpr (VEC) {
          const uint2 u = *reinterpret_cast<const uint2*>(p + nc);
          dr[i][0] = u.x;
          dr[i][DW - 1] = u.y;
        } else {
          dr[i][0] = __float_as_uint(p[na]);
          dr[i][DW - 1] = __float_as_uint(p[nb]);
        }
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(dy) + (int64_t)ri * ld;
        if constexpr (VEC) dr[i][0] = *reinterpret_cast<const uint32_t*>(p + nc);
        else dr[i][0] = (uint32_t)p[na] | (uint32_t)p[nb] << 16;
      }
    }
  };
  auto put = [&](int m, uint8_t* X, uint8_t* Y) {     // the loaded rows (of step m) as operands
    const int at = (oct * S + 2 * cp) * 16;
    const int live = to - (m + 8 * oct);              // rows below the end
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = __builtin_amdgcn_readlane(sr, i);
      const uint32_t c = byte == kF8NanByte ? 0x7F7Fu : xr[i];
      const v2b v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c, f8_scale(byte), false);
      w[i] = i < live ? __builtin_bit_cast(uint32_t, v) : 0u;
    }
    *reinterpret_cast<uint4*>(X + at) = make_uint4(low_halves(w[0], w[1]), low_halves(w[2], w[3]),
                                                   low_halves(w[4], w[5]), low_halves(w[6], w[7]));
    *reinterpret_cast<uint4*>(X + at + 16) =
        make_uint4(high_halves(w[0], w[1]), high_halves(w[2], w[3]), high_halves(w[4], w[5]),
                   high_halves(w[6], w[7]));
    if constexpr (DT == kBF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < live ? dr[i][0] : 0u;
      *reinterpret_cast<uint4*>(Y + at) = make_uint4(low_halves(w[0], w[1]), low_halves(w[2], w[3]),
                                                     low_halves(w[4], w[5]), low_halves(w[6], w[7]));
      *reinterpret_cast<uint4*>(Y + at + 16) =
          make_uint4(high_halves(w[0], w[1]), high_halves(w[2], w[3]), high_halves(w[4], w[5]),
                     high_halves(w[6], w[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {                   // the two columns
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (DT == kF32) v[i] = __uint_as_float(dr[i][j]);
          else {
            const __half2 h = *reinterpret_cast<const __half2*>(&dr[i][0]);
            v[i] = j == 0 ? __low2float(h) : __high2float(h);
          }
          if (i >= live) v[i] = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = lead(v[i], v[i]);
          *reinterpret_cast<uint4*>(Y + t * PANEL + at + 16 * j) =
              make_uint4(high_halves(w[0], w[1]), high_halves(w[2], w[3]), high_halves(w[4], w[5]),
                         high_halves(w[6], w[7]));
        }
      }
    }
  };

  const int wk = wave / WN, wn = wave % WN;
  const int lr = lane % 32, hf = lane / 32;
  v16f acc[FK][FN];
#pragma unroll
  for (int i = 0; i < FK; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v16f{0.0f};
  auto compute = [&](const uint8_t* X, const uint8_t* Y) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {                     // 16 rows each: pieces 2h + hf
      v8b a[FK];
#pragma unroll
      for (int i = 0; i < FK; ++i)
        a[i] = *reinterpret_cast<const v8b*>(X + ((2 * h + hf) * S + wk * (S / 2) + 32 * i + lr) * 16);
#pragma unroll
      for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v8b b = *reinterpret_cast<const v8b*>(
              Y + t * PANEL + ((2 * h + hf) * S + wn * (S / WN) + 32 * j + lr) * 16);
#pragma unroll
          for (int i = 0; i < FK; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b, acc[i][j], 0, 0, 0);
        }
    }
  };
  if (from < to) {
    load_tok(from);
    load(from);
    load_tok(from + kStepRows);
    put(from, X0, Y0);
    load(from + kStepRows);
    load_tok(from + 2 * kStepRows);
    // stage of step m is written by all waves at the barrier, the other one is read
    auto step = [&](int m, const uint8_t* X, const uint8_t* Y, uint8_t* Xn, uint8_t* Yn) {
      __syncthreads();
      put(m + kStepRows, Xn, Yn);
      load(m + 2 * kStepRows);
      load_tok(m + 3 * kStepRows);
      compute(X, Y);
    };
#pragma unroll 1
    for (int m = from; m < to; m += 2 * kStepRows) {
      step(m, X0, Y0, X1, Y1);
      if (m + kStepRows < to) step(m + kStepRows, X1, Y1, X0, Y0);
    }
  }
  // lane: column n = lane % 32 of a block, rows k = 8 (r / 4) + 4 hf + r % 4
#pragma unroll
  for (int i = 0; i < FK; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + wn * (S / WN) + 32 * j + lr;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = k0 + wk * (S / 2) + 32 * i + 8 * (r / 4) + 4 * hf + r % 4;
        if (k >= K || n >= N) continue;
        const int64_t o = (int64_t)k * N + n;
        if (!GR && parts > 1) part[(int64_t)blockIdx.y * K * N + o] = acc[i][j][r];
        else dw.put(out0 + o, acc[i][j][r]);
      }
    }
}

// the parts' sums, in order
__global__ __launch_bounds__(256) void k_f8_wgrad_join(const float* __restrict__ part, int parts,
                                                       int64_t count, OutY dw) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float v = 0.0f;
  for (int p = 0; p < parts; ++p) v += part[p * count + i];
  dw.put(i, v);
}

namespace {

constexpr int kTile = 256;

// parts of the rows of one matrix: doubled while the tiles fill at most half of the CUs and
// every part keeps 256 rows
int wgrad_parts(int64_t M, int64_t K, int64_t N) {
  const int64_t tiles = ((K + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  int p = 1;
  while (tiles * p * 2 <= device_cus() && M / (2 * p) >= 256) p *= 2;
  return p;
}

template <int DT, bool GR>
hipError_t wgrad_t(const uint8_t* qx, const uint8_t* sx, const void* dy, int64_t ld, int64_t M, int64_t K,
             int64_t N, const Route& rt, OutY dw, float* ws, hipStream_t stream) {
  const int64_t tiles = ((K + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int parts = GR ? 1 : wgrad_parts(M, K, N);
  const dim3 grid((unsigned)tiles, (unsigned)(GR ? rt.E : parts)), block(kTile * 2);
  if (!grid_fits(tiles, kTile * 2) || !grid_fits((K * N + 255) / 256, 256))
    return hipErrorInvalidConfiguration;
  constexpr int two = DT == kF32 ? 8 : 4;             // bytes of two elements of dy
  const bool vec = N % 2 == 0 && ld % 2 == 0 && reinterpret_cast<uintptr_t>(dy) % two == 0;
  if (vec)
    hipLaunchKernelGGL((k_f8_wgrad<kTile, DT, true, GR>), grid, block, 0, stream, qx, sx, dy, ld,
                       (int)M, (int)K, (int)N, rt, dw, parts, ws);
  else
    hipLaunchKernelGGL((k_f8_wgrad<kTile, DT, false, GR>), grid, block, 0, stream, qx, sx, dy, ld,
                       (int)M, (int)K, (int)N, rt, dw, parts, ws);
  if (parts > 1)
    hipLaunchKernelGGL(k_f8_wgrad_join, dim3((unsigned)((K * N + 255) / 256)), dim3(256), 0, stream,
                       ws, parts, K * N, dw);
  return hipGetLastError();
}

}  // namespace

int64_t f8_wgrad_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t E) {
  const int parts = E > 0 ? 1 : wgrad_parts(M, K, N);
  return parts > 1 ? (int64_t)parts * K * N * 4 : 0;
}

hipError_t launch_f8_wgrad(const uint8_t* qx, const uint8_t* sx, const void* dy, int64_t ld,
                           int64_t M, int64_t K, int64_t N, const Route& rt, OutY dw, void* ws,
                           hipStream_t stream) {
  float* p = static_cast<float*>(ws);
#define BGT_CALL(T)                                                              \
  return rt.E > 0 ? wgrad_t<T, true>(qx, sx, dy, ld, M, K, N, rt, dw, p, stream) \
                  : wgrad_t<T, false>(qx, sx, dy, ld, M, K, N, rt, dw, p, stream)
  if (dw.type == kF32) BGT_CALL(kF32);
  if (dw.type == kF16) BGT_CALL(kF16);
  BGT_CALL(kBF16);
#undef BGT_CALL
}

}  // namespace bgt
