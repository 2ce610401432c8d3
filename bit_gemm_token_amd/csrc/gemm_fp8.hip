// gemm_fp8.hip -- products of rows and weights held in 8 bits (gfx950).
//
//     y_mn = sum_g 2^(a_gm + b_gn) sum_{k in g} qx_mk qw_nk,      g: blocks of 128 k
//
// with e4m3 codes qx (M x K'), qw (N x K') and exponent bytes a (K'/128 x M), b (K'/128 x
// N'/128). The matrix instructions for 8-bit floats take an exponent byte for every lane's 32 k
// of either operand, so the blocks' scales cost no vector instruction and the sums stay in
// one fp32 accumulator. The same instruction aligns the products of a few k to the largest of
// them and keeps 13 bits below it (measured: 2^16 + 2^3 in one group of k gives 2^16), an
// error of about 1.4e-5 of the sum for normal data at K = 128: far below the rounding of a
// 16-bit output, but not of an fp32 one. Outputs in fp32 therefore take bf16 products of the
// same codes (e4m3 is exact in bf16, the products exact in fp32, four instructions in place of
// one), with the group's scale applied to its fp32 sum.
//
// The order of k within a group is free as long as both operands agree: a lane takes 16-byte
// pieces where they are contiguous for its neighbours.
#include <algorithm>
#include <type_traits>

#include "fp8_common.h"
#include "launch.h"

namespace bgt {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v8i join(const uint4& a, const uint4& b) {
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
// eight codes (words 2p, 2p + 1 of a lane's 32) as bf16, exact
__device__ __forceinline__ v8b widen8(const v8i& c, int p) {
  v8b r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * p + h], 1.0f, false);
    const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * p + h], 1.0f, true);
    r[4 * h + 0] = a[0]; r[4 * h + 1] = a[1]; r[4 * h + 2] = b[0]; r[4 * h + 3] = b[1];
  }
  return r;
}

// rows past the last expert's are zero: workgroup z of nz clears its share
__device__ __forceinline__ void zero_rows(const Route& rt, int N, OutY y, int z, int nz) {
  const int64_t from = (int64_t)clamp_route(rt.offs[rt.E], 0, rt.R) * N, to = (int64_t)rt.R * N;
  for (int64_t i = from + (int64_t)z * blockDim.x + threadIdx.x; i < to; i += (int64_t)nz * blockDim.x)
    y.put(i, 0.0f);
}
constexpr int kZeroWgs = 64;

// waves of a streaming workgroup with so many 16 x 16 blocks: registers
constexpr int stream_most(int blocks) { return blocks > 4 ? 8 : 16; }

}  // namespace

// =====================================================================
// Few rows: the weights stream once through registers
// =====================================================================
// A workgroup takes 16 NT weight rows (outputs n) and 16 MT rows of x; its waves take the groups
// in turn, keep D of them in flight in registers, and their sums meet in LDS in wave order.
// XT >= 0: x comes as elements of that type and every wave turns its own groups' blocks into
// codes (a block's scale needs no other wave); the workgroups of the first weight rows write
// codes and scales out.
template <int NT, int MT, int D, bool EX, int XT, bool GR>
__global__ __launch_bounds__(stream_most(NT * MT) * 64) void k_f8_stream(
    const void* __restrict__ x, int64_t ldx, int Kx, const uint8_t* __restrict__ sx,
    const uint8_t* __restrict__ qw, const uint8_t* __restrict__ sw, int M, int N, int K, OutY y,
    Route rt, uint8_t* __restrict__ q_out, uint8_t* __restrict__ s_out) {
  __shared__ float red[stream_most(NT * MT) * MT * 4 * 64];
  const int G = K / kGroup, B = (N + kGroup - 1) / kGroup;
  const int KS = blockDim.x / kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const int c = lane % 16, s4 = lane / 16;
  const int ntn = (N + 16 * NT - 1) / (16 * NT);
  int tn, tm, r0 = 0, rows = M;
  if constexpr (GR) {
    int e;
    const int main_wgs = (int)gridDim.x - kZeroWgs;
    if ((int)blockIdx.x >= main_wgs) {
      zero_rows(rt, N, y, blockIdx.x - main_wgs, kZeroWgs);
      return;
    }
    if (!grouped_tile(blockIdx.x, 16 * MT, ntn, rt, e, r0, rows, tm, tn)) return;
    qw += e * rt.wstride;
    sw += e * rt.sstride;
  } else {
    // the row blocks of one column of tiles follow each other on one XCD
    const int ntm = (M + 16 * MT - 1) / (16 * MT), j = blockIdx.x / 8;
    tn = j / ntm * 8 + blockIdx.x % 8;
    tm = j % ntm;
    if (tn >= ntn) return;
  }
  const int n0 = tn * 16 * NT, m0 = tm * 16 * MT;

  const uint8_t* wsrc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = n0 + 16 * i + c;
    wsrc[i] = qw + (int64_t)(n < N ? n : N - 1) * K + 16 * s4;
  }
  const uint8_t* ssrc = sw + n0 / kGroup;
  int64_t row[MT];
  bool live[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + c;
    live[i] = m < rows;
    row[i] = live[i] ? m : 0;
    if constexpr (GR) row[i] = clamp_route(rt.tok[r0 + row[i]], 0, rt.T - 1);
  }
  const int64_t Ms = GR ? rt.T : M;

  constexpr int XW = XT < 0 ? 2 : (XT == kF32 ? 8 : 4);      // 16-byte pieces of x a lane and group
  uint4 wb[D][NT][2], xb[D][MT][XW];
  uint8_t sb[D], ab[D][MT];
  auto fetch = [&](int j, int g) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wb[j][i][h] = *reinterpret_cast<const uint4*>(wsrc[i] + (int64_t)g * kGroup + 64 * h);
    sb[j] = ssrc[(int64_t)g * B];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int h = 0; h < XW; ++h) xb[j][i][h] = make_uint4(0, 0, 0, 0);
      ab[j][i] = 0;
      if constexpr (XT < 0) {
        if (live[i]) {
          const uint8_t* p = static_cast<const uint8_t*>(x) + row[i] * K + (int64_t)g * kGroup + 16 * s4;
          xb[j][i][0] = *reinterpret_cast<const uint4*>(p);
          xb[j][i][1] = *reinterpret_cast<const uint4*>(p + 64);
          ab[j][i] = sx[(int64_t)g * Ms + row[i]];
        }
      } else {
        constexpr int EB = XT == kF32 ? 4 : 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = g * kGroup + 64 * h + 16 * s4;       // 16 elements, all there or none
          if (live[i] && k < Kx) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + (row[i] * ldx + k) * EB);
#pragma unroll
            for (int u = 0; u < XW / 2; ++u) xb[j][i][h * (XW / 2) + u] = p[u];
          }
        }
      }
    }
  };
  v4f acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](int j, int g) {
    v8i xc[MT];
    uint32_t sxb[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if constexpr (XT < 0) {
        xc[i] = join(xb[j][i][0], xb[j][i][1]);
        sxb[i] = ab[j][i];
      } else {
        float v[32];
#pragma unroll
        for (int u = 0; u < XW; ++u) {
          const uint4 w = xb[j][i][u];
          if constexpr (XT == kF32) {
            v[4 * u + 0] = __uint_as_float(w.x); v[4 * u + 1] = __uint_as_float(w.y);
            v[4 * u + 2] = __uint_as_float(w.z); v[4 * u + 3] = __uint_as_float(w.w);
          } else {
            const float4 a = widen_x4<XT>(make_uint2(w.x, w.y)), b = widen_x4<XT>(make_uint2(w.z, w.w));
            v[8 * u + 0] = a.x; v[8 * u + 1] = a.y; v[8 * u + 2] = a.z; v[8 * u + 3] = a.w;
            v[8 * u + 4] = b.x; v[8 * u + 5] = b.y; v[8 * u + 6] = b.z; v[8 * u + 7] = b.w;
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < 32; ++u) top = umax(top, abs_bits(v[u]));
        top = umax(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
        top = umax(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
        const uint32_t byte = f8_scale_byte(top);
        const float inv = f8_inverse(byte);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          xc[i][u] = (int)f8_pack4(v[4 * u] * inv, v[4 * u + 1] * inv, v[4 * u + 2] * inv, v[4 * u + 3] * inv);
        sxb[i] = byte;
        if (tn == 0 && live[i]) {
          uint8_t* p = q_out + row[i] * K + (int64_t)g * kGroup + 16 * s4;
          *reinterpret_cast<uint4*>(p) = make_uint4(xc[i][0], xc[i][1], xc[i][2], xc[i][3]);
          *reinterpret_cast<uint4*>(p + 64) = make_uint4(xc[i][4], xc[i][5], xc[i][6], xc[i][7]);
          if (s4 == 0) s_out[(int64_t)g * M + row[i]] = (uint8_t)byte;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const v8i w = join(wb[j][i][0], wb[j][i][1]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (EX) {
          v4f p = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w, u), widen8(xc[m], u), p, 0, 0, 0);
          const float a = f8_scale(sxb[m]), b = f8_scale(sb[j]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][m][r] = acc[i][m][r] + p[r] * a * b;
        } else {
          acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, xc[m], acc[i][m], 0, 0, 0,
                                                                       (int)sb[j], 0, (int)sxb[m]);
        }
      }
    }
  };

#pragma unroll
  for (int j = 0; j < D; ++j)
    if (wave + j * KS < G) fetch(j, wave + j * KS);
#pragma unroll 1
  for (int g = wave; g < G; g += D * KS) {
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (g + j * KS < G) {
        compute(j, g + j * KS);
        if (g + (j + D) * KS < G) fetch(j, g + (j + D) * KS);
      }
    }
  }

  // lane: row m = 16 mt + lane % 16, outputs n = 16 nt + 4 (lane / 16) + r
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(wave * MT * 4 + m * 4 + r) * 64 + lane] = acc[i][m][r];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += blockDim.x) {
      const int n = t % 16, m = t / 16;
      const int at = (m / 16 * 4 + n % 4) * 64 + n / 4 * 16 + m % 16;
      if (m0 + m >= rows || n0 + 16 * i + n >= N) continue;
      float v = 0.0f;
      for (int w = 0; w < KS; ++w) v += red[w * MT * 256 + at];
      y.put((int64_t)(r0 + m0 + m) * N + n0 + 16 * i + n, v);
    }
  }
}

// =====================================================================
// Many rows: BN x BM output tiles through LDS
// =====================================================================
// WN x WM waves of 32 x 32 blocks (v_mfma_scale_f32_32x32x64_f8f6f4, weights as the first
// operand: a lane then holds runs of four outputs n of one row m). One step is one group of
// 128 k: BN weight rows and BM rows of x of 128 bytes each, copied straight into LDS
// (16-byte pieces XOR-swizzled by row, so that the 32 rows of an operand read fall on
// distinct banks), two stages, one barrier a step. 16-bit outputs leave through the stages'
// LDS as whole rows.
template <int BN, int BM, int WN, int WM, bool EX, bool GR>
__global__ __launch_bounds__(WN * WM * 64) __attribute__((amdgpu_waves_per_eu(2))) void k_f8_tile(
    const uint8_t* __restrict__ qx, const uint8_t* __restrict__ sx, const uint8_t* __restrict__ qw,
    const uint8_t* __restrict__ sw, int M, int N, int K, OutY y, Route rt) {
  constexpr int NW = WN * WM;
  constexpr int FN = BN / WN / 32, FM = BM / WM / 32;          // 32 x 32 blocks of a wave
  constexpr int STG = (BN + BM) * kGroup;
  constexpr int WCP = BN / 8 / NW, XCP = BM / 8 / NW;          // 1 KiB copies a wave and step
  static_assert(BN / WN <= kGroup, "a wave's weight rows share one scale");
  __shared__ __align__(16) uint8_t S0[STG];
  __shared__ __align__(16) uint8_t S1[STG];
  const int G = K / kGroup, B = (N + kGroup - 1) / kGroup;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = tid % kWave;
  const int wn = wave % WN, wm = wave / WN;
  const int lr = lane % 32, hf = lane / 32;
  const int ntn = (N + BN - 1) / BN;
  int tm, tn, r0 = 0;
  if constexpr (GR) {
    int e, rows;
    const int main_wgs = (int)gridDim.x - kZeroWgs;
    if ((int)blockIdx.x >= main_wgs) {
      zero_rows(rt, N, y, blockIdx.x - main_wgs, kZeroWgs);
      return;
    }
    if (!grouped_tile(blockIdx.x, BM, ntn, rt, e, r0, rows, tm, tn)) return;
    M = rows;
    qw += e * rt.wstride;
    sw += e * rt.sstride;
  } else {
    tile_of(blockIdx.x, (M + BM - 1) / BM, ntn, tm, tn);
  }
  const int m0 = tm * BM, n0 = tn * BN;
  auto source_row = [&](int m) -> int64_t {                    // of tile row m (past the end: the last)
    const int r = m0 + m < M ? m0 + m : M - 1;
    return GR ? clamp_route(rt.tok[r0 + r], 0, rt.T - 1) : r;
  };

  // copy i of this wave: rows 8 b .. 8 b + 7, b = NW i + wave; lane L fills row 8 b + L / 8,
  // slot L % 8 with the row's piece (L % 8) ^ ((row / 2) % 8)
  const uint8_t *wsrc[WCP], *xsrc[XCP];
#pragma unroll
  for (int i = 0; i < WCP; ++i) {
    const int r = 8 * (NW * i + wave) + lane / 8;
    wsrc[i] = qw + (int64_t)(n0 + r < N ? n0 + r : N - 1) * K + 16 * ((lane % 8) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int i = 0; i < XCP; ++i) {
    const int r = 8 * (NW * i + wave) + lane / 8;
    xsrc[i] = qx + source_row(r) * K + 16 * ((lane % 8) ^ ((r >> 1) & 7));
  }
  auto issue = [&](int g, uint8_t* S) {
#pragma unroll
    for (int i = 0; i < WCP; ++i)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(wsrc[i] + (int64_t)g * kGroup),
          (__attribute__((address_space(3))) void*)(S + (NW * i + wave) * 1024), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < XCP; ++i)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(xsrc[i] + (int64_t)g * kGroup),
          (__attribute__((address_space(3))) void*)(S + BN * kGroup + (NW * i + wave) * 1024), 16, 0, 0);
  };
  const int64_t Ms = GR ? rt.T : M;
  const uint8_t* ssrc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) ssrc[i] = sx + source_row(wm * (BM / WM) + 32 * i + lr);
  const int nb = (n0 + wn * (BN / WN)) / kGroup;
  const uint8_t* wscale = sw + (nb < B ? nb : B - 1);
  uint32_t sa[FM], sb, na[FM], nb1;
  auto scales = [&](int g) {
    nb1 = wscale[(int64_t)g * B];
#pragma unroll
    for (int i = 0; i < FM; ++i) na[i] = ssrc[i][(int64_t)g * Ms];
  };

  auto fragment = [&](const uint8_t* S, int r, int h) {       // 32 codes: pieces 4h + 2hf, + 1
    const uint8_t* p = S + r * kGroup;
    const int f = (r >> 1) & 7, u = 4 * h + 2 * hf;
    return join(*reinterpret_cast<const uint4*>(p + 16 * (u ^ f)),
                *reinterpret_cast<const uint4*>(p + 16 * ((u + 1) ^ f)));
  };
  v16f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[i][m] = v16f{0.0f};
  auto compute = [&](const uint8_t* S) {
    if constexpr (EX) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int m = 0; m < FM; ++m) {
          v16f p = v16f{0.0f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v8i w = fragment(S, wn * (BN / WN) + 32 * i + lr, h);
            const v8i xx = fragment(S + BN * kGroup, wm * (BM / WM) + 32 * m + lr, h);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(w, u), widen8(xx, u), p, 0, 0, 0);
          }
          const float a = f8_scale(sa[m]), b = f8_scale(sb);
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][m][r] = acc[i][m][r] + p[r] * a * b;
        }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v8i w[FN], xx[FM];
#pragma unroll
        for (int i = 0; i < FN; ++i) w[i] = fragment(S, wn * (BN / WN) + 32 * i + lr, h);
#pragma unroll
        for (int m = 0; m < FM; ++m) xx[m] = fragment(S + BN * kGroup, wm * (BM / WM) + 32 * m + lr, h);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int m = 0; m < FM; ++m)
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[i], xx[m], acc[i][m], 0, 0, 0,
                                                                        (int)sb, 0, (int)sa[m]);
      }
    }
  };
  auto step = [&](int g, uint8_t* cur, uint8_t* nxt) {
    wait_vm<0>();                                     // group g and its scales landed
    lds_barrier();                                    // ... in every wave, and nxt is read
    sb = nb1;
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = na[i];
    if (g + 1 < G) {
      scales(g + 1);
      issue(g + 1, nxt);
    }
    compute(cur);
    wait_lds0();
  };
  scales(0);
  issue(0, S0);
#pragma unroll 1
  for (int g = 0; g < G; g += 2) {
    step(g, S0, S1);
    if (g + 1 < G) step(g + 1, S1, S0);
  }

  if constexpr (EX) {                                 // fp32: runs of four outputs a lane
    const bool vec = N % 4 == 0 && reinterpret_cast<uintptr_t>(y.p) % 16 == 0;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int row = m0 + wm * (BM / WM) + 32 * m + lr;
        if (row >= M) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * (BN / WN) + 32 * i + 8 * q + 4 * hf;
          float* p = static_cast<float*>(y.p) + (int64_t)(r0 + row) * N + n;
          if (vec && n < N) {
            *reinterpret_cast<float4*>(p) = make_float4(acc[i][m][4 * q], acc[i][m][4 * q + 1],
                                                        acc[i][m][4 * q + 2], acc[i][m][4 * q + 3]);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < N) p[r] = acc[i][m][4 * q + r];
          }
        }
      }
    return;
  }
  // 16 bits: the tile as BM rows of BN outputs in the stages' LDS, RPS rows a stage, 16-byte
  // pieces XOR-swizzled by row; then whole rows out
  constexpr int RPS = STG / (2 * BN);
  static_assert(BM <= 2 * RPS, "the tile fits the stages");
  __syncthreads();                                    // every wave is done with the stages
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int r = wm * (BM / WM) + 32 * m + lr;
      uint8_t* p = (r < RPS ? S0 : S1) + (r < RPS ? r : r - RPS) * (2 * BN);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int piece = (wn * (BN / WN) + 32 * i) / 8 + q;
        const float *v = reinterpret_cast<const float*>(&acc[i][m]) + 4 * q;
        const uint2 w = y.type == kF16 ? make_uint2(narrow2<kF16>(v[0], v[1]), narrow2<kF16>(v[2], v[3]))
                                       : make_uint2(narrow2<kBF16>(v[0], v[1]), narrow2<kBF16>(v[2], v[3]));
        *reinterpret_cast<uint2*>(p + 16 * (piece ^ (r & 15)) + 8 * hf) = w;
      }
    }
  __syncthreads();
  constexpr int PIECES = BN / 8;
  const bool vec = N % 8 == 0 && reinterpret_cast<uintptr_t>(y.p) % 16 == 0;
  uint16_t* yp = static_cast<uint16_t*>(y.p);
#pragma unroll 4
  for (int t = tid; t < BM * PIECES; t += NW * 64) {
    const int r = t / PIECES, piece = t % PIECES;
    const uint8_t* p = (r < RPS ? S0 : S1) + (r < RPS ? r : r - RPS) * (2 * BN) + 16 * (piece ^ (r & 15));
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const int n = n0 + 8 * piece;
    if (m0 + r >= M || n >= N) continue;
    uint16_t* o = yp + (int64_t)(r0 + m0 + r) * N + n;
    if (vec) {
      *reinterpret_cast<uint4*>(o) = v;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (n + u < N) o[u] = h[u];
    }
  }
}

// ------------------------------------------------------------------ launchers
namespace {

// waves of a streaming workgroup: as many as leave each two groups, at most `most`
int stream_waves(int64_t G, int most) {
  int ks = 1;
  while (ks < most && 2 * ks * 2 <= G) ks *= 2;
  return ks;
}

template <int NT, int MT, int D, bool EX, int XT, bool GR>
hipError_t stream_t(const void* x, int64_t ldx, int64_t Kx, const uint8_t* sx, const uint8_t* qw,
              const uint8_t* sw, int64_t M, int64_t N, int64_t K, OutY y, const Route& rt,
              uint8_t* q_out, uint8_t* s_out, hipStream_t stream) {
  const int64_t ntn = (N + 16 * NT - 1) / (16 * NT);
  const int64_t wgs = GR ? (rt.R / (16 * MT) + std::min<int64_t>(rt.E, rt.R)) * ntn + kZeroWgs
                         : (ntn + 7) / 8 * 8 * ((M + 16 * MT - 1) / (16 * MT));
  const int ks = stream_waves(K / kGroup, stream_most(NT * MT));
  if (!grid_fits(wgs, ks * kWave)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_f8_stream<NT, MT, D, EX, XT, GR>), dim3((unsigned)wgs), dim3(ks * kWave), 0,
                     stream, x, ldx, (int)Kx, sx, qw, sw, (int)M, (int)N, (int)K, y, rt, q_out, s_out);
  return hipGetLastError();
}

template <bool EX, bool GR>
hipError_t stream_rows(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                 int64_t M, int64_t N, int64_t K, OutY y, const Route& rt, int64_t per,
                 hipStream_t stream) {
  if (per <= 16)
    return stream_t<1, 1, 4, EX, -1, GR>(qx, K, K, sx, qw, sw, M, N, K, y, rt, nullptr, nullptr, stream);
  if (per <= 32)
    return stream_t<1, 2, 2, EX, -1, GR>(qx, K, K, sx, qw, sw, M, N, K, y, rt, nullptr, nullptr, stream);
  return stream_t<2, 4, 1, EX, -1, GR>(qx, K, K, sx, qw, sw, M, N, K, y, rt, nullptr, nullptr, stream);
}

template <int BN, int BM, int WN, int WM, bool EX, bool GR>
hipError_t tile_t(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw, int64_t M,
            int64_t N, int64_t K, OutY y, const Route& rt, hipStream_t stream) {
  const int64_t ntn = (N + BN - 1) / BN;
  const int64_t wgs = GR ? (rt.R / BM + std::min<int64_t>(rt.E, rt.R)) * ntn + kZeroWgs
                         : (M + BM - 1) / BM * ntn;
  if (!grid_fits(wgs, WN * WM * 64)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_f8_tile<BN, BM, WN, WM, EX, GR>), dim3((unsigned)wgs), dim3(WN * WM * 64), 0,
                     stream, qx, sx, qw, sw, (int)M, (int)N, (int)K, y, rt);
  return hipGetLastError();
}

template <bool GR>
hipError_t launch_t(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw, int64_t M,
              int64_t N, int64_t K, OutY y, const Route& rt, hipStream_t stream) {
  const bool ex = y.type == kF32;
  const int64_t per = GR ? (rt.R + rt.E - 1) / rt.E : M;      // rows of a matrix
  if (per <= 256)
    return ex ? stream_rows<true, GR>(qx, sx, qw, sw, M, N, K, y, rt, per, stream)
              : stream_rows<false, GR>(qx, sx, qw, sw, M, N, K, y, rt, per, stream);
  return ex ? tile_t<128, 128, 2, 4, true, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream)
            : tile_t<256, 256, 2, 4, false, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream);
}

}  // namespace

hipError_t launch_w8a8_f8(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw,
                          const uint8_t* sw, int64_t M, int64_t N, int64_t K, OutY y,
                          hipStream_t stream) {
  return launch_t<false>(qx, sx, qw, sw, M, N, K, y, Route{}, stream);
}

hipError_t launch_w8a8_f8_moe(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw,
                              const uint8_t* sw, int64_t N, int64_t K, const Route& rt, OutY y,
                              hipStream_t stream) {
  return launch_t<true>(qx, sx, qw, sw, rt.T, N, K, y, rt, stream);
}

hipError_t launch_w8a8_f8_linear(const void* x, int type, int64_t ldx, int64_t Kx, const uint8_t* qw,
                                 const uint8_t* sw, int64_t M, int64_t N, int64_t K, uint8_t* q,
                                 uint8_t* s, OutY y, hipStream_t stream) {
  const bool fused = M <= 16 && Kx % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                     ldx * (type == kF32 ? 4 : 2) % 16 == 0;
  if (!fused) {
    const hipError_t e = launch_f8_rows(x, type, M, Kx, ldx, q, s, stream);
    return e != hipSuccess ? e : launch_w8a8_f8(q, s, qw, sw, M, N, K, y, stream);
  }
  const Route rt{};
  const bool ex = y.type == kF32;
#define BGT_FUSED(T)                                                                               \
  return ex ? stream_t<1, 1, 2, true, T, false>(x, ldx, Kx, nullptr, qw, sw, M, N, K, y, rt, q, s, stream) \
            : stream_t<1, 1, 2, false, T, false>(x, ldx, Kx, nullptr, qw, sw, M, N, K, y, rt, q, s, stream)
  if (type == kF32) BGT_FUSED(kF32);
  if (type == kF16) BGT_FUSED(kF16);
  BGT_FUSED(kBF16);
#undef BGT_FUSED
}

}  // namespace bgt
