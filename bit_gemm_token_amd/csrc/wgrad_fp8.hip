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
// consecutive m of one column in a lane. They are kept in LDS as they lie, rows of columns, and
// read through the transposing LDS read (four rows of 16 columns: a lane gets the four rows of
// its column). 16-bit floats of the matrix product's own type go to LDS straight from memory
// (aligned bf16 rows); codes and the other types pass through registers, a step ahead, where
// they are widened or split. Rows are XOR-swizzled by 64 bytes so that the four rows of a read
// lie on distinct banks. Two LDS stages, one barrier a step.
//
// What bounds it: 32 rows of a 256 x 256 tile are 1024 cycles of matrix instructions for each term
// of dy and, for bf16, as many of LDS traffic (96 KiB read, 32 KiB written), which have to overlap.
// 8192 rows, 4096 x 4096: bf16 223 us back to back (1230 TFLOP/s; a library product of bf16 operands
// 1361), fp16 415 (661, 1322 in terms), fp32 646 (425, 1276 in terms). fp32 tiles are 256 x 128, two
// workgroups a CU: the three terms of a 256 x 256 tile leave LDS for one. Two columns of eight rows a
// lane, paired by byte permutes, took 390, and of 4096 rows 345 and 469 (now 222 and 329-347).
#include <algorithm>

#include "fp8_common.h"
#include "launch.h"

namespace bgt {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

enum { kByElement, kByPiece, kStraight };             // how dy's rows come

__device__ const uint4 kZeroPiece = {0, 0, 0, 0};     // what rows behind the last are read from

// two leading parts of 8 significant bits as bf16, in one word each; v: what is left
__device__ __forceinline__ uint32_t lead2(float& a, float& b) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  a -= __uint_as_float(ua & 0xFFFF0000u);
  b -= __uint_as_float(ub & 0xFFFF0000u);
  return __builtin_amdgcn_perm(ub, ua, 0x07060302u);
}
constexpr int terms_of(int type) { return type == kBF16 ? 1 : type == kF16 ? 2 : 3; }

}  // namespace

// SK x SN outputs of dW a workgroup (2 x SN / 64 waves), ROWS rows a step; GR: blockIdx.y is the
// expert. parts > 1: blockIdx.y is a part of the rows, whose fp32 sums go to part[y] (K x N).
template <int SK, int SN, int ROWS, int DT, int LOAD, bool GR>
__global__ __launch_bounds__(SN * 2) __attribute__((amdgpu_waves_per_eu(2))) void k_f8_wgrad(
    const uint8_t* __restrict__ qx, const uint8_t* __restrict__ sx, const void* __restrict__ dy,
    int64_t ld, int M, int K, int N, Route rt, OutY dw, int parts, float* __restrict__ part) {
  static_assert(LOAD != kStraight || DT == kBF16, "only operands go straight to LDS");
  constexpr int NT = SN * 2, NW = NT / kWave, WN = SN / 64, TERMS = terms_of(DT);
  constexpr int FK = SK / 2 / 32, FN = 2;             // 32 x 32 blocks of a wave
  constexpr int XROW = SK * 2, YROW = SN * 2, PANEL = ROWS * YROW;   // bytes
  constexpr int RX = NT / (SK / 16), RY = NT / (SN / 8);  // rows of a pass of the threads
  constexpr int PX = ROWS / RX, PY = ROWS / RY;       // passes: 16 codes, 8 elements of dy a thread
  constexpr int WY = DT == kF32 ? 8 : 4;              // words of these
  __shared__ __align__(16) uint8_t X0[ROWS * XROW];
  __shared__ __align__(16) uint8_t X1[ROWS * XROW];
  __shared__ __align__(16) uint8_t Y0[TERMS * PANEL];
  __shared__ __align__(16) uint8_t Y1[TERMS * PANEL];
  const int Kp = (K + kGroup - 1) / kGroup * kGroup;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = tid % kWave;
  const int ntk = (K + SK - 1) / SK, ntn = (N + SN - 1) / SN;
  int tk, tn, from = 0, to = M;
  tile_of(blockIdx.x, ntk, ntn, tk, tn);
  const int64_t Ms = GR ? rt.T : M;
  int64_t out0 = 0;
  if constexpr (GR) {
    from = clamp_route(rt.offs[blockIdx.y], 0, rt.R);
    to = clamp_route(rt.offs[blockIdx.y + 1], from, rt.R);
    out0 = (int64_t)blockIdx.y * K * N;
  } else if (parts > 1) {                             // whole steps to each part
    const int steps = (M + ROWS - 1) / ROWS;
    from = (int)((int64_t)blockIdx.y * steps / parts) * ROWS;
    to = std::min(M, (int)((int64_t)(blockIdx.y + 1) * steps / parts) * ROWS);
  }
  const int k0 = tk * SK, n0 = tn * SN;
  // a tile's columns of dy come in pieces of 8; one that reaches past the end of the row starts
  // earlier (its columns are then computed twice, alike)
  auto column = [&](int piece) {
    const int n = n0 + 8 * piece;
    return LOAD == kByElement || n + 8 <= N ? n : N - 8;
  };
  // 16-byte piece c of row m of a panel
  auto place = [&](int row, int m, int c) { return m * row + (c ^ (m % 4 * 4)) * 16; };

  // codes of this thread: rows mx + RX p, columns 16 cx ..
  const int mx = tid / (SK / 16), cx = tid % (SK / 16);
  const int kc = k0 + 16 * cx < Kp ? k0 + 16 * cx : Kp - 16;   // past the end: never stored
  const uint8_t* scol = sx + (int64_t)(kc / kGroup) * Ms;
  // elements of dy: rows my + RY p, piece cy
  const int my = tid / (SN / 8), cy = tid % (SN / 8);
  uint4 xr[PX];
  uint32_t sr[PX];
  int tok[PX];                                        // a step ahead of the codes
  uint32_t yr[PY][WY];
  auto load_tok = [&](int m) {
    if constexpr (GR) {
#pragma unroll
      for (int p = 0; p < PX; ++p) {
        const int r = m + mx + RX * p;
        tok[p] = clamp_route(rt.tok[r < to ? r : to - 1], 0, rt.T - 1);
      }
    }
  };
  auto load = [&](int m) {                            // rows from m on; past the end: the last
#pragma unroll
    for (int p = 0; p < PX; ++p) {
      const int r = m + mx + RX * p;
      const int64_t src = GR ? tok[p] : (r < to ? r : to - 1);
      xr[p] = *reinterpret_cast<const uint4*>(qx + src * Kp + kc);
      sr[p] = scol[src];
    }
    if constexpr (LOAD != kStraight) {
      constexpr int B = DT == kF32 ? 4 : 2;
#pragma unroll
      for (int p = 0; p < PY; ++p) {
        const int r = m + my + RY * p;
        const uint8_t* row = static_cast<const uint8_t*>(dy) + (int64_t)(r < to ? r : to - 1) * ld * B;
        if constexpr (LOAD == kByPiece) {
          __builtin_memcpy(yr[p], row + (int64_t)column(cy) * B, 8 * B);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int n = column(cy) + e < N ? column(cy) + e : N - 1;
            if constexpr (DT == kF32) yr[p][e] = reinterpret_cast<const uint32_t*>(row)[n];
            else {
              const uint32_t h = reinterpret_cast<const uint16_t*>(row)[n];
              yr[p][e / 2] = e % 2 ? yr[p][e / 2] | h << 16 : h;
            }
          }
        }
      }
    }
  };
  auto issue = [&](int m, uint8_t* Y) {               // rows from m on straight to the panel
    if constexpr (LOAD == kStraight) {
#pragma unroll
      for (int i = 0; i < PY; ++i) {
        const int at = i * NW + wave;                 // 1 KiB each
        const int r = at * (512 / SN) + lane / (SN / 8);
        const int c = lane % (SN / 8) ^ (r % 4 * 4);
        const uint16_t* src = static_cast<const uint16_t*>(dy) + (int64_t)(m + r) * ld + column(c);
        const void* p = m + r < to ? static_cast<const void*>(src) : &kZeroPiece;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                         (__attribute__((address_space(3))) void*)(Y + at * 1024), 16, 0, 0);
      }
    }
  };
  auto put = [&](int m, uint8_t* X, uint8_t* Y) {     // the loaded rows (from m on) as operands
#pragma unroll
    for (int p = 0; p < PX; ++p) {
      const int r = mx + RX * p;
      const bool live = m + r < to;
      const float scale = f8_scale(live ? sr[p] : 127u);
      const uint32_t c[4] = {xr[p].x, xr[p].y, xr[p].z, xr[p].w};
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = live ? sr[p] == kF8NanByte ? 0x7F7F7F7F : (int)c[i] : 0;
        w[2 * i] = __builtin_bit_cast(uint32_t, (v2b)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, false));
        w[2 * i + 1] = __builtin_bit_cast(uint32_t, (v2b)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, true));
      }
      *reinterpret_cast<uint4*>(X + place(XROW, r, 2 * cx)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(X + place(XROW, r, 2 * cx + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    if constexpr (LOAD != kStraight) {
#pragma unroll
      for (int p = 0; p < PY; ++p) {
        const int r = my + RY * p;
        const bool live = m + r < to;
        uint8_t* out = Y + place(YROW, r, cy);
        if constexpr (DT == kBF16) {
          *reinterpret_cast<uint4*>(out) = live ? make_uint4(yr[p][0], yr[p][1], yr[p][2], yr[p][3])
                                                : make_uint4(0, 0, 0, 0);
        } else {
          uint32_t w[TERMS][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a, b;
            if constexpr (DT == kF32) {
              a = __uint_as_float(yr[p][2 * i]);
              b = __uint_as_float(yr[p][2 * i + 1]);
            } else {
              const __half2 h = __builtin_bit_cast(__half2, yr[p][i]);
              a = __low2float(h);
              b = __high2float(h);
            }
            // a quiet NaN keeps its mark in the leading part; past an infinity nothing is left
            a = live ? __builtin_canonicalizef(a) : 0.0f;
            b = live ? __builtin_canonicalizef(b) : 0.0f;
            const bool fa = __builtin_isfinite(a), fb = __builtin_isfinite(b);
            w[0][i] = lead2(a, b);
            a = fa ? a : 0.0f;
            b = fb ? b : 0.0f;
#pragma unroll
            for (int t = 1; t < TERMS; ++t) w[t][i] = lead2(a, b);
          }
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
            *reinterpret_cast<uint4*>(out + t * PANEL) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        }
      }
    }
  };

  const int wk = wave / WN, wn = wave % WN;
  const int lr = lane % 32, hf = lane / 32;
  // block b of 32 columns of a panel: this lane's place in its first four rows
  auto corner = [&](int row, int b) {
    const int r = lane % 16 / 4, c = 2 * b + lane / 16 % 2;
    return (8 * hf + r) * row + (c ^ (2 * r)) * 32 + lane % 4 * 8;
  };
  int ca[FK], cb[FN];
#pragma unroll
  for (int i = 0; i < FK; ++i) ca[i] = corner(XROW, wk * FK + i);
#pragma unroll
  for (int j = 0; j < FN; ++j) cb[j] = corner(YROW, wn * FN + j);
  auto operand = [&](const uint8_t* P, int at, int row) {      // eight rows of this lane's column
    typedef __attribute__((address_space(3))) v4s* Ptr;
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(P + at));
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(P + at + 4 * row));
    return __builtin_bit_cast(v8b, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  v16f acc[FK][FN];
#pragma unroll
  for (int i = 0; i < FK; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v16f{0.0f};
  auto compute = [&](const uint8_t* X, const uint8_t* Y, int h0, int h1) {   // 16 rows each
#pragma unroll
    for (int h = h0; h < h1; ++h) {
      v8b a[FK];
#pragma unroll
      for (int i = 0; i < FK; ++i) a[i] = operand(X, ca[i] + 16 * h * XROW, XROW);
#pragma unroll
      for (int t = TERMS - 1; t >= 0; --t)            // the least term first
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v8b b = operand(Y, cb[j] + t * PANEL + 16 * h * YROW, YROW);
#pragma unroll
          for (int i = 0; i < FK; ++i)
            acc[i][j] = DT == kF32 ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b, acc[i][j], 0, 0, 0)
                                   : __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a[i], acc[i][j], 0, 0, 0);
        }
    }
  };
  if (from < to) {
    load_tok(from);
    load(from);
    load_tok(from + ROWS);
    issue(from, Y0);
    put(from, X0, Y0);
    load(from + ROWS);
    load_tok(from + 2 * ROWS);
    auto step = [&](int m, const uint8_t* X, const uint8_t* Y, uint8_t* Xn, uint8_t* Yn) {
      asm volatile("" ::: "memory");                  // the last step's reads stay ahead of their wait
      if constexpr (LOAD == kStraight) wait_vm<0>();  // step m's rows of dy landed
      wait_lds0();                                    // ... and are written
      lds_barrier();                                  // ... in every wave, and the others are read
      asm volatile("" ::: "memory");
      issue(m + ROWS, Yn);
      // a long step's codes are widened between its halves (8192 rows, 4096 x 4096 bf16: 240 us,
      // ahead of the step 267); a short one's ahead (fp32 646 us, between 660; fp16 415 and 424)
      constexpr int H = ROWS / 16, HALF = SK == 256 && ROWS == 64 ? H / 2 : 0;
      compute(X, Y, 0, HALF);
      put(m + ROWS, Xn, Yn);
      load(m + 2 * ROWS);
      load_tok(m + 3 * ROWS);
      if constexpr (HALF > 0) __builtin_amdgcn_sched_barrier(0);
      compute(X, Y, HALF, H);
    };
#pragma unroll 1
    for (int m = from; m < to; m += 2 * ROWS) {
      step(m, X0, Y0, X1, Y1);
      if (m + ROWS < to) step(m + ROWS, X1, Y1, X0, Y0);
    }
    if constexpr (LOAD == kStraight) wait_vm<0>();
  }
  float* const sums = !GR && parts > 1 ? part + (int64_t)blockIdx.y * K * N : nullptr;
  if constexpr (DT == kF32) {
    // lane: column n = lane % 32 of a block, rows k = 8 (r / 4) + 4 hf + r % 4
    float* const y = sums ? sums : static_cast<float*>(dw.p) + out0;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int pos = wn * 64 + 32 * j + lr, n = column(pos / 8) + pos % 8;
      if (n0 + pos / 8 * 8 >= N || n >= N) continue;
#pragma unroll
      for (int i = 0; i < FK; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int k = k0 + wk * (SK / 2) + 32 * i + 8 * (r / 4) + 4 * hf + r % 4;
          if (k < K) __builtin_nontemporal_store(acc[i][j][r], y + (int64_t)k * N + n);
        }
    }
  } else if (sums) {
    // lane: row k = lane % 32 of a block, columns n = 8 (r / 4) + 4 hf + r % 4
#pragma unroll
    for (int i = 0; i < FK; ++i) {
      const int k = k0 + wk * (SK / 2) + 32 * i + lr;
      if (k >= K) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int piece = wn * 8 + 4 * j + q, n = column(piece) + 4 * hf;
          if (n0 + 8 * piece >= N) continue;
          float* o = sums + (int64_t)k * N + n;
          const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if constexpr (LOAD == kByElement) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < N) o[e] = v[e];
          } else {
            __builtin_memcpy(o, v, 16);
          }
        }
    }
  } else {
    // through this wave's 4 KiB of LDS: 32 rows of 64 outputs, pieces swizzled by row
    __syncthreads();                                  // every wave is done with the panels
    uint8_t* const P = (wave % 4 == 0 ? X0 : wave % 4 == 1 ? X1 : wave % 4 == 2 ? Y0 : Y1) + wave / 4 * 4096;
    static_assert(PANEL >= (NW + 3) / 4 * 4096 && SK >= SN, "a wave's part fits");
    const bool vec = N % 8 == 0 && reinterpret_cast<uintptr_t>(dw.p) % 16 == 0;
    uint16_t* const y = static_cast<uint16_t*>(dw.p) + out0;
#pragma unroll
    for (int i = 0; i < FK; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(P + lr * 128 + ((4 * j + q) ^ (lr % 8)) * 16 + 8 * hf) =
              make_uint2(narrow2<DT>(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                         narrow2<DT>(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
      wave_exchange();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 8 * t + lane / 8, c = lane % 8;
        const uint4 v = *reinterpret_cast<const uint4*>(P + row * 128 + (c ^ (row % 8)) * 16);
        const int k = k0 + wk * (SK / 2) + 32 * i + row, n = column(wn * 8 + c);
        if (k >= K || n0 + 8 * (wn * 8 + c) >= N) continue;
        uint16_t* o = y + (int64_t)k * N + n;
        if (vec) {
          store_once(o, v);
        } else {
          const uint16_t* e = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (n + u < N) o[u] = e[u];
        }
      }
      wave_exchange();
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

// Tiles and parts. Large tiles (256 x 256 outputs; fp32 256 x 128, two workgroups a CU) once they
// fill the card's CUs and keep a few steps (us, large and 128 x 128: 8192 rows, 4096 x 4096 bf16 240
// and 300, fp16 437 and 538, fp32 668 and 844; 1024 rows, 4096 x 14336 bf16 143 and 147; 230 rows,
// 8192 x 5632 bf16 52 and 43, fp16 67 and 62, fp32 87 and 93; 4096 rows, 1024 x 4096, 64 tiles of
// 256 x 256: bf16 95 and 53, fp32 172 and 138). Small ones fill the card with parts of the rows
// while a part keeps 512.
struct Plan {
  bool large;
  int64_t tiles;
  int parts;
};
Plan wgrad_plan(int type, int64_t M, int64_t K, int64_t N, int64_t E) {
  auto tiles = [&](int64_t k, int64_t n) { return ((K + k - 1) / k) * ((N + n - 1) / n); };
  const int64_t cus = device_cus(), rows = E > 0 ? M / E : M, times = E > 0 ? E : 1;
  const int64_t wide = type == kF32 ? 128 : 256;
  if (N >= 8 && tiles(256, 256) * times >= cus * 3 / 4 && rows >= (type == kF32 ? 128 : 512))
    return {true, tiles(256, wide), 1};
  Plan p{false, tiles(128, 128), 1};
  while (E == 0 && p.tiles * p.parts * 2 <= 2 * cus && M / (2 * p.parts) >= 512) p.parts *= 2;
  return p;
}

template <int SK, int SN, int ROWS, int DT, int LOAD, bool GR>
hipError_t wgrad_t(const Plan& p, const uint8_t* qx, const uint8_t* sx, const void* dy, int64_t ld, int64_t M,
                   int64_t K, int64_t N, const Route& rt, OutY dw, float* ws, hipStream_t stream) {
  if (!grid_fits(p.tiles, SN * 2) || (p.parts > 1 && !grid_fits((K * N + 255) / 256, 256)))
    return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_f8_wgrad<SK, SN, ROWS, DT, LOAD, GR>),
                     dim3((unsigned)p.tiles, (unsigned)(GR ? rt.E : p.parts)), dim3(SN * 2), 0, stream, qx, sx,
                     dy, ld, (int)M, (int)K, (int)N, rt, dw, p.parts, ws);
  if (p.parts > 1)
    hipLaunchKernelGGL(k_f8_wgrad_join, dim3((unsigned)((K * N + 255) / 256)), dim3(256), 0, stream,
                       ws, p.parts, K * N, dw);
  return hipGetLastError();
}

template <int DT, bool GR>
hipError_t wgrad_d(const uint8_t* qx, const uint8_t* sx, const void* dy, int64_t ld, int64_t M, int64_t K,
                   int64_t N, const Route& rt, OutY dw, float* ws, hipStream_t stream) {
  const Plan p = wgrad_plan(DT, GR ? rt.R : M, K, N, rt.E);
#define BGT_CALL(SK, SN, ROWS, LOAD) \
  return wgrad_t<SK, SN, ROWS, DT, LOAD, GR>(p, qx, sx, dy, ld, M, K, N, rt, dw, ws, stream)
  if (N < 8) BGT_CALL(128, 128, 32, kByElement);
  if constexpr (DT == kBF16) {
    if (N % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(dy) % 16 == 0) {
      if (p.large) BGT_CALL(256, 256, 64, kStraight);
      // two workgroups a CU hide less of a step's latency than four (256 tiles, 4096 rows: 53 us with
      // steps of 64 rows, 75 with 32), which need the shorter step (2816 tiles, 230 rows: 54 and 43)
      if (p.tiles * p.parts * (GR ? rt.E : 1) <= 2 * device_cus()) BGT_CALL(128, 128, 64, kStraight);
      BGT_CALL(128, 128, 32, kStraight);
    }
  }
  if (p.large) BGT_CALL(256, (DT == kF32 ? 128 : 256), 32, kByPiece);
  BGT_CALL(128, 128, 32, kByPiece);
#undef BGT_CALL
}

}  // namespace

int64_t f8_wgrad_ws_bytes(int64_t M, int64_t K, int64_t N) {
  const int parts = wgrad_plan(kF32, M, K, N, 0).parts;   // of rows enough for parts: every type's
  return parts > 1 ? (int64_t)parts * K * N * 4 : 0;
}

hipError_t launch_f8_wgrad(const uint8_t* qx, const uint8_t* sx, const void* dy, int64_t ld,
                           int64_t M, int64_t K, int64_t N, const Route& rt, OutY dw, void* ws,
                           hipStream_t stream) {
  float* p = static_cast<float*>(ws);
#define BGT_CALL(T)                                                              \
  return rt.E > 0 ? wgrad_d<T, true>(qx, sx, dy, ld, M, K, N, rt, dw, p, stream) \
                  : wgrad_d<T, false>(qx, sx, dy, ld, M, K, N, rt, dw, p, stream)
  if (dw.type == kF32) BGT_CALL(kF32);
  if (dw.type == kF16) BGT_CALL(kF16);
  BGT_CALL(kBF16);
#undef BGT_CALL
}

}  // namespace bgt
