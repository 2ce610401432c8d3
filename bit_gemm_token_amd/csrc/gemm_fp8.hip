// gemm_fp8.hip -- products of rows and weights held in 8 bits (gfx950).
//
//     y_mn = sum_g 2^(a_gm + b_gn) sum_{k in g} qx_mk qw_nk,      g: blocks of 128 k
//
// with e4m3 codes qx (M x K'), qw (N x K') and exponent bytes a (K'/128 x M), b (K'/128 x
// N'/128). The matrix instructions for 8-bit floats take an exponent byte for every lane's 32 k
// of either operand, so the blocks' scales cost no vector instruction and the sums stay in
// one fp32 accumulator. The same instruction aligns the products of eight k to the largest of them
// and cuts off what lies more than 13 bits below that one's leading bit (measured: of 2^16 + 2^3 in
// one group of k both are kept, + 2^2 is lost, of either sign), less than 7 * 2^-13 < 2^-10 of the
// magnitudes that a sum adds up.
// Measured besides the rounding: 1.8e-5 of the outputs' norm for normal rows and weights, 4.7e-5 for
// rows with channels twenty times as large. That is a hundredth and a thirtieth of a bf16 output's
// rounding error and a tenth and a quarter of an fp16 one's, but a sum whose large products cancel is
// left with it, and it is too much for fp32. Outputs in fp32, and those of few rows where the stream
// of weights hides it, therefore take bf16 products of the same codes (e4m3 is exact in bf16, the
// products exact in fp32, four instructions in place of one), with the sum of the two exponents
// applied to a group's fp32 sum at once: one alone may take it out of range (rows of 2^118 by weights
// of 2^-20).
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

// Rows past the last expert's are zero: workgroup z of nz clears its share, 16 bytes a lane at the
// element's alignment; a last, partial piece is a whole one moved back to end with them. (4096 tokens,
// 2 of 8 experts, 1024 into 14336 bf16, seven eighths dropped: 78 us, 333 an element a lane.)
__device__ __forceinline__ void zero_rows(const Route& rt, int N, OutY y, int z, int nz) {
  typedef uint32_t Piece __attribute__((ext_vector_type(4), aligned(2)));
  const int b = y.type == kF32 ? 4 : 2;
  const int64_t from = (int64_t)clamp_route(rt.offs[rt.E], 0, rt.R) * N, n = ((int64_t)rt.R * N - from) * b;
  const int64_t at = (int64_t)z * blockDim.x + threadIdx.x;
  if (n >= 16) {
    char* const tail = static_cast<char*>(y.p) + from * b;
    for (int64_t o = 16 * at; o < n; o += (int64_t)nz * blockDim.x * 16)
      *reinterpret_cast<Piece*>(tail + std::min(o, n - 16)) = Piece{};
  } else if (at * b < n) {
    y.put(from + at, 0.0f);
  }
}
constexpr int kZeroWgs = 64;
constexpr int kFusedRows = 8;                         // rows quantized by the product itself

// waves of a streaming workgroup at most: sixteen of 128 registers, or eight of 256 for 64 rows,
// whose fragments take 32 registers a group, and for chunks, whose next part of x takes as many
// again (64 rows of exact products by expert spill 44)
constexpr int stream_waves(int mt, bool ch) { return mt == 4 || ch ? 8 : 16; }

// blocks of bm rows of all experts' slots
__device__ __forceinline__ int route_blocks(const Route& rt, int bm) {
  int n = 0;
  for (int base = 0; base < rt.E; base += kWave)
    n += wave_sum(expert_row_tiles(rt, base + (int)threadIdx.x % kWave, bm));
  return __builtin_amdgcn_readfirstlane(n);
}
// block b of them: its expert e, that one's first slot a and slots, and the block tm within
__device__ __forceinline__ void route_block(const Route& rt, int bm, int b, int& e, int& a, int& rows,
                                            int& tm) {
  const int lane = threadIdx.x % kWave;
  for (int base = 0; base < rt.E; base += kWave) {
    const int nt = expert_row_tiles(rt, base + lane, bm);
    int incl = nt;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    const unsigned long long hit = __ballot(b >= incl - nt && b < incl);
    if (hit != 0ull) {
      const int l = (int)__builtin_ctzll(hit);
      e = __builtin_amdgcn_readfirstlane(base + l);
      tm = __builtin_amdgcn_readfirstlane(b - __shfl(incl - nt, l, kWave));
      a = clamp_route(rt.offs[e], 0, rt.R);
      rows = clamp_route(rt.offs[e + 1], a, rt.R) - a;
      return;
    }
    b -= __builtin_amdgcn_readfirstlane(__shfl(incl, kWave - 1, kWave));
  }
  e = a = rows = tm = 0;                              // no such block
}

}  // namespace

// =====================================================================
// Few rows: the weights stream once through registers
// =====================================================================
// An item is 16 weight rows (outputs n) for one block of 16 MT rows of x. A workgroup takes a run
// of items, weight rows innermost; its KS waves share the groups of K, GPW of each at a time.
//   CH false  KS * GPW groups are all of K: a wave keeps its groups' fragments of x in
//             registers over the run, so x is read once a workgroup, not once an item
//   CH true   longer K: chunks of KS * GPW groups, each with its part of x
// The next step's weights (and part of x) are on their way in registers. The waves' sums meet in
// LDS (two buffers, one barrier an item) in wave order; an output is stored one item late,
// before new loads are issued, so that no wait for loads waits for a store too.
//
// Of x whole 128-byte pieces of rows are loaded (reading 64 bytes of 16 rows an instruction, as
// the fragments lie, took 6.2 us more than an empty launch for 64 rows x 4096 in every workgroup,
// this 1.8) and become fragments by way of the wave's own LDS, 16-byte pieces XOR-swizzled by
// row.
// XT >= 0 (at most kFusedRows rows, CH false): x comes as elements of that type and every wave turns
// its own groups' blocks into codes (a block's scale needs no other wave); the workgroup of the first
// item writes codes and scales out. The elements are requested ahead of the weights and are codes by
// the time these arrive (1 x 4096 into 4096: 7.7 us behind them).
template <int MT, int GPW, bool CH, bool EX, int XT, bool GR>
__global__ __launch_bounds__(stream_waves(MT, CH) * 64) void k_f8_stream(
    const void* __restrict__ x, int64_t ldx, int Kx, const uint8_t* __restrict__ sx,
    const uint8_t* __restrict__ qw, const uint8_t* __restrict__ sw, int M, int N, int K, OutY y,
    Route rt, uint8_t* __restrict__ q_out, uint8_t* __restrict__ s_out) {
  constexpr int MOST = stream_waves(MT, CH);
  static_assert(XT < 0 || (MT == 1 && !CH), "a wave quantizes the x that it keeps");
  __shared__ float red[2][MOST * MT * 4 * 64];
  __shared__ __align__(16) uint8_t turn[MOST * MT * 2048];
  const int G = K / kGroup, B = (N + kGroup - 1) / kGroup;
  const int KS = blockDim.x / kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const int c = lane % 16, s4 = lane / 16;
  const int ntn = (N + 15) / 16;
  const int main_wgs = (int)gridDim.x - (GR ? kZeroWgs : 0);
  if (GR && (int)blockIdx.x >= main_wgs) {
    zero_rows(rt, N, y, blockIdx.x - main_wgs, kZeroWgs);
    return;
  }
  // 32-bit divisions, and none where there is nothing to divide: they precede the first load
  const uint32_t wg = blockIdx.x, wgs = (uint32_t)main_wgs;
  const uint32_t blocks = GR ? route_blocks(rt, 16 * MT) : (M + 16 * MT - 1) / (16 * MT);
  const uint32_t total = blocks * (uint32_t)ntn;
  uint32_t item = wg, last = wg + 1;
  if (total != wgs) {                                 // an equal run each, one more for the first
    const uint32_t each = total / wgs, more = total - each * wgs;
    item = wg * each + (wg < more ? wg : more);
    last = item + each + (wg < more ? 1 : 0);
  }
  if (item >= last) return;
  int rb = 0, tn = (int)item;
  if (blocks > 1) {
    rb = (int)(item / (uint32_t)ntn);
    tn = (int)(item - (uint32_t)rb * ntn);
  }
  const int chunks = CH ? (G + KS * GPW - 1) / (KS * GPW) : 1;
  const int64_t Ms = GR ? rt.T : M;

  // a block of rows: its expert, first slot (r0), row within (m0), rows of the expert
  struct Block {
    int e, r0, rows, m0;
  };
  auto locate = [&](int b) {
    Block k{0, 0, M, b * 16 * MT};
    if constexpr (GR) {
      int tm;
      route_block(rt, 16 * MT, b, k.e, k.r0, k.rows, tm);
      k.m0 = tm * 16 * MT;
    }
    return k;
  };
  Block at = locate(rb);

  // what is requested next: an item and, of long K, a chunk
  uint32_t fitem = item;
  int frb = rb, ftn = tn, fch = 0;
  Block fat = at;
  // rows of x as loaded (16 i + 8 h + lane / 8; -1: none) and of the scales (16 i + c)
  int xrow[MT][2], srow[MT];
  auto find_rows = [&](const Block& k) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = k.m0 + 16 * i + 8 * h + lane / 8;
        xrow[i][h] = m >= k.rows ? -1 : GR ? clamp_route(rt.tok[k.r0 + m], 0, rt.T - 1) : m;
      }
      const int m = k.m0 + 16 * i + c < k.rows ? k.m0 + 16 * i + c : k.rows - 1;
      srow[i] = GR ? clamp_route(rt.tok[k.r0 + m], 0, rt.T - 1) : m;
    }
  };
  uint4 wb[GPW][2], raw[GPW][MT][2];
  uint32_t sb[GPW], sxb[GPW][MT], sraw[GPW][MT];
  v8i xc[GPW][MT];
  constexpr bool WIDE = EX && !CH && MT == 1;         // x is kept widened, before the weights arrive
  v8b xw[WIDE ? GPW : 1][4];
  auto widen_x = [&](int j) {
    if constexpr (WIDE) {
#pragma unroll
      for (int u = 0; u < 4; ++u) xw[j][u] = widen8(xc[j][0], u);
    }
  };
  auto load_raw = [&](int ch) {
#pragma unroll
    for (int j = 0; j < GPW; ++j) {
      const int g = (ch * GPW + j) * KS + wave;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          raw[j][i][h] = make_uint4(0, 0, 0, 0);
          if (xrow[i][h] >= 0 && g < G)
            raw[j][i][h] = *reinterpret_cast<const uint4*>(
                static_cast<const uint8_t*>(x) + (int64_t)xrow[i][h] * K + (int64_t)g * kGroup + lane % 8 * 16);
        }
        sraw[j][i] = sx[(int64_t)(g < G ? g : G - 1) * Ms + srow[i]];
      }
    }
  };
  // loads of weights are unconditional, so that they go to the registers the last step used up
  // without copies: past the run's end all lanes read the weights' first bytes
  auto fetch = [&]() {
    const bool more = fitem < last;
    const int n = 16 * ftn + c;
    const uint8_t* p = qw + (GR ? fat.e * rt.wstride : 0);
    const uint8_t* ps = sw + (GR ? fat.e * rt.sstride : 0);
    p += more ? (int64_t)(n < N ? n : N - 1) * K + 16 * s4 : 0;
    ps += more ? ftn / 8 : 0;
#pragma unroll
    for (int j = 0; j < GPW; ++j) {
      // past the wave's groups: the last group again, which meets zero codes of x
      int g = (fch * GPW + j) * KS + wave;
      g = !more ? 0 : g < G ? g : G - 1;
      sb[j] = ps[(int64_t)g * B];
      wb[j][0] = *reinterpret_cast<const uint4*>(p + (int64_t)g * kGroup);
      wb[j][1] = *reinterpret_cast<const uint4*>(p + (int64_t)g * kGroup + 64);
    }
    if constexpr (CH)
      if (more) load_raw(fch);
    if (CH && ++fch < chunks) return;
    fch = 0;
    if (++fitem < last && ++ftn == ntn) {
      ftn = 0;
      fat = locate(++frb);
      if constexpr (CH) find_rows(fat);
    }
  };
  uint8_t* mine = turn + wave * MT * 2048;
  auto place = [](int row, int piece) { return row * 128 + 16 * (piece ^ ((row >> 1) & 7)); };
  auto read_x = [&](const uint8_t* p) {
    return join(*reinterpret_cast<const uint4*>(p + place(c, s4)),
                *reinterpret_cast<const uint4*>(p + place(c, s4 + 4)));
  };
  auto turn_x = [&]() {                               // raw -> fragments
#pragma unroll
    for (int j = 0; j < GPW; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint4*>(mine + i * 2048 + place(8 * h + lane / 8, lane % 8)) = raw[j][i][h];
        sxb[j][i] = sraw[j][i];
      }
      wave_exchange();
#pragma unroll
      for (int i = 0; i < MT; ++i) xc[j][i] = read_x(mine + i * 2048);
      widen_x(j);
      wave_exchange();                                // the next group takes the same place
    }
  };
  // elements: rows 4 r + lane / 16, eight a lane, a block in 16 lanes
  constexpr int XR = XT >= 0 ? kFusedRows / 4 : 1;
  float xv[XT >= 0 ? GPW : 1][XR][8];
  auto load_x = [&]() {
    if constexpr (XT >= 0) {
#pragma unroll
      for (int j = 0; j < GPW; ++j)
#pragma unroll
        for (int r = 0; r < XR; ++r) {
          const int g = j * KS + wave, row = 4 * r + s4, k = g * kGroup + 8 * c;
#pragma unroll
          for (int u = 0; u < 8; ++u) xv[j][r][u] = 0.0f;
          if (row < M && g < G && k < Kx) load8<XT>(x, row * ldx + k, xv[j][r]);
        }
    }
  };
  auto quantize_x = [&](bool write) {
    if constexpr (XT >= 0) {
#pragma unroll
      for (int j = 0; j < GPW; ++j) {
        const int g = j * KS + wave;
        sxb[j][0] = 127;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 4 * r + s4, k = g * kGroup + 8 * c;
          uint32_t byte = 127;
          uint2 q = make_uint2(0, 0);
          if (r < XR && 4 * r < M) {                  // uniform
            const float* const v = xv[j][r < XR ? r : 0];
            uint32_t top = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) top = umax(top, abs_bits(v[u]));
            byte = f8_scale_byte(max16(top));
            const float scale = f8_scale(byte);
            q.x = f8_pack4(v[0], v[1], v[2], v[3], scale);
            q.y = f8_pack4(v[4], v[5], v[6], v[7], scale);
            if (write && row < M && g < G) {
              *reinterpret_cast<uint2*>(q_out + (int64_t)row * K + k) = q;
              if (c == 0) s_out[(int64_t)g * M + row] = (uint8_t)byte;
            }
          }
          *reinterpret_cast<uint2*>(mine + place(row, c / 2) + c % 2 * 8) = q;
          // lane (c, s4) wants the byte of row c = 4 r + s: it lies in lanes 16 s ..
          const uint32_t of = (uint32_t)__shfl((int)byte, c % 4 * 16, kWave);
          if (c / 4 == r) sxb[j][0] = of;
        }
        wave_exchange();
        xc[j][0] = read_x(mine);
        widen_x(j);
        wave_exchange();
      }
    }
  };

  find_rows(at);
  if constexpr (XT >= 0) load_x();
  else if constexpr (!CH) load_raw(0);
  fetch();
  if constexpr (XT >= 0) quantize_x(item == 0);
  else if constexpr (!CH) turn_x();
  const bool single = (int)blockDim.x >= MT * 256;    // an output of an item a thread at most
  int buf = 0;
  int64_t late = -1;                                  // place and value of the output to store
  float value = 0.0f;
  auto sum = [&](int t, int64_t& o, float& v) {       // output t of the item over the waves
    const int n = t % 16, m = t / 16;
    const int of = (m / 16 * 4 + n % 4) * 64 + n / 4 * 16 + m % 16;
    if (at.m0 + m >= at.rows || 16 * tn + n >= N) return;
    v = 0.0f;
    if (KS == MOST) {                                 // all reads at once
#pragma unroll
      for (int w = 0; w < MOST; ++w) v += red[buf][w * MT * 256 + of];
    } else {
      for (int w = 0; w < KS; ++w) v += red[buf][w * MT * 256 + of];
    }
    o = (int64_t)(at.r0 + at.m0 + m) * N + 16 * tn + n;
  };
#pragma unroll 1
  while (item < last) {
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t worst[MT] = {};                          // of the exponent bytes: 255 makes the sum NaN
#pragma unroll 1
    for (int ch = 0; ch < chunks; ++ch) {
      if constexpr (CH) turn_x();
#pragma unroll
      for (int j = 0; j < GPW; ++j) {
        const v8i w = join(wb[j][0], wb[j][1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (EX) {
            v4f p = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w, u), WIDE ? xw[WIDE ? j : 0][u] : widen8(xc[j][m], u),
                                                          p, 0, 0, 0);
            const int e = (int)(sxb[j][m] + sb[j]) - 254;
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][r] = acc[m][r] + __builtin_ldexpf(p[r], e);
            worst[m] = umax(worst[m], umax(sxb[j][m], sb[j]));
          } else {
            acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, xc[j][m], acc[m], 0, 0, 0,
                                                                      (int)sb[j], 0, (int)sxb[j][m]);
          }
        }
      }
      if (late >= 0) y.put(late, value);
      late = -1;
      fetch();
    }
    // lane: row m = 16 mt + lane % 16, outputs n = 4 (lane / 16) + r
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[buf][(wave * MT * 4 + m * 4 + r) * 64 + lane] = EX && worst[m] == kF8NanByte ? kF8Nan : acc[m][r];
    }
    __syncthreads();
    if (single) {
      if ((int)threadIdx.x < MT * 256) sum(threadIdx.x, late, value);
    } else {
      for (int t = threadIdx.x; t < MT * 256; t += blockDim.x) {
        int64_t o = -1;
        float v = 0.0f;
        sum(t, o, v);
        if (o >= 0) y.put(o, v);
      }
    }
    buf ^= 1;
    if (++item < last && ++tn == ntn) {
      tn = 0;
      at = locate(++rb);
      if constexpr (!CH && XT < 0) {
        find_rows(at);
        load_raw(0);
        turn_x();
      }
    }
  }
  if (late >= 0) y.put(late, value);
}

template <bool B, class T, class F> struct Pick { using type = T; };
template <class T, class F> struct Pick<false, T, F> { using type = F; };

// =====================================================================
// Many rows: BN x BM output tiles through LDS
// =====================================================================
// WN x WM waves of 32 x 32 blocks (v_mfma_scale_f32_32x32x64_f8f6f4, weights as the first
// operand: a lane then holds runs of four outputs n of one row m). One step is one group of
// 128 k: BN weight rows and BM rows of x of 128 bytes each, copied straight into LDS
// (16-byte pieces XOR-swizzled by row, so that the 32 rows of an operand read fall on
// distinct banks), two stages, one barrier a step. 16-bit outputs leave through the stages'
// LDS as whole rows.
//
// The 256 x 256 tile reads the operands of 64 k while those of the 64 before them are multiplied
// (two sets of registers), so that a group's two LDS reads and its copies run under the products;
// its copies are 32-bit offsets from one base in scalar registers, for want of vector registers
// (8192 x 14336 into 4096: 391 us, 425 without; 8192^3 467 and 474). Smaller tiles lose by it
// (128 x 128, 8192^3: 576 and 532): more workgroups a CU do the same for them. Its 256 registers
// spill one or two. fp32: eight waves of at most 128 registers, so that two workgroups share a CU.
template <int BN, int BM, int WN, int WM, bool EX, bool GR>
__global__ __launch_bounds__(WN * WM * 64) __attribute__((amdgpu_waves_per_eu(EX ? 4 : 2))) void k_f8_tile(
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
  constexpr bool HALVES = BN == 256;
  const uint8_t* const wbase = qw + (int64_t)n0 * K;
  const uint8_t* const xbase = qx + (GR ? 0 : (int64_t)m0 * K);
  typename Pick<HALVES, uint32_t, int64_t>::type wofs[WCP], xofs[XCP];   // a CU's rows, or T x K, below 2^32
#pragma unroll
  for (int i = 0; i < WCP; ++i) {
    const int r = 8 * (NW * i + wave) + lane / 8;
    wofs[i] = (int64_t)(n0 + r < N ? r : N - 1 - n0) * K + 16 * ((lane % 8) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int i = 0; i < XCP; ++i) {
    const int r = 8 * (NW * i + wave) + lane / 8;
    xofs[i] = (source_row(r) - (GR ? 0 : m0)) * K + 16 * ((lane % 8) ^ ((r >> 1) & 7));
  }
  auto copy = [&](const uint8_t* base, auto ofs, int g, uint8_t* to) {   // 1 KiB a wave
    auto* const l = (__attribute__((address_space(3))) void*)to;
    if constexpr (HALVES)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, -1, 0x27000), l, 16, (int)ofs,
          g * kGroup, 0, 0);
    else
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(base + ofs + (int64_t)g * kGroup), l, 16, 0, 0);
  };
  auto issue = [&](int g, uint8_t* S) {
#pragma unroll
    for (int i = 0; i < WCP; ++i) copy(wbase, wofs[i], g, S + (NW * i + wave) * 1024);
#pragma unroll
    for (int i = 0; i < XCP; ++i) copy(xbase, xofs[i], g, S + BN * kGroup + (NW * i + wave) * 1024);
  };
  // fp32: a wave whose rows all lie past the end only copies (a branch that 16-bit outputs' shorter
  // steps lose more by: 1024 x 4096 into 4096 36 us, 28 without)
  const bool idle = EX && m0 + wm * (BM / WM) >= M;
  const int64_t Ms = GR ? rt.T : M;
  int ssrc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) ssrc[i] = (int)source_row(wm * (BM / WM) + 32 * i + lr);
  const int nb = (n0 + wn * (BN / WN)) / kGroup;
  const uint8_t* wscale = sw + (nb < B ? nb : B - 1);
  uint32_t sa[FM], sb, na[FM], nb1;
  auto scales = [&](int g) {
    nb1 = wscale[(int64_t)g * B];
    const uint8_t* const sg = sx + (int64_t)g * Ms;
#pragma unroll
    for (int i = 0; i < FM; ++i) na[i] = sg[ssrc[i]];
  };
  auto take_scales = [&] {
    sb = nb1;
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = na[i];
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
  auto read = [&](const uint8_t* S, int h, v8i* w, v8i* xx) {  // operands of 64 k
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = fragment(S, wn * (BN / WN) + 32 * i + lr, h);
#pragma unroll
    for (int m = 0; m < FM; ++m) xx[m] = fragment(S + BN * kGroup, wm * (BM / WM) + 32 * m + lr, h);
  };
  uint32_t worst[FM] = {};                             // fp32: of the exponent bytes, 255 makes the sum NaN
  auto multiply = [&](const v8i* w, const v8i* xx) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int m = 0; m < FM; ++m)
        acc[i][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[i], xx[m], acc[i][m], 0, 0, 0,
                                                                    (int)sb, 0, (int)sa[m]);
  };
  scales(0);
  issue(0, S0);
  if constexpr (HALVES) {
    v8i wa[FN], xa[FM], wb[FN], xb[FM];
    auto step = [&](int g, uint8_t* cur, uint8_t* nxt) {
      take_scales();
      scales(g + 1 < G ? g + 1 : G - 1);
      read(cur, 1, wb, xb);
      multiply(wa, xa);
      __builtin_amdgcn_sched_barrier(0);
      wait_lds0();                                    // cur is read, and group g + 1 landed
      wait_vm<0>();
      asm volatile("" ::: "memory");
      lds_barrier();                                  // ... in every wave
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      issue(g + 2 < G ? g + 2 : G - 1, cur);          // past the end: never read
      read(nxt, 0, wa, xa);
      multiply(wb, xb);
      __builtin_amdgcn_sched_barrier(0);
    };
    issue(G > 1 ? 1 : 0, S1);
    wait_vm<0>();
    asm volatile("" ::: "memory");
    lds_barrier();
    asm volatile("" ::: "memory");
    read(S0, 0, wa, xa);
#pragma unroll 1
    for (int g = 0; g < G; g += 2) {
      step(g, S0, S1);
      if (g + 1 < G) step(g + 1, S1, S0);
    }
    wait_vm<0>();
  } else {
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
            const int e = (int)(sa[m] + sb) - 254;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][m][r] = acc[i][m][r] + __builtin_ldexpf(p[r], e);
            worst[m] = umax(worst[m], umax(sa[m], sb));
          }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v8i w[FN], xx[FM];
          read(S, h, w, xx);
          multiply(w, xx);
        }
      }
    };
    auto step = [&](int g, uint8_t* cur, uint8_t* nxt) {
      wait_vm<0>();                                   // group g and its scales landed
      lds_barrier();                                  // ... in every wave, and nxt is read
      asm volatile("" ::: "memory");
      take_scales();
      if (g + 1 < G) {
        scales(g + 1);
        issue(g + 1, nxt);
      }
      if (!idle) compute(cur);
      asm volatile("" ::: "memory");                  // the reads stay ahead of their wait
      wait_lds0();
    };
#pragma unroll 1
    for (int g = 0; g < G; g += 2) {
      step(g, S0, S1);
      if (g + 1 < G) step(g + 1, S1, S0);
    }
  }

  if constexpr (EX) {                                 // fp32: runs of four outputs a lane
    const bool vec = N % 4 == 0 && reinterpret_cast<uintptr_t>(y.p) % 16 == 0;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int row = m0 + wm * (BM / WM) + 32 * m + lr;
        if (row >= M) continue;
        if (worst[m] == kF8NanByte) acc[i][m] = v16f{} + kF8Nan;
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
  constexpr int PIECES = BN / 8, SWZ = (PIECES < 16 ? PIECES : 16) - 1;
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
        *reinterpret_cast<uint2*>(p + 16 * (piece ^ (r & SWZ)) + 8 * hf) = w;
      }
    }
  __syncthreads();
  const bool vec = N % 8 == 0 && reinterpret_cast<uintptr_t>(y.p) % 16 == 0;
  uint16_t* yp = static_cast<uint16_t*>(y.p);
  // 128 MB and more of outputs are stored past the L2 and leave the rows and weights there that tiles
  // share. What the product gains its output's reader loses where it comes at once, and does not where
  // other calls come first (us, past the L2 and not): 8192 x 4096 into 8192, 128 MB: the product alone 229
  // and 248, with the quantization of its output after it 295 and 284, a feed-forward of two such
  // products, the gate and the product back 835 and 831; into 11008, 172 MB: 319 and 360, 413 and 408, 1149
  // and 1160; into 14336, 224 MB: 392 and 432, 487 and 491, 1391 and 1426. Below there is little either way (64
  // MB: 117 and 117, 138 and 141).
  const bool past = (int64_t)(GR ? rt.R : M) * N >= 1 << 26;
#pragma unroll 4
  for (int t = tid; t < BM * PIECES; t += NW * 64) {
    const int r = t / PIECES, piece = t % PIECES;
    const uint8_t* p = (r < RPS ? S0 : S1) + (r < RPS ? r : r - RPS) * (2 * BN) + 16 * (piece ^ (r & SWZ));
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const int n = n0 + 8 * piece;
    if (m0 + r >= M || n >= N) continue;
    uint16_t* o = yp + (int64_t)(r0 + m0 + r) * N + n;
    if (vec) {
      if (past) store_once(o, v);
      else *reinterpret_cast<uint4*>(o) = v;
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

// waves: as many as the groups; workgroups: as many as give a CU 16 waves (8 for 64 rows: registers),
// no more than items (of a route: than its slots may need). LDS is that of the most waves whatever
// their number: two workgroups of 16 rows fit a CU at once, one of 32 and 64 rows, so that those of
// few groups (below 8 and 16) follow one another with fewer waves. Without `run`, here and below: only
// whether the launch is within the grid's limits.
template <int MT, int GPW, bool CH, bool EX, int XT, bool GR>
hipError_t stream_t(const void* x, int64_t ldx, int64_t Kx, const uint8_t* sx, const uint8_t* qw,
                    const uint8_t* sw, int64_t M, int64_t N, int64_t K, OutY y, const Route& rt,
                    uint8_t* q_out, uint8_t* s_out, hipStream_t stream, bool run = true) {
  const int64_t G = K / kGroup;
  int waves = 1;
  while (waves < stream_waves(MT, CH) && waves < G) waves *= 2;
  const int64_t blocks = GR ? rt.R / (16 * MT) + std::min<int64_t>(rt.E, rt.R) : (M + 16 * MT - 1) / (16 * MT);
  const int64_t items = blocks * ((N + 15) / 16);
  const int64_t wgs = std::min<int64_t>(items, device_cus() * ((MT == 4 ? 8 : 16) / waves)) + (GR ? kZeroWgs : 0);
  if (items > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  if (!run) return hipSuccess;
  hipLaunchKernelGGL((k_f8_stream<MT, GPW, CH, EX, XT, GR>), dim3((unsigned)wgs), dim3(waves * kWave), 0,
                     stream, x, ldx, (int)Kx, sx, qw, sw, (int)M, (int)N, (int)K, y, rt, q_out, s_out);
  return hipGetLastError();
}

constexpr int kStreamGroups = 32;                     // groups of K whose x the waves keep
constexpr int kStreamRows = 64;                       // rows of a matrix that this kernel takes

template <bool EX, bool GR>
hipError_t stream_rows(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                       int64_t M, int64_t N, int64_t K, OutY y, const Route& rt, int64_t per,
                       hipStream_t stream, bool run) {
  const bool all = K <= kStreamGroups * kGroup;       // 16 waves of 2 groups, 8 of 4
  // experts' slots scatter about their mean, and one past the block reads its weights again
  if (GR) per += per / 2;
#define BGT_STREAM(MT, GPW, CH, EXACT) \
  return stream_t<MT, GPW, CH, EXACT, -1, GR>(qx, K, K, sx, qw, sw, M, N, K, y, rt, nullptr, nullptr, stream, run)
  // 16-bit outputs too take exact products where the weights' stream hides them (us, exact and by the
  // 8-bit instructions): 1 / 16 / 32 rows x 4096 into 22016 20.4 / 21.8 / 25.5 and 20.7 / 22.1 / 24.7; not 61
  // rows, 34.1 and 28.2, nor longer K, 1 x 14336 into 4096 16.9 and 15.1
  if (per <= 16) {
    if (all) BGT_STREAM(1, 2, false, true);
    BGT_STREAM(1, 2, true, EX);
  }
  if (per <= 32) {
    if (all) BGT_STREAM(2, 2, false, true);
    BGT_STREAM(2, 2, true, EX);
  }
  if (all) BGT_STREAM(4, 4, false, EX);
  BGT_STREAM(4, 2, true, EX);
#undef BGT_STREAM
}

template <int BN, int BM, int WN, int WM, bool EX, bool GR>
hipError_t tile_t(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw, int64_t M,
            int64_t N, int64_t K, OutY y, const Route& rt, hipStream_t stream, bool run) {
  const int64_t ntn = (N + BN - 1) / BN;
  const int64_t wgs = GR ? (rt.R / BM + std::min<int64_t>(rt.E, rt.R)) * ntn + kZeroWgs
                         : (M + BM - 1) / BM * ntn;
  if (!grid_fits(wgs, WN * WM * 64)) return hipErrorInvalidConfiguration;
  if (!run) return hipSuccess;
  hipLaunchKernelGGL((k_f8_tile<BN, BM, WN, WM, EX, GR>), dim3((unsigned)wgs), dim3(WN * WM * 64), 0,
                     stream, qx, sx, qw, sw, (int)M, (int)N, (int)K, y, rt);
  return hipGetLastError();
}

template <bool GR>
hipError_t launch_t(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                    int64_t M, int64_t N, int64_t K, OutY y, const Route& rt, hipStream_t stream,
                    bool run = true) {
  const bool ex = y.type == kF32;
  const int64_t per = GR ? (rt.R + rt.E - 1) / rt.E : M;      // rows of a matrix
  if (per <= kStreamRows)
    return ex ? stream_rows<true, GR>(qx, sx, qw, sw, M, N, K, y, rt, per, stream, run)
              : stream_rows<false, GR>(qx, sx, qw, sw, M, N, K, y, rt, per, stream, run);
  if (ex) return tile_t<128, 128, 2, 4, true, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream, run);
  // The largest tile that keeps the CUs busy, one workgroup each of 256 x 256, two and more of the
  // smaller ones (us): 8192 x 14336 into 4096, 512 tiles of 256 x 256: 393, of 128 x 128 459;
  // 1024 x 4096 into 14336, 224 tiles: 62.6 and 71.6; 2048 x 4096 into 4096, 128 tiles: 55.3, 38.1;
  // 512 x 4096 into 4096, 128 tiles of 128 x 128: 23.5, of 64 x 64 18.5. Experts' last tiles are
  // half empty on average.
  auto tiles = [&](int64_t t) {
    const int64_t rows = GR ? (2 * rt.R / t + rt.E) / 2 : (M + t - 1) / t;
    return rows * ((N + t - 1) / t);
  };
  const int64_t busy = (int64_t)device_cus() * 4 / 5;
  const bool near = !GR || (int64_t)rt.T * K < (1LL << 32);    // rows of x within 32-bit offsets
  if (tiles(256) >= busy && per >= 256 && near)
    return tile_t<256, 256, 4, 2, false, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream, run);
  if (tiles(128) >= busy)
    return tile_t<128, 128, 2, 2, false, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream, run);
  return tile_t<64, 64, 2, 2, false, GR>(qx, sx, qw, sw, M, N, K, y, rt, stream, run);
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
  // quantized by the product where its waves keep x (8 rows x 4096 into 4096: 8.4 us, one launch
  // more for the codes about 10), not for longer K, where every item would do it again
  const bool fused = M <= kFusedRows && K <= kStreamGroups * kGroup && Kx % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * (type == kF32 ? 4 : 2) % 16 == 0;
  const Route rt{};
  if (!fused) {                                       // the product's limits before the rows' launch
    hipError_t e = launch_t<false>(q, s, qw, sw, M, N, K, y, rt, stream, false);
    if (e == hipSuccess) e = launch_f8_rows(x, type, M, Kx, ldx, q, s, stream);
    return e != hipSuccess ? e : launch_w8a8_f8(q, s, qw, sw, M, N, K, y, stream);
  }
#define BGT_FUSED(T) \
  return stream_t<1, 2, false, true, T, false>(x, ldx, Kx, nullptr, qw, sw, M, N, K, y, rt, q, s, stream)
  if (type == kF32) BGT_FUSED(kF32);
  if (type == kF16) BGT_FUSED(kF16);
  BGT_FUSED(kBF16);
#undef BGT_FUSED
}

}  // namespace bgt
