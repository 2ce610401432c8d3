// gemv_w4a16.hip -- few rows of unquantized activations times 4-bit weights
// with a float scale per group of 128, dense and for expert-routed slots (gfx950).
//
//     y_ij = sum_l s_lj * p_ilj,   p_ilj = sum_{k in group l} x_ik q_kj
//
// x is fp16, bf16 or fp32; the codes q are small integers, exact in fp16 and
// bf16, so the group sums p run on the 16-bit matrix cores with fp32
// accumulation and each group takes one fp32 multiply-add per output.
//
// v_mfma_f32_16x16x32 (fp16 / bf16): lane L supplies row (A) or column (B)
// L%16 and the 8 k of slice L/16; result lane L, register r holds
// C[4*(L/16) + r][L%16]. A lane's 16 bytes of a packed block are four words of
// 8 consecutive k of its column (k = 64h + 16(L/16) + 8w + 0..7 of the group
// for word 2h + w), so word m is the B operand of MFMA m and the matching A
// operand is 8 consecutive elements of the lane's row of x.
//
// fp32 rows enter as three bf16 terms (8 + 8 + 8 significant bits, exact): row
// i becomes rows 3i, 3i+1, 3i+2 of A, whose products are added at the end.
//
// The weights' bytes bound it where they are many: 2 experts of 4096 x 14336, one
// token, 13.0 us (62 MB); 16 x 4096 x 22016 fp16 11.3 us (49 MB). Small products are
// bound by a launch and its round trips (1 x 4096 x 4096 4.1 us), few fp32 rows
// also by splitting them (3 x 11008 x 4096 10.2 us), and 17 to 64 rows by the rows:
// every workgroup reads all of them for its 16 to 64 columns, and more than 32 take
// the weights twice (4096 x 22016 fp16, 32 and 64 rows 15.6 and 29.3 us; 64 x 14336 x
// 4096 19.3).
#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace bgt {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloat8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
// loads of x at the alignment of its elements (one wide load all the same)
typedef uint32_t u4e __attribute__((ext_vector_type(4), aligned(2)));
typedef float f2e __attribute__((ext_vector_type(2), aligned(4)));

// words of a wave's LDS block, written and read as different types
typedef uint32_t u1a __attribute__((may_alias));
typedef uint32_t u4a __attribute__((ext_vector_type(4), may_alias));

// orders the wave's own LDS accesses (they execute in program order; this keeps
// the compiler from moving them across)
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// terms a row of x takes in A
template <int XT> constexpr int kTerms = XT == kF32 ? 3 : 1;

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t flip) {
  return (w & mask) ^ flip;
}
// upper halves of two words
__device__ __forceinline__ uint32_t pack_hi(uint32_t hi, uint32_t lo) {
  return perm(hi, lo, 0x07060302u);
}

// q / 16 in fp32 of the 4-bit two's complement q in the low nibble of byte B
template <int B>
__device__ __forceinline__ uint32_t sixteenth(uint32_t w) {
  uint32_t f;
#define BGT_SIXTEENTH(byte)                                                                 \
  asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:" byte      \
      : "=v"(f)                                                                             \
      : "v"(w))
  if constexpr (B == 0) BGT_SIXTEENTH("BYTE_0");
  if constexpr (B == 1) BGT_SIXTEENTH("BYTE_1");
  if constexpr (B == 2) BGT_SIXTEENTH("BYTE_2");
  if constexpr (B == 3) BGT_SIXTEENTH("BYTE_3");
#undef BGT_SIXTEENTH
  return f;
}

// 8 codes of a packed word as the B operand, k ascending. fp16: the nibbles of
// bytes (0,1) and (2,3) in the mantissas of 1024 + n and 1024 + 16 n, n = q + 8
// (sign bit flipped), less 1032, or times 1/16 less 72: exact. bf16: q / 16 in
// fp32 from the low nibble of each byte, the upper halves packed; scaled back
// with the group's scale (16, exact).
template <int XT>
__device__ __forceinline__ uint4 unpack(uint32_t w) {
  if constexpr (XT == kF16) {
    const half2v lo = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const half2v sc = {(_Float16)0.0625f, (_Float16)0.0625f};
    const half2v hi = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t u = perm(w, w, 0x01010000u), v = perm(w, w, 0x03030202u);
    const half2v a = __builtin_bit_cast(half2v, and_xor(u, 0x000F000Fu, 0x64086408u)) + lo;
    const half2v b = __builtin_bit_cast(half2v, and_xor(v, 0x000F000Fu, 0x64086408u)) + lo;
    const half2v c = __builtin_elementwise_fma(
        __builtin_bit_cast(half2v, and_xor(u, 0x00F000F0u, 0x64806480u)), sc, hi);
    const half2v d = __builtin_elementwise_fma(
        __builtin_bit_cast(half2v, and_xor(v, 0x00F000F0u, 0x64806480u)), sc, hi);
    return make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                      __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d));
  } else {
    const uint32_t h = w >> 4;
    return make_uint4(pack_hi(sixteenth<1>(w), sixteenth<0>(w)),
                      pack_hi(sixteenth<3>(w), sixteenth<2>(w)),
                      pack_hi(sixteenth<1>(h), sixteenth<0>(h)),
                      pack_hi(sixteenth<3>(h), sixteenth<2>(h)));
  }
}
template <int XT> constexpr float kCodeScale = XT == kF16 ? 1.0f : 16.0f;

template <int XT>
__device__ __forceinline__ v4f mfma(const uint4& a, const uint4& b, v4f c) {
  if constexpr (XT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfloat8, a),
                                                   __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------- rows of x as A
// The wave reads a group of each row in whole 256-byte runs and turns it into
// operands through an LDS block of its own (256 bytes a row; 16-byte pieces
// exchanged by row so that the 16 rows of an operand read fall on distinct
// banks). Loading operands directly, 16 bytes from each of 16 rows, takes the
// address path a request for every lane. No other wave touches the block.
// QR: rows in use, in fours (those past the last repeat it; the block's rows
// past 4*QR are never written, and nobody reads the outputs of either).
__device__ __forceinline__ uint4 lds_operand(const char* lds, int rb, int m) {
  const int lane = threadIdx.x % kWave, c = lane % 16;
  const int piece = 8 * (m / 2) + 2 * (lane / 16) + m % 2;
  const u4a v = *reinterpret_cast<const u4a*>(lds + (16 * rb + c) * 256 + (piece ^ c) * 16);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// fp16 / bf16: 16 lanes a row. load() takes the next group; the pointers run
// along (one pair of registers a quad; offsets from the group's number would
// keep one for every step of an unrolled loop).
template <int XT, int QR>
struct Rows {
  const uint16_t* row[QR];       // of row 4i + lane/16, at the lane's piece
  char* lds;
  // slot(i): row index in x of row i of this pass (i < nr); g: the first group
  template <typename F>
  __device__ __forceinline__ Rows(const void* xp, int64_t ldx, int nr, char* block, int g, F slot)
      : lds(block) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int i = 0; i < QR; ++i)
      row[i] = static_cast<const uint16_t*>(xp) + slot(min(4 * i + lane / 16, nr - 1)) * ldx +
               (int64_t)g * kGroup + 8 * (lane % 16);
  }
  struct Raw { u4e v[QR]; };
  __device__ __forceinline__ void load(Raw& r) {
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      r.v[i] = *reinterpret_cast<const u4e*>(row[i]);
      row[i] += kGroup;
    }
  }
  __device__ __forceinline__ void stage(const Raw& r) const {
    const int lane = threadIdx.x % kWave;
    wave_fence();                                  // the last group's reads come first
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int vr = 4 * i + lane / 16;
      *reinterpret_cast<u4a*>(lds + vr * 256 + ((lane % 16) ^ (vr % 16)) * 16) = r.v[i];
    }
    wave_fence();
  }
};

// fp32: 2 elements a lane; every element is split once, row i into rows 3i..3i+2
template <int QR>
struct Rows<kF32, QR> {
  static constexpr int ROWS = 4 * QR / 3;
  const float* x;
  int64_t off[ROWS];
  int nr;
  char* lds;
  template <typename F>
  __device__ __forceinline__ Rows(const void* xp, int64_t ldx, int rows, char* block, int g, F slot)
      : x(static_cast<const float*>(xp) + (int64_t)g * kGroup), nr(rows), lds(block) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      off[i] = (int64_t)__builtin_amdgcn_readfirstlane(slot(min(i, nr - 1))) * ldx;
  }
  struct Raw { f2e v[ROWS]; };
  __device__ __forceinline__ void load(Raw& r) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) r.v[i] = reinterpret_cast<const f2e*>(x + off[i])[lane];
    x += kGroup;
  }
  // v = hi + mid + lo by truncation, each exact in bf16 (its upper half). An
  // infinity stays whole in the first term; a NaN makes the second one NaN.
  __device__ __forceinline__ static void split(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = __float_as_uint(v);
    const float r1 = fabsf(v) == __builtin_inff() ? 0.0f : v - __uint_as_float(hi & 0xFFFF0000u);
    mid = __float_as_uint(r1);
    lo = __float_as_uint(r1 - __uint_as_float(mid & 0xFFFF0000u));
  }
  __device__ __forceinline__ void stage(const Raw& r) const {
    const int lane = threadIdx.x % kWave;
    wave_fence();                                  // the last group's reads come first
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i < nr) {
        uint32_t t0[3], t1[3];
        split(r.v[i].x, t0[0], t0[1], t0[2]);
        split(r.v[i].y, t1[0], t1[1], t1[2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const int vr = 3 * i + q;
          *reinterpret_cast<u1a*>(lds + vr * 256 + ((lane / 4) ^ (vr % 16)) * 16 + (lane % 4) * 4) =
              pack_hi(t1[q], t0[q]);
        }
      }
    }
    wave_fence();
  }
};

// ------------------------------------------------------------------- kernel
template <int QR> constexpr int kBlocks = (QR + 3) / 4;      // row blocks of 16

// The wave's groups [gb, ge) of NT column tiles.
// make_rows() is called once the first weights have been requested (the row
// list of routed slots is itself loaded).
template <int XT, int QR, int NT, typename F>
__device__ __forceinline__ void run_groups(F make_rows, const uint4* __restrict__ packed,
                                           const float* __restrict__ fscale, int t0, int tiles,
                                           int N, int G, int gb, int ge, char* lds,
                                           v4f (&acc)[kBlocks<QR>][NT]) {
  constexpr int MR = kBlocks<QR>;
  const int lane = threadIdx.x % kWave, c = lane % 16;
  // wave-uniform bases, the lane's part added by each load
  const uint4* wp[NT];
  const float* sp[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int t = min(t0 + nt, tiles - 1);         // a tile past the last repeats it, unused
    wp[nt] = packed + (int64_t)t * G * 64;
    sp[nt] = fscale + 16 * t;
  }
  typename Rows<XT, QR>::Raw a;
  uint4 w[2][NT];
  float s[2][NT];
  auto load = [&](int u, int g) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      w[u][nt] = (wp[nt] + (int64_t)g * 64)[lane];
      s[u][nt] = (sp[nt] + (int64_t)g * N)[c];
    }
  };
  // the four MFMAs of a group outermost: each operand is read once, and the
  // NT * MR sums advance side by side
  auto compute = [&](int u) {
    v4f p[MR][NT];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint4 op[MR];
#pragma unroll
      for (int rb = 0; rb < MR; ++rb) op[rb] = lds_operand(lds, rb, m);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4& q = w[u][nt];
        const uint4 b = unpack<XT>(m == 0 ? q.x : m == 1 ? q.y : m == 2 ? q.z : q.w);
#pragma unroll
        for (int rb = 0; rb < MR; ++rb)
          p[rb][nt] = mfma<XT>(op[rb], b, m == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : p[rb][nt]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float sc = s[u][nt] * kCodeScale<XT>;
#pragma unroll
      for (int rb = 0; rb < MR; ++rb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[rb][nt][r] = __builtin_fmaf(p[rb][nt][r], sc, acc[rb][nt][r]);
    }
  };
  if (gb >= ge) return;
  load(0, gb);
  Rows<XT, QR> rows = make_rows(gb, lds);
  rows.load(a);
  // A step hands its rows to LDS, requests the next group and computes its own,
  // so one group is on its way while one is computed (two on their way measured
  // no faster anywhere, and 6 to 12% slower with 16 rows: the registers cost
  // waves). The loop's steps load without a condition, so that the compiler's
  // wait counts are exact; the last one or two groups go through the tail.
  int g = gb;
  for (; g + 3 <= ge; g += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      rows.stage(a);
      load(u ^ 1, g + u + 1);
      rows.load(a);
      __builtin_amdgcn_sched_barrier(0);           // requests first, and no step's
      compute(u);                                  // waits before the last one's work
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  rows.stage(a);
  if (g + 1 < ge) {
    load(1, g + 1);
    rows.load(a);
    compute(0);
    rows.stage(a);
    compute(1);
  } else {
    compute(0);
  }
}

// One workgroup: NT column tiles of 16 for up to 4*QR / terms rows; its NW
// waves split the groups, and their partial outputs are added in wave order.
template <int XT, int QR, int NT, int NW>
__device__ __forceinline__ void run_rows(char* lds, const void* x, int64_t ldx, const uint4* packed,
                                         const float* fscale, int N, int G, OutY y, const Route& rt,
                                         bool routed, int first, int nr) {
  constexpr int TERMS = kTerms<XT>, MR = kBlocks<QR>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int c = lane % 16, s4 = lane / 16;
  const int t0 = blockIdx.x * NT;
  auto make_rows = [&](int g, char* block) {
    return Rows<XT, QR>(x, ldx, nr, block, g, [&](int i) {
      return routed ? clamp_route(rt.tok[first + i], 0, rt.T - 1) : first + i;
    });
  };
  v4f acc[MR][NT];
#pragma unroll
  for (int rb = 0; rb < MR; ++rb)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[rb][nt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  run_groups<XT, QR, NT>(make_rows, packed, fscale, t0, N / 16, N, G, G * wave / NW,
                            G * (wave + 1) / NW, lds + wave * MR * 4096, acc);
  float* part = reinterpret_cast<float*>(lds);     // [NW][16 MR][16 NT]
  __syncthreads();                                 // the waves' row blocks are done with
#pragma unroll
  for (int rb = 0; rb < MR; ++rb)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        part[((wave * MR + rb) * 16 + 4 * s4 + r) * (16 * NT) + 16 * nt + c] = acc[rb][nt][r];
  __syncthreads();
  for (int o = threadIdx.x; o < nr * 16 * NT; o += NW * 64) {
    const int i = o / (16 * NT), j = o % (16 * NT);
    if (16 * t0 + j < N) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int q = TERMS - 1; q >= 0; --q)
          v += part[(w * 16 * MR + i * TERMS + q) * (16 * NT) + j];
      y.put((int64_t)(first + i) * N + 16 * t0 + j, v);
    }
  }
  __syncthreads();
}

template <int QR, int NT, int NW>
constexpr int kLds = (NT < 4 ? 4 : NT) * 1024 * NW * kBlocks<QR>;

// dense: up to 4*QR / terms rows a pass, grid z over the passes
template <int XT, int QR, int NT, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2))) void k_w4a16(
    const void* __restrict__ x, int64_t ldx, const uint4* __restrict__ packed,
    const float* __restrict__ fscale, int M, int N, int G, OutY y) {
  __shared__ __attribute__((aligned(16))) char lds[kLds<QR, NT, NW>];
  constexpr int ROWS = 4 * QR / kTerms<XT>;
  const int r0 = blockIdx.z * ROWS;
  run_rows<XT, QR, NT, NW>(lds, x, ldx, packed, fscale, N, G, y, Route{}, false, r0,
                              min(ROWS, M - r0));
}

// The j-th pass over slots of one expert: the expert, the pass's first slot and slot
// count. An expert's slots make whole passes of ROWS and one of the rest; passes of
// more than `many` slots come before all others, and the first ones of the experts
// before their further ones. False: there are no more. Every wave reads the offsets
// 64 experts at a time.
template <int ROWS>
__device__ __forceinline__ bool find_pass(const Route& rt, int j, int many, int& e, int& first,
                                          int& rows) {
  const int lane = threadIdx.x % kWave;
  const bool whole_heavy = ROWS > many;
  for (int heavy = many < rt.R; heavy >= 0; --heavy)
    for (int base = 0; base < rt.E; base += kWave) {
      const int i = min(base + lane, rt.E - 1);
      const int a = clamp_route(rt.offs[i], 0, rt.R), b = clamp_route(rt.offs[i + 1], a, rt.R);
      const int n = base + lane < rt.E ? b - a : 0, whole = n / ROWS, rest = n % ROWS;
      const int mine = (whole_heavy == (heavy != 0) ? whole : 0) +
                       (rest > 0 && (rest > many) == (heavy != 0) ? 1 : 0);
      const unsigned long long some = __ballot(mine > 0);
      unsigned long long hit = 0;
      int local = 0;
      if (j < __popcll(some)) {
        hit = __ballot(mine > 0 && __popcll(some & ((2ull << lane) - 1)) == j + 1);
      } else {
        j -= __popcll(some);
        if (__ballot(mine > 1) == 0) continue;
        int upto = max(mine - 1, 0);
        for (int o = 1; o < kWave; o <<= 1) {
          const int below = __shfl_up(upto, o, kWave);
          if (lane >= o) upto += below;
        }
        const int before = upto - max(mine - 1, 0);
        hit = __ballot(j >= before && j < upto);
        if (hit == 0) {
          j -= __builtin_amdgcn_readfirstlane(__shfl(upto, kWave - 1, kWave));
          continue;
        }
        local = 1 + j - before;
      }
      // the one pass of a class that whole passes are not in is the rest
      const int pass = whole_heavy == (heavy != 0) ? local : whole;
      const int l = __builtin_ctzll(hit);
      e = __builtin_amdgcn_readfirstlane(base + l);
      first = __builtin_amdgcn_readfirstlane(__shfl(a + pass * ROWS, l, kWave));
      rows = __builtin_amdgcn_readfirstlane(__shfl(min(n - pass * ROWS, ROWS), l, kWave));
      return true;
    }
  return false;
}

// routed: grid y (and z, past 65535) deals out the passes of up to 4*QR / terms rows,
// not more than the slots can make, so the grid of a few slots has few rows. Passes
// of one expert run side by side (8 experts of 14336 x 4096, 122 slots, calls: 61 of
// them at two experts each 29.5 us, one after the other in a workgroup 50.2; 61 at one
// and 8 or 9 at the others 64 to 67 and 78.7; 12 to 20 each 54 and 56). The further
// passes find the weights in the Infinity Cache only where those of all busy experts
// fit it: of 64 experts of 14336 x 4096, 1.9 GB and 512 slots, 8 each 350 us, 20 at 16
// of them and 4 at the others 418 (351 as one pass each of up to 32 rows). A pass takes
// 16 or 24 rows of A where that is enough (20 slots each: 58 us as 24 rows, 62 as 32).
// The first y zeroes the rows past the last slot.
template <int XT, int QR, int NT, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2))) void k_w4a16_moe(
    const void* __restrict__ x, int64_t ldx, const uint4* __restrict__ packed,
    const float* __restrict__ fscale, int N, int G, OutY y, Route rt) {
  __shared__ __attribute__((aligned(16))) char lds[kLds<QR, NT, NW>];
  constexpr int TERMS = kTerms<XT>, ROWS = 4 * QR / TERMS;
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    const int c0 = 16 * NT * blockIdx.x, cols = min(16 * NT, N - c0);
    const int last = clamp_route(rt.offs[rt.E], 0, rt.R);
    for (int64_t o = threadIdx.x; o < (int64_t)(rt.R - last) * cols; o += NW * 64)
      y.put((last + o / cols) * N + c0 + o % cols, 0.0f);
  }
  // with blocks of 16 rows and larger ones in a launch the larger start first, so
  // that a CU's workgroups are of both kinds (8 experts of 14336 x 4096, 61
  // tokens: 57.1 -> 55.0 us)
  const int many = QR > 4 ? 16 / TERMS : rt.R;
  int e, first, nr;
  if (!find_pass<ROWS>(rt, blockIdx.z * gridDim.y + blockIdx.y, many, e, first, nr)) return;
  packed += (int64_t)e * rt.wstride / 16;
  fscale += (int64_t)e * rt.sstride;
  if (QR > 4 && nr * TERMS <= 16)
    run_rows<XT, 4, NT, NW>(lds, x, ldx, packed, fscale, N, G, y, rt, true, first, nr);
  else if (QR > 6 && nr * TERMS <= 24)
    run_rows<XT, 6, NT, NW>(lds, x, ldx, packed, fscale, N, G, y, rt, true, first, nr);
  else
    run_rows<XT, QR, NT, NW>(lds, x, ldx, packed, fscale, N, G, y, rt, true, first, nr);
}

template <int XT, int QR, int NT, int NW>
static void launch_dense(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale,
                         int M, int N, int K, OutY y, hipStream_t stream) {
  constexpr int ROWS = 4 * QR / kTerms<XT>;
  const int tiles = N / 16;
  const dim3 grid((tiles + NT - 1) / NT, 1, (M + ROWS - 1) / ROWS);
  hipLaunchKernelGGL((k_w4a16<XT, QR, NT, NW>), grid, dim3(NW * 64), 0, stream, x, ldx,
                     reinterpret_cast<const uint4*>(packed), fscale, M, N, K / kGroup, y);
}
template <int XT, int QR, int NT, int NW>
static void launch_routed(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale,
                          int N, int K, OutY y, const Route& rt, hipStream_t stream) {
  // the most passes that R slots of E experts make
  const int tiles = N / 16, busy = min(rt.E, rt.R);
  const int passes = busy + (rt.R - busy) / (4 * QR / kTerms<XT>);
  const int ny = min(passes, 65535), nz = (passes + ny - 1) / ny;
  hipLaunchKernelGGL((k_w4a16_moe<XT, QR, NT, NW>), dim3((tiles + NT - 1) / NT, ny, nz),
                     dim3(NW * 64), 0, stream, x, ldx, reinterpret_cast<const uint4*>(packed),
                     fscale, N, K / kGroup, y, rt);
}

// Column tiles a workgroup of more than one row quad takes, for `tiles` tiles in
// the whole launch (more than one a CU): what the busiest CU then has to do,
// each workgroup's rows counted as 0.3 tiles a quad. Sweeps (us), 2 / 3 / 4 tiles a
// workgroup, [taken]: 16 x 4096 fp16 at N = 8192 [6.9] / 7.1 / 8.0, 11008 8.1 / [7.5] /
// 8.1, 14336 9.0 / 10.2 / [8.7], 22016 13.0 / [11.7] / 14.2, 28672 17.5 / 15.7 / [13.8];
// 32 x 14336 fp16 at 8192 [19.7] / 24.9 / 26.2, 11008 37 / [25] / 30, 14336 43 / 48 /
// [37]; 8 experts of 14336 x 4096, 61 tokens 73.8 / 72.1 / [65.4]. It does not know that
// four tiles of 32 rows of 16 bits need more registers than there are (256, 25 to
// 34 of them spilled), which costs where K is short: 32 x 4096 fp16 at N =
// 14336 11.3 / 14.1 / [13.3], 22016 16.1 / [16.0] / 22.6, 28672 20.1 / 21.9 / [22.0], 32768
// 21.0 / 24.0 / [25.6]; 48 rows at 22016 28.3 / 26.2 / [29.5].
static int tiles_per_wg(int tiles, int qr) {
  const int cus = device_cus();
  int best = 2;
  float least = 0.0f;
  for (int nt = 2; nt <= 4; ++nt) {
    const int wgs = (tiles + nt - 1) / nt;
    const float cost = (float)((wgs + cus - 1) / cus) * ((float)nt + 0.3f * (float)qr);
    if (nt == 2 || cost <= least) { best = nt; least = cost; }
  }
  return best;
}

// f(QR, NT, NW) for rows of A, the tile count and the groups. Up to one tile a
// CU: a tile a workgroup, its groups over 8 waves (16 for few fp32 rows, which
// have the splitting to do: 3 x 11008 x 4096 10.7 -> 9.6 us). More: 4 waves, for
// up to 4 rows of A, whose rows cost little, with one tile (1 x 4096 x 11008
// bf16, 1 / 2 / 3 / 4 tiles: 6.2 / 7.9 / 7.3 / 8.7 us; 2 experts of 4096 x 14336,
// one token: 12.5 / 13.9 / 14.1 / 14.2), in launches of 192 MiB of weights and more
// with four: no mechanism is known, only the sweeps. One / four tiles, one row of
// bf16, one of fp16, four of fp16, one of fp32: 14336 x 22016 (150 MiB) 35 / 39, 34 / 36,
// 35 / 37, 41 / 44; 28672 (196 MiB) 44 / 44, 43 / 43, 47 / 43, 46 / 48; 32768 (224 MiB)
// 51 / 50, 58 / 49, 57 / 50, 53 / 50; 57344 (392 MiB) 85 / 96, 82 / 92, 91 / 90, 91 / 90;
// 4096 x 98304 (192 MiB) 43 / 43, 40 / 42, 42 / 41, 45 / 44; routed, one token of bf16, 6
// and 8 experts of 4096 x 14336 (168 and 224 MiB) 40 / 40 and 53 / 49. For more rows as
// tiles_per_wg says.
template <int XT, typename F>
static void with_shape(int rows, int tiles, int groups, F f) {
  constexpr int FEW = XT == kF32 ? 16 : 8;
  const bool one = tiles <= device_cus();
  if (rows <= 4) {
    if (one) f(IC<1>{}, IC<1>{}, IC<FEW>{});
    else if ((int64_t)tiles * groups < 192 * 1024) f(IC<1>{}, IC<1>{}, IC<4>{});
    else f(IC<1>{}, IC<4>{}, IC<4>{});
    return;
  }
  const auto by_tiles = [&](auto qr) {
    constexpr int QR = decltype(qr)::value;
    if (one) return f(qr, IC<1>{}, IC<QR <= 4 ? FEW : 8>{});
    const int nt = tiles_per_wg(tiles, QR);
    if (nt == 2) f(qr, IC<2>{}, IC<4>{});
    else if (nt == 3) f(qr, IC<3>{}, IC<4>{});
    else f(qr, IC<4>{}, IC<4>{});
  };
  if (rows <= 16) by_tiles(IC<4>{});
  else by_tiles(IC<8>{});
}

template <int XT>
static void dense_of_type(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale,
                          int M, int N, int K, OutY y, hipStream_t stream) {
  const int passes = (M * kTerms<XT> + 31) / 32;
  with_shape<XT>(M * kTerms<XT>, passes * (N / 16), K / kGroup, [&](auto qr, auto nt, auto nw) {
    launch_dense<XT, decltype(qr)::value, decltype(nt)::value, decltype(nw)::value>(
        x, ldx, packed, fscale, M, N, K, y, stream);
  });
}

template <int XT>
static void routed_of_type(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale,
                           int N, int K, OutY y, const Route& rt, hipStream_t stream) {
  // rows an expert gets at most, and half as many again as the mean: an expert
  // with more takes another pass over its weights, in other workgroups
  const int busy = min(rt.E, rt.R);
  const int rows = min(min(rt.T, rt.R), (3 * rt.R / rt.E + 1) / 2 + 1);
  with_shape<XT>(rows * kTerms<XT>, busy * (N / 16), K / kGroup, [&](auto qr, auto nt, auto nw) {
    launch_routed<XT, decltype(qr)::value, decltype(nt)::value, decltype(nw)::value>(
        x, ldx, packed, fscale, N, K, y, rt, stream);
  });
}

hipError_t launch_w4a16(const void* x, int x_type, int64_t ldx, const uint8_t* packed,
                        const float* fscale, int64_t M, int64_t N, int64_t K, OutY y,
                        hipStream_t stream) {
  const int m = (int)M, n = (int)N, k = (int)K;
  if (x_type == kF32) dense_of_type<kF32>(x, ldx, packed, fscale, m, n, k, y, stream);
  else if (x_type == kF16) dense_of_type<kF16>(x, ldx, packed, fscale, m, n, k, y, stream);
  else dense_of_type<kBF16>(x, ldx, packed, fscale, m, n, k, y, stream);
  return hipGetLastError();
}

hipError_t launch_w4a16_moe(const void* x, int x_type, int64_t ldx, int64_t T, const int32_t* offs,
                            const int32_t* tok, int64_t E, int64_t R, const uint8_t* packed,
                            const float* fscale, int64_t N, int64_t K, OutY y, hipStream_t stream) {
  const Route rt{offs, tok, (int)E, (int)T, (int)R, N * K / 2, (K / kGroup) * N};
  const int n = (int)N, k = (int)K;
  if (x_type == kF32) routed_of_type<kF32>(x, ldx, packed, fscale, n, k, y, rt, stream);
  else if (x_type == kF16) routed_of_type<kF16>(x, ldx, packed, fscale, n, k, y, rt, stream);
  else routed_of_type<kBF16>(x, ldx, packed, fscale, n, k, y, rt, stream);
  return hipGetLastError();
}

}  // namespace bgt
