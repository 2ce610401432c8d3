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
typedef float f4e __attribute__((ext_vector_type(4), aligned(4)));

// terms a row of x takes in A
template <int XT> constexpr int kTerms = XT == kF32 ? 3 : 1;

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

// The A operand of one MFMA: 8 consecutive elements of a row. fp16 elements are
// reordered to (0,2 1,3 4,6 5,7), the order in which unpack_f16 leaves codes.
template <int XT>
__device__ __forceinline__ uint4 load_a(const void* row, int k, int term) {
  if constexpr (XT == kF16) {
    const u4e d = *reinterpret_cast<const u4e*>(static_cast<const uint16_t*>(row) + k);
    return make_uint4(perm(d.y, d.x, 0x05040100u), perm(d.y, d.x, 0x07060302u),
                      perm(d.w, d.z, 0x05040100u), perm(d.w, d.z, 0x07060302u));
  } else if constexpr (XT == kBF16) {
    const u4e d = *reinterpret_cast<const u4e*>(static_cast<const uint16_t*>(row) + k);
    return make_uint4(d.x, d.y, d.z, d.w);
  } else {
    const f4e* p = reinterpret_cast<const f4e*>(static_cast<const float*>(row) + k);
    const f4e a = p[0], b = p[1];
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // v = hi + mid + lo by truncation, each exact in bf16; infinities and
      // NaN stay whole in the first term
      const uint32_t u = __float_as_uint(v[i]);
      const bool fin = (u & 0x7F800000u) != 0x7F800000u;
      const float hi = __uint_as_float(u & 0xFFFF0000u);
      const float r1 = v[i] - hi;
      const float mid = __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
      const float lo = r1 - mid;
      const uint32_t top = fin ? u : ((u & 0x007FFFFFu) ? 0x7FC00000u : u);
      t[i] = term == 0 ? top : (!fin ? 0u : __float_as_uint(term == 1 ? mid : lo));
    }
    return make_uint4(perm(t[1], t[0], 0x07060302u), perm(t[3], t[2], 0x07060302u),
                      perm(t[5], t[4], 0x07060302u), perm(t[7], t[6], 0x07060302u));
  }
}

// 8 codes of a packed word as the B operand. fp16: (1024 + n) - 1032 with
// n = q + 8 set in the mantissa (or 1024 + 16n, times 1/16): exact. bf16: 16 q
// by signed byte conversions, the upper halves packed; scaled back with the
// group's scale (1/16, exact).
template <int XT>
__device__ __forceinline__ uint4 unpack(uint32_t w) {
  if constexpr (XT == kF16) {
    const uint32_t n = w ^ 0x88888888u, n8 = n >> 8;
    const half2v lo = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const half2v sc = {(_Float16)0.0625f, (_Float16)0.0625f};
    const half2v hi = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t a = (n & 0x000F000Fu) | 0x64006400u, b = (n8 & 0x000F000Fu) | 0x64006400u;
    const uint32_t c = (n & 0x00F000F0u) | 0x64006400u, d = (n8 & 0x00F000F0u) | 0x64006400u;
    const half2v ah = __builtin_bit_cast(half2v, a) + lo, bh = __builtin_bit_cast(half2v, b) + lo;
    const half2v ch = __builtin_elementwise_fma(__builtin_bit_cast(half2v, c), sc, hi);
    const half2v dh = __builtin_elementwise_fma(__builtin_bit_cast(half2v, d), sc, hi);
    return make_uint4(__builtin_bit_cast(uint32_t, ah), __builtin_bit_cast(uint32_t, bh),
                      __builtin_bit_cast(uint32_t, ch), __builtin_bit_cast(uint32_t, dh));
  } else {
    uint32_t lo, hi;
    unpack_x16(w, lo, hi);
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __float_as_uint((float)(int8_t)(lo >> (8 * i)));
      f[4 + i] = __float_as_uint((float)(int8_t)(hi >> (8 * i)));
    }
    return make_uint4(perm(f[1], f[0], 0x07060302u), perm(f[3], f[2], 0x07060302u),
                      perm(f[5], f[4], 0x07060302u), perm(f[7], f[6], 0x07060302u));
  }
}
template <int XT> constexpr float kCodeScale = XT == kF16 ? 1.0f : 0.0625f;

template <int XT>
__device__ __forceinline__ v4f mfma(const uint4& a, const uint4& b, v4f c) {
  if constexpr (XT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfloat8, a),
                                                   __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}

// One workgroup: NT column tiles of 16 for up to 16*MR / terms rows; its NW
// waves split the groups, and their partial outputs are added in wave order.
template <int XT, int MR, int NT, int NW, bool GR>
__global__ __launch_bounds__(NW * 64) void k_w4a16(const void* __restrict__ x, int64_t ldx,
                                                   const uint4* __restrict__ packed,
                                                   const float* __restrict__ fscale, int M, int N,
                                                   int G, OutY y, Route rt) {
  constexpr int TERMS = kTerms<XT>, ROWS = 16 * MR / TERMS;
  __shared__ float part[NW][MR][16][16 * NT];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int c = lane % 16, s4 = lane / 16;
  const int t0 = blockIdx.x * NT, tiles = N / 16;
  int first = 0, rows = M;
  if constexpr (GR) {
    const int e = blockIdx.y;
    const int last = clamp_route(rt.offs[rt.E], 0, rt.R);
    if (e == rt.E) {                               // rows past the last slot are zero
      const int cols = min(16 * NT, N - 16 * t0);
      for (int r = last; r < rt.R; ++r)
        for (int j = threadIdx.x; j < cols; j += NW * 64) y.put((int64_t)r * N + 16 * t0 + j, 0.0f);
      return;
    }
    first = clamp_route(rt.offs[e], 0, rt.R);
    rows = clamp_route(rt.offs[e + 1], first, rt.R) - first;
    packed += (int64_t)e * rt.wstride / 16;
    fscale += (int64_t)e * rt.sstride;
  }
  const int gb = G * wave / NW, ge = G * (wave + 1) / NW;
  for (int pass = blockIdx.z; pass * ROWS < rows; pass += gridDim.z) {
    const int r0 = pass * ROWS, nr = min(ROWS, rows - r0);
    const char* arow[MR];
#pragma unroll
    for (int rb = 0; rb < MR; ++rb) {
      int i = first + r0 + min((rb * 16 + c) / TERMS, nr - 1);
      if constexpr (GR) i = clamp_route(rt.tok[i], 0, rt.T - 1);
      arow[rb] = static_cast<const char*>(x) + (int64_t)i * ldx * (XT == kF32 ? 4 : 2);
    }
    v4f acc[MR][NT];
#pragma unroll
    for (int rb = 0; rb < MR; ++rb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[rb][nt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int g = gb; g < ge; ++g) {
      uint4 a[MR][4];
#pragma unroll
      for (int rb = 0; rb < MR; ++rb)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          a[rb][m] = load_a<XT>(arow[rb], g * kGroup + 64 * (m / 2) + 16 * s4 + 8 * (m % 2),
                                (rb * 16 + c) % TERMS);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int t = min(t0 + nt, tiles - 1);
        const uint4 w = load_u4_nt(packed + ((int64_t)t * G + g) * 64 + lane);
        const float sc = fscale[(int64_t)g * N + 16 * t + c] * kCodeScale<XT>;
        const uint4 b0 = unpack<XT>(w.x), b1 = unpack<XT>(w.y), b2 = unpack<XT>(w.z),
                    b3 = unpack<XT>(w.w);
#pragma unroll
        for (int rb = 0; rb < MR; ++rb) {
          v4f p = {0.0f, 0.0f, 0.0f, 0.0f};
          p = mfma<XT>(a[rb][0], b0, p);
          p = mfma<XT>(a[rb][1], b1, p);
          p = mfma<XT>(a[rb][2], b2, p);
          p = mfma<XT>(a[rb][3], b3, p);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[rb][nt][r] = fmaf(p[r], sc, acc[rb][nt][r]);
        }
      }
    }
#pragma unroll
    for (int rb = 0; rb < MR; ++rb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][rb][4 * s4 + r][16 * nt + c] = acc[rb][nt][r];
    __syncthreads();
    for (int o = threadIdx.x; o < nr * 16 * NT; o += NW * 64) {
      const int i = o / (16 * NT), j = o % (16 * NT);
      if (16 * t0 + j < N) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
          for (int q = TERMS - 1; q >= 0; --q) {
            const int vr = i * TERMS + q;
            v += part[w][vr / 16][vr % 16][j];
          }
        y.put((int64_t)(first + r0 + i) * N + 16 * t0 + j, v);
      }
    }
    __syncthreads();
  }
}

template <int XT, int MR, bool GR>
static void launch_mr(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale, int M,
                      int N, int K, OutY y, const Route& rt, hipStream_t stream) {
  constexpr int ROWS = 16 * MR / kTerms<XT>;
  const int tiles = N / 16;
  const dim3 grid(tiles, GR ? rt.E + 1 : 1, GR ? 1 : (M + ROWS - 1) / ROWS);
  hipLaunchKernelGGL((k_w4a16<XT, MR, 1, 8, GR>), grid, dim3(512), 0, stream, x, ldx,
                     reinterpret_cast<const uint4*>(packed), fscale, M, N, K / kGroup, y, rt);
}

template <int XT, bool GR>
static void launch_type(const void* x, int64_t ldx, const uint8_t* packed, const float* fscale,
                        int M, int N, int K, OutY y, const Route& rt, hipStream_t stream) {
  const int blocks = (M * kTerms<XT> + 15) / 16;   // row blocks of A
  if (blocks <= 1) launch_mr<XT, 1, GR>(x, ldx, packed, fscale, M, N, K, y, rt, stream);
  else if (blocks == 2) launch_mr<XT, 2, GR>(x, ldx, packed, fscale, M, N, K, y, rt, stream);
  else launch_mr<XT, 4, GR>(x, ldx, packed, fscale, M, N, K, y, rt, stream);
}

hipError_t launch_w4a16(const void* x, int x_type, int64_t ldx, const uint8_t* packed,
                        const float* fscale, int64_t M, int64_t N, int64_t K, OutY y,
                        hipStream_t stream) {
  const Route none{};
  const int m = (int)M, n = (int)N, k = (int)K;
  if (x_type == kF32) launch_type<kF32, false>(x, ldx, packed, fscale, m, n, k, y, none, stream);
  else if (x_type == kF16) launch_type<kF16, false>(x, ldx, packed, fscale, m, n, k, y, none, stream);
  else launch_type<kBF16, false>(x, ldx, packed, fscale, m, n, k, y, none, stream);
  return hipGetLastError();
}

hipError_t launch_w4a16_moe(const void* x, int x_type, int64_t ldx, int64_t T, const int32_t* offs,
                            const int32_t* tok, int64_t E, int64_t R, const uint8_t* packed,
                            const float* fscale, int64_t N, int64_t K, OutY y, hipStream_t stream) {
  const Route rt{offs, tok, (int)E, (int)T, (int)R, N * K / 2, (K / kGroup) * N};
  const int m = (int)(T < R ? T : R), n = (int)N, k = (int)K;   // an expert's most rows
  if (x_type == kF32) launch_type<kF32, true>(x, ldx, packed, fscale, m, n, k, y, rt, stream);
  else if (x_type == kF16) launch_type<kF16, true>(x, ldx, packed, fscale, m, n, k, y, rt, stream);
  else launch_type<kBF16, true>(x, ldx, packed, fscale, m, n, k, y, rt, stream);
  return hipGetLastError();
}

}  // namespace bgt
