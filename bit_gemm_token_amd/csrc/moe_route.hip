// moe_route.hip -- routing of a mixture-of-experts layer (gfx950): the k
// experts of each token from the router's logits, the routed slots sorted by
// expert, and the gradient of the logits.
//
//   chosen experts of token t: its k largest logits, ties to the lower expert;
//   w_ti = exp(l_ti - m) / sum, the sum over the chosen experts or over all;
//   slots (t, i) sorted by expert, in order of (t, i) within an expert;
//   dl_j = p_j (dw_j - sum_i p_i dw_i) with p the same softmax.
//
// -inf and NaN logits are never chosen; a token with fewer than k others has
// expert -1 and weight 0 in its last places, and those slots are dropped.
//
// The work is a few bytes a token, so launches and round trips bound it: few
// tokens (one_launch) are chosen for and sorted by one workgroup in one launch;
// otherwise the choosing launch also leaves each workgroup's slot counts by
// expert, and a second launch sorts, every workgroup adding up the counts before
// its own.
// Kernel times: one token of 8 experts 3.6 us, 64 tokens of 256 experts, k = 8, 11.0 us
// (6.7 to choose, 4.3 to sort), 4096 tokens of 8 experts, k = 2, 8.9 us (3.8 and 5.1),
// 16381 tokens of 64 experts, k = 6, 12.6 us (6.7 and 5.9) and 5.3 us for the gradient;
// the sort alone of the last two 7.3 us (2.3 to count, 5.0 to place) and 8.9 (2.8, 6.1).
#include "device_common.h"
#include "launch.h"

namespace bgt {

constexpr int kMaxE = 256;          // experts
constexpr int kMaxK = 16;           // experts of a token
constexpr int kMaxChunks = 256;     // workgroups a sort is split into
constexpr int64_t kSingleSlots = 1024;  // slots one workgroup sorts
constexpr float kNegInf = -__builtin_inff();

// ------------------------------------------------------------- counting sort
// The slots of a workgroup are dealt to its waves in contiguous segments. Per
// (wave, expert) counts become first positions; then each wave walks its
// segment 64 slots at a time. A slot's place among its wave's equal slots is
// the number of lower lanes with the same expert, found by ballots over the
// bits of the expert, so the order is that of the slots and no atomic decides it.
template <int NW>
struct Sorter {
  int counts[NW][kMaxE];
  int base[kMaxE];      // first position of each expert's slots of this chunk
  int total;            // slots that have an expert

  __device__ __forceinline__ static int64_t segment(int64_t n) {
    return (n + NW * kWave - 1) / (NW * kWave) * kWave;
  }

  // counts[w][e] over the slots [s0, s1)
  __device__ __forceinline__ void count(const int32_t* ids, int64_t s0, int64_t s1, int E) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    for (int w = 0; w < NW; ++w)
      for (int e = threadIdx.x; e < E; e += NW * kWave) counts[w][e] = 0;
    __syncthreads();
    const int64_t a = s0 + wave * segment(s1 - s0), b = min(s1, a + segment(s1 - s0));
    for (int64_t s = a + lane; s < b; s += kWave) {
      const int e = ids[s];
      if (e >= 0 && e < E) atomicAdd(&counts[wave][e], 1);
    }
    __syncthreads();
  }

  // the counts of all waves of one expert
  __device__ __forceinline__ int counted(int e) const {
    int n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) n += counts[w][e];
    return n;
  }

  // base[e] = totals[e]'s exclusive prefix + before[e], by the first wave, 4
  // experts a lane; offs gets the prefixes where not null. totals may be base.
  __device__ __forceinline__ void scan(const int* totals, const int* before, int E, int32_t* offs) {
    if (threadIdx.x < kWave) {
      const int lane = threadIdx.x;
      int v[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i;
        v[i] = e < E ? totals[e] : 0;
        sum += v[i];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += u;
      }
      int run = incl - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i;
        if (e < E) {
          base[e] = run + (before ? before[e] : 0);
          if (offs) offs[e] = run;
        }
        run += v[i];
      }
      if (lane == kWave - 1) {
        total = incl;
        if (offs) offs[E] = incl;
      }
    }
    __syncthreads();
  }

  // tok and pos of the slots [s0, s1), given counts and base
  __device__ __forceinline__ void place(const int32_t* ids, int64_t s0, int64_t s1, int E, int k,
                                        int32_t* tok, int32_t* pos) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    for (int e = threadIdx.x; e < E; e += NW * kWave) {
      int run = base[e];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int c = counts[w][e];
        counts[w][e] = run;
        run += c;
      }
    }
    __syncthreads();
    const int64_t a = s0 + wave * segment(s1 - s0), b = min(s1, a + segment(s1 - s0));
    const unsigned long long below = (1ull << lane) - 1;
    int next = a + lane < b ? ids[a + lane] : -1;
    for (int64_t s = a; s < b; s += kWave) {
      const bool in = s + lane < b;
      const int e = next;
      next = s + kWave + lane < b ? ids[s + kWave + lane] : -1;
      const bool ok = e >= 0 && e < E;
      unsigned long long same = __ballot(ok);
      for (int bit = 1; bit < E; bit <<= 1) {
        const unsigned long long m = __ballot(ok && (e & bit));
        same &= (e & bit) ? m : ~m;
      }
      const int first = ok ? counts[wave][e] : 0;
      __builtin_amdgcn_wave_barrier();             // all lanes read before the leaders add
      const int p = first + __popcll(same & below);
      if (ok && (same & below) == 0) counts[wave][e] = first + __popcll(same);
      __builtin_amdgcn_wave_barrier();
      if (in) pos[s + lane] = ok ? p : -1;
      if (ok) tok[p] = (int)((uint32_t)(s + lane) / (uint32_t)k);   // slots fit 24 bits
    }
  }

  // the whole sort by one workgroup; ids may just have been written by it
  __device__ __forceinline__ void sort_all(const int32_t* ids, int64_t R, int E, int k,
                                           int32_t* offs, int32_t* tok, int32_t* pos) {
    count(ids, 0, R, E);
    for (int e = threadIdx.x; e < E; e += NW * kWave) base[e] = counted(e);
    __syncthreads();
    scan(base, nullptr, E, offs);
    place(ids, 0, R, E, k, tok, pos);
    for (int64_t r = total + threadIdx.x; r < R; r += NW * kWave) tok[r] = -1;
  }
};

template <int NW>
__global__ __launch_bounds__(NW * 64) void k_slot_sort(const int32_t* __restrict__ ids, int64_t R,
                                                       int E, int k, int32_t* __restrict__ offs,
                                                       int32_t* __restrict__ tok,
                                                       int32_t* __restrict__ pos) {
  __shared__ Sorter<NW> sh;
  sh.sort_all(ids, R, E, k, offs, tok, pos);
}

// chunk b's slot counts by expert
template <int NW>
__global__ __launch_bounds__(NW * 64) void k_slot_count(const int32_t* __restrict__ ids, int64_t R,
                                                        int64_t chunk, int E,
                                                        int32_t* __restrict__ counts) {
  __shared__ Sorter<NW> sh;
  const int64_t s0 = blockIdx.x * chunk;
  sh.count(ids, s0, min(R, s0 + chunk), E);
  for (int e = threadIdx.x; e < E; e += NW * kWave)
    counts[(int64_t)blockIdx.x * E + e] = sh.counted(e);
}

// chunk b's slots, given every chunk's counts. The threads add up the counts
// column by column, several of them to an expert (the reads of one column are
// independent: a few round trips in all).
template <int NW>
__global__ __launch_bounds__(NW * 64) void k_slot_place(const int32_t* __restrict__ ids, int64_t R,
                                                        int64_t chunk, int E, int k,
                                                        const int32_t* __restrict__ chunk_counts,
                                                        int32_t* __restrict__ offs,
                                                        int32_t* __restrict__ tok,
                                                        int32_t* __restrict__ pos) {
  __shared__ Sorter<NW> sh;
  __shared__ int before[kMaxE], totals[kMaxE];
  const int n = gridDim.x, b = blockIdx.x;
  for (int e = threadIdx.x; e < kMaxE; e += NW * kWave) before[e] = totals[e] = 0;
  int cols = 8;                                    // power of two from E on
  while (cols < E) cols <<= 1;
  const int e = threadIdx.x & (cols - 1), part = threadIdx.x / cols, parts = NW * kWave / cols;
  int below = 0, all = 0;
  if (e < E) {
#pragma unroll 8
    for (int i = part; i < n; i += parts) {
      const int c = chunk_counts[(int64_t)i * E + e];
      all += c;
      below += i < b ? c : 0;
    }
  }
  const int64_t s0 = b * chunk, s1 = min(R, s0 + chunk);
  sh.count(ids, s0, s1, E);                        // (synchronizes)
  if (e < E) {
    atomicAdd(&before[e], below);
    atomicAdd(&totals[e], all);
  }
  __syncthreads();
  sh.scan(totals, before, E, b == 0 ? offs : nullptr);
  sh.place(ids, s0, s1, E, k, tok, pos);
  for (int64_t r = sh.total + (int64_t)b * NW * kWave + threadIdx.x; r < R;
       r += (int64_t)n * NW * kWave)
    tok[r] = -1;
}

// ------------------------------------------------------- lanes of a token
// L neighbouring lanes share a token, V consecutive logits each (expert V*l + j
// in lane l): 4 each up to 32 experts, 8 beyond, so a wave works on 2 to 32
// tokens and an exchange among a token's lanes takes 1 to 5 steps.
typedef uint32_t u4e __attribute__((ext_vector_type(4), aligned(2)));

template <int IT, int V>
__device__ __forceinline__ void load_logits(const void* row, int e0, int E, float (&v)[V]) {
  constexpr int W = IT == kF32 ? 4 : 8;            // elements of 16 bytes
  const char* p = static_cast<const char*>(row) + (int64_t)e0 * (IT == kF32 ? 4 : 2);
  if (e0 + V <= E && V % W == 0) {
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
      const u4e u = *reinterpret_cast<const u4e*>(p + 16 * q);
      if constexpr (IT == kF32) {
        v[4 * q] = __uint_as_float(u.x); v[4 * q + 1] = __uint_as_float(u.y);
        v[4 * q + 2] = __uint_as_float(u.z); v[4 * q + 3] = __uint_as_float(u.w);
      } else {
        const float4 a = widen_x4<IT>(make_uint2(u.x, u.y));
        const float4 b = widen_x4<IT>(make_uint2(u.z, u.w));
        v[8 * q] = a.x; v[8 * q + 1] = a.y; v[8 * q + 2] = a.z; v[8 * q + 3] = a.w;
        v[8 * q + 4] = b.x; v[8 * q + 5] = b.y; v[8 * q + 6] = b.z; v[8 * q + 7] = b.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = e0 + j < E ? load_x1<IT>(p, j) : kNegInf;
  }
}

// v of the lane that step STEP pairs this one with: the neighbour, the next
// pair, the other half of 8 or of 16 (mirrored: by then the lanes of each half
// hold the same), the other 16. Up to 16 lanes these are register moves.
template <int STEP>
__device__ __forceinline__ int partner(int v) {
  // DPP controls: quad permutations 1,0,3,2 and 2,3,0,1, mirrors of 8 and of 16
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
  else if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
  else if constexpr (STEP == 4) return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
  else if constexpr (STEP == 8) return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);
  else return __shfl_xor(v, STEP, kWave);
}
template <int STEP>
__device__ __forceinline__ float partner(float v) {
  return __int_as_float(partner<STEP>(__float_as_int(v)));
}
template <int L, int STEP = 1>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (STEP < L) return lanes_sum<L, 2 * STEP>(v + partner<STEP>(v));
  else return v;
}
template <int L, int STEP = 1>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (STEP < L) return lanes_max<L, 2 * STEP>(fmaxf(v, partner<STEP>(v)));
  else return v;
}
// the largest value of the L lanes and its index, the lower one of equal ones
// (-1, of no value, is above all others)
template <int L, int STEP = 1>
__device__ __forceinline__ void lanes_best(float& best, int& at) {
  if constexpr (STEP < L) {
    const float b = partner<STEP>(best);
    const int a = partner<STEP>(at);
    if (b > best || (b == best && (unsigned)a < (unsigned)at)) { best = b; at = a; }
    lanes_best<L, 2 * STEP>(best, at);
  }
}

// --------------------------------------------------------------------- top k
// waves of a workgroup: 128 or 64 tokens at once with 2 or 4 lanes a token, 64, 32
// or 16 with 8, 16 or 32
template <int L> constexpr int kTopWaves = L <= 4 ? 4 : 8;

// Workgroup b chooses for tokens [b*tb, (b+1)*tb) and leaves its slots' counts
// by expert in chunk_counts[b], or, without chunk_counts (one workgroup), sorts.
// k rounds of a maximum over the token's lanes by (logit, lower expert first).
template <int IT, int L, int V>
__global__ __launch_bounds__(kTopWaves<L> * 64) void k_route_top(
    const void* __restrict__ logits, int64_t ld, int64_t T, int64_t tb, int E, int k, bool all,
    float* __restrict__ weights, int32_t* ids, int32_t* __restrict__ chunk_counts,
    int32_t* __restrict__ offs, int32_t* __restrict__ tok, int32_t* __restrict__ pos) {
  constexpr int THREADS = kTopWaves<L> * kWave, TOKENS = THREADS / L;
  __shared__ float top_e[TOKENS][kMaxK + 1];       // exp(l - m) and experts of this round's tokens
  __shared__ int top_id[TOKENS][kMaxK + 1];
  __shared__ float sums[TOKENS];
  __shared__ Sorter<kTopWaves<L>> sh;
  const int l = threadIdx.x % L, mine = threadIdx.x / L;
  const int64_t t0 = blockIdx.x * tb, t1 = min(T, t0 + tb);
  if (chunk_counts)
    for (int e = threadIdx.x; e < E; e += THREADS) sh.base[e] = 0;
  for (int64_t tr = t0; tr < t1; tr += TOKENS) {
    const int64_t t = tr + mine;
    float v[V];
    if (t < t1) {
      const char* row = static_cast<const char*>(logits) + t * ld * (IT == kF32 ? 4 : 2);
      load_logits<IT, V>(row, V * l, E, v);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = kNegInf;
    }
    // the largest of all (a NaN only matters to the sum over all)
    float m = kNegInf, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, v[j]);
    m = lanes_max<L>(m);
    if (!(m > kNegInf)) m = 0.0f;
    if (all) {
#pragma unroll
      for (int j = 0; j < V; ++j) sum += expf(v[j] - m);
      sum = lanes_sum<L>(sum);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = v[j] == v[j] ? v[j] : kNegInf;
    for (int i = 0; i < k; ++i) {
      float best = kNegInf;
      int at = -1;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (v[j] > best) { best = v[j]; at = V * l + j; }
      lanes_best<L>(best, at);
      const float e = at >= 0 ? expf(best - m) : 0.0f;
      if (!all) sum += e;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at == V * l + j) v[j] = kNegInf;
      if (l == 0) {
        top_e[mine][i] = e;
        top_id[mine][i] = at;
      }
    }
    if (l == 0) sums[mine] = sum;
    __syncthreads();
    const int n = (int)min((int64_t)TOKENS, t1 - tr) * k;
    for (int o = threadIdx.x; o < n; o += THREADS) {
      const int r = o / k, i = o - r * k, id = top_id[r][i];
      ids[tr * k + o] = id;
      weights[tr * k + o] = id >= 0 ? top_e[r][i] / sums[r] : 0.0f;
      if (chunk_counts && id >= 0) atomicAdd(&sh.base[id], 1);
    }
    __syncthreads();
  }
  if (chunk_counts) {
    for (int e = threadIdx.x; e < E; e += THREADS)
      chunk_counts[(int64_t)blockIdx.x * E + e] = sh.base[e];
  } else {
    sh.sort_all(ids, T * k, E, k, offs, tok, pos);
  }
}

// ------------------------------------------------------------------ gradient
template <int IT, int L, int V>
__global__ __launch_bounds__(256) void k_route_grad(const float* __restrict__ dw,
                                                    const void* __restrict__ logits, int64_t ld,
                                                    const int32_t* __restrict__ ids, int64_t T,
                                                    int E, int k, bool all, void* __restrict__ dl) {
  constexpr int TOKENS = 256 / L;
  __shared__ float sdw[TOKENS * kMaxK];
  __shared__ int sid[TOKENS * kMaxK];
  const int l = threadIdx.x % L, mine = threadIdx.x / L;
  const int64_t tr = (int64_t)blockIdx.x * TOKENS, t = tr + mine;
  const bool in = t < T;
  const int n = (int)min((int64_t)TOKENS, T - tr) * k;
  for (int o = threadIdx.x; o < n; o += 256) {
    // an id past E may fall on a lane's padding, where 0 * dweight would meet the sum
    const int id = ids[tr * k + o];
    sdw[o] = dw[tr * k + o];
    sid[o] = id >= 0 && id < E ? id : -1;
  }
  float v[V], d[V];
  if (in) {
    const char* row = static_cast<const char*>(logits) + t * ld * (IT == kF32 ? 4 : 2);
    load_logits<IT, V>(row, V * l, E, v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = kNegInf;
  }
  __syncthreads();
  unsigned hit = all ? ~0u : 0;                    // logits that the softmax is over
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.0f;
  if (in)
    for (int i = 0; i < k; ++i) {
      const int at = sid[mine * k + i] - V * l;
      const float g = sdw[mine * k + i];
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at == j) {
          d[j] = g;
          hit |= 1u << j;
        }
    }
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (!(hit >> j & 1)) v[j] = kNegInf;
    m = fmaxf(m, v[j]);
  }
  m = lanes_max<L>(m);
  if (!(m > kNegInf)) m = 0.0f;                    // nothing left: every p is 0
  float sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = expf(v[j] - m);
    sum += v[j];
  }
  sum = lanes_sum<L>(sum);
  if (sum == 0.0f) sum = 1.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] /= sum;
    dot = __builtin_fmaf(v[j], d[j], dot);
  }
  dot = lanes_sum<L>(dot);
  // the others' gradient is 0, also where the sum is not finite
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = hit >> j & 1 ? v[j] * (d[j] - dot) : 0.0f;
  const OutY out{dl, IT};
  const int64_t o = t * E + V * l;
  constexpr int W = IT == kF32 ? 4 : 8;
  if (in && V * l + V <= E && V % W == 0) {
    char* p = static_cast<char*>(dl) + o * (IT == kF32 ? 4 : 2);
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
      u4e u;
      if constexpr (IT == kF32)
        u = u4e{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])};
      else
        u = u4e{narrow2<IT>(v[8 * q], v[8 * q + 1]), narrow2<IT>(v[8 * q + 2], v[8 * q + 3]),
                narrow2<IT>(v[8 * q + 4], v[8 * q + 5]), narrow2<IT>(v[8 * q + 6], v[8 * q + 7])};
      *reinterpret_cast<u4e*>(p + 16 * q) = u;
    }
  } else if (in) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (V * l + j < E) out.put(o + j, v[j]);
  }
}

// ----------------------------------------------------------------- launchers
namespace {

template <typename F>
void with_lanes(int E, F f) {
  if (E <= 8) f(IC<2>{}, IC<4>{});
  else if (E <= 16) f(IC<4>{}, IC<4>{});
  else if (E <= 32) f(IC<8>{}, IC<4>{});
  else if (E <= 64) f(IC<8>{}, IC<8>{});
  else if (E <= 128) f(IC<16>{}, IC<8>{});
  else f(IC<32>{}, IC<8>{});
}
int tokens_at_once(int E) {
  int n = 0;
  with_lanes(E, [&](auto lanes, auto) {
    constexpr int L = decltype(lanes)::value;
    n = kTopWaves<L> * kWave / L;
  });
  return n;
}

// whether one workgroup chooses and sorts in one launch. Its rounds of tokens
// follow each other, about 0.75 + 0.5 k us each; two launches cost the host 2.6 us
// more and the device about 2. Kernels, one launch / two, us: 256 tokens of 8
// experts, k = 2 (2 rounds) 5.6 / 6.6, 512 (4 rounds) 8.8 / 6.7; 64 of 128, k = 8 (2
// rounds) 11.5 / 9.8, 128 (4) 20.5 / 10.0; 1024 of 8, k = 1 (8) 10.7 / 6.6; 1024 of
// 256, k = 1 (64) 85 / 8.3. Calls that are waited for: 25.3 / 27.6, 28.1 / 27.6; 30.5 /
// 29.4, 39.6 / 29.4; 30.1 / 28.6; 104 / 28.
bool one_launch(int64_t T, int64_t E, int64_t k) {
  const int64_t round = tokens_at_once((int)E), rounds = (T + round - 1) / round;
  return T * k <= kSingleSlots && (rounds - 1) * (3 + 2 * k) <= 21;
}

// tokens of a workgroup where several sort: one round of the choosing kernel,
// more where that would take over kMaxChunks workgroups
int64_t chunk_tokens(int64_t T, int64_t E) {
  const int64_t round = tokens_at_once((int)E);
  const int64_t need = (T + kMaxChunks - 1) / kMaxChunks;
  return (need + round - 1) / round * round;
}

template <int IT>
void launch_top(const void* logits, int64_t ld, int64_t T, int64_t tb, int E, int k, bool all,
                float* weights, int32_t* ids, int32_t* counts, int32_t* offs, int32_t* tok,
                int32_t* pos, hipStream_t stream) {
  with_lanes(E, [&](auto lanes, auto vals) {
    constexpr int L = decltype(lanes)::value, V = decltype(vals)::value;
    hipLaunchKernelGGL((k_route_top<IT, L, V>), dim3((unsigned)((T + tb - 1) / tb)),
                       dim3(kTopWaves<L> * 64), 0, stream, logits, ld, T, tb, E, k, all, weights, ids,
                       counts, offs, tok, pos);
  });
}

template <int IT>
void launch_grad(const float* dw, const void* logits, int64_t ld, const int32_t* ids, int64_t T,
                 int E, int k, bool all, void* dl, hipStream_t stream) {
  with_lanes(E, [&](auto lanes, auto vals) {
    constexpr int L = decltype(lanes)::value, V = decltype(vals)::value;
    hipLaunchKernelGGL((k_route_grad<IT, L, V>), dim3((unsigned)((T * L + 255) / 256)), dim3(256),
                       0, stream, dw, logits, ld, ids, T, E, k, all, dl);
  });
}

void launch_place(const int32_t* ids, int64_t R, int64_t chunk, int E, int k, const int32_t* counts,
                  int32_t* offs, int32_t* tok, int32_t* pos, hipStream_t stream) {
  hipLaunchKernelGGL((k_slot_place<16>), dim3((unsigned)((R + chunk - 1) / chunk)), dim3(1024), 0,
                     stream, ids, R, chunk, E, k, counts, offs, tok, pos);
}

}  // namespace

// the chunks' counts; one workgroup needs none. (Where one_launch holds the sort
// alone is one launch too, so this is enough for both.)
int64_t moe_sort_ws_bytes(int64_t T, int64_t E, int64_t k) {
  if (one_launch(T, E, k)) return 0;
  const int64_t tb = chunk_tokens(T, E);
  return (T + tb - 1) / tb * E * 4;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t T, int64_t E, int64_t k, int32_t* offs,
                           int32_t* tok, int32_t* pos, int32_t* ws, hipStream_t stream) {
  const int64_t R = T * k;
  if (R <= kSingleSlots) {
    hipLaunchKernelGGL((k_slot_sort<4>), dim3(1), dim3(256), 0, stream, ids, R, (int)E, (int)k, offs,
                       tok, pos);
    return hipGetLastError();
  }
  const int64_t chunk = chunk_tokens(T, E) * k;
  hipLaunchKernelGGL((k_slot_count<4>), dim3((unsigned)((R + chunk - 1) / chunk)), dim3(256), 0,
                     stream, ids, R, chunk, (int)E, ws);
  launch_place(ids, R, chunk, (int)E, (int)k, ws, offs, tok, pos, stream);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int type, int64_t ld, int64_t T, int64_t E,
                            int64_t k, bool all, float* weights, int32_t* ids, int32_t* offs,
                            int32_t* tok, int32_t* pos, int32_t* ws, hipStream_t stream) {
  const bool single = one_launch(T, E, k);
  const int64_t tb = single ? T : chunk_tokens(T, E);
  int32_t* counts = single ? nullptr : ws;
  const int e = (int)E, n = (int)k;
  const auto top = type == kF32   ? launch_top<kF32>
                   : type == kF16 ? launch_top<kF16>
                                  : launch_top<kBF16>;
  top(logits, ld, T, tb, e, n, all, weights, ids, counts, offs, tok, pos, stream);
  if (!single) launch_place(ids, T * k, tb * k, e, n, ws, offs, tok, pos, stream);
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const float* dw, const void* logits, int type, int64_t ld,
                                     const int32_t* ids, int64_t T, int64_t E, int64_t k, bool all,
                                     void* dlogits, hipStream_t stream) {
  const int e = (int)E, n = (int)k;
  if (type == kF32) launch_grad<kF32>(dw, logits, ld, ids, T, e, n, all, dlogits, stream);
  else if (type == kF16) launch_grad<kF16>(dw, logits, ld, ids, T, e, n, all, dlogits, stream);
  else launch_grad<kBF16>(dw, logits, ld, ids, T, e, n, all, dlogits, stream);
  return hipGetLastError();
}

}  // namespace bgt
