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
#include "device_common.h"
#include "launch.h"

namespace bgt {

constexpr int kMaxE = 256;          // experts
constexpr float kNegInf = -__builtin_inff();

// ------------------------------------------------------------- counting sort
// The slots of a chunk are dealt to the waves in contiguous segments. Per
// (wave, expert) counts, turned into first positions, then each wave walks its
// segment 64 slots at a time; a slot's place among its wave's equal slots is
// the number of lower lanes with the same expert, found by ballots over the
// bits of the expert, so the order is that of the slots and no atomic decides it.
struct SortShared {
  int base[kMaxE];      // first position of each expert's slots of this chunk
  int scan[kMaxE];
};

// counts[w][e] of the block's NW waves over slots [s0, s1)
template <int NW>
__device__ __forceinline__ void count_slots(const int32_t* ids, int64_t s0, int64_t s1, int E,
                                            int (*counts)[kMaxE]) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int i = threadIdx.x; i < NW * kMaxE; i += NW * kWave) (&counts[0][0])[i] = 0;
  __syncthreads();
  const int64_t seg = (s1 - s0 + NW * kWave - 1) / (NW * kWave) * kWave;
  const int64_t a = s0 + wave * seg, b = min(s1, a + seg);
  for (int64_t s = a + lane; s < b; s += kWave) {
    const int e = ids[s];
    if (e >= 0 && e < E) atomicAdd(&counts[wave][e], 1);
  }
  __syncthreads();
}

// exclusive prefix over the experts of v (thread e holds expert e's, e < kMaxE);
// every thread calls; scan[] holds the inclusive prefix afterwards
__device__ __forceinline__ int scan_experts(int v, int* scan) {
  const int e = threadIdx.x;
  if (e < kMaxE) scan[e] = v;
  __syncthreads();
  for (int o = 1; o < kMaxE; o <<= 1) {
    const int u = (e < kMaxE && e >= o) ? scan[e - o] : 0;
    __syncthreads();
    if (e < kMaxE) scan[e] += u;
    __syncthreads();
  }
  return e < kMaxE ? scan[e] - v : 0;
}

// positions of the slots [s0, s1) of this chunk, given sh.base
template <int NW>
__device__ __forceinline__ void place_slots(const int32_t* ids, int64_t s0, int64_t s1, int E,
                                            int k, int (*counts)[kMaxE], const SortShared& sh,
                                            int32_t* tok, int32_t* pos) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int e = threadIdx.x; e < E; e += NW * kWave) {
    int run = sh.base[e];
    for (int w = 0; w < NW; ++w) {
      const int c = counts[w][e];
      counts[w][e] = run;
      run += c;
    }
  }
  __syncthreads();
  const int64_t seg = (s1 - s0 + NW * kWave - 1) / (NW * kWave) * kWave;
  const int64_t a = s0 + wave * seg, b = min(s1, a + seg);
  const unsigned long long below = (1ull << lane) - 1;
  for (int64_t s = a; s < b; s += kWave) {
    const bool in = s + lane < b;
    int e = in ? ids[s + lane] : -1;
    const bool ok = e >= 0 && e < E;
    unsigned long long same = __ballot(ok);
    for (int bit = 1; bit < E; bit <<= 1) {
      const unsigned long long m = __ballot(ok && (e & bit));
      same &= (e & bit) ? m : ~m;
    }
    int first = 0;
    if (ok) first = counts[wave][e];
    __builtin_amdgcn_wave_barrier();               // all lanes read before the leaders add
    const int p = first + __popcll(same & below);
    if (ok && (same & below) == 0) counts[wave][e] = first + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) pos[s + lane] = ok ? p : -1;
    if (ok) tok[p] = (int)((s + lane) / k);
  }
}

// the whole sort by one workgroup
template <int NW>
__device__ __forceinline__ void sort_single(const int32_t* ids, int64_t R, int E, int k,
                                            int (*counts)[kMaxE], SortShared& sh, int32_t* offs,
                                            int32_t* tok, int32_t* pos) {
  count_slots<NW>(ids, 0, R, E, counts);
  int mine = 0;
  if ((int)threadIdx.x < E)
    for (int w = 0; w < NW; ++w) mine += counts[w][threadIdx.x];
  const int excl = scan_experts(mine, sh.scan);
  if ((int)threadIdx.x < E) {
    sh.base[threadIdx.x] = excl;
    offs[threadIdx.x] = excl;
  }
  if (threadIdx.x == 0) offs[E] = sh.scan[E - 1];
  __syncthreads();
  place_slots<NW>(ids, 0, R, E, k, counts, sh, tok, pos);
  for (int64_t r = sh.scan[E - 1] + threadIdx.x; r < R; r += NW * kWave) tok[r] = -1;
}

template <int NW>
__global__ __launch_bounds__(NW * 64) void k_sort_single(const int32_t* __restrict__ ids, int64_t R,
                                                         int E, int k, int32_t* __restrict__ offs,
                                                         int32_t* __restrict__ tok,
                                                         int32_t* __restrict__ pos) {
  __shared__ int counts[NW][kMaxE];
  __shared__ SortShared sh;
  sort_single<NW>(ids, R, E, k, counts, sh, offs, tok, pos);
}

// --------------------------------------------------------------------- top k
// L lanes share a token, V logits each (expert l + L v in lane l). k rounds of a
// maximum over the lanes by (logit, lower expert first).
template <int IT, int L, int V>
__global__ __launch_bounds__(256) void k_route_top(const void* __restrict__ logits, int64_t ld,
                                                   int64_t T, int E, int k, bool all,
                                                   float* __restrict__ weights,
                                                   int32_t* __restrict__ ids) {
  const int l = threadIdx.x % L;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const bool in = t < T;
  float v[V], orig[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = l + L * i;
    const float raw = in && e < E ? load_x1<IT>(logits, t * ld + e) : kNegInf;
    orig[i] = raw;
    v[i] = raw == raw ? raw : kNegInf;
  }
  float m = 0.0f, mine = 0.0f, sum = 0.0f;   // lane i keeps the i-th chosen logit
  int my_id = -1;
  for (int i = 0; i < k; ++i) {
    float best = kNegInf;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (v[j] > best) { best = v[j]; at = l + L * j; }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const float b = __shfl_xor(best, o, kWave);
      const int a = __shfl_xor(at, o, kWave);
      if (b > best || (b == best && a < at)) { best = b; at = a; }
    }
    const bool got = best > kNegInf;
    if (i == 0) m = got ? best : 0.0f;
    const float e = got ? expf(best - m) : 0.0f;
    sum += e;
    if (l == i % L) {
      mine = e;
      my_id = got ? at : -1;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (at == l + L * j) v[j] = kNegInf;
    if (l == i % L && in) {
      ids[t * k + i] = my_id;
      weights[t * k + i] = mine;
    }
  }
  if (all) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += expf(orig[j] - m);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  }
  for (int i = l; i < k; i += L)
    if (in) {
      const float w = weights[t * k + i];
      weights[t * k + i] = ids[t * k + i] >= 0 ? w / sum : 0.0f;
    }
}

// ------------------------------------------------------------------ gradient
template <int IT, int L, int V>
__global__ __launch_bounds__(256) void k_route_grad(const float* __restrict__ dw,
                                                    const void* __restrict__ logits, int64_t ld,
                                                    const int32_t* __restrict__ ids, int64_t T,
                                                    int E, int k, bool all, OutY out) {
  const int l = threadIdx.x % L;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const bool in = t < T;
  float v[V], d[V];
  bool hit[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = l + L * i;
    v[i] = in && e < E ? load_x1<IT>(logits, t * ld + e) : kNegInf;
    d[i] = 0.0f;
    hit[i] = false;
  }
  if (in)
    for (int i = 0; i < k; ++i) {
      const int id = ids[t * k + i];
      const float g = dw[t * k + i];
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (id == l + L * j) { d[j] = g; hit[j] = true; }
    }
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (!all && !hit[j]) v[j] = kNegInf;
    m = fmaxf(m, v[j]);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  if (!(m > kNegInf)) m = 0.0f;                    // nothing left: every p is 0
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = expf(v[j] - m);
    sum += v[j];
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (sum == 0.0f) sum = 1.0f;
  float dot = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] /= sum;
    dot += v[j] * d[j];
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = l + L * j;
    if (in && e < E) out.put(t * E + e, v[j] * (d[j] - dot));
  }
}

// ----------------------------------------------------------------- launchers
template <int IT, typename F>
static void with_lanes(int E, F f) {
  if (E <= 8) f(IC<8>{}, IC<1>{});
  else if (E <= 16) f(IC<16>{}, IC<1>{});
  else if (E <= 32) f(IC<32>{}, IC<1>{});
  else if (E <= 64) f(IC<64>{}, IC<1>{});
  else if (E <= 128) f(IC<64>{}, IC<2>{});
  else f(IC<64>{}, IC<4>{});
}

template <int IT>
static void launch_top(const void* logits, int64_t ld, int64_t T, int E, int k, bool all,
                       float* weights, int32_t* ids, hipStream_t stream) {
  with_lanes<IT>(E, [&](auto lanes, auto vals) {
    constexpr int L = decltype(lanes)::value, V = decltype(vals)::value;
    hipLaunchKernelGGL((k_route_top<IT, L, V>), dim3((unsigned)((T * L + 255) / 256)), dim3(256), 0,
                       stream, logits, ld, T, E, k, all, weights, ids);
  });
}

template <int IT>
static void launch_grad(const float* dw, const void* logits, int64_t ld, const int32_t* ids,
                        int64_t T, int E, int k, bool all, OutY out, hipStream_t stream) {
  with_lanes<IT>(E, [&](auto lanes, auto vals) {
    constexpr int L = decltype(lanes)::value, V = decltype(vals)::value;
    hipLaunchKernelGGL((k_route_grad<IT, L, V>), dim3((unsigned)((T * L + 255) / 256)), dim3(256),
                       0, stream, dw, logits, ld, ids, T, E, k, all, out);
  });
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t T, int64_t E, int64_t k, int32_t* offs,
                           int32_t* tok, int32_t* pos, int32_t* ws, hipStream_t stream) {
  (void)ws;
  hipLaunchKernelGGL((k_sort_single<16>), dim3(1), dim3(1024), 0, stream, ids, T * k, (int)E,
                     (int)k, offs, tok, pos);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int type, int64_t ld, int64_t T, int64_t E,
                            int64_t k, bool all, float* weights, int32_t* ids, int32_t* offs,
                            int32_t* tok, int32_t* pos, int32_t* ws, hipStream_t stream) {
  if (type == kF32) launch_top<kF32>(logits, ld, T, (int)E, (int)k, all, weights, ids, stream);
  else if (type == kF16) launch_top<kF16>(logits, ld, T, (int)E, (int)k, all, weights, ids, stream);
  else launch_top<kBF16>(logits, ld, T, (int)E, (int)k, all, weights, ids, stream);
  return launch_moe_sort(ids, T, E, k, offs, tok, pos, ws, stream);
}

hipError_t launch_moe_route_backward(const float* dw, const void* logits, int type, int64_t ld,
                                     const int32_t* ids, int64_t T, int64_t E, int64_t k, bool all,
                                     void* dlogits, hipStream_t stream) {
  const OutY out{dlogits, type};
  if (type == kF32) launch_grad<kF32>(dw, logits, ld, ids, T, (int)E, (int)k, all, out, stream);
  else if (type == kF16) launch_grad<kF16>(dw, logits, ld, ids, T, (int)E, (int)k, all, out, stream);
  else launch_grad<kBF16>(dw, logits, ld, ids, T, (int)E, (int)k, all, out, stream);
  return hipGetLastError();
}

// 0: one workgroup sorts
int64_t moe_sort_ws_bytes(int64_t T, int64_t E, int64_t k) {
  (void)T; (void)E; (void)k;
  return 0;
}

}  // namespace bgt
