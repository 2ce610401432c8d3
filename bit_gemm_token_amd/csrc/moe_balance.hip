// moe_balance.hip -- a router's balance loss with the experts' counts, and its gradient (gfx950).
//
//     p_t = softmax(l_t) over all E experts,   c_e = number of ids equal to e,   f_e = c_e / sum c,
//     loss = E sum_e f_e P_e,   P_e = (1 / T') sum_t p_te
//     dl_te = dloss (E / T') p_te (f_e - sum_j f_j p_tj)       (f is a constant of the gradient)
//
// T': the tokens with a logit other than -inf; the others (padding) have p_t = 0 and no gradient.
//
// A token's logits lie in L = 1 .. 64 lanes, four each, so that its softmax takes lane exchanges
// only; a lane adds up its own four experts' probabilities over its tokens in registers, the
// workgroup's sums go to the workspace and a second launch adds those in order (equal inputs
// give equal bits; counts are integers). Latency bounds both: a few dependent round trips.
#include "device_common.h"
#include "launch.h"

namespace bgt {

namespace {

constexpr int kEach = 4, kBThreads = 256, kBWaves = kBThreads / kWave;

// lanes of a token: the least power of two that holds E
int lanes_of(int64_t E) {
  int L = 1;
  while (L * kEach < E) L *= 2;
  return L;
}
// workgroups: at least 4 tokens for each group of lanes, at most 256
int balance_wgs(int64_t T, int64_t E) {
  const int64_t at_once = kBThreads / lanes_of(E);
  const int64_t w = (T + 4 * at_once - 1) / (4 * at_once);
  return (int)(w < 1 ? 1 : w > 256 ? 256 : w);
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
// the softmax of a token's logits over its L lanes; false where all are -inf (p = 0). The maximum
// passes over NaN, the sum does not: it is 0 only if every term is, so that a token of NaN and
// -inf alone is NaN too, as the formula is.
template <int L, int IT>
__device__ __forceinline__ bool softmax4(const void* logits, int64_t row, int e0, int E, float* p) {
  float v[kEach], top = -INFINITY;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    v[j] = e0 + j < E ? load_x1<IT>(logits, row + e0 + j) : -INFINITY;
    top = fmaxf(top, v[j]);
  }
  top = group_max<L>(top);
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    p[j] = expf(v[j] - top);
    sum += p[j];
  }
  sum = group_sum<L>(sum);
  const bool some = !(sum == 0.0f);
#pragma unroll
  for (int j = 0; j < kEach; ++j) p[j] = some ? p[j] / sum : 0.0f;
  return some;
}

// sums of one workgroup (W of them): [w][E] probabilities, then [w][E] counts, then [w] tokens
struct Parts {
  float* probs;
  int32_t* counts;
  int32_t* tokens;
};
__device__ __forceinline__ Parts parts_of(void* ws, int W, int E) {
  float* p = static_cast<float*>(ws);
  int32_t* c = reinterpret_cast<int32_t*>(p + (int64_t)W * E);
  return Parts{p, c, c + (int64_t)W * E};
}

// The experts' sums over W workgroups' parts, then loss. Threads of one expert take every
// slices-th part, U of them at once (256 parts of 64 experts: 34.5 us a thread an expert in turn, 6 so).
constexpr int kSlices = 16, kJoinThreads = 1024;
template <int THREADS, int U>
__device__ __forceinline__ void join_parts(Parts ps, int W, int E, float* loss, int32_t* counts,
                                           float* probs, int32_t* tokens) {
  __shared__ double psum[THREADS];
  __shared__ int csum[THREADS], valid;
  const int tid = threadIdx.x;
  const int slices = U == 1 ? 1 : E * kSlices <= THREADS ? kSlices : THREADS / E;
  const int e = U == 1 ? tid : tid % E, first = U == 1 ? tid >= E : tid / E;
  if (tid == 0) valid = 0;
  double p = 0.0;
  int c = 0;
  if (first < slices)
    for (int w0 = first; w0 < W; w0 += U * slices) {
      float a[U];
      int b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int w = w0 + u * slices < W ? w0 + u * slices : first;
        a[u] = ps.probs[(int64_t)w * E + e];
        b[u] = ps.counts[(int64_t)w * E + e];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (w0 + u * slices < W) {
          p += a[u];
          c += b[u];
        }
    }
  psum[tid] = p;
  csum[tid] = c;
  __syncthreads();
  if (tid < W) {                                      // W <= 256
    const int n = ps.tokens[tid];
    if (n > 0) atomicAdd(&valid, n);
  }
  p = 0.0;
  c = 0;
  if (tid < E)
    for (int s = 0; s < slices; ++s) {
      p += psum[s * E + tid];
      c += csum[s * E + tid];
    }
  __syncthreads();
  const int n = valid;
  const double mean = n > 0 ? p / n : 0.0;
  if (tid < E) {
    probs[tid] = (float)mean;
    counts[tid] = c;
  }
  psum[tid] = mean * c;
  csum[tid] = c;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {                 // E <= 256
    if (tid < o) {
      psum[tid] += psum[tid + o];
      csum[tid] += csum[tid + o];
    }
    __syncthreads();
  }
  if (tid == 0) {
    *loss = csum[0] > 0 ? (float)(E * psum[0] / csum[0]) : 0.0f;
    *tokens = n;
  }
}

}  // namespace

template <int L, int IT>
__global__ __launch_bounds__(kBThreads) void k_balance_parts(
    const void* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids, int T, int E, int k,
    void* ws, float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ tokens) {
  constexpr int AT = kBThreads / L;                   // tokens at once
  __shared__ float psum[kBWaves][L * kEach];
  __shared__ int csum[256], nsum;
  const int W = gridDim.x, tid = threadIdx.x, wave = tid / kWave;
  const int e0 = tid % L * kEach;
  csum[tid] = 0;
  if (tid == 0) nsum = 0;
  __syncthreads();
  const int t0 = (int)((int64_t)blockIdx.x * T / W), t1 = (int)((int64_t)(blockIdx.x + 1) * T / W);
  for (int64_t i = (int64_t)t0 * k + tid; i < (int64_t)t1 * k; i += kBThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&csum[e], 1);
  }
  float acc[kEach] = {0.0f, 0.0f, 0.0f, 0.0f};
  int n = 0;
  auto tokens_at = [&](int t, int u) {
    const bool live = t + u * AT < t1;
    float p[kEach];
    const bool some = softmax4<L, IT>(logits, (int64_t)(live ? t + u * AT : t) * ld, e0, E, p);
    n += live && some ? 1 : 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) acc[j] += live ? p[j] : 0.0f;
  };
  if (t1 - t0 <= AT) {
    if (t0 + tid / L < t1) tokens_at(t0 + tid / L, 0);
  } else {                                            // four at a time: their round trips overlap
    for (int t = t0 + tid / L; t < t1; t += 4 * AT)
#pragma unroll
      for (int u = 0; u < 4; ++u) tokens_at(t, u);
  }
  if (tid % L == 0 && n > 0) atomicAdd(&nsum, n);
#pragma unroll
  for (int o = L; o < kWave; o <<= 1)
#pragma unroll
    for (int j = 0; j < kEach; ++j) acc[j] += __shfl_xor(acc[j], o, kWave);
  if (tid % kWave < L)
#pragma unroll
    for (int j = 0; j < kEach; ++j) psum[wave][e0 + j] = acc[j];
  __syncthreads();
  const Parts ps = parts_of(ws, W, E);
  if (tid < E) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kBWaves; ++w) v += psum[w][tid];
    ps.probs[(int64_t)blockIdx.x * E + tid] = v;
    ps.counts[(int64_t)blockIdx.x * E + tid] = csum[tid];
  }
  if (tid == 0) ps.tokens[blockIdx.x] = nsum;
  if (W == 1) {
    __threadfence_block();
    __syncthreads();
    join_parts<kBThreads, 1>(ps, 1, E, loss, counts, probs, tokens);
  }
}

__global__ __launch_bounds__(kJoinThreads) void k_balance_join(
    void* ws, int W, int E, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ probs, int32_t* __restrict__ tokens) {
  join_parts<kJoinThreads, 16>(parts_of(ws, W, E), W, E, loss, counts, probs, tokens);
}

template <int L, int IT>
__global__ __launch_bounds__(kBThreads) void k_balance_grad(
    const float* __restrict__ dloss, const void* __restrict__ logits, int64_t ld,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens, int T, int E, OutY d) {
  const int tid = threadIdx.x, e0 = tid % L * kEach;
  float n = 0.0f, f[kEach];                           // n: exact up to 2^24, the counts of one call
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int c = counts[e0 + j < E ? e0 + j : E - 1]; // no branch, which would wait for each
    f[j] = e0 + j < E ? (float)c : 0.0f;
    n += f[j];
  }
  n = group_sum<L>(n);                                // sums over many ranks may pass 2^31
#pragma unroll
  for (int j = 0; j < kEach; ++j) f[j] = n > 0.0f ? f[j] / n : 0.0f;
  const int valid = *tokens;
  const float scale = valid > 0 ? *dloss * (float)E / (float)valid : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * (kBThreads / L) + tid / L; t < T;
       t += (int64_t)gridDim.x * (kBThreads / L)) {
    float p[kEach], dot = 0.0f;
    const bool some = softmax4<L, IT>(logits, t * ld, e0, E, p);
#pragma unroll
    for (int j = 0; j < kEach; ++j) dot += p[j] * f[j];
    dot = group_sum<L>(dot);
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (e0 + j < E) d.put(t * E + e0 + j, some ? scale * p[j] * (f[j] - dot) : 0.0f);
  }
}

int64_t moe_balance_ws_bytes(int64_t T, int64_t E) {
  return (int64_t)balance_wgs(T, E) * (2 * E + 1) * 4;
}

#define BGT_LANES(L, CALL)          \
  do {                              \
    switch (L) {                    \
      case 1: CALL(1); break;       \
      case 2: CALL(2); break;       \
      case 4: CALL(4); break;       \
      case 8: CALL(8); break;       \
      case 16: CALL(16); break;     \
      case 32: CALL(32); break;     \
      default: CALL(64); break;     \
    }                               \
  } while (0)

namespace {

template <int IT>
void balance_t(const void* logits, int64_t ld, const int32_t* ids, int T, int E, int k, void* ws,
               float* loss, int32_t* counts, float* probs, int32_t* tokens, hipStream_t stream) {
  const int W = balance_wgs(T, E);
#define BGT_CALL(L)                                                                              \
  hipLaunchKernelGGL((k_balance_parts<L, IT>), dim3(W), dim3(kBThreads), 0, stream, logits, ld, ids, \
                     T, E, k, ws, loss, counts, probs, tokens)
  BGT_LANES(lanes_of(E), BGT_CALL);
#undef BGT_CALL
  if (W > 1)
    hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(kJoinThreads), 0, stream, ws, W, E, loss, counts,
                       probs, tokens);
}

template <int IT>
void balance_grad_t(const float* dloss, const void* logits, int64_t ld, const int32_t* counts,
                    const int32_t* tokens, int T, int E, void* d, hipStream_t stream) {
  const int L = lanes_of(E);
  const int64_t w = ((int64_t)T * L + kBThreads - 1) / kBThreads;
  const int W = (int)(w < 2048 ? w : 2048);
#define BGT_CALL(L)                                                                               \
  hipLaunchKernelGGL((k_balance_grad<L, IT>), dim3(W), dim3(kBThreads), 0, stream, dloss, logits, ld, \
                     counts, tokens, T, E, OutY{d, IT})
  BGT_LANES(L, BGT_CALL);
#undef BGT_CALL
}

}  // namespace

hipError_t launch_moe_balance(const void* logits, int type, int64_t ld, const int32_t* ids,
                              int64_t T, int64_t E, int64_t k, float* loss, int32_t* counts,
                              float* probs, int32_t* tokens, void* ws, hipStream_t stream) {
  if (type == kF32) balance_t<kF32>(logits, ld, ids, (int)T, (int)E, (int)k, ws, loss, counts, probs, tokens, stream);
  else if (type == kF16) balance_t<kF16>(logits, ld, ids, (int)T, (int)E, (int)k, ws, loss, counts, probs, tokens, stream);
  else balance_t<kBF16>(logits, ld, ids, (int)T, (int)E, (int)k, ws, loss, counts, probs, tokens, stream);
  return hipGetLastError();
}

hipError_t launch_moe_balance_backward(const float* dloss, const void* logits, int type, int64_t ld,
                                       const int32_t* counts, const int32_t* tokens, int64_t T,
                                       int64_t E, void* dlogits, hipStream_t stream) {
  if (type == kF32) balance_grad_t<kF32>(dloss, logits, ld, counts, tokens, (int)T, (int)E, dlogits, stream);
  else if (type == kF16) balance_grad_t<kF16>(dloss, logits, ld, counts, tokens, (int)T, (int)E, dlogits, stream);
  else balance_grad_t<kBF16>(dloss, logits, ld, counts, tokens, (int)T, (int)E, dlogits, stream);
  return hipGetLastError();
}

}  // namespace bgt
