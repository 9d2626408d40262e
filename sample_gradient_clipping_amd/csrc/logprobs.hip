// Log probabilities of given tokens, entropy and best alternatives of rows of
// logits, and the gradient to the logits.  For a row z of V logits, target y:
//
//   lse  = m + log S,  S = sum_j e_j,  e_j = exp(z_j - m),  m = max_j z_j
//   logp = z_y - lse
//   H    = -sum_j p_j log p_j = log S - (sum_j e_j (z_j - m)) / S
//   dz_j = dlogp (1[j = y] - p_j) - dH p_j (log p_j + H),  p_j = exp(z_j - lse)
//
// The maximum and both sums are carried together (float32), one pass over the
// row: when the maximum moves by d = m - m', S' = e^d S and the weighted sum
// S1' = e^d (S1 + d S).  A term with e_j = 0 adds nothing to S1, so a logit of
// -inf is a token of probability 0 and not NaN.
#include <cmath>

#include "lm.hpp"

namespace dpf {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

struct Stats {
  float m, s, s1;
};

__device__ __forceinline__ Stats merge(const Stats& a, const Stats& b) {
  Stats r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m == r.m ? 0.f : a.m - r.m, db = b.m == r.m ? 0.f : b.m - r.m;
  const float ea = expf(da), eb = expf(db);   // 0 where that side is empty (da = -inf)
  r.s = ea * a.s + eb * b.s;
  r.s1 = (ea == 0.f ? 0.f : ea * (a.s1 + da * a.s)) + (eb == 0.f ? 0.f : eb * (b.s1 + db * b.s));
  return r;
}

__device__ __forceinline__ void add(Stats& a, float z) {
  if (z > a.m) {
    const float d = a.m - z, e = expf(d);
    a.s1 = e == 0.f ? 0.f : e * (a.s1 + d * a.s);
    a.s = e * a.s;
    a.m = z;
  }
  const float d = z == a.m ? z - z : z - a.m;   // infinities: inf - inf is NaN, as it should be
  if (z == kNegInf) return;
  const float e = expf(d);
  a.s += e;
  if (e != 0.f) a.s1 += e * d;
}

// (value, index) order of the alternatives: larger value first, then lower index.
__device__ __forceinline__ bool before(float v, int i, float w, int j) {
  return i >= 0 && (j < 0 || v > w || (v == w && i < j));
}

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / 64;

template <class E, int V>
__global__ void __launch_bounds__(kRowThreads) logprobs_kernel(LogprobArgs a) {
  __shared__ Stats ws[kRowWaves];
  __shared__ float wv[kRowWaves];
  __shared__ int wi[kRowWaves];
  const int64_t n = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (a.mask != nullptr && a.mask[n] == 0) {
    if (tid == 0) {
      if (a.logp != nullptr) a.logp[n] = 0.f;
      if (a.entropy != nullptr) a.entropy[n] = 0.f;
      if (a.lse != nullptr) a.lse[n] = 0.f;
    }
    if (tid < a.top_k) {
      a.top_logp[n * a.top_k + tid] = 0.f;
      a.top_ids[n * a.top_k + tid] = -1;
    }
    return;
  }
  const int64_t b = n / a.T, t = n - b * a.T;
  const typename E::storage* z =
      (const typename E::storage*)a.Z.data + b * a.Z.stride_b + t * a.Z.stride_t;
  Stats st = {kNegInf, 0.f, 0.f};
  for (int64_t j = (int64_t)tid * V; j < a.V; j += kRowThreads * V) {
    float x[V];
    load_f32<E, V>(z + j, x);
#pragma unroll
    for (int k = 0; k < V; ++k) add(st, x[k]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    Stats other = {__shfl_xor(st.m, o, 64), __shfl_xor(st.s, o, 64), __shfl_xor(st.s1, o, 64)};
    // the lower lane's side first in both, so that both compute the same
    st = (lane & o) ? merge(other, st) : merge(st, other);
  }
  if (lane == 0) ws[wave] = st;
  __syncthreads();
  st = ws[0];
  for (int w = 1; w < kRowWaves; ++w) st = merge(st, ws[w]);
  const float lse = st.m + logf(st.s);
  if (tid == 0) {
    if (a.lse != nullptr) a.lse[n] = lse;
    if (a.entropy != nullptr) a.entropy[n] = logf(st.s) - st.s1 / st.s;
    if (a.logp != nullptr) {
      const int64_t y = a.targets.at(b, t);
      a.logp[n] = y >= 0 && y < a.V ? E::to_float(z[y]) - lse : 0.f;
    }
  }
  float lv = 0.f;
  int li = -1;                                 // the last alternative found
  for (int q = 0; q < a.top_k; ++q) {
    float bv = kNegInf;
    int bi = -1;
    for (int64_t j = (int64_t)tid * V; j < a.V; j += kRowThreads * V) {
      float x[V];
      load_f32<E, V>(z + j, x);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int i = (int)(j + k);
        if (x[k] == x[k] && (q == 0 || (li >= 0 && before(lv, li, x[k], i))) && before(x[k], i, bv, bi)) {
          bv = x[k];
          bi = i;
        }
      }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const float ov = __shfl_xor(bv, o, 64);
      const int oi = __shfl_xor(bi, o, 64);
      if (before(ov, oi, bv, bi)) { bv = ov; bi = oi; }
    }
    __syncthreads();
    if (lane == 0) { wv[wave] = bv; wi[wave] = bi; }
    __syncthreads();
    lv = wv[0];
    li = wi[0];
    for (int w = 1; w < kRowWaves; ++w)
      if (before(wv[w], wi[w], lv, li)) { lv = wv[w]; li = wi[w]; }
    if (tid == 0) {
      a.top_logp[n * a.top_k + q] = li >= 0 ? lv - lse : __builtin_nanf("");
      a.top_ids[n * a.top_k + q] = li;
    }
  }
}

template <class E, class EO, int V>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(LogprobGradArgs a) {
  const int64_t n = blockIdx.x;
  const int64_t j = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
  if (j >= a.V) return;
  const int64_t b = n / a.T, t = n - b * a.T;
  typename EO::storage* dz =
      (typename EO::storage*)a.dZ.data + b * a.dZ.stride_b + t * a.dZ.stride_t + j;
  float x[V];
  if (a.mask != nullptr && a.mask[n] == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = 0.f;
    store_f32<EO, V>(dz, x);
    return;
  }
  load_f32<E, V>((const typename E::storage*)a.Z.data + b * a.Z.stride_b + t * a.Z.stride_t + j, x);
  const int64_t y = a.targets.data != nullptr ? a.targets.at(b, t) : -1;
  const float up = a.dlogp != nullptr && y >= 0 && y < a.V ? a.dlogp[n] : 0.f;
  const float lse = a.lse[n];
  const float dh = a.dentropy != nullptr ? a.dentropy[n] : 0.f;
  const float H = a.dentropy != nullptr ? a.entropy[n] : 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float lp = x[k] - lse, p = expf(lp);
    float g = (j + k == y ? up : 0.f) - up * p;
    if (a.dentropy != nullptr && p != 0.f) g -= dh * p * (lp + H);
    x[k] = g;
  }
  store_f32<EO, V>(dz, x);
}

int vec_of(const Act& z, int64_t V) {
  if (V % 8 == 0 && z.stride_t % 8 == 0 && z.stride_b % 8 == 0) return 8;
  if (V % 4 == 0 && z.stride_t % 4 == 0 && z.stride_b % 4 == 0) return 4;
  return 1;
}

template <class E, class EO>
void grad_v(const LogprobGradArgs& a, hipStream_t s) {
  const int v1 = vec_of(a.Z, a.V), v2 = vec_of(a.dZ, a.V), V = v1 < v2 ? v1 : v2;
  const dim3 grid((unsigned)a.N, (unsigned)((a.V + 256 * V - 1) / (256 * V)));
  if (V == 8) hipLaunchKernelGGL((logprobs_grad_kernel<E, EO, 8>), grid, dim3(256), 0, s, a);
  else if (V == 4) hipLaunchKernelGGL((logprobs_grad_kernel<E, EO, 4>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((logprobs_grad_kernel<E, EO, 1>), grid, dim3(256), 0, s, a);
}

template <class E>
void logprobs_v(const LogprobArgs& a, hipStream_t s) {
  const int V = vec_of(a.Z, a.V);
  const dim3 grid((unsigned)a.N);
  if (V == 8) hipLaunchKernelGGL((logprobs_kernel<E, 8>), grid, dim3(kRowThreads), 0, s, a);
  else if (V == 4) hipLaunchKernelGGL((logprobs_kernel<E, 4>), grid, dim3(kRowThreads), 0, s, a);
  else hipLaunchKernelGGL((logprobs_kernel<E, 1>), grid, dim3(kRowThreads), 0, s, a);
}

}  // namespace

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  timing_begin("token_logprobs", s);
  if (a.dtype == kBF16) logprobs_v<BF16>(a, s);
  else logprobs_v<F32>(a, s);
  timing_end("token_logprobs", s);
  return hipGetLastError();
}

hipError_t launch_token_logprobs_backward(const LogprobGradArgs& a, hipStream_t s) {
  timing_begin("token_logprobs_backward", s);
  if (a.dtype == kBF16) {
    if (a.out_dtype == kBF16) grad_v<BF16, BF16>(a, s);
    else grad_v<BF16, F32>(a, s);
  } else {
    if (a.out_dtype == kBF16) grad_v<F32, BF16>(a, s);
    else grad_v<F32, F32>(a, s);
  }
  timing_end("token_logprobs_backward", s);
  return hipGetLastError();
}

}  // namespace dpf
