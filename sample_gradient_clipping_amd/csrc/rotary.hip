// Norms of queries and keys per head, and their rotation by position, in one
// pass over both tensors:
//
//   n = w x / sqrt(mean(x^2) + eps)                       (with weights)
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),  t = position freqs[j]
//
// for the pairs j of a head: entries (j, j + pairs), or (2 j, 2 j + 1) when
// interleaved; entries past 2 pairs pass through.  Backward, with d the
// rotation's transpose of the output's gradient and r = 1 / sqrt(mean(x^2) + eps):
//
//   dx = r (d w - x r mean(d w x r)),   dw[b] = sum over the heads and positions of sample b of d x r
//
// (per sample, which is what clipping needs).
//
// HBM bounds both passes, so each entry is read and written once, in 16-byte
// pieces.  A lane holds two pieces whose entries are each other's partners (of
// the two halves, or neighbours), so the rotation stays within lanes; the lanes
// of a head add their squares by lane exchanges.  A position's cosines and sines
// serve all of its heads: a workgroup computes them once, into LDS, the angle in
// turns in float64 (in float32 a position of 10^6 would be off by 0.06 radians),
// reduced, then float32.  Rows and their sums are float32 throughout; outputs are
// rounded once.  8x2048, 40x128 bf16: 125 us forward, 200 backward, 5.0 to 5.4 TB/s
// (a large copy: 5.1).
#include "lm.hpp"

#include <algorithm>

namespace dpf {
namespace {

constexpr int kNT = 256;
constexpr int kMaxPairs = kRotaryMaxD / 2;
constexpr int kMaxTokens = 8;

// Where unit u's two pieces of V entries lie, and its first pair (rotated units).
struct Unit {
  int o1, o2, pair;
  bool turns;
};
template <int V>
__device__ __forceinline__ Unit unit_of(const RotaryArgs& a, int u) {
  const int turning = a.pairs / V;
  if (u >= turning) {
    const int o = 2 * a.pairs + (u - turning) * 2 * V;
    return {o, o + V, 0, false};
  }
  if (a.interleaved) return {2 * u * V, 2 * u * V + V, u * V, true};
  return {u * V, a.pairs + u * V, u * V, true};
}

// The rotation of a unit (s = -1: its transpose).
template <int V>
__device__ __forceinline__ void turn(const Unit& u, int interleaved, const float* cs, const float* sn, float s,
                                     float (&x)[V], float (&y)[V]) {
  if (!u.turns) return;
  if (V > 1 && interleaved) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const float c1 = cs[u.pair + k], s1 = s * sn[u.pair + k];
      const float c2 = cs[u.pair + V / 2 + k], s2 = s * sn[u.pair + V / 2 + k];
      const float a = x[2 * k], b = x[2 * k + 1], e = y[2 * k], f = y[2 * k + 1];
      x[2 * k] = a * c1 - b * s1;
      x[2 * k + 1] = b * c1 + a * s1;
      y[2 * k] = e * c2 - f * s2;
      y[2 * k + 1] = f * c2 + e * s2;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float c = cs[u.pair + k], t = s * sn[u.pair + k];
      const float a = x[k], b = y[k];
      x[k] = a * c - b * t;
      y[k] = b * c + a * t;
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int j = 1; j < G; j <<= 1) x += lane_xor(x, j);
  return x;
}

// cos and sin (times the amplitude) of the workgroup's positions into LDS.
__device__ __forceinline__ void angles(const RotaryArgs& a, int64_t n0, int tokens, float* cs, float* sn) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  for (int e = threadIdx.x; e < tokens * a.pairs; e += kNT) {
    const int64_t n = n0 + e / a.pairs;
    const int64_t b = n / a.T, t = n % a.T;
    const double at = a.positions.data == nullptr ? (double)t : (double)a.positions.at(b, t);
    const double turns = at * a.freqs[e % a.pairs] * kInvTwoPi;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    cs[e] = a.amplitude * c;
    sn[e] = a.amplitude * s;
  }
  __syncthreads();
}

template <class E, int V>
__device__ __forceinline__ void load_unit(const typename E::storage* row, const Unit& u, int D, float (&x)[V],
                                          float (&y)[V]) {
  if constexpr (V > 1) {
    load_f32<E, V>(row + u.o1, x);
    load_f32<E, V>(row + u.o2, y);
  } else {
    x[0] = E::to_float(row[u.o1]);
    y[0] = u.o2 < D ? E::to_float(row[u.o2]) : 0.0f;
  }
}
template <class E, int V>
__device__ __forceinline__ void store_unit(typename E::storage* row, const Unit& u, int D, const float (&x)[V],
                                           const float (&y)[V]) {
  store_f32<E, V>(row + u.o1, x);
  if (V > 1 || u.o2 < D) store_f32<E, V>(row + u.o2, y);
}

// G lanes per head row, NU units of 2 V entries each.
template <class E, int V, int G, int NU>
__global__ __launch_bounds__(kNT) void qk_norm_rotary_kernel(RotaryArgs a) {
  typedef typename E::storage S;
  __shared__ float cs[kMaxTokens * kMaxPairs], sn[kMaxTokens * kMaxPairs];
  const int64_t N = a.B * a.T, n0 = (int64_t)blockIdx.x * a.tokens;
  const int tokens = (int)min((int64_t)a.tokens, N - n0);
  angles(a, n0, tokens, cs, sn);
  const int lane = threadIdx.x & 63, g = lane % G, heads = a.Hq + a.Hk;
  const int units = (a.D + 2 * V - 1) / (2 * V);
  const float inv_d = 1.0f / (float)a.D;
  float wq1[NU][V], wq2[NU][V];
  for (int r = threadIdx.x / G; r < tokens * heads; r += kNT / G) {
    const int k = r / heads, hh = r % heads;
    const int64_t n = n0 + k, b = n / a.T, t = n % a.T;
    const bool is_q = hh < a.Hq;
    const Heads& in = is_q ? a.q : a.k;
    const Heads& out = is_q ? a.oq : a.ok;
    const int head = is_q ? hh : hh - a.Hq;
    const S* row = (const S*)in.data + b * in.sb + t * in.st + head * in.sh;
    S* to = (S*)out.data + b * out.sb + t * out.st + head * out.sh;
    const bool live = a.mask == nullptr || a.mask[n] != 0;
    const float* w = is_q ? a.wq : a.wk;
    float x[NU][V], y[NU][V], sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const Unit u = unit_of<V>(a, g + i * G);
      const bool in_row = g + i * G < units;
#pragma unroll
      for (int e = 0; e < V; ++e) x[i][e] = y[i][e] = wq1[i][e] = wq2[i][e] = 0.0f;
      if (live && in_row) {
        load_unit<E, V>(row, u, a.D, x[i], y[i]);
        if (w != nullptr) load_unit<F32, V>(w, u, a.D, wq1[i], wq2[i]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) sq = fmaf(x[i][e], x[i][e], fmaf(y[i][e], y[i][e], sq));
    }
    if (w != nullptr) {
      const float f = 1.0f / sqrtf(fmaf(group_sum<G>(sq), inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[i][e] *= f * wq1[i][e];
          y[i][e] *= f * wq2[i][e];
        }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (g + i * G >= units) continue;
      const Unit u = unit_of<V>(a, g + i * G);
      if (live) turn<V>(u, a.interleaved, cs + k * a.pairs, sn + k * a.pairs, 1.0f, x[i], y[i]);
      store_unit<E, V>(to, u, a.D, x[i], y[i]);
    }
  }
}

// Backward: a workgroup takes positions of one sample, all its queries' heads,
// then all its keys', and leaves their sums of d x r in part[workgroup][2][D]
// (lanes that hold the same entries are added in a fixed order through LDS).
template <class E, int V, int G, int NU>
__global__ __launch_bounds__(kNT) void qk_norm_rotary_backward_kernel(RotaryArgs a, int chunks) {
  typedef typename E::storage S;
  __shared__ float cs[kMaxTokens * kMaxPairs], sn[kMaxTokens * kMaxPairs];
  __shared__ float sums[kNT / 64][G == 64 ? 64 * NU * 2 : G * 2 * V];
  const int64_t b = blockIdx.x / chunks, t0 = (int64_t)(blockIdx.x % chunks) * a.tokens;
  const int tokens = (int)min((int64_t)a.tokens, a.T - t0);
  angles(a, b * a.T + t0, tokens, cs, sn);
  const int lane = threadIdx.x & 63, g = lane % G;
  const int units = (a.D + 2 * V - 1) / (2 * V);
  const float inv_d = 1.0f / (float)a.D;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const Heads& in = which == 0 ? a.q : a.k;
    const Heads& grad = which == 0 ? a.gq : a.gk;
    const Heads& out = which == 0 ? a.oq : a.ok;
    const int heads = which == 0 ? a.Hq : a.Hk;
    const float* w = which == 0 ? a.wq : a.wk;
    float w1[NU][V], w2[NU][V], dw1[NU][V], dw2[NU][V];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) w1[i][e] = w2[i][e] = dw1[i][e] = dw2[i][e] = 0.0f;
      if (w != nullptr && g + i * G < units)
        load_unit<F32, V>(w, unit_of<V>(a, g + i * G), a.D, w1[i], w2[i]);
    }
    for (int r = threadIdx.x / G; r < tokens * heads; r += kNT / G) {
      const int k = r / heads, head = r % heads;
      const int64_t t = t0 + k;
      const S* row = (const S*)in.data + b * in.sb + t * in.st + head * in.sh;
      const S* dy = (const S*)grad.data + b * grad.sb + t * grad.st + head * grad.sh;
      S* to = (S*)out.data + b * out.sb + t * out.st + head * out.sh;
      const bool live = a.mask == nullptr || a.mask[b * a.T + t] != 0;
      float x[NU][V], y[NU][V], d1[NU][V], d2[NU][V], sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const Unit u = unit_of<V>(a, g + i * G);
#pragma unroll
        for (int e = 0; e < V; ++e) x[i][e] = y[i][e] = d1[i][e] = d2[i][e] = 0.0f;
        if (live && g + i * G < units) {
          load_unit<E, V>(dy, u, a.D, d1[i], d2[i]);
          if (w != nullptr) load_unit<E, V>(row, u, a.D, x[i], y[i]);
          turn<V>(u, a.interleaved, cs + k * a.pairs, sn + k * a.pairs, -1.0f, d1[i], d2[i]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sq = fmaf(x[i][e], x[i][e], fmaf(y[i][e], y[i][e], sq));
      }
      if (w != nullptr) {
        const float f = 1.0f / sqrtf(fmaf(group_sum<G>(sq), inv_d, a.eps));
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x[i][e] *= f;
            y[i][e] *= f;
            dw1[i][e] = fmaf(d1[i][e], x[i][e], dw1[i][e]);
            dw2[i][e] = fmaf(d2[i][e], y[i][e], dw2[i][e]);
            d1[i][e] *= w1[i][e];
            d2[i][e] *= w2[i][e];
            dot = fmaf(d1[i][e], x[i][e], fmaf(d2[i][e], y[i][e], dot));
          }
        dot = group_sum<G>(dot) * inv_d;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            // a masked row's zeros, whatever the weights hold
            d1[i][e] = live ? f * (d1[i][e] - dot * x[i][e]) : 0.0f;
            d2[i][e] = live ? f * (d2[i][e] - dot * y[i][e]) : 0.0f;
          }
      }
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (g + i * G < units) store_unit<E, V>(to, unit_of<V>(a, g + i * G), a.D, d1[i], d2[i]);
    }
    if (w == nullptr) continue;
    // rows of a wave, then the waves, in order
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = G; j < 64; j <<= 1) {
          dw1[i][e] += lane_xor(dw1[i][e], j);
          dw2[i][e] += lane_xor(dw2[i][e], j);
        }
        if (lane < G) {
          float* s = sums[threadIdx.x >> 6] + (g + i * G) * 2 * V;
          s[e] = dw1[i][e];
          s[V + e] = dw2[i][e];
        }
      }
    __syncthreads();
    for (int e = threadIdx.x; e < units * 2 * V; e += kNT) {
      const Unit u = unit_of<V>(a, e / (2 * V));
      const int k = e % (2 * V), d = k < V ? u.o1 + k : u.o2 + k - V;
      float s = 0.0f;
#pragma unroll
      for (int wv = 0; wv < kNT / 64; ++wv) s += sums[wv][e];
      if (d < a.D) a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
    }
    __syncthreads();
  }
}

// dw[b][d] = the chunks' sums: kSlices threads per entry, each every kSlices-th
// chunk, then their sums in order.  Workgroups in rows of kRowOfGroups: one dimension
// of a launch holds fewer than 2^32 threads, and 2^20 samples of 128 entries need as many.
constexpr int64_t kRowOfGroups = 1 << 23;
constexpr int kSlices = 16, kEntries = kNT / kSlices;
__global__ __launch_bounds__(kNT) void qk_norm_weights_kernel(RotaryArgs a, int chunks) {
  __shared__ float sums[kSlices][kEntries];
  const int x = threadIdx.x % kEntries, k = threadIdx.x / kEntries;
  const int64_t e = (blockIdx.y * kRowOfGroups + blockIdx.x) * kEntries + x, b = e / (2 * a.D);
  const int i = (int)(e % (2 * a.D));
  float s = 0.0f;
  if (b < a.B) {
    const float* from = a.part + b * chunks * 2 * a.D + i;
#pragma unroll 8
    for (int c = k; c < chunks; c += kSlices) s += from[(int64_t)c * 2 * a.D];
  }
  sums[k][x] = s;
  __syncthreads();
  if (b >= a.B || k != 0) return;
#pragma unroll
  for (int j = 1; j < kSlices; ++j) s += sums[j][x];
  (i < a.D ? a.dwq : a.dwk)[b * a.D + i % a.D] = s;
}

int64_t chunks_of(const RotaryArgs& a) { return (a.T + a.tokens - 1) / a.tokens; }

template <class E, int V, int G, int NU>
hipError_t rotary_g(const RotaryArgs& a, bool backward, hipStream_t s) {
  if (!backward) {
    hipLaunchKernelGGL((qk_norm_rotary_kernel<E, V, G, NU>),
                       dim3((unsigned)((a.B * a.T + a.tokens - 1) / a.tokens)), dim3(kNT), 0, s, a);
  } else {
    hipLaunchKernelGGL((qk_norm_rotary_backward_kernel<E, V, G, NU>), dim3((unsigned)(a.B * chunks_of(a))),
                       dim3(kNT), 0, s, a, (int)chunks_of(a));
  }
  return hipGetLastError();
}

template <class E, int V>
hipError_t rotary_v(const RotaryArgs& a, bool backward, hipStream_t s) {
  const int units = a.D / (2 * V);
  if (units <= 4) return rotary_g<E, V, 4, 1>(a, backward, s);
  if (units <= 8) return rotary_g<E, V, 8, 1>(a, backward, s);
  if (units <= 16) return rotary_g<E, V, 16, 1>(a, backward, s);
  return rotary_g<E, V, 32, 1>(a, backward, s);
}

hipError_t rotary(const RotaryArgs& a, bool backward, hipStream_t s) {
  if (a.dtype == kBF16) {
    if (a.width == 8) return rotary_v<BF16, 8>(a, backward, s);
    if (a.width == 4) return rotary_v<BF16, 4>(a, backward, s);
    return rotary_g<BF16, 1, 64, 2>(a, backward, s);
  }
  if (a.width == 4) return rotary_v<F32, 4>(a, backward, s);
  return rotary_g<F32, 1, 64, 2>(a, backward, s);
}

bool pieces(const Heads& h, int V, int es, int64_t D) {
  return ((uintptr_t)h.data & (uintptr_t)(V * es - 1)) == 0 && h.sb % V == 0 && h.st % V == 0 &&
         h.sh % V == 0 && D % (2 * V) == 0;
}

}  // namespace

size_t rotary_plan(RotaryArgs& a, bool backward) {
  const int es = a.dtype == kBF16 ? 2 : 4;
  a.width = 1;
  for (int V = 16 / es; V >= 4 && a.width == 1; V /= 2) {
    bool ok = (2 * a.pairs) % (2 * V) == 0;
    for (const Heads* h : {&a.q, &a.k, &a.oq, &a.ok}) ok = ok && pieces(*h, V, es, a.D);
    if (backward) ok = ok && pieces(a.gq, V, es, a.D) && pieces(a.gk, V, es, a.D);
    for (const float* w : {a.wq, a.wk}) ok = ok && ((uintptr_t)w & 15) == 0;
    if (ok) a.width = V;
  }
  const int64_t N = a.B * a.T;
  if (!backward) {
    // several positions per workgroup where their heads are few and workgroups many
    const int heads = a.Hq + a.Hk, rows = a.width == 1 ? 4 : kNT / std::max(4, a.D / (2 * a.width));
    a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxTokens, 2 * rows / heads, N / 1024}));
    return 0;
  }
  a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxTokens, a.T, N / 1024}));
  return a.wq == nullptr ? 0 : (size_t)(a.B * chunks_of(a) * 2 * a.D);
}

hipError_t launch_qk_norm_rotary(const RotaryArgs& a, hipStream_t s) {
  timing_begin("qk_norm_rotary", s);
  const hipError_t e = rotary(a, false, s);
  timing_end("qk_norm_rotary", s);
  return e;
}

hipError_t launch_qk_norm_rotary_backward(const RotaryArgs& a, hipStream_t s) {
  timing_begin("qk_norm_rotary_backward", s);
  const hipError_t e = rotary(a, true, s);
  timing_end("qk_norm_rotary_backward", s);
  if (e != hipSuccess || a.wq == nullptr) return e;
  timing_begin("qk_norm_weights", s);
  const int64_t groups = (a.B * 2 * a.D + kEntries - 1) / kEntries;
  hipLaunchKernelGGL(qk_norm_weights_kernel,
                     dim3((unsigned)std::min(groups, kRowOfGroups), (unsigned)((groups + kRowOfGroups - 1) / kRowOfGroups)),
                     dim3(kNT), 0, s, a, (int)chunks_of(a));
  timing_end("qk_norm_weights", s);
  return hipGetLastError();
}

}  // namespace dpf
