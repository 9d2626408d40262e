// Log probabilities of given tokens, entropy and best alternatives of rows of
// logits, and the gradient to the logits.  For a row z of V logits, target y:
//
//   lse  = m + log S,  S = sum_j e_j,  e_j = exp(z_j - m),  m = max_j z_j
//   logp = z_y - lse
//   H    = -sum_j p_j log p_j = log S - S1 / S,  S1 = sum_j e_j (z_j - m)
//   dz_j = dlogp (1[j = y] - p_j) - dH p_j (log p_j + H),  p_j = exp(z_j - lse)
//
// Both directions are bound by the logits' bytes, so a row is read once.  A
// wave holds a chunk of it in registers (64 bf16 or 32 float32 logits a lane),
// takes the chunk's maximum, and adds to S and S1 relative to the largest
// maximum so far: where that moves by d = m - m', S' = e^d S and S1' =
// e^d (S1 + d S).  A wave does short rows alone; the eight waves of a
// workgroup share long ones, and where there are too few rows for the chip,
// several workgroups share a row and a second kernel joins their parts.
//
// The alternatives come from the same registers.  The K-th largest of a wave's
// 64 lane maxima is a bound that at least K of its logits reach and few others
// do; those are put in order by a sort over the lanes.  Where more than 64
// reach it (equal logits), the K best are picked one after another.
//
// Rows may start anywhere: the 16-byte loads are aligned, and the vectors
// that reach past either end of the row are read element by element.
#include <algorithm>
#include <cmath>

#include "lm.hpp"

namespace dpf {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kNoIndex = 0x7fffffff;
constexpr int kR = 8;                       // 16-byte vectors per lane and chunk
constexpr int kWaves = 8;                   // waves that share a long row
constexpr int kTopLanes = 32;               // lanes that hold the alternatives so far
constexpr float kFloor2 = -1000.f;          // below the least exponent: e = 0 there

static_assert(kMaxTopK <= kTopLanes, "one lane per alternative");

// m: maximum; s, s1: sums relative to it, s1 with the difference in powers of
// two (s1 ln 2 is S1).
struct Stats {
  float m, s, s1;
};

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(x) to about two units of the last place of the result whatever |x|: the
// product x log2(e) is rounded by up to |x| units, which the second factor
// makes good.
__device__ __forceinline__ float exp_hw(float x) {
  constexpr float kLog2eLow = 1.92596299e-8f;   // log2(e) - kLog2e
  const float t = x * kLog2e;
  float r = __builtin_fmaf(x, kLog2e, -t);
  r = __builtin_fmaf(x, kLog2eLow, r);
  const float e = exp2_hw(t);
  return e == 0.f ? 0.f : __builtin_fmaf(e, r * kLn2, e);   // x = -inf: r is NaN
}

// The sums relative to `to` instead of `from` (to >= from).
__device__ __forceinline__ void rebase(float from, float to, float& s, float& s1) {
  if (from == to) return;
  if (from == kNegInf) { s = s != s ? s : 0.f; s1 = 0.f; return; }   // nothing yet, or NaN
  const float d = (from - to) * kLog2e, e = exp2_hw(d);
  s1 = e == 0.f ? 0.f : e * (s1 + d * s);
  s *= e;
}

__device__ __forceinline__ Stats merge(Stats a, Stats b) {
  const float m = fmaxf(a.m, b.m);
  rebase(a.m, m, a.s, a.s1);
  rebase(b.m, m, b.s, b.s1);
  return Stats{m, a.s + b.s, a.s1 + b.s1};
}

// Larger value first, then the lower index; (-inf, kNoIndex) is no entry.
__device__ __forceinline__ bool before(float v, int i, float w, int j) {
  return v > w || (v == w && i < j);
}

// The 64 lanes' entries in order, lane 0 the first.
__device__ __forceinline__ void sort_lanes(float& v, int& i) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 2; k <= 64; k *= 2)
#pragma unroll
    for (int j = k / 2; j >= 1; j /= 2) {
      const float w = lane_xor(v, j);
      const int o = lane_xor(i, j);
      const bool first = ((lane & j) == 0) == ((lane & k) == 0);   // keep the better one
      if (before(w, o, v, i) == first) { v = w; i = o; }
    }
}

// The k-th largest of 64 lanes' values.
__device__ __forceinline__ float kth_of_lanes(float v, int k) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int n = 2; n <= 64; n *= 2)
#pragma unroll
    for (int j = n / 2; j >= 1; j /= 2) {
      const float w = lane_xor(v, j);
      const bool most = ((lane & j) == 0) == ((lane & n) == 0);
      v = most ? fmaxf(v, w) : fminf(v, w);
    }
  return __shfl(v, k - 1, 64);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, lane_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += lane_xor(v, o);
  return v;
}

// The chunk as it was loaded: without this the compiler keeps it widened to
// float32 as well, in twice the registers.
template <class Vec>
__device__ __forceinline__ void as_loaded(Vec (&x)[kR]) {
#pragma unroll
  for (int r = 0; r < kR; ++r) asm volatile("" : "+v"(x[r]));
}

// What one wave finds in its part of a row.
template <class E, bool TOP>
struct RowPart {
  static constexpr int kVec = E::kVec;            // logits per 16-byte load
  using S = typename E::storage;
  typedef Raw<E, kVec> Vec;

  Stats st;
  float tv;                                       // lanes 0 .. 31: alternatives so far
  int ti;
  // The vectors [v0, v1) of the row whose first aligned vector is at `z`
  // (`pre` elements before the row), this wave's share of them: vectors
  // v0 + `wave` * 64 + lane and so on, in steps of `waves` * 64.
  // `list`: 64 entries of LDS of this wave's own.
  __device__ __forceinline__ void run(const S* z, int pre, int V, int v0, int v1, int wave,
                                      int waves, int top_k, float2* list) {
    const int lane = threadIdx.x & 63;
    st = Stats{kNegInf, 0.f, 0.f};
    tv = kNegInf;
    ti = kNoIndex;
    float kth = kNegInf;                          // the top_k-th so far
    bool full = false;                            // there are top_k
    const int step = waves * 64;
    const int n = max(0, (v1 - v0 - wave * 64 + step - 1) / step);   // vectors of lane 0
    const int chunks = (n + kR - 1) / kR;
    int done = 0;
    for (int c = 0; c < chunks; ++c) {
      const int now = (n - done + (chunks - c) - 1) / (chunks - c);    // even chunks, <= kR
      Vec x[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= now) continue;
        const int v = v0 + wave * 64 + (done + r) * step + lane;
        const int j = v * kVec - pre;             // first index of the vector
        if (v < v1 && j >= 0 && j + kVec <= V) {
          x[r] = load_raw<E, kVec>(z + (int64_t)v * kVec);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const bool in = v < v1 && j + e >= 0 && j + e < V;
            x[r][e] = in ? z[(int64_t)v * kVec + e] : lowest();
          }
        }
      }
      float lm = kNegInf;
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (r < now)
#pragma unroll
          for (int e = 0; e < kVec; ++e) lm = fmaxf(lm, raw_f32<E, kVec>(x[r], e));
      const float m = fmaxf(st.m, wave_max(lm));
      as_loaded(x);
      rebase(st.m, m, st.s, st.s1);
      const float at = m == kNegInf ? 0.f : m;    // -inf - -inf would be NaN
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (r < now)
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const float d = (raw_f32<E, kVec>(x[r], e) - at) * kLog2e, p = exp2_hw(d);
            st.s += p;
            st.s1 += p * fmaxf(d, kFloor2);       // NaN is kept by s
          }
      st.m = m;
      as_loaded(x);
      if constexpr (TOP) alternatives(x, now, lm, pre, V, v0 + wave * 64 + done * step, v1, step, top_k, list, kth, full);
      done += now;
    }
    st.s = wave_sum(st.s);
    st.s1 = wave_sum(st.s1);
  }

  static __device__ __forceinline__ S lowest() {
    if constexpr (sizeof(S) == 2) return (S)0xff80u;
    else return kNegInf;
  }

  // Adds a chunk's best logits to the alternatives.  Later chunks hold higher
  // indices, so a logit equal to the last alternative comes after it.
  __device__ __forceinline__ void alternatives(const Vec (&x)[kR], int now, float lm, int pre, int V,
                                               int first, int v1, int step, int top_k,
                                               float2* list, float& kth, bool& full) {
    const int lane = threadIdx.x & 63;
    if (full && !(wave_max(lm) > kth)) return;
    float bound = kth_of_lanes(lm, top_k);
    // strictly above the last alternative, if there are enough of them
    const bool above = full && kth >= bound;
    if (above) bound = kth;
    int count = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if (r < now)
{
        float most = raw_f32<E, kVec>(x[r], 0);   // few vectors hold one
#pragma unroll
        for (int e = 1; e < kVec; ++e) most = fmaxf(most, raw_f32<E, kVec>(x[r], e));
        if (__ballot(above ? most > bound : most >= bound) == 0) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float v = raw_f32<E, kVec>(x[r], e);
          uint64_t hit = __ballot(above ? v > bound : v >= bound);
          if (hit != 0) {
            const int w = first + r * step + lane, j = w * kVec - pre + e;
            hit &= __ballot(w < v1 && j >= 0 && j < V);     // not the padding's -inf
            const int to = count + __popcll(hit & ((1ull << lane) - 1ull));
            if (((hit >> lane) & 1) && to < 64) list[to] = make_float2(v, __int_as_float(j));
            count += __popcll(hit);
          }
        }
      }
    if (count <= 64) {
      __builtin_amdgcn_wave_barrier();
      float v = kNegInf;
      int i = kNoIndex;
      if (lane < count) {
        const float2 c = list[lane];
        v = c.x;
        i = __float_as_int(c.y);
      }
      __builtin_amdgcn_wave_barrier();
      if (ti_any()) sort_lanes(v, i);             // the best 32 of these first
      join(v, i);
    } else {
      // Too many equal ones: the best, then the best after it, and so on.
      float bv = 0.f, mv = kNegInf;
      int bi = -1, mi = kNoIndex;
      for (int k = 0; k < top_k; ++k) {
        float cv = kNegInf;
        int ci = kNoIndex;
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (r < now)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              const float v = raw_f32<E, kVec>(x[r], e);
              const int w = first + r * step + lane, j = w * kVec - pre + e;
              if (v == v && w < v1 && j >= 0 && j < V && (k == 0 || before(bv, bi, v, j)) && before(v, j, cv, ci)) {
                cv = v;
                ci = j;
              }
            }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
          const float ov = lane_xor(cv, o);
          const int oi = lane_xor(ci, o);
          if (before(ov, oi, cv, ci)) { cv = ov; ci = oi; }
        }
        if (ci == kNoIndex) break;
        bv = cv;
        bi = ci;
        if (lane == k) { mv = cv; mi = ci; }
      }
      join(mv, mi);
    }
    full = __shfl(ti, top_k - 1, 64) != kNoIndex;
    if (full) kth = __shfl(tv, top_k - 1, 64);
  }

  __device__ __forceinline__ bool ti_any() const { return __ballot((threadIdx.x & 63) < kTopLanes && ti != kNoIndex) != 0; }

  // Takes the entries of all lanes (where there are alternatives already, only
  // the first 32 lanes', the best of them).
  __device__ __forceinline__ void join(float v, int i) {
    const int lane = threadIdx.x & 63;
    if (!ti_any()) {
      tv = v;
      ti = i;
    } else {
      const float up = __shfl(v, lane - kTopLanes, 64);
      const int ui = __shfl(i, lane - kTopLanes, 64);
      if (lane >= kTopLanes) { tv = up; ti = ui; }
    }
    sort_lanes(tv, ti);
    if (lane >= kTopLanes) { tv = kNegInf; ti = kNoIndex; }
  }
};

// The best of `n` entries in memory, by one wave, into lanes 0 .. 31.
__device__ __forceinline__ void best_of(const float2* e, int n, float& v, int& i) {
  const int lane = threadIdx.x & 63;
  v = kNegInf;
  i = kNoIndex;
  if (lane < n) { v = e[lane].x; i = __float_as_int(e[lane].y); }
  sort_lanes(v, i);
  for (int at = 64; at < n; at += 64 - kTopLanes) {
    const int k = at + lane - kTopLanes;
    if (lane >= kTopLanes) {
      v = k < n ? e[k].x : kNegInf;
      i = k < n ? __float_as_int(e[k].y) : kNoIndex;
    }
    sort_lanes(v, i);
  }
}

// One wave writes a row's results (entries in lanes 0 ..).
template <class E>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t n, const Stats& st, float v,
                                          int i, const typename E::storage* z) {
  const int lane = threadIdx.x & 63;
  const float log_s = logf(st.s), lse = st.m + log_s;
  if (lane == 0) {
    if (a.lse != nullptr) a.lse[n] = lse;
    if (a.entropy != nullptr) a.entropy[n] = log_s - kLn2 * (st.s1 / st.s);
    if (a.logp != nullptr) {
      const int64_t b = n / a.T, y = a.targets.at(b, n - b * a.T);
      a.logp[n] = y >= 0 && y < a.V ? E::to_float(z[y]) - lse : 0.f;
    }
  }
  if (lane < a.top_k) {
    a.top_logp[n * a.top_k + lane] = i != kNoIndex ? v - lse : __builtin_nanf("");
    a.top_ids[n * a.top_k + lane] = i != kNoIndex ? i : -1;
  }
}

__device__ __forceinline__ void write_masked(const LogprobArgs& a, int64_t n) {
  const int lane = threadIdx.x & 63;
  if (lane == 0) {
    if (a.logp != nullptr) a.logp[n] = 0.f;
    if (a.entropy != nullptr) a.entropy[n] = 0.f;
    if (a.lse != nullptr) a.lse[n] = 0.f;
  }
  if (lane < a.top_k) {
    a.top_logp[n * a.top_k + lane] = 0.f;
    a.top_ids[n * a.top_k + lane] = -1;
  }
}

template <class E>
__device__ __forceinline__ const typename E::storage* row_of(const Act& z, int64_t T, int64_t n) {
  const int64_t b = n / T;
  return (const typename E::storage*)z.data + b * z.stride_b + (n - b * T) * z.stride_t;
}
// Elements between the 16-byte boundary at or before p and p.
template <class E>
__device__ __forceinline__ int before_aligned(const typename E::storage* p) {
  return (int)(((uintptr_t)p & 15) / sizeof(typename E::storage));
}

// What a workgroup leaves of its part of a split row: the sums, then top_k
// entries.
__host__ __device__ __forceinline__ int part_words(int top_k) { return 4 + 2 * top_k; }

// WAVES waves per row and part; four rows per workgroup with one wave each.
template <class E, int WAVES, bool TOP>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) logprobs_kernel(LogprobArgs a,
                                                                                 int splits) {
  constexpr int kLists = WAVES == 1 ? 4 : WAVES;
  __shared__ float2 lists[kLists][64];
  __shared__ Stats stats[kLists];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int64_t n;
  int part = 0;
  if constexpr (WAVES == 1) {
    n = (int64_t)blockIdx.x * 4 + wave;
    if (n >= a.N) return;
  } else {
    n = blockIdx.x / splits;
    part = blockIdx.x % splits;
  }
  if (a.mask != nullptr && a.mask[n] == 0) {
    if ((WAVES == 1 || wave == 0) && part == 0) write_masked(a, n);
    return;
  }
  const typename E::storage* z = row_of<E>(a.Z, a.T, n);
  const int pre = before_aligned<E>(z), V = (int)a.V;
  const int vecs = (V + pre + E::kVec - 1) / E::kVec;
  const int v0 = (int)((int64_t)vecs * part / splits), v1 = (int)((int64_t)vecs * (part + 1) / splits);
  RowPart<E, TOP> p;
  p.run(z - pre, pre, V, v0, v1, WAVES == 1 ? 0 : wave, WAVES, a.top_k, lists[wave]);
  if constexpr (WAVES == 1) {
    write_row<E>(a, n, p.st, p.tv, p.ti, z);
  } else {
    if (lane == 0) stats[wave] = p.st;
    float2* best = &lists[0][0];
    __syncthreads();                             // the lists are free
    if constexpr (TOP) {
      if (lane < a.top_k) best[wave * a.top_k + lane] = make_float2(p.tv, __int_as_float(p.ti));
      __syncthreads();
    }
    if (wave != 0) return;
    Stats st = stats[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) st = merge(st, stats[w]);
    float v = kNegInf;
    int i = kNoIndex;
    if constexpr (TOP) best_of(best, WAVES * a.top_k, v, i);
    if (splits == 1) {
      write_row<E>(a, n, st, v, i, z);
    } else {
      float* o = (float*)a.ws + (n * splits + part) * part_words(a.top_k);
      if (lane == 0) { o[0] = st.m; o[1] = st.s; o[2] = st.s1; }
      if (lane < a.top_k) ((float2*)(o + 4))[lane] = make_float2(v, __int_as_float(i));
    }
  }
}

// Joins the parts of split rows, one wave per row: the sums in the parts'
// order, the alternatives by order.
template <class E>
__global__ void __launch_bounds__(64) logprobs_join_kernel(LogprobArgs a, int splits) {
  __shared__ float2 best[kTopLanes * 64];
  const int64_t n = blockIdx.x;
  const int lane = threadIdx.x;
  if (a.mask != nullptr && a.mask[n] == 0) return;
  const int words = part_words(a.top_k);
  const float* o = (const float*)a.ws + n * splits * words;
  Stats mine = {kNegInf, 0.f, 0.f};
  if (lane < splits) mine = Stats{o[lane * words], o[lane * words + 1], o[lane * words + 2]};
  for (int k = lane; k < splits * a.top_k; k += 64)
    best[k] = ((const float2*)(o + (k / a.top_k) * words + 4))[k % a.top_k];
  Stats st = {__shfl(mine.m, 0, 64), __shfl(mine.s, 0, 64), __shfl(mine.s1, 0, 64)};
  for (int w = 1; w < splits; ++w)
    st = merge(st, Stats{__shfl(mine.m, w, 64), __shfl(mine.s, w, 64), __shfl(mine.s1, w, 64)});
  __syncthreads();
  float v = kNegInf;
  int i = kNoIndex;
  if (a.top_k > 0) best_of(best, splits * a.top_k, v, i);
  write_row<E>(a, n, st, v, i, row_of<E>(a.Z, a.T, n));
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
constexpr int kGradVecs = 4;               // vectors per thread

// ALIGNED: both rows have the same distance to a multiple of 8 elements.
template <class E, class EO, bool ALIGNED>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(LogprobGradArgs a) {
  constexpr int V = ALIGNED ? 8 : 1;
  const int64_t n = blockIdx.x;
  const typename E::storage* z = row_of<E>(a.Z, a.T, n);
  typename EO::storage* dz = const_cast<typename EO::storage*>(row_of<EO>(a.dZ, a.T, n));
  const int len = (int)a.V;
  const int pre = ALIGNED ? (int)(((uintptr_t)z / sizeof(typename E::storage)) & 7) : 0;
  const int j0 = ((int)blockIdx.y * 256 * kGradVecs + (int)threadIdx.x) * V - pre;
  if ((int)blockIdx.y * 256 * kGradVecs * V - pre >= len) return;
  if (a.mask != nullptr && a.mask[n] == 0) {
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const int j = j0 + k * 256 * V;
      float x[V];
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = 0.f;
      if (j >= 0 && j + V <= len) {
        store_f32<EO, V>(dz + j, x);
      } else {
        for (int e = 0; e < V; ++e)
          if (j + e >= 0 && j + e < len) dz[j + e] = 0;
      }
    }
    return;
  }
  Raw<E, V> x[kGradVecs];
#pragma unroll
  for (int k = 0; k < kGradVecs; ++k) {
    const int j = j0 + k * 256 * V;
    if (j >= 0 && j + V <= len) {
      x[k] = load_raw<E, V>(z + j);
    } else if constexpr (V > 1) {
#pragma unroll
      for (int e = 0; e < V; ++e) x[k][e] = j + e >= 0 && j + e < len ? z[j + e] : (typename E::storage)0;
    } else {
      x[k] = 0;
    }
  }
  const int64_t b = n / a.T;
  const int64_t y = a.targets.data != nullptr ? a.targets.at(b, n - b * a.T) : -1;
  const float up = a.dlogp != nullptr && y >= 0 && y < a.V ? a.dlogp[n] : 0.f;
  const float lse = a.lse[n];
  const bool ent = a.dentropy != nullptr;
  const float dh = ent ? a.dentropy[n] : 0.f, H = ent ? a.entropy[n] : 0.f;
#pragma unroll
  for (int k = 0; k < kGradVecs; ++k) {
    const int j = j0 + k * 256 * V;
    float g[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float lp = raw_f32<E, V>(x[k], e) - lse, p = exp_hw(lp);
      g[e] = (j + e == y ? up : 0.f) - up * p;
      if (ent && p != 0.f) g[e] -= dh * p * (lp + H);
    }
    if (j >= 0 && j + V <= len) {
      store_f32<EO, V>(dz + j, g);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (j + e >= 0 && j + e < len) {
          float one[1] = {g[e]};
          store_f32<EO, 1>(dz + j + e, one);
        }
    }
  }
}

template <class E, class EO>
void grad_v(const LogprobGradArgs& a, hipStream_t s) {
  const bool al = (a.Z.stride_t - a.dZ.stride_t) % 8 == 0 && (a.Z.stride_b - a.dZ.stride_b) % 8 == 0 &&
                  ((uintptr_t)a.Z.data / sizeof(typename E::storage)) % 8 ==
                      ((uintptr_t)a.dZ.data / sizeof(typename EO::storage)) % 8;
  const int64_t per = 256 * kGradVecs * (al ? 8 : 1);
  const dim3 grid((unsigned)a.N, (unsigned)((a.V + (al ? 7 : 0) + per - 1) / per));
  if (al) hipLaunchKernelGGL((logprobs_grad_kernel<E, EO, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((logprobs_grad_kernel<E, EO, false>), grid, dim3(256), 0, s, a);
}

// One wave per row up to this many logits (one chunk of a wave).
template <class E>
constexpr int64_t wave_row() { return 64 * kR * E::kVec; }

// Workgroups per row: 1, or enough for half the compute units where the rows
// are fewer, parts of at least two chunks of a wave each.
int splits_of(const LogprobArgs& a) {
  const int64_t vec = a.dtype == kBF16 ? 8 : 4, most = 64;
  const int64_t parts = a.V / (kWaves * 64 * vec * 2);
  const int64_t want = (device_cus() / 2) / a.N;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(parts, want), most));
}

template <class E, bool TOP>
hipError_t logprobs_e(const LogprobArgs& a, hipStream_t s) {
  if (a.V <= wave_row<E>()) {
    hipLaunchKernelGGL((logprobs_kernel<E, 1, TOP>), dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, a, 1);
    return hipGetLastError();
  }
  const int splits = splits_of(a);
  hipLaunchKernelGGL((logprobs_kernel<E, kWaves, TOP>), dim3((unsigned)(a.N * splits)), dim3(kWaves * 64),
                     0, s, a, splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL(logprobs_join_kernel<E>, dim3((unsigned)a.N), dim3(64), 0, s, a, splits);
  return hipGetLastError();
}

}  // namespace

size_t logprobs_workspace_bytes(const LogprobArgs& a) {
  const int splits = a.V <= (a.dtype == kBF16 ? wave_row<BF16>() : wave_row<F32>()) ? 1 : splits_of(a);
  return splits == 1 ? 0 : (size_t)a.N * splits * part_words(a.top_k) * sizeof(float);
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  timing_begin("token_logprobs", s);
  hipError_t e;
  if (a.dtype == kBF16) e = a.top_k > 0 ? logprobs_e<BF16, true>(a, s) : logprobs_e<BF16, false>(a, s);
  else e = a.top_k > 0 ? logprobs_e<F32, true>(a, s) : logprobs_e<F32, false>(a, s);
  timing_end("token_logprobs", s);
  return e;
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
