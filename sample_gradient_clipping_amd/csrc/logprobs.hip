// Log probabilities of given tokens, entropy and best alternatives of rows of
// logits, and the gradient to the logits.  For a row z of V logits, target y:
//
//   lse  = m + log S,  S = sum_j e_j,  e_j = exp(z_j - m),  m = max_j z_j
//   logp = z_y - lse = (z_y - m) - log S
//   H    = -sum_j p_j log p_j = log S - S1 / S,  S1 = sum_j e_j (z_j - m)
//   dz_j = dlogp (1[j = y] - p_j) - dH p_j (log p_j + H),  p_j = exp(z_j - lse)
//
// Both directions are bound by the logits' bytes, so a row is read once.  A
// wave holds a chunk of it in registers (64 bf16 or 32 float32 logits a lane),
// takes the chunk's maximum, and adds to S and S1 relative to the largest
// maximum so far: where that moves by d = m - m', S' = e^d S and S1' =
// e^d (S1 + d S).  A wave does short rows alone, four or eight waves of a
// workgroup share long ones, and where there are too few rows for the chip,
// several workgroups share a row and a second kernel joins their parts.
//
// The alternatives come from the same registers.  The K-th largest of a wave's
// 64 lane maxima is a bound that at least K of its logits reach; the largest
// bound of any wave so far is in LDS, and the few logits that reach it are
// listed there.  What reaches the last bound of all is put in order by a sort
// over the lanes.  Which logits are listed on the way depends on the waves'
// pace, the result does not.  Where more than 64 of a chunk reach the bound
// (equal logits), the chunk is read again and the K best are picked one after
// another.
//
// Rows may start anywhere: the 16-byte loads are aligned, and the vectors
// that reach past either end of the row are read element by element.
//
// What it costs (MI355X).  16384 rows of 32000 bf16 logits: 181 to 186 us, 5.7 TB/s;
// with five alternatives 267 (their instructions bound it then: a bound and a
// scan per chunk of a wave), 2052 float32 rows of 50257 with eight 101 (4.1
// TB/s).  16384 float32 rows of 4096: 44, with five 59 us.  One row of
// 32000 with five: 11 us in one workgroup, most of it the latency of a chain
// of loads, maximum, bound, list and sort.  The gradient: 16384 x 32000 bf16
// 424 us (4.9 TB/s read and written, a copy's rate), 2052 x 50257 float32, half
// the rows masked, 127 (5.0 TB/s).
#include <algorithm>
#include <cmath>

#include "lm.hpp"

namespace dpf {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kR = 8;                       // 16-byte vectors per lane and chunk
constexpr int kWaves = 8;                   // waves that share a long row, at most
constexpr int kTopLanes = 32;               // lanes that hold the best so far in a sort of many
constexpr int kListed = 128;                // a wave's list: up to 64 entries and a chunk's 64
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

// Unsigned integers in the order of the floats (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ (u >> 31 != 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ (u >> 31 != 0 ? 0x80000000u : 0xffffffffu));
}

// An alternative as one number: the larger logit is the larger, and of equal
// ones that with the lower index.  0 is no alternative.
__device__ __forceinline__ uint64_t entry(float v, int i) {
  return (uint64_t)ordered(v) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(uint64_t e) { return from_ordered((uint32_t)(e >> 32)); }
__device__ __forceinline__ int index_of(uint64_t e) { return (int)~(uint32_t)e; }

__device__ __forceinline__ uint64_t entry_xor(uint64_t e, int o) {
  const uint32_t hi = (uint32_t)lane_xor((int)(e >> 32), o), lo = (uint32_t)lane_xor((int)(uint32_t)e, o);
  return (uint64_t)hi << 32 | lo;
}

// The 64 lanes' entries in order, lane 0 the first.
__device__ __forceinline__ uint64_t sort_lanes(uint64_t e) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 2; k <= 64; k *= 2)
#pragma unroll
    for (int j = k / 2; j >= 1; j /= 2) {
      const uint64_t o = entry_xor(e, j);
      const bool most = ((lane & j) == 0) == ((lane & k) == 0);   // keep the better one
      e = (o > e) == most ? o : e;
    }
  return e;
}

// A value that at least k of the 64 lanes' reach, k <= 32: the k-th largest of
// the 64, or for k <= 8 of the maxima of four lanes each, in half the steps.
__device__ __forceinline__ float kth_of_lanes(float v, int k) {
  const int lane = threadIdx.x & 63;
  const auto step = [&](int j, int n) {
    const float w = lane_xor(v, j);
    const bool most = ((lane & j) == 0) == ((lane & n) == 0);
    v = most ? fmaxf(v, w) : fminf(v, w);
  };
  if (k <= 8) {
    v = fmaxf(v, lane_xor(v, 32));
    v = fmaxf(v, lane_xor(v, 16));
#pragma unroll
    for (int n = 2; n <= 16; n *= 2)
#pragma unroll
      for (int j = n / 2; j >= 1; j /= 2) step(j, n == 16 ? 64 : n);
  } else {
#pragma unroll
    for (int n = 2; n <= 64; n *= 2)
#pragma unroll
      for (int j = n / 2; j >= 1; j /= 2) step(j, n);
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

// The best of `n` entries in memory, in order, by one wave: the first 32 lanes'.
__device__ __forceinline__ uint64_t best_of(const uint64_t* of, int n) {
  const int lane = threadIdx.x & 63;
  uint64_t e = lane < n ? of[lane] : 0;
  int at = 64;
  for (;;) {
    e = sort_lanes(e);
    if (at >= n) return e;
    const int k = at + lane - kTopLanes;
    if (lane >= kTopLanes) e = k < n ? of[k] : 0;
    at += 64 - kTopLanes;
  }
}

// What one wave finds in its part of a row.
template <class E, bool TOP>
struct RowPart {
  static constexpr int kVec = E::kVec;            // logits per 16-byte load
  using S = typename E::storage;
  typedef Raw<E, kVec> Vec;

  const S* z;                                     // the row's first aligned vector,
  int pre, V, v1;                                 // `pre` elements before the row
  int step;                                       // vectors from one of a lane's to its next
  int top_k;
  uint64_t* list;                                 // kListed entries of this wave's own
  uint32_t* bound;                                // ordered(the row's bound so far)

  Stats st;
  int count;                                      // entries in the list, <= 64 between chunks
  float kth;                                      // top_k of them reach this,
  bool full;                                      // if there are so many

  // This wave's share of the vectors [v0, v1): v0 + `wave` * 64 + lane and so
  // on, in steps of `waves` * 64.
  __device__ __forceinline__ void run(int v0, int wave, int waves) {
    const int lane = threadIdx.x & 63;
    st = Stats{kNegInf, 0.f, 0.f};
    count = 0;
    kth = kNegInf;
    full = false;
    step = waves * 64;
    const int n = max(0, (v1 - v0 - wave * 64 + step - 1) / step);   // vectors of lane 0
    const int chunks = (n + kR - 1) / kR;
    int done = 0;
    for (int c = 0; c < chunks; ++c) {
      const int now = (n - done + (chunks - c) - 1) / (chunks - c);    // even chunks, <= kR
      const int first = v0 + wave * 64 + done * step + lane;
      Vec x[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= now) continue;
        const int v = first + r * step;
        const int j = v * kVec - pre;             // first index of the vector
        if (v < v1 && j >= 0 && j + kVec <= V) {
          x[r] = load_raw<E, kVec>(z + (int64_t)v * kVec);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) x[r][e] = inside(v, e) ? z[(int64_t)v * kVec + e] : lowest();
        }
      }
      float lm = kNegInf;
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (r < now)
#pragma unroll
          for (int e = 0; e < kVec; ++e) lm = fmaxf(lm, raw_f32<E, kVec>(x[r], e));
      const float most = wave_max(lm), m = fmaxf(st.m, most);
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
      if constexpr (TOP) {
        as_loaded(x);
        alternatives(x, now, lm, most, first);
      }
      done += now;
    }
    st.s = wave_sum(st.s);
    st.s1 = wave_sum(st.s1);
  }

  // Element e of vector v is this part's.
  __device__ __forceinline__ bool inside(int v, int e) const {
    const int j = v * kVec - pre + e;
    return v < v1 && j >= 0 && j < V;
  }

  static __device__ __forceinline__ S lowest() {
    if constexpr (sizeof(S) == 2) return (S)0xff80u;
    else return kNegInf;
  }

  __device__ __forceinline__ float bound_now() const {
    return from_ordered(*(volatile const uint32_t*)bound);
  }
  __device__ __forceinline__ void raise_bound(float b) {
    if ((threadIdx.x & 63) == 0) atomicMax(bound, ordered(b));
  }

  // Lists a chunk's logits that reach the bound.  Later chunks hold higher
  // indices, so where top_k entries of this wave's reach it already, a logit
  // equal to it comes after them.
  __device__ __forceinline__ void alternatives(const Vec (&x)[kR], int now, float lm, float most,
                                               int first) {
    const int lane = threadIdx.x & 63;
    float b = bound_now();
    if (most < b || (full && kth == b && !(most > b))) return;
    const float of_chunk = kth_of_lanes(lm, top_k);
    if (of_chunk > b) {
      raise_bound(of_chunk);
      b = bound_now();                            // another wave's may be higher by now
      if (most < b) return;
    }
    const bool above = full && kth == b;
    int n = 0;                                    // that reach it
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if (r < now) {
        float vm = raw_f32<E, kVec>(x[r], 0);     // few vectors hold one
#pragma unroll
        for (int e = 1; e < kVec; ++e) vm = fmaxf(vm, raw_f32<E, kVec>(x[r], e));
        if (__ballot(above ? vm > b : vm >= b) == 0) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float v = raw_f32<E, kVec>(x[r], e);
          uint64_t hit = __ballot(above ? v > b : v >= b);
          if (hit != 0) {
            hit &= __ballot(inside(first + r * step, e));     // not the padding's -inf
            const int to = n + __popcll(hit & ((1ull << lane) - 1ull));
            if (((hit >> lane) & 1) && to < 64)
              list[count + to] = entry(v, (first + r * step) * kVec - pre + e);
            n += __popcll(hit);
          }
        }
      }
    __builtin_amdgcn_wave_barrier();
    const bool fits = n <= 64;
    if (fits) {
      count += n;
      if (n >= top_k) { full = true; kth = b; }
    }
    if (count > (fits ? 64 : 64 - top_k)) keep_best();
    if (!fits) pick(now, first);
  }

  // Shortens the list to its best top_k entries.
  __device__ __forceinline__ void keep_best() {
    const int lane = threadIdx.x & 63;
    const uint64_t e = best_of(list, count);
    __builtin_amdgcn_wave_barrier();
    if (lane < top_k) list[lane] = e;
    __builtin_amdgcn_wave_barrier();
    count = top_k;                                // it was longer
    full = true;
    kth = __shfl(value_of(e), top_k - 1, 64);
    raise_bound(kth);
  }

  // Too many equal ones: the best of the chunk, then the best after it, and so on.
  __device__ __forceinline__ void pick(int now, int first) {
    const int lane = threadIdx.x & 63;
    uint64_t last = ~0ull;
    int k = 0;
    for (; k < top_k; ++k) {
      uint64_t c = 0;
      for (int r = 0; r < now; ++r) {
        const int w = first + r * step;
#pragma unroll 1
        for (int e = 0; e < kVec; ++e) {
          if (!inside(w, e)) continue;
          const float v = E::to_float(z[(int64_t)w * kVec + e]);
          const uint64_t o = v == v ? entry(v, w * kVec - pre + e) : 0;
          if (o < last && o > c) c = o;
        }
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) {
        const uint64_t w = entry_xor(c, o);
        c = w > c ? w : c;
      }
      if (c == 0) break;
      last = c;
      if (lane == 0) list[count + k] = c;
    }
    __builtin_amdgcn_wave_barrier();
    count += k;
    if (k == top_k) {
      full = true;
      kth = value_of(last);
      raise_bound(kth);
    }
  }
};

// One wave writes a row's results (entries in lanes 0 ..).  Log probabilities are
// taken from the maximum, not from lse: that is rounded at the logits' size, and
// an offset common to a row's logits would show in them.
template <class E>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t n, const Stats& st, uint64_t e,
                                          const typename E::storage* z) {
  const int lane = threadIdx.x & 63;
  const float log_s = logf(st.s);
  if (lane == 0) {
    if (a.lse != nullptr) a.lse[n] = st.m + log_s;
    if (a.entropy != nullptr) a.entropy[n] = log_s - kLn2 * (st.s1 / st.s);
    if (a.logp != nullptr) {
      const int64_t b = n / a.T, y = a.targets.at(b, n - b * a.T);
      a.logp[n] = y >= 0 && y < a.V ? (E::to_float(z[y]) - st.m) - log_s : 0.f;
    }
  }
  if (lane < a.top_k) {
    a.top_logp[n * a.top_k + lane] = e != 0 ? (value_of(e) - st.m) - log_s : __builtin_nanf("");
    a.top_ids[n * a.top_k + lane] = e != 0 ? index_of(e) : -1;
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
  __shared__ uint64_t lists[TOP ? kLists : 1][TOP ? kListed : 1];
  __shared__ uint64_t best[TOP && WAVES > 1 ? WAVES * 64 : 1];
  __shared__ uint32_t bounds[kLists];
  __shared__ int listed;
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
  if constexpr (TOP) {
    if (lane == 0) bounds[wave] = ordered(kNegInf);
    if constexpr (WAVES == 1) {
      __builtin_amdgcn_wave_barrier();
    } else {
      if (threadIdx.x == 0) listed = 0;
      __syncthreads();
    }
  }
  const typename E::storage* z = row_of<E>(a.Z, a.T, n);
  RowPart<E, TOP> p;
  p.pre = before_aligned<E>(z);
  p.z = z - p.pre;
  p.V = (int)a.V;
  p.top_k = a.top_k;
  p.list = lists[TOP ? wave : 0];
  p.bound = &bounds[WAVES == 1 ? wave : 0];
  const int vecs = (p.V + p.pre + E::kVec - 1) / E::kVec;
  p.v1 = (int)((int64_t)vecs * (part + 1) / splits);
  p.run((int)((int64_t)vecs * part / splits), WAVES == 1 ? 0 : wave, WAVES);
  uint64_t top = 0;
  if constexpr (WAVES == 1) {
    if constexpr (TOP) top = best_of(p.list, p.count);
    write_row<E>(a, n, p.st, top, z);
  } else {
    if (lane == 0) stats[wave] = p.st;
    __syncthreads();
    if constexpr (TOP) {
      const uint64_t c = lane < p.count ? p.list[lane] : 0;
      const uint64_t hit = __ballot((uint32_t)(c >> 32) >= *p.bound);
      if (hit != 0) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&listed, __popcll(hit));
        at = __shfl(at, 0, 64);
        if ((hit >> lane) & 1) best[at + __popcll(hit & ((1ull << lane) - 1ull))] = c;
      }
      __syncthreads();
    }
    if (wave != 0) return;
    Stats st = stats[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) st = merge(st, stats[w]);
    if constexpr (TOP) top = best_of(best, listed);
    if (splits == 1) {
      write_row<E>(a, n, st, top, z);
    } else {
      float* o = (float*)a.ws + (n * splits + part) * part_words(a.top_k);
      if (lane == 0) { o[0] = st.m; o[1] = st.s; o[2] = st.s1; }
      if (lane < a.top_k) ((uint64_t*)(o + 4))[lane] = top;
    }
  }
}

// Joins the parts of split rows, one wave per row: the sums in the parts'
// order, the alternatives by order.
template <class E>
__global__ void __launch_bounds__(64) logprobs_join_kernel(LogprobArgs a, int splits) {
  __shared__ uint64_t best[kTopLanes * 64];
  const int64_t n = blockIdx.x;
  const int lane = threadIdx.x;
  if (a.mask != nullptr && a.mask[n] == 0) return;
  const int words = part_words(a.top_k);
  const float* o = (const float*)a.ws + n * splits * words;
  Stats mine = {kNegInf, 0.f, 0.f};
  if (lane < splits) mine = Stats{o[lane * words], o[lane * words + 1], o[lane * words + 2]};
  for (int k = lane; k < splits * a.top_k; k += 64)
    best[k] = ((const uint64_t*)(o + (k / a.top_k) * words + 4))[k % a.top_k];
  Stats st = {__shfl(mine.m, 0, 64), __shfl(mine.s, 0, 64), __shfl(mine.s1, 0, 64)};
  for (int w = 1; w < splits; ++w)
    st = merge(st, Stats{__shfl(mine.m, w, 64), __shfl(mine.s, w, 64), __shfl(mine.s1, w, 64)});
  __syncthreads();
  const uint64_t top = a.top_k > 0 ? best_of(best, splits * a.top_k) : 0;
  write_row<E>(a, n, st, top, row_of<E>(a.Z, a.T, n));
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

// Waves per row.  A wave alone needs no barrier and one bound, list and sort per
// row, but the chip needs rows for it; eight hold a long row at once.  In
// chunks of a wave (64 kR vectors, 8 KB), N rows, microseconds for 1, 4, 8 waves:
//   without alternatives  N 16384, 1.5 chunks 33 39 70; 4 105 100 125; 8 198 185 191
//                         N 1024, 6 chunks 20 14 14; 24 63 40 40
//   five alternatives     N 16384, 1.5 chunks 68 106 186; 4 146 154 258; 12 384 400 479
//                         N 4096, 2 chunks 30 35 55; 12 129 115 129; 24 220 201 200
//                         N 1024, 4 chunks 31 18 21; 24 126 67 61
template <class E>
int waves_of(const LogprobArgs& a) {
  const int64_t chunk = 64 * kR * E::kVec, chunks = (a.V + chunk - 1) / chunk;
  const int64_t alone = a.top_k > 0 ? a.N / 2048 : std::min<int64_t>(2, a.N / 2048);
  if (chunks <= std::max<int64_t>(1, alone)) return 1;
  return chunks <= a.N / 128 ? 4 : kWaves;
}
int waves_of(const LogprobArgs& a) {
  return a.dtype == kBF16 ? waves_of<BF16>(a) : waves_of<F32>(a);
}

// Workgroups per row: 1, or enough for half the compute units where the rows
// are fewer, parts of at least one chunk of each wave.  (Smaller parts are read
// no sooner and cost the join: in parts of a quarter of that, one row of 32000
// bf16 logits took 20 us in place of 11, one of 262144 float32 33 in place of
// 23, 64 rows of 50257 bf16 18 in place of 8.)
int splits_of(const LogprobArgs& a) {
  const int64_t vec = a.dtype == kBF16 ? 8 : 4, most = 64;
  const int64_t parts = a.V / (kWaves * 64 * vec * kR);
  const int64_t want = (device_cus() / 2) / a.N;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(parts, want), most));
}

template <class E, bool TOP>
hipError_t logprobs_e(const LogprobArgs& a, hipStream_t s) {
  const int waves = waves_of<E>(a);
  if (waves == 1) {
    hipLaunchKernelGGL((logprobs_kernel<E, 1, TOP>), dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, a, 1);
    return hipGetLastError();
  }
  if (waves == 4) {
    hipLaunchKernelGGL((logprobs_kernel<E, 4, TOP>), dim3((unsigned)a.N), dim3(256), 0, s, a, 1);
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
  const int splits = waves_of(a) < kWaves ? 1 : splits_of(a);
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
