// Embedding rows: the lookup, and the per-sample clipped gradient of the table.
//
//   out[b][t]  = scale * table[id_bt]
//   g_i[v]     = scale * sum over the active t of sample i with id_it = v of G_i[t]
//   n_i^2      = sum_v ||g_i[v]||^2
//   grad[v]    = (sum_i c_i g_i[v] + noise_std xi_v) / denom
//
// A position is active when its mask byte is not 0 and its id is in [0, V).
//
// The gradient works on the positions sorted by (token, position).  Equal
// tokens of one sample are then neighbours (a run), equal tokens of the whole
// batch too (a segment): a run's rows are summed before they are squared, and
// a segment's rows, each times its sample's clip factor, are one row of the
// result.  No [V, D] gradient of a sample is ever stored.
//
//  sort_hist, sort_scatter : stable radix sort by the token id, least
//                            significant digit first; inactive positions get
//                            the id V and end up last; the last pass also
//                            writes, per position, where its row of G starts
//                            and its sample, and per table row its segment
//  embed_blocks            : 16 positions of one run (segment) summed ahead
//  embed_norm              : one wave per run and column group
//  embed_long              : segments that hold such blocks
//  embed_accumulate        : every row of the result, noise included
#include <algorithm>
#include <type_traits>

#include "lm.hpp"

namespace dpf {
namespace {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
// L lanes per position (a power of two up to 64), V elements per lane and step.
template <class EI, class EO, int V>
__global__ void __launch_bounds__(256) lookup_kernel(LookupArgs a, int L) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int l = (int)(threadIdx.x & (unsigned)(L - 1));
  if (n >= a.N) return;
  const int64_t b = n / a.T, t = n - b * a.T;
  const int64_t id = a.ids.at(b, t);
  const bool active = (a.mask == nullptr || a.mask[n] != 0) && id >= 0 && id < a.V;
  const typename EI::storage* row =
      (const typename EI::storage*)a.table + (active ? id : 0) * a.stride_v;
  typename EO::storage* out = (typename EO::storage*)a.out + n * a.D;
#pragma unroll 4
  for (int64_t d = (int64_t)l * V; d < a.D; d += (int64_t)L * V) {
    float x[V];
    if (active) {
      load_f32<EI, V>(row + d, x);
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] *= a.scale;
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = 0.f;
    }
    store_f32<EO, V>(out + d, x);
  }
}

template <class EI, class EO>
void lookup_v(const LookupArgs& a, int V, hipStream_t s) {
  int L = 1;
  while (L < 64 && (int64_t)L * V < a.D) L *= 2;
  const dim3 grid((unsigned)((a.N * L + 255) / 256));
  if (V == 8) hipLaunchKernelGGL((lookup_kernel<EI, EO, 8>), grid, dim3(256), 0, s, a, L);
  else if (V == 4) hipLaunchKernelGGL((lookup_kernel<EI, EO, 4>), grid, dim3(256), 0, s, a, L);
  else hipLaunchKernelGGL((lookup_kernel<EI, EO, 1>), grid, dim3(256), 0, s, a, L);
}

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int kSortPer = 8;                              // most keys per thread and chunk
constexpr int kSortBlocks = 64;                          // workgroups, before chunks are looped over
constexpr int kMaxDigit = 9, kMaxBins = 1 << kMaxDigit;
static_assert(kMaxBins <= kSortThreads, "one thread per bin");

struct SortPlan {
  int passes, digit, per, blocks, chunks;   // keys per thread; chunks per workgroup
};

SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan p;
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;              // keys 0 .. V
  p.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  p.digit = (bits + p.passes - 1) / p.passes;
  p.per = 1;
  while (p.per < kSortPer && N > (int64_t)kSortBlocks * kSortThreads * p.per) p.per *= 2;
  const int64_t chunks = (N + kSortThreads * p.per - 1) / (kSortThreads * p.per);
  p.chunks = (int)((chunks + kSortBlocks - 1) / kSortBlocks);
  p.blocks = (int)((chunks + p.chunks - 1) / p.chunks);
  return p;
}

// Which of the two buffers pass q writes (q = -1: the last pass).
int embed_sorted(int64_t V, int q) {
  if (q < 0) q = sort_plan(1, V).passes - 1;
  return q & 1;
}

__device__ __forceinline__ uint32_t token_key(const EmbedArgs& a, uint32_t n) {
  if (a.mask != nullptr && a.mask[n] == 0) return (uint32_t)a.V;
  const uint32_t b = n / (uint32_t)a.T;
  const int64_t id = a.ids.at(b, n - b * (uint32_t)a.T);
  return id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

struct SortPass {
  const uint32_t *key, *pos;     // sorted so far (first pass: null)
  uint32_t *key_out, *pos_out;
  uint32_t *hist, *next_hist;    // [blocks, bins] of this pass and of the next (last: null)
  uint32_t N;
  int shift, digit, blocks, chunks, per;
};

// First pass: digit counts of each workgroup's keys.  Workgroups past `blocks`
// empty the segments and clear the later passes' counts, which the passes
// before them add up.
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(EmbedArgs a, SortPass p,
                                                                 int64_t later) {
  const int bins = 1 << p.digit;
  if ((int)blockIdx.x >= p.blocks) {
    const int64_t step = (int64_t)(gridDim.x - p.blocks) * kSortThreads;
    const int64_t at = (int64_t)(blockIdx.x - p.blocks) * kSortThreads + threadIdx.x;
    for (int64_t v = at; v < a.V; v += step) a.seg[v] = make_uint2(0xffffffffu, 0u);
    uint32_t* h = p.hist + (int64_t)p.blocks * bins;
    for (int64_t v = at; v < later; v += step) h[v] = 0u;
    return;
  }
  __shared__ uint32_t cnt[kMaxBins];
  if ((int)threadIdx.x < bins) cnt[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t len = (uint32_t)(p.chunks * p.per * kSortThreads), n0 = blockIdx.x * len;
  const uint32_t n1 = min(p.N, n0 + len);
  for (uint32_t n = n0 + threadIdx.x; n < n1; n += kSortThreads)
    atomicAdd(&cnt[token_key(a, n) & (uint32_t)(bins - 1)], 1u);
  __syncthreads();
  if ((int)threadIdx.x < bins) p.hist[(int64_t)blockIdx.x * bins + threadIdx.x] = cnt[threadIdx.x];
}

// Exclusive prefix sum of one value per thread over the workgroup.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < wave; ++w) before += tmp[w];
  return before + x - v;
}

// Moves every key (and its position) to its place in the digit's order.  A
// key's rank among equal digits counts the keys before it: those of earlier
// workgroups (from the histograms), chunks and waves, and within a wave's 64
// keys the lanes below it with the same digit (found by ballots on its bits).
// Each key's digit of the next pass is counted for the workgroup that will
// read it there.  The last pass writes what the kernels after it read: the
// row's offset in G and its sample, and the segments (keys that are equal
// arrive next to each other and in order, so the first and the last of them
// in a wave give the segment's ends; integer minimum and maximum, the same in
// any order).
template <int PER, bool FIRST, bool LAST>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(EmbedArgs a, SortPass p) {
  __shared__ uint32_t base[kMaxBins];
  __shared__ uint32_t wcnt[kSortWaves][kMaxBins];
  __shared__ uint32_t tmp[kSortWaves];
  const int bins = 1 << p.digit, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t chunk = kSortThreads * PER, len = chunk * p.chunks, n0 = blockIdx.x * len;
  for (int ch = 0; ch < p.chunks; ++ch) {
    const uint32_t c0 = n0 + ch * chunk;
    if (c0 >= p.N) break;
    uint32_t k[PER], q[PER], r[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t n = c0 + wave * (64 * PER) + i * 64 + lane;
      const bool in = n < p.N;
      k[i] = !in ? 0u : FIRST ? token_key(a, n) : p.key[n];
      q[i] = !in ? 0u : FIRST ? n : p.pos[n];
    }
    if (ch == 0) {
      uint32_t total = 0, before = 0;
      if (tid < bins) {
#pragma unroll 16
        for (int w = 0; w < p.blocks; ++w) {
          const uint32_t h = p.hist[w * bins + tid];
          before += w < (int)blockIdx.x ? h : 0u;
          total += h;
        }
      }
      const uint32_t ex = block_exclusive(total, tmp);
      if (tid < bins) base[tid] = ex + before;
    }
    for (int d = lane; d < bins; d += 64) wcnt[wave][d] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = c0 + wave * (64 * PER) + i * 64 + lane < p.N;
      const uint32_t d = (k[i] >> p.shift) & (uint32_t)(bins - 1);
      uint64_t same = __ballot(in);
      for (int j = 0; j < p.digit; ++j) {
        const uint64_t m = __ballot((d >> j) & 1u);
        same &= ((d >> j) & 1u) ? m : ~m;
      }
      const uint32_t below = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
      const uint32_t seen = in ? wcnt[wave][d] : 0u;
      r[i] = seen + below;
      __builtin_amdgcn_wave_barrier();
      if (in && below == 0) wcnt[wave][d] = seen + (uint32_t)__popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (tid < bins) {
      uint32_t at = base[tid];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = wcnt[w][tid];
        wcnt[w][tid] = at;
        at += c;
      }
      base[tid] = at;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t n = c0 + wave * (64 * PER) + i * 64 + lane;
      const bool in = n < p.N;
      const uint32_t key = k[i];
      const uint32_t to = in ? wcnt[wave][(key >> p.shift) & (uint32_t)(bins - 1)] + r[i] : 0u;
      const uint32_t prev = __shfl_up(key, 1, 64), next = __shfl_down(key, 1, 64);
      if (!in) continue;
      p.key_out[to] = key;
      p.pos_out[to] = q[i];
      if constexpr (!LAST) {
        const uint32_t nd = (key >> (p.shift + p.digit)) & (uint32_t)(bins - 1);
        atomicAdd(&p.next_hist[(to / len) * bins + nd], 1u);
      } else {
        const uint32_t b = q[i] / (uint32_t)a.T, t = q[i] - b * (uint32_t)a.T;
        a.off[to] = (int64_t)b * a.G.stride_b + (int64_t)t * a.G.stride_t;
        a.smp[to] = b;
        if (key < (uint32_t)a.V) {
          if (lane == 0 || prev != key) atomicMin(&a.seg[key].x, to);
          if (lane == 63 || n == p.N - 1 || next != key) atomicMax(&a.seg[key].y, to + 1);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Row sums
// ---------------------------------------------------------------------------
// Sorted positions in blocks of 16.  A block that lies inside one run (of one
// segment, for the clipped sum) is summed by itself first, so that no wave
// adds more than 30 rows and a partial per 16 others: a token that fills a
// tenth of the batch does not leave one wave with all its rows.
constexpr uint32_t kBlock = 16;
// Batches below this many positions go without (two launches less; a wave
// then adds at most this many rows).
constexpr int64_t kBlocksFrom = 256;

typedef __attribute__((address_space(4))) const uint32_t c_u32;
typedef __attribute__((address_space(4))) const int64_t c_i64;
typedef __attribute__((address_space(4))) const float c_f32;

// Wave-uniform reads of what an earlier kernel wrote, through the scalar cache.
__device__ __forceinline__ uint32_t su32(const uint32_t* p, uint32_t i) { return ((c_u32*)p)[i]; }
__device__ __forceinline__ int64_t si64(const int64_t* p, uint32_t i) { return ((c_i64*)p)[i]; }
__device__ __forceinline__ float sf32(const float* p, uint32_t i) { return ((c_f32*)p)[i]; }

// One wave's share of a row: U groups of 64 V columns from c0 on.
template <class E, int V, int U>
struct RowSum {
  float s[U][V];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) s[u][e] = 0.f;
  }
  // += w row; `row` at the wave's first column
  __device__ __forceinline__ void add(const typename E::storage* row, int64_t left, float w) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = (int64_t)(u * 64 + lane) * V;
      if (col < left) {
        float x[V];
        load_f32<E, V>(row + col, x);
#pragma unroll
        for (int e = 0; e < V; ++e) s[u][e] += w * x[e];
      }
    }
  }
  __device__ __forceinline__ void add_part(const float* part, int64_t left) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = (int64_t)(u * 64 + lane) * V;
      if (col < left) {
        float x[V];
        load_f32<F32, V>(part + col, x);
#pragma unroll
        for (int e = 0; e < V; ++e) s[u][e] += x[e];
      }
    }
  }
  __device__ __forceinline__ void store(float* part, int64_t left) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = (int64_t)(u * 64 + lane) * V;
      if (col < left) store_f32<F32, V>(part + col, s[u]);
    }
  }
  // The rows of sorted positions [i, end), whole blocks of 16 from `parts`
  // (null: none); weights c[sample] * scale, or 1.
  template <bool WEIGHTED>
  __device__ __forceinline__ void range(const EmbedArgs& a, const float* parts, int64_t c0,
                                        uint32_t i, uint32_t end) {
    const typename E::storage* G = (const typename E::storage*)a.G.data + c0;
    const int64_t left = a.D - c0;
    const uint32_t b0 = (i + kBlock - 1) / kBlock, b1 = end / kBlock;
    const bool blocks = parts != nullptr && b1 > b0;
    const uint32_t head = blocks ? b0 * kBlock : end;
#pragma unroll 4
    for (; i < head; ++i) add(G + si64(a.off, i), left, WEIGHTED ? sf32(a.c, su32(a.smp, i)) * a.scale : 1.f);
    if (!blocks) return;
#pragma unroll 4
    for (uint32_t b = b0; b < b1; ++b) add_part(parts + (int64_t)b * a.D + c0, left);
#pragma unroll 4
    for (i = b1 * kBlock; i < end; ++i)
      add(G + si64(a.off, i), left, WEIGHTED ? sf32(a.c, su32(a.smp, i)) * a.scale : 1.f);
  }
};

__device__ __forceinline__ uint32_t wave_of_grid() {
  return blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// The blocks inside one run (WEIGHTED: one segment), one wave per block and
// column group.
template <class E, int V, int U, bool WEIGHTED>
__global__ void __launch_bounds__(256) embed_blocks_kernel(EmbedArgs a, const uint32_t* key,
                                                           uint32_t N) {
  const uint32_t b = wave_of_grid(), i = b * kBlock;
  if (i + kBlock > N) return;
  const uint32_t v = su32(key, i);
  if (v >= (uint32_t)a.V || v != su32(key, i + kBlock - 1)) return;
  if (!WEIGHTED && su32(a.smp, i) != su32(a.smp, i + kBlock - 1)) return;
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * U);
  RowSum<E, V, U> sum;
  sum.zero();
  sum.template range<WEIGHTED>(a, nullptr, c0, i, i + kBlock);
  sum.store(a.blocks + (int64_t)b * a.D + c0, a.D - c0);
}

// Segments with a block of their own: their whole sum, in place of the first
// such block's.
template <class E, int V, int U>
__global__ void __launch_bounds__(256) embed_long_kernel(EmbedArgs a, const uint32_t* key,
                                                         uint32_t N) {
  const uint32_t b = wave_of_grid(), i = b * kBlock;
  if (i + kBlock > N) return;
  const uint32_t v = su32(key, i);
  if (v >= (uint32_t)a.V || v != su32(key, i + kBlock - 1)) return;
  const uint32_t first = su32(&a.seg[v].x, 0), end = su32(&a.seg[v].y, 0);
  if ((first + kBlock - 1) / kBlock != b) return;
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * U);
  RowSum<E, V, U> sum;
  sum.zero();
  sum.template range<true>(a, a.blocks, c0, first, end);
  sum.store(a.blocks + (int64_t)b * a.D + c0, a.D - c0);
}

// One wave per sorted position and column group.  The first position of a run
// sums the run's rows (float32, in order) and squares the sum (float64); the
// others write 0.  partials[position][column group], positions in their
// original order, so that a sample's are contiguous.
template <class E, int V, int U>
__global__ void __launch_bounds__(256) embed_norm_kernel(EmbedArgs a, const uint32_t* key,
                                                         const uint32_t* pos, uint32_t N) {
  const int lane = threadIdx.x & 63;
  const uint32_t k = wave_of_grid();
  if (k >= N) return;
  double* dst = a.partials + (int64_t)su32(pos, k) * gridDim.y + blockIdx.y;
  const uint32_t v = su32(key, k), b = su32(a.smp, k);
  if (v >= (uint32_t)a.V || (k > 0 && su32(key, k - 1) == v && su32(a.smp, k - 1) == b)) {
    if (lane == 0) *dst = 0.0;
    return;
  }
  uint32_t end = k + 1;
  for (;;) {                       // the run's end, 64 positions at a time
    const uint32_t i = end + lane;
    const uint64_t other = __ballot(i >= N || key[i] != v || a.smp[i] != b);
    if (other != 0) { end += __builtin_ctzll(other); break; }
    end += 64;
  }
  end = __builtin_amdgcn_readfirstlane(end);
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * U);
  RowSum<E, V, U> sum;
  sum.zero();
  sum.template range<false>(a, a.blocks, c0, k, end);
  double sq = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < V; ++e) sq += (double)sum.s[u][e] * (double)sum.s[u][e];
  sq = wave_sum_f64(sq);
  if (lane == 0) *dst = sq * (double)a.scale * (double)a.scale;
}

// One wave per row of the result and U groups of 256 columns (gridDim.y of
// them at a time).  A thread's four values are one Philox block: with D % 4
// != 0 (AL false) the groups start at the block that holds the row's first
// value, and each row keeps its own part of a shared block.
template <class E, int U, bool AL>
__global__ void __launch_bounds__(256) embed_accumulate_kernel(EmbedArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t v = wave_of_grid();
  if (v >= (uint32_t)a.V) return;
  const uint32_t first = su32(&a.seg[v].x, 0), end = su32(&a.seg[v].y, 0);
  const uint32_t b0 = (first + kBlock - 1) / kBlock;
  const bool empty = first >= end;
  const bool summed = !empty && a.blocks != nullptr && (b0 + 1) * kBlock <= end;
  const int64_t row0 = (int64_t)v * a.D, start = AL ? row0 : row0 & ~(int64_t)3;
  const int64_t D = a.D;
  const float rd = 1.0f / a.denom;
  for (int64_t g0 = (int64_t)blockIdx.y * (256 * U); start + g0 < row0 + D;
       g0 += (int64_t)gridDim.y * (256 * U)) {
    int64_t col[U];                // first of the thread's four columns (may be below 0)
#pragma unroll
    for (int u = 0; u < U; ++u) col[u] = start - row0 + g0 + (u * 64 + lane) * 4;
    float old[U][4], sum[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[u][e] = old[u][e] = 0.f;
      if (a.beta && col[u] < D) {
        float* o = a.out + row0 + col[u];
        if (AL || (col[u] >= 0 && col[u] + 4 <= D)) {
          load_f32<F32, 4>(o, old[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col[u] + e >= 0 && col[u] + e < D) old[u][e] = o[e];
        }
      }
    }
    if (summed) {
      const float* part = a.blocks + (int64_t)b0 * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (col[u] >= D) continue;
        if (AL) {
          load_f32<F32, 4>(part + col[u], sum[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col[u] + e >= 0 && col[u] + e < D) sum[u][e] = part[col[u] + e];
        }
      }
    } else if (!empty) {
#pragma unroll 2
      for (uint32_t i = first; i < end; ++i) {
        const typename E::storage* row = (const typename E::storage*)a.G.data + si64(a.off, i);
        const float w = sf32(a.c, su32(a.smp, i)) * a.scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (col[u] >= D) continue;
          if (AL) {
            float x[4];
            load_f32<E, 4>(row + col[u], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u][e] += w * x[e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col[u] + e >= 0 && col[u] + e < D) sum[u][e] += w * E::to_float(row[col[u] + e]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (col[u] >= D) continue;
      const int64_t e0 = row0 + col[u];
      if (a.noise_std != 0.0f) {
        const f32x4 z = normals_of_block(philox_block(a.seed, a.offset + (uint64_t)(e0 >> 2)));
        sum[u][0] += a.noise_std * z.x; sum[u][1] += a.noise_std * z.y;
        sum[u][2] += a.noise_std * z.z; sum[u][3] += a.noise_std * z.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[u][e] = old[u][e] + sum[u][e] * rd;
      float* o = a.out + e0;
      if (AL || (col[u] >= 0 && col[u] + 4 <= D)) {
        store_f32<F32, 4>(o, sum[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col[u] + e >= 0 && col[u] + e < D) o[e] = sum[u][e];
      }
    }
  }
}

// Elements per load for rows of D that start stride_b, stride_t apart.
int row_vec(const Act& G, int64_t D) {
  if (D % 8 == 0 && G.stride_t % 8 == 0 && G.stride_b % 8 == 0) return 8;
  if (D % 4 == 0 && G.stride_t % 4 == 0 && G.stride_b % 4 == 0) return 4;
  return 1;
}

// Groups of 64 V columns that a wave of the row sums takes: the count up to 3
// that leaves the fewest idle.
int row_groups(int64_t D, int V) {
  const int64_t steps = (D + 64 * V - 1) / (64 * V);
  int best = 1;
  for (int u = 2; u <= 3; ++u)
    if ((steps + u - 1) / u * u <= (steps + best - 1) / best * best) best = u;
  return best;
}

int64_t row_parts(int64_t D, int V) {
  const int64_t cols = 64 * (int64_t)V * row_groups(D, V);
  return (D + cols - 1) / cols;
}

bool use_blocks(const EmbedArgs& a) { return a.B * a.T >= kBlocksFrom; }

// Calls f with the element type, V and U of a call's row sums.
template <class F>
void with_rows(const EmbedArgs& a, F&& f) {
  const int V = row_vec(a.G, a.D), U = row_groups(a.D, V);
  auto u = [&](auto e, auto v) {
    if (U == 1) f(e, v, std::integral_constant<int, 1>());
    else if (U == 2) f(e, v, std::integral_constant<int, 2>());
    else f(e, v, std::integral_constant<int, 3>());
  };
  auto vv = [&](auto e) {
    if (V == 8) u(e, std::integral_constant<int, 8>());
    else if (V == 4) u(e, std::integral_constant<int, 4>());
    else u(e, std::integral_constant<int, 1>());
  };
  if (a.dtype == kBF16) vv(BF16());
  else vv(F32());
}

template <int PER>
void launch_scatter(const EmbedArgs& a, const SortPass& p, bool first, bool last, hipStream_t s) {
  const dim3 grid((unsigned)p.blocks), block(kSortThreads);
  if (first && last) hipLaunchKernelGGL((sort_scatter_kernel<PER, true, true>), grid, block, 0, s, a, p);
  else if (first) hipLaunchKernelGGL((sort_scatter_kernel<PER, true, false>), grid, block, 0, s, a, p);
  else if (last) hipLaunchKernelGGL((sort_scatter_kernel<PER, false, true>), grid, block, 0, s, a, p);
  else hipLaunchKernelGGL((sort_scatter_kernel<PER, false, false>), grid, block, 0, s, a, p);
}

}  // namespace

hipError_t launch_embedding_lookup(const LookupArgs& a, hipStream_t s) {
  const int V = a.D % 8 == 0 && a.stride_v % 8 == 0 ? 8 : a.D % 4 == 0 && a.stride_v % 4 == 0 ? 4 : 1;
  timing_begin("embedding_lookup", s);
  if (a.table_dtype == kBF16) {
    if (a.out_dtype == kBF16) lookup_v<BF16, BF16>(a, V, s);
    else lookup_v<BF16, F32>(a, V, s);
  } else {
    if (a.out_dtype == kBF16) lookup_v<F32, BF16>(a, V, s);
    else lookup_v<F32, F32>(a, V, s);
  }
  timing_end("embedding_lookup", s);
  return hipGetLastError();
}

int64_t embed_hist_words(int64_t N, int64_t V) {
  const SortPlan p = sort_plan(N, V);
  return ((int64_t)p.blocks << p.digit) * p.passes;
}

int64_t embed_block_floats(const EmbedArgs& a) {
  return use_blocks(a) ? a.B * a.T / kBlock * a.D : 0;
}

int embed_norm_parts(const EmbedArgs& a) { return (int)row_parts(a.D, row_vec(a.G, a.D)); }

hipError_t launch_embed_sort(const EmbedArgs& a, hipStream_t s) {
  const int64_t N = a.B * a.T;
  const SortPlan p = sort_plan(N, a.V);
  const int64_t words = (int64_t)p.blocks << p.digit;
  timing_begin("embed_sort", s);
  for (int q = 0; q < p.passes; ++q) {
    const bool first = q == 0, last = q + 1 == p.passes;
    SortPass w{};
    if (!first) {
      w.key = a.key[embed_sorted(a.V, q - 1)];
      w.pos = a.pos[embed_sorted(a.V, q - 1)];
    }
    w.key_out = a.key[embed_sorted(a.V, q)];
    w.pos_out = a.pos[embed_sorted(a.V, q)];
    w.hist = a.hist + q * words;
    w.next_hist = last ? nullptr : w.hist + words;
    w.N = (uint32_t)N;
    w.shift = q * p.digit;
    w.digit = p.digit;
    w.blocks = p.blocks;
    w.chunks = p.chunks;
    w.per = p.per;
    if (first) {
      const int64_t later = words * (p.passes - 1);
      const int clear = (int)std::min<int64_t>(
          256, (std::max(a.V, later) + kSortThreads - 1) / kSortThreads);
      hipLaunchKernelGGL(sort_hist_kernel, dim3((unsigned)(p.blocks + clear)), dim3(kSortThreads), 0,
                         s, a, w, later);
    }
    if (p.per == 1) launch_scatter<1>(a, w, first, last, s);
    else if (p.per == 2) launch_scatter<2>(a, w, first, last, s);
    else if (p.per == 4) launch_scatter<4>(a, w, first, last, s);
    else launch_scatter<8>(a, w, first, last, s);
  }
  timing_end("embed_sort", s);
  return hipGetLastError();
}

hipError_t launch_embed_norm(const EmbedArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)(a.B * a.T);
  const unsigned parts = (unsigned)embed_norm_parts(a);
  const uint32_t *key = a.key[embed_sorted(a.V, -1)], *pos = a.pos[embed_sorted(a.V, -1)];
  EmbedArgs q = a;
  if (a.T < (int64_t)kBlock) q.blocks = nullptr;   // no run is as long
  timing_begin("embed_norm", s);
  with_rows(a, [&](auto e, auto v, auto u) {
    using E = decltype(e);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    if (q.blocks != nullptr)
      hipLaunchKernelGGL((embed_blocks_kernel<E, V, U, false>), dim3((N / kBlock + 3) / 4, parts),
                         dim3(256), 0, s, q, key, N);
    hipLaunchKernelGGL((embed_norm_kernel<E, V, U>), dim3((N + 3) / 4, parts), dim3(256), 0, s, q,
                       key, pos, N);
  });
  timing_end("embed_norm", s);
  return hipGetLastError();
}

namespace {

template <class E, bool AL>
void accumulate_u(const EmbedArgs& a, int U, dim3 grid, hipStream_t s) {
  switch (U) {
    case 1: hipLaunchKernelGGL((embed_accumulate_kernel<E, 1, AL>), grid, dim3(256), 0, s, a); break;
    case 2: hipLaunchKernelGGL((embed_accumulate_kernel<E, 2, AL>), grid, dim3(256), 0, s, a); break;
    case 3: hipLaunchKernelGGL((embed_accumulate_kernel<E, 3, AL>), grid, dim3(256), 0, s, a); break;
    case 4: hipLaunchKernelGGL((embed_accumulate_kernel<E, 4, AL>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((embed_accumulate_kernel<E, 5, AL>), grid, dim3(256), 0, s, a);
  }
}

}  // namespace

hipError_t launch_embed_accumulate(const EmbedArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)(a.B * a.T);
  const unsigned parts = (unsigned)embed_norm_parts(a);
  const uint32_t* key = a.key[embed_sorted(a.V, -1)];
  timing_begin("embed_accumulate", s);
  if (a.blocks != nullptr)
    with_rows(a, [&](auto e, auto v, auto u) {
      using E = decltype(e);
      constexpr int V = decltype(v)::value, U = decltype(u)::value;
      const dim3 grid((N / kBlock + 3) / 4, parts);
      hipLaunchKernelGGL((embed_blocks_kernel<E, V, U, true>), grid, dim3(256), 0, s, a, key, N);
      hipLaunchKernelGGL((embed_long_kernel<E, V, U>), grid, dim3(256), 0, s, a, key, N);
    });
  const bool al = row_vec(a.G, a.D) >= 4;
  // an unaligned row can touch one Philox block more
  const int64_t steps = (a.D + (al ? 0 : 3) + 255) / 256;
  int U = 1;
  for (int u = 2; u <= 5; ++u)
    if ((steps + u - 1) / u * u <= (steps + U - 1) / U * U) U = u;
  // Column groups side by side only where the rows alone leave the chip idle.
  const int64_t groups = (steps + U - 1) / U, want = (int64_t)device_cus() * 32;
  const int64_t gy = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(groups, 65535), want / a.V));
  const dim3 grid((unsigned)((a.V + 3) / 4), (unsigned)gy);
  if (a.dtype == kBF16) {
    if (al) accumulate_u<BF16, true>(a, U, grid, s);
    else accumulate_u<BF16, false>(a, U, grid, s);
  } else {
    if (al) accumulate_u<F32, true>(a, U, grid, s);
    else accumulate_u<F32, false>(a, U, grid, s);
  }
  timing_end("embed_accumulate", s);
  return hipGetLastError();
}

}  // namespace dpf
