// Embedding rows: the lookup, and the per-sample clipped gradient of the table.
//
//   out[b][t]  = scale * table[id_bt]                    (float32, then rounded)
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
//                            and its sample
//  sort_small              : the same in one workgroup, up to 2048 positions
//  embed_segments          : each row's positions (with norms, embed_norm's
//                            work)
//  embed_blocks            : 8 positions of one run (segment) summed ahead
//  embed_norm              : one wave per 8 sorted positions and column group
//  embed_accumulate        : every row of the result, noise included
//
// What it costs (MI355X).  Lookup of 16384 rows of 5120 bf16: 52 us, 4.3 TB/s of
// distinct rows read and rows written; of 16: 3.3 us.  Gradient of 16384
// positions, 8.7 thousand active, 5120 bf16 columns, added into 32000 rows of
// which 3.4 thousand have a token: 125 us.  The norms read G (89 MB) in 25 us,
// the result takes 51 (G again, 140 MB of rows read and written: 4.5 TB/s); the
// sort's three launches 16, the block sums 10 twice, the clip factors 5: a few
// thousand rows each, bound by the latency of dependent loads.  Of 32 x 512
// positions, 768 columns, 50257 rows with noise: 80 us, 47 of them the result,
// which the noise's arithmetic bounds (39 million normals; 154 MB written).
// Of 132 positions in 99 float32 columns: 16 us in four launches, 22 a call.
#include <algorithm>
#include <type_traits>

#include "lm.hpp"

namespace dpf {
namespace {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
// L lanes per position (a power of two up to 64), V elements per lane and step:
// a row is one or a few 16-byte loads of each lane, all in flight together, and
// a wave's stores are whole lines.
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

// Mask byte and id are fetched together: both are the caller's memory whatever
// they hold, and a chain of two loads costs a microsecond more.
__device__ __forceinline__ uint32_t token_key(const EmbedArgs& a, uint32_t n) {
  const uint8_t m = a.mask != nullptr ? a.mask[n] : 1;
  const uint32_t b = n / (uint32_t)a.T;
  const int64_t id = a.ids.at(b, n - b * (uint32_t)a.T);
  return m != 0 && id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

// What the kernels after the sort read of a position, in one load: its token,
// its sample, and where its row of G starts (elements).
__device__ __forceinline__ uint4 record(const EmbedArgs& a, uint32_t key, uint32_t n) {
  const uint32_t b = n / (uint32_t)a.T, t = n - b * (uint32_t)a.T;
  const int64_t off = (int64_t)b * a.G.stride_b + (int64_t)t * a.G.stride_t;
  return make_uint4(key, b, (uint32_t)off, (uint32_t)(off >> 32));
}
__device__ __forceinline__ int64_t record_off(const uint4& r) {
  return (int64_t)(((uint64_t)r.w << 32) | r.z);
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
// read it there: in LDS first (a frequent token would otherwise queue up its
// global atomics), then added up, integers, so the same in any order.  The last
// pass writes what the kernels after it read: the row's offset in G and its
// sample.
template <int PER, bool FIRST, bool LAST>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(EmbedArgs a, SortPass p) {
  extern __shared__ uint32_t next_cnt[];         // [blocks, bins], not in the last pass
  __shared__ uint32_t base[kMaxBins];
  __shared__ uint32_t wcnt[kSortWaves][kMaxBins];
  __shared__ uint32_t tmp[kSortWaves];
  const int bins = 1 << p.digit, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if constexpr (!LAST)
    for (int i = tid; i < p.blocks * bins; i += kSortThreads) next_cnt[i] = 0u;
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
      if (!in) continue;
      p.pos_out[to] = q[i];
      if constexpr (!LAST) {
        p.key_out[to] = key;
        const uint32_t nd = (key >> (p.shift + p.digit)) & (uint32_t)(bins - 1);
        atomicAdd(&next_cnt[(to / len) * bins + nd], 1u);
      } else {
        a.rec[to] = record(a, key, q[i]);
      }
    }
    __syncthreads();
  }
  if constexpr (!LAST)
    for (int i = tid; i < p.blocks * bins; i += kSortThreads)
      if (const uint32_t n = next_cnt[i]) atomicAdd(&p.next_hist[i], n);
}

// Up to 2048 positions: every pass in one workgroup, keys and the order so
// far in LDS, so that a call has one launch instead of one per digit and one
// more.  The other workgroups empty the segments.
constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64, kSmallPer = 2;
constexpr int64_t kSmallN = kSmallThreads * kSmallPer;

template <int PER>
constexpr int small_lds() {
  return kSmallThreads * PER * (4 + 2 * 2) + kSmallWaves * kMaxBins * 2 + kSmallWaves * 4;
}

template <int PER>
__global__ void __launch_bounds__(kSmallThreads) sort_small_kernel(EmbedArgs a, uint32_t N,
                                                                   int passes, int digit,
                                                                   uint32_t* pos_out) {
  extern __shared__ __attribute__((aligned(16))) unsigned char mem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x != 0) {
    for (int64_t v = (int64_t)(blockIdx.x - 1) * kSmallThreads + tid; v < a.V;
         v += (int64_t)(gridDim.x - 1) * kSmallThreads)
      a.seg[v] = make_uint2(0xffffffffu, 0u);
    return;
  }
  uint32_t* key = (uint32_t*)mem;                                  // by position
  uint16_t* perm = (uint16_t*)(key + kSmallThreads * PER);         // two orders
  uint16_t* wcnt = perm + 2 * kSmallThreads * PER;                 // [wave][bin]
  uint32_t* tmp = (uint32_t*)(wcnt + kSmallWaves * kMaxBins);
  const int bins = 1 << digit;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t n = tid + i * kSmallThreads;
    if (n < N) key[n] = token_key(a, n);
  }
  __syncthreads();
  for (int p = 0; p < passes; ++p) {
    const uint16_t* from = perm + (p & 1) * kSmallThreads * PER;
    uint16_t* to = perm + ((p + 1) & 1) * kSmallThreads * PER;
    for (int d = lane; d < bins; d += 64) wcnt[wave * kMaxBins + d] = 0;
    __builtin_amdgcn_wave_barrier();
    uint16_t src[PER], dig[PER], r[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t n = wave * (64 * PER) + i * 64 + lane;
      src[i] = n >= N ? 0 : p == 0 ? (uint16_t)n : from[n];
      dig[i] = n >= N ? 0 : (uint16_t)((key[src[i]] >> (p * digit)) & (uint32_t)(bins - 1));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = wave * (64 * PER) + i * 64 + lane < N;
      const uint32_t d = dig[i];
      uint64_t same = __ballot(in);
      for (int j = 0; j < digit; ++j) {
        const uint64_t m = __ballot((d >> j) & 1u);
        same &= ((d >> j) & 1u) ? m : ~m;
      }
      const uint32_t below = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
      const uint32_t seen = in ? wcnt[wave * kMaxBins + d] : 0u;
      r[i] = (uint16_t)(seen + below);
      __builtin_amdgcn_wave_barrier();
      if (in && below == 0) wcnt[wave * kMaxBins + d] = (uint16_t)(seen + (uint32_t)__popcll(same));
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    uint32_t total = 0;
    if (tid < bins)
      for (int w = 0; w < kSmallWaves; ++w) total += wcnt[w * kMaxBins + tid];
    uint32_t at = block_exclusive(total, tmp);
    if (tid < bins)
      for (int w = 0; w < kSmallWaves; ++w) {
        const uint32_t c = wcnt[w * kMaxBins + tid];
        wcnt[w * kMaxBins + tid] = (uint16_t)at;
        at += c;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (wave * (64 * PER) + i * 64 + lane < N) to[wcnt[wave * kMaxBins + dig[i]] + r[i]] = src[i];
    __syncthreads();
  }
  const uint16_t* order = perm + (passes & 1) * kSmallThreads * PER;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t k = tid + i * kSmallThreads;
    if (k >= N) break;
    const uint32_t n = order[k];
    pos_out[k] = n;
    a.rec[k] = record(a, key[n], n);
  }
}

// The segments, from neighbours' tokens (emptied by the sort).
__global__ void __launch_bounds__(256) embed_segments_kernel(EmbedArgs a, uint32_t N) {
  const uint32_t k = blockIdx.x * 256 + threadIdx.x;
  if (k >= N) return;
  const uint32_t v = a.rec[k].x;
  if (v >= (uint32_t)a.V) return;
  if (k == 0 || a.rec[k - 1].x != v) a.seg[v].x = k;
  if (k == N - 1 || a.rec[k + 1].x != v) a.seg[v].y = k + 1;
}

// ---------------------------------------------------------------------------
// Row sums
// ---------------------------------------------------------------------------
// Sorted positions in blocks of 8.  A block that lies inside one run (of one
// segment, for the clipped sum) is summed by itself first, so that no wave
// adds more than 14 rows and a partial per 8 others: a token that fills a
// tenth of the batch does not leave one wave with all its rows.
constexpr uint32_t kBlock = 8;
// Batches below this many positions go without (two launches less, 4 to 5 us
// each; a wave then adds at most this many rows, 32 batches of loads).
constexpr int64_t kBlocksFrom = 256;
// Samples of at most this many positions have no runs worth summing ahead for
// the norms: norms of 256 x 64 positions of 768 columns 29.3 us without, 30.9
// with (one token throughout: 34.1 and 33.5); of 32 x 512 31.0 and 31.6 (86.5 and
// 42.1); of 8 x 2048 of 5120 columns 69.6 and 64.5 (546 and 161).
constexpr int64_t kShortRuns = 64;

typedef __attribute__((address_space(4))) const uint32_t c_u32;

// Wave-uniform reads of what an earlier kernel wrote, through the scalar cache.
__device__ __forceinline__ uint32_t su32(const uint32_t* p, uint32_t i) { return ((c_u32*)p)[i]; }

__device__ __forceinline__ int64_t lane_i64(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Rows (or partials) j .. cnt - 1 in batches whose loads are all in flight
// together: as many of MOST as there are, then the binary rest.
template <int MOST, class F>
__device__ __forceinline__ void in_batches(int cnt, F&& f) {
  int j = 0;
  for (; j + MOST <= cnt; j += MOST) f(j, std::integral_constant<int, MOST>());
  if constexpr (MOST >= 8)
    if (cnt - j >= 4) { f(j, std::integral_constant<int, 4>()); j += 4; }
  if constexpr (MOST >= 4)
    if (cnt - j >= 2) { f(j, std::integral_constant<int, 2>()); j += 2; }
  if (cnt - j >= 1) f(j, std::integral_constant<int, 1>());
}

// f(offsets, weights, count) for the sorted positions [i, end), 64 at a time,
// one position's in each lane (to go round by lane reads).  Weights c[sample]
// * scale, or 1.
template <bool WEIGHTED, class F>
__device__ __forceinline__ void over_rows(const EmbedArgs& a, uint32_t i, uint32_t end, F&& f) {
  const int lane = threadIdx.x & 63;
  for (; i < end; i += 64) {
    const int cnt = (int)min(64u, end - i);
    const uint32_t k = i + min(lane, cnt - 1);
    const uint4 r = a.rec[k];
    const int64_t off = record_off(r);
    const float w = WEIGHTED ? a.c[r.y] * a.scale : 1.f;
    f(off, w, cnt);
  }
}

// One wave's share of a row: U groups of 64 V columns from c0 on.
template <class E, int V, int U>
struct RowSum {
  // Rows loaded ahead: up to 96 registers of them.
  static constexpr int kMost = U * V * (int)sizeof(typename E::storage) / 4 <= 12 ? 8 : 4;
  float s[U][V];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) s[u][e] = 0.f;
  }
  // This lane's column of group u, within the row also where the group is
  // not (what is loaded there is never stored).
  static __device__ __forceinline__ int64_t column(int u, int64_t left) {
    const int64_t col = (int64_t)(u * 64 + (threadIdx.x & 63)) * V;
    return col < left ? col : left - V;
  }
  // += w row, for K rows given at the wave's first column
  template <class S, int K, class P, class W>
  __device__ __forceinline__ void add(int64_t left, P&& row, W&& weight) {
    Raw<S, V> x[K][U];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const typename S::storage* p = row(k);
#pragma unroll
      for (int u = 0; u < U; ++u) x[k][u] = load_raw<S, V>(p + column(u, left));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float w = weight(k);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) s[u][e] += w * raw_f32<S, V>(x[k][u], e);
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
  // The rows whose offsets and weights the first cnt lanes hold.
  __device__ __forceinline__ void batch(const EmbedArgs& a, int64_t c0, int64_t off, float w,
                                        int cnt) {
    const typename E::storage* G = (const typename E::storage*)a.G.data + c0;
    in_batches<kMost>(cnt, [&](int j, auto kk) {
      add<E, decltype(kk)::value>(a.D - c0, [&](int k) { return G + lane_i64(off, j + k); },
                                  [&](int k) { return lane_f32(w, j + k); });
    });
  }
  template <bool WEIGHTED>
  __device__ __forceinline__ void rows(const EmbedArgs& a, int64_t c0, uint32_t i, uint32_t end) {
    over_rows<WEIGHTED>(a, i, end, [&](int64_t off, float w, int cnt) { batch(a, c0, off, w, cnt); });
  }
  __device__ __forceinline__ void parts(const EmbedArgs& a, int64_t c0, uint32_t b, uint32_t end) {
    const float* p = a.blocks + (int64_t)b * a.D + c0;
    in_batches<U * V <= 16 ? 8 : 4>((int)(end - b), [&](int j, auto kk) {
      add<F32, decltype(kk)::value>(a.D - c0, [&](int k) { return p + (int64_t)(j + k) * a.D; },
                                    [](int) { return 1.f; });
    });
  }
};

__device__ __forceinline__ uint32_t wave_of_grid() {
  return blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// The blocks inside one run (WEIGHTED: one segment), one wave per block and
// column group.
template <class E, int V, int U, bool WEIGHTED>
__global__ void __launch_bounds__(256) embed_blocks_kernel(EmbedArgs a, uint32_t N) {
  const uint32_t b = wave_of_grid(), i = b * kBlock;
  if (i + kBlock > N) return;
  const uint4 r = a.rec[i + min(threadIdx.x & 63u, kBlock - 1)];
  const uint32_t v = __builtin_amdgcn_readlane(r.x, 0);
  if (v >= (uint32_t)a.V || v != __builtin_amdgcn_readlane(r.x, kBlock - 1)) return;
  if (!WEIGHTED && __builtin_amdgcn_readlane(r.y, 0) != __builtin_amdgcn_readlane(r.y, kBlock - 1)) return;
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * U);
  RowSum<E, V, U> sum;
  sum.zero();
  sum.batch(a, c0, record_off(r), WEIGHTED ? a.c[r.y] * a.scale : 1.f, kBlock);
  sum.store(a.blocks + (int64_t)b * a.D + c0, a.D - c0);
}

// One wave per 8 sorted positions and column group, for the runs that start
// there: the 8 rows are loaded together (most runs have one or two), a run's
// rows are summed (float32, in order) and the sum squared (float64).  A run
// that starts before the 8 is skipped, one that goes on past them is followed
// to its end.  partials[position][column group], positions in their original
// order, so that a sample's are contiguous; a run's value is written at its
// last position among the 8, and 0 at the others.
constexpr int kWindow = kBlock;
template <class E, int V, int U>
__global__ void __launch_bounds__(256) embed_norm_kernel(EmbedArgs a, const uint32_t* pos,
                                                         uint32_t N) {
  const int lane = threadIdx.x & 63;
  const uint32_t base = wave_of_grid() * kWindow;
  if (base >= N) return;
  // lane l: sorted position base + l - 1
  const bool in = base + lane >= 1 && base + lane - 1 < N;
  const uint4 r = a.rec[in ? base + lane - 1 : 0];
  const uint32_t where = lane < kWindow && base + lane < N ? pos[base + lane] : 0u;
  const int64_t off = record_off(r);
  const uint32_t pk = __shfl_up(r.x, 1, 64), pb = __shfl_up(r.y, 1, 64);
  const bool pin = __shfl_up((int)in, 1, 64) != 0 && lane > 0;
  // bit l: position base + l - 1 is of the same token (run) as the one before it
  const uint64_t same = __ballot(in && pin && pk == r.x);
  const uint64_t cont = same & __ballot(pb == r.y);
  const uint64_t act = __ballot(in && r.x < (uint32_t)a.V) >> 1;
  if (blockIdx.y == 0 && lane >= 1 && lane <= kWindow && in && r.x < (uint32_t)a.V) {
    if (!((same >> lane) & 1)) a.seg[r.x].x = base + lane - 1;
    if (!((same >> (lane + 1)) & 1)) a.seg[r.x].y = base + lane;
  }
  const int lead = __builtin_ctzll(~(cont >> 1));
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * U), left = a.D - c0;
  const typename E::storage* G = (const typename E::storage*)a.G.data + c0;
  double q[kWindow];
  RowSum<E, V, U> sum;
  Raw<E, V> x[kWindow][U];
#pragma unroll
  for (int j = 0; j < kWindow; ++j) {
    q[j] = 0.0;
    if (j < lead || !((act >> j) & 1)) continue;
    const typename E::storage* row = G + lane_i64(off, j + 1);
#pragma unroll
    for (int u = 0; u < U; ++u) x[j][u] = load_raw<E, V>(row + sum.column(u, left));
  }
  // V squares in float32, everything above in float64 (a conversion and a
  // float64 multiply per value would be as long as the loads).  Where a lane's
  // V squares leave float32's range, or come so near its lower end that one of
  // them may have, the wave squares in float64 (the check: 0.3 us of 29 at
  // 256 x 64 positions of 768 columns, 0.8 of 66 at 8 x 2048 of 5120).
  auto squares = [&]() {
    double s = 0.0;
    bool inside = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) v += sum.s[u][e] * sum.s[u][e];
      s += (int64_t)(u * 64 + lane) * V < left ? (double)v : 0.0;
      inside = inside && v >= 0x1p-96f && v < __builtin_huge_valf();
    }
    if (__ballot(!inside) != 0) {
      s = 0.0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const double d = (int64_t)(u * 64 + lane) * V < left ? (double)sum.s[u][e] : 0.0;
          s += d * d;
        }
    }
    return s;
  };
#pragma unroll
  for (int j = 0; j < kWindow; ++j) {
    if (j < lead || !((act >> j) & 1)) continue;
    const bool more = (cont >> (j + 1)) & 1, goes_on = (cont >> (j + 2)) & 1;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e)
        sum.s[u][e] = (more ? sum.s[u][e] : 0.f) + raw_f32<E, V>(x[j][u], e);
    if (!goes_on) {
      q[j] = squares();
    } else if (j == kWindow - 1) {
      const uint32_t v = __builtin_amdgcn_readlane(r.x, j + 1), b = __builtin_amdgcn_readlane(r.y, j + 1);
      const uint32_t i = base + kWindow;
      uint32_t end = i + (uint32_t)__builtin_ctzll(~(cont >> (kWindow + 1)));
      while (end >= base + 63 && end < N) {          // past the lanes' positions
        const uint32_t k = end + lane;
        const uint4 o = a.rec[min(k, N - 1)];
        const uint64_t other = __ballot(k >= N || o.x != v || o.y != b);
        end += other != 0 ? (uint32_t)__builtin_ctzll(other) : 64u;
        if (other != 0) break;
      }
      end = __builtin_amdgcn_readfirstlane(end);
      uint32_t rest = i;                             // a block starts here
      if (a.blocks != nullptr) {
        rest = end / kBlock * kBlock;
        sum.parts(a, c0, i / kBlock, rest / kBlock);
      }
      sum.template rows<false>(a, c0, rest, end);
      q[j] = squares();
    }
  }
  // all eight sums over the wave: halves of the values change sides while
  // there are several, then the lanes of one value add up; lane 8 j has q[j]
#pragma unroll
  for (int n = kWindow / 2, o = 32; n >= 1; n /= 2, o /= 2)
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const double keep = (lane & o) ? q[j + n] : q[j], give = (lane & o) ? q[j] : q[j + n];
      q[j] = keep + lane_xor(give, o);
    }
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) q[0] += lane_xor(q[0], o);
  const uint32_t at = __shfl(where, lane >> 3, 64);
  if ((lane & 7) == 0 && base + (lane >> 3) < N)
    a.partials[(int64_t)at * gridDim.y + blockIdx.y] = q[0] * (double)a.scale * (double)a.scale;
}

// The rows of the result in U groups of 256 columns (gridDim.y of them at a
// time).  A thread's four values are one Philox block: with D % 4 != 0 (AL
// false) the groups start at the block that holds the row's first value, and
// each row keeps its own part of a shared block.
//
// The first `shared` workgroups look for segments with a block of their own,
// one candidate each.  There the four waves take a quarter of the blocks, the
// first the rows before them too and the last the rows after, and the four
// sums are added in order.  The other rows get one wave each, so that the
// longest segments are summed next to them and not before them.
template <class E, int U, bool AL>
__global__ void __launch_bounds__(256) embed_accumulate_kernel(EmbedArgs a, uint32_t shared) {
  __shared__ f32x4 part[3][U][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool share = blockIdx.x < shared;
  uint32_t v, b0, b1 = 0;
  if (share) {
    b0 = blockIdx.x;
    v = su32(&a.rec[b0 * kBlock].x, 0);
    if (v >= (uint32_t)a.V || v != su32(&a.rec[b0 * kBlock + kBlock - 1].x, 0)) return;
  } else {
    v = (blockIdx.x - shared) * 4 + wave;
    if (v >= (uint32_t)a.V) return;
  }
  const uint32_t first = su32(&a.seg[v].x, 0), end = su32(&a.seg[v].y, 0);
  const bool empty = first >= end;
  if (share) {
    if ((first + kBlock - 1) / kBlock != b0) return;         // not its first block
    b1 = end / kBlock;
  } else {
    if (empty && a.beta && a.noise_std == 0.0f) return;      // nothing is added to it
    b0 = (first + kBlock - 1) / kBlock;
    if (shared != 0 && !empty && (b0 + 1) * kBlock <= end) return;   // done by a workgroup
  }
  // this wave's rows, and after them its blocks [pb, pe)
  const uint32_t r0 = share && wave == 3 ? b1 * kBlock : first;
  const uint32_t r1 = !share || wave == 3 ? end : wave == 0 ? b0 * kBlock : first;
  const uint32_t pb = b0 + (b1 - b0) * wave / 4, pe = b0 + (b1 - b0) * (wave + 1) / 4;
  const int64_t row0 = (int64_t)v * a.D, start = AL ? row0 : row0 & ~(int64_t)3;
  const int64_t D = a.D;
  const float rd = 1.0f / a.denom;
  for (int64_t g0 = (int64_t)blockIdx.y * (256 * U); start + g0 < row0 + D;
       g0 += (int64_t)gridDim.y * (256 * U)) {
    // First of the thread's four columns (may be below 0), and a place within
    // the row to load from also where they are not.
    int64_t col[U], in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      col[u] = start - row0 + g0 + (u * 64 + lane) * 4;
      in[u] = AL ? (col[u] < D ? col[u] : D - 4) : col[u];
    }
    // Four values of a row of `S`: one load, or (AL false) element by element.
    auto fetch = [&](auto e, const auto* row, int u) {
      using S = decltype(e);
      Raw<S, 4> x;
      if constexpr (AL) {
        x = load_raw<S, 4>(row + in[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t c = in[u] + k;
          x[k] = row[c < 0 ? 0 : c < D ? c : D - 1];
        }
      }
      return x;
    };
    f32x4 old[U];
    float sum[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[u][e] = 0.f;
      old[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // The result is read and written once: past the caches, which G needs.
    if (a.beta && (!share || wave == 0))
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (AL) old[u] = __builtin_nontemporal_load((const f32x4*)(a.out + row0 + in[u]));
        else old[u] = fetch(F32(), a.out + row0, u);
      }
    over_rows<true>(a, r0, r1, [&](int64_t off, float w, int cnt) {
      in_batches<4>(cnt, [&](int j, auto kk) {
        constexpr int K = decltype(kk)::value;
        Raw<E, 4> x[K][U];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int u = 0; u < U; ++u)
            x[k][u] = fetch(E(), (const typename E::storage*)a.G.data + lane_i64(off, j + k), u);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float wk = lane_f32(w, j + k);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u][e] += wk * raw_f32<E, 4>(x[k][u], e);
        }
      });
    });
    if (share) {
      in_batches<sizeof(typename E::storage)>((int)(pe - pb), [&](int j, auto kk) {
        constexpr int K = decltype(kk)::value;
        f32x4 x[K][U];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int u = 0; u < U; ++u) x[k][u] = fetch(F32(), a.blocks + (int64_t)(pb + j + k) * D, u);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u][e] += x[k][u][e];
      });
      if (wave > 0)
#pragma unroll
        for (int u = 0; u < U; ++u)
          part[wave - 1][u][lane] = f32x4{sum[u][0], sum[u][1], sum[u][2], sum[u][3]};
      __syncthreads();
      if (wave == 0)
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const f32x4 x = part[w][u][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u][e] += x[e];
          }
      __syncthreads();                           // before the next columns' parts
      if (wave > 0) continue;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (col[u] >= D) continue;
      const int64_t e0 = row0 + col[u];
      if (a.noise_std != 0.0f) {
        const f32x4 z = normals_of_block_hw(philox_block_xor3(a.seed, a.offset + (uint64_t)(e0 >> 2)));
        sum[u][0] += a.noise_std * z.x; sum[u][1] += a.noise_std * z.y;
        sum[u][2] += a.noise_std * z.z; sum[u][3] += a.noise_std * z.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[u][e] = old[u][e] + sum[u][e] * rd;
      float* o = a.out + e0;
      if (AL || (col[u] >= 0 && col[u] + 4 <= D)) {
        __builtin_nontemporal_store(f32x4{sum[u][0], sum[u][1], sum[u][2], sum[u][3]}, (f32x4*)o);
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
  const unsigned lds = last ? 0u : (unsigned)(p.blocks << p.digit) * 4u;
  if (first && last) hipLaunchKernelGGL((sort_scatter_kernel<PER, true, true>), grid, block, lds, s, a, p);
  else if (first) hipLaunchKernelGGL((sort_scatter_kernel<PER, true, false>), grid, block, lds, s, a, p);
  else if (last) hipLaunchKernelGGL((sort_scatter_kernel<PER, false, true>), grid, block, lds, s, a, p);
  else hipLaunchKernelGGL((sort_scatter_kernel<PER, false, false>), grid, block, lds, s, a, p);
}

template <int PER>
hipError_t launch_small(const EmbedArgs& a, const SortPlan& p, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)sort_small_kernel<PER>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               small_lds<PER>());
  if (once != hipSuccess) return once;
  const int at = embed_sorted(a.V, -1);
  const int clear = (int)std::min<int64_t>(256, (a.V + kSmallThreads - 1) / kSmallThreads);
  hipLaunchKernelGGL((sort_small_kernel<PER>), dim3((unsigned)(1 + clear)), dim3(kSmallThreads),
                     small_lds<PER>(), s, a, (uint32_t)(a.B * a.T), p.passes, p.digit, a.pos[at]);
  return hipGetLastError();
}

// More LDS than the default limit, once per scatter kernel that counts the
// next digit.
template <int PER>
hipError_t scatter_attributes() {
  const int most = kSortBlocks * kMaxBins * 4;
  static hipError_t once = [&] {
    hipError_t e = hipFuncSetAttribute((const void*)sort_scatter_kernel<PER, true, false>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == hipSuccess)
      e = hipFuncSetAttribute((const void*)sort_scatter_kernel<PER, false, false>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, most);
    return e;
  }();
  return once;
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
  if (N <= kSmallN) {
    const hipError_t e = N <= kSmallThreads ? launch_small<1>(a, p, s) : launch_small<2>(a, p, s);
    timing_end("embed_sort", s);
    return e;
  }
  const hipError_t ready = p.per == 1 ? scatter_attributes<1>() : p.per == 2 ? scatter_attributes<2>()
                         : p.per == 4 ? scatter_attributes<4>() : scatter_attributes<8>();
  if (ready != hipSuccess) return ready;
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

hipError_t launch_embed_segments(const EmbedArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)(a.B * a.T);
  hipLaunchKernelGGL(embed_segments_kernel, dim3((N + 255) / 256), dim3(256), 0, s, a, N);
  return hipGetLastError();
}

hipError_t launch_embed_norm(const EmbedArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)(a.B * a.T);
  const unsigned parts = (unsigned)embed_norm_parts(a);
  const uint32_t* pos = a.pos[embed_sorted(a.V, -1)];
  EmbedArgs q = a;
  if (a.T <= kShortRuns) q.blocks = nullptr;
  timing_begin("embed_norm", s);
  with_rows(a, [&](auto e, auto v, auto u) {
    using E = decltype(e);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    if (q.blocks != nullptr)
      hipLaunchKernelGGL((embed_blocks_kernel<E, V, U, false>), dim3((N / kBlock + 3) / 4, parts),
                         dim3(256), 0, s, q, N);
    hipLaunchKernelGGL((embed_norm_kernel<E, V, U>), dim3((N + 4 * kWindow - 1) / (4 * kWindow), parts),
                       dim3(256), 0, s, q, pos, N);
  });
  timing_end("embed_norm", s);
  return hipGetLastError();
}

namespace {

template <class E, bool AL>
void accumulate_u(const EmbedArgs& a, int U, dim3 grid, uint32_t shared, hipStream_t s) {
  switch (U) {
    case 1: hipLaunchKernelGGL((embed_accumulate_kernel<E, 1, AL>), grid, dim3(256), 0, s, a, shared); break;
    case 2: hipLaunchKernelGGL((embed_accumulate_kernel<E, 2, AL>), grid, dim3(256), 0, s, a, shared); break;
    case 3: hipLaunchKernelGGL((embed_accumulate_kernel<E, 3, AL>), grid, dim3(256), 0, s, a, shared); break;
    case 4: hipLaunchKernelGGL((embed_accumulate_kernel<E, 4, AL>), grid, dim3(256), 0, s, a, shared); break;
    default: hipLaunchKernelGGL((embed_accumulate_kernel<E, 5, AL>), grid, dim3(256), 0, s, a, shared);
  }
}

}  // namespace

hipError_t launch_embed_accumulate(const EmbedArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)(a.B * a.T);
  const unsigned parts = (unsigned)embed_norm_parts(a);
  const uint32_t shared = a.blocks != nullptr ? N / kBlock : 0;
  timing_begin("embed_accumulate", s);
  if (a.blocks != nullptr)
    with_rows(a, [&](auto e, auto v, auto u) {
      using E = decltype(e);
      constexpr int V = decltype(v)::value, U = decltype(u)::value;
      const dim3 grid((N / kBlock + 3) / 4, parts);
      hipLaunchKernelGGL((embed_blocks_kernel<E, V, U, true>), grid, dim3(256), 0, s, a, N);
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
  const dim3 grid((unsigned)(shared + (a.V + 3) / 4), (unsigned)gy);
  if (a.dtype == kBF16) {
    if (al) accumulate_u<BF16, true>(a, U, grid, shared, s);
    else accumulate_u<BF16, false>(a, U, grid, shared, s);
  } else {
    if (al) accumulate_u<F32, true>(a, U, grid, shared, s);
    else accumulate_u<F32, false>(a, U, grid, shared, s);
  }
  timing_end("embed_accumulate", s);
  return hipGetLastError();
}

}  // namespace dpf
