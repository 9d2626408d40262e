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
//                            the id V and end up last
//  embed_rows              : per sorted position, where its row of G starts
//                            and its sample; per table row, its segment
//  embed_norm              : one wave per run and column block
//  embed_accumulate        : every row of the result, noise included
#include <algorithm>

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
constexpr int kSortPer = 4;                              // keys per thread and chunk
constexpr int kSortChunk = kSortThreads * kSortPer;
constexpr int kSortBlocks = 128;                         // most workgroups
constexpr int kMaxDigit = 9, kMaxBins = 1 << kMaxDigit;

struct SortPlan {
  int bits, passes, digit, blocks, chunks;   // chunks per workgroup
};

SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan p;
  p.bits = 1;
  while (((int64_t)1 << p.bits) <= V) ++p.bits;          // keys 0 .. V
  p.passes = (p.bits + kMaxDigit - 1) / kMaxDigit;
  p.digit = (p.bits + p.passes - 1) / p.passes;
  const int64_t chunks = (N + kSortChunk - 1) / kSortChunk;
  p.chunks = (int)((chunks + kSortBlocks - 1) / kSortBlocks);
  p.blocks = (int)((chunks + p.chunks - 1) / p.chunks);
  return p;
}

__device__ __forceinline__ uint32_t token_key(const EmbedArgs& a, int64_t n) {
  if (a.mask != nullptr && a.mask[n] == 0) return (uint32_t)a.V;
  const int64_t b = n / a.T;
  const int64_t id = a.ids.at(b, n - b * a.T);
  return id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

// Digit counts of each workgroup's keys.  Workgroups past `blocks` (first
// pass) clear the segments.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(EmbedArgs a, const uint32_t* key,
                                                                 int64_t N, int shift, int bins,
                                                                 int blocks, int chunks) {
  if (FIRST && (int)blockIdx.x >= blocks) {
    const int64_t step = (int64_t)(gridDim.x - blocks) * kSortThreads;
    for (int64_t v = (int64_t)(blockIdx.x - blocks) * kSortThreads + threadIdx.x; v < a.V; v += step)
      a.seg[v] = make_uint2(0u, 0u);
    return;
  }
  __shared__ uint32_t cnt[kMaxBins];
  for (int d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * chunks * kSortChunk;
  const int64_t n1 = min(N, n0 + (int64_t)chunks * kSortChunk);
  for (int64_t n = n0 + threadIdx.x; n < n1; n += kSortThreads) {
    const uint32_t k = FIRST ? token_key(a, n) : key[n];
    atomicAdd(&cnt[(k >> shift) & (uint32_t)(bins - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) a.hist[(int64_t)blockIdx.x * bins + d] = cnt[d];
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
  __syncthreads();
  return before + x - v;
}

// Moves every key (and its position) to its place in the digit's order.  A
// key's rank among equal digits counts the keys before it: those of earlier
// workgroups (from the histograms), chunks and waves, and within a wave's 64
// keys the lanes below it with the same digit (found by ballots on its bits).
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(
    EmbedArgs a, const uint32_t* key, const uint32_t* pos, uint32_t* key_out, uint32_t* pos_out,
    int64_t N, int shift, int digit, int blocks, int chunks) {
  __shared__ uint32_t base[kMaxBins];
  __shared__ uint32_t wcnt[kSortWaves][kMaxBins];
  __shared__ uint32_t tmp[kSortWaves];
  const int bins = 1 << digit, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  {
    uint32_t total = 0, before = 0;
    if (tid < bins) {
#pragma unroll 8
      for (int w = 0; w < blocks; ++w) {
        const uint32_t h = a.hist[(int64_t)w * bins + tid];
        before += w < (int)blockIdx.x ? h : 0u;
        total += h;
      }
    }
    const uint32_t ex = block_exclusive(total, tmp);
    if (tid < bins) base[tid] = ex + before;
  }
  const int64_t n0 = (int64_t)blockIdx.x * chunks * kSortChunk;
  for (int ch = 0; ch < chunks; ++ch) {
    const int64_t c0 = n0 + (int64_t)ch * kSortChunk;
    if (c0 >= N) break;
    for (int d = lane; d < bins; d += 64) wcnt[wave][d] = 0;
    __syncthreads();
    uint32_t k[kSortPer], p[kSortPer], r[kSortPer];
#pragma unroll
    for (int i = 0; i < kSortPer; ++i) {
      const int64_t n = c0 + wave * (64 * kSortPer) + i * 64 + lane;
      const bool in = n < N;
      k[i] = !in ? 0u : FIRST ? token_key(a, n) : key[n];
      p[i] = !in ? 0u : FIRST ? (uint32_t)n : pos[n];
      const uint32_t d = (k[i] >> shift) & (uint32_t)(bins - 1);
      uint64_t same = __ballot(in);
      for (int j = 0; j < digit; ++j) {
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
    for (int d = tid; d < bins; d += kSortThreads) {
      uint32_t at = base[d];
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = wcnt[w][d];
        wcnt[w][d] = at;
        at += c;
      }
      base[d] = at;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortPer; ++i) {
      const int64_t n = c0 + wave * (64 * kSortPer) + i * 64 + lane;
      if (n < N) {
        const uint32_t to = wcnt[wave][(k[i] >> shift) & (uint32_t)(bins - 1)] + r[i];
        key_out[to] = k[i];
        pos_out[to] = p[i];
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) embed_rows_kernel(EmbedArgs a, const uint32_t* key,
                                                         const uint32_t* pos, int64_t N) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (k >= N) return;
  const uint32_t v = key[k], p = pos[k];
  const uint32_t b = p / (uint32_t)a.T, t = p - b * (uint32_t)a.T;
  a.off[k] = (int64_t)b * a.G.stride_b + (int64_t)t * a.G.stride_t;
  a.smp[k] = b;
  if (v >= (uint32_t)a.V) return;
  if (k == 0 || key[k - 1] != v) a.seg[v].x = (uint32_t)k;
  if (k == N - 1 || key[k + 1] != v) a.seg[v].y = (uint32_t)(k + 1);
}

// ---------------------------------------------------------------------------
// Norms
// ---------------------------------------------------------------------------
constexpr int kNormU = 2;   // column groups of 64 V per wave

// One wave per sorted position and column block.  The first position of a run
// sums the run's rows (float32, in order) and squares the sum (float64); the
// others write 0.  partials[position][column block], positions in their
// original order, so that a sample's are contiguous.
template <class E, int V>
__global__ void __launch_bounds__(256) embed_norm_kernel(EmbedArgs a, const uint32_t* key,
                                                         const uint32_t* pos, int64_t N) {
  const int lane = threadIdx.x & 63;
  const int64_t k = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (k >= N) return;
  double* dst = a.partials + (int64_t)pos[k] * gridDim.y + blockIdx.y;
  const uint32_t v = key[k], b = a.smp[k];
  if (v >= (uint32_t)a.V || (k > 0 && key[k - 1] == v && a.smp[k - 1] == b)) {
    if (lane == 0) *dst = 0.0;
    return;
  }
  const typename E::storage* G = (const typename E::storage*)a.G.data;
  float sum[kNormU][V];
#pragma unroll
  for (int u = 0; u < kNormU; ++u)
#pragma unroll
    for (int e = 0; e < V; ++e) sum[u][e] = 0.f;
  const int64_t c0 = (int64_t)blockIdx.y * (64 * V * kNormU) + lane * V;
  for (int64_t i = k; i < N && key[i] == v && a.smp[i] == b; ++i) {
    const typename E::storage* row = G + a.off[i];
#pragma unroll
    for (int u = 0; u < kNormU; ++u) {
      const int64_t col = c0 + u * 64 * V;
      if (col < a.D) {
        float x[V];
        load_f32<E, V>(row + col, x);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[u][e] += x[e];
      }
    }
  }
  double sq = 0.0;
#pragma unroll
  for (int u = 0; u < kNormU; ++u)
#pragma unroll
    for (int e = 0; e < V; ++e) sq += (double)sum[u][e] * (double)sum[u][e];
  sq = wave_sum_f64(sq);
  if (lane == 0) *dst = sq * (double)a.scale * (double)a.scale;
}

// ---------------------------------------------------------------------------
// Clipped sum
// ---------------------------------------------------------------------------
// D % 4 == 0: 4 columns (one Philox block) per thread, L lanes per row.
template <class E>
__global__ void __launch_bounds__(256) embed_accumulate_kernel(EmbedArgs a, int L) {
  const int64_t v = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int64_t col = ((int64_t)blockIdx.y * L + (threadIdx.x & (unsigned)(L - 1))) * 4;
  if (v >= a.V || col >= a.D) return;
  const typename E::storage* G = (const typename E::storage*)a.G.data + col;
  const uint2 seg = a.seg[v];
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t i = seg.x; i < seg.y; ++i) {
    float x[4];
    load_f32<E, 4>(G + a.off[i], x);
    const float w = a.c[a.smp[i]] * a.scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += w * x[e];
  }
  const float r = 1.0f / a.denom;
  const int64_t e0 = v * a.D + col;
  if (a.noise_std != 0.0f) {
    const f32x4 z = normals_of_block(philox_block(a.seed, a.offset + (uint64_t)(e0 >> 2)));
    sum[0] += a.noise_std * z.x; sum[1] += a.noise_std * z.y;
    sum[2] += a.noise_std * z.z; sum[3] += a.noise_std * z.w;
  }
  float* o = a.out + e0;
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] *= r;
  if (a.beta) {
    float old[4];
    load_f32<F32, 4>(o, old);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += old[e];
  }
  store_f32<F32, 4>(o, sum);
}

// Any D and strides: 4 consecutive elements of the flat result per thread.
template <class E>
__global__ void __launch_bounds__(256) embed_accumulate_flat_kernel(EmbedArgs a) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t e0 = 4 * j, total = a.V * a.D;
  if (e0 >= total) return;
  float z[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.noise_std != 0.0f) {
    const f32x4 w = normals_of_block(philox_block(a.seed, a.offset + (uint64_t)j));
    z[0] = w.x; z[1] = w.y; z[2] = w.z; z[3] = w.w;
  }
  const float r = 1.0f / a.denom;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t e = e0 + q;
    if (e >= total) break;
    const int64_t v = e / a.D, col = e - v * a.D;
    const uint2 seg = a.seg[v];
    float sum = 0.f;
    for (uint32_t i = seg.x; i < seg.y; ++i)
      sum += a.c[a.smp[i]] * a.scale * E::to_float(((const typename E::storage*)a.G.data)[a.off[i] + col]);
    sum = (sum + a.noise_std * z[q]) * r;
    a.out[e] = a.beta ? a.out[e] + sum : sum;
  }
}

// Elements per load for rows of D that start stride_b, stride_t apart.
int row_vec(const Act& G, int64_t D) {
  if (D % 8 == 0 && G.stride_t % 8 == 0 && G.stride_b % 8 == 0) return 8;
  if (D % 4 == 0 && G.stride_t % 4 == 0 && G.stride_b % 4 == 0) return 4;
  return 1;
}

template <class E>
void norm_v(const EmbedArgs& a, int V, dim3 grid, const uint32_t* key, const uint32_t* pos,
            int64_t N, hipStream_t s) {
  if (V == 8) hipLaunchKernelGGL((embed_norm_kernel<E, 8>), grid, dim3(256), 0, s, a, key, pos, N);
  else if (V == 4) hipLaunchKernelGGL((embed_norm_kernel<E, 4>), grid, dim3(256), 0, s, a, key, pos, N);
  else hipLaunchKernelGGL((embed_norm_kernel<E, 1>), grid, dim3(256), 0, s, a, key, pos, N);
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
  return (int64_t)p.blocks << p.digit;
}

int embed_norm_parts(const EmbedArgs& a) {
  const int cols = 64 * row_vec(a.G, a.D) * kNormU;
  return (int)((a.D + cols - 1) / cols);
}

int embed_sorted(int64_t V) { return (sort_plan(1, V).passes & 1) ? 0 : 1; }

hipError_t launch_embed_sort(const EmbedArgs& a, hipStream_t s) {
  const int64_t N = a.B * a.T;
  const SortPlan p = sort_plan(N, a.V);
  const int bins = 1 << p.digit;
  timing_begin("embed_sort", s);
  for (int q = 0; q < p.passes; ++q) {
    const int shift = q * p.digit, to = q & 1, from = to ^ 1;
    if (q == 0) {
      const int clear = (int)std::min<int64_t>(256, (a.V + kSortThreads - 1) / kSortThreads);
      hipLaunchKernelGGL((sort_hist_kernel<true>), dim3((unsigned)(p.blocks + clear)),
                         dim3(kSortThreads), 0, s, a, (const uint32_t*)nullptr, N, shift, bins,
                         p.blocks, p.chunks);
      hipLaunchKernelGGL((sort_scatter_kernel<true>), dim3((unsigned)p.blocks), dim3(kSortThreads),
                         0, s, a, (const uint32_t*)nullptr, (const uint32_t*)nullptr, a.key[to],
                         a.pos[to], N, shift, p.digit, p.blocks, p.chunks);
    } else {
      hipLaunchKernelGGL((sort_hist_kernel<false>), dim3((unsigned)p.blocks), dim3(kSortThreads), 0,
                         s, a, (const uint32_t*)a.key[from], N, shift, bins, p.blocks, p.chunks);
      hipLaunchKernelGGL((sort_scatter_kernel<false>), dim3((unsigned)p.blocks), dim3(kSortThreads),
                         0, s, a, (const uint32_t*)a.key[from], (const uint32_t*)a.pos[from],
                         a.key[to], a.pos[to], N, shift, p.digit, p.blocks, p.chunks);
    }
  }
  const int at = embed_sorted(a.V);
  hipLaunchKernelGGL(embed_rows_kernel, dim3((unsigned)((N + 255) / 256)), dim3(256), 0, s, a,
                     (const uint32_t*)a.key[at], (const uint32_t*)a.pos[at], N);
  timing_end("embed_sort", s);
  return hipGetLastError();
}

hipError_t launch_embed_norm(const EmbedArgs& a, hipStream_t s) {
  const int64_t N = a.B * a.T;
  const int at = embed_sorted(a.V), V = row_vec(a.G, a.D);
  const dim3 grid((unsigned)((N + 3) / 4), (unsigned)embed_norm_parts(a));
  timing_begin("embed_norm", s);
  if (a.dtype == kBF16) norm_v<BF16>(a, V, grid, a.key[at], a.pos[at], N, s);
  else norm_v<F32>(a, V, grid, a.key[at], a.pos[at], N, s);
  timing_end("embed_norm", s);
  return hipGetLastError();
}

hipError_t launch_embed_accumulate(const EmbedArgs& a, hipStream_t s) {
  timing_begin("embed_accumulate", s);
  if (row_vec(a.G, a.D) >= 4) {
    int L = 1;
    while (L < 256 && (int64_t)L * 4 < a.D) L *= 2;
    const dim3 grid((unsigned)((a.V + 256 / L - 1) / (256 / L)), (unsigned)((a.D + 4 * L - 1) / (4 * L)));
    if (a.dtype == kBF16) hipLaunchKernelGGL((embed_accumulate_kernel<BF16>), grid, dim3(256), 0, s, a, L);
    else hipLaunchKernelGGL((embed_accumulate_kernel<F32>), grid, dim3(256), 0, s, a, L);
  } else {
    const dim3 grid((unsigned)((a.V * a.D + 1023) / 1024));
    if (a.dtype == kBF16) hipLaunchKernelGGL((embed_accumulate_flat_kernel<BF16>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((embed_accumulate_flat_kernel<F32>), grid, dim3(256), 0, s, a);
  }
  timing_end("embed_accumulate", s);
  return hipGetLastError();
}

}  // namespace dpf
