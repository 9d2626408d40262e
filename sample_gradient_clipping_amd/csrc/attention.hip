// Attention over the positions of each sample, forward.
//
//   position p of query i:  p = Tk - Tq + i   (the queries are the last Tq positions)
//   A(i) = keys j of p's segment with mask[j] != 0, j <= p if causal; empty
//          where mask[p] = 0
//   s_ij = scale q_i . k_j,  lse_i = log sum_A e^{s_ij},  out_i = sum_A e^{s_ij - lse_i} v_j
//
// One pass over the keys with a running maximum and sum.  A workgroup of four
// waves takes 128 queries of one head, each wave 32; tiles of keys and values
// go through LDS, twice buffered, by direct loads.  Scores are computed
// transposed, S^T = K Q^T: a lane then holds one query's scores, so that the
// softmax is arithmetic within lanes (one exchange between the two lane halves
// per tile, for the maximum), and the exponentials are, as they lie in the
// accumulator's registers, the right operand of O^T = V^T P^T (with the rows of
// V read in the accumulator's order by the transposing LDS reads).  The
// exponentials are rounded to bf16 for that product (what its operand type
// holds); their sum is that of the unrounded ones (lse is float32), and it, the
// maximum and the output stay in float32.
#include "attn.hpp"

#include <algorithm>

namespace dpf {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kNT = 64 * kWaves;
constexpr int kQ = 32 * kWaves;         // queries of a workgroup
// The running maximum follows the scores only where they rise above it by more
// than this (in powers of two): the weights then stay below 2^8, and a tile that
// raises no maximum rescales nothing.
constexpr float kSlack = 8.0f;

template <class E> struct KeysOf;
template <> struct KeysOf<BF16> { static constexpr int kKeys = 64; };
template <> struct KeysOf<F32> { static constexpr int kKeys = 32; };

// ---------------------------------------------------------------------------
// Mask and segments
// ---------------------------------------------------------------------------
// Each wave takes 64 positions of a sample.  lo: the first active position of
// the segment, end: one past its last active one (0, 0 for an inactive
// position), so a causal row with one key has lo == p and any other with one
// key end == lo + 1.  Segment numbers do not decrease, so the start of the
// first position's segment and the end of the last one's are found by 64-way
// search, the boundaries between by a vote.
__device__ __forceinline__ int first_from(const int32_t* id, int l, int r, int32_t least, int lane) {
  // smallest index in [l, r) whose id is >= least, else r
  while (l < r) {
    const int step = (r - l + 63) / 64;
    const int at = l + lane * step;
    const bool in = at < r;
    const uint64_t hit = __ballot(in && id[in ? at : l] >= least);
    const int probes = __popcll(__ballot(in));
    if (hit == 0) {
      l = l + (probes - 1) * step + 1;
    } else {
      const int f = __ffsll((unsigned long long)hit) - 1;
      r = l + f * step;
      l = f > 0 ? l + (f - 1) * step + 1 : r;
    }
  }
  return r;
}

__global__ __launch_bounds__(256) void attn_ranges_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63, T = a.Tk, blocks = (T + 255) / 256;
  const int b = blockIdx.x / blocks;
  const int t0 = 64 * (int)(blockIdx.x % blocks * 4 + (threadIdx.x >> 6));
  if (t0 >= T) return;
  const int64_t row = (int64_t)b * T;
  const int t = t0 + lane, n = min(64, T - t0);
  const bool inside = lane < n;
  const bool act = inside && (a.mask == nullptr || a.mask[row + t] != 0);
  const uint64_t live = __ballot(act);
  if (lane < 2) a.bits[(int64_t)b * a.nwords + t0 / 32 + lane] = (uint32_t)(live >> (32 * lane));
  // segments: their starts within the wave, the first one's start, the last one's end
  uint64_t starts = 0;
  int s0 = 0, e0 = T;
  if (a.segments != nullptr) {
    const int32_t* id = a.segments + row;
    const int32_t own = id[inside ? t : t0];
    const int32_t before = __shfl_up(own, 1);
    starts = __ballot(inside && lane > 0 && own != before);
    s0 = first_from(id, 0, t0, __shfl(own, 0), lane);
    const int32_t last = __shfl(own, n - 1);
    e0 = last == INT32_MAX ? T : first_from(id, t0 + n, T, last + 1, lane);
  }
  // the first active position in [s0, t0), the last in [t0 + n, e0)
  int f0 = -1, l0 = -1;
  if (live != 0) {
    if (a.mask == nullptr) {
      if (s0 < t0) f0 = s0;
      if (e0 > t0 + n) l0 = e0 - 1;
    } else {
      for (int at = s0; at < t0 && f0 < 0; at += 64) {
        const uint64_t m = __ballot(at + lane < t0 && a.mask[row + min(at + lane, T - 1)] != 0);
        if (m != 0) f0 = at + __ffsll((unsigned long long)m) - 1;
      }
      if (!a.causal)
        for (int at = e0; at > t0 + n && l0 < 0; at -= 64) {
          const int k = at - 64 + lane;
          const uint64_t m = __ballot(k >= t0 + n && a.mask[row + max(k, 0)] != 0);
          if (m != 0) l0 = at - 64 + 63 - __clzll((long long)m);
        }
    }
  }
  if (!inside) return;
  int lo = 0, end = 0;
  if (act) {
    const uint64_t upto = lane == 63 ? ~0ull : (2ull << lane) - 1;
    const uint64_t below = starts & upto, above = starts & ~upto;
    if (below != 0) {
      const int s = 63 - __clzll((long long)below);
      lo = t0 + __ffsll((unsigned long long)(live >> s << s)) - 1;
    } else {
      lo = f0 >= 0 ? f0 : t0 + __ffsll((unsigned long long)live) - 1;
    }
    if (above != 0) {
      const int e = __ffsll((unsigned long long)above) - 1;      // > lane
      end = t0 + 64 - __clzll((long long)(live & ((1ull << e) - 1)));
    } else if (a.causal && a.mask != nullptr) {
      end = e0;    // not tightened: a causal row ends at itself
    } else {
      end = l0 >= 0 ? l0 + 1 : t0 + 64 - __clzll((long long)live);
    }
  }
  a.lo[row + t] = lo;
  a.end[row + t] = end;
}

// ---------------------------------------------------------------------------
// A wave's 32 queries and one tile of keys
// ---------------------------------------------------------------------------
template <class E, int DP>
struct State {
  f32x16 o[DP / 32];    // O^T: this lane's query, relative to m
  float m, l;           // maximum used (times log2 e) and this lane half's sum
};

// The tile goes by blocks of 32 keys: while the matrix cores take the scores of
// the next block, or the outputs of the last one, the vector unit takes the
// exponentials of this one.  The order is written out, step by step between
// fences, with every LDS operand read kAhead products early: left to itself the
// compiler waits for each read, and puts all exponentials before all products.
template <class E, int DP, int KEYS>
__device__ __forceinline__ void attend(const Places& kt, const Places& vt,
                                       const Chunk<E> (&qf)[Shape<E, DP>::kG], State<E, DP>& st, float c,
                                       int k0, Span keys, bool full, const uint32_t (&live)[KEYS / 32],
                                       int lane) {
  constexpr int NB = KEYS / 32, G = Shape<E, DP>::kG, DB = DP / 32, CS = ColumnSteps<E>::kN;
  const int h = lane >> 5;
  f32x16 s[2];
  Weights<E> p[2];
  float m = 0.0f, sum[2] = {};

  const auto exponential = [&](int n, int j) {
    float x = __builtin_amdgcn_exp2f(fmaf(s[n & 1][j], c, -m));
    asm volatile("" : "+v"(x));    // here, not where it is used first
    s[n & 1][j] = x;
    sum[j & 1] += x;
  };
  // scores of block n, with the exponentials of block n - 1 between the products
  const auto scores = [&](int n) {
    Chunk<E> k[kAhead];
    f32x16 x = {};
#pragma unroll
    for (int g = 0; g < kAhead; ++g) k[g] = row_frag<E, DP>(kt, 32 * n, g);
    fence();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      x = mma<E>(k[g % kAhead], qf[g], x);
      if (g + kAhead < G) k[g % kAhead] = row_frag<E, DP>(kt, 32 * n, g + kAhead);
      if (n > 0) {
#pragma unroll
        for (int j = 16 * g / G; j < 16 * (g + 1) / G; ++j) exponential(n - 1, j);
      }
      fence();
    }
    s[n & 1] = x;
  };
  // outputs from block n, with the exponentials of block n + 1 between the products
  const auto outputs = [&](int n, bool more) {
    constexpr int N = DB * CS;
    Column<E> v[kAhead];
    const auto read = [&](int t) { return column_frag<E, DP>(vt, 32 * n, t % DB, t / DB, lane); };
#pragma unroll
    for (int t = 0; t < kAhead; ++t) v[t] = read(t);
    fence();
#pragma unroll
    for (int t = 0; t < N; ++t) {
      st.o[t % DB] = mma_column<E>(v[t % kAhead], p[n & 1], t / DB, st.o[t % DB]);
      if (t + kAhead < N) v[t % kAhead] = read(t + kAhead);
      if (more) {
#pragma unroll
        for (int j = 16 * t / N; j < 16 * (t + 1) / N; ++j) exponential(n + 1, j);
      }
      fence();
    }
  };
  // masks block n and moves the running maximum to it
  const auto settle = [&](int n) {
    if (!full) {
      apart();
      const uint32_t w = live[n] >> (4 * h);
      const int first = keys.lo - k0 - 32 * n - 4 * h, past = keys.end - k0 - 32 * n - 4 * h;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int r = 8 * (j >> 2) + (j & 3);
        const bool in = r >= first && r < past && ((w >> r) & 1);
        s[n & 1][j] = in ? s[n & 1][j] : -INFINITY;
      }
    }
    float top = s[n & 1][0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, s[n & 1][j]);
    top = fmaxf(top, lane_xor(top, 32)) * c;
    if (__any(top > st.m + kSlack)) {
      apart();
      const float to = fmaxf(st.m, top);
      const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - to);
      st.m = to;
      st.l = (st.l + (sum[0] + sum[1])) * f;
      sum[0] = sum[1] = 0.0f;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 16; ++j) st.o[db][j] *= f;
      // the block before, whose weights are still to be used
      if (n > 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[(n - 1) & 1][j] *= f;
      }
    }
    m = st.m == -INFINITY ? 0.0f : st.m;
  };

  scores(0);
  settle(0);
#pragma unroll
  for (int n = 1; n < NB; ++n) {
    scores(n);
    settle(n);
    p[(n - 1) & 1].set(s[(n - 1) & 1]);
    outputs(n - 1, true);
  }
  if (NB == 1) {
#pragma unroll
    for (int j = 0; j < 16; ++j) exponential(0, j);
  }
  p[(NB - 1) & 1].set(s[(NB - 1) & 1]);
  outputs(NB - 1, false);
  st.l += sum[0] + sum[1];
}

template <class E, int DP, bool VEC>
__global__ __launch_bounds__(kNT, sizeof(typename E::storage) == 2 ? 2 : 1) void
attention_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  constexpr int KEYS = KeysOf<E>::kKeys;
  constexpr int kTile = KEYS * Sh::kRowBytes;
  extern __shared__ __attribute__((aligned(kTileAlign))) unsigned char smem[];   // [2][K, V] tiles
  __shared__ int bound[2][kWaves];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int tiles = (a.Tq + kQ - 1) / kQ;
  int head, tile;
  if (!place(a.B * a.Hq, tiles, &head, &tile)) return;
  tile = tiles - 1 - tile;
  const int b = head / a.Hq, hq = head % a.Hq, hk = hq / (a.Hq / a.Hkv);
  const int i = tile * kQ + wave * 32 + (lane & 31), p = a.Tk - a.Tq + i;
  const bool valid = i < a.Tq;
  Span keys = valid ? span_of(a, b, p) : Span{0, 0};
  if (a.causal && valid) keys.end = min(keys.end, p + 1);
  const bool some = keys.lo < keys.end;
  // what any query of the wave needs, and what all of them may see
  const int wlo = wave_min(some ? keys.lo : INT32_MAX), wend = wave_max(some ? keys.end : 0);
  const int full_lo = wave_max(some ? keys.lo : 0), full_end = wave_min(some ? keys.end : INT32_MAX);
  if (lane == 0) {
    bound[0][wave] = wlo;
    bound[1][wave] = wend;
  }
  __syncthreads();
  int lo = bound[0][0], end = bound[1][0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    lo = min(lo, bound[0][w]);
    end = max(end, bound[1][w]);
  }
  lo = uniform(lo);
  end = uniform(end);
  State<E, DP> st;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db) st.o[db] = f32x16{};
  st.m = -INFINITY;
  st.l = 0.0f;
  if (lo < end) {
    const int64_t kat = b * a.k.sb + hk * a.k.sh, vat = b * a.v.sb + hk * a.v.sh;
    uint32_t live[KEYS / 32], next[KEYS / 32];
    int k0 = lo / KEYS * KEYS;
    uint64_t m = live_keys<KEYS>(a, b, k0, live);
    const Loader<E, DP, KEYS, kWaves, VEC> load_k(a.k, a.D, wave, lane), load_v(a.v, a.D, wave, lane);
    load_k(smem, a.k, kat, k0, a.Tk, m);
    load_v(smem + kTile, a.v, vat, k0, a.Tk, m);
    Chunk<E> qf[Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.q.data + b * a.q.sb + hq * a.q.sh + (int64_t)i * a.q.st, some,
                               a.D, lane, qf);
    const float c = a.scale * kLog2e;
    const Places at = places<E, DP>(lane);
    int buf = 0;
    for (; k0 < end; k0 += KEYS, buf ^= 1) {
      unsigned char* here = smem + buf * 2 * kTile;
      unsigned char* there = smem + (buf ^ 1) * 2 * kTile;
      if constexpr (VEC) wait_loads();
      tile_barrier();        // this tile is there; the other one has been read
      if (k0 + KEYS < end) {
        m = live_keys<KEYS>(a, b, k0 + KEYS, next);
        load_k(there, a.k, kat, k0 + KEYS, a.Tk, m);
        load_v(there + kTile, a.v, vat, k0 + KEYS, a.Tk, m);
      }
      if (k0 < wend && k0 + KEYS > wlo) {
        const bool full = k0 >= full_lo && k0 + KEYS <= full_end && all_live<KEYS>(live);
        const uint32_t base = lds_addr(here);
        attend<E, DP, KEYS>(in_tile(at, base), in_tile(at, base + kTile), qf, st, c, k0, keys, full, live,
                            lane);
      }
#pragma unroll
      for (int n = 0; n < KEYS / 32; ++n) live[n] = next[n];
    }
  }
  if (!valid) return;
  const float l = st.l + lane_xor(st.l, 32);
  S* out = (S*)a.o.data + b * a.o.sb + hq * a.o.sh + (int64_t)i * a.o.st;
  store_row<E, DP, VEC>(out, st.o, some, 1.0f / l, a.D, lane);
  if (lane < 32)
    a.lse[((int64_t)b * a.Hq + hq) * a.Tq + i] = some ? kLn2 * (st.m + __log2f(l)) : 0.0f;
}

// ---------------------------------------------------------------------------
// Few queries over many keys
// ---------------------------------------------------------------------------
// Up to 32 (query, head of the group) pairs are one wave's rows, so the group's keys and values are read once; the tiles of
// keys are dealt to the waves of a.splits workgroups, each with tiles of LDS of
// its own (no barriers until the end).  A workgroup joins its waves through
// LDS; several workgroups' results are joined by a second kernel.
template <class E> struct FewOf;
template <> struct FewOf<BF16> { static constexpr int kWaves = 4; };
template <> struct FewOf<F32> { static constexpr int kWaves = 2; };
constexpr int kFewKeys = 32;

template <class E, int DP, bool VEC>
__global__ __launch_bounds__(64 * FewOf<E>::kWaves, 1) void attention_few_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  constexpr int NW = FewOf<E>::kWaves, KEYS = kFewKeys;
  constexpr int kTile = KEYS * Sh::kRowBytes;
  extern __shared__ __attribute__((aligned(kTileAlign))) unsigned char smem[];   // [wave][2][K, V], then joins
  __shared__ float ms[NW][32], ls[NW][32];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int split = blockIdx.x % a.splits, head = blockIdx.x / a.splits;
  const int hk = head % a.Hkv, b = head / a.Hkv;
  const int group = a.Hq / a.Hkv, rows = a.Tq * group;
  const int r = lane & 31;
  const bool valid = r < rows;
  const int i = valid ? r / group : 0, hq = hk * group + (valid ? r % group : 0), p = a.Tk - a.Tq + i;
  Span keys = valid ? span_of(a, b, p) : Span{0, 0};
  if (a.causal && valid) keys.end = min(keys.end, p + 1);
  const bool some = keys.lo < keys.end;
  const int lo = wave_min(some ? keys.lo : INT32_MAX), end = wave_max(some ? keys.end : 0);
  const int full_lo = wave_max(some ? keys.lo : 0), full_end = wave_min(some ? keys.end : INT32_MAX);
  State<E, DP> st;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db) st.o[db] = f32x16{};
  st.m = -INFINITY;
  st.l = 0.0f;
  unsigned char* mine = smem + wave * 4 * kTile;
  if (lo < end) {
    const int64_t kat = b * a.k.sb + hk * a.k.sh, vat = b * a.v.sb + hk * a.v.sh;
    const int step = a.splits * NW * KEYS;
    int k0 = lo / KEYS * KEYS + (split * NW + wave) * KEYS;
    uint32_t live[1] = {}, next[1] = {};
    const Loader<E, DP, KEYS, 1, VEC> load_k(a.k, a.D, 0, lane), load_v(a.v, a.D, 0, lane);
    const auto fetch = [&](int at, unsigned char* to) {
      const uint64_t m = live_keys<KEYS>(a, b, at, next);
      load_k(to, a.k, kat, at, a.Tk, m);
      load_v(to + kTile, a.v, vat, at, a.Tk, m);
    };
    if (k0 < end) fetch(k0, mine);
    live[0] = next[0];
    Chunk<E> qf[Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.q.data + b * a.q.sb + hq * a.q.sh + (int64_t)i * a.q.st, some,
                               a.D, lane, qf);
    const float c = a.scale * kLog2e;
    const Places at = places<E, DP>(lane);
    int buf = 0;
    for (; k0 < end; k0 += step, buf ^= 1) {
      unsigned char* here = mine + buf * 2 * kTile;
      wait_loads();
      wait_lds();
      __builtin_amdgcn_wave_barrier();
      if (k0 + step < end) fetch(k0 + step, mine + (buf ^ 1) * 2 * kTile);
      const bool full = k0 >= full_lo && k0 + KEYS <= full_end && live[0] == ~0u;
      const uint32_t base = lds_addr(here);
      attend<E, DP, KEYS>(in_tile(at, base), in_tile(at, base + kTile), qf, st, c, k0, keys, full, live,
                          lane);
      live[0] = next[0];
    }
  }
  // join the waves: weights 2^(m_w - M)
  const float l = st.l + lane_xor(st.l, 32);
  __syncthreads();                        // every wave is done with its tiles
  float* own = (float*)smem + wave * 32 * DP;
  if (lane < 32) {
    ms[wave][lane] = st.m;
    ls[wave][lane] = l;
  }
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int j = 0; j < 16; ++j)
      own[(lane & 31) * DP + 32 * db + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3)] = st.o[db][j];
  __syncthreads();
  float* po = a.part + (int64_t)blockIdx.x * rows * (DP + 2);     // [row][DP + 2]: O, M, L
  for (int e = threadIdx.x; e < rows * DP; e += 64 * NW) {
    const int row = e / DP, d = e % DP;
    float M = ms[0][row];
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, ms[w][row]);
    float o = 0.0f, L = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ms[w][row] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ms[w][row] - M);
      // a wave without keys of this row holds zeros
      o += f * ((float*)smem)[(w * 32 + row) * DP + d];
      L += f * ls[w][row];
    }
    if (a.splits > 1) {
      po[row * (DP + 2) + d] = o;
      if (d == 0) {
        po[row * (DP + 2) + DP] = M;
        po[row * (DP + 2) + DP + 1] = L;
      }
      continue;
    }
    const int qi = row / group, qh = hk * group + row % group;
    const Span sp = span_of(a, b, a.Tk - a.Tq + qi);
    const bool any = sp.lo < sp.end;
    if (d < a.D) {
      const float y[1] = {any ? o / L : 0.0f};
      store_f32<E, 1>((S*)a.o.data + b * a.o.sb + qh * a.o.sh + (int64_t)qi * a.o.st + d, y);
    }
    if (d == 0) a.lse[((int64_t)b * a.Hq + qh) * a.Tq + qi] = any ? kLn2 * (M + __log2f(L)) : 0.0f;
  }
}

// One wave joins the parts of one row.
template <class E, int DP>
__global__ __launch_bounds__(64) void attention_join_kernel(AttnArgs a) {
  typedef typename E::storage S;
  const int lane = threadIdx.x, group = a.Hq / a.Hkv, rows = a.Tq * group;
  const int rr = blockIdx.x % rows, head = blockIdx.x / rows, hk = head % a.Hkv, b = head / a.Hkv;
  const int qi = rr / group, qh = hk * group + rr % group;
  const float* po = a.part + ((int64_t)head * a.splits * rows + rr) * (DP + 2);
  const int64_t step = (int64_t)rows * (DP + 2);
  float M = -INFINITY;
  for (int s = 0; s < a.splits; ++s) M = fmaxf(M, po[s * step + DP]);
  float o[DP / 64] = {}, L = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float m = po[s * step + DP];
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
    L += f * po[s * step + DP + 1];
#pragma unroll
    for (int k = 0; k < DP / 64; ++k) o[k] += f * po[s * step + 64 * k + lane];
  }
  const Span sp = span_of(a, b, a.Tk - a.Tq + qi);
  const bool any = sp.lo < sp.end;
#pragma unroll
  for (int k = 0; k < DP / 64; ++k)
    if (64 * k + lane < a.D) {
      const float y[1] = {any ? o[k] / L : 0.0f};
      store_f32<E, 1>((S*)a.o.data + b * a.o.sb + qh * a.o.sh + (int64_t)qi * a.o.st + 64 * k + lane, y);
    }
  if (lane == 0) a.lse[((int64_t)b * a.Hq + qh) * a.Tq + qi] = any ? kLn2 * (M + __log2f(L)) : 0.0f;
}

// ---------------------------------------------------------------------------
template <class E, int DP, bool VEC>
hipError_t forward(const AttnArgs& a, hipStream_t s) {
  typedef Shape<E, DP> Sh;
  if (a.splits > 0) {
    constexpr int NW = FewOf<E>::kWaves;
    constexpr int lds = std::max(NW * 4 * kFewKeys * Sh::kRowBytes, NW * 32 * DP * 4);
    static hipError_t once = hipFuncSetAttribute((const void*)attention_few_kernel<E, DP, VEC>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (once != hipSuccess) return once;
    const unsigned heads = (unsigned)(a.B * a.Hkv), rows = (unsigned)(a.Tq * (a.Hq / a.Hkv));
    hipLaunchKernelGGL((attention_few_kernel<E, DP, VEC>), dim3(heads * a.splits), dim3(64 * NW), lds, s, a);
    if (a.splits > 1)
      hipLaunchKernelGGL((attention_join_kernel<E, DP>), dim3(heads * rows), dim3(64), 0, s, a);
    return hipGetLastError();
  }
  constexpr int lds = 4 * KeysOf<E>::kKeys * Sh::kRowBytes;
  static hipError_t once = hipFuncSetAttribute((const void*)attention_kernel<E, DP, VEC>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (once != hipSuccess) return once;
  const int64_t tiles = (a.Tq + kQ - 1) / kQ, heads = (int64_t)a.B * a.Hq;
  hipLaunchKernelGGL((attention_kernel<E, DP, VEC>), dim3((unsigned)((heads + 7) / 8 * 8 * tiles)),
                     dim3(kNT), lds, s, a);
  return hipGetLastError();
}

template <class E>
hipError_t forward_e(const AttnArgs& a, hipStream_t s) {
  if (a.D <= 64) return a.vec ? forward<E, 64, true>(a, s) : forward<E, 64, false>(a, s);
  return a.vec ? forward<E, 128, true>(a, s) : forward<E, 128, false>(a, s);
}

}  // namespace
}  // namespace attn

size_t attention_part_floats(AttnArgs& a) {
  const int64_t rows = (int64_t)a.Tq * (a.Hq / a.Hkv);
  a.splits = 0;
  if (rows > 32) return 0;
  const int64_t heads = (int64_t)a.B * a.Hkv;
  const int waves = a.dtype == kBF16 ? attn::FewOf<BF16>::kWaves : attn::FewOf<F32>::kWaves;
  const int64_t most = (a.Tk + waves * attn::kFewKeys * 2 - 1) / (waves * attn::kFewKeys * 2);
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>({most, (512 + heads - 1) / heads, 64}));
  return a.splits == 1 ? 0 : (size_t)(heads * a.splits * rows) * ((a.D <= 64 ? 64 : 128) + 2);
}

hipError_t launch_attn_ranges(const AttnArgs& a, hipStream_t s) {
  timing_begin("attention_ranges", s);
  hipLaunchKernelGGL(attn::attn_ranges_kernel, dim3((unsigned)((a.Tk + 255) / 256 * a.B)), dim3(256), 0, s, a);
  timing_end("attention_ranges", s);
  return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t s) {
  timing_begin("attention", s);
  const hipError_t e = a.dtype == kBF16 ? attn::forward_e<BF16>(a, s) : attn::forward_e<F32>(a, s);
  timing_end("attention", s);
  return e;
}

}  // namespace dpf
