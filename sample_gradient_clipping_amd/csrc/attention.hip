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
//
// 8x2048, 40x128 bf16: 410 us, 840 TFLOP/s.  A tile of 32 x 32 x 128 takes 16 matrix
// instructions (512 cycles) and about 126 vector ones (500 cycles, 256 of them the
// exponentials), 71 scalar and 24 LDS ones; of a compute unit's busy time the matrix
// units work 46%, the vector units 58%.  Tiles of 32 keys are what leaves registers for
// three waves per SIMD (64 keys, two waves: 444 us).
#include "attn.hpp"

#include <algorithm>

namespace dpf {
namespace attn {
namespace {

// The running maximum follows the scores only where they rise above it by more
// than this (in powers of two): the weights then stay below 2^8, and a tile that
// raises no maximum rescales nothing.
constexpr float kSlack = 8.0f;

// ---------------------------------------------------------------------------
// Mask and segments
// ---------------------------------------------------------------------------
// Each wave takes 64 positions of a sample.  lo: the first active position of
// the segment, end: one past its last active one (0, 0 for an inactive
// position), so a causal row with one key has lo == p and any other with one
// key end == lo + 1.  Segment numbers do not decrease, so the start of the
// first position's segment and the end of the last one's are found by 64-way
// search, the boundaries between by a vote.  A chain of latencies: 3 to 5 us without a
// mask or where padding is short.  The first active position before the wave's own is
// looked for 64 mask bytes at a time from the segment's start (not causal: the last one
// from its end), one round trip each: left-padded samples of 8192 positions take 20 us
// with 4096 of them padded, 34 with 7680, 65536 with half of them padded 175, and 2^20
// so 2.5 ms, beside 43, 10, 370 and 370 us of a single token's attention.
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
// A wave's 32 queries against tiles of 32 keys
// ---------------------------------------------------------------------------
constexpr int kKeys = 32;

template <class E, int DP>
struct State {
  f32x16 o[DP / 32];    // O^T: this lane's query, relative to m
  float m, l;           // maximum used (times log2 e) and this lane half's sum
};

// What of a tile a lane's query sees: keys [lo, end) with their bit of `live`.
struct Sight {
  int lo, end;
  uint32_t live;
  bool full;            // every query of the wave sees every key of the tile
};

// The scores of a tile, masked; returns their maximum, unscaled.  Every LDS operand
// is read kAhead products early, and fences keep that order: left to itself the
// compiler waits for each read.
template <class E, int DP>
__device__ __forceinline__ float scores(const Places& kt, const Chunk<E> (&qf)[Shape<E, DP>::kG], f32x16& s,
                                        int k0, const Sight& see, int lane) {
  constexpr int G = Shape<E, DP>::kG;
  Chunk<E> k[kAhead];
#pragma unroll
  for (int g = 0; g < kAhead; ++g) k[g] = row_frag<E, DP>(kt, 0, g);
  fence();
  s = f32x16{};
#pragma unroll
  for (int g = 0; g < G; ++g) {
    s = mma<E>(k[g % kAhead], qf[g], s);
    if (g + kAhead < G) k[g % kAhead] = row_frag<E, DP>(kt, 0, g + kAhead);
    fence();
  }
  if (!see.full) {
    apart();
    const int h = lane >> 5;
    const uint32_t w = see.live >> (4 * h);
    const int first = see.lo - k0 - 4 * h, past = see.end - k0 - 4 * h;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int r = 8 * (j >> 2) + (j & 3);
      const bool in = r >= first && r < past && ((w >> r) & 1);
      s[j] = in ? s[j] : -INFINITY;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 16; ++j) top = fmaxf(top, s[j]);
  return top;
}

// Adds a tile's weighted values, its scores in s.
template <class E, int DP>
__device__ __forceinline__ void values(const Places& vt, State<E, DP>& st, f32x16& s, float c, int lane) {
  constexpr int DB = DP / 32, N = DB * ColumnSteps<E>::kN;
  const float m = st.m == -INFINITY ? 0.0f : st.m;
  const auto read = [&](int t) { return column_frag<E, DP>(vt, 0, t % DB, t / DB, lane); };
  Column<E> v[kAhead];
#pragma unroll
  for (int t = 0; t < kAhead; ++t) v[t] = read(t);
  fence();
  float sum[2] = {};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float x = __builtin_amdgcn_exp2f(fmaf(s[j], c, -m));
    asm volatile("" : "+v"(x));    // here, not where it is used first
    s[j] = x;
    sum[j & 1] += x;
  }
  Weights<E> p;
  p.set(s);
  st.l += sum[0] + sum[1];
  fence();
#pragma unroll
  for (int t = 0; t < N; ++t) {
    st.o[t % DB] = mma_column<E>(v[t % kAhead], p, t / DB, st.o[t % DB]);
    if (t + kAhead < N) v[t % kAhead] = read(t + kAhead);
    fence();
  }
}

// Moves the running maximum to the scores of maximum `top`.
template <class E, int DP>
__device__ __forceinline__ void settle(State<E, DP>& st, float top, float c) {
  top = fmaxf(top, lane_xor(top, 32)) * c;
  if (__any(top > st.m + kSlack)) {
    apart();
    const float to = fmaxf(st.m, top);
    const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - to);
    st.m = to;
    st.l *= f;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int j = 0; j < 16; ++j) st.o[db][j] *= f;
  }
}

// The mask of a sample of up to kRowMask positions, in scalar registers: its call
// needs no launch for ranges (32x128, 16x64: 18.5 us with one, 13.3 without).
struct RowMask {
  static_assert(kRowMask == 256, "four words");
  uint64_t m0, m1, m2, m3;
  __device__ __forceinline__ void read(const AttnArgs& a, int b, int lane) {
    const uint8_t* row = a.mask + (int64_t)b * a.Tk;
    const auto part = [&](int k) { return __ballot(row[min(k, a.Tk - 1)] != 0 && k < a.Tk); };
    m0 = part(lane);
    m1 = part(64 + lane);
    m2 = part(128 + lane);
    m3 = part(192 + lane);
  }
  __device__ __forceinline__ Span span() const {      // from the first active position to the last
    const auto first = [](uint64_t m) { return __ffsll((unsigned long long)m) - 1; };
    const auto past = [](uint64_t m) { return 64 - __clzll((long long)m); };
    return {m0 ? first(m0) : m1 ? 64 + first(m1) : m2 ? 128 + first(m2) : 192 + first(m3),
            m3 ? 192 + past(m3) : m2 ? 128 + past(m2) : m1 ? 64 + past(m1) : past(m0)};
  }
  __device__ __forceinline__ uint32_t word(int k0) const {      // of positions k0 .. k0 + 31
    const uint64_t low = k0 < 64 ? m0 : m1, high = k0 < 192 ? m2 : m3;
    return (uint32_t)((k0 < 128 ? low : high) >> (k0 & 32));
  }
};

// NW waves, 32 queries each, share the tiles.
template <class E, int DP, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, sizeof(typename E::storage) == 4 ? 1 : !VEC ? 2 : DP == 64 ? 4 : 3) void
attention_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  constexpr int kQ = 32 * NW;             // queries of a workgroup
  constexpr int kTile = kKeys * Sh::kRowBytes;
  extern __shared__ __attribute__((aligned(kTileAlign))) unsigned char smem[];   // K [2], V [2] tiles
  __shared__ int bound[2][NW];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int tiles = (a.Tq + kQ - 1) / kQ;
  int head, tile;
  place(a.B * a.Hq, tiles, max(heads_at_once<E>(a), a.Hq / a.Hkv), &head, &tile);
  tile = tiles - 1 - tile;
  const int b = head / a.Hq, hq = head % a.Hq, hk = hq / (a.Hq / a.Hkv);
  const int i = tile * kQ + wave * 32 + (lane & 31), p = a.Tk - a.Tq + i;
  const bool valid = i < a.Tq;
  const bool row_mask = a.mask != nullptr && a.lo == nullptr;
  RowMask row;
  Span keys = {0, 0};
  if (row_mask) {
    row.read(a, b, lane);
    if (valid && a.mask[(int64_t)b * a.Tk + p] != 0) keys = row.span();
  } else if (valid) {
    keys = span_of(a, b, p);
  }
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
  for (int w = 1; w < NW; ++w) {
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
    Loader<E, DP, kKeys, NW, VEC> load_k(a.k, a.Tk, a.D, wave, lane), load_v(a.v, a.Tk, a.D, wave, lane);
    const float c = a.scale * kLog2e;
    const Places pl = places<E, DP>(lane);
    const uint32_t kt = lds_addr(smem), vt = kt + 2 * kTile;
    const int first = lo / kKeys, tiles = (end + kKeys - 1) / kKeys - first;
    const auto place_of = [&](int t) { return (first + t) * kKeys; };
    Sight see{keys.lo, keys.end, 0, false};
    const auto look = [&](int t) {
      uint32_t live[1];
      uint64_t m;
      if (row_mask) m = live[0] = row.word(place_of(t));
      else m = live_keys<kKeys>(a, b, place_of(t), live);
      see.live = live[0];
      see.full = place_of(t) >= full_lo && place_of(t) + kKeys <= full_end && live[0] == ~0u;
      return m;
    };
    load_k.start(a.k, kat, place_of(0));
    load_v.start(a.v, vat, place_of(0));
    const auto fetch = [&](int t) {
      if (t >= tiles) return;
      const uint64_t m = look(t);
      // keys' rows of masked positions need no zeros: their scores are selected away
      load_k(kt + (t & 1) * kTile, place_of(t), ~0ull);
      load_v(vt + (t & 1) * kTile, place_of(t), m);
    };
    fetch(0);
    Chunk<E> qf[Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.q.data, b * a.q.sb + hq * a.q.sh + (int64_t)i * a.q.st, some,
                               a.D, lane, qf);
    f32x16 s;
    for (int t = 0; t < tiles; ++t) {
      const Sight now = see;
      wait_loads();
      tile_barrier();        // this tile is there; the other one has been read
      fetch(t + 1);
      if (place_of(t) < wend && place_of(t) + kKeys > wlo) {
        const Places kn = in_tile(pl, kt + (t & 1) * kTile), vn = in_tile(pl, vt + (t & 1) * kTile);
        settle<E, DP>(st, scores<E, DP>(kn, qf, s, place_of(t), now, lane), c);
        values<E, DP>(vn, st, s, c, lane);
      }
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
// Up to 32 (query, head of the group) pairs are one wave's rows, so the group's
// keys and values are read once; the tiles of keys are dealt to the waves of
// a.splits workgroups, each with tiles of LDS of its own (no barriers until the
// end).  A workgroup joins its waves through LDS; several workgroups' results are
// joined by a second kernel.  HBM bounds it: what counts is that all compute units
// start at once and end together, so there are as many workgroups as compute
// units, not more (16x1 over 4096, 40/8x128: 58 us in one round of 256, 65 in two;
// 1x1 over 65536, 32/8x128: 64 and 86); half of them still draw most of what HBM
// gives.  Where the heads alone are more, workgroups of two waves, two to a compute
// unit (100x8 heads over 1000: 80 us, 90 with four waves).  Float32 tiles leave room
// for two waves.
constexpr int kUnits = 256;
int few_waves(const AttnArgs& a) {
  return a.dtype == kBF16 && (int64_t)a.B * a.Hkv <= kUnits ? 4 : 2;
}

template <class E, int DP, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, 1) void attention_few_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  constexpr int KEYS = kKeys;
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
    const int stride = a.splits * NW * KEYS;
    int k0 = lo / KEYS * KEYS + (split * NW + wave) * KEYS;
    uint32_t live[1] = {}, next[1] = {};
    Loader<E, DP, KEYS, 1, VEC> load_k(a.k, a.Tk, a.D, 0, lane), load_v(a.v, a.Tk, a.D, 0, lane);
    load_k.start(a.k, kat, k0);
    load_v.start(a.v, vat, k0);
    const auto fetch = [&](int at, uint32_t to) {
      const uint64_t m = live_keys<KEYS>(a, b, at, next);
      load_k(to, at, m);
      load_v(to + kTile, at, m);
    };
    const uint32_t own_tiles = lds_addr(mine);
    if (k0 < end) fetch(k0, own_tiles);
    live[0] = next[0];
    Chunk<E> qf[Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.q.data, b * a.q.sb + hq * a.q.sh + (int64_t)i * a.q.st, some,
                               a.D, lane, qf);
    const float c = a.scale * kLog2e;
    const Places at = places<E, DP>(lane);
    int buf = 0;
    for (; k0 < end; k0 += stride, buf ^= 1) {
      wait_loads();
      wait_lds();
      __builtin_amdgcn_wave_barrier();
      if (k0 + stride < end) fetch(k0 + stride, own_tiles + (buf ^ 1) * 2 * kTile);
      const Sight see{keys.lo, keys.end, live[0],
                      k0 >= full_lo && k0 + KEYS <= full_end && live[0] == ~0u};
      const uint32_t base = own_tiles + buf * 2 * kTile;
      const Places kt = in_tile(at, base), vt = in_tile(at, base + kTile);
      f32x16 s;
      settle<E, DP>(st, scores<E, DP>(kt, qf, s, k0, see, lane), c);
      values<E, DP>(vt, st, s, c, lane);
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
  // lane s has split s's maximum and sum (at most 64 of them)
  const bool in = lane < a.splits;
  const float m = in ? po[lane * step + DP] : -INFINITY, l = in ? po[lane * step + DP + 1] : 0.0f;
  float M = m;
#pragma unroll
  for (int j = 1; j < 64; j <<= 1) M = fmaxf(M, lane_xor(M, j));
  const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
  float o[DP / 64] = {}, L = f * l;
#pragma unroll
  for (int j = 1; j < 64; j <<= 1) L += lane_xor(L, j);
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) {
    const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), s));
#pragma unroll
    for (int k = 0; k < DP / 64; ++k) o[k] += w * po[s * step + 64 * k + lane];
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
template <class E, int DP, int NW, bool VEC>
hipError_t tiled(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = 4 * kKeys * Shape<E, DP>::kRowBytes;
  static hipError_t once = hipFuncSetAttribute((const void*)attention_kernel<E, DP, NW, VEC>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (once != hipSuccess) return once;
  const int64_t tiles = (a.Tq + 32 * NW - 1) / (32 * NW);
  hipLaunchKernelGGL((attention_kernel<E, DP, NW, VEC>), dim3((unsigned)(a.B * a.Hq * tiles)), dim3(64 * NW),
                     lds, s, a);
  return hipGetLastError();
}

template <class E, int DP, int NW, bool VEC>
hipError_t few(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = std::max(NW * 4 * kKeys * Shape<E, DP>::kRowBytes, NW * 32 * DP * 4);
  static hipError_t once = hipFuncSetAttribute((const void*)attention_few_kernel<E, DP, NW, VEC>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (once != hipSuccess) return once;
  const unsigned heads = (unsigned)(a.B * a.Hkv), rows = (unsigned)(a.Tq * (a.Hq / a.Hkv));
  hipLaunchKernelGGL((attention_few_kernel<E, DP, NW, VEC>), dim3(heads * a.splits), dim3(64 * NW), lds, s, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((attention_join_kernel<E, DP>), dim3(heads * rows), dim3(64), 0, s, a);
  return hipGetLastError();
}

template <class E, int DP, bool VEC>
hipError_t forward(const AttnArgs& a, hipStream_t s) {
  if (a.splits == 0) return tiled<E, DP, 4, VEC>(a, s);
  if constexpr (sizeof(typename E::storage) == 2)
    if (few_waves(a) == 4) return few<E, DP, 4, VEC>(a, s);
  return few<E, DP, 2, VEC>(a, s);
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
  const int keys = attn::few_waves(a) * attn::kKeys * 2;
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>({(a.Tk + keys - 1) / keys, attn::kUnits / heads, 64}));
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
