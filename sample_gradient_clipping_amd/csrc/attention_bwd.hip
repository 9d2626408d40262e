// Attention over the positions of each sample, backward.
//
//   P_ij = e^{s_ij - lse_i},  delta_i = dO_i . O_i
//   dS_ij = P_ij (dO_i . v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i
//
// Two kernels, each a pass with sums of its own in registers, so that nothing is
// added to memory in an order that changes: one over the keys for dq (which
// takes delta too), one over the queries of all heads of a group for dk and dv.
// Both form S and dO V^T again: seven products for the five of the formula, in
// exchange for no atomics and no array of queries by keys.  P and dS lie in the
// accumulators as the right operands of the products that sum over their rows;
// they are rounded to bf16 there (what the operand type holds), all sums are
// float32.
//
// A query that sees one key only has P = 1 and dS = 0 exactly; its delta comes
// from the rounded output and would leave a difference that is all rounding, so
// such a pair's dS is set to 0.
//
// 8x2048, 40x128 bf16: dq 590 us, dk and dv 850 (870 and 810 TFLOP/s of the products
// run); 32x512, 12x64: 57 and 68.  Matrix instructions and the exponentials' vector
// work bound both, at two waves per SIMD (the sums take 64 and 128 registers).
#include "attn.hpp"

namespace dpf {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kNT = 64 * kWaves;
constexpr int kRows = 32 * kWaves;      // queries (keys) of a workgroup

// ---------------------------------------------------------------------------
// dq and delta: as the forward pass, each wave 32 queries (its lanes), tiles of
// keys and values through LDS.  SHARE, where the workgroups would be few: the four
// waves of a workgroup have the same 32 queries, each with tiles of its own every
// fourth step of 32 keys, and the first adds their sums in order.
// ---------------------------------------------------------------------------
template <class E, int DP, bool SHARE>
struct Dq {
  static constexpr int kQueries = SHARE ? 32 : kRows;
  static constexpr int kN = sizeof(typename E::storage) == 2 && !SHARE ? 64 : 32;     // keys of a tile
  static constexpr int kTile = kN * Shape<E, DP>::kRowBytes;
  // pairs of tiles of a set, sets of a workgroup
  static constexpr int kPairs = SHARE && kTile * 16 > 150 * 1024 ? 1 : 2;
  static constexpr int kSets = SHARE ? kWaves : 1;
  static constexpr int kLds = kSets * kPairs * 2 * kTile;
  static_assert(!SHARE || kLds >= (kWaves - 1) * DP * 32 * 4, "room for the waves' sums");
  static_assert(kLds <= 156 * 1024, "LDS");
};

template <class E, int DP, bool VEC, bool SHARE>
__global__ __launch_bounds__(kNT, sizeof(typename E::storage) == 2 && VEC && !SHARE ? 2 : 1) void
attention_dq_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  typedef Dq<E, DP, SHARE> Z;
  constexpr int KEYS = Z::kN, kTile = Z::kTile;
  extern __shared__ __attribute__((aligned(kTileAlign))) unsigned char smem[];   // [sets][pairs][K, V] tiles
  __shared__ int bound[2][kWaves];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5;
  const int tiles = (a.Tq + Z::kQueries - 1) / Z::kQueries;
  int head, tile;
  place(a.B * a.Hq, tiles, max(heads_at_once<E>(a), a.Hq / a.Hkv), &head, &tile);
  tile = tiles - 1 - tile;
  const int b = head / a.Hq, hq = head % a.Hq, hk = hq / (a.Hq / a.Hkv);
  const int i = tile * Z::kQueries + (SHARE ? 0 : wave * 32) + (lane & 31), p = a.Tk - a.Tq + i;
  const bool valid = i < a.Tq;
  Span keys = valid ? span_of(a, b, p) : Span{0, 0};
  if (a.causal && valid) keys.end = min(keys.end, p + 1);
  const bool some = keys.lo < keys.end, lone = keys.end - keys.lo == 1;
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
  f32x16 dq[Sh::kDB];
#pragma unroll
  for (int db = 0; db < Sh::kDB; ++db) dq[db] = f32x16{};
  const int64_t at = ((int64_t)b * a.Hq + hq) * a.Tq + i;
  if (lo < end) {
    const int64_t kat = b * a.k.sb + hk * a.k.sh, vat = b * a.v.sb + hk * a.v.sh;
    uint32_t live[KEYS / 32], next[KEYS / 32];
    constexpr int kStride = KEYS * Z::kSets, kLoaders = SHARE ? 1 : kWaves;
    int k0 = lo / KEYS * KEYS + (SHARE ? wave * KEYS : 0);
    uint64_t m = 0;
    Loader<E, DP, KEYS, kLoaders, VEC> load_k(a.k, a.Tk, a.D, SHARE ? 0 : wave, lane),
        load_v(a.v, a.Tk, a.D, SHARE ? 0 : wave, lane);
    load_k.start(a.k, kat, k0);
    load_v.start(a.v, vat, k0);
    const uint32_t tiles_at = lds_addr(smem) + (SHARE ? wave * Z::kPairs * 2 * kTile : 0);
    const auto fetch = [&](int at, uint32_t to, uint32_t (&bits)[KEYS / 32]) {
      m = live_keys<KEYS>(a, b, at, bits);
      load_k(to, at, m);
      load_v(to + kTile, at, m);
    };
    if (!SHARE || k0 < end) fetch(k0, tiles_at, live);
    Chunk<E> qf[Sh::kG], gf[Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.o.data, b * a.o.sb + hq * a.o.sh + (int64_t)i * a.o.st, some,
                               a.D, lane, qf);
    row_frags_from<E, DP, VEC>((const S*)a.dout.data, b * a.dout.sb + hq * a.dout.sh +
                               (int64_t)i * a.dout.st, some, a.D, lane, gf);
    float delta = 0.0f;
#pragma unroll
    for (int g = 0; g < Sh::kG; ++g)
#pragma unroll
      for (int k = 0; k < 16 / Sh::kES; ++k)
        delta = fmaf(E::to_float(qf[g][k]), E::to_float(gf[g][k]), delta);
    delta += lane_xor(delta, 32);
    row_frags_from<E, DP, VEC>((const S*)a.q.data, b * a.q.sb + hq * a.q.sh + (int64_t)i * a.q.st, some,
                               a.D, lane, qf);
    const float base = some ? -a.lse[at] / a.scale : 0.0f;
    if (valid && h == 0 && (!SHARE || wave == 0)) a.delta[at] = delta;
    const float c = a.scale * kLog2e;
    const Places pl = places<E, DP>(lane);
    int buf = 0;
    bool full = false;
    // S starts from -lse / scale and dO V^T from -delta: P = 2^(c S), dS = P dP
    const auto start = [&](f32x16& s, f32x16& dp) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        s[j] = base;
        dp[j] = -delta;
      }
    };
    const auto mask = [&](int n, f32x16& s) {
      if (full) return;
      apart();
      const uint32_t w0 = live[0], w1 = live[KEYS / 32 - 1], w = lone ? 0u : (n == 0 ? w0 : w1) >> (4 * h);
      const int first = keys.lo - k0 - 32 * n - 4 * h, past = keys.end - k0 - 32 * n - 4 * h;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int r = 8 * (j >> 2) + (j & 3);
        const bool in = r >= first && r < past && ((w >> r) & 1);
        s[j] = in ? s[j] : -INFINITY;
      }
    };
    // a row's sum_j P_ij (dO_i . v_j - delta_i) over the keys of a tile
    const auto rest = [&](uint32_t here) {
      float sum = 0.0f;
#pragma unroll 1
      for (int n = 0; n < KEYS / 32; ++n) {
        const Places kt = in_tile(pl, here + n * 32 * Sh::kRowBytes);
        const Places vt = in_tile(pl, here + kTile + n * 32 * Sh::kRowBytes);
        f32x16 s, dp;
        start(s, dp);
#pragma unroll
        for (int g = 0; g < Sh::kG; ++g) {
          s = mma<E>(row_frag<E, DP>(kt, 0, g), qf[g], s);
          dp = mma<E>(row_frag<E, DP>(vt, 0, g), gf[g], dp);
          fence();
        }
        mask(n, s);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum = fmaf(__builtin_amdgcn_exp2f(s[j] * c), dp[j], sum);
      }
      return sum + lane_xor(sum, 32);
    };
    const auto all_seen = [&] { return k0 >= full_lo && k0 + KEYS <= full_end && all_live<KEYS>(live); };
    // Where the keys are few, delta is sum_j P_ij dO_i . v_j: from the rounded output
    // it is off by 2^-9 of |dO| |O|, which shows there.
    // A wave's keys in one tile, or (SHARE) a tile or none for each wave:
    const bool once = sizeof(S) == 2 && (SHARE ? (end - 1) / KEYS - lo / KEYS < kWaves
                                               : wlo / KEYS == (wend - 1) / KEYS);
    if constexpr (SHARE && sizeof(S) == 2) {
      if (once) {
        __shared__ float sums[kWaves][32];
        float sum = 0.0f;
        if (k0 < end) {
          if constexpr (VEC) wait_loads();
          wait_lds();
          asm volatile("" ::: "memory");
          full = all_seen();
          sum = rest(tiles_at);
        }
        if (h == 0) sums[wave][lane] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) delta += sums[w][lane & 31];
        if (some && h == 0 && wave == 0) a.delta[at] = delta;
      }
    }
    for (; k0 < end; k0 += kStride, buf ^= Z::kPairs - 1) {
      const uint32_t here = tiles_at + buf * 2 * kTile, there = tiles_at + (buf ^ 1) * 2 * kTile;
      if constexpr (VEC) wait_loads();
      // this tile is there; the other one has been read
      if constexpr (SHARE) {
        wait_lds();
        asm volatile("" ::: "memory");
      } else {
        tile_barrier();
      }
      if (Z::kPairs == 2 && k0 + kStride < end) fetch(k0 + kStride, there, next);
      if (k0 < wend && k0 + KEYS > wlo) {
        full = all_seen();
        if constexpr (sizeof(S) == 2) {
          if (!SHARE && once) {
            delta += rest(here);                  // dP started from -delta
            if (some && h == 0) a.delta[((int64_t)b * a.Hq + hq) * a.Tq + i] = delta;
          }
          // per block of 32 keys G products for S, G for dP with the exponentials
          // between them, 2 DB for dq; operands read kAhead products early
          constexpr int G = Sh::kG, DB = Sh::kDB, T = 2 * G + 2 * DB;
#pragma unroll 1
          for (int n = 0; n < KEYS / 32; ++n) {
            const Places kt = in_tile(pl, here + n * 32 * Sh::kRowBytes);
            const Places vt = in_tile(pl, here + kTile + n * 32 * Sh::kRowBytes);
            const auto operand = [&](int t) -> u16x8 {
              if (t < G) return row_frag<E, DP>(kt, 0, t);
              if (t < 2 * G) return row_frag<E, DP>(vt, 0, t - G);
              return column_frag<E, DP>(kt, 0, (t - 2 * G) % DB, (t - 2 * G) / DB, lane);
            };
            u16x8 x[kAhead];
            f32x16 s, dp;
            Weights<E> w;
            start(s, dp);
#pragma unroll
            for (int t = 0; t < kAhead; ++t) x[t] = operand(t);
            fence();
#pragma unroll
            for (int t = 0; t < T; ++t) {
              const u16x8 y = x[t % kAhead];
              if (t < G) s = mma<E>(y, qf[t], s);
              else if (t < 2 * G) dp = mma<E>(y, gf[t - G], dp);
              else dq[(t - 2 * G) % DB] = mma_column<E>(y, w, (t - 2 * G) / DB, dq[(t - 2 * G) % DB]);
              if (t + kAhead < T) x[t % kAhead] = operand(t + kAhead);
              if (t >= G && t < 2 * G) {
#pragma unroll
                for (int j = 16 * (t - G) / G; j < 16 * (t - G + 1) / G; ++j) {
                  float e = __builtin_amdgcn_exp2f(s[j] * c);
                  asm volatile("" : "+v"(e));
                  s[j] = e;
                }
              }
              fence();
              if (t == G - 1) mask(n, s);
              if (t == 2 * G - 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j) dp[j] *= s[j];
                w.set(dp);
              }
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < KEYS / 32; ++n) {
            const Places kt = in_tile(pl, here + n * 32 * Sh::kRowBytes);
            const Places vt = in_tile(pl, here + kTile + n * 32 * Sh::kRowBytes);
            f32x16 s, dp;
            start(s, dp);
#pragma unroll
            for (int g = 0; g < Sh::kG; ++g) s = mma<E>(row_frag<E, DP>(kt, 0, g), qf[g], s);
#pragma unroll
            for (int g = 0; g < Sh::kG; ++g) dp = mma<E>(row_frag<E, DP>(vt, 0, g), gf[g], dp);
            mask(n, s);
#pragma unroll
            for (int j = 0; j < 16; ++j) dp[j] *= __builtin_amdgcn_exp2f(s[j] * c);
            Weights<E> w;
            w.set(dp);
#pragma unroll
            for (int db = 0; db < Sh::kDB; ++db)
              dq[db] = mma_columns<E, DP>(kt, 0, db, w, dq[db], lane);
          }
        }
      }
      if (Z::kPairs == 1 && k0 + kStride < end) {      // one pair of tiles: the next after this has been read
        wait_lds();
        asm volatile("" ::: "memory");
        fetch(k0 + kStride, tiles_at, next);
      }
#pragma unroll
      for (int n = 0; n < KEYS / 32; ++n) live[n] = next[n];
    }
    if constexpr (SHARE) {     // the waves' sums, added in their order by the first
      float* const sums = (float*)smem;
      __syncthreads();
      if (wave > 0) {
#pragma unroll
        for (int db = 0; db < Sh::kDB; ++db)
#pragma unroll
          for (int j = 0; j < 16; ++j) sums[(((wave - 1) * Sh::kDB + db) * 16 + j) * 64 + lane] = dq[db][j];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
          for (int db = 0; db < Sh::kDB; ++db)
#pragma unroll
            for (int j = 0; j < 16; ++j) dq[db][j] += sums[((w * Sh::kDB + db) * 16 + j) * 64 + lane];
      }
    }
  } else if (valid && h == 0 && (!SHARE || wave == 0)) {
    a.delta[at] = 0.0f;
  }
  if (!valid || (SHARE && wave > 0)) return;
  store_row<E, DP, VEC>((S*)a.dq.data + b * a.dq.sb + hq * a.dq.sh + (int64_t)i * a.dq.st, dq,
                        some, a.scale, a.D, lane);
}

// ---------------------------------------------------------------------------
// dk and dv: each wave 32 keys (its lanes), whose rows of K it holds in registers,
// and of V in registers (heads of 64) or LDS (heads of 128, whose sums take 128
// registers: a wave with both in registers would have its SIMD alone, and nothing
// to overlap its exponentials with); tiles of queries and of their output
// gradients go through LDS, for each head of the group in turn.
//
// SHARE, where the workgroups would be few: the four waves of a workgroup have the
// same 32 keys, each with tiles of its own every fourth (head, queries) step, and
// the first adds their sums in order.
// ---------------------------------------------------------------------------
template <class E, int DP, bool SHARE>
struct Dkv {
  static constexpr int kKeys = SHARE ? 32 : kRows;                  // keys of a workgroup
  // queries of a tile
  static constexpr int kN = sizeof(typename E::storage) == 2 && DP == 64 && !SHARE ? 64 : 32;
  static constexpr int kTile = kN * Shape<E, DP>::kRowBytes;
  static constexpr bool kValuesInLds = DP == 128;
  static constexpr int kValues = kValuesInLds ? kKeys * Shape<E, DP>::kRowBytes : 0;
  // pairs of tiles of a set, sets of a workgroup
  static constexpr int kPairs = SHARE && kTile * 16 + kValues > 150 * 1024 ? 1 : 2;
  static constexpr int kSets = SHARE ? kWaves : 1;
  static constexpr int kLds = kValues + kSets * kPairs * 2 * kTile;
  // sums of all waves but one, where the tiles were
  static_assert(!SHARE || kLds - kValues >= (kWaves - 1) * DP * 64 * 4, "room for the waves' sums");
  static_assert(kLds <= 156 * 1024, "LDS");
};

template <class E, int DP, bool VEC, bool SHARE>
__global__ __launch_bounds__(kNT, sizeof(typename E::storage) == 2 && !SHARE ? 2 : 1) void
attention_dkv_kernel(AttnArgs a) {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  typedef Dkv<E, DP, SHARE> Z;
  constexpr int N = Z::kN, kTile = Z::kTile;
  extern __shared__ __attribute__((aligned(kTileAlign))) unsigned char shared_tiles[];   // V, [sets][pairs][Q, dO]
  __shared__ int bound[2][kWaves];
  __shared__ __attribute__((aligned(16))) float row_lse[Z::kSets][2][N],
      row_delta[Z::kSets][2][N];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5;
  const int set = SHARE ? wave : 0;
  const uint32_t smem = lds_addr(shared_tiles) + Z::kValues + set * Z::kPairs * 2 * kTile;
  const int tiles = (a.Tk + Z::kKeys - 1) / Z::kKeys, group = a.Hq / a.Hkv, off = a.Tk - a.Tq;
  int head, tile;
  place(a.B * a.Hkv, tiles, heads_at_once<E>(a), &head, &tile);
  const int b = head / a.Hkv, hk = head % a.Hkv;
  const int j0 = tile * Z::kKeys + (SHARE ? 0 : wave * 32) + (lane & 31);
  const bool valid = j0 < a.Tk;
  const Span sp = valid ? span_of(a, b, j0) : Span{0, 0};
  // positions whose queries see this key: [from, past), active
  int from = a.causal ? j0 : sp.lo;
  const int past = sp.end;
  const bool lone = a.causal ? sp.lo == j0 : sp.end - sp.lo == 1;   // position j0 sees only this key
  from = max(from, off);
  const bool some = from < past && sp.lo < sp.end;
  const int wlo = wave_min(some ? from : INT32_MAX), wend = wave_max(some ? past : 0);
  const int full_lo = wave_max(some ? from : 0), full_end = wave_min(some ? past : INT32_MAX);
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
  f32x16 dk[Sh::kDB], dv[Sh::kDB];
#pragma unroll
  for (int db = 0; db < Sh::kDB; ++db) dk[db] = dv[db] = f32x16{};
  if (lo < end) {
    const int p_first = lo / N * N, steps = (end - p_first + N - 1) / N;
    const float c = a.scale * kLog2e;
    const Places pl = places<E, DP>(lane);
    Chunk<E> kf[Sh::kG], vf[Z::kValuesInLds ? 1 : Sh::kG];
    row_frags_from<E, DP, VEC>((const S*)a.k.data, b * a.k.sb + hk * a.k.sh + (int64_t)j0 * a.k.st, some,
                               a.D, lane, kf);
    if constexpr (Z::kValuesInLds) {
      // what an inactive key's row holds reaches nothing but its own sums, which
      // are not used
      constexpr int kR = SHARE ? 32 : 64;
      Loader<E, DP, kR, kWaves, VEC> load_v(a.v, a.Tk, a.D, wave, lane);
      load_v.start(a.v, b * a.v.sb + hk * a.v.sh, tile * Z::kKeys);
#pragma unroll
      for (int r = 0; r < Z::kKeys; r += kR)
        load_v(lds_addr(shared_tiles) + r * Sh::kRowBytes, tile * Z::kKeys + r, ~0ull);
    } else {
      row_frags_from<E, DP, VEC>((const S*)a.v.data, b * a.v.sb + hk * a.v.sh + (int64_t)j0 * a.v.st,
                                 some, a.D, lane, vf);
    }
    const float inv_scale = -1.0f / a.scale;
    const Places values = in_tile(pl, lds_addr(shared_tiles) + (SHARE ? 0 : 32 * wave) * Sh::kRowBytes);
    const auto value_frag = [&](int g) {
      if constexpr (Z::kValuesInLds) return row_frag<E, DP>(values, 0, g);
      else return vf[g];
    };
    uint32_t live[N / 32], next[N / 32];
    // this thread's row of the next tile: its lse (kind 0) or delta (kind 1)
    float value = 0.0f;
    const int row = SHARE ? lane & 31 : threadIdx.x & 63, kind = SHARE ? h : wave;
    constexpr int kLoaders = SHARE ? 1 : kWaves;
    Loader<E, DP, N, kLoaders, VEC> load_q(a.q, a.Tq, a.D, SHARE ? 0 : wave, lane),
        load_g(a.dout, a.Tq, a.D, SHARE ? 0 : wave, lane);
    const auto fetch = [&](int p0, int hq, int buf) {
      uint64_t m = live_keys<N>(a, b, p0, next);
      if (p0 < off) m &= ~0ull << (off - p0);        // no queries at these positions
      if (SHARE || p0 == p_first) {                  // the next head
        load_q.start(a.q, b * a.q.sb + hq * a.q.sh, p0 - off);
        load_g.start(a.dout, b * a.dout.sb + hq * a.dout.sh, p0 - off);
      }
      const uint32_t to = smem + buf * 2 * kTile;
      load_q(to, p0 - off, m);
      load_g(to + kTile, p0 - off, m);
      const int i = p0 - off + row;
      value = 0.0f;
      if (kind < 2 && row < N && i >= 0 && i < a.Tq && ((m >> row) & 1)) {
        const int64_t e = ((int64_t)b * a.Hq + hq) * a.Tq + i;
        value = kind == 0 ? a.lse[e] * inv_scale : -a.delta[e];
      }
    };
    const auto keep = [&](int buf) {
      if (kind < 2 && row < N) (kind == 0 ? row_lse : row_delta)[set][buf][row] = value;
    };
    constexpr int kStride = Z::kSets;      // a wave of SHARE takes every fourth step
    const int all = steps * group;
    const auto position = [&](int it) { return p_first + it % steps * N; };
    const auto query_head = [&](int it) { return hk * group + it / steps; };
    int buf = 0, p0 = position(set), hq = query_head(set);
    if (set < all) {
      fetch(p0, hq, 0);
      keep(0);
    }
    if (SHARE && Z::kValuesInLds) {
      if constexpr (VEC) wait_loads();
      tile_barrier();        // the values are there
    }
    for (int it = set; it < all; it += kStride, buf ^= Z::kPairs - 1) {
#pragma unroll
      for (int n = 0; n < N / 32; ++n) live[n] = next[n];
      int p1 = p0 + N, hq1 = hq;
      if (SHARE) {
        p1 = position(it + kStride);
        hq1 = query_head(it + kStride);
      } else if (p1 >= end) {
        p1 = p_first;
        ++hq1;
      }
      if constexpr (VEC) wait_loads();
      // this tile is there; the other one has been read
      if constexpr (SHARE) {
        wait_lds();
        asm volatile("" ::: "memory");
      } else {
        tile_barrier();
      }
      const bool more = it + kStride < all;
      if (more && Z::kPairs == 2) fetch(p1, hq1, buf ^ 1);
      if (p0 < wend && p0 + N > wlo) {
        const uint32_t here = smem + buf * 2 * kTile;
        const Places qt = in_tile(pl, here), gt = in_tile(pl, here + kTile);
        const bool full = p0 >= full_lo && p0 + N <= full_end && all_live<N>(live);
        // S starts from -lse / scale and dO V^T from -delta: P = 2^(c S), dS = P dP
        const auto start = [&](const float* from_rows, int n, f32x16& x) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 y = *(const f32x4*)&from_rows[32 * n + 8 * q + 4 * h];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * q + k] = y[k];
          }
        };
        const auto mask = [&](int n, f32x16& s) {
          if (full) return;
          apart();
          const uint32_t w = live[n] >> (4 * h);
          const int base = p0 + 32 * n + 4 * h, first = from - base, stop = past - base;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int r = 8 * (j >> 2) + (j & 3);
            const bool in = r >= first && r < stop && ((w >> r) & 1);
            s[j] = in ? s[j] : -INFINITY;
          }
        };
        // position j0's only key is j0: dS = 0
        const auto alone = [&](int n, f32x16& dp) {
          if (full) return;
          apart();
          const int self = lone ? j0 - (p0 + 32 * n + 4 * h) : -1;
#pragma unroll
          for (int j = 0; j < 16; ++j) dp[j] = 8 * (j >> 2) + (j & 3) == self ? 0.0f : dp[j];
        };
        if constexpr (sizeof(S) == 2) {
          // per block of 32 queries G products for S, G for dP with the
          // exponentials between them, 2 DB for dv with dS between them, 2 DB for
          // dk; operands read kAhead products early
          constexpr int G = Sh::kG, DB = Sh::kDB, T = 2 * G + 4 * DB;
#pragma unroll
          for (int n = 0; n < N / 32; ++n) {
            const auto operand = [&](int t) -> u16x8 {
              if (t < G) return row_frag<E, DP>(qt, 32 * n, t);
              if (t < 2 * G) return row_frag<E, DP>(gt, 32 * n, t - G);
              const int u = (t - 2 * G) % (2 * DB);
              return column_frag<E, DP>(t < 2 * G + 2 * DB ? gt : qt, 32 * n, u % DB, u / DB, lane);
            };
            u16x8 x[kAhead], v[2];
            f32x16 s, dp;
            Weights<E> pw, dw;
            start(row_lse[set][buf], n, s);
#pragma unroll
            for (int t = 0; t < kAhead; ++t) x[t] = operand(t);
            fence();
#pragma unroll
            for (int t = 0; t < T; ++t) {
              const u16x8 y = x[t % kAhead];
              const int u = (t - 2 * G) % (2 * DB), db = u % DB, half = u / DB;
              if (t < G) s = mma<E>(y, kf[t], s);
              else if (t < 2 * G) dp = mma<E>(y, v[t % 2], dp);
              else if (t < 2 * G + 2 * DB) dv[db] = mma_column<E>(y, pw, half, dv[db]);
              else dk[db] = mma_column<E>(y, dw, half, dk[db]);
              if (t + kAhead < T) x[t % kAhead] = operand(t + kAhead);
              if (t + 2 >= G && t + 2 < 2 * G) v[t % 2] = value_frag(t + 2 - G);
              if (t == G - 2) start(row_delta[set][buf], n, dp);
              if (t >= G && t < 2 * G) {
#pragma unroll
                for (int j = 16 * (t - G) / G; j < 16 * (t - G + 1) / G; ++j) {
                  float e = __builtin_amdgcn_exp2f(s[j] * c);
                  asm volatile("" : "+v"(e));
                  s[j] = e;
                }
              }
              if (t >= 2 * G && t < 2 * G + 2 * DB) {
#pragma unroll
                for (int j = 16 * u / (2 * DB); j < 16 * (u + 1) / (2 * DB); ++j) {
                  float e = dp[j] * s[j];
                  asm volatile("" : "+v"(e));
                  dp[j] = e;
                }
              }
              fence();
              if (t == G - 1) mask(n, s);
              if (t == 2 * G - 1) {
                alone(n, dp);
                pw.set(s);
              }
              if (t == 2 * G + 2 * DB - 1) dw.set(dp);
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < N / 32; ++n) {
            f32x16 s, dp;
            start(row_lse[set][buf], n, s);
            start(row_delta[set][buf], n, dp);
#pragma unroll
            for (int g = 0; g < Sh::kG; ++g) s = mma<E>(row_frag<E, DP>(qt, 32 * n, g), kf[g], s);
#pragma unroll
            for (int g = 0; g < Sh::kG; ++g) dp = mma<E>(row_frag<E, DP>(gt, 32 * n, g), value_frag(g), dp);
            mask(n, s);
            alone(n, dp);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              s[j] = __builtin_amdgcn_exp2f(s[j] * c);
              dp[j] *= s[j];
            }
            Weights<E> pw, dw;
            pw.set(s);
            dw.set(dp);
#pragma unroll
            for (int db = 0; db < Sh::kDB; ++db) {
              dv[db] = mma_columns<E, DP>(gt, 32 * n, db, pw, dv[db], lane);
              dk[db] = mma_columns<E, DP>(qt, 32 * n, db, dw, dk[db], lane);
            }
          }
        }
      }
      if (more && Z::kPairs == 1) {      // one pair of tiles: the next after this has been read
        wait_lds();
        asm volatile("" ::: "memory");
        fetch(p1, hq1, 0);
      }
      if (more) keep(Z::kPairs == 2 ? buf ^ 1 : 0);
      p0 = p1;
      hq = hq1;
    }
    if constexpr (SHARE) {     // the waves' sums, added in their order by the first
      float* const sums = (float*)(shared_tiles + Z::kValues);
      __syncthreads();
      if (wave > 0) {
#pragma unroll
        for (int db = 0; db < Sh::kDB; ++db)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int at = (((wave - 1) * Sh::kDB + db) * 16 + j) * 128 + lane;
            sums[at] = dk[db][j];
            sums[at + 64] = dv[db][j];
          }
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
          for (int db = 0; db < Sh::kDB; ++db)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int at = ((w * Sh::kDB + db) * 16 + j) * 128 + lane;
              dk[db][j] += sums[at];
              dv[db][j] += sums[at + 64];
            }
      }
    }
  }
  if (!valid || (SHARE && wave > 0)) return;
  store_row<E, DP, VEC>((S*)a.dk.data + b * a.dk.sb + hk * a.dk.sh + (int64_t)j0 * a.dk.st, dk,
                        some, a.scale, a.D, lane);
  store_row<E, DP, VEC>((S*)a.dv.data + b * a.dv.sb + hk * a.dv.sh + (int64_t)j0 * a.dv.st, dv,
                        some, 1.0f, a.D, lane);
}

// Few workgroups leave compute units idle and give a wave a long chain of steps.
// With and without SHARE, us (bf16, f32; workgroups as without, steps of 32):
//                                            dq                       dk and dv
//   48, 16 steps, heads of 64     12.5 / 18.4  26.2 / 69.6   15.6 / 21.4  36.6 /  111
//   96, 16 steps, heads of 64            19.3  33.5 / 70.2   22.4 / 21.3  49.6 /  111
//  128, 32 steps, heads of 128    33.6 / 36.4   106 /  250   48.8 / 53.4   157 /  375
//  128, 320 steps, heads of 128                               217 /  436  1155 / 3633
//  192, 8 steps, heads of 64                                 28.2 / 15.8  62.4 / 62.6
//  256, 64 steps, heads of 128           60.6   345 /  489    129 /   97   519 /  739
// Up to 32 rows leave three waves of four without work: with SHARE, dk and dv of
// 512x32, 16/2x64 f32 100 us, without 251; of 512x32, 16/8x128 bf16, whose workgroups
// then have a compute unit alone, 253 and 91.
template <class E>
bool shared(int64_t rows, int64_t groups, int64_t steps) {
  constexpr bool kWide = sizeof(typename E::storage) == 4;
  return groups <= 64 || (kWide && rows <= 32 && steps > 1) ||
         (groups <= (kWide ? 256 : 128) && steps >= (kWide ? 16 : 32));
}

template <class E, int DP, bool VEC, bool SHARE>
hipError_t queries(const AttnArgs& a, hipStream_t s) {
  typedef Dq<E, DP, SHARE> Z;
  static hipError_t once = hipFuncSetAttribute((const void*)attention_dq_kernel<E, DP, VEC, SHARE>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, Z::kLds);
  if (once != hipSuccess) return once;
  const int64_t groups = (int64_t)a.B * a.Hq * ((a.Tq + Z::kQueries - 1) / Z::kQueries);
  timing_begin("attention_dq", s);
  hipLaunchKernelGGL((attention_dq_kernel<E, DP, VEC, SHARE>), dim3((unsigned)groups), dim3(kNT), Z::kLds, s, a);
  timing_end("attention_dq", s);
  return hipGetLastError();
}

template <class E, int DP, bool VEC, bool SHARE>
hipError_t keys(const AttnArgs& a, hipStream_t s) {
  typedef Dkv<E, DP, SHARE> Z;
  static hipError_t once = hipFuncSetAttribute((const void*)attention_dkv_kernel<E, DP, VEC, SHARE>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, Z::kLds);
  if (once != hipSuccess) return once;
  const int64_t groups = (int64_t)a.B * a.Hkv * ((a.Tk + Z::kKeys - 1) / Z::kKeys);
  timing_begin("attention_dkv", s);
  hipLaunchKernelGGL((attention_dkv_kernel<E, DP, VEC, SHARE>), dim3((unsigned)groups), dim3(kNT), Z::kLds, s,
                     a);
  timing_end("attention_dkv", s);
  return hipGetLastError();
}

template <class E, int DP, bool VEC>
hipError_t backward(const AttnArgs& a, hipStream_t s) {
  const int64_t q = (int64_t)a.B * a.Hq * ((a.Tq + kRows - 1) / kRows);
  const int64_t k = (int64_t)a.B * a.Hkv * ((a.Tk + kRows - 1) / kRows);
  const hipError_t e = shared<E>(a.Tq, q, (a.Tk + 31) / 32) ? queries<E, DP, VEC, true>(a, s)
                                                      : queries<E, DP, VEC, false>(a, s);
  if (e != hipSuccess) return e;
  return shared<E>(a.Tk, k, (int64_t)(a.Hq / a.Hkv) * ((a.Tq + 31) / 32)) ? keys<E, DP, VEC, true>(a, s)
                                                                    : keys<E, DP, VEC, false>(a, s);
}

template <class E>
hipError_t backward_e(const AttnArgs& a, hipStream_t s) {
  if (a.D <= 64) return a.vec ? backward<E, 64, true>(a, s) : backward<E, 64, false>(a, s);
  return a.vec ? backward<E, 128, true>(a, s) : backward<E, 128, false>(a, s);
}

}  // namespace
}  // namespace attn

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
  return a.dtype == kBF16 ? attn::backward_e<BF16>(a, s) : attn::backward_e<F32>(a, s);
}

}  // namespace dpf
