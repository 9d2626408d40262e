// Attention: arguments of the kernels, and the tiles they share (attention.hip,
// attention_bwd.hip).
#pragma once

#include <type_traits>

#include "lm.hpp"

namespace dpf {

constexpr int kAttnMaxD = 128;
constexpr int64_t kAttnMaxT = (int64_t)1 << 22;
// Batch x heads x tiles of 32 rows: of the queries, and of the keys where their gradients are taken.
constexpr int64_t kAttnMaxTiles = (int64_t)1 << 22;
constexpr int64_t kAttnMaxPositions = (int64_t)1 << 31;   // batch x Tk: 256 to a workgroup of `ranges`

struct AttnArgs {
  Heads q, k, v, o;         // o: the output (forward), read by the backward
  Heads dout, dq, dk, dv;   // backward only
  float* lse;               // [B, Hq, Tq], written (forward) or read (backward)
  float* delta;             // [B, Hq, Tq] workspace of the backward
  int dtype;
  int B, Tq, Tk, Hq, Hkv, D;
  int causal;
  float scale;              // > 0
  // Padding and packing (null without): what `ranges` makes of mask and segments.
  const uint8_t* mask;      // [B, Tk]
  const int32_t* segments;  // [B, Tk], not decreasing along T
  int32_t *lo, *end;        // [B, Tk] workspace
  uint32_t* bits;           // [B, nwords] workspace: bit t % 32 of word t / 32, active
  int nwords;               // 2 ceil(Tk / 64)
  int vec;                  // every row is 16-byte aligned and whole 16-byte pieces
  float* part;              // attention_part_floats: partial results of keys split over workgroups
  int splits;
};

// Workspace of mask and segments, and of split keys, in elements.
constexpr int kRowMask = 256;             // positions whose mask a wave keeps by itself (forward)
inline int attn_words(int64_t Tk) { return (int)(2 * ((Tk + 63) / 64)); }
// Fills a.splits; 0 floats without a split.
size_t attention_part_floats(AttnArgs& a);
hipError_t launch_attn_ranges(const AttnArgs& a, hipStream_t s);
hipError_t launch_attention(const AttnArgs& a, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s);

namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kOOB = 0x7ffffff0;          // past every buffer's end: such a load gives zeros

// A position's keys are [lo, end) less the inactive ones, up to itself when
// causal.  Without mask and segments [0, Tk).
struct Span { int lo, end; };
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b, int p) {
  if (a.lo == nullptr) return {0, a.Tk};
  const int64_t e = (int64_t)b * a.Tk + p;
  return {max(a.lo[e], 0), min(a.end[e], a.Tk)};     // no address from memory unchecked
}

// LDS tiles: rows of DP elements in 16-byte chunks, chunk c of row r stored at
// c ^ swz(r), so that 16 rows' equal chunks lie in different banks (row
// fragments, 16 bytes per lane) and so do 64 bytes of each of 4 rows (the
// transposing reads).
template <class E, int DP>
struct Shape {
  typedef typename E::storage S;
  static constexpr int kES = (int)sizeof(S);
  static constexpr int kRowBytes = DP * kES;
  static constexpr int kChunks = kRowBytes / 16;    // of a row: 8, 16 or 32
  static constexpr int kG = kChunks / 2;            // row fragments: two chunks, one per lane half
  static constexpr int kRowsPerDma = 64 / kChunks;
  static constexpr int kDB = DP / 32;               // 32-wide blocks of the head
};

template <int CHUNKS>
__device__ __forceinline__ int swz(int row) {
  if constexpr (CHUNKS == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  else return ((row & 3) << 2) | ((row >> 2) & 3);
}

// 16 bytes per lane from rsrc at voffset straight into LDS at lds + at + 16 * lane;
// awaited with wait_loads.
template <int AT>
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, int voffset, uint32_t lds) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voffset), "s"(rsrc), "s"(lds), "n"(AT)
               : "memory", "scc");
}
// Until every load this wave has queued is there.  The builtin, not assembly: the
// compiler has to know that its own loads are back too, or it waits for the next
// tile's along with them at their first use in the loop.
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0) expcnt(7) lgkmcnt(15)
  asm volatile("" ::: "memory");
}
// Until this wave's LDS reads are back: what they read may then be overwritten.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // vmcnt(63) expcnt(7) lgkmcnt(0)
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void tile_barrier() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)p;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Keeps what follows in a branch of its own: where the compiler runs it always
// and selects, a full tile pays for its mask (128 instructions of 370 per tile).
__device__ __forceinline__ void apart() { asm volatile("; masked" ::); }

template <int J, int PER, class F>
__device__ __forceinline__ void each(const F& f) {
  if constexpr (J < PER) {
    f(std::integral_constant<int, J>());
    each<J + 1, PER>(f);
  }
}

// 16 bytes of a row: 8 bf16 or 4 float32 elements, the operand of one
// 32x32x16 or four 32x32x2 products (k = lane half, then element).
template <class E> struct ChunkOf;
template <> struct ChunkOf<BF16> { typedef u16x8 type; };
template <> struct ChunkOf<F32> { typedef f32x4 type; };
template <class E> using Chunk = typename ChunkOf<E>::type;

// Entries d .. of a row of D (zeros past D, and all zeros where !in, though the row
// is read: it lies inside the tensor), of any alignment: the last piece is read from
// further back, so that nothing past the row is touched, and moved down.
template <class E>
__device__ __forceinline__ Chunk<E> load_piece(const typename E::storage* row, int d, int D, bool in) {
  typedef typename E::storage S;
  constexpr int kN = 16 / sizeof(S);
  Chunk<E> x = {};
  if (D >= kN) {
    const int back = max(min(d, D) + kN - D, 0);
    unsigned __int128 y;
    __builtin_memcpy(&y, row + (min(d, D) - back), 16);
    y = in && d < D ? y >> (8 * (int)sizeof(S) * (back & (kN - 1))) : 0;
    x = __builtin_bit_cast(Chunk<E>, y);
  } else {
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (in && d + k < D) x[k] = row[d + k];
  }
  return x;
}

// Brings rows [row0, row0 + ROWS) of one head's `rows` rows into an LDS tile, by
// NW waves (wave w of them).  Rows outside [0, rows) and those whose bit of `live`
// is 0 become zeros (of a negative row0 the caller's live has zeros there), and so
// does what lies past D.  VEC: direct loads to LDS, in flight until wait_loads.
// Scalar instructions are not free (a wave issues one in about five cycles): a
// lane's offsets within a tile are formed once and a buffer descriptor serves the
// 2^30 bytes after its first row, so that a tile costs a dozen of them.  Not VEC:
// through registers, in pieces of any alignment, there after a barrier.
template <class E, int DP, int ROWS, int NW, bool VEC>
struct Loader {
  typedef Shape<E, DP> Sh;
  typedef typename E::storage S;
  static constexpr int kPer = VEC ? ROWS / Sh::kRowsPerDma / NW : 1;
  static_assert(kPer >= 1, "a wave's share of a tile");
  const char* head;
  __amdgpu_buffer_rsrc_t rsrc;
  int first;              // row of the descriptor's base
  int off[kPer];
  int stride, rows, D, wave, lane;
  __device__ __forceinline__ Loader(const Heads& h, int n, int d, int w, int l)
      : head(nullptr), first(0), rows(n), D(d), wave(w), lane(l) {
    stride = (int)(h.st * Sh::kES);
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int row = (w * kPer + j) * Sh::kRowsPerDma + l / Sh::kChunks;
        const int chunk = (l % Sh::kChunks) ^ swz<Sh::kChunks>(row);
        off[j] = 16 * chunk < d * Sh::kES ? row * stride + 16 * chunk : kOOB;
      }
    }
  }
  // The head at element `at` of h, tiles from row0 on.
  __device__ __forceinline__ void start(const Heads& h, int64_t at, int row0) {
    head = (const char*)h.data + at * Sh::kES;
    if constexpr (VEC) base_at(row0);
    else stride = 0, strides = h.st;
  }
  int64_t strides;        // not VEC: of a row, in elements
  __device__ __forceinline__ void base_at(int row0) {
    first = row0;
    const int n = rows - row0;
    const uint64_t left = (uint64_t)(uint32_t)(n - 1) * (uint32_t)stride + (uint32_t)(D * Sh::kES);
    rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)(head + (int64_t)row0 * stride), (short)0,
                                             n <= 0 ? 0 : left < 0x7fff0000ull ? (int)left : 0x7fff0000,
                                             0x00020000);
  }
  __device__ __forceinline__ void operator()(uint32_t tile, int row0, uint64_t live) {
    if constexpr (VEC) {
      if ((int64_t)(row0 - first) * stride > (1 << 30)) base_at(row0);
      // an out-of-range offset stays one: it is above every descriptor's 2^31 bytes
      const int at = (row0 - first) * stride;
      const uint32_t to = uniform((int)tile + wave * kPer * 1024);
      constexpr uint64_t kAll = ROWS >= 64 ? ~0ull : (1ull << (ROWS & 63)) - 1;
      int now[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) now[j] = off[j] + at;
      if ((live & kAll) != kAll) {
        apart();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int row = (wave * kPer + j) * Sh::kRowsPerDma + lane / Sh::kChunks;
          now[j] = (live >> row) & 1 ? now[j] : kOOB;
        }
      }
      each<0, kPer>([&](auto j) { dma16<1024 * j>(rsrc, now[j], to); });
    } else {
      // all loads in flight, a piece outside from the head's first row and not used
      constexpr int kEach = ROWS * Sh::kChunks / (64 * NW);
      Chunk<E> x[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int e = (j * NW + wave) * 64 + lane, row = e / Sh::kChunks, i = row0 + row;
        const bool in = i >= 0 && i < rows && ((live >> row) & 1);
        x[j] = load_piece<E>((const S*)head + (in ? i : 0) * strides, e % Sh::kChunks * (16 / Sh::kES), D, in);
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int e = (j * NW + wave) * 64 + lane, row = e / Sh::kChunks;
        *(__attribute__((address_space(3))) Chunk<E>*)(uintptr_t)(
            tile + row * Sh::kRowBytes + 16 * ((e % Sh::kChunks) ^ swz<Sh::kChunks>(row))) = x[j];
      }
    }
  }
};

template <class E>
__device__ __forceinline__ f32x16 mma(const Chunk<E>& x, const Chunk<E>& y, f32x16 c) {
  if constexpr (sizeof(typename E::storage) == 2) {
    return mfma_32x32x16(x, y, c);
  } else {
    c = mfma_32x32x2(x.x, y.x, c);
    c = mfma_32x32x2(x.y, y.y, c);
    c = mfma_32x32x2(x.z, y.z, c);
    return mfma_32x32x2(x.w, y.w, c);
  }
}

// Where a lane's fragments lie in a tile at LDS address `tile` (a multiple of
// kTileAlign): fragment g of row lane % 32 at row ^ (g << 5), the transposing reads
// of the 32-wide block db and row quarter r at col ^ (db << 6 | r << 5), both plus
// whole rows (of at least as many bytes as the exclusive ors touch).
constexpr int kTileAlign = 512;
struct Places {
  uint32_t row, col;
};
template <class E, int DP>
__device__ __forceinline__ Places places(int lane) {
  typedef Shape<E, DP> Sh;
  const int h = lane >> 5, r = lane & 31, j = lane & 15, q = j >> 2;
  Places p;
  p.row = r * Sh::kRowBytes + 16 * (h ^ swz<Sh::kChunks>(r));
  p.col = (4 * h + q) * Sh::kRowBytes + 8 * (j & 1) +
          16 * ((2 * ((lane >> 4) & 1) + ((j & 3) >> 1)) ^ swz<Sh::kChunks>(4 * h + q));
  return p;
}
// The places of a tile, not derived from those of others: the addresses are then
// formed where they are used (one exclusive or each) instead of being kept in
// registers for every tile.
__device__ __forceinline__ Places in_tile(const Places& p, uint32_t tile) {
  Places x{p.row + tile, p.col + tile};
  asm volatile("" : "+v"(x.row), "+v"(x.col));
  return x;
}

template <class T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *(const __attribute__((address_space(3))) T*)(uintptr_t)at;
}

// Row fragment g of rows row0 + 0..31 of an LDS tile.
template <class E, int DP>
__device__ __forceinline__ Chunk<E> row_frag(const Places& at, int row0, int g) {
  return lds_at<Chunk<E>>((at.row ^ (g << 5)) + row0 * Shape<E, DP>::kRowBytes);
}

// The row fragments of one row in memory (this lane's: at element `at` of the array
// `safe`), zeros where !live.
template <class E, int DP, bool VEC>
__device__ __forceinline__ void row_frags_from(const typename E::storage* safe, int64_t at, bool live, int D, int lane,
                                               Chunk<E> (&f)[Shape<E, DP>::kG]) {
  typedef Shape<E, DP> Sh;
  constexpr int kN = 16 / Sh::kES;
  const typename E::storage* const row = safe + at;
#pragma unroll
  for (int g = 0; g < Sh::kG; ++g) {
    const int d = (2 * g + (lane >> 5)) * kN;
    if constexpr (VEC) {
      f[g] = Chunk<E>{};
      if (live && d < D) f[g] = *(const Chunk<E>*)(row + d);
    } else {
      f[g] = load_piece<E>(live ? row : safe, d, D, live);
    }
  }
}

// Two values as bf16, to nearest even, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}

// What a 32x32 accumulator holds per lane (register j: row 8 (j / 4) + 4 half
// + j % 4), as the right operand of products that sum over its 32 rows: for
// bf16 two fragments of 8 rows each (rounded to nearest even), for float32 the
// values themselves.
template <class E> struct Weights;
template <> struct Weights<BF16> {
  u16x8 f[2];
  __device__ __forceinline__ void set(const f32x16& p) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack_bf16(p[8 * s + 2 * k], p[8 * s + 2 * k + 1]);
      f[s] = __builtin_bit_cast(u16x8, w);
    }
  }
};
template <> struct Weights<F32> {
  f32x16 p;
  __device__ __forceinline__ void set(const f32x16& x) { p = x; }
};

// acc += (rows row0 .. row0 + 31 of the tile, columns 32 db ..)^T times w, in
// kColumnSteps products (bf16: two of 16 rows; float32: 16 of two).
template <class E> struct ColumnSteps;
template <> struct ColumnSteps<BF16> { static constexpr int kN = 2; };
template <> struct ColumnSteps<F32> { static constexpr int kN = 16; };

// The left operand of step s.
template <class E> struct ColumnOf;
template <> struct ColumnOf<BF16> { typedef u16x8 type; };
template <> struct ColumnOf<F32> { typedef float type; };
template <class E> using Column = typename ColumnOf<E>::type;

template <class E, int DP>
__device__ __forceinline__ Column<E> column_frag(const Places& at, int row0, int db, int s, int lane) {
  typedef Shape<E, DP> Sh;
  if constexpr (sizeof(typename E::storage) == 2) {
    u16x4 part[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
      part[r] = __builtin_bit_cast(u16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(uintptr_t)(
          (at.col ^ (db << 6 | r << 5)) + (row0 + 16 * s + 8 * r) * Sh::kRowBytes)));
    return __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    // col is made for the transposing reads: its row and its chunk differ here
    const int h = lane >> 5, d = 32 * db + (lane & 31), row = 8 * (s >> 2) + 4 * h + (s & 3);
    const int chunk = (d >> 2) ^ swz<Sh::kChunks>(row);
    const uint32_t tile = at.row - places<E, DP>(lane).row;
    return lds_at<float>(tile + (row0 + row) * Sh::kRowBytes + 16 * chunk + 4 * (d & 3));
  }
}
template <class E>
__device__ __forceinline__ f32x16 mma_column(const Column<E>& x, const Weights<E>& w, int s, const f32x16& acc) {
  if constexpr (sizeof(typename E::storage) == 2) return mfma_32x32x16(x, w.f[s], acc);
  else return mfma_32x32x2(x, w.p[s], acc);
}
template <class E, int DP>
__device__ __forceinline__ f32x16 mma_columns(const Places& at, int row0, int db, const Weights<E>& w,
                                              f32x16 acc, int lane) {
#pragma unroll
  for (int s = 0; s < ColumnSteps<E>::kN; ++s)
    acc = mma_column<E>(column_frag<E, DP>(at, row0, db, s, lane), w, s, acc);
  return acc;
}

// Products that an operand is read ahead of its own: an LDS read takes longer than
// a product.
constexpr int kAhead = 4;

__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Stores this lane's columns of the transposed result (registers of block db:
// entries 32 db + 8 (j / 4) + 4 half + j % 4 of the row) times f, zeros where
// !live, whatever the registers hold.
template <class E, int DP, bool VEC>
__device__ __forceinline__ void store_row(typename E::storage* row, const f32x16 (&acc)[DP / 32], bool live,
                                          float f, int D, int lane) {
  const int h = lane >> 5;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 32 * db + 8 * i + 4 * h;
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = live ? acc[db][4 * i + k] * f : 0.0f;
      typedef typename E::storage S;
      typedef S four __attribute__((ext_vector_type(4)));
      four y;
      if constexpr (sizeof(S) == 2) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        y = __builtin_bit_cast(four, u2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])});
      } else {
        y = four{x[0], x[1], x[2], x[3]};
      }
      if constexpr (VEC) {
        if (d < D) *(four*)(row + d) = y;
      } else {
        if (d + 4 <= D) {
          __builtin_memcpy(row + d, &y, sizeof(y));
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (d + k < D) row[d + k] = y[k];
        }
      }
    }
}

__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int j = 1; j < 64; j <<= 1) x = min(x, lane_xor(x, j));
  return uniform(x);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int j = 1; j < 64; j <<= 1) x = max(x, lane_xor(x, j));
  return uniform(x);
}

// The active bits of keys k0 .. k0 + KEYS - 1 (k0 a multiple of KEYS).
template <int KEYS>
__device__ __forceinline__ uint64_t live_keys(const AttnArgs& a, int b, int k0,
                                              uint32_t (&w)[KEYS / 32]) {
  if (a.bits == nullptr) {
#pragma unroll
    for (int n = 0; n < KEYS / 32; ++n) w[n] = ~0u;
    return ~0ull;
  }
  const uint32_t* p = a.bits + (int64_t)b * a.nwords + k0 / 32;
#pragma unroll
  for (int n = 0; n < KEYS / 32; ++n) w[n] = uniform(p[n]);
  return KEYS == 64 ? ((uint64_t)w[KEYS / 32 - 1] << 32) | w[0] : (uint64_t)w[0];
}

template <int KEYS>
__device__ __forceinline__ bool all_live(const uint32_t (&w)[KEYS / 32]) {
  uint32_t x = ~0u;
#pragma unroll
  for (int n = 0; n < KEYS / 32; ++n) x &= w[n];
  return x == ~0u;
}

// Heads of a set (see place) that read keys and values of their own: a large set
// balances better, but its keys and values leave the L2 of 4 MB (gradients of
// 8x2048, 40x128 in sets of 4, 5, 8: 1402, 1411, 1460 us; of 32x512, 12x64: 119, 122,
// 116).  Heads of a group count once.
template <class E>
__device__ __forceinline__ int heads_at_once(const AttnArgs& a) {
  return (int64_t)a.Tk * a.D * (int)sizeof(typename E::storage) > 256 * 1024 ? 4 : 8;
}

// Head and tile of a workgroup (heads * tiles of them).  Workgroups that read the
// same keys and values (the tiles of a head, the heads of a group) are given to one
// XCD one after another, so that they find them in its L2; the heads left over by
// eight go to all XCDs, tile by tile.  An XCD takes its heads in sets of up to
// `at_once`, a set's first tiles (callers count from the longest ones of a causal
// call) before its next: head after head, the last head's long tiles came last and
// left compute units idle (8x2048, 40x128: 442 us, in sets of 4 408; packed 1x8192,
// 40/8x128: 264, in sets of 5 219).
__device__ __forceinline__ void place(int heads, int tiles, int at_once, int* head, int* tile) {
  const int L = blockIdx.x, each = heads / 8, rest = heads % 8, whole = 8 * each * tiles;
  if (L < whole) {
    const int sets = (each + at_once - 1) / at_once, most = (each + sets - 1) / sets;
    const int at = L >> 3, set = at / (most * tiles), in_set = at % (most * tiles);
    const int n = min(most, each - set * most);
    *head = (L & 7) * each + set * most + in_set % n;
    *tile = in_set / n;
  } else {
    *head = 8 * each + (L - whole) % rest;
    *tile = (L - whole) / rest;
  }
}

}  // namespace attn
}  // namespace dpf
