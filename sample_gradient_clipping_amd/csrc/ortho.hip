// Orthogonalised update by Newton-Schulz products.  For a matrix U [R, C]:
//
//   X_0 = U / max(||U||_F, eps)
//   X <- a X + (b A + c A^2) X,  A = X X^T      (R <= C; else X (b A + c A^2), A = X^T X)
//
// `steps` times: each singular value s of X goes to a s + b s^3 + c s^5, which
// the coefficients drive towards 1, and the singular vectors stay.  Computed as
//
//   A' = A + (b / 2c) I,  B = c A'^2 + (a - b^2 / 4c) I,  X <- B X
//
// so that every product's result is only scaled, shifted on its diagonal and
// stored: nothing is read back (with c = 0: B = b A + a I, and no square).  A
// shift that is large beside A's eigenvalues would take A's low bits with it:
// then the square is c A^2, and a pass over it adds b A + a I (completed_square
// below).  The optimizer step forms U from the gradient and the momentum, and
// subtracts the result from the weight.
//
// Products.  Every operand is kept as two half-precision matrices hi + lo
// (hi = half(v), lo = half(v - hi), 22 bits together), scaled by a power of two
// so that its largest possible value is just below half's largest.  A product
// is three MFMA products, hi hi + hi lo + lo hi, summed in float32: what is left
// out, lo lo, is 2^-22 of the product, below float32's own rounding of a
// sum.  The small singular values are what needs this: a step multiplies
// them by up to a, and an error in X as large as bfloat16's rounding would be
// multiplied with them.
//
// A and B are symmetric: only the tiles on and above the
// diagonal are computed, and stored twice.
//
// Layouts.  X stays as U is stored.  With R <= C the products contract X's
// rows (K-inner operands) for A, and B X contracts over rows of X (K-outer
// operands, B read as its own transpose).  With R > C it is the other way
// round, so two kernels serve both shapes and nothing is ever transposed.  In
// memory the halves alternate, 16 hi and then the same 16 lo, so that a step
// of 16 along K takes both from one place.  All dimensions are padded with
// zeros to whole tiles.
//
// Product kernel.  Tiles of 256 x 256 on 8 waves (128 x 64 each) or 128 x 128
// on 4 (64 x 64; two workgroups per compute unit), K in steps of 16.  A step's
// operands go from memory to LDS directly (16 bytes a lane), into a ring of
// five slots, four steps ahead (ten slots and nine steps where the grid leaves a
// compute unit to one workgroup of 4 waves: a step is then shorter than a load
// takes); LDS chunks are permuted so that the fragment
// reads hit every bank once.  Per step a wave reads its fragments one block
// ahead of the MFMAs, 3 MFMAs per block and half pair: 24 (12) MFMAs on 12 (8)
// fragments, so LDS is busy for two thirds of the MFMAs' time.  One barrier
// per step, in its middle: it certifies that the next step has landed and that
// every wave is done with the step before, whose slot is then refilled.
//
// Where a product has too few tiles for the chip, several workgroups share a
// tile's steps and leave float32 parts that a second kernel adds in order.
// Matrices that fit into LDS take one workgroup for the whole call, other
// thin ones (up to 96 rows or columns) two launches a step.
//
// What it costs (MI355X).  The MFMAs bound it.  A 13824 x 5120 step takes 15.6
// to 16.4 ms: five times X^T X 0.91 ms (1250 TFLOP/s of half-precision products),
// the square 0.34 (1210), B X 1.89 (1150), where a large half-precision library
// product reaches 1170; norm and split 0.15 and 0.18 (1.1 and 0.7 GB: 7 and 4
// TB/s).  The clock falls to 2.0 to 2.1 GHz under these, so that keeping the
// MFMAs busier than half the cycles buys little.  Twelve 768 x 768 take 490 us:
// per step 31 each for the symmetric products (600 TFLOP/s: 252 tiles of 128 on
// 256 compute units, one wave per SIMD) and 41 for B X (790: 432 tiles on 512
// places).  One 768 x 768 takes 295, 1024 x 4096 450 us, 4096 x 4096 3.9 ms;
// 64 x 32 20 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lm.hpp"

namespace dpf {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kSumBlocks = 2048;    // most workgroups of one matrix's norm

__device__ __forceinline__ f32x16 mma16(const u16x8& a, const u16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A matrix as pairs of halves: element (r, c) at r ld + 2 (c - c % 16) + c % 16,
// its lo part 16 further; the next matrix of the stack `next` further.
struct Pair {
  uint16_t* p;
  int64_t ld, next;
  __device__ __forceinline__ Pair at(int64_t k) const { return Pair{p + k * next, ld, next}; }
  __device__ __forceinline__ uint16_t* elem(int64_t r, int64_t c) const {
    return p + r * ld + 2 * c - (c & 15);
  }
};

// Four elements of a row (c a multiple of 4).
__device__ __forceinline__ void store_pair(const Pair& p, int64_t r, int64_t c, const float (&v)[4]) {
  f16x4 h, l;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = (_Float16)v[k];
    l[k] = (_Float16)(v[k] - (float)h[k]);
  }
  uint16_t* e = p.elem(r, c);
  *(f16x4*)e = h;
  *(f16x4*)(e + 16) = l;
}

// ---------------------------------------------------------------------------
// Momentum and norm
// ---------------------------------------------------------------------------
template <class E, bool MUON>
__device__ __forceinline__ float update_at(const OrthoArgs& a, int64_t e) {
  if constexpr (MUON) {
    const float g = a.grad[e], m = a.momentum[e];
    return a.nesterov ? g + a.beta * m : m;
  } else {
    return E::to_float(((const typename E::storage*)a.in)[e]);
  }
}

// V consecutive elements of the update from element e on; `first` pass: the
// momentum is moved on.
template <class E, bool MUON, int V, bool FIRST>
__device__ __forceinline__ void update_from(const OrthoArgs& a, int64_t e, float (&u)[V]) {
  if constexpr (MUON) {
    float g[V], m[V];
    load_f32<F32, V>(a.grad + e, g);
    load_f32<F32, V>(a.momentum + e, m);
    if constexpr (FIRST) {
#pragma unroll
      for (int k = 0; k < V; ++k) m[k] = a.beta * m[k] + g[k];
      store_f32<F32, V>(a.momentum + e, m);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) u[k] = a.nesterov ? g[k] + a.beta * m[k] : m[k];
  } else {
    load_f32<E, V>((const typename E::storage*)a.in + e, u);
  }
}

// V: 4 where a matrix's elements are a multiple of 4, else 1.
template <class E, bool MUON, int V>
__global__ void __launch_bounds__(256) ortho_norm_kernel(OrthoArgs a, double* part) {
  __shared__ double red[4];
  const int64_t len = a.R * a.C, base = (int64_t)blockIdx.y * len;
  double sq = 0.0;
  const int64_t step = (int64_t)gridDim.x * 256 * V;
#pragma unroll 4
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < len; i += step) {
    float u[V];
    update_from<E, MUON, V, true>(a, base + i, u);
#pragma unroll
    for (int k = 0; k < V; ++k) sq += (double)u[k] * (double)u[k];
  }
  sq = block_sum_f64(sq, red);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sq;
}

// X_0 times 2^sx as a pair, zero in the padding.  A norm that is not finite
// makes the whole matrix NaN.  A norm below eps leaves X_0 small, and half has
// few exponents: X is then kept times unit = 2^e, the largest power that no
// step can carry past the range (a step takes s to at most |a| s + |b| s^3 +
// |c| s^5), and A and the result are scaled back.
constexpr int kMaxUnit = 100;
__device__ __forceinline__ double input_scale(const OrthoArgs& a, double sq, float pow_x, int* unit) {
  const double norm = sqrt(sq);
  int e = 0;
  if (norm < a.eps && norm > 0.0) {
    double v = norm / a.eps, most = v;
    for (int k = 0; k < a.steps && most < 1.0; ++k) {
      v *= fabs(a.a) + v * v * (fabs(a.b) + v * v * fabs(a.c));
      most = fmax(most, v);
    }
    if (most < 1.0) e = min(kMaxUnit, ilogb(1.0 / most));
  }
  *unit = e;
  return norm < __builtin_huge_val() ? ldexp((double)pow_x, e) / (norm > a.eps ? norm : a.eps)
                                     : __builtin_nan("");
}

// V: 4 where C is a multiple of 4, else 1.
template <class E, bool MUON, int V>
__global__ void __launch_bounds__(256) ortho_split_kernel(OrthoArgs a, const double* part, int nb,
                                                          Pair X, int Rp, int Cp, float pow_x,
                                                          float* unit) {
  __shared__ double scale;
  if (threadIdx.x < 64) {
    double sq = 0.0;
    for (int k = threadIdx.x; k < nb; k += 64) sq += part[(int64_t)blockIdx.y * nb + k];
    sq = wave_sum_f64(sq);
    if (threadIdx.x == 0) {
      int e;
      scale = input_scale(a, sq, pow_x, &e);
      if (blockIdx.x == 0) unit[blockIdx.y] = ldexpf(1.0f, -e);
    }
  }
  __syncthreads();
  const double f = scale;
  const Pair x = X.at(blockIdx.y);
  const int64_t base = (int64_t)blockIdx.y * a.R * a.C;
  const int per = Cp / 4, R = (int)a.R, C = (int)a.C;   // lanes of a row
  // rows in steps of the grid's, a row's groups of four side by side
  const int64_t total = (int64_t)Rp * per, step = (int64_t)gridDim.x * 256;
  const int64_t q0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int r = (int)(q0 / per), c4 = (int)(q0 - (int64_t)r * per);
  const int dr = (int)(step / per), dc = (int)(step - (int64_t)dr * per);
#pragma unroll 2
  for (int64_t q = q0; q < total; q += step) {
    const int c = 4 * c4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < R && c < C) {
      const int64_t e = base + (int64_t)r * C + c;
      if constexpr (V == 4) {
        update_from<E, MUON, 4, false>(a, e, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < C) {
            float one[1];
            update_from<E, MUON, 1, false>(a, e + k, one);
            v[k] = one[0];
          }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r < R && c + k < C ? (float)((double)v[k] * f) : 0.f;
    store_pair(x, r, c, v);
    r += dr;
    c4 += dc;
    if (c4 >= per) { c4 -= per; ++r; }
  }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// D[M][N] = f sum_k L(M, k) R(N, k), symmetric ones plus `shift` on the
// diagonal; stored as pairs, or (the last one) to the caller's matrix.
enum Mode { kStore = 0, kFinal = 1 };
struct ProductArgs {
  Pair L, R, out;
  int steps;              // K / 16
  int mt, nt;             // tiles of M and N (symmetric: mt == nt)
  int tiles;              // per matrix
  int64_t total;          // steps of all tiles of all matrices
  int groups;             // workgroups that share them
  float* parts;           // [2 groups][tile] float32 parts of shared tiles
  int sym, mode, dtype;
  float f, shift;
  const float* unit;      // [n] 1 / unit of each matrix's X
  int units;              // power of it that is part of f
  // kFinal
  int64_t rows, cols;
  void* dst;              // [rows, cols] of dtype, or the weight (float32)
  int muon;
  float decay, size;
};

template <int TILE, int WAVES, int SLOTS>
struct Shape {
  static constexpr int kTile = TILE, kWaves = WAVES, kSlots = SLOTS;
  static constexpr int kAhead = kSlots - 1;                 // steps between a slot's load and its use
  static constexpr int kNT = kWaves * 64;
  static constexpr int kWR = 2, kWC = kWaves / 2;           // wave grid, M by N
  static constexpr int kBA = TILE / kWR / 32, kBO = TILE / kWC / 32;   // 32 x 32 blocks of a wave
  static constexpr int kOpBytes = TILE * 64;                // one operand's step
  static constexpr int kSlotBytes = 2 * kOpBytes;
  static constexpr int kLds = kSlots * kSlotBytes;
  static constexpr int kFloats = TILE * TILE;               // one tile's accumulators
  static constexpr int kDma = kOpBytes / 1024 / kWaves;     // loads of a wave per operand and step
  static_assert(kOpBytes == 2 * 1024 * kWaves && kBO == 2, "the main loop's order of reads and loads");
};

// 16 bytes per lane from rsrc at voffset straight into LDS at m0 + 16 * lane;
// awaited explicitly (wait_dma).
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voffset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voffset), "s"(rsrc), "s"(lds)
               : "memory");
}

// Until at most LOADS of this wave's latest loads are in flight.
template <int LOADS>
__device__ __forceinline__ void wait_dma() {
  static_assert(LOADS < 64, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
}

// A barrier without the compiler's wait for every outstanding LDS read: what
// other waves may overwrite after it has been used by MFMAs before it.
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)p;
}

// `live` false: a buffer of no bytes, whose loads touch no memory and give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, bool live) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, live ? 0x7fffffff : 0, 0x00020000);
}

// LDS image of one operand's step, and its loads.
//   K-inner: [TILE rows][64 bytes]: k 0-7 hi, 8-15 hi, 0-7 lo, 8-15 lo, 16-byte
//            chunk c of row r at c ^ ((r >> 2) & 3).
//   K-outer: [16 k][TILE columns, 64 bytes per 16]: the chunk's index with its
//            bits 2 and 3 inverted by k's low bits (four rows of a transposing
//            read fall on different banks) and the hi/lo bit by bit 2 (so do
//            the two 16-column halves of a block).
template <class S, bool KI>
struct Operand {
  static constexpr int TILE = S::kTile;
  const char* base;               // this tile's next step
  int64_t step;                   // bytes between steps
  uint32_t off[S::kDma];          // per lane: the wave's loads
  __device__ __forceinline__ void start(const Pair& p, int64_t m0, int64_t k0) {
    const int64_t ldb = p.ld * 2;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    base = (const char*)p.p + (KI ? m0 * ldb + k0 * 64 : m0 * 4 + k0 * 16 * ldb);
    step = KI ? 64 : 16 * ldb;
#pragma unroll
    for (int j = 0; j < S::kDma; ++j) {
      const int d = wave * S::kDma + j;
      if constexpr (KI) {
        const int row = d * 16 + (lane >> 2), c = (lane & 3) ^ ((row >> 2) & 3);
        off[j] = (uint32_t)(row * ldb + c * 16);
      } else {
        constexpr int kCpr = TILE / 4;
        const int k = (d * 64 + lane) / kCpr, q = ((d * 64 + lane) % kCpr) ^ ((k & 3) << 2);
        off[j] = (uint32_t)(k * ldb + (q ^ (((q >> 2) & 1) << 1)) * 16);
      }
    }
  }
  // Load j of the next step into its slot; the last one moves on.
  __device__ __forceinline__ void load(int j, uint32_t lds, int wave, bool live) {
    dma16(rsrc_of(base, live), off[j], lds + (uint32_t)(wave * S::kDma + j) * 1024u);
    if (j + 1 == S::kDma) base += step;
  }
};

// This lane's fragment reads of an operand: blocks of 32 from block `b0` on, the
// hi half at the address and lo at address ^ 32.
template <int TILE, bool KI>
struct FragLane {
  uint32_t even, odd;             // for blocks b0 + 0, 2, .. and b0 + 1, 3, ..
  __device__ __forceinline__ void start(int b0) {
    const int lane = threadIdx.x & 63;
    if constexpr (KI) {
      const int c = (lane >> 5) ^ ((lane >> 2) & 3);
      even = odd = (uint32_t)(b0 * 2048 + (lane & 31) * 64 + c * 16);
    } else {
      const int k = 8 * (lane >> 5) + ((lane & 15) >> 2), kb = (k >> 1) & 1;
      const int lp = ((lane >> 4) & 1) * 4 + ((lane & 3) >> 1);
      const int c = lp ^ (((lp >> 2) & 1) << 1) ^ ((k & 1) << 2);
      const uint32_t at = (uint32_t)(k * TILE * 4 + b0 * 128 + c * 16 + (lane & 1) * 8);
      const uint32_t swap = (uint32_t)(kb * 128);      // an even block and the next change places
      even = (b0 & 1) ? at - swap : at + swap;
      odd = (b0 & 1) ? at + swap : at - swap;
    }
  }
  template <int I>
  __device__ __forceinline__ u16x8 read(const unsigned char* op, bool lo) const {
    const uint32_t at = ((I & 1) ? odd : even) ^ (lo ? 32u : 0u);
    if constexpr (KI) {
      return *(const u16x8*)(op + at + I * 2048);
    } else {
      const u16x4 a = lds_read_tr16((const uint16_t*)(op + at + I * 128));
      const u16x4 b = lds_read_tr16((const uint16_t*)(op + at + I * 128 + 4 * TILE * 4));
      u16x8 f;
      f.s0 = a.s0; f.s1 = a.s1; f.s2 = a.s2; f.s3 = a.s3;
      f.s4 = b.s0; f.s5 = b.s1; f.s6 = b.s2; f.s7 = b.s3;
      return f;
    }
  }
};

// Tile t of a matrix: groups of four tile rows, within them column by column,
// so that the tiles in flight on one XCD share operand strips in its L2; with
// `sym` those on and above the diagonal.
__device__ __forceinline__ void tile_of(const ProductArgs& p, int t, int* ti, int* tj) {
  int r0 = 0;
  for (;;) {
    const int h = min(4, p.mt - r0);
    const int count = p.sym ? h * (p.nt - r0) - h * (h - 1) / 2 : h * p.nt;
    if (t < count) {
      if (!p.sym) {
        *ti = r0 + t % h;
        *tj = t / h;
        return;
      }
      const int head = h * (h + 1) / 2;          // the triangle at the diagonal
      if (t < head) {
        int j = 0;
        while (t > j) { t -= j + 1; ++j; }
        *ti = r0 + t;
        *tj = r0 + j;
      } else {
        *ti = r0 + (t - head) % h;
        *tj = r0 + h + (t - head) / h;
      }
      return;
    }
    t -= count;
    r0 += h;
  }
}

__device__ __forceinline__ int64_t first_step(const ProductArgs& p, int w) {
  return p.total * w / p.groups;
}

// Workgroups go round the eight XCDs; each XCD takes a contiguous share.
__device__ __forceinline__ int logical_group(int id, int groups) {
  const int q = groups / 8, r = groups % 8, x = id % 8;
  return x * q + min(x, r) + id / 8;
}

// Block row i of every wave of a tile (64 rows of the result), scaled, shifted
// on the diagonal, and stored.  The accumulators hold 8 bytes of each of 32
// rows; they go through LDS, so that memory sees whole lines.
constexpr int kStageRows = 64;
template <int TILE>
constexpr int stage_bytes() {
  const int rows = kStageRows * (TILE * 4 + 16), mirror = TILE * (kStageRows * 4 + 16);
  return rows > mirror ? rows : mirror;
}

template <class S>
__device__ __forceinline__ void store_rows(const ProductArgs& p, int64_t mat, int ti, int tj, int i,
                                           const f32x16 (&acc)[S::kBO],
                                           unsigned char* lds) {
  constexpr int TILE = S::kTile;
  static_assert(S::kWR * 32 == kStageRows, "two blocks of 32 rows");
  static_assert(stage_bytes<TILE>() <= S::kLds, "the stage fits into the ring");
  constexpr int kLine = TILE * 4 + 16, kMirrorLine = kStageRows * 4 + 16;
  // Hidden from the optimiser, which would otherwise keep these addresses in
  // registers through the main loop.
  int tid = (int)threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int wave = tid >> 6, lane = tid & 63;
  const int wm = wave / S::kWC, wn = wave % S::kWC;
  const int64_t m0 = (int64_t)ti * TILE, n0 = (int64_t)tj * TILE;
  // stage row s holds row m0 + (s / 32) * kBA * 32 + i * 32 + s % 32
  const int srow = wm * 32 + (lane & 31);
  const int64_t r = m0 + (wm * S::kBA + i) * 32 + (lane & 31);
  float f = p.f;
  for (int k = 0; k < p.units; ++k) f *= p.unit[mat];
  const bool mirror = p.sym && ti != tj;
  __syncthreads();                                  // the ring, or the last rows, are read
  if (p.mode == kFinal) {
#pragma unroll
    for (int j = 0; j < S::kBO; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(f32x4*)(lds + srow * kLine + ((wn * S::kBO + j) * 32 + (8 * g + 4 * (lane >> 5))) * 4) =
            f32x4{f * acc[j][4 * g], f * acc[j][4 * g + 1], f * acc[j][4 * g + 2], f * acc[j][4 * g + 3]};
  } else {
    // the tile column of this lane's diagonal element, if it has one
    const int diag = p.sym && ti == tj ? (int)(r - n0) : -1;
#pragma unroll
    for (int j = 0; j < S::kBO; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = (wn * S::kBO + j) * 32 + (8 * g + 4 * (lane >> 5));
        f16x4 h, l;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = f * acc[j][4 * g + k] + (c + k == diag ? p.shift : 0.f);
          h[k] = (_Float16)x;
          l[k] = (_Float16)(x - (float)h[k]);
        }
        unsigned char* e = lds + srow * kLine + (2 * c - (c & 15)) * 2;
        *(f16x4*)e = h;
        *(f16x4*)(e + 32) = l;
      }
  }
  __syncthreads();
  constexpr int kChunks = TILE / 4;                 // 16-byte chunks of a stage row
  if (p.mode == kStore) {
    const Pair out = p.out.at(mat);
#pragma unroll 4
    for (int q = tid; q < kStageRows * kChunks; q += S::kNT) {
      const int s = q / kChunks, c = q % kChunks;
      const int64_t row = m0 + (s >> 5) * (S::kBA * 32) + i * 32 + (s & 31);
      *(u32x4*)((char*)(out.p + row * out.ld) + n0 * 4 + c * 16) = *(const u32x4*)(lds + s * kLine + c * 16);
    }
    if (!mirror) return;
    // the same values as columns: row n0 + c of the result, 32 of its columns
    // (128 bytes) per block of rows
    __syncthreads();
#pragma unroll
    for (int j = 0; j < S::kBO; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int c = (wn * S::kBO + j) * 32 + acc_row(k, lane), q = (lane & 31);
        const float x = f * acc[j][k];
        const _Float16 h = (_Float16)x, l = (_Float16)(x - (float)h);
        unsigned char* e = lds + c * kMirrorLine + wm * 128 + (2 * q - (q & 15)) * 2;
        *(_Float16*)e = h;
        *(_Float16*)(e + 32) = l;
      }
    __syncthreads();
#pragma unroll 4
    for (int q = tid; q < TILE * 16; q += S::kNT) {
      const int c = q >> 4, half = (q >> 3) & 1, x = q & 7;
      const int64_t col = m0 + half * (S::kBA * 32) + i * 32;
      *(u32x4*)((char*)(out.p + (n0 + c) * out.ld) + col * 4 + x * 16) =
          *(const u32x4*)(lds + c * kMirrorLine + half * 128 + x * 16);
    }
    return;
  }
  for (int q = tid; q < kStageRows * kChunks; q += S::kNT) {
    const int s = q / kChunks;
    const int64_t row = m0 + (s >> 5) * (S::kBA * 32) + i * 32 + (s & 31), c = n0 + (q % kChunks) * 4;
    if (row >= p.rows || c >= p.cols) continue;
    const f32x4 x = *(const f32x4*)(lds + s * kLine + (q % kChunks) * 16);
    const int64_t e = (mat * p.rows + row) * p.cols + c;
    if (p.cols % 4 == 0) {                          // whole and aligned
      if (p.muon) {
        f32x4* w = (f32x4*)((float*)p.dst + e);
        f32x4 old = *w;
#pragma unroll
        for (int k = 0; k < 4; ++k) old[k] = p.decay * old[k] - p.size * x[k];
        *w = old;
      } else {
        float y[4] = {x[0], x[1], x[2], x[3]};
        if (p.dtype == kBF16) store_f32<BF16, 4>((uint16_t*)p.dst + e, y);
        else store_f32<F32, 4>((float*)p.dst + e, y);
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c + k >= p.cols) break;
      if (p.muon) {
        float* w = (float*)p.dst + e + k;
        *w = p.decay * *w - p.size * x[k];
      } else if (p.dtype == kBF16) {
        ((uint16_t*)p.dst)[e + k] = f32_to_bf16_rne(x[k]);
      } else {
        ((float*)p.dst)[e + k] = x[k];
      }
    }
  }
}

__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

template <class S, bool KI>
__global__ void __launch_bounds__(S::kNT, 2) ortho_product_kernel(ProductArgs p) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  constexpr int TILE = S::kTile, kLoads = 2 * S::kDma, kAhead = S::kAhead, kSlots = S::kSlots;
  constexpr int BA = S::kBA, BO = S::kBO;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = logical_group(blockIdx.x, p.groups);
  const int64_t s0 = first_step(p, w), s1 = first_step(p, w + 1);
  FragLane<TILE, KI> fl, fr;
  fl.start(wave / S::kWC * BA);
  fr.start(wave % S::kWC * BO);
  const uint32_t lds0 = lds_addr(lds);
  bool first = true;
  for (int64_t at = s0; at < s1;) {
    const int64_t tile = at / p.steps;
    const int mat = __builtin_amdgcn_readfirstlane((int)(tile / p.tiles));
    const int k0 = __builtin_amdgcn_readfirstlane((int)(at - tile * p.steps));
    // steps of this piece
    const int n = __builtin_amdgcn_readfirstlane((int)min((int64_t)(p.steps - k0), s1 - at));
    int ti, tj;
    tile_of(p, (int)(tile - (int64_t)mat * p.tiles), &ti, &tj);
    ti = __builtin_amdgcn_readfirstlane(ti);
    tj = __builtin_amdgcn_readfirstlane(tj);
    Operand<S, KI> ol, orr;
    ol.start(p.L.at(mat), (int64_t)ti * TILE, k0);
    orr.start(p.R.at(mat), (int64_t)tj * TILE, k0);
    f32x16 acc[BA][BO];
#pragma unroll
    for (int i = 0; i < BA; ++i)
#pragma unroll
      for (int j = 0; j < BO; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    if (!first) __syncthreads();                 // the last piece's slots are read
    // Load d (operand d % 2) of a step, into the slot at `to`.  Steps past the
    // last are loaded too, as nothing (`live`): the loop has no branch then,
    // and a wave always has the same number of loads in flight.
    auto dma = [&](int d, uint32_t to, bool live) {
      if (d & 1) orr.load(d >> 1, to + S::kOpBytes, wave, live);
      else ol.load(d >> 1, to, wave, live);
    };
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int d = 0; d < kLoads; ++d) dma(d, lds0 + (uint32_t)s * S::kSlotBytes, s < n);
    wait_dma<kLoads * (kAhead - 1)>();
    step_barrier();
    // Fragments [.. block][hi, lo]: of the step at hand and, as they are used
    // up, of the next.
    constexpr int NL = BA == 4 ? 1 : 2;
    u16x8 L[NL][BA][2], R[2][BO][2];
    auto read_l = [&](auto buf, auto i, int lo, const unsigned char* slot) {
      L[decltype(buf)::value][decltype(i)::value][lo] = fl.template read<decltype(i)::value>(slot, lo != 0);
    };
    auto read_r = [&](auto buf, auto j, int lo, const unsigned char* slot) {
      R[decltype(buf)::value][decltype(j)::value][lo] =
          fr.template read<decltype(j)::value>(slot + S::kOpBytes, lo != 0);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
#pragma unroll
    for (int lo = 0; lo < 2; ++lo) {
      read_r(I0(), I0(), lo, lds);
      if constexpr (BO > 1) read_r(I0(), I1(), lo, lds);
      read_l(I0(), I0(), lo, lds);
      read_l(I0(), I1(), lo, lds);
    }
    int slot = 0;
    uint32_t fill = lds0 + kAhead * S::kSlotBytes;      // where step t + kAhead goes
    // One step.  Between any two MFMAs at most one fragment read or one load is
    // issued: all waves pass the barrier together, and a burst of them there
    // would leave the matrix units waiting.
    auto step = [&](int t, auto par) {
      using P = decltype(par);
      using Q = std::integral_constant<int, P::value ^ 1>;
      const unsigned char* cur = lds + slot * S::kSlotBytes;
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      const unsigned char* next = lds + slot * S::kSlotBytes;
      const bool live = t + kAhead < n;
      // Block row i: lo hi, hi lo, hi hi; `then(k)` after MFMA k.
      auto products = [&](int i, const u16x8 (&l)[2], auto&& then) {
#pragma unroll
        for (int k = 0; k < 3 * BO; ++k) {
          const int q = k / BO, j = k % BO;
          acc[i][j] = mma16(R[P::value][j][q == 0 ? 1 : 0], l[q == 1 ? 1 : 0], acc[i][j]);
          sched_fence();
          then(k);
          sched_fence();
        }
      };
      auto barrier = [&]() {
        wait_dma<kLoads * (kAhead - 2)>();
        step_barrier();
      };
      if constexpr (BA == 4) {
        products(0, L[0][0], [&](int k) {
          if (k < 2) read_l(I0(), I2(), k, cur);
        });
        products(1, L[0][1], [&](int k) {
          if (k < 2) read_l(I0(), I3(), k, cur);
        });
        barrier();
        products(2, L[0][2], [&](int k) {
          if (k == 0 || k == 2) dma(k / 2, fill, live);
          else if (k == 1 || k == 3) read_r(Q(), I0(), k >> 1, next);
          else read_r(Q(), I1(), k & 1, next);
        });
        products(3, L[0][3], [&](int k) {
          if (k == 0 || k == 2) dma(2 + k / 2, fill, live);
          else if (k == 1 || k == 3) read_l(I0(), I0(), k >> 1, next);
          else read_l(I0(), I1(), k & 1, next);
        });
      } else {
        // everything of the next step is read during this one
        barrier();
        products(0, L[P::value][0], [&](int k) {
          if (k < 2) read_r(Q(), I0(), k, next);
          else if (k < 4) read_r(Q(), I1(), k & 1, next);
          else dma(k - 4, fill, live);
        });
        products(1, L[P::value][1], [&](int k) {
          if (k < 2) read_l(Q(), I0(), k, next);
          else if (k < 4) read_l(Q(), I1(), k & 1, next);
          else dma(k - 2, fill, live);
        });
      }
      fill = fill == lds0 + (kSlots - 1) * S::kSlotBytes ? lds0 : fill + S::kSlotBytes;
    };
    int t = 0;
    for (; t + 1 < n; t += 2) {
      step(t, I0());
      step(t + 1, I1());
    }
    if (t < n) step(t, I0());
    wait_dma<0>();                               // nothing is left in flight into LDS
    if (n == p.steps) {
#pragma unroll
      for (int i = 0; i < BA; ++i) store_rows<S>(p, mat, ti, tj, i, acc[i], lds);
    } else {
      // part: four accumulators of every thread side by side
      float* o = p.parts + (int64_t)(2 * w + (first ? 0 : 1)) * S::kFloats + threadIdx.x * 4;
#pragma unroll
      for (int i = 0; i < BA; ++i)
#pragma unroll
        for (int j = 0; j < BO; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *(f32x4*)(o + ((i * BO + j) * 4 + g) * S::kNT * 4) =
                f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    }
    first = false;
    at += n;
  }
}

// The tiles that workgroups share: their parts in order, then as above.  One
// workgroup per first inner boundary of a tile and block row of its waves.
template <class S>
__global__ void __launch_bounds__(S::kNT) ortho_fixup_kernel(ProductArgs p) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int b = blockIdx.x + 1, i = blockIdx.y;
  const int64_t s = first_step(p, b), tile = s / p.steps, begin = tile * p.steps;
  if (s == begin || first_step(p, b - 1) > begin) return;
  f32x16 acc[S::kBO];
#pragma unroll
  for (int j = 0; j < S::kBO; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
  for (int w = b - 1; w < p.groups && first_step(p, w) < begin + p.steps; ++w) {
    const float* o = p.parts + (int64_t)(2 * w + (first_step(p, w) >= begin ? 0 : 1)) * S::kFloats +
                     threadIdx.x * 4 + (int64_t)i * S::kBO * 4 * S::kNT * 4;
#pragma unroll
    for (int j = 0; j < S::kBO; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 x = *(const f32x4*)(o + (j * 4 + g) * S::kNT * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][4 * g + k] += x[k];
      }
  }
  const int64_t mat = tile / p.tiles;
  int ti, tj;
  tile_of(p, (int)(tile - mat * p.tiles), &ti, &tj);
  store_rows<S>(p, mat, ti, tj, i, acc, lds);
}

// B += add A, plus `shift` on the diagonal: 8 elements of n matrices [mp, mp] a
// thread, hi and lo of both in one 16-byte load each.  Bound by memory (201 MB
// for 4096 x 4096), below that by its launch: five steps of 768 x 768 take 304 us
// with it and 292 with the completed square, of 1920 x 1920 655 and 625, of
// 4096 x 4096 3.95 and 3.83 ms.
__global__ void __launch_bounds__(256) ortho_add_kernel(Pair A, Pair B, int64_t n, int mp, float add,
                                                        float shift) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (e >= n * mp * mp) return;
  const int64_t row = e / mp;                       // of all matrices
  const int c = (int)(e - row * mp), diag = (int)(row % mp) - c;
  const int64_t at = row * A.ld + 2 * c - (c & 15);
  typedef _Float16 half8 __attribute__((ext_vector_type(8)));
  const half8 ah = *(const half8*)(A.p + at), al = *(const half8*)(A.p + at + 16);
  half8 bh = *(const half8*)(B.p + at), bl = *(const half8*)(B.p + at + 16);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = ((float)bh[k] + (float)bl[k]) + add * ((float)ah[k] + (float)al[k]) +
                    (k == diag ? shift : 0.f);
    bh[k] = (_Float16)x;
    bl[k] = (_Float16)(x - (float)bh[k]);
  }
  *(half8*)(B.p + at) = bh;
  *(half8*)(B.p + at + 16) = bl;
}

// ---------------------------------------------------------------------------
// Small matrices
// ---------------------------------------------------------------------------
// A matrix whose pairs fit into LDS next to its m x m product: the whole call
// in one workgroup of 8 waves (a launch per product costs more than the
// product).  X is kept with its smaller dimension first, A and then B in the
// same place; each wave computes 32 x 32 blocks in registers and they are
// stored after a barrier, in place: 64 x 32 20 us, 128 x 128 75 (latency of LDS
// reads and barriers; 182 for 64 x 32 with a launch per product).  Here B = b A + c A^2 and X <- a X + B X as
// they stand: reading back costs nothing in LDS, and a few large entries (a
// row, a number) do not average out what the shifted diagonals round off.
constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / 64;
constexpr int kSmallBlocks = 5;                   // blocks of X per wave, at most
constexpr int kSmallSquare = 2;                   // and of A
constexpr int kSmallLds = 156 * 1024;

// What the products' results are multiplied by, and the diagonal shifts.
struct StepFactors {
  float gram, gram_shift, square, square_shift, apply;
  float add_b, add_shift;                         // of the pass after the square, or 0
};
// The same for B = b A + c A^2 and X <- a X + B X.
struct AddFactors {
  float gram, add_b, square, add_x, apply;
};
struct SmallArgs {
  OrthoArgs a;
  int flip, m, k, mp, kp;                         // X: [m, k], padded to 32
  float pow_x;
  AddFactors f[kOrthoMaxSteps];
};

// One matrix in LDS: hi and lo planes, rows `ld` halves apart.
struct Planes {
  uint16_t *hi, *lo;
  int ld;
  __device__ __forceinline__ u16x8 inner(bool low, int m0, int k0) const {   // rows m0 .., k0 .. + 15
    const int lane = threadIdx.x & 63;
    return *(const u16x8*)((low ? lo : hi) + (m0 + (lane & 31)) * ld + k0 + 8 * (lane >> 5));
  }
  __device__ __forceinline__ u16x8 outer(bool low, int m0, int k0) const {   // columns m0 .., rows k0 ..
    const int lane = threadIdx.x & 63;
    const uint16_t* p = (low ? lo : hi) + (k0 + 8 * (lane >> 5) + ((lane & 15) >> 2)) * ld + m0 +
                        16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const u16x4 a = lds_read_tr16(p), b = lds_read_tr16(p + 4 * ld);
    u16x8 f;
    f.s0 = a.s0; f.s1 = a.s1; f.s2 = a.s2; f.s3 = a.s3;
    f.s4 = b.s0; f.s5 = b.s1; f.s6 = b.s2; f.s7 = b.s3;
    return f;
  }
  __device__ __forceinline__ void put(int r, int c, float v) const {
    const _Float16 h = (_Float16)v, l = (_Float16)(v - (float)h);
    hi[r * ld + c] = __builtin_bit_cast(uint16_t, h);
    lo[r * ld + c] = __builtin_bit_cast(uint16_t, l);
  }
  // old f0 + f1 acc for this lane's values of a block, in place
  __device__ __forceinline__ void update(int r0, int c0, float f0, float f1, const f32x16& acc) const {
    const int lane = threadIdx.x & 63, r = r0 + acc_col(lane);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int e = r * ld + c0 + acc_row(4 * g, lane);
      f16x4 h, l;
      if (f0 != 0.f) {
        h = *(const f16x4*)(hi + e);
        l = *(const f16x4*)(lo + e);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float old = f0 != 0.f ? f0 * ((float)h[k] + (float)l[k]) : 0.f;
        const float v = old + f1 * acc[4 * g + k];
        h[k] = (_Float16)v;
        l[k] = (_Float16)(v - (float)h[k]);
      }
      *(f16x4*)(hi + e) = h;
      *(f16x4*)(lo + e) = l;
    }
  }
};

__device__ __forceinline__ f32x16 zero16() {
  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  return acc;
}

// acc + block (r0, c0) of L R^T (fragments from `l` and `r`), K in steps of 16.
template <class FL, class FR>
__device__ __forceinline__ f32x16 small_block(int K, FL&& l, FR&& r, f32x16 acc = zero16()) {
#pragma unroll 2
  for (int k0 = 0; k0 < K; k0 += 16) {
    const u16x8 lh = l(false, k0), ll = l(true, k0), rh = r(false, k0), rl = r(true, k0);
    acc = mma16(rl, lh, acc);
    acc = mma16(rh, ll, acc);
    acc = mma16(rh, lh, acc);
  }
  return acc;
}

template <class E, bool MUON>
__global__ void __launch_bounds__(kSmallThreads) ortho_small_kernel(SmallArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ double red[kSmallWaves], scale;
  __shared__ int unit;
  const OrthoArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = p.m * p.k, C = (int)a.C;
  const int64_t base = (int64_t)blockIdx.x * len;
  const int ldx = p.kp + 8, lda = p.mp + 8;
  const Planes X{(uint16_t*)lds, (uint16_t*)lds + p.mp * ldx, ldx};
  uint16_t* ap = X.lo + p.mp * ldx;
  const Planes A{ap, ap + p.mp * lda, lda};
  double sq = 0.0;
  for (int i = tid; i < len; i += kSmallThreads) {
    const int64_t e = base + i;
    if constexpr (MUON) a.momentum[e] = a.beta * a.momentum[e] + a.grad[e];
    const float u = update_at<E, MUON>(a, e);
    sq += (double)u * (double)u;
  }
  for (int i = tid; i < p.mp * ldx; i += kSmallThreads) ((uint32_t*)lds)[i] = 0u;   // both planes
  sq = block_sum_f64(sq, red);
  if (tid == 0) scale = input_scale(a, sq, p.pow_x, &unit);
  __syncthreads();
  for (int i = tid; i < len; i += kSmallThreads) {
    const int r = i / C, c = i - r * C;
    const float v = (float)((double)update_at<E, MUON>(a, base + i) * scale);
    if (p.flip) X.put(c, r, v);
    else X.put(r, c, v);
  }
  const float inv = ldexpf(1.0f, -unit);
  const int mb = p.mp / 32, kb = p.kp / 32;
  for (int s = 0; s < a.steps; ++s) {
    const AddFactors f = p.f[s];
    __syncthreads();
    f32x16 acc[kSmallSquare];
    // f(q, r0, c0) for this wave's blocks of A
    auto squares = [&](auto&& g) {
#pragma unroll
      for (int q = 0; q < kSmallSquare; ++q) {
        const int n = wave + q * kSmallWaves;
        if (n < mb * mb) g(q, n / mb * 32, n % mb * 32);
      }
    };
    squares([&](int q, int r0, int c0) {                    // A
      acc[q] = small_block(p.kp, [&](bool low, int k) { return X.inner(low, r0, k); },
                           [&](bool low, int k) { return X.inner(low, c0, k); });
      A.update(r0, c0, 0.f, f.gram * inv * inv, acc[q]);
    });
    __syncthreads();
    squares([&](int q, int r0, int c0) {                    // B
      acc[q] = small_block(p.mp, [&](bool low, int k) { return A.inner(low, r0, k); },
                           [&](bool low, int k) { return A.inner(low, c0, k); });
    });
    __syncthreads();
    squares([&](int q, int r0, int c0) { A.update(r0, c0, f.add_b, f.square, acc[q]); });
    __syncthreads();
    auto block = [&](int n) {
      return small_block(p.mp, [&](bool low, int k) { return A.inner(low, n / kb * 32, k); },
                         [&](bool low, int k) { return X.outer(low, n % kb * 32, k); });
    };
    if (s + 1 < a.steps) {
      f32x16 x[kSmallBlocks];
#pragma unroll
      for (int q = 0; q < kSmallBlocks; ++q)
        if (wave + q * kSmallWaves < mb * kb) x[q] = block(wave + q * kSmallWaves);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kSmallBlocks; ++q) {
        const int n = wave + q * kSmallWaves;
        if (n < mb * kb) X.update(n / kb * 32, n % kb * 32, f.add_x, f.apply, x[q]);
      }
      continue;
    }
#pragma unroll 1
    for (int n = wave; n < mb * kb; n += kSmallWaves) {       // the result
      const f32x16 x = block(n);
      const int r = n / kb * 32 + acc_col(lane), c0 = n % kb * 32;
      if (r >= p.m) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = c0 + acc_row(j, lane);
        if (c >= p.k) continue;
        const int at = r * ldx + c;
        const float old = (float)__builtin_bit_cast(_Float16, X.hi[at]) +
                          (float)__builtin_bit_cast(_Float16, X.lo[at]);
        const float v = (f.add_x * old + f.apply * x[j]) * inv;
        const int64_t e = base + (p.flip ? c * C + r : r * C + c);
        if constexpr (MUON) {
          a.W[e] = a.decay * a.W[e] - a.size * v;
        } else {
          float one[1] = {v};
          store_f32<E, 1>((typename E::storage*)a.out + e, one);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Thin matrices
// ---------------------------------------------------------------------------
// m x k with m <= 96 and too long for one workgroup: two launches a step in
// place of four.  X is cut into strips of 128 columns, each kept as the image of
// its planes in LDS.  A workgroup takes a strip (or several) through X <- a X +
// B X and at once adds its X X^T to the next step's A, of which it leaves a part
// (the 32 x 32 blocks on and above the diagonal); one workgroup per matrix adds
// the parts in order and makes B = b A + c A^2.  Bound by the latency of its
// twelve launches' short chains (memory, LDS, barrier, store), 5 to 8 us each.
// Against the tiles of 128: 16 x 5120 65 us (250), 35 x 4850 105 (247), 5120 x 64
// 94 (257), 90 x 600 115 (164), 96 x 20000 297 (395), stacks of 256 64 x 1000 285
// (576), of 64 90 x 1000 216 (258).  With m = 128 it was no faster (128 x 5120
// 280 against 254: the parts of A, and one workgroup per compute unit).
constexpr int kThinCols = 128, kThinMost = 96;    // columns of a strip, rows of X at most
// blocks of X per wave
constexpr int kThinX = (kThinMost / 32 * (kThinCols / 32) + kSmallWaves - 1) / kSmallWaves;
constexpr int kThinLd = kThinCols + 8;

struct ThinArgs {
  OrthoArgs a;
  int flip, m, k, mp;             // X: [m, k], m padded to 32
  int strips, parts;              // strips, and workgroups that share them
  int nb;                         // norm partials per matrix
  const double* sq;
  float* unit;                    // [n]
  uint16_t* X;                    // [n][strips][hi, lo][mp][kThinCols]
  uint16_t* B;                    // [n][hi, lo][mp][mp]
  float* part;                    // [n][parts][blocks][32 * 32]
  float pow_x;
  AddFactors f;
};

__host__ __device__ constexpr int tri_blocks(int mb) { return mb * (mb + 1) / 2; }
// Block q on or above the diagonal, row by row.
__device__ __forceinline__ void tri_block(int q, int mb, int* r0, int* c0) {
  int r = 0;
  while (q >= mb - r) q -= mb - r++;
  *r0 = 32 * r;
  *c0 = 32 * (r + q);
}

// `rows` rows of `cols` halves between memory (contiguous, the lo plane after the
// hi plane) and planes in LDS, 16 bytes a lane.
template <bool STORE>
__device__ __forceinline__ void copy_planes(const Planes& x, uint16_t* g, int rows, int cols) {
  const int per = cols / 8, plane = rows * per;
  for (int i = threadIdx.x; i < 2 * plane; i += kSmallThreads) {
    const int j = i < plane ? i : i - plane, r = j / per, c = (j - r * per) * 8;
    u16x8* l = (u16x8*)((i < plane ? x.hi : x.lo) + r * x.ld + c);
    u16x8* m = (u16x8*)g + i;
    if constexpr (STORE) *m = *l;
    else *l = *m;
  }
}

enum ThinStage { kThinFirst = 0, kThinStep = 1, kThinLast = 2 };

template <class E, bool MUON, int STAGE>
__global__ void __launch_bounds__(kSmallThreads) ortho_strip_kernel(ThinArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ double scale;
  const OrthoArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int mp = p.mp, mb = mp / 32, kb = kThinCols / 32, C = (int)a.C;
  const int64_t n = blockIdx.y, base = n * p.m * p.k;
  const Planes X{(uint16_t*)lds, (uint16_t*)lds + mp * kThinLd, kThinLd};
  uint16_t* bp = X.lo + mp * kThinLd;
  const Planes B{bp, bp + mp * (mp + 8), mp + 8};
  if constexpr (STAGE == kThinFirst) {
    if (tid < 64) {
      double sq = 0.0;
      for (int i = tid; i < p.nb; i += 64) sq += p.sq[n * p.nb + i];
      sq = wave_sum_f64(sq);
      if (tid == 0) {
        int e;
        scale = input_scale(a, sq, p.pow_x, &e);
        if (blockIdx.x == 0) p.unit[n] = ldexpf(1.0f, -e);
      }
    }
  } else {
    copy_planes<false>(B, p.B + n * 2 * mp * mp, mp, mp);
  }
  f32x16 sums[kSmallSquare];
#pragma unroll
  for (int q = 0; q < kSmallSquare; ++q) sums[q] = zero16();
  const int s0 = (int)((int64_t)p.strips * blockIdx.x / p.parts);
  const int s1 = (int)((int64_t)p.strips * (blockIdx.x + 1) / p.parts);
  for (int strip = s0; strip < s1; ++strip) {
    uint16_t* image = p.X + (n * p.strips + strip) * (2 * mp * kThinCols);
    const int col0 = strip * kThinCols;
    __syncthreads();                              // the last strip is done with
    if constexpr (STAGE == kThinFirst) {
      for (int i = tid; i < mp * kThinCols; i += kSmallThreads) {
        // along the input's rows
        const int r = p.flip ? i % mp : i / kThinCols, c = p.flip ? i / mp : i % kThinCols;
        float v = 0.f;
        if (r < p.m && col0 + c < p.k) {
          const int64_t e = base + (p.flip ? (int64_t)(col0 + c) * C + r : (int64_t)r * C + col0 + c);
          v = (float)((double)update_at<E, MUON>(a, e) * scale);
        }
        X.put(r, c, v);
      }
      __syncthreads();
    } else {
      copy_planes<false>(X, image, mp, kThinCols);
      __syncthreads();
      f32x16 x[kThinX];
#pragma unroll
      for (int q = 0; q < kThinX; ++q) {
        const int i = wave + q * kSmallWaves;
        if (i < mb * kb)
          x[q] = small_block(mp, [&](bool low, int k) { return B.inner(low, i / kb * 32, k); },
                             [&](bool low, int k) { return X.outer(low, i % kb * 32, k); });
      }
      __syncthreads();
      if constexpr (STAGE == kThinStep) {
#pragma unroll
        for (int q = 0; q < kThinX; ++q) {
          const int i = wave + q * kSmallWaves;
          if (i < mb * kb) X.update(i / kb * 32, i % kb * 32, p.f.add_x, p.f.apply, x[q]);
        }
        __syncthreads();
      } else {
        const float inv = p.unit[n];
#pragma unroll
        for (int q = 0; q < kThinX; ++q) {
          const int i = wave + q * kSmallWaves;
          const int r = i / kb * 32 + acc_col(lane), c0 = i % kb * 32;
          if (i >= mb * kb || r >= p.m) continue;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int c = c0 + acc_row(j, lane);
            if (col0 + c >= p.k) continue;
            const int at = r * kThinLd + c;
            const float old = (float)__builtin_bit_cast(_Float16, X.hi[at]) +
                              (float)__builtin_bit_cast(_Float16, X.lo[at]);
            const float v = (p.f.add_x * old + p.f.apply * x[q][j]) * inv;
            const int64_t e = base + (p.flip ? (int64_t)(col0 + c) * C + r : (int64_t)r * C + col0 + c);
            if constexpr (MUON) {
              a.W[e] = a.decay * a.W[e] - a.size * v;
            } else {
              float one[1] = {v};
              store_f32<E, 1>((typename E::storage*)a.out + e, one);
            }
          }
        }
      }
    }
    if constexpr (STAGE != kThinLast) {
      copy_planes<true>(X, image, mp, kThinCols);
#pragma unroll
      for (int q = 0; q < kSmallSquare; ++q) {
        const int i = wave + q * kSmallWaves;
        if (i >= tri_blocks(mb)) continue;
        int r0, c0;
        tri_block(i, mb, &r0, &c0);
        sums[q] = small_block(kThinCols, [&](bool low, int k) { return X.inner(low, r0, k); },
                              [&](bool low, int k) { return X.inner(low, c0, k); }, sums[q]);
      }
    }
  }
  if constexpr (STAGE != kThinLast) {
    float* part = p.part + (n * p.parts + blockIdx.x) * (tri_blocks(mb) * 1024);
#pragma unroll
    for (int q = 0; q < kSmallSquare; ++q) {
      const int i = wave + q * kSmallWaves;
      if (i >= tri_blocks(mb)) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        ((f32x4*)part)[i * 256 + g * 64 + lane] =
            f32x4{sums[q][4 * g], sums[q][4 * g + 1], sums[q][4 * g + 2], sums[q][4 * g + 3]};
    }
  }
}

// B of one matrix from the strips' parts of A.
__global__ void __launch_bounds__(kSmallThreads) ortho_thin_square_kernel(ThinArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, wave = tid >> 6, mp = p.mp, mb = mp / 32, ld = mp + 8;
  const int64_t n = blockIdx.x;
  const Planes A{(uint16_t*)lds, (uint16_t*)lds + mp * ld, ld};
  const int values = tri_blocks(mb) * 256;        // four of each part
  const f32x4* part = (const f32x4*)p.part + n * p.parts * values;
  const float inv = p.unit[n], f = p.f.gram * inv * inv;
  for (int i = tid; i < values; i += kSmallThreads) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < p.parts; ++k) {
      const f32x4 v = part[(int64_t)k * values + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    int r0, c0;
    tri_block(i / 256, mb, &r0, &c0);
    const int lane = i & 63, r = r0 + acc_col(lane), c = c0 + acc_row(4 * (i >> 6 & 3), lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      A.put(r, c + e, f * sum[e]);
      if (r0 != c0) A.put(c + e, r, f * sum[e]);
    }
  }
  __syncthreads();
  f32x16 acc[kSmallSquare];
#pragma unroll
  for (int q = 0; q < kSmallSquare; ++q) {
    const int i = wave + q * kSmallWaves;
    if (i < mb * mb)
      acc[q] = small_block(mp, [&](bool low, int k) { return A.inner(low, i / mb * 32, k); },
                           [&](bool low, int k) { return A.inner(low, i % mb * 32, k); });
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSmallSquare; ++q) {
    const int i = wave + q * kSmallWaves;
    if (i < mb * mb) A.update(i / mb * 32, i % mb * 32, p.f.add_b, p.f.square, acc[q]);
  }
  __syncthreads();
  copy_planes<true>(A, p.B + n * 2 * mp * mp, mp, mp);
}

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
// The largest |a s + b s^3 + c s^5| over 0 <= s <= top.
double poly_bound(double a, double b, double c, double top) {
  auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
  double most = std::max(f(0.0), f(top));
  // a + 3 b q + 5 c q^2 = 0, q = s^2
  double q[2];
  int n = 0;
  if (c != 0.0) {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0.0)
      for (int k = 0; k < 2; ++k) q[n++] = (-3 * b + (k ? 1 : -1) * std::sqrt(d)) / (10 * c);
  } else if (b != 0.0) {
    q[n++] = -a / (3 * b);
  }
  for (int k = 0; k < n; ++k)
    if (q[k] > 0.0 && q[k] < top * top) most = std::max(most, f(std::sqrt(q[k])));
  return most;
}

// The largest |x + y q + z q^2| over 0 <= q <= top.
double quad_bound(double x, double y, double z, double top) {
  auto f = [&](double q) { return std::fabs(x + q * (y + q * z)); };
  double most = std::max(f(0.0), f(top));
  if (z != 0.0) {
    const double q = -y / (2 * z);
    if (q > 0.0 && q < top) most = std::max(most, f(q));
  }
  return most;
}

constexpr double kRoom = 1.01;   // rounding may pass a bound a little

// The power of two that brings values up to `bound` just below 2^15.
int scale_of(double bound) {
  if (!(bound > 0.0)) return 0;
  return std::min(24, (int)std::floor(std::log2(32768.0 / bound)));
}

struct Plan {
  bool flip;                   // R > C
  int tile;
  int64_t m, Rp, Cp, mp;       // padded
  int nb;                      // norm workgroups per matrix
  int64_t groups_sym, groups_full, groups_square;
  int small;                   // LDS bytes of the one-workgroup kernel, or 0
  int strips, thin_parts;      // of a thin matrix, or 0
  size_t x, a, part, unit, parts, total;   // bytes of one X pair, one A pair; offsets
};

int64_t up(int64_t v, int64_t t) { return (v + t - 1) / t * t; }

// Microseconds of a product on `groups` workgroups, measured: a step of a
// 128 x 128 tile takes 0.37 with the compute unit to itself and 0.75 next to
// another, of a 256 x 256 tile 1.05; shared tiles cost a launch and their
// parts' way through memory.
double product_us(int64_t tiles, int64_t steps, int tile, int64_t groups) {
  const int64_t cus = device_cus();
  if (groups != tiles)
    return (double)(tiles * steps) / groups * (groups <= cus ? 0.37 : 0.75) + 5.0 + 0.06 * groups;
  if (tile == 256) return (double)((tiles + cus - 1) / cus * steps) * 1.05;
  if (tiles <= cus) return steps * 0.37;
  return (double)((tiles + 2 * cus - 1) / (2 * cus) * steps) * 0.75;
}

// Workgroups for `tiles` tiles of `steps` steps: one per tile, or, where there
// are too few tiles for the compute units, several that share each (at least 8
// steps each): one 768 x 768 matrix takes 287 us with three to a tile, 355
// whole; twelve of them 528 whole, 586 with two to a tile.  Tiles of 256 are
// taken where there are enough of them (4096 x 4096: 3.87 ms, 4.05 with 128;
// 3000 x 3000: 2.50 against 2.17), and never shared: that was slower even with
// a fifth of the chip idle (5120 x 5120 7.8 ms whole, 8.5 shared; the clock
// rises when units idle).
int64_t groups_of(int64_t tiles, int64_t steps, int tile) {
  int64_t best = tiles;
  if (tile == 256) return best;
  for (int64_t share = 2; share * 8 <= steps && tiles * share <= 2 * device_cus(); ++share)
    if (product_us(tiles, steps, tile, tiles * share) < product_us(tiles, steps, tile, best))
      best = tiles * share;
  return best;
}

int64_t sym_tiles(int64_t mt) { return mt * (mt + 1) / 2; }

void plan_tiles(Plan& p, const OrthoArgs& a, int tile) {
  p.tile = tile;
  p.Rp = up(a.R, tile);
  p.Cp = up(a.C, tile);
  p.mp = up(p.m, tile);
  const int64_t mt = p.mp / tile, k = (p.flip ? p.Rp : p.Cp) / 16;
  p.groups_sym = groups_of(a.n * sym_tiles(mt), k, tile);
  p.groups_square = groups_of(a.n * sym_tiles(mt), p.mp / 16, tile);
  p.groups_full = groups_of(a.n * (p.Rp / tile) * (p.Cp / tile), p.mp / 16, tile);
}

// Time of an iteration.
double plan_cost(const Plan& p, const OrthoArgs& a) {
  const int64_t mt = p.mp / p.tile, k = (p.flip ? p.Rp : p.Cp) / 16;
  return product_us(a.n * sym_tiles(mt), k, p.tile, p.groups_sym) +
         product_us(a.n * sym_tiles(mt), p.mp / 16, p.tile, p.groups_square) +
         product_us(a.n * (p.Rp / p.tile) * (p.Cp / p.tile), p.mp / 16, p.tile, p.groups_full);
}

// The small kernel's LDS for X [mp, kp] (0: does not fit).
int small_lds(int64_t mp, int64_t kp) {
  if (mp > 128 || mp / 32 * (kp / 32) > kSmallWaves * kSmallBlocks) return 0;
  const int64_t bytes = 4 * mp * (kp + 8) + 4 * mp * (mp + 8);
  return bytes <= kSmallLds ? (int)bytes : 0;
}

// Workgroups that share a thin matrix's strips: enough for two per compute
// unit over the stack, and few enough that the one workgroup which adds their
// parts does not take longer than the strips (192 blocks of 4 KB).
int thin_parts(int64_t n, int strips, int blocks) {
  const int64_t want = std::max<int64_t>(1, 2 * device_cus() / n);
  return (int)std::min<int64_t>({strips, want, std::max(16, 192 / blocks), 64});
}

Plan plan_of(const OrthoArgs& a) {
  Plan p{};
  p.flip = a.R > a.C;
  p.m = std::min(a.R, a.C);
  p.small = small_lds(up(p.m, 32), up(std::max(a.R, a.C), 32));
  if (p.small != 0) return p;
  p.nb = (int)std::min<int64_t>(kSumBlocks, (a.R * a.C + 4095) / 4096);
  if (p.m <= kThinMost) {
    p.mp = up(p.m, 32);
    p.strips = (int)((std::max(a.R, a.C) + kThinCols - 1) / kThinCols);
    const int blocks = tri_blocks((int)(p.mp / 32));
    p.thin_parts = thin_parts(a.n, p.strips, blocks);
    p.x = (size_t)a.n * p.strips * (size_t)p.mp * kThinCols * 4;
    p.a = (size_t)(a.n * p.mp * p.mp) * 4;
    p.part = p.x + p.a;
    p.unit = p.part + (size_t)a.n * p.nb * sizeof(double);
    p.parts = (size_t)up((int64_t)(p.unit + (size_t)a.n * sizeof(float)), 256);
    p.total = p.parts + (size_t)a.n * p.thin_parts * blocks * 1024 * sizeof(float);
    return p;
  }
  if (a.tile != 0) {
    plan_tiles(p, a, a.tile);
  } else {
    plan_tiles(p, a, 256);
    const double large = plan_cost(p, a);
    plan_tiles(p, a, 128);
    if (large < plan_cost(p, a)) plan_tiles(p, a, 256);
  }
  p.x = (size_t)(a.n * p.Rp * p.Cp) * 4;
  p.a = (size_t)(a.n * p.mp * p.mp) * 4;
  p.part = 2 * p.x + 2 * p.a;
  p.unit = p.part + (size_t)a.n * p.nb * sizeof(double);
  p.parts = (size_t)up((int64_t)(p.unit + (size_t)a.n * sizeof(float)), 256);
  const int64_t mt = p.mp / p.tile, full = (p.Rp / p.tile) * (p.Cp / p.tile);
  int64_t shared = 0;          // the most workgroups of a product that shares tiles
  if (p.groups_sym != a.n * sym_tiles(mt)) shared = std::max<int64_t>(shared, p.groups_sym);
  if (p.groups_square != a.n * sym_tiles(mt)) shared = std::max<int64_t>(shared, p.groups_square);
  if (p.groups_full != a.n * full) shared = std::max<int64_t>(shared, p.groups_full);
  p.total = p.parts + (size_t)(2 * shared) * p.tile * p.tile * sizeof(float);
  return p;
}

template <class S, bool KI>
hipError_t launch_product_k(const ProductArgs& p, int64_t tiles, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)ortho_product_kernel<S, KI>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (once != hipSuccess) return once;
  hipLaunchKernelGGL((ortho_product_kernel<S, KI>), dim3((unsigned)p.groups), dim3(S::kNT), S::kLds, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.groups == tiles) return e;
  if constexpr (S::kTile == 128)
    hipLaunchKernelGGL((ortho_fixup_kernel<S>), dim3((unsigned)(p.groups - 1), S::kBA), dim3(S::kNT),
                       stage_bytes<S::kTile>(), s, p);
  return hipGetLastError();
}

template <class S>
hipError_t launch_product_s(const ProductArgs& p, bool ki, int64_t tiles, hipStream_t s) {
  return ki ? launch_product_k<S, true>(p, tiles, s) : launch_product_k<S, false>(p, tiles, s);
}

hipError_t launch_product(ProductArgs p, int tile, bool ki, int64_t n, int64_t groups,
                          hipStream_t s) {
  p.tiles = p.sym ? p.mt * (p.mt + 1) / 2 : p.mt * p.nt;
  const int64_t tiles = p.tiles * n;
  p.total = tiles * p.steps;
  p.groups = (int)groups;
  if (tile == 256) return launch_product_s<Shape<256, 8, 5>>(p, ki, tiles, s);
  if (groups <= device_cus()) return launch_product_s<Shape<128, 4, 10>>(p, ki, tiles, s);
  return launch_product_s<Shape<128, 4, 5>>(p, ki, tiles, s);
}

template <class E, bool MUON>
hipError_t launch_norm(const OrthoArgs& a, const Plan& p, double* part, hipStream_t s) {
  const dim3 grid((unsigned)p.nb, (unsigned)a.n);
  if (a.R * a.C % 4 == 0) hipLaunchKernelGGL((ortho_norm_kernel<E, MUON, 4>), grid, dim3(256), 0, s, a, part);
  else hipLaunchKernelGGL((ortho_norm_kernel<E, MUON, 1>), grid, dim3(256), 0, s, a, part);
  return hipGetLastError();
}

template <class E, bool MUON>
hipError_t launch_input(const OrthoArgs& a, const Plan& p, double* part, float* unit, Pair X,
                        float pow_x, hipStream_t s) {
  const hipError_t e = launch_norm<E, MUON>(a, p, part, s);
  if (e != hipSuccess) return e;
  const dim3 blocks((unsigned)std::min<int64_t>(8192, (p.Rp * p.Cp / 4 + 1023) / 1024), (unsigned)a.n);
  if (a.C % 4 == 0)
    hipLaunchKernelGGL((ortho_split_kernel<E, MUON, 4>), blocks, dim3(256), 0, s, a, (const double*)part,
                       p.nb, X, (int)p.Rp, (int)p.Cp, pow_x, unit);
  else
    hipLaunchKernelGGL((ortho_split_kernel<E, MUON, 1>), blocks, dim3(256), 0, s, a, (const double*)part,
                       p.nb, X, (int)p.Rp, (int)p.Cp, pow_x, unit);
  return hipGetLastError();
}

}  // namespace

bool ortho_coeffs_ok(const OrthoArgs& a) {
  double top = 1.0;
  for (int k = 0; k < a.steps; ++k) {
    top = kRoom * poly_bound(a.a, a.b, a.c, top);
    if (!(top <= 4.0)) return false;
  }
  return true;
}

size_t ortho_workspace_bytes(const OrthoArgs& a) { return plan_of(a).total; }

namespace {

// Whether the square is completed.  A' is rounded at the shift's size, 2^-23
// |b / 2c|, which B takes times b; in b A + c A^2 the rounding of A, whose
// eigenvalues are at most about 1, stands there instead.  So the shift may be
// little more than that (the limit of 3/2 has (2, -1.5, 0.5) at it), and what
// the diagonal takes back, b^2 / 4c, no larger than a.  Error against float64
// after 5 steps of a 160 x 200 matrix (these roundings in numpy), completed and
// not: (3.4445, -4.775, 2.0315) 1.3e-6 and 1.4e-6 (plain float32 products
// 1.6e-6), (2, -1.5, 0.5) 6e-7 and 6e-7 (2.3e-7), (1.5, -0.5, 0.01) 7.5e-6 and
// 5.4e-7 (9.3e-8), (1.5, -0.5, 1e-6) 6.0e-3 and 5.4e-7 (9.4e-8).
bool completed_square(const OrthoArgs& a) {
  return std::fabs(a.b) <= 3 * std::fabs(a.c) && a.b * a.b <= 4 * std::fabs(a.a * a.c);
}

// The factors of a step whose X is kept times 2^sx with singular values up to
// *top; *top and the power of the next X come back.  A' and B are kept times
// the powers that their largest values allow.
StepFactors step_factors(const OrthoArgs& a, double* top, int* sx, bool last) {
  const double most = *top * *top;                // of A's eigenvalues
  const bool square = a.c != 0.0, completed = square && completed_square(a);
  const double shift = completed ? a.b / (2 * a.c) : 0.0;
  int sb = scale_of(kRoom * quad_bound(a.a, a.b, a.c, most));
  if (square && !completed) sb = std::min(sb, scale_of(kRoom * std::fabs(a.c) * most * most));
  const int sa = square ? scale_of(kRoom * quad_bound(shift, 1.0, 0.0, most)) : sb;
  *top = kRoom * poly_bound(a.a, a.b, a.c, *top);
  const int next = last ? 0 : scale_of(kRoom * *top);
  StepFactors f{};
  f.gram = (float)((square ? 1.0 : a.b) * std::ldexp(1.0, sa - 2 * *sx));
  f.gram_shift = (float)((square ? shift : a.a) * std::ldexp(1.0, sa));
  f.square = (float)(a.c * std::ldexp(1.0, sb - 2 * sa));
  if (completed) {
    // from the shift as it was rounded, so that the two cancel in full
    const double rounded = std::ldexp((double)f.gram_shift, -sa);
    f.square_shift = (float)((a.a - a.c * rounded * rounded) * std::ldexp(1.0, sb));
  } else if (square) {
    f.add_b = (float)(a.b * std::ldexp(1.0, sb - sa));
    f.add_shift = (float)(a.a * std::ldexp(1.0, sb));
  }
  f.apply = (float)std::ldexp(1.0, next - sb - *sx);
  *sx = next;
  return f;
}

AddFactors add_factors(const OrthoArgs& a, double* top, int* sx, bool last) {
  const double most = *top * *top;
  const int sa = scale_of(kRoom * most), sb = scale_of(kRoom * quad_bound(0.0, a.b, a.c, most));
  *top = kRoom * poly_bound(a.a, a.b, a.c, *top);
  const int next = last ? 0 : scale_of(kRoom * *top);
  AddFactors f;
  f.gram = (float)std::ldexp(1.0, sa - 2 * *sx);
  f.add_b = (float)(a.b * std::ldexp(1.0, sb - sa));
  f.square = (float)(a.c * std::ldexp(1.0, sb - 2 * sa));
  f.add_x = (float)(a.a * std::ldexp(1.0, next - *sx));
  f.apply = (float)std::ldexp(1.0, next - sb - *sx);
  *sx = next;
  return f;
}

template <class E, bool MUON>
hipError_t launch_small(const SmallArgs& q, int lds, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)ortho_small_kernel<E, MUON>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
  if (once != hipSuccess) return once;
  hipLaunchKernelGGL((ortho_small_kernel<E, MUON>), dim3((unsigned)q.a.n), dim3(kSmallThreads), lds, s, q);
  return hipGetLastError();
}

template <class E, bool MUON, int STAGE>
hipError_t launch_strips(const ThinArgs& q, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)ortho_strip_kernel<E, MUON, STAGE>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
  if (once != hipSuccess) return once;
  const int lds = 4 * q.mp * kThinLd + 4 * q.mp * (q.mp + 8);
  hipLaunchKernelGGL((ortho_strip_kernel<E, MUON, STAGE>), dim3((unsigned)q.parts, (unsigned)q.a.n),
                     dim3(kSmallThreads), lds, s, q);
  return hipGetLastError();
}

template <class E, bool MUON>
hipError_t launch_thin(const OrthoArgs& a, const Plan& p, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)ortho_thin_square_kernel,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
  if (once != hipSuccess) return once;
  char* ws = (char*)a.ws;
  double top = 1.0;
  int sx = scale_of(top * kRoom);
  ThinArgs q{};
  q.a = a;
  q.flip = p.flip ? 1 : 0;
  q.m = (int)p.m;
  q.k = (int)std::max(a.R, a.C);
  q.mp = (int)p.mp;
  q.strips = p.strips;
  q.parts = p.thin_parts;
  q.nb = p.nb;
  q.sq = (const double*)(ws + p.part);
  q.unit = (float*)(ws + p.unit);
  q.X = (uint16_t*)ws;
  q.B = (uint16_t*)(ws + p.x);
  q.part = (float*)(ws + p.parts);
  q.pow_x = std::ldexp(1.f, sx);
  hipError_t e = launch_norm<E, MUON>(a, p, (double*)(ws + p.part), s);
  if (e == hipSuccess) e = launch_strips<E, MUON, kThinFirst>(q, s);
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    q.f = add_factors(a, &top, &sx, k + 1 == a.steps);
    hipLaunchKernelGGL(ortho_thin_square_kernel, dim3((unsigned)a.n), dim3(kSmallThreads),
                       4 * q.mp * (q.mp + 8), s, q);
    if ((e = hipGetLastError()) != hipSuccess) break;
    e = k + 1 < a.steps ? launch_strips<E, MUON, kThinStep>(q, s) : launch_strips<E, MUON, kThinLast>(q, s);
  }
  return e;
}

}  // namespace

hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s) {
  const Plan p = plan_of(a);
  double top = 1.0;
  int sx = scale_of(top * kRoom);
  if (p.small != 0) {
    SmallArgs q{};
    q.a = a;
    q.flip = p.flip ? 1 : 0;
    q.m = (int)p.m;
    q.k = (int)std::max(a.R, a.C);
    q.mp = (int)up(q.m, 32);
    q.kp = (int)up(q.k, 32);
    q.pow_x = std::ldexp(1.f, sx);
    for (int k = 0; k < a.steps; ++k) q.f[k] = add_factors(a, &top, &sx, k + 1 == a.steps);
    timing_begin("ortho_small", s);
    const hipError_t e = a.W != nullptr       ? launch_small<F32, true>(q, p.small, s)
                         : a.dtype == kBF16 ? launch_small<BF16, false>(q, p.small, s)
                                            : launch_small<F32, false>(q, p.small, s);
    timing_end("ortho_small", s);
    return e;
  }
  if (p.strips != 0) {
    timing_begin("ortho_thin", s);
    const hipError_t e = a.W != nullptr       ? launch_thin<F32, true>(a, p, s)
                         : a.dtype == kBF16 ? launch_thin<BF16, false>(a, p, s)
                                            : launch_thin<F32, false>(a, p, s);
    timing_end("ortho_thin", s);
    return e;
  }
  char* ws = (char*)a.ws;
  auto pair = [&](size_t off, int64_t rows, int64_t cols) {
    return Pair{(uint16_t*)(ws + off), 2 * cols, 2 * rows * cols};
  };
  const Pair X[2] = {pair(0, p.Rp, p.Cp), pair(p.x, p.Rp, p.Cp)};
  const Pair A = pair(2 * p.x, p.mp, p.mp), B = pair(2 * p.x + p.a, p.mp, p.mp);
  double* part = (double*)(ws + p.part);
  float* unit = (float*)(ws + p.unit);
  timing_begin("ortho_input", s);
  hipError_t e;
  if (a.W != nullptr) e = launch_input<F32, true>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  else if (a.dtype == kBF16) e = launch_input<BF16, false>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  else e = launch_input<F32, false>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  timing_end("ortho_input", s);
  const int mt = (int)(p.mp / p.tile);
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    const Pair& Xk = X[k & 1];
    const bool last = k + 1 == a.steps;
    const StepFactors f = step_factors(a, &top, &sx, last);
    ProductArgs q{};
    q.unit = unit;
    q.parts = (float*)(ws + p.parts);
    // A' from X X^T (R <= C: K-inner) or X^T X (K-outer)
    q.L = q.R = Xk;
    q.out = A;
    q.steps = (int)((p.flip ? p.Rp : p.Cp) / 16);
    q.mt = q.nt = mt;
    q.sym = 1;
    q.mode = kStore;
    q.units = 2;
    q.f = f.gram;
    q.shift = f.gram_shift;
    timing_begin("ortho_gram", s);
    e = launch_product(q, p.tile, !p.flip, a.n, p.groups_sym, s);
    timing_end("ortho_gram", s);
    if (e != hipSuccess) break;
    const bool square = a.c != 0.0;
    if (square) {
      q.L = q.R = A;
      q.out = B;
      q.steps = (int)(p.mp / 16);
      q.units = 0;
      q.f = f.square;
      q.shift = f.square_shift;
      timing_begin("ortho_square", s);
      e = launch_product(q, p.tile, !p.flip, a.n, p.groups_square, s);
      timing_end("ortho_square", s);
      if (e != hipSuccess) break;
      if (!completed_square(a)) {
        const int64_t threads = a.n * p.mp * p.mp / 8;
        timing_begin("ortho_add", s);
        hipLaunchKernelGGL(ortho_add_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, A, B,
                           a.n, (int)p.mp, f.add_b, f.add_shift);
        timing_end("ortho_add", s);
        if ((e = hipGetLastError()) != hipSuccess) break;
      }
    }
    // X <- B X (K-outer) or X B (K-inner)
    q.L = p.flip ? Xk : square ? B : A;
    q.R = p.flip ? (square ? B : A) : Xk;
    q.out = X[(k + 1) & 1];
    q.steps = (int)(p.mp / 16);
    q.mt = (int)(p.Rp / p.tile);
    q.nt = (int)(p.Cp / p.tile);
    q.sym = 0;
    q.mode = last ? kFinal : kStore;
    q.units = last ? 1 : 0;
    q.f = f.apply;
    q.rows = a.R;
    q.cols = a.C;
    q.dst = a.W != nullptr ? (void*)a.W : a.out;
    q.dtype = a.dtype;
    q.muon = a.W != nullptr ? 1 : 0;
    q.decay = a.decay;
    q.size = a.size;
    timing_begin("ortho_apply", s);
    e = launch_product(q, p.tile, p.flip, a.n, p.groups_full, s);
    timing_end("ortho_apply", s);
  }
  return e;
}

}  // namespace dpf
