// Orthogonalised update by Newton-Schulz products.  For a matrix U [R, C]:
//
//   X_0 = U / max(||U||_F, eps)
//   X <- a X + (b A + c A^2) X,  A = X X^T      (R <= C; else X (b A + c A^2), A = X^T X)
//
// `steps` times: each singular value s of X goes to a s + b s^3 + c s^5, which
// the coefficients drive towards 1, and the singular vectors stay.  The
// optimizer step forms U from the gradient and the momentum, and subtracts the
// result from the weight.
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
// A and B = b A + c A^2 are symmetric: only the tiles on and above the
// diagonal are computed, and stored twice.
//
// Layouts.  X stays as U is stored.  With R <= C the products contract X's
// rows (K-inner operands) for A, and B X contracts over rows of X (K-outer
// operands, B read as its own transpose).  With R > C it is the other way
// round, so two kernels serve both shapes and nothing is ever transposed.
#include <algorithm>
#include <cmath>

#include "lm.hpp"
#include "tiles.hpp"

namespace dpf {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kNT = 256;            // 4 waves, 2 x 2
constexpr int kKT = 32;             // K per LDS step
constexpr int kPad = 8;             // LDS row padding (halves)
constexpr int kSumBlocks = 256;     // most workgroups of one matrix's norm

__device__ __forceinline__ f32x16 mma16(const u16x8& a, const u16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two half planes of a matrix, rows ld elements apart; the next matrix of the
// stack starts `next` elements further.
struct Pair {
  uint16_t *hi, *lo;
  int64_t ld, next;
  __device__ __forceinline__ Pair at(int64_t k) const { return Pair{hi + k * next, lo + k * next, ld, next}; }
};

__device__ __forceinline__ void store_pair(const Pair& p, int64_t e, const float (&v)[4]) {
  f16x4 h, l;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = (_Float16)v[k];
    l[k] = (_Float16)(v[k] - (float)h[k]);
  }
  *(f16x4*)(p.hi + e) = h;
  *(f16x4*)(p.lo + e) = l;
}

__device__ __forceinline__ void load_pair(const Pair& p, int64_t e, float (&v)[4]) {
  const f16x4 h = *(const f16x4*)(p.hi + e), l = *(const f16x4*)(p.lo + e);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = (float)h[k] + (float)l[k];
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

template <class E, bool MUON>
__global__ void __launch_bounds__(256) ortho_norm_kernel(OrthoArgs a, double* part) {
  __shared__ double red[4];
  const int64_t len = a.R * a.C, base = (int64_t)blockIdx.y * len;
  double sq = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < len; i += (int64_t)gridDim.x * 256) {
    const int64_t e = base + i;
    if constexpr (MUON) a.momentum[e] = a.beta * a.momentum[e] + a.grad[e];
    const float u = update_at<E, MUON>(a, e);
    sq += (double)u * (double)u;
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
template <class E, bool MUON>
__global__ void __launch_bounds__(256) ortho_split_kernel(OrthoArgs a, const double* part, int nb,
                                                          Pair X, int64_t Rp, float pow_x,
                                                          float* unit) {
  __shared__ double scale;
  if (threadIdx.x < 64) {
    double sq = 0.0;
    for (int k = threadIdx.x; k < nb; k += 64) sq += part[(int64_t)blockIdx.y * nb + k];
    sq = wave_sum_f64(sq);
    if (threadIdx.x == 0) {
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
      scale = norm < __builtin_huge_val()
                  ? ldexp((double)pow_x, e) / (norm > a.eps ? norm : a.eps)
                  : __builtin_nan("");
      if (blockIdx.x == 0) unit[blockIdx.y] = ldexpf(1.0f, -e);
    }
  }
  __syncthreads();
  const double f = scale;
  const Pair x = X.at(blockIdx.y);
  const int64_t total = Rp * X.ld / 4, base = (int64_t)blockIdx.y * a.R * a.C;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    const int64_t r = 4 * q / X.ld, c = 4 * q - r * X.ld;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = r < a.R && c + k < a.C
                 ? (float)((double)update_at<E, MUON>(a, base + r * a.C + c + k) * f)
                 : 0.f;
    store_pair(x, 4 * q, v);
  }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// D[M][N] = sum_k L(M, k) R(N, k); then, by mode, with f0, f1 powers of two
// times coefficients:
enum Mode {
  kStore = 0,    // out = f1 D
  kAddStore = 1, // out = f0 add + f1 D
  kFinal = 2     // result = f0 add + f1 D, to the caller's matrix
};
struct ProductArgs {
  Pair L, R, add, out;
  int64_t K;
  int mt, nt;             // tiles of M and N (symmetric: mt == nt)
  int sym, mode, dtype;
  float f0, f1;
  const float* unit;      // [n] 1 / unit of each matrix's X
  int units;              // power of it that scales f1 D (kStore) or the result (kFinal)
  // kFinal
  int64_t rows, cols;
  void* dst;              // [rows, cols] of dtype, or the weight (float32)
  int muon;
  float decay, size;
};

// Chunk q of an operand's TILE x kKT slice, in global memory and in LDS.
template <int TILE, bool KI>
struct Slice {
  static constexpr int kCpr = (KI ? kKT : TILE) / 8;
  static constexpr int kLd = (KI ? kKT : TILE) + kPad;
  static constexpr int kPlane = (KI ? TILE : kKT) * kLd;     // halves
  static constexpr int kN = TILE * kKT / 8 / kNT;
  u32x4 h[kN], l[kN];
  __device__ __forceinline__ void load(const Pair& p, int64_t m0, int64_t k0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int q = threadIdx.x + kNT * i, row = q / kCpr, cc = q % kCpr;
      const int64_t e = KI ? (m0 + row) * p.ld + k0 + cc * 8 : (k0 + row) * p.ld + m0 + cc * 8;
      h[i] = *(const u32x4*)(p.hi + e);
      l[i] = *(const u32x4*)(p.lo + e);
    }
  }
  __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int q = threadIdx.x + kNT * i, row = q / kCpr, cc = q % kCpr;
      *(u32x4*)(lds + row * kLd + cc * 8) = h[i];
      *(u32x4*)(lds + kPlane + row * kLd + cc * 8) = l[i];
    }
  }
  static __device__ __forceinline__ u16x8 frag(const uint16_t* plane, int m0, int ks) {
    if constexpr (KI) return frag_kinner<BF16, kLd>(plane, m0, ks);
    else return frag_kouter<BF16, kLd>(plane, m0, ks);
  }
};

template <int TILE, bool KI>
constexpr int product_lds() { return 2 * 4 * Slice<TILE, KI>::kPlane * 2; }

template <int TILE, bool KI>
__global__ void __launch_bounds__(kNT) ortho_product_kernel(ProductArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  using S = Slice<TILE, KI>;
  constexpr int NB = TILE / 64;
  const int tiles = p.sym ? p.mt * (p.mt + 1) / 2 : p.mt * p.nt;
  const int64_t mat = blockIdx.x / tiles;
  int t = blockIdx.x % tiles, ti, tj;
  if (p.sym) {           // row by row of the upper triangle
    ti = 0;
    while (t >= p.mt - ti) { t -= p.mt - ti; ++ti; }
    tj = ti + t;
  } else {
    ti = t / p.nt;
    tj = t % p.nt;
  }
  const Pair Lp = p.L.at(mat), Rp = p.R.at(mat);
  const int64_t m0 = (int64_t)ti * TILE, n0 = (int64_t)tj * TILE;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, wm = wave >> 1, wn = wave & 1;
  f32x16 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  S sl, sr;
  sl.load(Lp, m0, 0);
  sr.load(Rp, n0, 0);
  sl.store(lds);
  sr.store(lds + 2 * S::kPlane);
  __syncthreads();
  const int64_t nk = p.K / kKT;
  for (int64_t kk = 0; kk < nk; ++kk) {
    const bool more = kk + 1 < nk;
    if (more) {
      sl.load(Lp, m0, (kk + 1) * kKT);
      sr.load(Rp, n0, (kk + 1) * kKT);
    }
    const uint16_t* buf = lds + (kk & 1) * 4 * S::kPlane;
#pragma unroll
    for (int ks = 0; ks < kKT / 16; ++ks) {
      u16x8 lh[NB], ll[NB], rh[NB], rl[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        lh[i] = S::frag(buf, (wm * NB + i) * 32, ks);
        ll[i] = S::frag(buf + S::kPlane, (wm * NB + i) * 32, ks);
        rh[i] = S::frag(buf + 2 * S::kPlane, (wn * NB + i) * 32, ks);
        rl[i] = S::frag(buf + 3 * S::kPlane, (wn * NB + i) * 32, ks);
      }
      // the N side is the MFMA's row operand: a lane's accumulators are then
      // runs of four columns of one row of D
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          acc[i][j] = mma16(rl[j], lh[i], acc[i][j]);
          acc[i][j] = mma16(rh[j], ll[i], acc[i][j]);
          acc[i][j] = mma16(rh[j], lh[i], acc[i][j]);
        }
    }
    if (!more) break;
    uint16_t* next = lds + ((kk + 1) & 1) * 4 * S::kPlane;
    sl.store(next);
    sr.store(next + 2 * S::kPlane);
    __syncthreads();
  }
  const Pair add = p.add.at(mat), out = p.out.at(mat);
  float f0 = p.f0, f1 = p.f1;
  for (int k = 0; k < p.units; ++k) { f0 *= p.unit[mat]; f1 *= p.unit[mat]; }
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t r = m0 + (wm * NB + i) * 32 + acc_col(lane);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = n0 + (wn * NB + j) * 32 + acc_row(4 * g, lane);
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = f1 * acc[i][j][4 * g + k];
        if (p.mode != kStore) {
          float w[4];
          load_pair(add, r * add.ld + c, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] += f0 * w[k];
        }
        if (p.mode != kFinal) {
          store_pair(out, r * out.ld + c, v);
          if (p.sym && ti != tj) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const _Float16 h = (_Float16)v[k], l = (_Float16)(v[k] - (float)h);
              out.hi[(c + k) * out.ld + r] = __builtin_bit_cast(uint16_t, h);
              out.lo[(c + k) * out.ld + r] = __builtin_bit_cast(uint16_t, l);
            }
          }
          continue;
        }
        if (r >= p.rows) continue;
        const int64_t e = (mat * p.rows + r) * p.cols + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c + k >= p.cols) break;
          if (p.muon) {
            float* w = (float*)p.dst + e + k;
            *w = p.decay * *w - p.size * v[k];
          } else if (p.dtype == kBF16) {
            ((uint16_t*)p.dst)[e + k] = f32_to_bf16_rne(v[k]);
          } else {
            ((float*)p.dst)[e + k] = v[k];
          }
        }
      }
    }
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

// The largest |b q + c q^2| over 0 <= q <= top.
double quad_bound(double b, double c, double top) {
  auto f = [&](double q) { return std::fabs(q * (b + q * c)); };
  double most = f(top);
  if (c != 0.0) {
    const double q = -b / (2 * c);
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
  size_t x, a, part, unit, total;   // bytes of one X pair, one A pair; offsets
};

int64_t up(int64_t v, int64_t t) { return (v + t - 1) / t * t; }

Plan plan_of(const OrthoArgs& a) {
  Plan p;
  p.flip = a.R > a.C;
  p.m = std::min(a.R, a.C);
  const int64_t t128 = up(a.R, 128) / 128 * (up(a.C, 128) / 128) * a.n;
  p.tile = t128 >= device_cus() ? 128 : 64;
  p.Rp = up(a.R, p.tile);
  p.Cp = up(a.C, p.tile);
  p.mp = up(p.m, p.tile);
  p.nb = (int)std::min<int64_t>(kSumBlocks, (a.R * a.C + 4095) / 4096);
  p.x = (size_t)(a.n * p.Rp * p.Cp) * 4;
  p.a = (size_t)(a.n * p.mp * p.mp) * 4;
  p.part = 2 * p.x + 2 * p.a;
  p.unit = p.part + (size_t)a.n * p.nb * sizeof(double);
  p.total = p.unit + (size_t)a.n * sizeof(float);
  return p;
}

template <int TILE, bool KI>
hipError_t launch_product_t(const ProductArgs& p, int64_t n, hipStream_t s) {
  static hipError_t once = hipFuncSetAttribute((const void*)ortho_product_kernel<TILE, KI>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               product_lds<TILE, KI>());
  if (once != hipSuccess) return once;
  const int64_t tiles = p.sym ? (int64_t)p.mt * (p.mt + 1) / 2 : (int64_t)p.mt * p.nt;
  hipLaunchKernelGGL((ortho_product_kernel<TILE, KI>), dim3((unsigned)(tiles * n)), dim3(kNT),
                     (product_lds<TILE, KI>()), s, p);
  return hipGetLastError();
}

hipError_t launch_product(const ProductArgs& p, int tile, bool ki, int64_t n, hipStream_t s) {
  if (tile == 128) return ki ? launch_product_t<128, true>(p, n, s) : launch_product_t<128, false>(p, n, s);
  return ki ? launch_product_t<64, true>(p, n, s) : launch_product_t<64, false>(p, n, s);
}

template <class E, bool MUON>
hipError_t launch_input(const OrthoArgs& a, const Plan& p, double* part, float* unit, Pair X,
                        float pow_x, hipStream_t s) {
  hipLaunchKernelGGL((ortho_norm_kernel<E, MUON>), dim3((unsigned)p.nb, (unsigned)a.n), dim3(256), 0,
                     s, a, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t blocks = std::min<int64_t>(2048, (p.Rp * p.Cp / 4 + 255) / 256);
  hipLaunchKernelGGL((ortho_split_kernel<E, MUON>), dim3((unsigned)blocks, (unsigned)a.n), dim3(256),
                     0, s, a, (const double*)part, p.nb, X, p.Rp, pow_x, unit);
  return hipGetLastError();
}

}  // namespace

bool ortho_coeffs_ok(const OrthoArgs& a) {
  double top = 1.0;
  for (int k = 0; k < a.steps; ++k) {
    top = kRoom * poly_bound(a.a, a.b, a.c, top);
    if (!(top <= 4.0)) return false;
    if (!(quad_bound(a.b, a.c, top * top) <= 1e4)) return false;
  }
  return true;
}

size_t ortho_workspace_bytes(const OrthoArgs& a) { return plan_of(a).total; }

hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s) {
  const Plan p = plan_of(a);
  char* ws = (char*)a.ws;
  auto pair = [&](size_t off, int64_t rows, int64_t ld) {
    uint16_t* hi = (uint16_t*)(ws + off);
    return Pair{hi, hi + a.n * rows * ld, ld, rows * ld};
  };
  Pair X[2] = {pair(0, p.Rp, p.Cp), pair(p.x, p.Rp, p.Cp)};
  const Pair A = pair(2 * p.x, p.mp, p.mp), B = pair(2 * p.x + p.a, p.mp, p.mp);
  double* part = (double*)(ws + p.part);
  float* unit = (float*)(ws + p.unit);
  double top = 1.0;
  int sx = scale_of(top * kRoom);
  timing_begin("ortho_input", s);
  hipError_t e;
  if (a.W != nullptr) e = launch_input<F32, true>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  else if (a.dtype == kBF16) e = launch_input<BF16, false>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  else e = launch_input<F32, false>(a, p, part, unit, X[0], std::ldexp(1.f, sx), s);
  timing_end("ortho_input", s);
  const int mt = (int)(p.mp / p.tile);
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    const Pair& Xk = X[k & 1];
    const int sa = scale_of(kRoom * top * top), sb = scale_of(kRoom * quad_bound(a.b, a.c, top * top));
    top = kRoom * poly_bound(a.a, a.b, a.c, top);
    const bool last = k + 1 == a.steps;
    const int sn = last ? 0 : scale_of(kRoom * top);
    ProductArgs q{};
    q.unit = unit;
    // A = X X^T (R <= C: K-inner) or X^T X (K-outer)
    q.L = q.R = Xk;
    q.out = q.add = A;
    q.K = p.flip ? p.Rp : p.Cp;
    q.mt = q.nt = mt;
    q.sym = 1;
    q.mode = kStore;
    q.units = 2;
    q.f1 = (float)std::ldexp(1.0, sa - 2 * sx);
    timing_begin("ortho_gram", s);
    e = launch_product(q, p.tile, !p.flip, a.n, s);
    timing_end("ortho_gram", s);
    if (e != hipSuccess) break;
    // B = b A + c A A
    q.L = q.R = q.add = A;
    q.out = B;
    q.K = p.mp;
    q.mode = kAddStore;
    q.units = 0;
    q.f0 = (float)(a.b * std::ldexp(1.0, sb - sa));
    q.f1 = (float)(a.c * std::ldexp(1.0, sb - 2 * sa));
    timing_begin("ortho_square", s);
    e = launch_product(q, p.tile, !p.flip, a.n, s);
    timing_end("ortho_square", s);
    if (e != hipSuccess) break;
    // X <- a X + B X (K-outer) or a X + X B (K-inner)
    q.L = p.flip ? Xk : B;
    q.R = p.flip ? B : Xk;
    q.add = Xk;
    q.out = X[(k + 1) & 1];
    q.mt = (int)(p.Rp / p.tile);
    q.nt = (int)(p.Cp / p.tile);
    q.sym = 0;
    q.mode = last ? kFinal : kAddStore;
    q.units = last ? 1 : 0;
    q.f0 = (float)(a.a * std::ldexp(1.0, sn - sx));
    q.f1 = (float)std::ldexp(1.0, sn - sb - sx);
    q.rows = a.R;
    q.cols = a.C;
    q.dst = a.W != nullptr ? (void*)a.W : a.out;
    q.dtype = a.dtype;
    q.muon = a.W != nullptr ? 1 : 0;
    q.decay = a.decay;
    q.size = a.size;
    timing_begin("ortho_apply", s);
    e = launch_product(q, p.tile, p.flip, a.n, s);
    timing_end("ortho_apply", s);
    sx = sn;
  }
  return e;
}

}  // namespace dpf
