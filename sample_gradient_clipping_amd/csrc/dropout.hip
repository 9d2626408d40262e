// Dropout with a counter-based mask that is never stored:
//
//   y_e = r_e + (bits_e >= limit ? factor x_e : 0),  limit = round(65536 p), factor = 65536 / (65536 - limit)
//
// bits_e: the 16-bit half e mod 8 (low half of each word first) of Philox block
// offset + e / 8, e the row-major index in [B, T, D].  Half words are enough to
// hold p to 2^-17 with a mean that is exact for the p they hold, and one block
// then serves eight entries: at four it would cost as much as the memory traffic.
// HBM bounds the pass: a thread takes the eight entries of one block, 16 bytes
// at a time (8x2048x5120 bf16 with residual: 87 us, 5.8 TB/s).
#include "lm.hpp"

namespace dpf {
namespace {

constexpr int kNT = 256;

__device__ __forceinline__ uint32_t half_of(const u32x4& w, int k) {
  const uint32_t x = w[k >> 1];
  return k & 1 ? x >> 16 : x & 0xffffu;
}

template <class E, bool RESIDUAL>
__global__ __launch_bounds__(kNT) void dropout_kernel(DropoutArgs a) {
  typedef typename E::storage S;
  const int64_t j = (int64_t)blockIdx.x * kNT + threadIdx.x, pieces = a.D / 8;
  const int64_t n = j / pieces;
  if (n >= a.B * a.T) return;
  const int64_t b = n / a.T, t = n % a.T, d = (j - n * pieces) * 8;
  S* y = (S*)a.Y.data + b * a.Y.stride_b + t * a.Y.stride_t + d;
  float out[8] = {};
  if (a.mask == nullptr || a.mask[n] != 0) {
    const Raw<E, 8> x = load_raw<E, 8>((const S*)a.X.data + b * a.X.stride_b + t * a.X.stride_t + d);
    Raw<E, 8> r = {};
    if constexpr (RESIDUAL) r = load_raw<E, 8>((const S*)a.R.data + b * a.R.stride_b + t * a.R.stride_t + d);
    const u32x4 w = philox_block_xor3(a.seed, a.offset + (uint64_t)j, 1u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      out[k] = half_of(w, k) >= a.limit ? a.factor * raw_f32<E, 8>(x, k) : 0.0f;
      if constexpr (RESIDUAL) out[k] += raw_f32<E, 8>(r, k);
    }
  }
  store_f32<E, 8>(y, out);
}

// Rows of any length and alignment: a thread still takes one block, its entries
// one by one (they may lie in two rows, or more).
template <class E>
__global__ __launch_bounds__(kNT) void dropout_any_kernel(DropoutArgs a) {
  typedef typename E::storage S;
  const int64_t total = a.B * a.T * a.D;
  const int64_t j = (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (j * 8 >= total) return;
  const u32x4 w = philox_block_xor3(a.seed, a.offset + (uint64_t)j, 1u);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t e = j * 8 + k;
    if (e >= total) return;
    const int64_t n = e / a.D, d = e - n * a.D, b = n / a.T, t = n % a.T;
    float out[1] = {0.0f};
    if (a.mask == nullptr || a.mask[n] != 0) {
      if (half_of(w, k) >= a.limit)
        out[0] = a.factor * E::to_float(((const S*)a.X.data)[b * a.X.stride_b + t * a.X.stride_t + d]);
      if (a.R.data != nullptr)
        out[0] += E::to_float(((const S*)a.R.data)[b * a.R.stride_b + t * a.R.stride_t + d]);
    }
    store_f32<E, 1>((S*)a.Y.data + b * a.Y.stride_b + t * a.Y.stride_t + d, out);
  }
}

template <class E>
void dropout_e(const DropoutArgs& a, hipStream_t s) {
  const int64_t blocks = (a.B * a.T * a.D + 7) / 8;
  const dim3 grid((unsigned)((blocks + kNT - 1) / kNT));
  if (!a.vec) hipLaunchKernelGGL((dropout_any_kernel<E>), grid, dim3(kNT), 0, s, a);
  else if (a.R.data != nullptr) hipLaunchKernelGGL((dropout_kernel<E, true>), grid, dim3(kNT), 0, s, a);
  else hipLaunchKernelGGL((dropout_kernel<E, false>), grid, dim3(kNT), 0, s, a);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  timing_begin("dropout", s);
  if (a.dtype == kBF16) dropout_e<BF16>(a, s);
  else dropout_e<F32>(a, s);
  timing_end("dropout", s);
  return hipGetLastError();
}

}  // namespace dpf
