// Internal interface of the operators at a language model's two ends and of
// its optimizer: embedding rows, token log probabilities, the orthogonalised
// update.
#pragma once

#include "kernels.hpp"

namespace dpf {

// [B, T] token ids in device memory (int32, or int64 when wide), rows
// stride_b elements apart.
struct Ids {
  const void* data;
  int wide;
  int64_t stride_b;
  __device__ __forceinline__ int64_t at(int64_t b, int64_t t) const {
    const int64_t e = b * stride_b + t;
    return wide ? ((const int64_t*)data)[e] : (int64_t)((const int32_t*)data)[e];
  }
};

// V consecutive elements (V = 1, 4 or 8; V > 1: naturally aligned) as float32,
// and back (bf16 rounded to nearest even).
template <class E, int V>
__device__ __forceinline__ void load_f32(const typename E::storage* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = E::to_float(p[0]);
  } else if constexpr (sizeof(typename E::storage) == 4) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const f32x4 w = *(const f32x4*)(p + k);
      x[k] = w.x; x[k + 1] = w.y; x[k + 2] = w.z; x[k + 3] = w.w;
    }
  } else if constexpr (V == 4) {
    const u16x4 w = *(const u16x4*)p;
    x[0] = E::to_float(w.s0); x[1] = E::to_float(w.s1);
    x[2] = E::to_float(w.s2); x[3] = E::to_float(w.s3);
  } else {
    const u16x8 w = *(const u16x8*)p;
    x[0] = E::to_float(w.s0); x[1] = E::to_float(w.s1);
    x[2] = E::to_float(w.s2); x[3] = E::to_float(w.s3);
    x[4] = E::to_float(w.s4); x[5] = E::to_float(w.s5);
    x[6] = E::to_float(w.s6); x[7] = E::to_float(w.s7);
  }
}

// The same elements as they are in memory: a load whose conversion can come
// later, so that several are in flight (a conversion beside the load waits for
// it wherever a branch stands between the two and the next).
template <class E, int V>
struct RawOf {
  typedef typename E::storage S;
  static constexpr int kBytes = V * (int)sizeof(S);
  typedef S type __attribute__((ext_vector_type(V), aligned(kBytes < 16 ? kBytes : 16)));
};
template <class E>
struct RawOf<E, 1> {
  typedef typename E::storage type;
};
template <class E, int V>
using Raw = typename RawOf<E, V>::type;

template <class E, int V>
__device__ __forceinline__ Raw<E, V> load_raw(const typename E::storage* p) {
  return *(const Raw<E, V>*)p;
}
template <class E, int V>
__device__ __forceinline__ float raw_f32(const Raw<E, V>& r, int k) {
  if constexpr (V == 1) return E::to_float(r);
  else return E::to_float(r[k]);
}

template <class E, int V>
__device__ __forceinline__ void store_f32(typename E::storage* p, const float (&x)[V]) {
  if constexpr (sizeof(typename E::storage) == 4) {
    if constexpr (V == 1) {
      p[0] = x[0];
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        f32x4 w; w.x = x[k]; w.y = x[k + 1]; w.z = x[k + 2]; w.w = x[k + 3];
        *(f32x4*)(p + k) = w;
      }
    }
  } else if constexpr (V == 1) {
    p[0] = f32_to_bf16_rne(x[0]);
  } else if constexpr (V == 4) {
    u16x4 w;
    w.s0 = f32_to_bf16_rne(x[0]); w.s1 = f32_to_bf16_rne(x[1]);
    w.s2 = f32_to_bf16_rne(x[2]); w.s3 = f32_to_bf16_rne(x[3]);
    *(u16x4*)p = w;
  } else {
    u16x8 w;
    w.s0 = f32_to_bf16_rne(x[0]); w.s1 = f32_to_bf16_rne(x[1]);
    w.s2 = f32_to_bf16_rne(x[2]); w.s3 = f32_to_bf16_rne(x[3]);
    w.s4 = f32_to_bf16_rne(x[4]); w.s5 = f32_to_bf16_rne(x[5]);
    w.s6 = f32_to_bf16_rne(x[6]); w.s7 = f32_to_bf16_rne(x[7]);
    *(u16x8*)p = w;
  }
}

// The value of lane l ^ j (j a power of two known when compiled, every lane
// active), without going through LDS as a shuffle does: within 16 lanes by
// data-parallel moves, across them by gfx950's lane swaps.  A chain of 21
// such steps sorts a wave, so their latency counts.
__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int j) {
  const uint32_t lane = threadIdx.x & 63;
  switch (j) {
    case 1: return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true);   // quad 1 0 3 2
    case 2: return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true);   // quad 2 3 0 1
    case 4: {                                              // mirrored in 8, then in 4
      const uint32_t h = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true);
      return __builtin_amdgcn_update_dpp(0, h, 0x1B, 0xf, 0xf, true);
    }
    case 8: return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true);  // 16 rotated by 8
    case 16: {
      const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      return (lane & 16) ? s[0] : s[1];
    }
    default: {
      const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      return (lane & 32) ? s[0] : s[1];
    }
  }
}
__device__ __forceinline__ int lane_xor(int v, int j) { return (int)lane_xor((uint32_t)v, j); }
__device__ __forceinline__ float lane_xor(float v, int j) {
  return __uint_as_float(lane_xor(__float_as_uint(v), j));
}
__device__ __forceinline__ double lane_xor(double v, int j) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = lane_xor((uint32_t)b, j), hi = lane_xor((uint32_t)(b >> 32), j);
  return __builtin_bit_cast(double, (hi << 32) | lo);
}

// philox_block's words, with gfx950's three-way xor: 20 instructions of a block's
// 100 less.
__device__ __forceinline__ u32x4 philox_block_xor3(uint64_t seed, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = 0u, c3 = 0u;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)kPhiloxM0 * c0, p1 = (uint64_t)kPhiloxM1 * c2;
    c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, 0x96);
    c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, 0x96);
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
    k0 += kPhiloxW0;
    k1 += kPhiloxW1;
  }
  u32x4 w;
  w.x = c0; w.y = c1; w.z = c2; w.w = c3;
  return w;
}

// The four normals of a Philox block, as normals_of_block, with the radius
// through the hardware's logarithm and square root: over all 2^23 uniforms it
// is within 4.9e-7 of the exact value (the library functions: 5.7e-7) in far
// fewer instructions.  The hardware's sine and cosine are no replacement: near
// their zeros they are off by 11 units of the last place.
__device__ __forceinline__ f32x4 normals_of_block_hw(u32x4 w) {
  constexpr float kM2Ln2 = -1.3862943611198906f;
  const float r01 = __builtin_amdgcn_sqrtf(kM2Ln2 * __builtin_amdgcn_logf(word_to_uniform(w.x)));
  const float r23 = __builtin_amdgcn_sqrtf(kM2Ln2 * __builtin_amdgcn_logf(word_to_uniform(w.z)));
  float s1, c1, s3, c3;
  sincospif(2.0f * word_to_uniform(w.y), &s1, &c1);
  sincospif(2.0f * word_to_uniform(w.w), &s3, &c3);
  f32x4 z;
  z.x = r01 * c1; z.y = r01 * s1; z.z = r23 * c3; z.w = r23 * s3;
  return z;
}

// Embedding (embedding.hip).
struct LookupArgs {
  Ids ids;
  const uint8_t* mask;      // [B, T] or null
  int64_t N, T;             // N = B * T positions
  const void* table;        // [V, D], rows stride_v elements apart
  int table_dtype;
  int64_t V, D, stride_v;
  float scale;
  void* out;                // [B, T, D] contiguous
  int out_dtype;
};
hipError_t launch_embedding_lookup(const LookupArgs& a, hipStream_t s);

struct EmbedArgs {
  Ids ids;
  const uint8_t* mask;      // [B, T] or null
  Act G;                    // [B, T, D]
  int dtype;
  int64_t B, T, V, D;
  float scale;
  // workspace
  uint32_t *key[2], *pos[2];   // [N] each: sort buffers, ping and pong
  uint32_t* hist;              // embed_hist_words
  uint2* seg;                  // [V] sorted range [x, y) of each row, x > y where it has none
  uint4* rec;                  // [N] each sorted position's token, sample and offset in G
  double* partials;            // [N, embed_norm_parts] squared run norms
  float* blocks;               // [N / 8, D] sums of blocks of positions, or null
  // clipped sum
  const float* c;              // [B]
  float noise_std;
  uint64_t seed, offset;
  float denom;
  int beta;
  float* out;                  // [V, D]
};
// Launch limits (threads of one grid dimension stay below 2^32).
constexpr int64_t kEmbedMaxN = (int64_t)1 << 25, kEmbedMaxV = (int64_t)1 << 24;
constexpr int64_t kEmbedMaxD = (int64_t)1 << 22, kEmbedMaxTable = (int64_t)1 << 33;
// Elements of a.hist and a.blocks (0: null), partials per sorted position.
int64_t embed_hist_words(int64_t N, int64_t V);
int64_t embed_block_floats(const EmbedArgs& a);
int embed_norm_parts(const EmbedArgs& a);
// Sorts the positions by (token, position); fills rec, empties seg.
hipError_t launch_embed_sort(const EmbedArgs& a, hipStream_t s);
// Fills seg, for calls that do not take the norms (which fill it too).
hipError_t launch_embed_segments(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embed_norm(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embed_accumulate(const EmbedArgs& a, hipStream_t s);

// Token log probabilities (logprobs.hip).
constexpr int kMaxTopK = 32;
constexpr int64_t kLogprobsMaxN = (int64_t)1 << 24, kLogprobsMaxV = (int64_t)1 << 23;
struct LogprobArgs {
  Act Z;                    // logits [B, T, V]
  int dtype;
  int64_t N, T, V;          // N = B * T rows
  Ids targets;              // data null: none
  const uint8_t* mask;      // [B, T] or null
  int top_k;
  float *logp, *entropy, *lse;   // [B, T] each, or null
  float* top_logp;          // [B, T, top_k]
  int32_t* top_ids;         // [B, T, top_k]
  void* ws;                 // logprobs_workspace_bytes(a)
};
// Workspace of a call whose rows are split over workgroups (0: none).
size_t logprobs_workspace_bytes(const LogprobArgs& a);
hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s);

struct LogprobGradArgs {
  Act Z, dZ;                // logits and their gradient, [B, T, V]
  int dtype, out_dtype;
  int64_t N, T, V;
  Ids targets;              // data null: none
  const uint8_t* mask;
  const float *lse, *entropy;      // [B, T] from the forward call
  const float *dlogp, *dentropy;   // [B, T], either may be null
};
hipError_t launch_token_logprobs_backward(const LogprobGradArgs& a, hipStream_t s);

// Orthogonalised update (ortho.hip): n matrices [R, C] stacked contiguously.
constexpr int kOrthoMaxSteps = 32;
struct OrthoArgs {
  int64_t n, R, C;
  int steps;
  double a, b, c, eps;      // X <- a X + b (X X^T) X + c (X X^T)^2 X
  // orthogonalize: out = NS(in); both of dtype
  const void* in;
  void* out;
  int dtype;
  // optimizer step (W not null): momentum <- beta momentum + grad, then
  // W <- decay W - size NS(update)
  const float* grad;
  float *momentum, *W;
  float beta, decay, size;
  int nesterov;
  int tile;                 // 128 or 256 wide products, 0: the faster by their cost
  void* ws;                 // ortho_workspace_bytes(a)
};
// False where the coefficients let a singular value grow past 4 within the
// steps (the half-precision factors are scaled for that range).
bool ortho_coeffs_ok(const OrthoArgs& a);
size_t ortho_workspace_bytes(const OrthoArgs& a);
hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s);

}  // namespace dpf
