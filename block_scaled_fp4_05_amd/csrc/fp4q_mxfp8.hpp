// fp4q_mxfp8.hpp -- device pieces of the kernels that write MXFP8 (fp4q_mxfp8.hip, fp4q_rotary.hip).
//
// One 16-byte chunk of a row is what a lane loads at a time: eight bf16 or four fp32
// elements, so a load instruction covers whole cache lines and four (bf16) or eight (fp32)
// neighbouring lanes hold one 32-element block.
#pragma once
#include "fp4q_dev.hpp"

namespace fp4q {
namespace {

typedef float f32x2m __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2m __attribute__((ext_vector_type(2)));

// Two fp32 values to packed bf16, nearest even (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2m{a, b}), bf16x2m));
}

template <typename T>
struct Chunk {
  static constexpr int N = 16 / (int)sizeof(T);   // elements per chunk
  static constexpr int LANES = 32 / N;            // lanes per 32-element block
};

__device__ __forceinline__ void unpack(const u32x4_t& w, float (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack(const u32x4_t& w, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[2 * i] = bf16_lo(w[i]), o[2 * i + 1] = bf16_hi(w[i]);
}
__device__ __forceinline__ u32x4_t pack(const float (&v)[4]) {
  return u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}
__device__ __forceinline__ u32x4_t pack(const float (&v)[8]) {
  return u32x4_t{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]), to_bf16x2(v[6], v[7])};
}

template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk_nt(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
}
template <typename T>
__device__ __forceinline__ void store_chunk_nt(T* p, const u32x4_t& w) {
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
}

// Maximum over the lanes of one block of non-negative values (see lane_xor_max); after the
// two steps within a quad its four lanes agree, so mirroring eight lanes swaps the quads.
template <int LANES>
__device__ __forceinline__ float block_max(float m) {
  m = lane_xor_max<1>(m);
  m = lane_xor_max<2>(m);
  if constexpr (LANES == 8) {
    const int o = __builtin_amdgcn_mov_dpp(__float_as_int(m), 0x141, 0xF, 0xF, false);   // row_half_mirror
    m = __uint_as_float(max(__float_as_uint(m), (uint32_t)o));
  }
  return m;
}

// The scale code of a block whose largest finite magnitude has the bits b: 448 = 1.75 * 2^8,
// so a significand up to 1.75 takes the exponent less 8, a larger one the next.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t b) {
  return (uint32_t)max((int)((b + 0x1FFFFFu) >> 23) - 8, 0);
}

// One lane's chunk of a block -> its codes (N bytes, in place order) and the block's scale code.
// The maximum ignores NaN by itself (fmax); an infinity is rare enough to be looked for only
// when the maximum is one.
template <typename T, int N>
__device__ __forceinline__ uint32_t mx8_encode(const float (&v)[N], uint32_t (&w)[N / 4]) {
  constexpr int LANES = Chunk<T>::LANES;
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
  float bm = block_max<LANES>(m);
  if (__builtin_expect(__any(bm == __builtin_inff()), 0)) {
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = __builtin_fabsf(v[i]);
      if (a < __builtin_inff()) m = __builtin_fmaxf(m, a);
    }
    bm = block_max<LANES>(m);
  }
  const uint32_t code = mx8_scale(__float_as_uint(bm));
  const float inv = __uint_as_float((254u - code) << 23);   // 2^(127 - code): code <= 247
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    uint32_t t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, t, true);
  }
  return code;
}

__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[2]) {
  __builtin_nontemporal_store(u32x2_t{w[0], w[1]}, reinterpret_cast<u32x2_t*>(p));
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[1]) {
  __builtin_nontemporal_store(w[0], reinterpret_cast<uint32_t*>(p));
}

}  // namespace
}  // namespace fp4q
