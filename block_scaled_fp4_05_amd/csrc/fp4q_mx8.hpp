// fp4q_mx8.hpp -- device pieces shared by the products of MXFP8 activations and MXFP4
// weights (fp4q_gemm8.hip, fp4q_moe.hip).
//
// v_mfma_scale_f32_{16x16x128,32x32x64}_f8f6f4 takes one operand in E4M3 and the other in
// E2M1.  Lane layout (checked with an in-bounds probe, both operand orders), for R = 16 or 32
// rows per operand, lane l holding row l % R of its operand and q = l / R:
//  - E2M1: 16 bytes, K elements 32 q .. 32 q + 31;
//  - E4M3: 32 bytes, the first 16 at K = 16 q .., the last 16 at K = (instruction's K) / 2 + 16 q ..;
//  - the scale byte of lane l is that of K block q (32 elements) of its row, for both.
// The E4M3 products of one small group are aligned to the group's largest and cut about 13
// bits below it, groups are joined in fp32: on Gaussian operands a result is about 5e-6
// (2-norm) from the exact one, against 2.6e-2 for rounding an operand to E4M3.
#pragma once
#include "fp4q_internal.hpp"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

typedef int v8i_m __attribute__((ext_vector_type(8)));
typedef float v4f_m __attribute__((ext_vector_type(4)));
typedef float v16f_m __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_m __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_w __attribute__((ext_vector_type(4), aligned(4)));   // four words at a word's alignment
typedef uint32_t u32x2_m __attribute__((ext_vector_type(2)));
typedef float f32x2_m __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_m __attribute__((ext_vector_type(2)));

// Operand registers of the builtin: 16 bytes of E2M1 (the upper half is not read), or two
// 16-byte pieces of E4M3.
__device__ __forceinline__ v8i_m frag4(u32x4_m w) {
  return v8i_m{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
}
__device__ __forceinline__ v8i_m frag8(u32x4_m lo, u32x4_m hi) {
  return v8i_m{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// acc[row of w][row of x] += w (16 rows, E2M1) x^T (16 rows, E4M3) over 128 K elements; sw / sx
// hold the lane's scale byte in byte 0.  Register r of lane l is row 4 (l / 16) + r, column l % 16.
__device__ __forceinline__ v4f_m mma_w4x8(v8i_m w, v8i_m x, v4f_m acc, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, 0, 0, (int)sw, 0, (int)sx);
}

// acc += x (32 rows, E4M3) w^T (32 rows, E2M1) over 64 K elements; the lane's scale byte is byte 0
// (_lo) or byte 2 (_hi) of its word.  Register t is row 8 (t / 4) + 4 (l / 32) + t % 4, column l % 32.
__device__ __forceinline__ v16f_m mma_x8w4_lo(v8i_m x, v8i_m w, v16f_m acc, uint32_t sx, uint32_t sw) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, w, acc, 0, 4, 0, (int)sx, 0, (int)sw);
}
__device__ __forceinline__ v16f_m mma_x8w4_hi(v8i_m x, v8i_m w, v16f_m acc, uint32_t sx, uint32_t sw) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, w, acc, 0, 4, 2, (int)sx, 2, (int)sw);
}

// Scale words s .. s + 3 of a row of n words (four blocks each, little end first), in one load
// where the row has four: a load of one word per row costs the address unit as much as 16 bytes
// per lane.  Words past the row's end repeat its last.
// The row is at `base` (the same for the wave) + `row` bytes.
__device__ __forceinline__ u32x4_m scale_words(const uint8_t* base, uint32_t row, int s, int n) {
  u32x4_m v;
  if (n >= 4) {
    const int at = min(s, n - 4), down = min(s - at, 3);
    v = *reinterpret_cast<const u32x4_w*>(base + 4 * at + row);
    const uint32_t one = 0u - (uint32_t)(down & 1), two = 0u - (uint32_t)(down >> 1);
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = (v[j] & ~one) | (v[j + 1] & one);
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = (v[j] & ~two) | (v[j + 2] & two);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(base + 4 * min(s + j, n - 1) + row);
  }
  return v;
}

// From a register whose lanes 16 i .. 16 i + 15 belong to row tile i, four registers with tile i's
// lanes in all four groups of 16: v_permlane16_swap exchanges the odd groups of its first operand
// with the even groups of its second, v_permlane32_swap the upper half with the lower half.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&o)[4]) {
  const auto a = __builtin_amdgcn_permlane16_swap(w, w, false, false);         // 0 0 2 2 and 1 1 3 3
  const auto e = __builtin_amdgcn_permlane32_swap(a[0], a[0], false, false);   // 0 0 0 0 and 2 2 2 2
  const auto f = __builtin_amdgcn_permlane32_swap(a[1], a[1], false, false);
  o[0] = e[0], o[2] = e[1], o[1] = f[0], o[3] = f[1];
}

// Likewise two, from a register whose even groups belong to tile 0 and odd ones to tile 1; one is its
// own.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&o)[2]) {
  const auto a = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  o[0] = a[0], o[1] = a[1];
}
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&o)[1]) { o[0] = w; }

// 16 bytes at `base` (the same for the wave) + `off`: the address costs a lane one register.
__device__ __forceinline__ u32x4_m load16(const uint8_t* base, uint32_t off) {
  return *reinterpret_cast<const u32x4_m*>(base + off);
}

// Orders a wave's LDS writes before its other lanes' reads, and those before the next writes: no
// instruction (the hardware keeps a wave's LDS accesses in order), only a limit on the compiler.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// T tiles of 16 rows x 128 bytes that were loaded by lines (lane l: w[i][0] is 16-byte chunk l % 8 of row
// l / 8 of tile i, w[i][1] that of row 8 + l / 8) to the matrix instruction's layout (lane l: chunks l / 16,
// in lo, and 4 + l / 16, in hi, of row l % 16), through 2 KB each of the wave's own LDS, with no barrier
// of the workgroup.  Chunk c of row i sits at c ^ (i % 8): neither side has bank conflicts.
template <int T>
__device__ __forceinline__ void deal(u32x4_m (*block)[128], const u32x4_m (&w)[T][2], u32x4_m (&lo)[T],
                                     u32x4_m (&hi)[T]) {
  const int l = threadIdx.x & 63, r = l & 15, q = l >> 4, put = (l & 56) + ((l & 7) ^ (l >> 3));
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < T; ++i) block[i][put] = w[i][0], block[i][put + 64] = w[i][1];
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < T; ++i) lo[i] = block[i][r * 8 + (q ^ (r & 7))], hi[i] = block[i][r * 8 + ((q + 4) ^ (r & 7))];
}

// Likewise T tiles of 16 rows x 64 bytes (lane l: chunk l % 4 of row l / 4) to one fragment each, through 1 KB
// for one tile after the other; chunk c of row i sits at c ^ (i / 2 % 4).
template <int T>
__device__ __forceinline__ void deal(u32x4_m* block, const u32x4_m (&w)[T], u32x4_m (&frag)[T]) {
  const int l = threadIdx.x & 63, r = l & 15, q = l >> 4;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    wave_lds_fence();
    block[(l & 60) + ((l & 3) ^ ((l >> 3) & 3))] = w[i];
    wave_lds_fence();
    frag[i] = block[r * 4 + (q ^ ((r >> 1) & 3))];
  }
}

// Two fp32 values to packed bf16, nearest even (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_m{a, b}), bf16x2_m));
}

}  // namespace fp4q
