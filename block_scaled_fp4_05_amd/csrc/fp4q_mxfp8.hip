// MXFP8 (E4M3 elements, an E8M0 scale per 32): the quantizer, its inverse, the RMS norm that
// ends in it and that norm's gradient.
#include "fp4q_mxfp8.hpp"

#include <type_traits>

namespace fp4q {
namespace {

// -----------------------------------------------------------------------------------------
// Quantizer: a stream over the chunks of the whole tensor (cols % 32 == 0, so blocks and
// chunks ignore the row boundaries).  Four chunks per thread, all loads first.  Bound by memory: bf16
// 16384 x 4096 (203 MB) in 32.3 us, 6.3 TB/s; fp32 (338 MB) 54 us, 6.2 TB/s; a few rows take one launch (2.9 us).
// -----------------------------------------------------------------------------------------
constexpr int kQuantChunks = 4;   // chunks per thread

template <typename T>
__global__ __launch_bounds__(256) void k_mxfp8(const T* __restrict__ x, int64_t chunks, uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ scales) {
  constexpr int N = Chunk<T>::N, LANES = Chunk<T>::LANES;
  const int64_t c0 = (int64_t)blockIdx.x * (256 * kQuantChunks) + threadIdx.x;
  u32x4_t in[kQuantChunks];
#pragma unroll
  for (int j = 0; j < kQuantChunks; ++j) {
    const int64_t c = c0 + 256 * j;
    in[j] = c < chunks ? load_chunk_nt(x + c * N) : u32x4_t{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int j = 0; j < kQuantChunks; ++j) {
    const int64_t c = c0 + 256 * j;
    float v[N];
    uint32_t w[N / 4];
    unpack(in[j], v);
    const uint32_t code = mx8_encode<T>(v, w);
    if (c < chunks) {
      store_codes(codes + c * N, w);
      if ((threadIdx.x & (LANES - 1)) == 0) scales[c / LANES] = (uint8_t)code;
    }
  }
}

// Eight codes per lane.  Bound by memory: 16384 x 4096 to bf16 33 us, 6.1 TB/s; to fp32, two 16-byte stores 32
// bytes apart per lane, 99 us, 3.4 TB/s.
template <bool BF16OUT>
__global__ __launch_bounds__(256) void k_dequant_mxfp8(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int64_t n8,
                                                       void* __restrict__ y) {
  // the grid is capped (a launch has at most 2^32 threads), so a workgroup may take several pieces
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < n8; g += (int64_t)gridDim.x * 256) {
    const u32x2_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(codes + g * 8));
    const uint32_t sc = scales[g >> 2];
    const float s = sc == 255u ? __builtin_nanf("") : e8m0_value(sc);
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
      v[4 * h] = lo[0] * s, v[4 * h + 1] = lo[1] * s, v[4 * h + 2] = hi[0] * s, v[4 * h + 3] = hi[1] * s;
    }
    if constexpr (BF16OUT) {
      store_chunk_nt(static_cast<uint16_t*>(y) + g * 8, pack(v));
    } else {
      float* d = static_cast<float*>(y) + g * 8;
      store_chunk_nt(d, pack(reinterpret_cast<const float(&)[4]>(v[0])));
      store_chunk_nt(d + 4, pack(reinterpret_cast<const float(&)[4]>(v[4])));
    }
  }
}

// -----------------------------------------------------------------------------------------
// RMS norm.  s = x + residual, r = 1 / sqrt(mean(s^2) + eps), n = s r gain, MXFP8(n).
// A workgroup keeps one row at a time in registers (V chunks per thread, chunk
// t + NT j for thread t), so x is read once; it walks rows blockIdx.x, + gridDim.x, ... with
// the gain in registers and the next row's loads in flight while this row is reduced.
// Bound by memory: bf16 8192 x 4096 with residual and sum (236 MB) in 42 us, 5.6 TB/s; bf16 4096 x 8192
// 44 us; fp32 8192 x 4096 74 us, 5.8 TB/s; one row 3.4 us, a launch and one trip to memory.  A row whose
// 32 elements per thread would need more than 256 threads is spread over more threads first: held by
// 256, 4096 x 8192 took 77 us, with its registers spilled.
// -----------------------------------------------------------------------------------------
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sum over the workgroup, the same bits in every thread.  `parity` alternates between calls,
// so one barrier per call is enough: a buffer is written again only after the barrier of the
// call in between, which every wave passes after reading it.
template <typename F>
__device__ __forceinline__ F group_sum(F v, F (*part)[16], int parity) {
  v = wave_sum(v);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[parity][threadIdx.x >> 6] = v;
  lds_barrier();
  F s = part[parity][0];
  for (int i = 1; i < waves; ++i) s += part[parity][i];
  return s;
}

// 1 / sqrt(v) in two parts, to well past fp32: one Newton step in double from the fp32 root.  0,
// infinity and NaN as the fp32 root gives them.
struct Root {
  float hi, lo;
};
__device__ __forceinline__ Root inverse_root(double v) {
  const float r0 = 1.0f / __builtin_sqrtf((float)v);
  if (!(r0 > 0.0f && r0 < __builtin_inff())) return Root{r0, 0.0f};
  const double d = (double)r0, r = d + d * 0.5 * (1.0 - v * d * d);
  const float hi = (float)r;
  return Root{hi, (float)(r - (double)hi)};
}

// s r gain to twice fp32: (p + e) gain.
//
// Rounded to fp32 and then to a code it would be rounded twice: n just past a point halfway between two
// codes can land on it and go to the even one.  Those points, and the scale's boundaries (1.75 2^k), have at
// most five significant bits, so only an n whose kBelowHalf last bits are all zero can be wrong (one in 2^19);
// it is moved to the next fp32 number on the side of the exact product, which rounds as that would.  Of the 33.5
// million codes of bf16 8192 x 4096 that leaves 2 or 3 other than the exact ones (the sum of squares is fp32),
// where rounding twice left some 20, now and then with a scale and its block.  us without / with, with a residual:
// bf16 8192 x 4096 44.2 / 42.4, 16384 x 2048 47.2 / 46.4, 4096 x 8192 44.0 / 44.6, 2048 x 16384 50.6 / 53.3, 1024 x 32768
// 51 / 52.5; without one 16384 x 2048 29.9 / 31.4.
constexpr int kBelowHalf = 19;
struct Product {
  float p, e, gain;
  __device__ __forceinline__ Product(float s, Root r, float g)
      : p(s * r.hi), e(__builtin_fmaf(s, r.lo, __builtin_fmaf(s, r.hi, -(s * r.hi)))), gain(g) {}
  // To nearest; `zeros` rises to its trailing zeros, which a zero has none of (v_ffbl_b32 gives -1; a zero
  // is common where a residual cancels).  The sign of a zero is the product's.
  __device__ __forceinline__ float rounded(int& zeros) const {
    const float n = __builtin_fmaf(p, gain, e * gain);
    int t;   // (in place of a count that the compiler guards against zero)
    asm("v_ffbl_b32 %0, %1" : "=v"(t) : "v"(n));
    zeros = max(zeros, t);
    return __builtin_copysignf(n, __uint_as_float(__float_as_uint(p) ^ __float_as_uint(gain)));
  }
  __device__ __forceinline__ float beside_boundary(float n) const {
    const uint32_t b = __float_as_uint(n);
    const float over = __builtin_fmaf(e, gain, __builtin_fmaf(p, gain, -n)), m = __builtin_fabsf(n);   // over: what n leaves out
    if ((b & ((1u << kBelowHalf) - 1u)) != 0u || !(m > 0.0f && m < __builtin_inff()) || over == 0.0f) return n;
    return __uint_as_float((over > 0.0f) == (n > 0.0f) ? b + 1u : b - 1u);
  }
};

// The same pointer, which the compiler takes for another one: what is read through it is not
// hoisted out of the loop over rows into registers that are not there.
__device__ __forceinline__ const float* per_row(const float* p) {
  asm volatile("" : "+s"(p));
  return p;
}
template <int N>
__device__ __forceinline__ void load_gain(const float* __restrict__ gain, int c, int chunks, float (&g)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4_t none = {0.0f, 0.0f, 0.0f, 0.0f};
    const f32x4_t v = c < chunks ? *reinterpret_cast<const f32x4_t*>(gain + (int64_t)c * N + i) : none;
#pragma unroll
    for (int k = 0; k < 4; ++k) g[i + k] = v[k];
  }
}

template <typename T, int V>
__global__ __launch_bounds__(1024) void k_rmsnorm(const T* x, const T* res, int rows, int cols,
                                                  const float* gain, float eps,
                                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, T* sum,
                                                  float* __restrict__ rstd, T* __restrict__ y) {
  constexpr int N = Chunk<T>::N, LANES = Chunk<T>::LANES;
  // The gain stays in registers and the next row is fetched a row ahead; with 32 elements per
  // thread that would spill, so there the gain comes from L2 for each row.
  constexpr bool HOLD = V * N < 32;
  __shared__ double part[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, chunks = cols / N;
  float g[HOLD ? V : 1][N];
  if constexpr (HOLD) {
#pragma unroll
    for (int j = 0; j < V; ++j) load_gain(gain, tid + nt * j, chunks, g[j]);
  }
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  u32x4_t xin[V], rin[V];
  auto fetch = [&](int64_t row) {
    const int64_t at = row * cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + nt * j;
      const bool ok = row < rows && c < chunks;
      xin[j] = ok ? load_chunk_nt(x + at + c * N) : zero;
      rin[j] = ok && res ? load_chunk_nt(res + at + c * N) : zero;
    }
  };
  const double inv_n = 1.0 / (double)cols;
  if constexpr (HOLD) fetch(blockIdx.x);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    if constexpr (!HOLD) fetch(row);
    float s[V][N];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      unpack(xin[j], s[j]);
      if (res) {
        float r[N];
        unpack(rin[j], r);
#pragma unroll
        for (int i = 0; i < N; ++i) s[j][i] += r[i];
      }
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) q = __builtin_fmaf(s[j][i], s[j][i], q);
      ss += q;
    }
    const int64_t at = row * cols;
    if (sum) {   // before the next row is fetched: sum may be x or res, whose this row is in registers
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (tid + nt * j < chunks) store_chunk_nt(sum + at + (tid + nt * j) * N, pack(s[j]));
    }
    if constexpr (HOLD) fetch(row + gridDim.x);
    else gain = per_row(gain);
    const Root r = inverse_root(group_sum((double)ss, part, parity) * inv_n + (double)eps);
    if (rstd && tid == 0) rstd[row] = r.hi;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + nt * j;
      if constexpr (!HOLD) {
        __builtin_amdgcn_sched_barrier(0);   // one chunk's gain at a time
        load_gain(gain, c, chunks, g[0]);
      }
      const float* gj = g[HOLD ? j : 0];
      float n[N];
      int zeros = 0;   // most trailing zeros of an n
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = Product(s[j][i], r, gj[i]).rounded(zeros);
      if (y && c < chunks) store_chunk_nt(y + at + c * N, pack(n));
      if (__builtin_expect(__any(zeros >= kBelowHalf), 0)) {
        Root again = r;   // taken for another: the products are formed again, not kept in registers for this
        asm volatile("" : "+v"(again.hi), "+v"(again.lo));
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = Product(s[j][i], again, gj[i]).beside_boundary(n[i]);
      }
      uint32_t w[N / 4];
      const uint32_t code = mx8_encode<T>(n, w);
      if (c < chunks) {
        store_codes(codes + at + c * N, w);
        if ((tid & (LANES - 1)) == 0) scales[(at >> 5) + c / LANES] = (uint8_t)code;
      }
    }
  }
}

// Gradient: a = dy gain, dx = r a - s r^3 mean(a s) + dsum, dgain = sum over rows of dy s r.  With x = s r,
// of size 1 whatever the row's, dx = r (a - x mean(a x)) + dsum: r^3 would leave fp32's range for rows of
// 1e13 and more, or 1e-13 and less.  The same walk; each workgroup also adds up dy s r over its rows, in registers
// for kRun rows at a time and these runs in its row of partial sums (one running sum was off by 3400
// roundings after 2^24 equal rows; runs keep that below 360), which k_rmsnorm_dgain adds in a fixed order.
// Bound by memory: bf16 8192 x 4096 with dsum (268 MB) in 51 us, 5.3 TB/s, and 5.0 us for the partial sums
// (16.8 MB from the last-level cache); fp32 92 us, 5.8 TB/s, and 4.8.
constexpr int kRun = 64;

// RUNS: more than one run (see BackwardRuns).
template <typename T, int V, bool RUNS>
__global__ __launch_bounds__(1024) void k_rmsnorm_backward(const T* dy, const T* __restrict__ s_in, const T* dsum,
                                                           int rows, int cols, const float* gain,
                                                           const float* __restrict__ rstd, T* dx,
                                                           float* __restrict__ partial) {
  constexpr int N = Chunk<T>::N;
  constexpr bool HOLD = V * N < 32;   // as above; where not, dsum is read late too
  __shared__ float part[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, chunks = cols / N;
  float g[HOLD ? V : 1][N], dg[V][N];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (HOLD) load_gain(gain, tid + nt * j, chunks, g[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) dg[j][i] = 0.0f;
  }
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  const float inv_n = 1.0f / (float)cols;
  int parity = 0, run = 0;   // rows in dg
  bool later = false;        // earlier runs are in `partial`
  const auto end_run = [&]() {
    float* to = partial + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + nt * j;
      if (c < chunks) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          f32x4_t v = {dg[j][i], dg[j][i + 1], dg[j][i + 2], dg[j][i + 3]};
          f32x4_t* p = reinterpret_cast<f32x4_t*>(to + c * N + i);
          if (RUNS && later) v += *p;
          *p = v;
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) dg[j][i] = 0.0f;
    }
    later = true;
    run = 0;
  };
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    const int64_t at = row * cols;
    u32x4_t din[V], sin[V], uin[HOLD ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + nt * j;
      din[j] = c < chunks ? load_chunk_nt(dy + at + c * N) : zero;
      sin[j] = c < chunks ? load_chunk_nt(s_in + at + c * N) : zero;
      if constexpr (HOLD) uin[j] = c < chunks && dsum ? load_chunk_nt(dsum + at + c * N) : zero;
    }
    if constexpr (!HOLD) gain = per_row(gain);
    const float r = rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d[N], s[N], q = 0.0f;
      unpack(din[j], d);
      unpack(sin[j], s);
      if constexpr (!HOLD) {
        __builtin_amdgcn_sched_barrier(0);
        load_gain(gain, tid + nt * j, chunks, g[0]);
      }
      const float* gj = g[HOLD ? j : 0];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = s[i] * r;
        q = __builtin_fmaf(d[i] * gj[i], x, q);
        dg[j][i] = __builtin_fmaf(d[i], x, dg[j][i]);
      }
      dot += q;
    }
    if constexpr (!HOLD) gain = per_row(gain);
    const float k = group_sum(dot, part, parity) * inv_n;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + nt * j;
      float d[N], s[N], u[N];
      unpack(din[j], d);
      unpack(sin[j], s);
      if constexpr (!HOLD) {
        __builtin_amdgcn_sched_barrier(0);
        uin[0] = c < chunks && dsum ? load_chunk_nt(dsum + at + c * N) : zero;
        load_gain(gain, c, chunks, g[0]);
      }
      const float* gj = g[HOLD ? j : 0];
      unpack(uin[HOLD ? j : 0], u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float t = r * (d[i] * gj[i] - s[i] * r * k);
        u[i] = dsum ? t + u[i] : t;
      }
      if (c < chunks) store_chunk_nt(dx + at + c * N, pack(u));
    }
    if constexpr (RUNS)
      if (++run == kRun) end_run();
  }
  if (!RUNS || run > 0) end_run();   // (every workgroup has a row: see backward_groups)
}

// dgain[c] = sum over the partial rows: 32 columns per workgroup, 32 threads per column, each
// adding every 32nd row, then a fixed tree.
__global__ __launch_bounds__(1024) void k_rmsnorm_dgain(const float* __restrict__ partial, int parts, int cols,
                                                        float* __restrict__ dgain) {
  __shared__ float t[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;   // cols % 32 == 0
  float v = 0.0f;
  constexpr int U = 16;   // loads in flight per thread; rows past the last add zero
  for (int r = ry; r < parts; r += 32 * U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = partial[(int64_t)min(r + 32 * u, parts - 1) * cols + c];
#pragma unroll
    for (int u = 0; u < U; ++u) v += r + 32 * u < parts ? x[u] : 0.0f;
  }
  t[ry][cx] = v;
  __syncthreads();
  for (int h = 16; h >= 1; h >>= 1) {
    if (ry < h) t[ry][cx] += t[ry + h][cx];
    __syncthreads();
  }
  if (ry == 0) dgain[c] = t[0][cx];
}

// Threads and chunks per thread for a row of `chunks` chunks: 256 threads with the fewest chunks
// each (powers of two up to 16 elements) that hold the row in registers, else 512 or 1024 threads
// of 16 elements, else 1024 of 32 (FP4Q_NORM_MAX_COLS is 1024 x 32).  From the width alone, so
// that a row's sums, and with them its results, are the same whatever number of rows it comes with.
struct RowShape {
  int v, threads;
};
template <typename T>
RowShape row_shape(int64_t cols) {
  const int64_t chunks = cols / Chunk<T>::N;
  constexpr int kMost = 32 / Chunk<T>::N;
  for (int limit : {256, 512, 1024})
    for (int v = 1; v < kMost; v *= 2) {
      const int64_t t = (chunks + v - 1) / v;
      if (t <= limit) return RowShape{v, (int)((t + 63) / 64 * 64)};
    }
  return RowShape{kMost, 1024};
}

template <template <typename, int> class K, typename T>
auto by_chunks(int v) {
  if constexpr (Chunk<T>::N == 4) {
    if (v == 8) return K<T, 8>::fn();
  }
  return v == 1 ? K<T, 1>::fn() : v == 2 ? K<T, 2>::fn() : K<T, 4>::fn();
}
template <typename T, int V>
struct NormKernel {
  static auto fn() { return k_rmsnorm<T, V>; }
};
// The gradient with more than one run: where a workgroup has more than kRun rows, and for fp32 rows of more
// than 16384 columns, whose registers spill less in that form (4096 x 20000 351 us, one run 433). Elsewhere
// it costs registers: bf16 4096 x 20000 177 us, one run 158.
template <typename T, int V>
struct BackwardRuns {
  static auto fn() { return k_rmsnorm_backward<T, V, true>; }
};
template <typename T, int V>
struct BackwardOnce {
  static auto fn() { return k_rmsnorm_backward<T, V, V == 8>; }
};

// Workgroups of the gradient, each with its row of partial sums: what the card holds at once (four
// of 256 threads on each of its 256 units, or as many threads in larger ones).
int64_t backward_groups(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 4096 ? 1024 : cols <= 8192 ? 512 : 256;
  return rows < most ? rows : most;
}

template <typename T>
void rmsnorm(const T* x, const T* res, int64_t rows, int64_t cols, const float* gain, float eps, uint8_t* codes,
             uint8_t* scales, T* sum, float* rstd, T* y, hipStream_t st) {
  const RowShape s = row_shape<T>(cols);
  const int grid = (int)(rows < 2048 ? rows : 2048);
  by_chunks<NormKernel, T>(s.v)<<<grid, s.threads, 0, st>>>(x, res, (int)rows, (int)cols, gain, eps, codes, scales, sum,
                                                            rstd, y);
}

template <typename T>
void rmsnorm_backward(const T* dy, const T* s_in, const T* dsum, int64_t rows, int64_t cols, const float* gain,
                      const float* rstd, T* dx, float* dgain, float* partial, hipStream_t st) {
  const RowShape s = row_shape<T>(cols);
  const int grid = (int)backward_groups(rows, cols);
  const auto kernel = rows > (int64_t)kRun * grid ? by_chunks<BackwardRuns, T>(s.v) : by_chunks<BackwardOnce, T>(s.v);
  kernel<<<grid, s.threads, 0, st>>>(dy, s_in, dsum, (int)rows, (int)cols, gain, rstd, dx, partial);
  k_rmsnorm_dgain<<<(unsigned)(cols / 32), 1024, 0, st>>>(partial, grid, (int)cols, dgain);
}

}  // namespace

void launch_mxfp8(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                  hipStream_t st) {
  const int64_t chunks = rows * cols / (dtype == 1 ? 8 : 4);
  const unsigned grid = (unsigned)((chunks + 256 * kQuantChunks - 1) / (256 * kQuantChunks));
  if (dtype == 1) k_mxfp8<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(x), chunks, codes, scales);
  else k_mxfp8<float><<<grid, 256, 0, st>>>(static_cast<const float*>(x), chunks, codes, scales);
}

void launch_dequant_mxfp8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int out_dtype,
                          void* y, hipStream_t st) {
  const int64_t n8 = rows * cols / 8;
  const int64_t pieces = (n8 + 255) / 256;
  const unsigned grid = (unsigned)(pieces < (1 << 23) ? pieces : (1 << 23));
  if (out_dtype == 1) k_dequant_mxfp8<true><<<grid, 256, 0, st>>>(codes, scales, n8, y);
  else k_dequant_mxfp8<false><<<grid, 256, 0, st>>>(codes, scales, n8, y);
}

void launch_rmsnorm(const void* x, const void* residual, int dtype, int64_t rows, int64_t cols, const float* gain,
                    float eps, uint8_t* codes, uint8_t* scales, void* sum, float* rstd, void* y, hipStream_t st) {
  if (dtype == 1)
    rmsnorm(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual), rows, cols, gain, eps, codes,
            scales, static_cast<uint16_t*>(sum), rstd, static_cast<uint16_t*>(y), st);
  else
    rmsnorm(static_cast<const float*>(x), static_cast<const float*>(residual), rows, cols, gain, eps, codes, scales,
            static_cast<float*>(sum), rstd, static_cast<float*>(y), st);
}

int64_t rmsnorm_backward_scratch(int64_t rows, int64_t cols) {
  return backward_groups(rows, cols) * cols * 4;
}

void launch_rmsnorm_backward(const void* dy, const void* s, const void* dsum, int dtype, int64_t rows, int64_t cols,
                             const float* gain, const float* rstd, void* dx, float* dgain, void* scratch,
                             hipStream_t st) {
  float* partial = static_cast<float*>(scratch);
  if (dtype == 1)
    rmsnorm_backward(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(s),
                     static_cast<const uint16_t*>(dsum), rows, cols, gain, rstd, static_cast<uint16_t*>(dx), dgain,
                     partial, st);
  else
    rmsnorm_backward(static_cast<const float*>(dy), static_cast<const float*>(s), static_cast<const float*>(dsum),
                     rows, cols, gain, rstd, static_cast<float*>(dx), dgain, partial, st);
}

}  // namespace fp4q
