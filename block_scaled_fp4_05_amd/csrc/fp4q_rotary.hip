// Rotary positions: the table of cosines and sines, the rotation of queries and keys with its
// gradient, and the append of keys (rotated on the way) and values to a paged MXFP8 cache.
//
// A pair (x1, x2) of a head turns by the angle of its position and frequency:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin.
// The pairs of a head of `rot` rotated elements are (i, i + rot/2) in the half layout and
// (2i, 2i+1) in the interleaved one.  The map is m times a rotation, so its gradient is the same with -sin.
#include "fp4q_kv.hpp"
#include "fp4q_mxfp8.hpp"

#include <type_traits>

namespace fp4q {
namespace {

// -----------------------------------------------------------------------------------------
// Table.  Angles of far positions need 64 bits (2^17 radians leave fp32 seven bits of the turn).
// A lane takes one frequency and kTableRun positions in a row: one sine and cosine of the first angle and of
// the frequency, then each next position by a product with the latter in binary64, whose rounding
// grows by about 2^-52 a step.
// -----------------------------------------------------------------------------------------
constexpr int kTableRun = 16;

__global__ __launch_bounds__(256) void k_rotary_table(int64_t positions, int half, double base, double factor,
                                                      double original, double low, double high, double amplitude,
                                                      f32x2* __restrict__ table) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t run = at / half;
  const int i = (int)(at - run * half);
  const int64_t p0 = run * kTableRun;
  if (p0 >= positions) return;
  double f = pow(base, -(double)i / (double)half);
  if (factor != 1.0) {
    const double turns = original * f * 0.15915494309189533577;   // 1 / (2 pi)
    const double keep = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
    f *= keep + (1.0 - keep) / factor;
  }
  double s, c, ds, dc;
  sincos((double)p0 * f, &s, &c);
  sincos(f, &ds, &dc);
  for (int j = 0; j < kTableRun && p0 + j < positions; ++j) {
    table[(p0 + j) * half + i] = f32x2{(float)(amplitude * c), (float)(amplitude * s)};
    const double c1 = fma(c, dc, -(s * ds));
    s = fma(s, dc, c * ds);
    c = c1;
  }
}

// -----------------------------------------------------------------------------------------
// Rotation of x [tokens][heads][head_dim].  A lane's item is the same in every head it takes: a chunk (16
// bytes) of both halves' partners, a chunk of interleaved pairs, or a chunk that is copied; so its
// cosines and sines are loaded once for all of them.
// -----------------------------------------------------------------------------------------
struct RotaryArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  const f32x2* table;
  int64_t table_rows, x_token, x_head, y_token, y_head;   // strides in elements
  int64_t tokens;
  int heads, head_dim, half;
  float sign;   // 1, or -1 for the gradient
  bool interleaved;
};

__device__ __forceinline__ void turn(float a, float b, f32x2 cs, float& ya, float& yb) {
  ya = __builtin_fmaf(a, cs.x, -(b * cs.y));
  yb = __builtin_fmaf(b, cs.x, a * cs.y);
}

template <typename T>
__device__ __forceinline__ float widen(T v) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)v << 16);
  else return v;
}
template <typename T>
__device__ __forceinline__ T narrow(float v) {
  if constexpr (sizeof(T) == 2) return (uint16_t)to_bf16x2(v, 0.0f);
  else return v;
}

// Items of 16 bytes: rot/2 a multiple of the chunk in the half layout.  256 threads take one token: thread t
// has item t % items of heads t / items, + 256 / items, ...
template <typename T, bool INTERLEAVED>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a) {
  constexpr int N = Chunk<T>::N;
  const int64_t t = blockIdx.x;
  const int pos = a.positions[t];
  if (pos < 0 || pos >= a.table_rows) return;   // padding
  const int rot = 2 * a.half;
  const int turned = INTERLEAVED ? a.head_dim / N : a.half / N;              // items with a rotation (interleaved: or a part of one)
  const int items = INTERLEAVED ? turned : turned + (a.head_dim - rot) / N;
  const T* x = static_cast<const T*>(a.x) + t * a.x_token;
  T* y = static_cast<T*>(a.y) + t * a.y_token;
  for (int first = 0; first < items; first += 256) {   // one round unless a head has over 256 items
    const int now = min(items - first, 256), per = 256 / now;
    const int item = first + (int)threadIdx.x % now, h0 = (int)threadIdx.x / now;
    if (h0 >= per) continue;
    constexpr int P = INTERLEAVED ? N / 2 : N;   // pairs per item
    f32x2 cs[P];
    const f32x2* row = a.table + (int64_t)pos * a.half;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = item * P + i;
      const f32x2 v = row[min(p, a.half - 1)];
      cs[i] = p < a.half ? f32x2{v.x, a.sign * v.y} : f32x2{1.0f, 0.0f};
    }
    if (INTERLEAVED || item < turned) {
      for (int h = h0; h < a.heads; h += per) {
        const int64_t xa = h * a.x_head + item * N, ya = h * a.y_head + item * N;
        float u[N], o[N];
        if constexpr (INTERLEAVED) {
          unpack(load_chunk(x + xa), u);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            turn(u[2 * i], u[2 * i + 1], cs[i], o[2 * i], o[2 * i + 1]);
            if (item * P + i >= a.half) o[2 * i] = u[2 * i], o[2 * i + 1] = u[2 * i + 1];   // past the rotated part
          }
          *reinterpret_cast<u32x4_t*>(y + ya) = pack(o);
        } else {
          float v[N], q[N];
          unpack(load_chunk(x + xa), u);
          unpack(load_chunk(x + xa + a.half), v);
#pragma unroll
          for (int i = 0; i < N; ++i) turn(u[i], v[i], cs[i], o[i], q[i]);
          *reinterpret_cast<u32x4_t*>(y + ya) = pack(o);
          *reinterpret_cast<u32x4_t*>(y + ya + a.half) = pack(q);
        }
      }
    } else {
      const int e = rot + (item - turned) * N;
      for (int h = h0; h < a.heads; h += per)
        *reinterpret_cast<u32x4_t*>(y + h * a.y_head + e) = load_chunk(x + h * a.x_head + e);
    }
  }
}

// Half layout where rot/2 is no multiple of the chunk: one pair, or one copied element, per item.
template <typename T>
__global__ __launch_bounds__(256) void k_rotary_pairs(RotaryArgs a) {
  const int64_t t = blockIdx.x;
  const int pos = a.positions[t];
  if (pos < 0 || pos >= a.table_rows) return;
  const T* x = static_cast<const T*>(a.x) + t * a.x_token;
  T* y = static_cast<T*>(a.y) + t * a.y_token;
  const int items = a.head_dim - a.half;   // pairs, then the elements past the rotated part
  for (int i = threadIdx.x; i < items * a.heads; i += 256) {
    const int h = i / items, e = i - h * items;
    const T* xh = x + h * a.x_head;
    T* yh = y + h * a.y_head;
    if (e < a.half) {
      const f32x2 v = a.table[(int64_t)pos * a.half + e];
      float o, q;
      turn(widen(xh[e]), widen(xh[e + a.half]), f32x2{v.x, a.sign * v.y}, o, q);
      yh[e] = narrow<T>(o), yh[e + a.half] = narrow<T>(q);
    } else {
      yh[e + a.half] = xh[e + a.half];
    }
  }
}

// -----------------------------------------------------------------------------------------
// Append.  One workgroup per token; a lane takes one chunk (8 bf16 or 4 fp32) of the token's keys
// or values, so that neighbouring lanes hold the 32-element blocks as in the quantizer.
//
// A rotated key is rounded once, from the value of x1 cos - x2 sin: the products are exact in binary64, their
// difference is rounded to 53 bits and then to odd in fp32, which E4M3's rounding does not see.
// -----------------------------------------------------------------------------------------
struct AppendArgs {
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const f32x2* table;
  int64_t table_rows;
  int half;
  bool interleaved, aligned;   // aligned: a chunk's partners are a chunk
  const int32_t *positions, *q_starts, *kv_lens, *page_table;
  int seqs, max_pages, page_shift, heads, head_dim;
  int64_t pages;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
};

// fp32 next to r towards zero with its last bit set where r is no fp32 number: rounds to fewer bits as r does.
__device__ __forceinline__ float to_odd(double r) {
  const float f = (float)r;
  const double back = (double)f;
  if (back == r) return f;
  const uint32_t b = __float_as_uint(f) - (__builtin_fabs(back) > __builtin_fabs(r) ? 1u : 0u);
  return __uint_as_float(b | 1u);
}

template <typename T>
__device__ __forceinline__ void turned_key(const T* __restrict__ x, int e0, const f32x2* __restrict__ row, int half,
                                           bool interleaved, bool aligned, float (&v)[Chunk<T>::N]) {
  constexpr int N = Chunk<T>::N;
  unpack(load_chunk(x + e0), v);
  if (e0 >= 2 * half) return;
  float w[N];
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = v[i ^ 1];
  } else if (aligned) {
    unpack(load_chunk(x + (e0 < half ? e0 + half : e0 - half)), w);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + i;
      w[i] = e < 2 * half ? widen(x[e < half ? e + half : e - half]) : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i;
    const bool second = interleaved ? (i & 1) != 0 : e >= half;
    const int p = interleaved ? e >> 1 : second ? e - half : e;
    if (e < 2 * half) {
      const f32x2 cs = row[p];
      const double far = (double)w[i] * (double)cs.y;
      v[i] = to_odd(__builtin_fma((double)v[i], (double)cs.x, second ? far : -far));
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
  constexpr int N = Chunk<T>::N, LANES = Chunk<T>::LANES;
  const int t = blockIdx.x;
  const int s = wave_sequence(a.q_starts, a.seqs, t);
  if (s < 0) return;
  const int end = a.q_starts[s + 1];
  const int64_t place = (int64_t)a.kv_lens[s] - ((int64_t)end - t);   // the token's in its sequence
  if (place < 0 || (place >> a.page_shift) >= a.max_pages) return;
  const int at = (int)place;
  const int page = a.page_table[(int64_t)s * a.max_pages + (at >> a.page_shift)];
  if (page < 0 || page >= a.pages) return;
  const int pos = a.positions ? a.positions[t] : at;
  const bool known = pos >= 0 && pos < a.table_rows;
  const f32x2* row = a.table + (known ? (int64_t)pos * a.half : 0);
  const int per = a.head_dim / N, chunks = a.heads * per;
  const int in_page = at & ((1 << a.page_shift) - 1);
  // whole blocks per wave: 2 * chunks is a multiple of LANES, and so is 256
  for (int i = threadIdx.x; i < 2 * chunks; i += 256) {
    const bool key = i < chunks;
    const int c = key ? i : i - chunks, h = c / per, e0 = (c - h * per) * N;
    float v[N];
    uint32_t w[N / 4];
    if (key) {
      const T* x = static_cast<const T*>(a.k) + t * a.k_token + h * a.k_head;
      if (a.table && known) {
        turned_key(x, e0, row, a.half, a.interleaved, a.aligned, v);
      } else {
        unpack(load_chunk(x + e0), v);
        if (a.table) {   // no such row of the table: a key that no one takes for one
#pragma unroll
          for (int j = 0; j < N; ++j) v[j] = __builtin_nanf("");
        }
      }
    } else {
      unpack(load_chunk(static_cast<const T*>(a.v) + t * a.v_token + h * a.v_head + e0), v);
    }
    const uint32_t code = mx8_encode<T>(v, w);
    const int64_t r = (((int64_t)page * a.heads + h) << a.page_shift) + in_page;
    uint8_t* codes = (key ? a.k_codes : a.v_codes) + r * a.head_dim + e0;
    if constexpr (N == 8) *reinterpret_cast<u32x2_t*>(codes) = u32x2_t{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(codes) = w[0];
    if ((threadIdx.x & (LANES - 1)) == 0) (key ? a.k_scales : a.v_scales)[r * (a.head_dim / 32) + e0 / 32] = (uint8_t)code;
  }
}

}  // namespace

void launch_rotary_table(int64_t positions, int rot, double base, double factor, double original, double low,
                         double high, double amplitude, float* table, hipStream_t st) {
  const int half = rot / 2;
  const int64_t threads = (positions + kTableRun - 1) / kTableRun * half;
  k_rotary_table<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(positions, half, base, factor, original, low, high,
                                                                   amplitude, reinterpret_cast<f32x2*>(table));
}

void launch_rotary(const Rotary& r, hipStream_t st) {
  const RotaryArgs a{r.x, r.y, r.positions, reinterpret_cast<const f32x2*>(r.table), r.table_rows, r.x_token, r.x_head,
                     r.y_token, r.y_head, r.tokens, r.heads, r.head_dim, r.rot / 2, r.backward ? -1.0f : 1.0f,
                     r.interleaved};
  const unsigned grid = (unsigned)r.tokens;
  const int n = r.dtype ? 8 : 4;
  if (r.interleaved) {
    if (r.dtype) k_rotary<uint16_t, true><<<grid, 256, 0, st>>>(a);
    else k_rotary<float, true><<<grid, 256, 0, st>>>(a);
  } else if (a.half % n == 0) {
    if (r.dtype) k_rotary<uint16_t, false><<<grid, 256, 0, st>>>(a);
    else k_rotary<float, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (r.dtype) k_rotary_pairs<uint16_t><<<grid, 256, 0, st>>>(a);
    else k_rotary_pairs<float><<<grid, 256, 0, st>>>(a);
  }
}

void launch_kv_append(const KvCache& c, const KvBatch& b, const KvAppend& p, hipStream_t st) {
  const int n = p.dtype ? 8 : 4, half = p.table ? p.rot / 2 : 0;
  const AppendArgs a{p.k, p.v, p.k_token, p.k_head, p.v_token, p.v_head, reinterpret_cast<const f32x2*>(p.table),
                     p.table_rows, half, p.interleaved, half % n == 0, p.positions, b.q_starts, b.kv_lens,
                     b.page_table, (int)b.seqs, (int)b.max_pages, c.page_shift, (int)c.heads, (int)c.head_dim, c.pages,
                     c.k_codes, c.k_scales, c.v_codes, c.v_scales};
  const unsigned grid = (unsigned)p.tokens;
  if (p.dtype) k_kv_append<uint16_t><<<grid, 256, 0, st>>>(a);
  else k_kv_append<float><<<grid, 256, 0, st>>>(a);
}

}  // namespace fp4q
