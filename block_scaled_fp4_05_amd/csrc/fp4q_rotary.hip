// Rotary positions: the table of cosines and sines, the rotation of queries and keys with its
// gradient, and the append of keys (rotated on the way) and values to a paged MXFP8 cache.
//
// A pair (x1, x2) of a head turns by the angle of its position and frequency:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin.
// The pairs of a head of `rot` rotated elements are (i, i + rot/2) in the half layout and
// (2i, 2i+1) in the interleaved one.  The map is m times a rotation, so its gradient is the same with -sin.
#include "fp4q_kv.hpp"
#include "fp4q_mx8.hpp"
#include "fp4q_mxfp8.hpp"

#include <type_traits>

namespace fp4q {
namespace {

// -----------------------------------------------------------------------------------------
// Table.  Angles of far positions need 64 bits (2^17 radians leave fp32 seven bits of the turn).
// A lane takes one frequency and kTableRun positions in a row: one sine and cosine of the first angle and of
// the frequency, then each next position by a product with the latter in binary64, whose rounding
// grows by about 2^-52 a step.  Bound by its stores: 131072 positions of 64 pairs (67 MB) 13.2 us, 5.1 TB/s (14.0 with
// ordinary ones).
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
    __builtin_nontemporal_store(f32x2{(float)(amplitude * c), (float)(amplitude * s)}, table + (p0 + j) * half + i);
    const double c1 = fma(c, dc, -(s * ds));
    s = fma(s, dc, c * ds);
    c = c1;
  }
}

// -----------------------------------------------------------------------------------------
// Rotation of x [tokens][heads][head_dim].  A lane's item is the same in every head it takes: a chunk (16
// bytes) of both halves' partners, a chunk of interleaved pairs, or a chunk that is copied; so its
// cosines and sines are loaded once for all of them.  Bound by memory: 8192 tokens of 40 heads of 128 in bf16 inside rows of
// 48 (172 MB) 30.0 us, 5.7 TB/s (33.5 with ordinary stores); 1021 tokens of 12 fp32 heads of 96, interleaved, 4 us, one
// launch and trip to memory.  A wave per token and five heads per lane: 36 us.
// -----------------------------------------------------------------------------------------
struct RotaryArgs {
  const void* x;
  void* y;
  const int32_t* positions;
  const f32x2* table;
  int64_t table_rows, x_token, x_head, y_token, y_head;   // strides in elements
  int heads, head_dim, half;
  float sign;   // 1, or -1 for the gradient
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

// Items of 16 bytes: rot/2 a multiple of the chunk in the half layout.  A workgroup takes a token: thread t has item
// t % items of heads t / items, + 256 / items, ...; the token's row of the table comes by way of LDS (see k_kv_append).
template <typename T, bool INTERLEAVED>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a) {
  constexpr int N = Chunk<T>::N, P = INTERLEAVED ? N / 2 : N;   // P: pairs per item
  extern __shared__ __align__(16) f32x2 row[];                  // [half]
  const int64_t t = blockIdx.x;
  const int pos = a.positions[t];
  if (pos < 0 || pos >= a.table_rows) return;   // padding
  for (int i = threadIdx.x; i < a.half; i += 256) row[i] = a.table[(int64_t)pos * a.half + i];
  const int rot = 2 * a.half;
  const int turned = INTERLEAVED ? a.head_dim / N : a.half / N;              // items with a rotation (interleaved: or a part of one)
  const int items = INTERLEAVED ? turned : turned + (a.head_dim - rot) / N;  // at most 256
  const int per = 256 / items, item = (int)threadIdx.x % items, h0 = (int)threadIdx.x / items;
  const bool turns = INTERLEAVED || item < turned;
  const int e = turns ? item * N : rot + (item - turned) * N;
  const T* x = static_cast<const T*>(a.x) + t * a.x_token + e;
  T* y = static_cast<T*>(a.y) + t * a.y_token + e;
  __syncthreads();
  if (h0 >= per) return;
  f32x2 cs[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const f32x2 v = row[min(item * P + i, a.half - 1)];
    cs[i] = f32x2{v.x, a.sign * v.y};
  }
  for (int h = h0; h < a.heads; h += per) {
    const T* p = x + h * a.x_head;
    T* q = y + h * a.y_head;
    const u32x4_t one = load_chunk(p);
    if (!turns) {
      store_chunk_nt(q, one);
      continue;
    }
    float u[N], o[N];
    unpack(one, u);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        turn(u[2 * i], u[2 * i + 1], cs[i], o[2 * i], o[2 * i + 1]);
        if (item * P + i >= a.half) o[2 * i] = u[2 * i], o[2 * i + 1] = u[2 * i + 1];   // past the rotated part
      }
    } else {
      float v[N], w[N];
      unpack(load_chunk(p + a.half), v);
#pragma unroll
      for (int i = 0; i < N; ++i) turn(u[i], v[i], cs[i], o[i], w[i]);
      store_chunk_nt(q + a.half, pack(w));
    }
    store_chunk_nt(q, pack(o));
  }
}

// Half layout where rot/2 is no multiple of the chunk: a lane has one pair, or one copied element, of the heads that its
// wave takes, wave w those of w, w + 4, ..., four of them in flight.
template <typename T>
__global__ __launch_bounds__(256) void k_rotary_pairs(RotaryArgs a) {
  constexpr int AHEAD = 4;
  const int64_t t = blockIdx.x;
  const int pos = a.positions[t], wave = threadIdx.x >> 6;
  if (pos < 0 || pos >= a.table_rows) return;
  const T* x = static_cast<const T*>(a.x) + t * a.x_token;
  T* y = static_cast<T*>(a.y) + t * a.y_token;
  const int items = a.head_dim - a.half;   // pairs, then the elements past the rotated part
  for (int e = threadIdx.x & 63; e < items; e += 64) {
    const bool pair = e < a.half;
    f32x2 cs = a.table[(int64_t)pos * a.half + (pair ? e : 0)];
    cs.y *= a.sign;
    for (int h0 = wave; h0 < a.heads; h0 += 4 * AHEAD) {
      T one[AHEAD], two[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const T* p = x + min(h0 + 4 * j, a.heads - 1) * a.x_head + e;
        two[j] = p[a.half];
        if (pair) one[j] = p[0];
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (h0 + 4 * j >= a.heads) break;
        T* p = y + (h0 + 4 * j) * a.y_head + e;
        if (pair) {
          float o, q;
          turn(widen(one[j]), widen(two[j]), cs, o, q);
          p[0] = narrow<T>(o), p[a.half] = narrow<T>(q);
        } else {
          p[a.half] = two[j];
        }
      }
    }
  }
}

// -----------------------------------------------------------------------------------------
// Append.  A workgroup takes kAppendTokens tokens; a lane one chunk (8 bf16 or 4 fp32) of each one's keys
// or values, so that neighbouring lanes hold the 32-element blocks as in the quantizer.
//
// A rotated key is rounded once, from the value of x1 cos - x2 sin.  In fp32 that value is off by some 2^-23 of it, which
// changes a code only next to a point halfway between two codes, or a scale next to its boundaries (1.75 2^k).  These have
// at most five significant bits, so a result whose last 19 are within kNear of zero (one in 2^15) is computed again:
// the products are exact in binary64, their difference is rounded to 53 bits and then to odd in fp32, which rounds to a
// code as the difference does.  (All in binary64: 13460 tokens of 8 heads of 128 in 32 us, against 25.)
// -----------------------------------------------------------------------------------------
constexpr int kAppendTokens = 2;

struct AppendArgs {
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const f32x2* table;
  int64_t table_rows;
  int half;
  const int32_t *positions, *q_starts, *kv_lens, *page_table;
  int tokens, seqs, max_pages, page_shift, heads, head_dim;
  int64_t pages;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
};

// fp32 next to r towards zero with its last bit set where r is no fp32 number: rounds to fewer bits as r does (past fp32's
// range its largest number).
__device__ __forceinline__ float to_odd(double r) {
  const float f = (float)r;
  const double back = (double)f;
  if (back == r) return f;
  const uint32_t b = __float_as_uint(f) - (__builtin_fabs(back) > __builtin_fabs(r) ? 1u : 0u);
  return __uint_as_float(b | 1u);
}

// x cos - other sin, rounded once in the sense of to_odd; other: an element's partner, its sign turned for the second
// element of a pair.
__device__ __forceinline__ float turned_exactly(float x, float other, f32x2 cs) {
  return to_odd(__builtin_fma((double)x, (double)cs.x, -((double)other * (double)cs.y)));
}
// In fp32, within three roundings of the result; `near` falls to kNearLimit or below where that may not do.
constexpr uint32_t kNear = 16;
constexpr uint32_t kNearLimit = (2 * kNear) << 13;   // of the last 19 bits in the upper ones' place
constexpr uint32_t kTiny = 30;   // and so it may in blocks with a scale code below this, whose results lose bits
__device__ __forceinline__ float turned(float x, float other, f32x2 cs, uint32_t& near) {
  const float far = other * cs.y;
  const float y = __builtin_fmaf(x, cs.x, -far) - __builtin_fmaf(other, cs.y, -far);
  near = min(near, (__float_as_uint(y) << 13) + (kNear << 13));
  return y;
}

// Where a token's keys and values go and its row of the table.
struct Place {
  int64_t row;     // (page heads << page_shift) + row in the page: head h is (h << page_shift) further; -1: nowhere
  int pos;         // -1: no such row
};

// Of token t in sequence s (-1: none) with kv positions, whose tokens end before q_end.
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t, int s, int q_end, int kv) {
  Place p{-1, -1};
  const int64_t at = (int64_t)kv - ((int64_t)q_end - t);   // its place in the sequence
  if (s < 0 || at < 0 || (at >> a.page_shift) >= a.max_pages) return p;
  const auto* table = (const __attribute__((address_space(4))) int32_t*)a.page_table;   // scalar loads
  const int page = table[(int64_t)s * a.max_pages + (at >> a.page_shift)];
  const int64_t pos = a.positions ? a.positions[t] : at;
  if (pos >= 0 && pos < a.table_rows) p.pos = (int)pos;
  if (page >= 0 && page < a.pages) p.row = (((int64_t)page * a.heads) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
  return p;
}

// Of the tokens t0, t0 + 1, ...: up to 63 sequences are held by the wave's lanes, in one trip to memory.
template <int TOKENS>
__device__ __forceinline__ void find_places(const AppendArgs& a, int t0, Place (&p)[TOKENS]) {
  const int lane = threadIdx.x & 63;
  if (a.seqs < 64) {
    const int start = a.q_starts[min(lane, a.seqs)], kv = a.kv_lens[min(lane, a.seqs - 1)];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int t = t0 + j, s = __popcll(__ballot(lane <= a.seqs && start <= t)) - 1;
      const bool some = s >= 0 && s < a.seqs && t < a.tokens;
      const int at = some ? s : 0;
      p[j] = place_of(a, t, some ? s : -1, __builtin_amdgcn_readlane(start, at + 1), __builtin_amdgcn_readlane(kv, at));
    }
  } else {
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int t = t0 + j, s = t < a.tokens ? __builtin_amdgcn_readfirstlane(wave_sequence(a.q_starts, a.seqs, t)) : -1;
      p[j] = place_of(a, t, s, s < 0 ? 0 : __builtin_amdgcn_readfirstlane(a.q_starts[s + 1]),
                      s < 0 ? 0 : __builtin_amdgcn_readfirstlane(a.kv_lens[s]));
    }
  }
}

template <int N>
__device__ __forceinline__ void put_codes(uint8_t* p, const uint32_t (&w)[N / 4]) {
  if constexpr (N == 8) *reinterpret_cast<u32x2_t*>(p) = u32x2_t{w[0], w[1]};
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// How keys are turned: not; in interleaved pairs; in halves, whose chunks meet chunks or not.
enum Layout { kPlain, kPairs, kHalfChunks, kHalfAny };

template <typename T, Layout L>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
  constexpr int N = Chunk<T>::N, LANES = Chunk<T>::LANES, TOKENS = kAppendTokens;
  extern __shared__ __align__(16) f32x2 rows[];   // [tokens][half]
  const int t0 = blockIdx.x * TOKENS, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = a.head_dim / N, chunks = a.heads * per, rot = 2 * a.half;
  // A lane's chunk is the same in every token: its loads go out before the tokens' places are known.
  Place place[TOKENS];
  for (int first = 0; first < 2 * chunks; first += 256) {
    const bool live = first + (int)threadIdx.x < 2 * chunks;
    const int i = min(first + (int)threadIdx.x, 2 * chunks - 1);
    const bool key = i < chunks;
    const int c = key ? i : i - chunks, h = c / per, e0 = (c - h * per) * N;
    const bool turns = L != kPlain && key && e0 < rot;
    const T* x = key ? static_cast<const T*>(a.k) + h * a.k_head + e0 : static_cast<const T*>(a.v) + h * a.v_head + e0;
    const int64_t step = key ? a.k_token : a.v_token;
    const int to_partner = e0 < a.half ? a.half : -a.half;
    u32x4_t own[TOKENS], partner[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const T* p = x + min(t0 + j, a.tokens - 1) * step;
      own[j] = load_chunk(p);
      if constexpr (L == kHalfChunks) partner[j] = turns ? load_chunk(p + to_partner) : own[j];
    }
    if (first == 0) find_places<TOKENS>(a, t0, place);
    if (L != kPlain && first == 0) {
      // The tokens' rows of the table by way of LDS: a lane's pairs lie 64 bytes from its neighbour's, which costs the
      // address unit as much as 64 lines for one load (13460 tokens of 8 heads of 128 in 32 us).
      for (int j = wave; j < TOKENS; j += 4) {
        int pos = place[0].pos;
#pragma unroll
        for (int k = 1; k < TOKENS; ++k) pos = j == k ? place[k].pos : pos;
        const f32x2* row = a.table + (int64_t)max(pos, 0) * a.half;
        for (int n = lane; n < a.half; n += 64) rows[j * a.half + n] = row[n];
      }
      __syncthreads();
    }
    const int pair = e0 >= a.half ? e0 - a.half : e0;
    const uint32_t signs = e0 < a.half ? 0u : sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
    const uint32_t in_page = (uint32_t)(h << a.page_shift) * (uint32_t)a.head_dim + (uint32_t)e0;
    uint8_t* codes = (key ? a.k_codes : a.v_codes) + in_page;
    uint8_t* scales = (key ? a.k_scales : a.v_scales) + in_page / 32;
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int64_t at = place[j].row;
      const int pos = place[j].pos;
      if (at < 0) continue;
      float v[N];
      uint32_t w[N / 4];
      unpack(own[j], v);
      if (L != kPlain && key && pos < 0) {   // no such row of the table: a key that no one takes for one
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = __builtin_nanf("");
      }
      uint32_t near = ~0u;
      // the chunk's elements through f(element, other, cosine and sine)
      auto turn_all = [&](auto f) {
        if constexpr (L == kPairs) {
          const f32x2* row = rows + j * a.half;
#pragma unroll
          for (int n = 0; n < N; n += 2) {
            if (e0 + n >= rot) continue;
            const f32x2 c_ = row[(e0 + n) >> 1];
            const float y0 = f(v[n], v[n + 1], c_), y1 = f(v[n + 1], -v[n], c_);
            v[n] = y0, v[n + 1] = y1;
          }
        } else if constexpr (L == kHalfChunks) {
          float u[N];
          unpack(partner[j] ^ signs, u);
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = f(v[n], u[n], rows[j * a.half + pair + n]);
        } else if constexpr (L == kHalfAny) {
          const T* p = x + (int64_t)(t0 + j) * step;
          const f32x2* row = rows + j * a.half;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const int e = e0 + n;
            const bool second = e >= a.half;
            if (e >= rot) continue;
            const float u = widen(p[n + (second ? -a.half : a.half)]);
            v[n] = f(v[n], second ? -u : u, row[second ? e - a.half : e]);
          }
        }
      };
      const bool turn_it = turns && pos >= 0;
      if (turn_it) turn_all([&](float x_, float w_, f32x2 c_) { return turned(x_, w_, c_, near); });
      uint32_t code = mx8_encode<T>(v, w);
      if constexpr (L != kPlain) {
        if (__builtin_expect(__any(turn_it && (near <= kNearLimit || code < kTiny)), 0)) {
          if (turn_it) {
            unpack(own[j], v);
            turn_all([&](float x_, float w_, f32x2 c_) { return turned_exactly(x_, w_, c_); });
          }
          code = mx8_encode<T>(v, w);
        }
      }
      const int64_t token = at * a.head_dim;
      if (live) put_codes<N>(codes + token, w);
      if (live && (threadIdx.x & (LANES - 1)) == 0) scales[token / 32] = (uint8_t)code;
    }
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
                     r.y_token, r.y_head, r.heads, r.head_dim, r.rot / 2, r.backward ? -1.0f : 1.0f};
  const unsigned grid = (unsigned)r.tokens, lds = (unsigned)a.half * 8u;
  const int n = r.dtype ? 8 : 4;
  if (r.interleaved) {
    if (r.dtype) k_rotary<uint16_t, true><<<grid, 256, lds, st>>>(a);
    else k_rotary<float, true><<<grid, 256, lds, st>>>(a);
  } else if (a.half % n == 0) {
    if (r.dtype) k_rotary<uint16_t, false><<<grid, 256, lds, st>>>(a);
    else k_rotary<float, false><<<grid, 256, lds, st>>>(a);
  } else {
    if (r.dtype) k_rotary_pairs<uint16_t><<<grid, 256, 0, st>>>(a);
    else k_rotary_pairs<float><<<grid, 256, 0, st>>>(a);
  }
}

template <typename T>
void append(const AppendArgs& a, Layout l, hipStream_t st) {
  const unsigned grid = (unsigned)((a.tokens + kAppendTokens - 1) / kAppendTokens);
  const unsigned lds = kAppendTokens * (unsigned)a.half * 8u;
  if (l == kPlain) k_kv_append<T, kPlain><<<grid, 256, 0, st>>>(a);
  else if (l == kPairs) k_kv_append<T, kPairs><<<grid, 256, lds, st>>>(a);
  else if (l == kHalfChunks) k_kv_append<T, kHalfChunks><<<grid, 256, lds, st>>>(a);
  else k_kv_append<T, kHalfAny><<<grid, 256, lds, st>>>(a);
}

void launch_kv_append(const KvCache& c, const KvBatch& b, const KvAppend& p, hipStream_t st) {
  const int n = p.dtype ? 8 : 4, half = p.table ? p.rot / 2 : 0;
  const AppendArgs a{p.k, p.v, p.k_token, p.k_head, p.v_token, p.v_head, reinterpret_cast<const f32x2*>(p.table),
                     p.table_rows, half, p.positions, b.q_starts, b.kv_lens, b.page_table, (int)p.tokens, (int)b.seqs,
                     (int)b.max_pages, c.page_shift, (int)c.heads, (int)c.head_dim, c.pages, c.k_codes, c.k_scales,
                     c.v_codes, c.v_scales};
  const Layout l = !p.table ? kPlain : p.interleaved ? kPairs : half % n == 0 ? kHalfChunks : kHalfAny;
  if (p.dtype) append<uint16_t>(a, l, st);
  else append<float>(a, l, st);
}

}  // namespace fp4q
