// Attention over a paged MXFP8 cache of keys and values.
//
// For a query row q with the keys lo <= j < hi of its sequence:
//   s_j = scale q . k_j,  m = max s_j,  p_j = exp(s_j - m),  l = sum p_j,
//   o = sum p_j v_j / l,  lse = m + ln l.
// One pass over the keys with running m, l and o: where m rises, l and o are multiplied by exp(old m - m).
// Parts of the keys that different waves, workgroups or passes took are joined by the same rule.
//
// The queries of one key/value head (all of its query heads, of all the tokens of an item) are the
// rows of one product.  S^T = K Q^T and O^T = V^T P^T run on the bf16 MFMA with fp32 sums: E4M3 times a power of two
// is exact in bf16, so the codes are converted as they are used, the queries are bf16 already, and only P is rounded
// to it (half a step, 2^-8 of each p_j at most; l sums the unrounded ones).  (S on the block-scaled MFMA, from the
// codes as they lie and the queries split into two E4M3 parts, needs no conversion of keys and as many MFMA cycles, but
// its cut of the products left 1e-6 to 5e-6 of lse against 1e-7.)  S^T leaves a lane the scores of one row
// and four neighbouring keys per 16, which is the layout that P^T's operand needs, given that V^T's takes its keys
// in the same order.
#include "fp4q_dev.hpp"
#include "fp4q_kv.hpp"
#include "fp4q_mx8.hpp"

#include <algorithm>

namespace fp4q {
namespace {

typedef short v4s_a __attribute__((ext_vector_type(4)));
typedef __bf16 v8b_a __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_a __attribute__((ext_vector_type(4)));

constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 32;       // keys that a wave takes at a time
constexpr int kWaves = 4;
constexpr int kHalf = 16;       // keys of one MFMA, from a multiple of 16 on: never in two pages, whose least size it is
constexpr int kMaxPages = 4096; // page ids of a workgroup's keys

struct AttnArgs {
  const uint16_t* q;
  int64_t q_token, q_head;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t *q_starts, *kv_lens, *page_table, *group_starts, *shared_lens;
  int64_t pages, max_kv, max_shared;
  int max_q, tokens, seqs, groups, kv_heads, per_kv, page_shift, max_pages, window;
  bool causal, shared_pass;   // shared_pass: the items are groups and their shared keys
  int chunk, chunks, row_tiles;             // keys per workgroup, workgroups per row tile, row tiles per item
  int most_chunks, shared_chunk;            // of the own pass; keys per workgroup of the shared pass
  float scale_log2;                         // scale log2(e)
  uint16_t* out;
  float *lse, *part_o, *part_ml;            // partial results: [slot][token][head][head_dim], [..][2]
};

// The keys that an item's workgroups go through, from a multiple of 16 on.
struct Range {
  int first, end;
};

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Shared keys of a group: whole pages, no more than the call's bound covers.
__device__ __forceinline__ int shared_keys(const AttnArgs& a, int group) {
  const int n = clamp_to(a.shared_lens[group], 0, (int)a.max_shared);
  return n >> a.page_shift << a.page_shift;
}

// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const AttnArgs& a, int s) {
  if (a.groups == 0) return -1;
  const int g = lane_find(a.group_starts, a.groups, s);
  return g >= 0 && s < a.group_starts[g + 1] ? g : -1;
}

// Own keys of a sequence: what its group does not share, from the first that its window's first query sees.
// A length out of bounds gives no keys (and NaN, see `broken`).
__device__ __forceinline__ bool broken(const AttnArgs& a, int kv) { return kv < 0 || kv > a.max_kv; }
__device__ __forceinline__ Range own_range(const AttnArgs& a, int kv, int q_len, int shared) {
  if (broken(a, kv)) return Range{0, 0};
  int first = shared;
  if (a.window > 0) first = max(first, kv - min(q_len, a.max_q) + 1 - a.window);
  first = min(first, kv) & ~(kHalf - 1);
  return Range{first, kv};
}
__device__ __forceinline__ int own_chunks(const AttnArgs& a, Range r) {
  return clamp_to((r.end - r.first + a.chunk - 1) / a.chunk, 1, a.most_chunks);
}
__device__ __forceinline__ int shared_chunks(const AttnArgs& a, int shared) {
  return (shared + a.shared_chunk - 1) / a.shared_chunk;
}

// The keys lo .. hi-1 that the query token t of sequence s sees.
__device__ __forceinline__ Range visible(const AttnArgs& a, int s, int t) {
  const int kv = a.kv_lens[s];
  if (broken(a, kv)) return Range{0, 0};
  const int64_t pos = (int64_t)kv - ((int64_t)a.q_starts[s + 1] - t);
  Range r{0, kv};
  if (a.causal) r.end = (int)max((int64_t)0, min(pos + 1, (int64_t)kv));
  if (a.window > 0) r.first = (int)max((int64_t)0, min(pos + 1 - a.window, (int64_t)kv));
  return r;
}

// Maximum and sum over the lanes l, l ^ 16, l ^ 32, l ^ 48, the same bits in all four.
__device__ __forceinline__ float quad_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float m = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Whether one of 16 E4M3 codes under this scale may be no finite number: a NaN code, or a scale past which
// 448 overflows.
__device__ __forceinline__ bool suspect(const u32x4_m& w, uint32_t scale) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return any != 0 || scale > 246u;
}

// 16 E4M3 codes to bf16 (exact where the value is normal; a product past the range is infinite).
__device__ __forceinline__ void to_bf16(const u32x4_m& w, uint32_t scale, u32x4_m (&o)[2]) {
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, false));
    o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, true));
  }
}
// Per half word: all ones where a bf16 is infinite or NaN.
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  const uint32_t lo = (v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
  return lo | hi;
}

// Four rows and 16 columns of bf16 in LDS, transposed: lane i of 16 gives the place of columns 4 (i % 4) .. + 3 of
// row i / 4 and gets column i of the four rows.
__device__ __forceinline__ v4s_a read_transposed(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s_a*)(__attribute__((address_space(3))) void*)p);
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// -----------------------------------------------------------------------------------------
// Few rows per key/value head: the keys' bytes are what counts.  A workgroup takes `chunk` keys of one
// head; each of its four waves takes every fourth tile of 32 keys for all 16 R rows, with the next tile's loads in
// flight, and no barrier until the waves' results are joined at the end.
// -----------------------------------------------------------------------------------------
template <int D>
struct Wave {
  static constexpr int ROW = 2 * D + 32;           // bytes of a row of V in LDS: 16 rows' 32-byte pieces on different banks
  static constexpr int LOADS = D / 64;             // 16-byte loads per lane for 16 rows of K or V
  static constexpr int SB = D / 32;                // scale bytes of a row
  static constexpr int LINE = D / 16;              // lanes to a row of V
};

template <int D>
struct Fetch {   // one tile
  u32x4_m k[2][Wave<D>::LOADS], v[2][Wave<D>::LOADS];
  uint32_t ks[2][D == 256 ? 2 : 1], vs[2][Wave<D>::LOADS];   // ks: the scale bytes of a lane's row
};

template <int D, int R>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_stream(AttnArgs a) {
  using W = Wave<D>;
  __shared__ __align__(16) uint8_t lds_v[kWaves][kTile * W::ROW];
  __shared__ float lds_ml[kWaves][16 * R][2];
  extern __shared__ int lds_page[];   // the chunk's pages

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g4 = lane >> 4;
  int id = blockIdx.x;
  const int chunk_at = id % a.chunks;
  id /= a.chunks;
  const int row_tile = id % a.row_tiles;
  id /= a.row_tiles;
  const int head = id % a.kv_heads, item = id / a.kv_heads;

  // The item's rows and keys.
  int s0, t0, t1, slot = 0;   // first sequence, tokens
  Range range;
  bool direct = false, bad = false;
  if (a.shared_pass) {
    s0 = clamp_to(a.group_starts[item], 0, a.seqs);
    const int s1 = clamp_to(a.group_starts[item + 1], s0, a.seqs);
    t0 = clamp_to(a.q_starts[s0], 0, a.tokens), t1 = clamp_to(a.q_starts[s1], t0, a.tokens);
    range = Range{0, shared_keys(a, item)};
    if (s1 == s0) return;
    slot = chunk_at;
    if (chunk_at >= shared_chunks(a, range.end)) return;
  } else {
    s0 = item;
    t0 = clamp_to(a.q_starts[s0], 0, a.tokens), t1 = clamp_to(a.q_starts[s0 + 1], t0, a.tokens);
    const int g = group_of(a, s0), shared = g >= 0 ? shared_keys(a, g) : 0, kv = a.kv_lens[s0];
    bad = broken(a, kv);
    range = own_range(a, kv, t1 - t0, shared);
    const int mine = own_chunks(a, range), before = shared_chunks(a, shared);
    if (chunk_at >= mine) return;
    direct = mine + before == 1;
    slot = before + chunk_at;
  }
  const int rows = (a.shared_pass ? t1 - t0 : min(t1 - t0, a.max_q)) * a.per_kv, row0 = row_tile * 16 * R;
  if (row0 >= rows) return;
  const int c0 = range.first + chunk_at * (a.shared_pass ? a.shared_chunk : a.chunk);
  const int c1 = min(c0 + (a.shared_pass ? a.shared_chunk : a.chunk), range.end);

  // Pages of the chunk; an id that is none counts as -1.
  const int p0 = c0 >> a.page_shift, np = c1 > c0 ? ((c1 - 1) >> a.page_shift) - p0 + 1 : 0;
  for (int i = threadIdx.x; i < np; i += 256) {
    const int id_ = p0 + i < a.max_pages ? a.page_table[(int64_t)s0 * a.max_pages + p0 + i] : -1;
    lds_page[i] = id_ < 0 || id_ >= a.pages ? -1 : id_;
  }

  // Queries, the MFMA's second operand: lane (n, g4) holds elements 64 i + 16 g4 .. + 15 of row n, as it does of the keys.
  v8b_a qf[R][W::LOADS][2];
  int lo[R], hi[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + n, rows - 1);   // behind the last row: that one again, not stored
    const int t = t0 + row / a.per_kv, h = head * a.per_kv + row % a.per_kv;
    const Range seen = visible(a, a.shared_pass ? clamp_to(lane_find(a.q_starts, a.seqs, t), 0, a.seqs - 1) : s0, t);
    lo[r] = seen.first, hi[r] = min(seen.end, c1);
    const uint16_t* x = a.q + t * a.q_token + h * a.q_head;
#pragma unroll
    for (int i = 0; i < W::LOADS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) qf[r][i][j] = *reinterpret_cast<const v8b_a*>(x + 64 * i + 16 * g4 + 8 * j);
  }
  // Keys that some row sees, and those that all do.
  int lo_min = lo[0], lo_max = lo[0], hi_min = hi[0], hi_max = hi[0];
#pragma unroll
  for (int r = 1; r < R; ++r) {
    lo_min = min(lo_min, lo[r]), lo_max = max(lo_max, lo[r]), hi_min = min(hi_min, hi[r]), hi_max = max(hi_max, hi[r]);
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) {
    lo_min = min(lo_min, __shfl_xor(lo_min, x, 64)), lo_max = max(lo_max, __shfl_xor(lo_max, x, 64));
    hi_min = min(hi_min, __shfl_xor(hi_min, x, 64)), hi_max = max(hi_max, __shfl_xor(hi_max, x, 64));
  }
  lo_min = __builtin_amdgcn_readfirstlane(lo_min), lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min), hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  __syncthreads();

  const int64_t head_rows = (int64_t)1 << a.page_shift;
  auto fetch = [&](int key0, Fetch<D>& f) {   // keys key0 .. key0 + 31; past the chunk's pages: those of its last
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int key = key0 + 16 * b, at = min((key >> a.page_shift) - p0, np - 1);
      const int page = __builtin_amdgcn_readfirstlane(lds_page[at]);
      const int64_t r0 = ((int64_t)max(page, 0) * a.kv_heads + head) * head_rows + (key & (int)(head_rows - 1));
      const uint8_t *kc = a.k_codes + r0 * D, *vc = a.v_codes + r0 * D, *ks = a.k_scales + r0 * W::SB,
                    *vs = a.v_scales + r0 * W::SB;
#pragma unroll
      for (int i = 0; i < W::LOADS; ++i) {
        f.k[b][i] = load16(kc, (uint32_t)(n * D + 64 * i + 16 * g4));
        f.v[b][i] = load16(vc, (uint32_t)(1024 * i + 16 * lane));
        f.vs[b][i] = vs[(64 / W::LINE * i + lane / W::LINE) * W::SB + (lane % W::LINE) / 2];
      }
      if constexpr (D == 64) {
        f.ks[b][0] = *reinterpret_cast<const uint16_t*>(ks + n * 2);
      } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) f.ks[b][i] = *reinterpret_cast<const uint32_t*>(ks + n * W::SB + 4 * i);
      }
      if (page < 0) {
#pragma unroll
        for (uint32_t& w : f.ks[b]) w = 0xFFFFFFFFu;
      }
    }
  };

  v4f_m acc[R][D / 16];
  float m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -kInf, l[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[r][i] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  }
  uint8_t* mine = lds_v[wave];
  // Where a lane's transposed reads start: key 4 g4 + n / 4, elements 4 (n % 4) ..
  const uint8_t* tr = mine + (4 * g4 + (n >> 2)) * W::ROW + 8 * (n & 3);

  const int begin = c0 + kTile * wave, stop = min(c1, hi_max);
  Fetch<D> f;
  if (begin < stop) fetch(begin, f);
  for (int key0 = begin; key0 < stop; key0 += kTile * kWaves) {
    const Fetch<D> now = f;
    if (key0 + kTile * kWaves < stop) fetch(key0 + kTile * kWaves, f);
    if (key0 + kTile <= lo_min) continue;
    const bool edge = key0 < lo_max || key0 + kTile > hi_min;   // some row does not see some key

    // Values to LDS as bf16.  Rows behind the chunk may hold anything: they become zeros.
    u32x4_m vb[2][W::LOADS][2];
    bool odd = false;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < W::LOADS; ++i) {
        u32x4_m w = now.v[b][i];
        uint32_t sc = now.vs[b][i];
        if (edge) {
          if (key0 + 16 * b + 64 / W::LINE * i + lane / W::LINE >= c1) w = u32x4_m{0u, 0u, 0u, 0u}, sc = 127u;
          odd |= suspect(w, sc);
        }
        to_bf16(w, sc, vb[b][i]);
      }
    odd = edge && __any(odd);
    auto put = [&](bool zero_odd, bool marks) {
      wave_lds_fence();
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < W::LOADS; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            u32x4_m w = vb[b][i][j];
            if (zero_odd || marks) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t o = odd_halves(w[e]);
                w[e] = marks ? o & 0x3F803F80u : w[e] & ~o;
              }
            }
            *reinterpret_cast<u32x4_m*>(mine + (16 * b + 64 / W::LINE * i + lane / W::LINE) * W::ROW +
                                        32 * (lane % W::LINE) + 16 * j) = w;
          }
      wave_lds_fence();
    };
    put(odd, false);

    // Scores: register j of half b is key key0 + 16 b + 4 g4 + j, row n.
    v4f_m s4[R][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int r = 0; r < R; ++r) s4[r][b] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < W::LOADS; ++i) {   // elements 64 i + 16 g4 ..: the row's scale byte 2 i + g4 / 2
        u32x4_m kb[2];
        to_bf16(now.k[b][i], now.ks[b][i / 2] >> (16 * (i & 1) + 8 * (g4 >> 1)) & 0xFFu, kb);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < R; ++r)
            s4[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b_a, kb[j]), qf[r][i][j], s4[r][b], 0, 0, 0);
      }
    }
    v8b_a p[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float sc[8];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4f_m c = s4[r][b];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[4 * b + j] = c[j] * a.scale_log2;
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = key0 + 16 * (i >> 2) + 4 * g4 + (i & 3);
          if (key < lo[r] || key >= hi[r]) sc[i] = -kInf;
        }
      }
      float top = sc[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, sc[i]);
      const float mt = __builtin_fmaxf(m[r], quad_max(top));
      if (__any(mt > m[r])) {
        const float keep = mt == -kInf ? 1.0f : exp2_of(m[r] - mt);
        m[r] = mt, l[r] *= keep;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc[r][i] *= keep;
      }
      const float base = m[r] == -kInf ? 0.0f : m[r];
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = exp2_of(sc[2 * i] - base), y = exp2_of(sc[2 * i + 1] - base);
        l[r] += x + y;
        w[i] = bf16_pair(x, y);
      }
      p[r] = __builtin_bit_cast(v8b_a, u32x4_m{w[0], w[1], w[2], w[3]});
    }
    // O^T += V^T P^T, 16 elements of the head at a time.
    auto product = [&](int i, const v8b_a& pr, v4f_m c) {
      const v4s_a x = read_transposed(tr + 32 * i), y = read_transposed(tr + 16 * W::ROW + 32 * i);
      const v8b_a vf = __builtin_bit_cast(v8b_a, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pr, c, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r][i] = product(i, p[r], acc[r][i]);
    if (__builtin_expect(odd, 0)) {
      // Values that are no finite numbers, in a tile that not every row sees whole: 0 times them would be NaN, so
      // the product above took zeros in their place, and the rows that see one get a NaN here.
      put(false, true);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint32_t see[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 16 * (i >> 1) + 4 * g4 + 2 * (i & 1);
          see[i] = (key >= lo[r] && key < hi[r] ? 0x3F80u : 0u) | (key + 1 >= lo[r] && key + 1 < hi[r] ? 0x3F800000u : 0u);
        }
        const v8b_a pr = __builtin_bit_cast(v8b_a, u32x4_m{see[0], see[1], see[2], see[3]});
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const v4f_m hit = product(i, pr, v4f_m{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (hit[j] > 0.0f) acc[r][i][j] = __builtin_nanf("");
        }
      }
    }
  }

  // Join the waves in their order.
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float sum = quad_sum(l[r]);
    if (g4 == 0) lds_ml[wave][16 * r + n][0] = m[r], lds_ml[wave][16 * r + n][1] = sum;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // 16 rows of D floats per wave in the place of its values
    wave_lds_fence();
    float* o = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<v4f_m*>(o + n * (D + 4) + 16 * i + 4 * g4) = acc[r][i];
    __syncthreads();
    constexpr int PER = 16 * D / 256;   // elements per thread, of one row
    const int row = threadIdx.x / (256 / 16), e0 = (threadIdx.x % 16) * PER, at = row0 + 16 * r + row;
    if (at < rows) {
      float top = -kInf, sum = 0.0f, v[PER];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, lds_ml[w][16 * r + row][0]);
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = lds_ml[w][16 * r + row][0], f_ = mw == -kInf ? 0.0f : exp2_of(mw - top);
        sum += f_ * lds_ml[w][16 * r + row][1];   // 0 times a NaN stays one
        const float* src = reinterpret_cast<const float*>(lds_v[w]) + row * (D + 4) + e0;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = __builtin_fmaf(f_, src[e], v[e]);
      }
      const int t = t0 + at / a.per_kv, h = head * a.per_kv + at % a.per_kv;
      const int64_t place = (int64_t)t * a.kv_heads * a.per_kv + h;
      if (direct) {
        // nothing seen: zeros; only scores of -infinity, or a length out of bounds: NaN
        const Range seen = visible(a, s0, t);
        float inv = 1.0f / sum, out_lse = (top + __builtin_amdgcn_logf(sum)) * kLn2;
        if (sum == 0.0f) {
          const bool none = seen.end <= seen.first && !bad;
          inv = none ? 0.0f : __builtin_nanf(""), out_lse = none ? -kInf : __builtin_nanf("");
        }
#pragma unroll
        for (int e = 0; e < PER; e += 4)
          *reinterpret_cast<u32x2_m*>(a.out + place * D + e0 + e) =
              u32x2_m{bf16_pair(v[e] * inv, v[e + 1] * inv), bf16_pair(v[e + 2] * inv, v[e + 3] * inv)};
        if (a.lse && e0 == 0) a.lse[place] = out_lse;
      } else {
        const int64_t p = (int64_t)slot * a.tokens * a.kv_heads * a.per_kv + place;
#pragma unroll
        for (int e = 0; e < PER; e += 4) *reinterpret_cast<v4f_m*>(a.part_o + p * D + e0 + e) = v4f_m{v[e], v[e + 1], v[e + 2], v[e + 3]};
        if (e0 == 0) *reinterpret_cast<f32x2_m*>(a.part_ml + 2 * p) = f32x2_m{top, sum};
      }
    }
    __syncthreads();
  }
}

// Joins the slots of each row in their order: one wave per query row.  Slots: those of its group's shared keys, then
// its sequence's own.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  const int q_heads = a.kv_heads * a.per_kv, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), all = (int64_t)a.tokens * q_heads;
  if (row >= all) return;
  const int t = __builtin_amdgcn_readfirstlane((int)(row / q_heads));
  const int s = wave_find(a.q_starts, a.seqs, t);
  if (s < 0 || t >= a.q_starts[s + 1]) return;   // no sequence's token
  const int t0 = clamp_to(a.q_starts[s], 0, a.tokens), t1 = clamp_to(a.q_starts[s + 1], t0, a.tokens);
  if (t - t0 >= a.max_q) return;   // past the call's bound: not computed
  const int g = group_of(a, s), shared = g >= 0 ? shared_keys(a, g) : 0, kv = a.kv_lens[s];
  const int slots = shared_chunks(a, shared) + own_chunks(a, own_range(a, kv, t1 - t0, shared));
  if (slots == 1) return;   // written already
  constexpr int PER = D / 64;
  float top = -kInf, sum = 0.0f, v[PER];
  for (int i = 0; i < slots; ++i) top = __builtin_fmaxf(top, a.part_ml[2 * (i * all + row)]);
#pragma unroll
  for (int e = 0; e < PER; ++e) v[e] = 0.0f;
  for (int i = 0; i < slots; ++i) {
    const int64_t p = i * all + row;
    const float m = a.part_ml[2 * p], f = m == -kInf ? 0.0f : exp2_of(m - top);
    sum += f * a.part_ml[2 * p + 1];
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = __builtin_fmaf(f, a.part_o[p * D + PER * lane + e], v[e]);
  }
  float inv = 1.0f / sum, out_lse = (top + __builtin_amdgcn_logf(sum)) * kLn2;
  if (sum == 0.0f) {
    const Range seen = visible(a, s, t);
    const bool none = seen.end <= seen.first && !broken(a, kv);
    inv = none ? 0.0f : __builtin_nanf(""), out_lse = none ? -kInf : __builtin_nanf("");
  }
  uint16_t* o = a.out + row * D + PER * lane;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = (uint16_t)bf16_pair(v[e] * inv, 0.0f);
  if (a.lse && lane == 0) a.lse[row] = out_lse;
}

// How a pass is cut: rows per workgroup, keys per workgroup.
struct Cut {
  int r, row_tiles, chunk, chunks;
  int64_t grid;
};
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in one launch
constexpr int kFill = 1024;                            // workgroups that fill the card twice over

// `rows` and `keys`: the most that one of the `items` has.  Keys are split only until the card is full.
Cut cut(int64_t items, const KvCache& cache, int64_t rows, int64_t keys) {
  Cut c;
  c.r = rows <= 16 || cache.head_dim > 128 ? 1 : 2;   // (two 16-row tiles of 256 elements spill registers)
  c.row_tiles = (int)std::min<int64_t>((rows + 16 * c.r - 1) / (16 * c.r), INT32_MAX);
  const int64_t units = items * cache.heads * c.row_tiles, step = kTile * kWaves;
  const int64_t want = std::max<int64_t>(1, kFill / units);
  int64_t chunk = (keys + want - 1) / want;
  // lengths differ: pieces that are all alike keep the longest sequence from being the last
  if (c.row_tiles == 1) chunk = std::min<int64_t>(chunk, std::max<int64_t>(2048, keys / 64));
  chunk = std::max<int64_t>(step, (chunk + step - 1) / step * step);
  c.chunk = (int)std::min<int64_t>(chunk, (int64_t)kMaxPages << cache.page_shift);
  c.chunks = (int)std::max<int64_t>(1, (keys + c.chunk - 1) / c.chunk);
  c.grid = units * c.chunks;
  return c;
}

struct Plan {
  Cut own, shared;
  int64_t slots;
};
Plan plan(const KvCache& c, const KvBatch& b, const Attention& a) {
  const int64_t per_kv = a.q_heads / c.heads;
  const int64_t max_q = std::min(a.tokens, b.max_q_len);
  int64_t keys = b.max_kv_len;
  if (a.window > 0) keys = std::min(keys, a.window + max_q - 1);
  Plan p;
  p.own = cut(b.seqs, c, max_q * per_kv, keys + kHalf - 1);
  p.shared = Cut{1, 1, kTile * kWaves, 0, 0};
  if (b.groups > 0 && b.max_shared_len > 0)
    p.shared = cut(b.groups, c, a.tokens * per_kv, b.max_shared_len);
  p.slots = p.own.chunks + p.shared.chunks;
  return p;
}

template <int D>
void launch(const KvCache& c, const KvBatch& b, const Attention& t, hipStream_t st) {
  const Plan p = plan(c, b, t);
  const int64_t rows = t.tokens * t.q_heads;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(t.q), a.q_token = t.q_token, a.q_head = t.q_head;
  a.k_codes = c.k_codes, a.k_scales = c.k_scales, a.v_codes = c.v_codes, a.v_scales = c.v_scales;
  a.q_starts = b.q_starts, a.kv_lens = b.kv_lens, a.page_table = b.page_table, a.group_starts = b.group_starts;
  a.shared_lens = b.shared_lens;
  a.pages = c.pages, a.max_kv = b.max_kv_len, a.max_q = (int)std::min(t.tokens, b.max_q_len), a.tokens = (int)t.tokens, a.seqs = (int)b.seqs;
  a.groups = p.shared.chunks > 0 ? (int)b.groups : 0;
  a.kv_heads = (int)c.heads, a.per_kv = (int)(t.q_heads / c.heads), a.page_shift = c.page_shift;
  a.max_pages = (int)b.max_pages, a.window = (int)std::min<int64_t>(t.window, 1 << 30), a.causal = t.causal;
  a.max_shared = b.max_shared_len;
  a.scale_log2 = t.scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(t.out), a.lse = t.lse;
  a.part_o = static_cast<float*>(t.scratch), a.part_ml = a.part_o + p.slots * rows * D;
  a.most_chunks = p.own.chunks, a.shared_chunk = p.shared.chunk;
  auto pass = [&](const Cut& k, bool shared) {
    a.shared_pass = shared, a.chunk = p.own.chunk, a.chunks = k.chunks, a.row_tiles = k.row_tiles;
    const unsigned lds = (unsigned)((k.chunk >> c.page_shift) + 2) * 4u;
    if (k.r == 1) k_attn_stream<D, 1><<<(unsigned)k.grid, 256, lds, st>>>(a);
    if constexpr (D <= 128)
      if (k.r == 2) k_attn_stream<D, 2><<<(unsigned)k.grid, 256, lds, st>>>(a);
  };
  if (a.groups > 0) pass(p.shared, true);
  pass(p.own, false);
  if (p.slots > 1) k_attn_join<D><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(a);
}

}  // namespace

bool attention_fits(const KvCache& c, const KvBatch& b, const Attention& a) {
  const Plan p = plan(c, b, a);
  return p.own.grid <= kMaxGrid && p.shared.grid <= kMaxGrid && (a.tokens * a.q_heads + 3) / 4 <= kMaxGrid;
}

int64_t attention_scratch(const KvCache& c, const KvBatch& b, const Attention& a) {
  const int64_t slots = plan(c, b, a).slots;
  return slots > 1 ? slots * a.tokens * a.q_heads * (c.head_dim + 2) * 4 : 16;
}

void launch_attention(const KvCache& c, const KvBatch& b, const Attention& a, hipStream_t st) {
  if (c.head_dim == 64) launch<64>(c, b, a, st);
  else if (c.head_dim == 128) launch<128>(c, b, a, st);
  else launch<256>(c, b, a, st);
}

}  // namespace fp4q
