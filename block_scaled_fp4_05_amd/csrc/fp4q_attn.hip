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
// is exact in bf16, so the codes are converted as they are used, the queries are bf16 already, and only P is rounded:
// where rows are few to two bf16 parts, 2^-16 of each p_j at most, since their products cost next to nothing there (64 sequences
// of up to 16384 keys 118.2 us, with one part 118.0; 8 tokens of 64 sequences 117.8, 116.0), where they are many to one,
// 2^-8, since there the products count (two parts: prompts 264 us instead of 207, a prefix that 64 sequences share 50 instead of 47).
// l sums the unrounded p_j.  (S on the block-scaled MFMA, from the
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
constexpr int kMaxPages = 1024; // page ids of a workgroup of many_rows
constexpr int kFewRows = 32;    // rows of a sequence and key/value head up to which few_rows takes it
constexpr int kRowTile = 128;   // rows of a workgroup of many_rows

// A pass of many_rows over its items' row tiles: pieces of `chunk` keys.
struct Pass {
  int items, row_tiles, chunk, chunks;   // row_tiles: the most that an item has; chunks: the most pieces of one; 0: no such pass
  uint32_t grid;                         // workgroups: one for each key/value head, piece and place of a row tile
  bool line;                             // places are those of `tiles_before`; else row_tiles for each item
};

struct AttnArgs {
  const uint16_t* q;
  int64_t q_token, q_head;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t *q_starts, *kv_lens, *page_table, *group_starts, *shared_lens;
  int64_t pages, max_kv, max_shared;
  int max_q, tokens, seqs, groups, kv_heads, per_kv, page_shift, max_pages, window;
  bool causal;
  float scale_log2;                         // scale log2(e)
  uint16_t* out;
  float* lse;
  int shares, unit_shift;                   // workgroups of few_rows, whose units have 2^unit_shift keys
  // many_rows, two passes: groups with the keys that they share, sequences with their own
  Pass shared, own;
  // Partial results, each with its m and l: of the shared pass [piece][token][head][head_dim], behind them many_rows'
  // own pieces or few_rows' whole results of sequences that share keys; of pairs that several workgroups of
  // few_rows took, two pieces of piece_rows to a workgroup.
  int piece_rows, most_rows;                // most_rows: that a pair has
  float *part_o, *part_ml, *piece_o, *piece_ml;
  int* taken;                               // [sequence][kv head][2 row tiles][4]: first workgroup, number of them, shared pieces
};

// The keys that an item's workgroups go through, from a multiple of 16 on.
struct Range {
  int first, end;
};

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ bool broken(const AttnArgs& a, int kv) { return kv < 0 || kv > a.max_kv; }

// Shared keys of a group: whole pages, no more than the call's bound covers, and none past the end of its first
// sequence, whose page table they are read by.
__device__ __forceinline__ int shared_keys(const AttnArgs& a, int group) {
  const int kv = a.kv_lens[clamp_to(a.group_starts[group], 0, a.seqs - 1)];
  const int n = broken(a, kv) ? 0 : clamp_to(a.shared_lens[group], 0, min(kv, (int)a.max_shared));
  return n >> a.page_shift << a.page_shift;
}

// The group of sequence s (the same in the whole wave), or -1.
__device__ __forceinline__ int group_of(const AttnArgs& a, int s) {
  if (a.groups == 0) return -1;
  return wave_sequence(a.group_starts, a.groups, s);
}

// Own keys of a sequence: what its group does not share; under a window, from the first key that the first of the n
// tokens that the call computes sees to the last one's own.  Their places go by the sequence's real length, q_end - t0
// tokens from t0 on, of which n may be fewer.  None where it ends within the shared ones.  A length out of bounds gives no
// keys (and NaN, see `broken`).
__device__ __forceinline__ Range own_range(const AttnArgs& a, int kv, int q_end, int t0, int n, int shared) {
  if (broken(a, kv)) return Range{0, 0};
  int first = shared, end = kv;
  if (a.window > 0) {
    const int64_t pos = (int64_t)kv - ((int64_t)q_end - t0);   // the first token's
    first = (int)max((int64_t)first, min(pos + 1 - a.window, (int64_t)kv));
    end = (int)max((int64_t)0, min(pos + n, (int64_t)kv));
  }
  first &= ~(kHalf - 1);   // whole pages are shared: none of their keys
  return first < end ? Range{first, end} : Range{0, 0};
}
__device__ __forceinline__ int own_pieces(const AttnArgs& a, Range r) {
  return clamp_to((r.end - r.first + a.own.chunk - 1) / a.own.chunk, 1, max(a.own.chunks, 1));
}
__device__ __forceinline__ int shared_pieces(const AttnArgs& a, int shared) {
  return (shared + a.shared.chunk - 1) / a.shared.chunk;
}

// The keys lo .. hi-1 that the query token t of a sequence sees, which has kv positions and whose tokens end
// before q_end.
__device__ __forceinline__ Range visible(const AttnArgs& a, int kv, int q_end, int t) {
  if (broken(a, kv)) return Range{0, 0};
  const int64_t pos = (int64_t)kv - ((int64_t)q_end - t);
  Range r{0, kv};
  if (a.causal) r.end = (int)max((int64_t)0, min(pos + 1, (int64_t)kv));
  if (a.window > 0) r.first = (int)max((int64_t)0, min(pos + 1 - a.window, (int64_t)kv));
  return r;
}
// Those of them before c1: from first to end, first <= end.
__device__ __forceinline__ Range visible_to(const AttnArgs& a, int kv, int q_end, int t, int c1) {
  Range r = visible(a, kv, q_end, t);
  r.end = max(min(r.end, c1), r.first);
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

// Four pairs of bf16 with zeros in place of what is infinite or NaN.
__device__ __forceinline__ u32x4_m only_finite(u32x4_m v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] &= ~odd_halves(v[e]);
  return v;
}
// Two pairs of bf16 values of a key that a row sees: NaN in the sums of those that are infinite or NaN.
__device__ __forceinline__ void poison(u32x2_m v, float& a, float& b, float& c, float& d) {
  const uint32_t x = odd_halves(v.x), y = odd_halves(v.y);
  a = x & 0xFFFFu ? __builtin_nanf("") : a, b = x >> 16 ? __builtin_nanf("") : b;
  c = y & 0xFFFFu ? __builtin_nanf("") : c, d = y >> 16 ? __builtin_nanf("") : d;
}

// Four rows and 16 columns of bf16 in LDS, transposed: lane i of 16 gives the place of columns 4 (i % 4) .. + 3 of
// row i / 4 and gets column i of the four rows.
__device__ __forceinline__ v4s_a read_transposed(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s_a*)(__attribute__((address_space(3))) void*)p);
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Where the products count (many_rows) a row's m need not be its largest score so far: it follows only where that
// is more than 2^kLag times larger, so that l and o, which have fp32's range, are rarely multiplied (prompts of 1021 to 4096
// tokens 215 -> 205 us).
constexpr float kLag = 8.0f;
// There p = 2^(s c - m), c = scale log2(e), with the product inside the fma: exact, while m is a rounded one.  Any m does as
// long as p stays in range, but past 2^24 m's rounding counts in whole powers of two (at 2^36 p was infinite or zero for
// every row).  From there on the product is rounded first, as m's was, so that the largest score gives p = 1; few_rows
// always does so.  Looked at where m changes, it costs 0.2 % (prompts 204.7 us without, 205.1 with; in every tile 205.8).
constexpr float kFar = 0x1p24f;

// What a workgroup works on: the rows of an item (a sequence's query tokens, or in the shared pass a group's, times the
// query heads of one key/value head) and a piece of its keys.
struct Work {
  int head, seq, t0, rows;      // the item's first sequence and token, its rows
  int kv, q_end;                // of a sequence
  int c0, c1;                   // keys
  int slot;                     // of the partial result; -1: the result is whole and goes to the output
};

// Tokens of sequence s that the call computes, from t0 on; q_end: where all of its tokens end.
__device__ __forceinline__ int own_tokens(const AttnArgs& a, int s, int& t0, int& q_end) {
  t0 = clamp_to(a.q_starts[s], 0, a.tokens), q_end = a.q_starts[s + 1];
  return min(clamp_to(q_end, t0, a.tokens) - t0, a.max_q);
}

// Row tiles of a pass in a line, item after item, of which the host knows the sum of the lengths only.  Item i, whose rows
// are those from row r on, has the places from min(i row_tiles, r / 128 + min(i, r / least)) on, least being the fewest rows
// that an item with a tile has: both grow by its tiles at least, so no two tiles share a place, a search in the
// starts finds a place's item without any sum over the items, and the line is no longer than what the host takes for r and i (`cut`).
template <bool SHARED>
__device__ __forceinline__ int first_token(const AttnArgs& a, int i) {
  return clamp_to(a.q_starts[SHARED ? clamp_to(a.group_starts[i], 0, a.seqs) : i], 0, a.tokens);
}
template <bool SHARED>
__device__ __forceinline__ int tiles_before(const AttnArgs& a, int i) {
  const int start = first_token<SHARED>(a, i), rows = start * a.per_kv;
  const int places = rows / kRowTile + min(i, SHARED ? start : rows / (kFewRows + 1));
  return (int)min((int64_t)i * (SHARED ? a.shared : a.own).row_tiles, (int64_t)places);
}

template <bool SHARED>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int place, int head, int piece, Work& w, int& row0) {
  const Pass& pass = SHARED ? a.shared : a.own;
  w.head = head;
  int item, tile;   // of the item's tiles from the last on, which under a causal mask has the most keys
  if (__builtin_expect(pass.line, 0)) {
    item = __builtin_amdgcn_readfirstlane(wave_last(pass.items, [&](int i) { return tiles_before<SHARED>(a, i) <= place; }));
    if (item < 0) return false;
    tile = place - tiles_before<SHARED>(a, item);
  } else {
    item = place % pass.items, tile = place / pass.items;
  }
  int n, first, end;
  if constexpr (SHARED) {
    w.seq = clamp_to(a.group_starts[item], 0, a.seqs);
    const int s1 = clamp_to(a.group_starts[item + 1], w.seq, a.seqs), shared = shared_keys(a, item);
    if (s1 == w.seq || piece >= shared_pieces(a, shared)) return false;
    w.t0 = clamp_to(a.q_starts[w.seq], 0, a.tokens), n = clamp_to(a.q_starts[s1], w.t0, a.tokens) - w.t0;
    first = 0, end = shared, w.slot = piece;
  } else {
    w.seq = item;
    n = own_tokens(a, item, w.t0, w.q_end), w.kv = a.kv_lens[item];
    if (n * a.per_kv <= kFewRows) return false;   // few_rows'
    const int g = group_of(a, item), shared = g >= 0 ? shared_keys(a, g) : 0;
    const Range own = own_range(a, w.kv, w.q_end, w.t0, n, shared);
    const int pieces = own_pieces(a, own);
    if (piece >= pieces) return false;
    first = own.first, end = own.end;
    w.slot = pieces + shared_pieces(a, shared) == 1 ? -1 : a.shared.chunks + piece;
  }
  w.rows = n * a.per_kv;
  const int last = pass.line ? (w.rows - 1) / kRowTile : pass.row_tiles - 1;
  if (tile > last || (last - tile) * kRowTile >= w.rows) return false;
  row0 = (last - tile) * kRowTile;
  w.c0 = min(first + piece * pass.chunk, end), w.c1 = min(w.c0 + pass.chunk, end);
  return true;
}

// The page ids of a workgroup's keys to LDS; an id that is none becomes -1.
__device__ __forceinline__ int load_pages(const AttnArgs& a, const Work& w, int* pages) {
  const int p0 = w.c0 >> a.page_shift, n = w.c1 > w.c0 ? ((w.c1 - 1) >> a.page_shift) - p0 + 1 : 0;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int id = p0 + i < a.max_pages ? a.page_table[(int64_t)w.seq * a.max_pages + p0 + i] : -1;
    pages[i] = id < 0 || id >= a.pages ? -1 : id;
  }
  return n;
}

// 1 / l and lse of a row that is complete.  Nothing seen: zeros and -infinity; only scores of -infinity, or a length
// out of bounds: NaN.
__device__ __forceinline__ float finish(const AttnArgs& a, int seq, int t, float top, float sum, float& lse) {
  lse = (top + __builtin_amdgcn_logf(sum)) * kLn2;
  if (sum != 0.0f) return 1.0f / sum;
  const Range seen = visible(a, a.kv_lens[seq], a.q_starts[seq + 1], t);
  const bool none = seen.end <= seen.first && !broken(a, a.kv_lens[seq]);
  lse = none ? -kInf : __builtin_nanf("");
  return none ? 0.0f : __builtin_nanf("");
}

// -----------------------------------------------------------------------------------------
// Few rows per key/value head: the keys' bytes are what counts.  The work is a line of units, 128 keys (more where they would pass 2^30) of a pair
// (sequence and key/value head) with all of its 16 R rows, sequence by sequence, and every workgroup takes the same
// number of units in a row, so that lengths, which the host does not know, balance.  It finds its place by a
// prefix sum over the sequences, takes pair after pair, and writes what it has of each: the output where it took a pair
// whole, else a piece for k_attn_join.  Within a pair each of its four waves takes every fourth tile of 32 keys, with the
// next tile's loads in flight, and no barrier until the waves' results are joined at the pair's end.
//
// 64 single tokens of 32 query and 8 key/value heads of 128 on 301 to 16384 keys (554 MB): 108 us and 7 in the join.
// The same loads alone, in the same order, take 95 us, 5.8 TB/s: bound by memory, and by some 12 us in which the
// workgroups find their places and end.  Alternatives: two tiles of loads in flight per wave 121 together, three
// workgroups on a CU (spills) 136, a workgroup per pair and fixed piece of its keys 127.  On few keys it is the chain of
// trips to memory (lengths, page ids, codes; then the join) that bounds: one token on 4000 keys 7 + 4 us, 3 to 5
// tokens of 7 sequences with windows of 1000 keys as many.
// -----------------------------------------------------------------------------------------
constexpr int kUnit = kTile * kWaves;
constexpr int kUnitShift = 7;
static_assert(kUnit == 1 << kUnitShift, "");

// Units and row tiles of a sequence's pairs.
struct Pairs {
  int kv, q_end, t0, rows;
  int tiles, units;             // units of one pair; the sequence has kv_heads * tiles pairs
  Range keys;
  int shared;                   // keys before them, of its group, that come from elsewhere
};
template <int R>
__device__ __forceinline__ Pairs pairs_of(const AttnArgs& a, int s) {
  Pairs p;
  const int q_start = a.q_starts[s];
  p.kv = a.kv_lens[s], p.q_end = a.q_starts[s + 1];
  p.t0 = clamp_to(q_start, 0, a.tokens);
  const int n = min(clamp_to(p.q_end, p.t0, a.tokens) - p.t0, a.max_q);
  p.rows = n * a.per_kv;
  p.tiles = p.rows <= kFewRows ? (p.rows + 16 * R - 1) / (16 * R) : 0;
  p.shared = 0;
  if (a.groups > 0) {
    const int g = lane_find(a.group_starts, a.groups + 1, s);
    if (g >= 0 && g < a.groups) p.shared = shared_keys(a, g);
  }
  p.keys = own_range(a, p.kv, p.q_end, p.t0, n, p.shared);
  p.units = max(1, ((p.keys.end - p.keys.first - 1) >> a.unit_shift) + 1);
  return p;
}

// The same value, held once for the wave: it is the same in all lanes.
__device__ __forceinline__ Pairs uniform(const Pairs& p) {
  auto one = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  return Pairs{one(p.kv), one(p.q_end), one(p.t0), one(p.rows), one(p.tiles), one(p.units), Range{one(p.keys.first), one(p.keys.end)}, one(p.shared)};
}

__device__ __forceinline__ int wave_scan(int v) {   // inclusive sum over the lanes up to this one
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const int o = __shfl_up(v, x, 64);
    if ((int)(threadIdx.x & 63) >= x) v += o;
  }
  return v;
}

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
  uint32_t none[2];                                          // all ones where the page is none: NaN scales
};

template <int D, int R>
struct FewLds {
  __align__(16) uint8_t v[kWaves][kTile * Wave<D>::ROW];
  float ml[kWaves][16 * R][2];
  int before[257];   // units per key/value head before each block of sequences
};

template <int D, int R>
__device__ __forceinline__ void few_rows(const AttnArgs& a, int me, FewLds<D, R>& lds) {
  using W = Wave<D>;
  auto& lds_v = lds.v;
  auto& lds_ml = lds.ml;
  auto& lds_before = lds.before;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g4 = lane >> 4;
  const int block = (a.seqs + 255) >> 8;   // sequences to a block: one up to 256
  {
    int mine = 0;
    for (int s = threadIdx.x * block; s < min((int)(threadIdx.x + 1) * block, a.seqs); ++s) {
      const Pairs p = pairs_of<R>(a, s);
      mine += p.tiles * p.units;
    }
    const int upto = wave_scan(mine);
    if (lane == 63) lds_ml[0][wave][0] = __int_as_float(upto);
    __syncthreads();
    int before = 0;
    for (int u = 0; u < wave; ++u) before += __float_as_int(lds_ml[0][u][0]);
    lds_before[threadIdx.x + 1] = before + upto;
    if (threadIdx.x == 0) lds_before[0] = 0;
    __syncthreads();
  }
  const int all = lds_before[256] * a.kv_heads, each = (all + a.shares - 1) / a.shares;
  int unit = __builtin_amdgcn_readfirstlane((int)min((int64_t)me * each, (int64_t)all));
  const int unit_end = __builtin_amdgcn_readfirstlane(min(unit + each, all));

  while (unit < unit_end) {
  // The sequence that has the unit, and its first one.
  int seq, seq_unit;
  {
    int count = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) count += __popcll(__ballot(lds_before[64 * i + lane + 1] * a.kv_heads <= unit));
    seq = count * block, seq_unit = lds_before[count];
    if (block > 1) {
      while (seq < a.seqs) {   // 64 sequences at a time
        const Pairs p = pairs_of<R>(a, min(seq + lane, a.seqs - 1));
        const int mine = seq + lane < a.seqs ? p.tiles * p.units : 0, upto = seq_unit + wave_scan(mine);
        const uint64_t past = __ballot(upto * a.kv_heads > unit);
        if (past) {
          const int at = __builtin_ctzll(past);
          seq_unit = __shfl(upto - mine, at, 64), seq += at;
          break;
        }
        seq_unit = __shfl(upto, 63, 64), seq += 64;
      }
    }
    seq = __builtin_amdgcn_readfirstlane(seq), seq_unit = __builtin_amdgcn_readfirstlane(seq_unit) * a.kv_heads;
  }
  if (seq >= a.seqs) break;
  const Pairs pairs = uniform(pairs_of<R>(a, seq));
  // Lengths that change under the call (a mistake of its caller's) could name a pair that is none.
  if (unit < seq_unit || unit - seq_unit >= (int64_t)pairs.units * pairs.tiles * a.kv_heads) break;
  const int pair = (unit - seq_unit) / pairs.units, pair_unit = seq_unit + pair * pairs.units, k0 = unit - pair_unit;
  const int units = min(pairs.units - k0, unit_end - unit);
  const int head = pair % a.kv_heads, row_tile = pair / a.kv_heads, rows = pairs.rows, row0 = row_tile * 16 * R, t0 = pairs.t0;
  const int c0 = pairs.keys.first + (k0 << a.unit_shift);
  const int c1 = k0 + units == pairs.units ? pairs.keys.end : c0 + (units << a.unit_shift);
  const bool whole = units == pairs.units;
  if (k0 == 0 && threadIdx.x == 0) {   // who has the pair: for k_attn_join
    int* at = a.taken + 4 * (((int64_t)seq * a.kv_heads + head) * 2 + row_tile);
    at[0] = me, at[1] = (pair_unit + pairs.units - 1) / each - me + 1, at[2] = shared_pieces(a, pairs.shared);
  }
  unit += units;

  // Queries, the MFMA's second operand: lane (n, g4) holds elements 64 i + 16 g4 .. + 15 of row n, as it does of the keys.
  v8b_a qf[R][W::LOADS][2];
  int lo[R], hi[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + n, rows - 1);   // behind the last row: that one again, not stored
    const int t = t0 + row / a.per_kv, h = head * a.per_kv + row % a.per_kv;
    const Range seen = visible_to(a, pairs.kv, pairs.q_end, t, c1);
    lo[r] = seen.first, hi[r] = seen.end;
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

  // Pages of the two halves of a tile, by scalar loads (a vector load's wait would be one for the rows asked for
  // before it, too).  Past the keys: those of the last.
  const int64_t head_rows = (int64_t)1 << a.page_shift;
  const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.page_table + (int64_t)seq * a.max_pages);
  auto fetch = [&](int key0, Fetch<D>& f) {   // keys key0 .. key0 + 31
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int key = key0 + 16 * b, page = table[min(min(key, c1 - 1) >> a.page_shift, a.max_pages - 1)];
      const bool none = page < 0 || page >= a.pages;
      const int64_t r0 = ((int64_t)(none ? 0 : page) * a.kv_heads + head) * head_rows + (key & (int)(head_rows - 1));
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
      f.none[b] = none ? 0xFFFFFFFFu : 0u;   // (applied where the scales are used: here it would wait for them)
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
  // One tile of keys, in f, and the loads of the one after the next into f as soon as that is free.
  auto step = [&](int key0, Fetch<D>& f) {
    const bool edge = key0 < lo_max || key0 + kTile > hi_min;   // some row does not see some key

    // Values to LDS as bf16.  Rows behind the chunk may hold anything: they become zeros.  So do values that are not finite
    // in a tile that not every row sees whole, since 0 times them is NaN: rows that see them get theirs below.
    bool odd = false;
    if (edge) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < W::LOADS; ++i) {
          if (key0 + 16 * b + 64 / W::LINE * i + lane / W::LINE >= c1) f.v[b][i] = u32x4_m{0u, 0u, 0u, 0u}, f.vs[b][i] = 127u;
          odd |= suspect(f.v[b][i], f.vs[b][i]);
        }
      odd = __any(odd);
    }
    auto put = [&](bool finite) {
      wave_lds_fence();
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < W::LOADS; ++i) {
          u32x4_m vb[2];
          to_bf16(f.v[b][i], f.vs[b][i], vb);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<u32x4_m*>(mine + (16 * b + 64 / W::LINE * i + lane / W::LINE) * W::ROW + 32 * (lane % W::LINE) + 16 * j) =
                finite ? only_finite(vb[j]) : vb[j];
        }
      wave_lds_fence();
    };
    put(false);
    if (__builtin_expect(odd, 0)) {
      for (int k = 0; k < kTile; ++k)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if ((uint32_t)(key0 + k - lo[r]) < (uint32_t)(hi[r] - lo[r]))
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              v4f_m& c = acc[r][i];
              float c0 = c[0], c1_ = c[1], c2 = c[2], c3 = c[3];
              poison(*reinterpret_cast<const u32x2_m*>(mine + k * W::ROW + 32 * i + 8 * g4), c0, c1_, c2, c3);
              c = v4f_m{c0, c1_, c2, c3};
            }
      put(true);
    }

    // Scores: register j of half b is key key0 + 16 b + 4 g4 + j, row n.
    v4f_m s4[R][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int r = 0; r < R; ++r) s4[r][b] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < W::LOADS; ++i) {   // elements 64 i + 16 g4 ..: the row's scale byte 2 i + g4 / 2
        u32x4_m kb[2];
        to_bf16(f.k[b][i], (f.ks[b][i / 2] | f.none[b]) >> (16 * (i & 1) + 8 * (g4 >> 1)) & 0xFFu, kb);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < R; ++r)
            s4[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b_a, kb[j]), qf[r][i][j], s4[r][b], 0, 0, 0);
      }
    }
    if (key0 + kUnit < stop) fetch(key0 + kUnit, f);
    v8b_a p[R][2];   // in two parts, the second what the first's rounding left
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
          if ((uint32_t)(key - lo[r]) >= (uint32_t)(hi[r] - lo[r])) sc[i] = -kInf;
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
      u32x4_m w[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = exp2_of(sc[2 * i] - base), y = exp2_of(sc[2 * i + 1] - base);
        l[r] += x + y;
        w[0][i] = bf16_pair(x, y);
        w[1][i] = bf16_pair(x - bf16_lo(w[0][i]), y - bf16_hi(w[0][i]));
      }
      p[r][0] = __builtin_bit_cast(v8b_a, w[0]), p[r][1] = __builtin_bit_cast(v8b_a, w[1]);
    }
    // O^T += V^T P^T, 32 elements of the head at a time.
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      v8b_a v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const v4s_a x = read_transposed(tr + 32 * (i + u)), y = read_transposed(tr + 16 * W::ROW + 32 * (i + u));
        v[u] = __builtin_bit_cast(v8b_a, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r][i + u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[u], p[r][j], acc[r][i + u], 0, 0, 0);
    }
  };
  {
    const int from = begin + max(lo_min - begin, 0) / kUnit * kUnit;   // the first tile that some row sees
    Fetch<D> f;
    if (from < stop) fetch(from, f);
    for (int key0 = from; key0 < stop; key0 += kUnit) step(key0, f);
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
      for (int u = 0; u < kWaves; ++u) top = __builtin_fmaxf(top, lds_ml[u][16 * r + row][0]);
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = 0.0f;
#pragma unroll
      for (int u = 0; u < kWaves; ++u) {
        const float mu = lds_ml[u][16 * r + row][0], part = mu == -kInf ? 0.0f : exp2_of(mu - top);
        sum += part * lds_ml[u][16 * r + row][1];   // 0 times a NaN stays one
        const float* src = reinterpret_cast<const float*>(lds_v[u]) + row * (D + 4) + e0;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = __builtin_fmaf(part, src[e], v[e]);
      }
      const int t = t0 + at / a.per_kv, h = head * a.per_kv + at % a.per_kv;
      const int64_t place = (int64_t)t * a.kv_heads * a.per_kv + h;
      if (whole && pairs.shared == 0) {
        float out_lse;
        const float inv = finish(a, seq, t, top, sum, out_lse);
#pragma unroll
        for (int e = 0; e < PER; e += 4)
          *reinterpret_cast<u32x2_m*>(a.out + place * D + e0 + e) =
              u32x2_m{bf16_pair(v[e] * inv, v[e + 1] * inv), bf16_pair(v[e + 2] * inv, v[e + 3] * inv)};
        if (a.lse && e0 == 0) a.lse[place] = out_lse;
      } else {
        // a whole result, or the workgroup's piece of the pair that it begins with (0) or ends with (1)
        const int64_t p = whole ? (int64_t)a.shared.chunks * a.tokens * a.kv_heads * a.per_kv + place
                                : (int64_t)(2 * me + (k0 == 0)) * a.piece_rows + 16 * r + row;
        float *po = whole ? a.part_o : a.piece_o, *pm = whole ? a.part_ml : a.piece_ml;
#pragma unroll
        for (int e = 0; e < PER; e += 4) *reinterpret_cast<v4f_m*>(po + p * D + e0 + e) = v4f_m{v[e], v[e + 1], v[e + 2], v[e + 3]};
        if (e0 == 0) *reinterpret_cast<f32x2_m*>(pm + 2 * p) = f32x2_m{top, sum};
      }
    }
    __syncthreads();
  }
  }
}

// -----------------------------------------------------------------------------------------
// Many rows per key/value head (prompts, a prefix shared by many sequences): the matrix products are what counts.
// The four waves of a workgroup take 32 rows each and go through the same tiles of 64 keys, staged through
// LDS as bf16 for all of them.  The next tile's loads are in flight during a tile, and its LDS buffer is the other of
// two, so one barrier per tile.
//
// Prompts of 1021 to 4096 tokens, 32 query and 8 key/value heads of 128, causal (180 GFLOP): 204 us, 880 TFLOP/s.
// The MFMA pipe is busy for 36 % of it, and the vector instructions (exponentials, conversions of codes, P to
// bf16) take about as long, so no one part bounds it: without the exponentials 196, without any of the softmax 186, without
// the loads 196.  Alternatives: 64 rows to a wave (spills) 482; the next tile's scores during this one's exponentials,
// with two sets of scores (spills), 224; two tiles of loads in flight 225.
// 64 queries of 32 heads on a shared prefix of 16384 keys: 40 us and 8 in the join; one workgroup on a CU goes through 16
// tiles of some 2 us each, bound by their latencies.
// -----------------------------------------------------------------------------------------
template <int D>
struct Tile {
  static constexpr int KEYS = 64;
  static constexpr int K_ROW = 2 * D + 16;  // bytes of a row of K in LDS: the 16-byte pieces of 16 rows on different banks
  static constexpr int V_ROW = 2 * D + 64;  // of V: the 64 bytes of four rows that half a transposed read covers, too
  static constexpr int LOADS = D / 64;      // 16-byte loads per lane for the 16 rows that a wave stages
  static constexpr int SB = D / 32;         // scale bytes of a row
  static constexpr int LINE = D / 16;       // lanes to a row
  static constexpr int BUFFER = KEYS * (K_ROW + V_ROW);
};

// Maximum and sum over lanes l and l ^ 32, the same bits in both.
__device__ __forceinline__ float pair_max(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ v16f_m zeros16() {
  return v16f_m{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
}

template <int D>
struct ManyLds {
  __align__(16) uint8_t tile[2 * Tile<D>::BUFFER];
  int bounds[kWaves][4], odd[2][kWaves], page[kMaxPages + 2];
};

template <int D, bool SHARED>
__device__ __forceinline__ void many_rows(const AttnArgs& a, uint32_t id, ManyLds<D>& shared_lds) {
  using T = Tile<D>;
  uint8_t* lds = shared_lds.tile;
  auto& lds_bounds = shared_lds.bounds;
  auto& lds_odd = shared_lds.odd;
  int* lds_page = shared_lds.page;
  const Pass& pass = SHARED ? a.shared : a.own;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, half = lane >> 5;
  // Heads first, since workgroups go to the eight XCDs in turn and those of one head read the same keys.
  const int head = id % a.kv_heads, piece = id / a.kv_heads % pass.chunks;
  Work w;
  int row0;
  if (!find_work<SHARED>(a, id / (pass.chunks * a.kv_heads), head, piece, w, row0)) return;
  const int rows = w.rows, c1 = w.c1;
  const int np = load_pages(a, w, lds_page), p0 = w.c0 >> a.page_shift;

  // Queries: lane (n, half) holds elements 32 i + 16 half .. + 15 of row n, as it does of the keys.
  v8b_a qf[D / 32][2];
  int lo, hi;
  {
    const int row = min(row0 + 32 * wave + n, rows - 1);   // behind the last row: that one again, not stored
    const int t = w.t0 + row / a.per_kv, h = head * a.per_kv + row % a.per_kv;
    int kv = w.kv, q_end = w.q_end;
    if constexpr (SHARED) {
      const int s = clamp_to(lane_find(a.q_starts, a.seqs, t), 0, a.seqs - 1);
      kv = a.kv_lens[s], q_end = a.q_starts[s + 1];
    }
    const Range seen = visible_to(a, kv, q_end, t, c1);
    lo = seen.first, hi = seen.end;
    const uint16_t* x = a.q + t * a.q_token + h * a.q_head;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) qf[i][j] = *reinterpret_cast<const v8b_a*>(x + 32 * i + 16 * half + 8 * j);
  }
  int lo_min = lo, lo_max = lo, hi_min = hi, hi_max = hi;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    lo_min = min(lo_min, __shfl_xor(lo_min, x, 64)), lo_max = max(lo_max, __shfl_xor(lo_max, x, 64));
    hi_min = min(hi_min, __shfl_xor(hi_min, x, 64)), hi_max = max(hi_max, __shfl_xor(hi_max, x, 64));
  }
  lo_min = __builtin_amdgcn_readfirstlane(lo_min), lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min), hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  if (lane == 0) lds_bounds[wave][0] = lo_min, lds_bounds[wave][1] = lo_max, lds_bounds[wave][2] = hi_min, lds_bounds[wave][3] = hi_max;
  __syncthreads();
  int all_lo_min = lo_min, all_lo_max = lo_max, all_hi_min = hi_min, all_hi_max = hi_max;   // over the workgroup's rows
#pragma unroll
  for (int u = 0; u < kWaves; ++u) {
    all_lo_min = min(all_lo_min, lds_bounds[u][0]), all_lo_max = max(all_lo_max, lds_bounds[u][1]);
    all_hi_min = min(all_hi_min, lds_bounds[u][2]), all_hi_max = max(all_hi_max, lds_bounds[u][3]);
  }
  const int begin = __builtin_amdgcn_readfirstlane(w.c0 + max(all_lo_min - w.c0, 0) / T::KEYS * T::KEYS);
  const int stop = __builtin_amdgcn_readfirstlane(min(c1, all_hi_max));

  // A wave stages keys 16 wave .. + 15 of a tile, which are in one page.
  const int64_t head_rows = (int64_t)1 << a.page_shift;
  u32x4_m fk[T::LOADS], fv[T::LOADS];
  uint32_t fks[T::LOADS], fvs[T::LOADS], none = 0;
  auto row_of = [&](int key, int& page) {
    page = __builtin_amdgcn_readfirstlane(lds_page[min((key >> a.page_shift) - p0, np - 1)]);
    return ((int64_t)max(page, 0) * a.kv_heads + head) * head_rows + (key & (int)(head_rows - 1));
  };
  auto fetch = [&](int key0) {
    int page;
    const int64_t r0 = row_of(key0 + 16 * wave, page);
    const uint8_t *kc = a.k_codes + r0 * D, *vc = a.v_codes + r0 * D, *ks = a.k_scales + r0 * T::SB, *vs = a.v_scales + r0 * T::SB;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const uint32_t sb = (uint32_t)((64 / T::LINE * i + lane / T::LINE) * T::SB + lane % T::LINE / 2);
      fk[i] = load16(kc, (uint32_t)(1024 * i + 16 * lane)), fks[i] = ks[sb];
      fv[i] = load16(vc, (uint32_t)(1024 * i + 16 * lane)), fvs[i] = vs[sb];
    }
    none = (uint32_t)(page >> 31) & 255u;   // (applied where the scales are used: here it would wait for them)
  };
  auto store = [&](int key0, int buf) {
    uint8_t* b = lds + buf * T::BUFFER;
    bool odd = false;
    const bool edge = key0 < all_lo_max || key0 + T::KEYS > all_hi_min;
    if (edge) {   // see few_rows
#pragma unroll
      for (int i = 0; i < T::LOADS; ++i) {
        if (key0 + 16 * wave + 64 / T::LINE * i + lane / T::LINE >= c1) fv[i] = u32x4_m{0u, 0u, 0u, 0u}, fvs[i] = 127u;
        odd |= suspect(fv[i], fvs[i]);
      }
      odd = __any(odd);
    }
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int row = 16 * wave + 64 / T::LINE * i + lane / T::LINE, col = lane % T::LINE;
      u32x4_m kb[2], vb[2];
      to_bf16(fk[i], fks[i] | none, kb);
      to_bf16(fv[i], fvs[i], vb);
      if (__builtin_expect(odd, 0)) vb[0] = only_finite(vb[0]), vb[1] = only_finite(vb[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<u32x4_m*>(b + row * T::K_ROW + 32 * col + 16 * j) = kb[j];
        *reinterpret_cast<u32x4_m*>(b + T::KEYS * T::K_ROW + row * T::V_ROW + 32 * col + 16 * j) = vb[j];
      }
    }
    if (lane == 0) lds_odd[buf][wave] = odd;
  };

  v16f_m acc[D / 32];
  float m = -kInf, l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = zeros16();
  bool far = false;   // some row's m is past kFar
  const bool idle = row0 + 32 * wave >= rows;

  auto compute = [&](int key0, int buf) {
    const uint8_t* b = lds + buf * T::BUFFER;
    const bool edge = key0 < lo_max || key0 + T::KEYS > hi_min;
    const int odd = lds_odd[buf][0] | lds_odd[buf][1] | lds_odd[buf][2] | lds_odd[buf][3];
    // Scores: register t of tile kt is key key0 + 32 kt + 8 (t / 4) + 4 half + t % 4, row n.
    v16f_m sc[2] = {zeros16(), zeros16()};
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
          sc[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              *reinterpret_cast<const v8b_a*>(b + (32 * kt + n) * T::K_ROW + 64 * i + 32 * half + 16 * j), qf[i][j], sc[kt], 0, 0, 0);
    // fragments are read six ahead of their products
    __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
    for (int i = 0; i < D / 8 - 6; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
    if (edge) {
      asm volatile("");   // a branch: the compiler would compare and select in every tile
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int key = key0 + 8 * (i >> 2) + 4 * half + (i & 3);
        if ((uint32_t)(key - lo) >= (uint32_t)(hi - lo)) sc[i >> 4][i & 15] = -kInf;
      }
    }
    float top = sc[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = __builtin_fmaxf(top, sc[i >> 4][i & 15]);
    const float mt = __builtin_fmaxf(m, pair_max(top) * a.scale_log2);
    if (__any(mt > m + kLag)) {
      const float keep = mt == -kInf ? 1.0f : exp2_of(m - mt);
      m = mt, l *= keep;
      far = __any(__builtin_fabsf(m) > kFar && m != -kInf);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] *= keep;
    }
    float base = m == -kInf ? 0.0f : m, factor = a.scale_log2;
    if (__builtin_expect(far, 0)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) sc[i >> 4][i & 15] = sc[i >> 4][i & 15] * a.scale_log2 - base;
      base = 0.0f, factor = 1.0f;
    }
    v8b_a p[4];   // 16 keys each
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      u32x4_m words;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = exp2_of(__builtin_fmaf(sc[step >> 1][8 * (step & 1) + 2 * i], factor, -base));
        const float y = exp2_of(__builtin_fmaf(sc[step >> 1][8 * (step & 1) + 2 * i + 1], factor, -base));
        l += x + y;
        words[i] = bf16_pair(x, y);
      }
      p[step] = __builtin_bit_cast(v8b_a, words);
    }
    // O^T += V^T P^T: keys 16 step .. + 15, elements 32 i .. + 31
    const uint8_t* tr = b + T::KEYS * T::K_ROW + (4 * half + ((lane & 15) >> 2)) * T::V_ROW + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
#pragma unroll
    for (int step = 0; step < 4; ++step)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint8_t* at = tr + 16 * step * T::V_ROW + 64 * i;
        const v4s_a x = read_transposed(at), y = read_transposed(at + 8 * T::V_ROW);
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(v8b_a, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7)), p[step], acc[i], 0, 0, 0);
      }
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 1);
#pragma unroll
    for (int i = 0; i < D / 8 - 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 4, 1);
    if (__builtin_expect(odd != 0, 0)) {
      for (int key = key0; key < min(key0 + T::KEYS, c1); ++key) {
        int page;
        const int64_t row = row_of(key, page);
        if ((uint32_t)(key - lo) >= (uint32_t)(hi - lo)) continue;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const float s = __uint_as_float((uint32_t)a.v_scales[row * T::SB + i] << 23);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(a.v_codes + row * D + 32 * i + 2 * j + 4 * half);
            float c0 = acc[i][j], c1_ = acc[i][j + 1], c2 = acc[i][j + 2], c3 = acc[i][j + 3];
            poison(u32x2_m{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, s, false)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, s, true))}, c0, c1_, c2, c3);
            acc[i][j] = c0, acc[i][j + 1] = c1_, acc[i][j + 2] = c2, acc[i][j + 3] = c3;
          }
        }
      }
    }
  };

  if (begin < stop) {
    fetch(begin);
    store(begin, 0);
    lds_barrier();
    int buf = 0;
    for (int key0 = begin; key0 < stop; key0 += T::KEYS, buf ^= 1) {
      const bool more = key0 + T::KEYS < stop;
      if (more) fetch(key0 + T::KEYS);
      if (!idle && key0 < hi_max && key0 + T::KEYS > lo_min) compute(key0, buf);
      if (more) store(key0 + T::KEYS, buf ^ 1);
      lds_barrier();
    }
  }

  // Register t of tile i is element 32 i + 8 (t / 4) + 4 half + t % 4 of row n.
  const float sum = pair_sum(l);
  const int at = row0 + 32 * wave + n;
  if (at >= rows) return;
  const int t = w.t0 + at / a.per_kv, h = head * a.per_kv + at % a.per_kv;
  const int64_t place = (int64_t)t * a.kv_heads * a.per_kv + h;
  if (w.slot < 0) {
    float out_lse;
    const float inv = finish(a, w.seq, t, m, sum, out_lse);
    uint16_t* o = a.out + place * D + 4 * half;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<u32x2_m*>(o + 32 * i + 2 * j) =
            u32x2_m{bf16_pair(acc[i][j] * inv, acc[i][j + 1] * inv), bf16_pair(acc[i][j + 2] * inv, acc[i][j + 3] * inv)};
    if (a.lse && half == 0) a.lse[place] = out_lse;
  } else {
    const int64_t p = (int64_t)w.slot * a.tokens * a.kv_heads * a.per_kv + place;
    float* o = a.part_o + p * D + 4 * half;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; j += 4) *reinterpret_cast<v4f_m*>(o + 32 * i + 2 * j) = v4f_m{acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]};
    if (half == 0) *reinterpret_cast<f32x2_m*>(a.part_ml + 2 * p) = f32x2_m{m, sum};
  }
}

// Workgroups on a CU, by registers and LDS.
template <int D, int R>
constexpr int kFewPerCu = D == 64 ? 5 - R : D == 128 ? 2 : 1;
template <int D>
constexpr int kManyPerCu = D <= 128 ? 2 : 1;

template <int D, int R>
__global__ __launch_bounds__(256, (kFewPerCu<D, R>)) void k_attn_few(AttnArgs a) {
  __shared__ FewLds<D, R> lds;
  few_rows<D, R>(a, blockIdx.x, lds);
}

// One launch for all: the shared pass, the sequences with many rows, and those with few, which wait for memory while
// the others multiply.  first: workgroups of the launches before.
template <int D, int R>
__global__ __launch_bounds__(256, kManyPerCu<D>) void k_attn_all(AttnArgs a, uint32_t first) {
  __shared__ union {
    FewLds<D, R> few;
    ManyLds<D> many;
  } lds;
  const uint32_t id = first + blockIdx.x;
  if (id < a.shared.grid) many_rows<D, true>(a, id, lds.many);
  else if (id < a.shared.grid + a.own.grid) many_rows<D, false>(a, id - a.shared.grid, lds.many);
  else few_rows<D, R>(a, id - a.shared.grid - a.own.grid, lds.few);
}

// Joins the partial results of each row.  MANY: the rows of all tokens, and of them those of sequences that many_rows
// took, a wave for each, since they are many and have few pieces (the last 512 tokens of 2048, 32
// heads, 69 us together with a workgroup for each row and 45 so).  Else the most
// rows of every pair that few_rows took, a workgroup for each: wave w takes every fourth piece in rounds of eight
// with their loads in flight, then the waves are added in their order.  2048 rows 6 to 8 us (11 MB), 32 rows
// 3.5 to 4.5: two trips to memory, one after the other, what each row has and then its pieces.
// first: workgroups of the launches before.
template <int D, int R, bool MANY>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, uint32_t first) {
  constexpr int PER = D / 64, AHEAD = MANY ? 4 : 8, WAVES = MANY ? 1 : kWaves;   // WAVES: that share a row
  __shared__ float lds_o[kWaves][D], lds_ml[kWaves][2];
  const int q_heads = a.kv_heads * a.per_kv, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t all = (int64_t)a.tokens * q_heads;
  const uint32_t id = first + blockIdx.x;
  int s, t, h, t0, q_end;
  int4 taken = {0, 0, 0, 0};
  if constexpr (MANY) {
    const int64_t mine = (int64_t)id * kWaves + wave;
    if (mine >= all) return;
    t = (int)mine / q_heads, h = (int)mine % q_heads;
    s = wave_sequence(a.q_starts, a.seqs, t);
    if (s < 0) return;
  } else {
    const int in_pair = id % a.most_rows, pair = id / a.most_rows;
    s = pair / a.kv_heads, t = in_pair / a.per_kv, h = pair % a.kv_heads * a.per_kv + in_pair % a.per_kv;
    // asked for along with the sequence's tokens; without any it means nothing
    taken = *reinterpret_cast<const int4*>(a.taken + 4 * ((int64_t)pair * 2 + in_pair / (16 * R)));
    // (and so where lengths change under the call, but then it is used)
    taken.x = clamp_to(taken.x, 0, a.shares - 1), taken.y = clamp_to(taken.y, 1, a.shares - taken.x);
    taken.z = clamp_to(taken.z, 0, a.shared.chunks);
  }
  const int n = own_tokens(a, s, t0, q_end);
  if constexpr (!MANY) t += t0;
  if (t - t0 >= n || n * a.per_kv > kFewRows != MANY) return;
  const int64_t row = (int64_t)t * q_heads + h;
  // Where they are: `before` of the shared keys, then the own ones.
  int before = 0, own, at = 0;
  bool pieces = false;
  if constexpr (MANY) {
    int shared = 0;
    if (a.groups > 0) {
      const int g = group_of(a, s);
      shared = g >= 0 ? shared_keys(a, g) : 0, before = shared_pieces(a, shared);
    }
    own = own_pieces(a, own_range(a, a.kv_lens[s], q_end, t0, n, shared));
  } else {
    before = taken.z, own = taken.y, pieces = own > 1;
    at = (2 * taken.x + 1) * a.piece_rows + ((t - t0) * a.per_kv + h % a.per_kv) % (16 * R);
  }
  const int count = before + own;
  if (count == 1) return;   // written already
  // number i, as an index of rows
  auto place = [&](int i) -> int64_t {
    if (i < before) return i * all + row;
    i -= before;
    if (!pieces) return (a.shared.chunks + i) * all + row;
    return at + (i == 0 ? 0 : (2 * i - 1) * a.piece_rows);   // the first ends with the pair, the others begin with it
  };
  float top = -kInf, sum = 0.0f, v[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) v[e] = 0.0f;
  for (int i0 = MANY ? 0 : wave; i0 < count; i0 += WAVES * AHEAD) {
    float o[AHEAD][PER], m[AHEAD], l[AHEAD], most = top;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int slot = i0 + WAVES * i, in = min(slot, count - 1);
      const int64_t p = place(in);
      const bool piece = pieces && in >= before;
      const float *po = (piece ? a.piece_o : a.part_o) + p * D + PER * lane, *pm = (piece ? a.piece_ml : a.part_ml) + 2 * p;
      const f32x2_m ml = *reinterpret_cast<const f32x2_m*>(pm);
      m[i] = slot < count ? ml.x : -kInf, l[i] = slot < count ? ml.y : 0.0f;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[i][e] = po[e];
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) most = __builtin_fmaxf(most, m[i]);
    const float keep = top == -kInf ? 0.0f : exp2_of(top - most);
    sum *= keep;
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] *= keep;
    top = most;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (i0 + WAVES * i >= count) break;
      const float part = m[i] == -kInf ? 0.0f : exp2_of(m[i] - top);
      sum += part * l[i];   // 0 times a NaN stays one
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = __builtin_fmaf(part, o[i][e], v[e]);
    }
  }
  float out_lse;
  if constexpr (MANY) {
    const float inv = finish(a, s, t, top, sum, out_lse);
    uint16_t* o = a.out + row * D + PER * lane;
    if constexpr (PER == 1) {
      o[0] = (uint16_t)bf16_pair(v[0] * inv, 0.0f);
    } else {
#pragma unroll
      for (int e = 0; e < PER; e += 2) *reinterpret_cast<uint32_t*>(o + e) = bf16_pair(v[e] * inv, v[e + 1] * inv);
    }
    if (a.lse && lane == 0) a.lse[row] = out_lse;
    return;
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) lds_o[wave][PER * lane + e] = v[e];
  if (lane == 0) lds_ml[wave][0] = top, lds_ml[wave][1] = sum;
  __syncthreads();
  if (threadIdx.x >= D) return;
  top = -kInf, sum = 0.0f;
  float r = 0.0f;
#pragma unroll
  for (int u = 0; u < kWaves; ++u) top = __builtin_fmaxf(top, lds_ml[u][0]);
#pragma unroll
  for (int u = 0; u < kWaves; ++u) {
    const float part = lds_ml[u][0] == -kInf ? 0.0f : exp2_of(lds_ml[u][0] - top);
    sum += part * lds_ml[u][1];
    r = __builtin_fmaf(part, lds_o[u][threadIdx.x], r);
  }
  const float inv = finish(a, s, t, top, sum, out_lse);
  a.out[row * D + threadIdx.x] = (uint16_t)bf16_pair(r * inv, 0.0f);
  if (a.lse && threadIdx.x == 0) a.lse[row] = out_lse;
}

constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in one launch
constexpr int64_t kMaxScratch = (int64_t)1 << 38;
constexpr int kCus = 256;

// `rows` and `keys`: the most that one of the `items` has, of `all` rows; least: the fewest that one with a tile has.  Where
// places for every item's most tiles are more than three times what the rows can need, the tiles go in a line: such places
// and a line, 255 single tokens and a chunk of 2048 on 8192 keys (50 times) 1790 and 1066 us, 16 groups of 16 tokens on
// prefixes of 16384 (5.6 times) 505 and 275, 32 sequences of 1 to 600 tokens (5 times) 298 and 235, a prompt of 4096 with four
// of 512 (3.2 times) 168 and 168, with four of 1024 (2.5 times) 193 and 198, three prompts of 1021 to 4096 (1.7 times) 199 and
// 209: in a line the longest tiles do not all come first.
// Keys are split until every CU has a workgroup, and where the pieces stay long, until it has the two that it holds and that
// hide each other's waits; more and smaller pieces cost more in joining them.  One against two workgroups on a CU, 64 queries of 32 heads on a prefix of 16384 keys 42 and 50 us,
// of 32768 64 and 67, of 65536 109 and 100 (pieces of 2048), of 131072 194 and 171; the last 512 tokens of 8192 112 and 97;
// 1024 of 4096, of which the one has no pieces to join, 99 and 102, of 8192 187 and 173.
constexpr int kLongPiece = 2048;
Pass cut(int64_t items, const KvCache& cache, int64_t rows, int64_t all, int64_t least, int64_t keys, int64_t& grid) {
  const int64_t row_tiles = (rows + kRowTile - 1) / kRowTile, tiles = (all + kRowTile - 1) / kRowTile + std::min(items, all / least) - 1;
  const bool line = items * row_tiles > 3 * tiles;
  const int64_t units = cache.heads * (line ? tiles : items * row_tiles);
  const int64_t want = std::max<int64_t>(1, kCus / units);
  int64_t chunk = (keys + want - 1) / want;
  if (const int64_t two = 2 * kCus / units; cache.head_dim <= 128 && two > want && keys >= two * kLongPiece) chunk = (keys + two - 1) / two;
  chunk = std::max<int64_t>(kUnit, (chunk + kUnit - 1) / kUnit * kUnit);
  chunk = std::min<int64_t>(chunk, (int64_t)kMaxPages << cache.page_shift);
  const int64_t chunks = (keys + chunk - 1) / chunk;
  grid += units * chunks;
  return Pass{(int)items, (int)row_tiles, (int)chunk, (int)chunks, (uint32_t)(units * chunks), line};
}

struct Plan {
  int r;                    // row tiles of few_rows' workgroups
  int64_t few, grid;        // its workgroups; all
  int unit_shift;
  int64_t most_rows, piece_rows;   // of a pair, and in one of its row tiles
  Pass own, shared;
  bool join_few, join_many;
  int64_t slots;            // partial results per row; the other parts of the scratch, in bytes from its start
  int64_t part_ml, piece_o, piece_ml, taken, scratch;
};
Plan plan(const KvCache& c, const KvBatch& b, const Attention& a) {
  const int64_t per_kv = a.q_heads / c.heads, max_q = std::min(a.tokens, b.max_q_len), rows = a.tokens * a.q_heads;
  int64_t keys = b.max_kv_len;
  if (a.window > 0) keys = std::min(keys, a.window + max_q - 1);
  keys += kHalf - 1;
  Plan p{};
  p.most_rows = std::min<int64_t>(max_q * per_kv, kFewRows);
  p.r = p.most_rows <= 16 || c.head_dim > 128 ? 1 : 2;   // (two 16-row tiles of 256 elements spill registers)
  p.piece_rows = std::min<int64_t>(p.most_rows, 16 * p.r);
  const int per_cu = c.head_dim == 64 ? (p.r == 1 ? kFewPerCu<64, 1> : kFewPerCu<64, 2>) : c.head_dim == 128 ? kFewPerCu<128, 1> : kFewPerCu<256, 1>;
  const int64_t pairs = b.seqs * c.heads * ((p.most_rows + 16 * p.r - 1) / (16 * p.r));   // up to 2^27
  p.unit_shift = kUnitShift;
  while (pairs * (((keys - 1) >> p.unit_shift) + 1) > ((int64_t)1 << 30)) ++p.unit_shift;   // they are counted in 32 bits
  const int64_t pair_units = ((keys - 1) >> p.unit_shift) + 1;
  p.few = p.grid = std::min<int64_t>(kCus * per_cu, pairs * pair_units);
  const bool many = max_q * per_kv > kFewRows, shares = b.groups > 0 && b.max_shared_len > 0;
  const int64_t most = a.tokens * per_kv;
  p.own = many ? cut(b.seqs, c, max_q * per_kv, most, kFewRows + 1, keys, p.grid) : Pass{0, 0, kUnit, 0, 0, false};
  p.shared = shares ? cut(b.groups, c, most, most, per_kv, b.max_shared_len, p.grid) : Pass{0, 0, kUnit, 0, 0, false};
  p.join_few = pair_units > 1 || shares, p.join_many = many && (p.own.chunks > 1 || shares);
  p.slots = p.shared.chunks + std::max(p.own.chunks > 1 || shares ? p.own.chunks : 0, shares ? 1 : 0);
  auto put = [&](int64_t& at, int64_t bytes) { at = p.scratch, p.scratch += (bytes + 15) / 16 * 16; };
  int64_t part_o;
  put(part_o, p.slots * rows * c.head_dim * 4);
  put(p.part_ml, p.slots * rows * 8);
  put(p.piece_o, p.few * 2 * p.piece_rows * c.head_dim * 4);
  put(p.piece_ml, p.few * 2 * p.piece_rows * 8);
  put(p.taken, b.seqs * c.heads * 32);
  return p;
}

// As many launches as `all` workgroups of 256 threads need: one takes no more than 2^32 - 1 threads.
template <typename F>
void in_launches(int64_t all, F launch) {
  for (int64_t first = 0; first < all; first += kMaxGrid) launch((unsigned)std::min(all - first, kMaxGrid), (uint32_t)first);
}

template <int D, int R>
void launch_all(const AttnArgs& a, const Plan& p, int64_t rows, hipStream_t st) {
  if (p.grid > p.few)
    in_launches(p.grid, [&](unsigned grid, uint32_t first) { k_attn_all<D, R><<<grid, 256, 0, st>>>(a, first); });
  else k_attn_few<D, R><<<(unsigned)p.grid, 256, 0, st>>>(a);
  if (p.join_few)
    in_launches((int64_t)a.seqs * a.kv_heads * a.most_rows, [&](unsigned grid, uint32_t first) { k_attn_join<D, R, false><<<grid, 256, 0, st>>>(a, first); });
  if (p.join_many)
    in_launches((rows + kWaves - 1) / kWaves, [&](unsigned grid, uint32_t first) { k_attn_join<D, 1, true><<<grid, 256, 0, st>>>(a, first); });
}

template <int D>
void launch(const KvCache& c, const KvBatch& b, const Attention& t, hipStream_t st) {
  const Plan p = plan(c, b, t);
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(t.q), a.q_token = t.q_token, a.q_head = t.q_head;
  a.k_codes = c.k_codes, a.k_scales = c.k_scales, a.v_codes = c.v_codes, a.v_scales = c.v_scales;
  a.q_starts = b.q_starts, a.kv_lens = b.kv_lens, a.page_table = b.page_table, a.group_starts = b.group_starts;
  a.shared_lens = b.shared_lens;
  a.pages = c.pages, a.max_kv = b.max_kv_len, a.max_shared = b.max_shared_len;
  a.max_q = (int)std::min(t.tokens, b.max_q_len), a.tokens = (int)t.tokens, a.seqs = (int)b.seqs;
  a.groups = p.shared.chunks > 0 ? (int)b.groups : 0;
  a.kv_heads = (int)c.heads, a.per_kv = (int)(t.q_heads / c.heads), a.page_shift = c.page_shift;
  a.max_pages = (int)b.max_pages, a.window = (int)std::min<int64_t>(t.window, 1 << 30), a.causal = t.causal;
  a.scale_log2 = t.scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(t.out), a.lse = t.lse;
  a.shares = (int)p.few, a.unit_shift = p.unit_shift, a.shared = p.shared, a.own = p.own;
  a.piece_rows = (int)p.piece_rows, a.most_rows = (int)p.most_rows;
  char* s = static_cast<char*>(t.scratch);
  a.part_o = reinterpret_cast<float*>(s), a.part_ml = reinterpret_cast<float*>(s + p.part_ml);
  a.piece_o = reinterpret_cast<float*>(s + p.piece_o), a.piece_ml = reinterpret_cast<float*>(s + p.piece_ml);
  a.taken = reinterpret_cast<int*>(s + p.taken);
  const int64_t rows = t.tokens * t.q_heads;
  if constexpr (D <= 128)
    if (p.r == 2) return launch_all<D, 2>(a, p, rows, st);
  launch_all<D, 1>(a, p, rows, st);
}

}  // namespace

// Workgroups fit in 32 bits, too, where the scratch does: a pass has at most 3 (1 + 1/128) for each row and piece of it, which
// take at least 256 bytes.
bool attention_fits(const KvCache& c, const KvBatch& b, const Attention& a) { return plan(c, b, a).scratch <= kMaxScratch; }

int64_t attention_scratch(const KvCache& c, const KvBatch& b, const Attention& a) { return plan(c, b, a).scratch; }

void launch_attention(const KvCache& c, const KvBatch& b, const Attention& a, hipStream_t st) {
  if (c.head_dim == 64) launch<64>(c, b, a, st);
  else if (c.head_dim == 128) launch<128>(c, b, a, st);
  else launch<256>(c, b, a, st);
}

}  // namespace fp4q
