// A mixture-of-experts layer for a few tokens over MXFP4 expert weights, in two launches, and up to
// two more for the router:
//
//   k_moe_logits   l = router_x router_w^T                                 (router only)
//   k_moe_topk     each token's experts and weights          (router, more than one token)
//   k_moe_up       per expert and 32 hidden columns: its tokens' gate and up products,
//                  silu(gate) * up, rounded to MXFP8
//   k_moe_down     per 16 output columns: every expert's down product, weighted and added up
//
// Bound by reading each used expert's weights once; the tokens are the 16 columns of a matrix
// instruction whatever their number, so up to 16 tokens of one expert cost what one does.  No sum
// depends on the order in which workgroups run.  Weights are loaded by whole lines and dealt out to the
// matrix instruction's layout through LDS (deal): loads in that layout, 16 rows per 16 lanes, took
// 62 us for the up product below and 39 for the down product.
//
// The 8-bit matrix arithmetic cuts a product about 13 bits below the largest of its group (fp4q_mx8.hpp).
// In the gate and up sums (5e-6 to 1.2e-5 of their norm) that moves one hidden code of about a thousand across
// a boundary of MXFP8: y before its rounding is 0.8e-3 (64 tokens) to 1.4e-3 (one) of its norm from the exact layer's,
// and 1.8e-3 to 2.1e-3 after the rounding to bf16, which alone is 1.65e-3 away.  Sums that cut nothing would need
// both operands widened to bf16 in registers first, and half of the matrix rate.
//
// Measured, 64 tokens, 4 of 32 experts, d 4096, hidden 2048 (428 MB of weights), us: logits 4.8, top-k 4.7,
// up 52 (285 MB, 5.4 TB/s), down 37 (143 MB, 3.9 TB/s).  One token, 4 of 64 experts, d 2048, hidden 1024
// (14 MB): 3.2, -, 7.3, 5.8, each a launch and one trip to memory, up and down on 128 of the 256 CUs.
#include "fp4q_dev.hpp"
#include "fp4q_mx8.hpp"

namespace fp4q {
namespace {

constexpr int kCus = 256;   // compute units of the GPU
constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = kMaxTokens * 16;   // tokens x top-k

// Order of logits as unsigned integers: NaN above everything, -0 equal to +0, none of them 0 (the
// lowest, -infinity, is ~0xFF800000).
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// -----------------------------------------------------------------------------------------
// Router logits: 16 experts x 16 tokens per workgroup, over a quarter of d that its four waves split
// and join in LDS in wave order; whoever reads a logit adds its quarters up (logit_of).  (One
// workgroup over all of d: 10.2 us for 64 tokens, 32 experts and d = 4096, all of it the address
// unit of the few CUs that had a workgroup.)  fp32 inputs go through the fp32 matrix instruction,
// so nothing is rounded but the sums.
// -----------------------------------------------------------------------------------------
constexpr int kQuarters = 4;

// Logit at `at` = token * experts + expert of the quarters' arrays of n.
__device__ __forceinline__ float logit_of(const float* part, int at, int n) {
  return ((part[at] + part[at + n]) + part[at + 2 * n]) + part[at + 3 * n];
}

typedef __bf16 bf16x8_m __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f_m router_mma(u32x4_m w, u32x4_m x, v4f_m acc, const uint16_t*) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_m, w), __builtin_bit_cast(bf16x8_m, x), acc,
                                                 0, 0, 0);
}
__device__ __forceinline__ v4f_m router_mma(u32x4_m w, u32x4_m x, v4f_m acc, const float*) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[i]), acc, 0, 0, 0);
  return acc;
}

template <typename T>
__global__ __launch_bounds__(256) void k_moe_logits(const T* __restrict__ x, const T* __restrict__ w, int tokens,
                                                     int d, int experts, float* __restrict__ logits) {
  __shared__ v4f_m sums[4][64];
  constexpr int N = 16 / (int)sizeof(T);   // elements per lane and load; a step is 4 N
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const T* wp = w + (int64_t)min(e0 + r, experts - 1) * d + N * q;
  const T* xp = x + (int64_t)min(t0 + r, tokens - 1) * d + N * q;
  const int steps = d / (4 * N), share = 4 * blockIdx.z + wave;
  const int first = steps * share / 16, last = steps * (share + 1) / 16;
  v4f_m acc = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 4;   // steps whose loads are in flight together; past the end the last one again, unused
  for (int s = first; s < last; s += U) {
    u32x4_m wv[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = 4 * N * min(s + u, last - 1);
      wv[u] = *reinterpret_cast<const u32x4_m*>(wp + at);
      xv[u] = *reinterpret_cast<const u32x4_m*>(xp + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < last) acc = router_mma(wv[u], xv[u], acc, (const T*)nullptr);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    v4f_m v = sums[0][lane];
#pragma unroll
    for (int i = 1; i < 4; ++i) v += sums[i][lane];
    float* to = logits + (int64_t)blockIdx.z * tokens * experts;
    const int t = t0 + r;   // column: token; rows 4 q ..: experts
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t < tokens && e0 + 4 * q + i < experts) to[t * experts + e0 + 4 * q + i] = v[i];
  }
}

// The largest of a wave's 64 values, in every lane: neighbours, quads and halves of 16 lanes by DPP,
// then the groups of 16 by lane swaps.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// Each token's top-k, one wave per token: k rounds of a maximum over the logits' keys that each lane
// keeps for its experts (lane, lane + 64, ...), the lowest expert of those that have it, then the
// softmax over the k.  Bound by the chain of k maxima: 4.7 us for 64 tokens, 32 experts and k = 4, of
// which 3 are the launch and the logits' trip from L2.
__global__ __launch_bounds__(64) void k_moe_topk(const float* __restrict__ logits, int experts, int topk,
                                                 int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr int kPerLane = 512 / 64;
  const int lane = threadIdx.x, t = blockIdx.x, n = gridDim.x * experts;
  uint32_t key[kPerLane];   // 0: taken, or no expert (a logit's key is larger: see logit_key)
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < experts ? logit_key(logit_of(logits, t * experts + e, n)) : 0u;
  }
  int chosen = 0;   // lane j: the j-th choice
  for (int j = 0; j < topk; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) best = max(best, key[i]);
    best = wave_max_u32(best);
    int e = -1;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const uint64_t m = __ballot(key[i] == best);
      if (e < 0 && m) e = 64 * i + __builtin_ctzll(m);
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) key[i] = lane + 64 * i == e ? 0u : key[i];
    if (lane == j) chosen = e;
  }
  // every lane adds the exponentials in the order of the choices
  const float own = lane < topk ? logit_of(logits, t * experts + chosen, n) : 0.0f, top = __shfl(own, 0, 64);
  const float w = expf(own - top);
  float total = 0.0f;
  for (int j = 0; j < topk; ++j) total += __shfl(w, j, 64);
  if (lane < topk) {
    ids[t * topk + lane] = chosen;
    weights[t * topk + lane] = w / total;
  }
}

// Arguments of the expert kernels.
struct Moe {
  const uint8_t *xc, *xs;       // MXFP8 tokens [tokens][d]
  const uint8_t *w13c, *w13s;   // MXFP4 [experts][2 hidden][d]: gate rows, then up rows
  const uint8_t *w2c, *w2s;     // MXFP4 [experts][d][hidden]
  int tokens, d, hidden, experts, topk;
  int slots;                    // workgroup columns of k_moe_up: see there
  int32_t* ids;                 // [tokens][topk]; routing one token, k_moe_up writes them
  float* weights;               // [tokens][topk]; routing one token, k_moe_down writes them
  const float* logits;          // [4][experts], routing one token only
  uint8_t *hc, *hs;             // scratch: MXFP8 hidden rows [tokens * topk][hidden]
  int splits;                   // workgroups per row tile of k_moe_down
  float* partial;               // scratch: their sums [row tile][splits][64][rows of the tile]
  int* arrived;                 // scratch: how many of a row tile's have finished; k_moe_up clears it
  void* y;
};

// Which pairs (token * topk + place) chose expert `e`, in order, in `list`; returns how many.  Whole
// workgroup; ends with a barrier.  A token that names an expert twice counts once, by its first
// place; k_moe_down adds the weights up.
struct RouteLds {
  union {
    int16_t id[kMaxPairs];
    uint32_t key[512];
  };
  uint16_t list[kMaxTokens];
  int count, found;
};

__device__ int pairs_of_expert(const Moe& a, int e, RouteLds& r) {
  const int lane = threadIdx.x & 63, pairs = a.tokens * a.topk;
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int v = a.ids[p];
    r.id[p] = v >= 0 && v < a.experts ? (int16_t)v : (int16_t)-1;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
      const int p = p0 + lane;
      bool hit = p < pairs && r.id[p] == e;
      if (hit)
        for (int f = p - p % a.topk; f < p; ++f) hit = hit && r.id[f] != e;
      const uint64_t m = __ballot(hit);
      if (hit) r.list[n + __popcll(m & ((1ull << lane) - 1ull))] = (uint16_t)p;
      n += __popcll(m);
    }
    if (lane == 0) r.count = n;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(r.count);
}

// The single token's choice number `want`: the place of an expert among the logits is the number of
// larger ones, ties to the lower index.
__device__ int choice_of_one(const Moe& a, int want, RouteLds& r) {
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) r.key[e] = logit_key(logit_of(a.logits, e, a.experts));
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    const uint32_t own = r.key[e];
    int place = 0;
#pragma unroll 8
    for (int f = 0; f < a.experts; ++f) {
      const uint32_t k = r.key[f];
      place += k > own || (k == own && f < e);
    }
    if (place == want) r.found = e;   // places are distinct: exactly one thread
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(r.found);
}

// Sums of a workgroup's waves on their way to one: [wave][row tile][q][17 columns] of four rows each
// (the 17th column spreads the readers over the banks).
typedef v4f_m UpSums[4][4][17];
// A wave's LDS: its weights on their way to the matrix instruction's layout, then its sums.
union UpPlace {
  u32x4_m tiles[4][128];
  UpSums sums;
};

// The weights of a workgroup's 32 hidden columns over two K steps: four row tiles of 16, two of gate,
// two of up, as loaded (see deal).
struct UpWeights {
  u32x4_m w[4][2];
};
struct UpRows {
  const uint8_t *codes, *scales;   // of the first tile's first row; the others are uniform distances away
  int64_t up;                      // rows from gate to up
  uint32_t row;                    // the lane's row of a tile's first eight, in bytes of codes
  uint32_t srow;                   // the scales of row lane % 16 of tile lane / 16
  __device__ __forceinline__ int64_t rows(int i) const { return (i & 1 ? 16 : 0) + (i >> 1 ? up : 0); }
};
__device__ __forceinline__ UpRows up_rows(const Moe& a, int e, int h0) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t row = (int64_t)e * 2 * a.hidden + h0;
  UpRows u{a.w13c + row * (a.d / 2), a.w13s + row * (a.d / 32), a.hidden, (uint32_t)((lane >> 3) * (a.d / 2)), 0};
  u.srow = (uint32_t)((u.rows(q) + r) * (a.d / 32));
  return u;
}
// First K step of a wave, of W that share d.
template <int W>
__device__ __forceinline__ int up_first(const Moe& a, int wave) {
  return a.d / 128 * wave / W;
}
// Steps s and s + 1 (past the row's end its last bytes again, unused).
__device__ __forceinline__ void load_up(const Moe& a, const UpRows& u, int s, UpWeights& d) {
  const uint32_t at = u.row + (uint32_t)min(s * 64 + (int)(threadIdx.x & 7) * 16, a.d / 2 - 16);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) d.w[i][h] = load16(u.codes + (u.rows(i) + 8 * h) * (a.d / 2), at);
}

// Gate and up products for G groups of 16 tokens, and the hidden activations of them.  `ahead`: this
// wave's first weights, loaded.
template <int G, int W>
__device__ void up_tiles(const Moe& a, const UpRows& rows, int h0, const uint16_t* list, int n,
                         UpWeights& ahead, UpPlace* places) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int U = G == 1 ? 2 : 1;   // steps whose tokens are in flight: with more groups the registers go to the sums
  const int nk = a.d / 128, first = up_first<W>(a, wave), last = up_first<W>(a, wave + 1);
  // the lane's tokens (64 of 64 K bytes at most; columns past n repeat the last and are not stored),
  // and the one of group q % G whose scales it loads for all
  const auto token = [&](int g) { return (uint32_t)list[min(16 * g + r, n - 1)] / (uint32_t)a.topk; };
  uint32_t xc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) xc[g] = token(g) * (uint32_t)a.d + 16 * q;
  const uint32_t xs = token(q % G) * (uint32_t)(a.d / 32);
  v4f_m acc[4][G];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[i][g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = first; s < last; s += 4) {
    const u32x4_m sw = scale_words(rows.scales, rows.srow, s, nk);   // the four tiles' at once
    const u32x4_m sx = scale_words(a.xs, xs, s, nk);
#pragma unroll
    for (int h = 0; h < 4; h += 2) {
      if (s + h >= last) break;
      u32x4_m xl[U][G], xh[U][G], w[2][4];
      const auto load_x = [&](int k, int to) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint8_t* p = a.xc + min(s + h + k, last - 1) * 128;
          xl[to][g] = load16(p, xc[g]);
          xh[to][g] = load16(p + 64, xc[g]);
        }
      };
#pragma unroll
      for (int k = 0; k < U; ++k) load_x(k, k);
      if (s + h > first) load_up(a, rows, s + h, ahead);
      deal(places[wave].tiles, ahead.w, w[0], w[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (s + h + k >= last) break;
        if (U == 1 && k == 1) load_x(1, 0);
        uint32_t tile[4], group[G];
        spread(sw[h + k], tile);
        spread(sx[h + k], group);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[i][g] = mma_w4x8(frag4(w[k][i]), frag8(xl[k % U][g], xh[k % U][g]), acc[i][g], tile[i] >> (8 * q),
                                 group[g] >> (8 * q));
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) places[wave].sums[i][q][r] = acc[i][g];
    __syncthreads();
    // thread -> token column c, hidden column i; 32 neighbouring lanes hold one MXFP8 block
    const int i = threadIdx.x & 31;
#pragma unroll
    for (int c = threadIdx.x >> 5; c < 16; c += 2 * W) {
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) {
        gate += places[v].sums[i >> 4][(i >> 2) & 3][c][i & 3];
        up += places[v].sums[2 + (i >> 4)][(i >> 2) & 3][c][i & 3];
      }
      const float h = gate / (1.0f + expf(-gate)) * up;
      float m = __builtin_fabsf(h);
      m = m < __builtin_inff() ? m : 0.0f;   // the scale is that of the finite values
      m = lane_xor_max<1>(m);
      m = lane_xor_max<2>(m);
#pragma unroll
      for (int off = 4; off <= 16; off *= 2) m = __builtin_fmaxf(m, __shfl_xor(m, off, 64));
      const uint32_t code = (uint32_t)max((int)((__float_as_uint(m) + 0x1FFFFFu) >> 23) - 8, 0);
      const float inv = __uint_as_float((254u - code) << 23);
      const uint32_t byte = __builtin_amdgcn_cvt_pk_fp8_f32(h * inv, 0.0f, 0, false) & 0xFFu;
      if (16 * g + c < n) {
        const int64_t p = list[16 * g + c];
        a.hc[p * a.hidden + h0 + i] = (uint8_t)byte;
        if (i == 0) a.hs[p * (a.hidden / 32) + h0 / 32] = (uint8_t)code;
      }
    }
  }
}

// Grid: hidden / 32 tiles x slots: 32 columns of gate and of up make one MXFP8 block, so a workgroup
// rounds its activations without help from others.  The waves split d; the weights of one workgroup
// travel while another's are multiplied.  The activation stays fp32 until its one rounding to MXFP8, the
// form in which the down product takes it.  G: groups of 16 tokens per pass over the expert's weights.
// ROUTE: one token, whose choices come from the logits and are written to a.ids.
// (Bounds: 128 registers spill with G = 2: 64 tokens, 4 of 12 experts, d 4096 took 67.5 us against 57.2.)
template <int G, int W, bool ROUTE>
__global__ __launch_bounds__(64 * W, G == 4 ? 2 : G == 2 ? 3 : 4) void k_moe_up(Moe a) {
  __shared__ UpPlace places[W];
  __shared__ RouteLds r;
  // the arrival counts of the launch that follows; any workgroups do, before the first can leave
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < a.d / 16;
       i += gridDim.x * gridDim.y * blockDim.x)
    a.arrived[i] = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = up_first<W>(a, wave), last = up_first<W>(a, wave + 1), h0 = blockIdx.x * 32;
  // Workgroup column -> expert.  With at least as many choices as experts there is a column per
  // expert; with fewer there is one per choice, and the one that holds an expert's first choice
  // takes it.
  const bool by_choice = a.slots != a.experts;
  int e = blockIdx.y;
  if constexpr (ROUTE) e = choice_of_one(a, blockIdx.y, r);
  else if (by_choice) e = a.ids[blockIdx.y];
  if (e < 0 || e >= a.experts) return;
  // The first weights travel while the expert's tokens are looked up, where few workgroups turn out to
  // have none (2 choices per expert: one in seven).  us of the layer without / with, 64 tokens: 4 of 32, d
  // 4096 95.8 / 93.5; 4, 3 and 2 of 128, d 2048 82.1 / 81.6, 73.2 / 76.6 and 62.2 / 69.0.
  const bool early = ROUTE || a.tokens * a.topk >= 2 * a.experts;
  const UpRows rows = up_rows(a, e, h0);
  UpWeights ahead;
  if (early && first < last) load_up(a, rows, first, ahead);
  int n;
  if constexpr (ROUTE) {
    if (threadIdx.x == 0) {
      r.list[0] = (uint16_t)blockIdx.y;
      if (blockIdx.x == 0) a.ids[blockIdx.y] = e;
    }
    __syncthreads();
    n = 1;
  } else {
    n = pairs_of_expert(a, e, r);
    if (n == 0 || (by_choice && r.list[0] != blockIdx.y)) return;
  }
  for (int i = 0; i < n; i += 16 * G) {
    if (i > 0) __syncthreads();   // the sums' places take weights again
    if ((i > 0 || !early) && first < last) load_up(a, rows, first, ahead);
    up_tiles<G, W>(a, rows, h0, r.list + i, min(n - i, 16 * G), ahead, places);
  }
}

constexpr int kDownWaves = 16;
// Most K steps of a unit of work, all of whose weights are in flight together: fewer where the sums
// of four groups need the registers.
constexpr int down_steps(int g) { return g == 4 ? 2 : 4; }
constexpr int kNone = 0xFFFF;   // no expert

// Weights of one unit of work: up to ST K steps of one expert's RT tiles of 16 output rows.
template <int RT, int ST>
struct DownUnit {
  u32x4_m w[ST][RT];   // as loaded (see deal)
  u32x4_m sw;   // of row lane % 16 of tile lane / 16 % RT
};
template <int RT, int ST>
__device__ __forceinline__ void load_unit(const Moe& a, int e, int n0, int s0, int s1, DownUnit<RT, ST>& d) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t row = (int64_t)e * a.d + n0, cols = a.hidden / 2;
  const uint8_t* wc = a.w2c + row * cols;
  const uint32_t at = (uint32_t)((lane >> 2) * cols + 16 * (lane & 3));
#pragma unroll
  for (int u = 0; u < ST; ++u)   // past the unit's end the last step again, unused
#pragma unroll
    for (int i = 0; i < RT; ++i) d.w[u][i] = load16(wc + (16 * i * cols + min(s0 + u, s1 - 1) * 64), at);
  d.sw = scale_words(a.w2s + row * (a.hidden / 32), (uint32_t)((16 * (q % RT) + r) * (a.hidden / 32)), s0,
                     a.hidden / 128);
}

// The unit's product with its expert's hidden rows, added with the pairs' weights to this wave's
// own sums (out[token][16 RT]).
template <int G, int RT, int ST>
__device__ __forceinline__ void down_unit(const Moe& a, const DownUnit<RT, ST>& d, int s0, int s1, const uint16_t* list,
                                          int n, const float* wts, float (*out)[16 * RT], u32x4_m* block) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  // the lane's hidden rows (1024 of 64 K bytes at most), and the one whose scales it loads for all
  uint32_t hc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) hc[g] = list[min(16 * g + r, n - 1)] * (uint32_t)a.hidden + 16 * q;
  const u32x4_m sh =
      scale_words(a.hs, list[min(16 * (q % G) + r, n - 1)] * (uint32_t)(a.hidden / 32), s0, a.hidden / 128);
  v4f_m acc[RT][G];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[i][g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < ST; ++u) {
    if (s0 + u >= s1) break;
    uint32_t tile[RT], group[G];
    spread(d.sw[u], tile);
    spread(sh[u], group);
    u32x4_m dealt[RT];
    deal(block, d.w[u], dealt);
    v8i_m w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i] = frag4(dealt[i]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t* p = a.hc + (s0 + u) * 128;
      const v8i_m h = frag8(load16(p, hc[g]), load16(p + 64, hc[g]));
#pragma unroll
      for (int i = 0; i < RT; ++i)
        acc[i][g] = mma_w4x8(w[i], h, acc[i][g], tile[i] >> (8 * q), group[g] >> (8 * q));
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (16 * g + r < n) {
      const int p = list[16 * g + r];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v4f_m* o = reinterpret_cast<v4f_m*>(&out[p / a.topk][16 * i + 4 * q]);
        *o += wts[p] * acc[i][g];
      }
    }
}

template <bool BF16OUT>
__device__ __forceinline__ void store_y(const Moe& a, int t, int col, float v0, float v1) {
  const int64_t at = (int64_t)t * a.d + col;
  if constexpr (BF16OUT) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + at) = bf16_pair(v0, v1);
  else *reinterpret_cast<f32x2_m*>(static_cast<float*>(a.y) + at) = f32x2_m{v0, v1};
}

// y[t] = sum over its experts e of weight(t, e) h(t, e) w2[e]^T, in fp32, rounded once.
// Grid: d / (16 RT) x splits.  Work units are (used expert in rising order, range of its K steps), dealt
// in turn to the waves of all the splits; each wave adds into sums of its own.  A workgroup joins
// its waves in order; with several splits the last workgroup of a row tile to finish joins them in
// order (their number is fixed by the shape), so the sums do not depend on who that is.
// TOK: token capacity; G: groups of 16 tokens per pass over an expert's weights; ROUTE: one token, whose
// weights come from its choices' logits and are written to a.weights.
template <int TOK, int G, int RT, bool ROUTE, bool BF16OUT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(Moe a) {
  constexpr int kPairs = 16 * TOK;
  constexpr int kRows = 16 * RT, ST = down_steps(G);
  __shared__ __align__(16) float out[kDownWaves][TOK][kRows];
  __shared__ u32x4_m place16[kDownWaves][64];   // each wave's to deal weights out
  __shared__ int16_t id[kPairs];
  __shared__ float wts[kPairs];
  __shared__ int count[512];            // by expert: pairs, then the first place in `sorted`
  __shared__ uint16_t sorted[kPairs];   // pairs by expert
  __shared__ uint16_t expert[kPairs], start[kPairs + 1];   // the used experts and their first place in `sorted`
  __shared__ int used, last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * kRows, pairs = a.tokens * a.topk;
  // K steps per unit: enough units for every wave, at most what one unit's registers hold
  const int nk = a.hidden / 128, workers = kDownWaves * gridDim.y;
  DownUnit<RT, ST> now, next;
  int u = wave * gridDim.y + blockIdx.y;
  const auto unit_steps = [&](int active) { return min(max(active * nk / workers, 1), ST); };
  // One token: its choices are the units' experts as they stand, so nothing is sorted and the first
  // weights travel while the rest is set up.  (An expert's repeats become kNone below: their units are
  // skipped, k_moe_up has written the hidden row of its first place only.)
  const bool single = ROUTE || (TOK == 16 && a.tokens == 1);
  if (single) {
    const int per = unit_steps(a.topk), parts = (nk + per - 1) / per, s0 = u % parts * per;
    const int e = u < a.topk * parts ? a.ids[u / parts] : -1;
    if (e >= 0 && e < a.experts) load_unit(a, e, n0, s0, min(s0 + per, nk), now);
  }
  // a pair's expert and weight, one thread per pair
  int e = -1;
  float w = 0.0f;
  if (tid < pairs) {
    e = a.ids[tid];
    if constexpr (ROUTE) w = logit_of(a.logits, e, a.experts);
    else w = a.weights[tid];
    if (e < 0 || e >= a.experts) e = -1;
    id[tid] = (int16_t)e;
    wts[tid] = w;
  }
  if (tid < 512) count[tid] = 0;
  for (int i = tid; i < kDownWaves * TOK * kRows / 4; i += 64 * kDownWaves)
    reinterpret_cast<v4f_m*>(out)[i] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  int place = 0;
  if (tid < pairs) {
    const int p0 = tid - tid % a.topk;
    if constexpr (ROUTE) {   // softmax over the token's choices; the first is the largest
      const float top = wts[p0];
      float total = 0.0f;
      for (int j = 0; j < a.topk; ++j) total += expf(wts[p0 + j] - top);
      w = expf(w - top) / total;
      if (blockIdx.x == 0 && blockIdx.y == 0) a.weights[tid] = w;
    } else if (e >= 0) {   // an expert's first place takes its repeats' weights; they take no part
      for (int f = p0; f < tid; ++f)
        if (id[f] == e) e = -1;
      if (e >= 0)
        for (int f = tid + 1; f < p0 + a.topk; ++f)
          if (id[f] == e) w += wts[f];
    }
    if (single) {
      sorted[tid] = start[tid] = (uint16_t)tid;
      expert[tid] = (uint16_t)e;   // kNone: the unit is skipped
      if (tid == 0) used = start[pairs] = (uint16_t)pairs;
    } else if (e >= 0) {
      place = atomicAdd(&count[e], 1);   // the order among an expert's pairs changes no sum
    }
  }
  __syncthreads();
  if (tid < pairs) wts[tid] = w;
  if (!single && wave == 0) {   // eight experts per lane: prefix sums of pairs (low half) and used experts (high half)
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = count[8 * lane + i];
      sum += c[i] + (c[i] ? 1 << 16 : 0);
    }
    int run = sum;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const int v = __shfl_up(run, off, 64);
      if (lane >= off) run += v;
    }
    if (lane == 63) used = run >> 16, start[run >> 16] = (uint16_t)(run & 0xFFFF);
    run -= sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      count[8 * lane + i] = run & 0xFFFF;
      if (c[i]) {
        expert[run >> 16] = (uint16_t)(8 * lane + i);
        start[run >> 16] = (uint16_t)(run & 0xFFFF);
        run += c[i] + (1 << 16);
      }
    }
  }
  __syncthreads();
  if (!single) {
    if (e >= 0) sorted[count[e] + place] = (uint16_t)tid;
    __syncthreads();
  }
  const int active = __builtin_amdgcn_readfirstlane(used);
  const int per = unit_steps(active), parts = (nk + per - 1) / per;
  const int units = active * parts;
  const auto load = [&](int u, DownUnit<RT, ST>& d) {
    const int s0 = u % parts * per, e = __builtin_amdgcn_readfirstlane(expert[u / parts]);
    if (e != kNone) load_unit(a, e, n0, s0, min(s0 + per, nk), d);
  };
  if (!single && u < units) load(u, now);
  for (; u < units; u += workers) {
    if (u + workers < units) load(u + workers, next);   // travels while this unit is multiplied
    const int s0 = u % parts * per, s1 = min(s0 + per, nk);
    const int first = __builtin_amdgcn_readfirstlane(start[u / parts]);
    const int n = __builtin_amdgcn_readfirstlane(start[u / parts + 1]) - first;
    const bool none = __builtin_amdgcn_readfirstlane(expert[u / parts]) == kNone;
    for (int i = 0; i < n && !none; i += 16 * G)
      down_unit<G, RT, ST>(a, now, s0, s1, sorted + first + i, min(n - i, 16 * G), wts, out[wave], place16[wave]);
    now = next;
  }
  __syncthreads();
  const int splits = gridDim.y;
  constexpr int kPer = kRows / 2;   // two neighbouring columns per thread
  float* joined = a.partial + (int64_t)blockIdx.x * splits * (kMaxTokens * kRows);
  float* part = joined + blockIdx.y * (kMaxTokens * kRows);
  for (int i = tid; i < a.tokens * kPer; i += 64 * kDownWaves) {
    const int t = i / kPer, c = i % kPer * 2;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) s0 += out[v][t][c], s1 += out[v][t][c + 1];
    if (splits == 1) {
      store_y<BF16OUT>(a, t, n0 + c, s0, s1);
    } else {
      // agent scope: the joining workgroup may sit on another die
      __hip_atomic_store(part + 2 * i, s0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(part + 2 * i + 1, s1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (splits == 1) return;
  // The sums are written and read past the caches (agent-scope atomics), so all it takes is that
  // every wave's stores have arrived before the count rises; a fence here would write back and
  // invalidate the die's L2 (60 us on this launch).
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(&a.arrived[blockIdx.x], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
  __syncthreads();
  if (!last) return;
  for (int i = tid; i < a.tokens * kPer; i += 64 * kDownWaves) {
    float s0 = 0.0f, s1 = 0.0f;
    for (int v = 0; v < splits; ++v) {
      const float* p = joined + v * (kMaxTokens * kRows) + 2 * i;
      s0 += __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s1 += __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    store_y<BF16OUT>(a, i / kPer, n0 + i % kPer * 2, s0, s1);
  }
}

// Row tiles per workgroup of the down product: with many tokens two, so that each hidden fragment
// loaded is multiplied twice (us of the layer with one / two, 4 of 32 experts, d 4096: 64 tokens 97.7 / 94,
// 24 tokens 88.2 / 86; 16 tokens 84.5 / 81.7, 4 tokens 44.8 / 45.1, 2 tokens 25.7 / 27.0).
constexpr int row_tiles(int tokens) { return tokens <= 16 ? 1 : 2; }

// Groups of 16 tokens that a pass over an expert's weights takes, from the mean number of tokens per
// expert: a further pass reads them from L2, more groups take registers from the loads in flight (and
// multiply columns that few experts fill).  us of the layer with one / two / four groups, 64 tokens, d 4096
// and hidden 2048, then d 2048 and hidden 1024:
//   mean  8 (4 of 32, 8 of 64)   92 / 109 / 139    60 / 73 / 94
//   mean 16 (4 of 16)            68 /  71 / 82      32 / 31 / 37
//   mean 19 (4 of 13)            67 /  65 / 78      37 / 35 / 44
//   mean 25 (4 of 10)            61 /  56 / 70      33 / 33 / 39
//   mean 32 (4 of 8)             56 /  55 / 53      30 / 31 / 32
//   mean 42 (4 of 6)             62 /  62 / 61      33 / 33 / 32
//   mean 64 (8 of 8)             79 /  71 / 67      45 / 43 / 45
//   mean 64 (4 of 4)             53 /  48 / 47      32 / 29 / 30
// (32 tokens, d 4096, mean 32, 4 of 4: 33.7 / 31.6.)  A hot expert costs little: that all 64 tokens of 4
// of 32 choose one, which takes four passes over it, 98 us against 92.
int groups(const Moe& a) {
  const int mean = a.tokens * a.topk / a.experts;
  return a.tokens <= 16 || mean <= 16 ? 1 : a.tokens <= 32 || mean <= 32 ? 2 : 4;
}

template <int G, bool ROUTE>
void run_up(const Moe& a, hipStream_t st) {
  // Waves per workgroup: eight where all workgroups are on the GPU at once then (16 waves of G = 1 fit a
  // CU by their registers, 12 or 8 of the others, and so two workgroups of eight or one); else four, which
  // leave a CU fewer waves at a time without loads in flight.  us of the layer with four / eight, 64 tokens, d 4096:
  // G = 1, hidden 2048, 8 of 64, 4 of 32, 4 of 16 172 / 181, 92 / 94, 68 / 69, hidden 1024, 4 of 16 42.7 / 41.3; G = 2,
  // hidden 2048, 4 of 12, 4 of 8 57 / 65, 55 / 60, hidden 1024, 4 of 8 43 / 39; G = 4, hidden 2048, 8 of 8, 4 of 4
  // 67 / 78, 53 / 48.  One token, 4 of 32: 20.0 / 19.5.
  const dim3 grid(a.hidden / 32, a.slots);
  const bool eight = (int64_t)grid.x * grid.y <= (G == 1 ? 2 : 1) * kCus;
  if (eight) k_moe_up<G, 8, ROUTE><<<grid, 512, 0, st>>>(a);
  else k_moe_up<G, 4, ROUTE><<<grid, 256, 0, st>>>(a);
}

template <int TOK, int G, int RT, bool ROUTE>
void run_down(const Moe& a, bool bf16_out, hipStream_t st) {
  const dim3 grid(a.d / (16 * RT), a.splits);
  if (bf16_out) k_moe_down<TOK, G, RT, ROUTE, true><<<grid, 64 * kDownWaves, 0, st>>>(a);
  else k_moe_down<TOK, G, RT, ROUTE, false><<<grid, 64 * kDownWaves, 0, st>>>(a);
}

void run(const Moe& a, bool bf16_out, hipStream_t st) {
  const int g = groups(a);
  if (g == 1) run_up<1, false>(a, st);
  else if (g == 2) run_up<2, false>(a, st);
  else run_up<4, false>(a, st);
  if (a.tokens <= 16) run_down<16, 1, row_tiles(16), false>(a, bf16_out, st);
  else if (g == 1) run_down<64, 1, row_tiles(64), false>(a, bf16_out, st);
  else if (g == 2) run_down<64, 2, row_tiles(64), false>(a, bf16_out, st);
  else run_down<64, 4, row_tiles(64), false>(a, bf16_out, st);
}

// Workgroups that share a row tile of the down product: as many as there are CUs for each tile, but
// no more than leaves a wave a full unit of work (the join takes 2 us), up to eight.
int down_splits(int64_t tokens, int64_t d, int64_t hidden, int64_t experts, int64_t topk) {
  const int64_t used = tokens * topk < experts ? tokens * topk : experts;
  const int64_t cus = kCus / (d / (16 * row_tiles(tokens))), work = used * (hidden / 128) / (4 * kDownWaves);
  const int64_t s = cus < work ? cus : work;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// Scratch: logits, hidden codes, hidden scales, the down splits' sums and arrival counts.
struct Layout {
  int64_t logits, codes, scales, partial, arrived, bytes;
};
Layout layout(int64_t tokens, int64_t d, int64_t hidden, int64_t experts, int64_t topk) {
  Layout l;
  l.logits = 0;
  l.codes = up16(kQuarters * tokens * experts * 4);
  l.scales = l.codes + up16(tokens * topk * hidden);
  l.partial = l.scales + up16(tokens * topk * (hidden / 32));
  const int splits = down_splits(tokens, d, hidden, experts, topk);
  l.arrived = l.partial + (splits > 1 ? d * splits * kMaxTokens * 4 : 0);
  l.bytes = l.arrived + up16(d / 16 * 4);
  return l;
}

}  // namespace

int64_t moe_scratch(int64_t tokens, int64_t d, int64_t hidden, int64_t experts, int64_t topk) {
  return layout(tokens, d, hidden, experts, topk).bytes;
}

void launch_moe(const MoeArgs& m, hipStream_t st) {
  Moe a;
  a.xc = m.x_codes, a.xs = m.x_scales, a.w13c = m.w13_codes, a.w13s = m.w13_scales, a.w2c = m.w2_codes;
  a.w2s = m.w2_scales, a.tokens = m.tokens, a.d = m.d, a.hidden = m.hidden, a.experts = m.experts, a.topk = m.topk;
  a.slots = m.tokens * m.topk < m.experts ? m.tokens * m.topk : m.experts;
  a.splits = down_splits(m.tokens, m.d, m.hidden, m.experts, m.topk);
  a.ids = m.ids, a.weights = m.weights, a.y = m.y;
  const Layout l = layout(m.tokens, m.d, m.hidden, m.experts, m.topk);
  uint8_t* scratch = static_cast<uint8_t*>(m.scratch);
  float* logits = reinterpret_cast<float*>(scratch + l.logits);
  a.logits = logits;
  a.hc = scratch + l.codes;
  a.hs = scratch + l.scales;
  a.partial = reinterpret_cast<float*>(scratch + l.partial);
  a.arrived = reinterpret_cast<int*>(scratch + l.arrived);
  if (!m.router_w) {
    run(a, m.bf16_out, st);
    return;
  }
  const dim3 grid((m.experts + 15) / 16, (m.tokens + 15) / 16, kQuarters);
  if (m.router_bf16)
    k_moe_logits<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(m.router_x),
                                                  static_cast<const uint16_t*>(m.router_w), m.tokens, m.d, m.experts,
                                                  logits);
  else
    k_moe_logits<float><<<grid, 256, 0, st>>>(static_cast<const float*>(m.router_x),
                                               static_cast<const float*>(m.router_w), m.tokens, m.d, m.experts, logits);
  if (m.tokens == 1 && m.topk < m.experts) {   // the expert kernels read the logits themselves: a launch less
    run_up<1, true>(a, st);
    run_down<16, 1, row_tiles(16), true>(a, m.bf16_out, st);
    return;
  }
  k_moe_topk<<<m.tokens, 64, 0, st>>>(logits, m.experts, m.topk, m.ids, m.weights);
  run(a, m.bf16_out, st);
}

}  // namespace fp4q
