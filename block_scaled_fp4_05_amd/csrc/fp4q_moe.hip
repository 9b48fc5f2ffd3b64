// A mixture-of-experts layer for a few tokens over MXFP4 expert weights, in two launches, three
// with the router:
//
//   k_moe_logits   l = router_x router_w^T                                 (router only)
//   k_moe_up       per expert and 32 hidden columns: its tokens' gate and up products,
//                  silu(gate) * up, rounded to MXFP8
//   k_moe_down     per 16 output columns: every expert's down product, weighted and added up
//
// Bound by reading each used expert's weights once; the tokens are the 16 columns of a matrix
// instruction whatever their number, so up to 16 tokens of one expert cost what one does.  No sum
// depends on the order in which workgroups run.
#include "fp4q_dev.hpp"
#include "fp4q_mx8.hpp"

namespace fp4q {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = kMaxTokens * 16;   // tokens x top-k

// Order of logits as unsigned integers: NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// -----------------------------------------------------------------------------------------
// Router logits: 16 experts x 16 tokens per workgroup, sixteen waves that split d and join in
// LDS in wave order.  fp32 inputs go through the fp32 matrix instruction, so nothing is rounded
// but the sums.
// -----------------------------------------------------------------------------------------
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
__global__ __launch_bounds__(1024) void k_moe_logits(const T* __restrict__ x, const T* __restrict__ w, int tokens,
                                                     int d, int experts, float* __restrict__ logits) {
  __shared__ v4f_m sums[16][64];
  constexpr int N = 16 / (int)sizeof(T);   // elements per lane and load; a step is 4 N
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const T* wp = w + (int64_t)min(e0 + r, experts - 1) * d + N * q;
  const T* xp = x + (int64_t)min(t0 + r, tokens - 1) * d + N * q;
  const int steps = d / (4 * N), first = steps * wave / 16, last = steps * (wave + 1) / 16;
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
    for (int i = 1; i < 16; ++i) v += sums[i][lane];
    const int t = t0 + r;   // column: token; rows 4 q ..: experts
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t < tokens && e0 + 4 * q + i < experts) logits[(int64_t)t * experts + e0 + 4 * q + i] = v[i];
  }
}

// Arguments of the expert kernels.
struct Moe {
  const uint8_t *xc, *xs;       // MXFP8 tokens [tokens][d]
  const uint8_t *w13c, *w13s;   // MXFP4 [experts][2 hidden][d]: gate rows, then up rows
  const uint8_t *w2c, *w2s;     // MXFP4 [experts][d][hidden]
  int tokens, d, hidden, experts, topk;
  int slots;                    // workgroup columns of k_moe_up: see expert_of_slot
  int32_t* ids;                 // [tokens][topk]; read, or written by k_moe_up when routing
  float* weights;               // [tokens][topk]; read, or written by k_moe_down when routing
  const float* logits;          // [tokens][experts], routing only
  uint8_t *hc, *hs;             // scratch: MXFP8 hidden rows [tokens * topk][hidden]
  void* y;
};

// The choice of expert `e` by each token as pair indices (token * topk + rank) in `list`, in
// order; returns how many.  Whole workgroup; ends with a barrier.
//
// With given ids: a token that names an expert twice counts once (its first place; k_moe_down
// adds the weights up).  When routing: the rank of e among a token's logits is the number of
// larger ones, ties to the lower index, so no sort is needed.
template <bool ROUTE>
__device__ int pairs_of_expert(const Moe& a, int e, uint16_t* list, int* count, bool publish) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if constexpr (!ROUTE) {
    if (wave == 0) {
      int n = 0;
      const int pairs = a.tokens * a.topk;
      for (int p0 = 0; p0 < pairs; p0 += 64) {
        const int p = p0 + lane;
        bool hit = p < pairs && a.ids[p] == e;
        if (hit)
          for (int f = p - p % a.topk; f < p; ++f) hit = hit && a.ids[f] != e;
        const uint64_t m = __ballot(hit);
        if (hit) list[n + __popcll(m & ((1ull << lane) - 1ull))] = (uint16_t)p;
        n += __popcll(m);
      }
      if (lane == 0) *count = n;
    }
  } else {
    // bit t of `chosen`: token t's place for e, found by one wave per token
    __shared__ uint8_t place[kMaxTokens];
    for (int t = wave; t < a.tokens; t += waves) {
      const float* l = a.logits + (int64_t)t * a.experts;
      const uint32_t own = logit_key(l[e]);
      int rank = 0;
      for (int f0 = 0; f0 < a.experts; f0 += 64) {
        const int f = f0 + lane;
        const uint32_t k = f < a.experts ? logit_key(l[f]) : 0u;
        rank += __popcll(__ballot(f < a.experts && (k > own || (k == own && f < e))));
      }
      if (lane == 0) {
        place[t] = (uint8_t)min(rank, 255);
        if (publish && rank < a.topk) a.ids[t * a.topk + rank] = e;
      }
    }
    __syncthreads();
    if (wave == 0) {
      const int rank = lane < a.tokens ? place[lane] : 255;
      const bool hit = rank < a.topk;
      const uint64_t m = __ballot(hit);
      if (hit) list[__popcll(m & ((1ull << lane) - 1ull))] = (uint16_t)(lane * a.topk + rank);
      if (lane == 0) *count = __popcll(m);
    }
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*count);
}

// Workgroup column -> expert.  With at least as many choices as experts there is a column per
// expert; with fewer there is one per choice, and the one that holds an expert's first choice
// takes it (the caller compares).  -1: nothing to do.
template <bool ROUTE>
__device__ int expert_of_slot(const Moe& a, int slot, int* found) {
  if (a.slots == a.experts) return slot;
  if constexpr (!ROUTE) {
    const int e = a.ids[slot];
    return e >= 0 && e < a.experts ? e : -1;
  } else {
    const int t = slot / a.topk, want = slot % a.topk;
    const float* l = a.logits + (int64_t)t * a.experts;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      const uint32_t own = logit_key(l[e]);
      int rank = 0;
      for (int f = 0; f < a.experts; ++f) {
        const uint32_t k = logit_key(l[f]);
        rank += k > own || (k == own && f < e);
      }
      if (rank == want) *found = e;   // ranks are distinct: exactly one thread
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*found);
  }
}

constexpr int kUpWaves = 8;

// Sums of the eight waves on their way to one: [wave][row tile][q][17 columns] of four rows each
// (the 17th column spreads the readers over the banks).
typedef v4f_m UpSums[kUpWaves][4][4][17];

// Gate and up products of 32 hidden columns (four row tiles of 16: two of gate, two of up) for
// G groups of 16 tokens, and the hidden activations of them.
template <int G>
__device__ void up_tiles(const Moe& a, int e, int h0, const uint16_t* list, int n, UpSums sums) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = a.d / 128, first = nk * wave / kUpWaves, last = nk * (wave + 1) / kUpWaves;
  const int64_t cols = a.d / 2, scols = a.d / 32;
  const uint8_t* wc[4];
  const uint8_t* ws[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = ((int64_t)e * 2 + (i >> 1)) * a.hidden + h0 + 16 * (i & 1) + r;
    wc[i] = a.w13c + row * cols + 16 * q;
    ws[i] = a.w13s + row * scols;
  }
  const uint8_t* xc[G];
  const uint8_t* xs[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int t = list[min(16 * g + r, n - 1)] / a.topk;   // columns past n repeat the last; not stored
    xc[g] = a.xc + (int64_t)t * a.d + 16 * q;
    xs[g] = a.xs + (int64_t)t * scols;
  }
  v4f_m acc[4][G];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[i][g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 2;   // steps whose weights are in flight together; past the end the last one again, unused
  for (int s = first; s < last; s += U) {
    u32x4_m w[U][4];
    uint32_t sw[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(s + u, last - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[u][i] = *reinterpret_cast<const u32x4_m*>(wc[i] + at * 64);
        sw[u][i] = *reinterpret_cast<const uint32_t*>(ws[i] + at * 4);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= last) break;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint8_t* p = xc[g] + (s + u) * 128;
        const u32x4_m lo = *reinterpret_cast<const u32x4_m*>(p), hi = *reinterpret_cast<const u32x4_m*>(p + 64);
        const uint32_t sx = *reinterpret_cast<const uint32_t*>(xs[g] + (s + u) * 4) >> (8 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i][g] = mma_w4x8(frag4(w[u][i]), frag8(lo, hi), acc[i][g], sw[u][i] >> (8 * q), sx);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][i][q][r] = acc[i][g];
    __syncthreads();
    // thread -> token column c, hidden column i; 32 neighbouring lanes hold one MXFP8 block
    const int c = threadIdx.x >> 5, i = threadIdx.x & 31;
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int v = 0; v < kUpWaves; ++v) {
      gate += sums[v][i >> 4][(i >> 2) & 3][c][i & 3];
      up += sums[v][2 + (i >> 4)][(i >> 2) & 3][c][i & 3];
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

// Grid: hidden / 32 tiles x slots.  GMAX: groups of 16 tokens an expert can have.
template <int GMAX, bool ROUTE>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(Moe a) {
  __shared__ UpSums sums;
  __shared__ uint16_t list[kMaxTokens];
  __shared__ int count, found;
  const int e = expert_of_slot<ROUTE>(a, blockIdx.y, &found);
  if (e < 0) return;
  const int n = pairs_of_expert<ROUTE>(a, e, list, &count, blockIdx.x == 0);
  if (n == 0 || (a.slots != a.experts && list[0] != blockIdx.y)) return;
  const int h0 = blockIdx.x * 32;
  if (GMAX == 1 || n <= 16) up_tiles<1>(a, e, h0, list, n, sums);
  else if (GMAX == 2 || n <= 32) up_tiles<2>(a, e, h0, list, n, sums);
  else up_tiles<GMAX < 4 ? 1 : 4>(a, e, h0, list, n, sums);
}

constexpr int kDownWaves = 16;
constexpr int kDownSteps = 4;   // most K steps of a unit of work

// One expert's down product for 16 output rows over K steps [s0, s1), at most kDownSteps, added with the pairs'
// weights to this wave's own sums (out[token][16]).
template <int G>
__device__ void down_tile(const Moe& a, int e, int n0, int s0, int s1, const uint16_t* list, int n, const float* wts,
                          float (*out)[16]) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t row = (int64_t)e * a.d + n0 + r, cols = a.hidden / 2, scols = a.hidden / 32;
  const uint8_t* wc = a.w2c + row * cols + 16 * q;
  const uint8_t* ws = a.w2s + row * scols;
  const uint8_t* hc[G];
  const uint8_t* hs[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t p = list[min(16 * g + r, n - 1)];
    hc[g] = a.hc + p * a.hidden + 16 * q;
    hs[g] = a.hs + p * scols;
  }
  v4f_m acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_m w[kDownSteps];   // all of the unit's weights in flight; past its end the last step again, unused
  uint32_t sw[kDownSteps];
#pragma unroll
  for (int u = 0; u < kDownSteps; ++u) {
    const int at = min(s0 + u, s1 - 1);
    w[u] = *reinterpret_cast<const u32x4_m*>(wc + at * 64);
    sw[u] = *reinterpret_cast<const uint32_t*>(ws + at * 4);
  }
#pragma unroll
  for (int u = 0; u < kDownSteps; ++u) {
    if (s0 + u >= s1) break;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t* p = hc[g] + (s0 + u) * 128;
      const u32x4_m lo = *reinterpret_cast<const u32x4_m*>(p), hi = *reinterpret_cast<const u32x4_m*>(p + 64);
      const uint32_t sh = *reinterpret_cast<const uint32_t*>(hs[g] + (s0 + u) * 4) >> (8 * q);
      acc[g] = mma_w4x8(frag4(w[u]), frag8(lo, hi), acc[g], sw[u] >> (8 * q), sh);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (16 * g + r < n) {
      const int p = list[16 * g + r];
      v4f_m* o = reinterpret_cast<v4f_m*>(&out[p / a.topk][4 * q]);
      *o += wts[p] * acc[g];
    }
}

// Grid: d / 16.  Work units are (used expert in rising order, range of its K steps), dealt to the
// waves in turn; each wave adds into sums of its own, which are joined in wave order.
template <int GMAX, bool ROUTE, bool BF16OUT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(Moe a) {
  constexpr int kTokens = 16 * GMAX;   // a.tokens is at most this
  __shared__ __align__(16) float out[kDownWaves][kTokens][16];
  __shared__ int16_t id[kMaxPairs];
  __shared__ float wts[kMaxPairs];
  __shared__ uint64_t used[8];         // experts that a token chose: experts <= 512
  __shared__ uint16_t lists[kDownWaves][kMaxTokens];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16;
  if (tid < 8) used[tid] = 0;
  for (int i = tid; i < kDownWaves * kTokens * 4; i += 64 * kDownWaves)
    reinterpret_cast<v4f_m*>(out)[i] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  if (tid < a.tokens) {   // one thread per token: its choices, weights and repeats
    const int p0 = tid * a.topk;
    float total = 0.0f, top = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
      const int e = a.ids[p0 + j];
      float w;
      if constexpr (ROUTE) {
        const float l = a.logits[(int64_t)tid * a.experts + e];
        if (j == 0) top = l;
        w = expf(l - top);
        total += w;
      } else {
        w = a.weights[p0 + j];
      }
      wts[p0 + j] = w;
      bool keep = e >= 0 && e < a.experts;
      if constexpr (!ROUTE) {
        for (int f = 0; keep && f < j; ++f)
          if (id[p0 + f] == e) {   // an earlier place holds this expert: its weight takes this one's too
            wts[p0 + f] += w;
            keep = false;
          }
      }
      id[p0 + j] = keep ? (int16_t)e : (int16_t)-1;
      if (keep) atomicOr(reinterpret_cast<unsigned long long*>(&used[e >> 6]), 1ull << (e & 63));
    }
    if constexpr (ROUTE) {
      for (int j = 0; j < a.topk; ++j) {
        const float w = wts[p0 + j] / total;
        wts[p0 + j] = w;
        if (blockIdx.x == 0) a.weights[p0 + j] = w;
      }
    }
  }
  __syncthreads();
  int active = 0;
  for (int i = 0; i < 8; ++i) active += __popcll(used[i]);
  // K steps per unit: enough units for every wave, at most four steps' loads in flight
  const int nk = a.hidden / 128, pairs = a.tokens * a.topk;
  const int per = min(max(active * nk / kDownWaves, 1), kDownSteps), parts = (nk + per - 1) / per;
  uint16_t* list = lists[wave];
  int unit = 0;   // first unit of the current expert
  for (int word = 0; word < 8; ++word) {
    // the builtin returns int: the low half must not be widened with its sign
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)used[word]);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(used[word] >> 32));
    uint64_t m = ((uint64_t)hi << 32) | lo;
    for (; m; m &= m - 1, unit += parts) {
      const int e = 64 * word + __builtin_ctzll(m);
      int k = (wave - unit % kDownWaves + kDownWaves) % kDownWaves;   // this wave's first part, if any
      if (k >= parts) continue;
      int n = 0;
      for (int p0 = 0; p0 < pairs; p0 += 64) {
        const bool hit = p0 + lane < pairs && id[p0 + lane] == e;
        const uint64_t b = __ballot(hit);
        if (hit) list[n + __popcll(b & ((1ull << lane) - 1ull))] = (uint16_t)(p0 + lane);
        n += __popcll(b);
      }
      __builtin_amdgcn_wave_barrier();   // the list is this wave's own: LDS keeps its order
      for (; k < parts; k += kDownWaves) {
        const int s0 = k * per, s1 = min(s0 + per, nk);
        if (GMAX == 1 || n <= 16) down_tile<1>(a, e, n0, s0, s1, list, n, wts, out[wave]);
        else if (GMAX == 2 || n <= 32) down_tile<2>(a, e, n0, s0, s1, list, n, wts, out[wave]);
        else down_tile<GMAX < 4 ? 1 : 4>(a, e, n0, s0, s1, list, n, wts, out[wave]);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * 8; i += 64 * kDownWaves) {   // two neighbouring columns per thread
    const int t = i >> 3, c = (i & 7) * 2;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) s0 += out[v][t][c], s1 += out[v][t][c + 1];
    const int64_t at = (int64_t)t * a.d + n0 + c;
    if constexpr (BF16OUT) {
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + at) = bf16_pair(s0, s1);
    } else {
      *reinterpret_cast<f32x2_m*>(static_cast<float*>(a.y) + at) = f32x2_m{s0, s1};
    }
  }
}

template <int GMAX, bool ROUTE>
void run(const Moe& a, bool bf16_out, hipStream_t st) {
  k_moe_up<GMAX, ROUTE><<<dim3(a.hidden / 32, a.slots), 64 * kUpWaves, 0, st>>>(a);
  if (bf16_out) k_moe_down<GMAX, ROUTE, true><<<a.d / 16, 64 * kDownWaves, 0, st>>>(a);
  else k_moe_down<GMAX, ROUTE, false><<<a.d / 16, 64 * kDownWaves, 0, st>>>(a);
}

template <bool ROUTE>
void run_tokens(const Moe& a, bool bf16_out, hipStream_t st) {
  if (a.tokens <= 16) run<1, ROUTE>(a, bf16_out, st);
  else if (a.tokens <= 32) run<2, ROUTE>(a, bf16_out, st);
  else run<4, ROUTE>(a, bf16_out, st);
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

// Scratch: logits, hidden codes, hidden scales.
int64_t moe_scratch(int64_t tokens, int64_t hidden, int64_t experts, int64_t topk) {
  return up16(tokens * experts * 4) + up16(tokens * topk * hidden) + up16(tokens * topk * (hidden / 32));
}

void launch_moe(const MoeArgs& m, hipStream_t st) {
  Moe a;
  a.xc = m.x_codes, a.xs = m.x_scales, a.w13c = m.w13_codes, a.w13s = m.w13_scales, a.w2c = m.w2_codes;
  a.w2s = m.w2_scales, a.tokens = m.tokens, a.d = m.d, a.hidden = m.hidden, a.experts = m.experts, a.topk = m.topk;
  a.slots = m.tokens * m.topk < m.experts ? m.tokens * m.topk : m.experts;
  a.ids = m.ids, a.weights = m.weights, a.y = m.y;
  float* logits = static_cast<float*>(m.scratch);
  a.logits = logits;
  a.hc = static_cast<uint8_t*>(m.scratch) + up16((int64_t)m.tokens * m.experts * 4);
  a.hs = a.hc + up16((int64_t)m.tokens * m.topk * m.hidden);
  if (!m.router_w) {
    run_tokens<false>(a, m.bf16_out, st);
    return;
  }
  const dim3 grid((m.experts + 15) / 16, (m.tokens + 15) / 16);
  if (m.router_bf16)
    k_moe_logits<uint16_t><<<grid, 1024, 0, st>>>(static_cast<const uint16_t*>(m.router_x),
                                                  static_cast<const uint16_t*>(m.router_w), m.tokens, m.d, m.experts,
                                                  logits);
  else
    k_moe_logits<float><<<grid, 1024, 0, st>>>(static_cast<const float*>(m.router_x),
                                               static_cast<const float*>(m.router_w), m.tokens, m.d, m.experts, logits);
  run_tokens<true>(a, m.bf16_out, st);
}

}  // namespace fp4q
