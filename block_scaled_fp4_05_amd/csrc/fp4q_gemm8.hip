// C = A B^T with A [m][k] in MXFP8 (activations) and B [n][k] in MXFP4 (weights), both along k,
// accumulated in fp32.
//
//   C[i][j] = sum over K blocks b of 2^(ea + eb - 254) * sum over t in b of a[i][t] b[j][t]
//
// Two forms: few rows of A (k_gemm8_rows, bound by reading B once) and tiles in LDS
// (k_gemm8_tile, bound by the matrix cores).
#include "fp4q_mx8.hpp"

namespace fp4q {
namespace {

// -----------------------------------------------------------------------------------------
// Few rows.  A workgroup takes 16 rows of B and every row of A (G groups of 16); its waves
// split k into contiguous ranges and join their sums in LDS, in wave order.  B's codes go from
// memory to the matrix core's registers without a stop, since no two waves want the same ones.
// -----------------------------------------------------------------------------------------
template <int G, int WAVES, bool BF16OUT>
__global__ __launch_bounds__(64 * WAVES) void k_gemm8_rows(const uint8_t* __restrict__ ac,
                                                           const uint8_t* __restrict__ as,
                                                           const uint8_t* __restrict__ bc,
                                                           const uint8_t* __restrict__ bs, int M, int N, int K,
                                                           void* __restrict__ cout) {
  __shared__ v4f_m sums[WAVES][G][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int nk = K / 128;
  const int first = (int)((int64_t)nk * wave / WAVES), last = (int)((int64_t)nk * (wave + 1) / WAVES);
  // rows past an operand's end read its last row; their results are not stored
  const int64_t brow = min(n0 + r, N - 1);
  const uint8_t* bcp = bc + brow * (K / 2) + 16 * q;
  const uint8_t* bsp = bs + brow * (K / 32);
  const uint8_t* acp[G];
  const uint8_t* asp[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t arow = min(16 * g + r, M - 1);
    acp[g] = ac + arow * K + 16 * q;
    asp[g] = as + arow * (K / 32);
  }
  v4f_m acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 4;   // steps whose loads are in flight together
  int s = first;
  for (; s + U <= last; s += U) {
    u32x4_m b[U];
    uint32_t sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      b[u] = *reinterpret_cast<const u32x4_m*>(bcp + (int64_t)(s + u) * 64);
      sb[u] = *reinterpret_cast<const uint32_t*>(bsp + (s + u) * 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint8_t* p = acp[g] + (int64_t)(s + u) * 128;
        const u32x4_m lo = *reinterpret_cast<const u32x4_m*>(p), hi = *reinterpret_cast<const u32x4_m*>(p + 64);
        const uint32_t sa = *reinterpret_cast<const uint32_t*>(asp[g] + (s + u) * 4);
        acc[g] = mma_w4x8(frag4(b[u]), frag8(lo, hi), acc[g], sb[u] >> (8 * q), sa >> (8 * q));
      }
  }
  for (; s < last; ++s) {
    const u32x4_m b = *reinterpret_cast<const u32x4_m*>(bcp + (int64_t)s * 64);
    const uint32_t sb = *reinterpret_cast<const uint32_t*>(bsp + s * 4);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t* p = acp[g] + (int64_t)s * 128;
      const u32x4_m lo = *reinterpret_cast<const u32x4_m*>(p), hi = *reinterpret_cast<const u32x4_m*>(p + 64);
      const uint32_t sa = *reinterpret_cast<const uint32_t*>(asp[g] + s * 4);
      acc[g] = mma_w4x8(frag4(b), frag8(lo, hi), acc[g], sb >> (8 * q), sa >> (8 * q));
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) sums[wave][g][lane] = acc[g];
  __syncthreads();
  for (int t = threadIdx.x; t < G * 64; t += 64 * WAVES) {
    const int g = t >> 6, l = t & 63;
    v4f_m v = sums[0][g][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w][g][l];
    const int row = 16 * g + (l & 15), col = n0 + 4 * (l >> 4);
    if (row >= M || col >= N) continue;
    const int64_t at = (int64_t)row * N + col;
    const bool whole = (N & 3) == 0;   // then col + 4 <= N and the address is a multiple of four elements
    if constexpr (BF16OUT) {
      const uint32_t p0 = bf16_pair(v[0], v[1]), p1 = bf16_pair(v[2], v[3]);
      uint16_t* c = static_cast<uint16_t*>(cout) + at;
      if (whole) {
        *reinterpret_cast<u32x2_m*>(c) = u32x2_m{p0, p1};
      } else {
        c[0] = (uint16_t)p0;
        if (col + 1 < N) c[1] = (uint16_t)(p0 >> 16);
        if (col + 2 < N) c[2] = (uint16_t)p1;
        if (col + 3 < N) c[3] = (uint16_t)(p1 >> 16);
      }
    } else {
      float* c = static_cast<float*>(cout) + at;
      if (whole) {
        *reinterpret_cast<v4f_m*>(c) = v;
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (col + x < N) c[x] = v[x];
      }
    }
  }
}

// -----------------------------------------------------------------------------------------
// Tiles.  Four waves, 2 x 2, each 32 MI x 32 NJ of C in 32 x 32 blocks; a K step is 128
// elements: 128 bytes of A and 64 of B per row, copied straight into one of S LDS stages by
// global_load_lds.
// -----------------------------------------------------------------------------------------

// 16-byte chunk c of staged row r sits at position c ^ swz: 16 consecutive rows at one chunk
// fall in distinct bank groups, for rows of eight chunks (A) and of four (B).
__device__ __forceinline__ uint32_t swz_a(uint32_t r) {
  return ((r >> 1) & 1u) | (((r >> 2) & 1u) << 1) | (((r ^ (r >> 3)) & 1u) << 2);
}
__device__ __forceinline__ uint32_t swz_b(uint32_t r) { return ((r >> 2) & 1u) | ((((r >> 1) ^ (r >> 3)) & 1u) << 1); }
// Word d of a row's 16 scale bytes (four steps) sits at position d ^ swz_s(row).
__device__ __forceinline__ uint32_t swz_s(uint32_t r) { return (r >> 3) & 3u; }

// One wave's copy of 64 pieces of 16 (4) bytes into 64 consecutive ones of LDS.
__device__ __forceinline__ void copy16(const void* from, void* lds) {
  __builtin_amdgcn_global_load_lds(from, lds, 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void* from, void* lds) {
  __builtin_amdgcn_global_load_lds(from, lds, 4, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Barrier that leaves later steps' loads in flight; each wave has waited for its own loads of
// the step about to be read, and its LDS reads are complete.
__device__ __forceinline__ void tile_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// Workgroup b -> tile.  The workgroups of one XCD (b % 8) take a contiguous range of an order
// that walks groups of four tile rows column by column, so they share rows in its L2.
__device__ __forceinline__ void tile_of(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, q = total >> 3, r = total & 7, x = b & 7;
  const int t = x * q + min(x, r) + (b >> 3);
  constexpr int kRows = 4;
  const int group = t / (kRows * tiles_n), first = group * kRows, gh = min(kRows, tiles_m - first);
  const int rem = t - group * kRows * tiles_n;
  tn = rem / gh;
  tm = first + rem % gh;
}

template <int MI, int NJ, int S>
struct TileLds {
  static constexpr int BM = 64 * MI, BN = 64 * NJ;
  struct Stage {
    u32x4_m a[BM * 8];
    u32x4_m b[BN * 4];
  };
  struct Scales {   // four steps: 16 bytes per row, A's rows, then B's
    uint32_t w[(BM + BN) * 4];
  };
  struct Loop {
    Stage st[S];
    Scales sc[3];
  };
  union {
    Loop loop;
    uint16_t out[4][32 * MI * 32 * NJ];   // each wave's block of C on its way out, bf16
  };
  // loads per wave and step: codes, and the next scale chunk's slices of 64 rows dealt over its
  // four steps (a chunk of only two slices is loaded twice)
  static constexpr int kSlices = (MI + NJ) >= 4 ? (MI + NJ) / 4 : 1;
  static constexpr int kLoads = 2 * MI + NJ + kSlices;
};

template <int MI, int NJ>
struct Frags {
  v8i_m a[MI], b[NJ];
};

template <int MI, int NJ, int S, bool BF16OUT>
__global__ __launch_bounds__(256) void k_gemm8_tile(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                    const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
                                                    int M, int N, int K, int tiles_m, int tiles_n,
                                                    void* __restrict__ cout) {
  using Lds = TileLds<MI, NJ, S>;
  static_assert((MI + NJ) % 4 == 0 || (MI == 1 && NJ == 1), "scale slices per step");
  __shared__ Lds lds_;
  auto* st = lds_.loop.st;
  auto* sc = lds_.loop.sc;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * Lds::BM, n0 = tn * Lds::BN;
  const int nk = K / 128;
  const int64_t lda = K, ldb = K / 2, lds = K / 32;   // bytes per row

  // A's chunk p = 256 j + tid is row 32 j + tid / 8, position tid % 8; B's is row 64 j + tid / 4,
  // position tid % 4.  Rows past the matrix read its last row (their C rows or columns are not
  // stored), steps past k the last step (never used).
  const int ra = tid >> 3, rb = tid >> 2;
  const int ca = (tid & 7) ^ (int)swz_a((uint32_t)ra), cb = (tid & 3) ^ (int)swz_b((uint32_t)rb);
  uint32_t oa[2 * MI], ob[NJ];   // the lane's row past its group's first, in bytes (< 2^31: k <= 2^25)
#pragma unroll
  for (int j = 0; j < 2 * MI; ++j)
    oa[j] = (uint32_t)((min(m0 + 32 * j + ra, M - 1) - min(m0 + 32 * j, M - 1)) * (int)lda);
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    ob[j] = (uint32_t)((min(n0 + 64 * j + rb, N - 1) - min(n0 + 64 * j, N - 1)) * (int)ldb);
  // Scale slice i of a chunk: 64 rows of A (i < MI) or of B; this lane fetches row 16 wave +
  // lane / 4 of it, word 4 chunk + ((lane % 4) ^ swz_s(row)), clamped to the row's last.
  const int srow = 16 * wave + (lane >> 2);
  const int sword = (lane & 3) ^ (int)swz_s((uint32_t)srow);
  auto issue_scales = [&](int chunk, int i) {
    const bool of_a = i < MI;   // uniform selects: a branch here would cut the step into pieces
    const uint8_t* from = of_a ? as : bs;
    const int row = (of_a ? m0 + 64 * i : n0 + 64 * (i - MI)) + srow, end = of_a ? M : N;
    copy4(from + (int64_t)min(row, end - 1) * lds + 4 * min(4 * chunk + sword, nk - 1),
          &sc[chunk % 3].w[(64 * i + 16 * wave) * 4]);
  };
  auto issue = [&](int ks) {
    auto& s = st[ks % S];
    const int kc = min(ks, nk - 1);
#pragma unroll
    for (int j = 0; j < 2 * MI; ++j)
      copy16(ac + (int64_t)min(m0 + 32 * j, M - 1) * lda + (oa[j] + (uint32_t)(kc * 128 + ca * 16)),
             &s.a[j * 256 + wave * 64]);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      copy16(bc + (int64_t)min(n0 + 64 * j, N - 1) * ldb + (ob[j] + (uint32_t)(kc * 64 + cb * 16)),
             &s.b[j * 256 + wave * 64]);
    const int chunk = (ks >> 2) + 1, part = ks & 3;
    if constexpr (MI + NJ >= 4) {
#pragma unroll
      for (int i = 0; i < Lds::kSlices; ++i) issue_scales(chunk, part * Lds::kSlices + i);
    } else {
      issue_scales(chunk, part & 1);
    }
  };

  // Fragment addresses: row (wave's first + 32 i + fr); sub-step u (64 K elements) takes A's
  // chunks 4 u + fh and 4 u + 2 + fh and B's chunk 2 u + fh.
  const int wm = wave & 1, wn = wave >> 1, fr = lane & 31, fh = lane >> 5;
  const uint32_t za = swz_a((uint32_t)fr), zb = swz_b((uint32_t)fr), zs = swz_s((uint32_t)fr);
  const int rowA = wm * 32 * MI + fr, rowB = wn * 32 * NJ + fr;
  auto read = [&](int ks, int u, Frags<MI, NJ>& f) {
    const auto& s = st[ks % S];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const u32x4_m* p = s.a + (rowA + 32 * i) * 8;
      f.a[i] = frag8(p[(uint32_t)(4 * u + fh) ^ za], p[(uint32_t)(4 * u + 2 + fh) ^ za]);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) f.b[j] = frag4(s.b[(rowB + 32 * j) * 4 + ((uint32_t)(2 * u + fh) ^ zb)]);
  };
  // Scale words of a step, shifted so that byte 2 u is the lane's block of sub-step u.
  auto read_scales = [&](int ks, uint32_t* wa, uint32_t* wb) {
    const auto& c = sc[(ks >> 2) % 3];
    const uint32_t d = (uint32_t)(ks & 3) ^ zs;
#pragma unroll
    for (int i = 0; i < MI; ++i) wa[i] = c.w[(rowA + 32 * i) * 4 + d] >> (8 * fh);
#pragma unroll
    for (int j = 0; j < NJ; ++j) wb[j] = c.w[(Lds::BM + rowB + 32 * j) * 4 + d] >> (8 * fh);
  };

  v16f_m acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v16f_m{};

  // While one sub-step's MFMAs run, the next one's fragments are read.  The barrier that
  // publishes step ks + 1 sits between the two sub-steps of step ks, when all of step ks is in
  // registers; its stage then takes step ks + S.  Step ks + 1 has landed once only the loads of
  // the S - 2 steps after it are outstanding.
#pragma unroll
  for (int i = 0; i < MI + NJ; ++i) issue_scales(0, i);
#pragma unroll
  for (int s = 0; s < S; ++s) issue(s);
  wait_loads<(S - 1) * Lds::kLoads>();
  tile_barrier();
  Frags<MI, NJ> f0, f1;
  uint32_t wa[MI], wb[NJ];
  read(0, 0, f0);
  read_scales(0, wa, wb);
  for (int ks = 0; ks < nk; ++ks) {
    read(ks, 1, f1);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = mma_x8w4_lo(f0.a[i], f0.b[j], acc[i][j], wa[i], wb[j]);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t va[MI], vb[NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i) va[i] = wa[i];
#pragma unroll
    for (int j = 0; j < NJ; ++j) vb[j] = wb[j];
    wait_loads<(S - 2) * Lds::kLoads>();
    tile_barrier();
    issue(ks + S);
    read_scales(ks + 1, wa, wb);
    read(ks + 1, 0, f0);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = mma_x8w4_hi(f1.a[i], f1.b[j], acc[i][j], va[i], vb[j]);
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_loads<0>();   // the loads past k land before LDS is used again

  // Register t of block (i, j) is row 8 (t / 4) + 4 fh + t % 4, column fr of that block.
  const int br = m0 + wm * 32 * MI, bc0 = n0 + wn * 32 * NJ;
  if constexpr (BF16OUT) {
    // through LDS, so that a store writes 16 bytes of a row
    tile_barrier();
    uint16_t* e = lds_.out[wave];
    constexpr int W = 32 * NJ, LPR = W / 8;   // columns of the block, lanes per row
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
          const uint32_t p = bf16_pair(acc[i][j][t], acc[i][j][t + 1]);
          uint16_t* d = e + (32 * i + 8 * (t >> 2) + 4 * fh + (t & 3)) * W + 32 * j + fr;
          d[0] = (uint16_t)p;
          d[W] = (uint16_t)(p >> 16);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    uint16_t* c16 = static_cast<uint16_t*>(cout);
    const bool vec = (N & 7) == 0;
    for (int it = 0; it < 32 * MI * LPR / 64; ++it) {
      const int row = it * (64 / LPR) + lane / LPR, c8 = (lane % LPR) * 8;
      if (br + row >= M) continue;
      uint16_t* dst = c16 + (int64_t)(br + row) * N + bc0 + c8;
      const uint16_t* src = e + row * W + c8;
      if (vec && bc0 + c8 + 8 <= N) {
        *reinterpret_cast<u32x4_m*>(dst) = *reinterpret_cast<const u32x4_m*>(src);
      } else {
        for (int x = 0; x < 8 && bc0 + c8 + x < N; ++x) dst[x] = src[x];
      }
    }
  } else {
    float* c32 = static_cast<float*>(cout);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int col = bc0 + 32 * j + fr;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const int row = br + 32 * i + 8 * (t >> 2) + 4 * fh + (t & 3);
          if (row < M && col < N) c32[(int64_t)row * N + col] = acc[i][j][t];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

struct Gemm8 {
  const uint8_t *ac, *as, *bc, *bs;
  int m, n, k;
  void* c;
  hipStream_t st;
};

template <int MI, int NJ, int S, bool BF16OUT>
bool run_tile(const Gemm8& g) {
  const int64_t tm = (g.m + (int64_t)64 * MI - 1) / (64 * MI), tn = (g.n + (int64_t)64 * NJ - 1) / (64 * NJ);
  if (tm * tn > (1 << 24) - 1) return false;   // a launch has at most 2^32 threads
  k_gemm8_tile<MI, NJ, S, BF16OUT><<<(unsigned)(tm * tn), 256, 0, g.st>>>(g.ac, g.as, g.bc, g.bs, g.m, g.n, g.k,
                                                                          (int)tm, (int)tn, g.c);
  return true;
}

template <int G, bool BF16OUT>
void run_rows(const Gemm8& g) {
  const unsigned grid = (unsigned)((g.n + (int64_t)15) / 16);
  k_gemm8_rows<G, 8, BF16OUT><<<grid, 512, 0, g.st>>>(g.ac, g.as, g.bc, g.bs, g.m, g.n, g.k, g.c);
}

template <bool BF16OUT>
bool run(const Gemm8& g) {
  if (g.m <= 64) {
    if ((g.n + (int64_t)15) / 16 > (1 << 22)) return false;
    if (g.m <= 16) run_rows<1, BF16OUT>(g);
    else if (g.m <= 32) run_rows<2, BF16OUT>(g);
    else run_rows<4, BF16OUT>(g);
    return true;
  }
  const auto tiles = [&](int t) { return ((g.m + (int64_t)t - 1) / t) * ((g.n + (int64_t)t - 1) / t); };
  if (tiles(256) >= 192) return run_tile<4, 4, 2, BF16OUT>(g);
  if (tiles(128) >= 192) return run_tile<2, 2, 2, BF16OUT>(g);
  return run_tile<1, 1, 4, BF16OUT>(g);
}

}  // namespace

bool launch_gemm_mxfp8_mxfp4(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int64_t m,
                             int64_t n, int64_t k, bool bf16_out, void* c, hipStream_t st) {
  const Gemm8 g{ac, as, bc, bs, (int)m, (int)n, (int)k, c, st};
  return bf16_out ? run<true>(g) : run<false>(g);
}

}  // namespace fp4q
