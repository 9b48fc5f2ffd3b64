// C = A B^T with A [m][k] in MXFP8 (activations) and B [n][k] in MXFP4 (weights), both along k,
// accumulated in fp32.
//
//   C[i][j] = sum over K blocks b of 2^(ea + eb - 254) * sum over t in b of a[i][t] b[j][t]
//
// Two forms: few rows of A (k_gemm8_rows, bound by reading B once) and tiles in LDS
// (k_gemm8_tile, bound by the matrix cores).
#include "fp4q_mx8.hpp"
#include <type_traits>

namespace fp4q {
namespace {

// -----------------------------------------------------------------------------------------
// Few rows.  A workgroup takes 16 NT rows of B and 16 G rows of A; its waves split k into
// contiguous ranges and join their sums in LDS, in wave order.
//
// A matrix instruction's lanes 0..15 hold 16 different rows, and a load in that layout touches 16
// lines per 16 lanes, which holds a CU at about 13 bytes per clock.  So eight lanes load 128 bytes
// of a row, and a pass through the wave's own part of LDS (no barrier) deals the rows out: 16-byte
// chunk c of row i sits at c ^ (i % 8).  (us, loads in the instruction's layout against these: 32 rows
// of A, n 28672, k 8192 58.5 / 38; 16 rows, n 4096, k 14336 16.5 / 12.5; one row, where A's lines
// are few either way and DIRECT loads its fragments, n 28672, k 8192 33.4 / 26.2.)
// Bound by reading B: one row, n 28672, k 8192 (125 MB) at 4.8 TB/s; below some 20 MB by the launch
// and one trip to memory: one row, n 4096, k 4096 (8.9 MB) 3.9 us.
// -----------------------------------------------------------------------------------------
template <int G, int NT, int WAVES, bool DIRECT, bool BF16OUT>
__global__ __launch_bounds__(64 * WAVES, G == 1 && NT <= 2 ? 4 : 2) void k_gemm8_rows(const uint8_t* __restrict__ ac,
                                                           const uint8_t* __restrict__ as,
                                                           const uint8_t* __restrict__ bc,
                                                           const uint8_t* __restrict__ bs, int M, int N, int K,
                                                           void* __restrict__ cout) {
  // per wave: NT blocks of B (two steps each) and 2 G blocks of A (one step each), 16 rows x 128 bytes
  constexpr int kBlocks = NT + (DIRECT ? 0 : 2 * G);
  union Lds {
    u32x4_m blocks[WAVES][kBlocks][128];
    v4f_m sums[WAVES][NT * G][64];
  };
  __shared__ Lds lds_;
  auto& sums = lds_.sums;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * (16 * NT);
  const int m0 = blockIdx.y * (16 * G);
  const int nk = K / 128;
  const int first = (int)((int64_t)nk * wave / WAVES), last = (int)((int64_t)nk * (wave + 1) / WAVES);
  // Rows past an operand's end read its last row; their results are not stored.
  const int lr = lane >> 3, lc = (lane & 7) * 16;
  const uint8_t *b0 = bc + (int64_t)n0 * (K / 2), *a0 = ac + (int64_t)m0 * K;
  uint32_t bo[NT][2], ao[G][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int t = 0; t < NT; ++t) bo[t][h] = (uint32_t)((min(n0 + 16 * t + 8 * h + lr, N - 1) - n0) * (K / 2));
#pragma unroll
    for (int g = 0; g < G; ++g) ao[g][h] = (uint32_t)((min(m0 + 16 * g + (DIRECT ? r : 8 * h + lr), M - 1) - m0) * K);
  }
  // Scale words likewise: lanes 16 i .. hold row tile i's (B's tiles, then A's), dealt out by lane swaps.
  constexpr int kTiles = NT + G, kWords = (kTiles + 3) / 4;
  const uint8_t* sp[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int tile = 4 * i + q;
    const int row = tile < NT ? min(n0 + 16 * tile + r, N - 1) : min(m0 + 16 * (tile - NT) + r, M - 1);
    sp[i] = (tile < NT ? bs : as) + (int64_t)row * (K / 32);
  }
  v4f_m acc[NT][G];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[t][g] = v4f_m{0.0f, 0.0f, 0.0f, 0.0f};
  // Four steps' loads in flight, the next four's issued before the last two are multiplied.
  struct Group {
    u32x4_m b[2][NT][2], a[4][G][2], sc[kWords];
  } f;
  const auto fetch = [&](int s) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (s + 2 * p < last)   // (a row that ends within the two steps: its last bytes again, not used)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            f.b[p][t][h] = load16(b0, bo[t][h] + (uint32_t)min(s * 64 + 128 * p + lc, K / 2 - 16));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s + u < last)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            f.a[u][g][h] = load16(a0, ao[g][h] + (uint32_t)((s + u) * 128 + (DIRECT ? 64 * h + 16 * q : lc)));
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (4 * i + q < kTiles) f.sc[i] = scale_words(sp[i], 0, s, nk);
  };
  auto* block = lds_.blocks[wave];
  const int put = lr * 8 + ((lane & 7) ^ lr);
  const auto get = [&](int blk, int c) { return block[blk][r * 8 + (c ^ (r & 7))]; };
  if (first < last) fetch(first);
  for (int s = first; s < last; s += 4) {
    u32x4_m a[4][G][2];   // DIRECT: the fragments as loaded
    if constexpr (DIRECT)
#pragma unroll
      for (int i = 0; i < 8 * G; ++i) a[i / (2 * G)][i / 2 % G][i & 1] = f.a[i / (2 * G)][i / 2 % G][i & 1];
    uint32_t sw[4][4 * kWords];   // by step and tile, the lane's byte first
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t o[4];
        spread(f.sc[i][u], o);
#pragma unroll
        for (int j = 0; j < 4; ++j) sw[u][4 * i + j] = o[j] >> (8 * q);
      }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < NT; ++t) block[t][put + 64 * h] = f.b[p][t][h];
        if constexpr (!DIRECT)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int g = 0; g < G; ++g) block[NT + u * G + g][put + 64 * h] = f.a[2 * p + u][g][h];
      }
      wave_lds_fence();
      if (p == 1 && s + 4 < last) fetch(s + 4);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (s + 2 * p + u < last) {
          v8i_m w[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) w[t] = frag4(get(t, 4 * u + q));
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const v8i_m x = DIRECT ? frag8(a[2 * p + u][g][0], a[2 * p + u][g][1])
                                   : frag8(get(NT + u * G + g, q), get(NT + u * G + g, 4 + q));
#pragma unroll
            for (int t = 0; t < NT; ++t)
              acc[t][g] = mma_w4x8(w[t], x, acc[t][g], sw[2 * p + u][t], sw[2 * p + u][NT + g]);
          }
        }
      wave_lds_fence();
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < G; ++g) sums[wave][t * G + g][lane] = acc[t][g];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * G * 64; i += 64 * WAVES) {
    const int tg = i >> 6, l = i & 63;
    v4f_m v = sums[0][tg][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w][tg][l];
    const int row = m0 + 16 * (tg % G) + (l & 15), col = n0 + 16 * (tg / G) + 4 * (l >> 4);
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
// Bound, on large shapes, by the matrix cores with their copies beside them (an E4M3 operand runs at
// the 8-bit rate): 8192^3 in 388 to 408 us from run to run, 2.7 to 2.8 PFLOP/s, MFMA busy 65 % of the cycles (to
// fp32 415); with few tiles by each workgroup's own chain of K steps: 193 x 4099 x 4224 in 16.7 us, 33 steps of
// half a microsecond on 132 of the 256 CUs, each bringing in 14 bytes per clock of the 32 it could.
// -----------------------------------------------------------------------------------------

// 16-byte chunk c of staged row r sits at position c ^ swz: 16 consecutive rows at one chunk
// fall in distinct bank groups, for rows of eight chunks (A) and of four (B).
__device__ __forceinline__ uint32_t swz_a(uint32_t r) {
  return ((r >> 1) & 1u) | (((r >> 2) & 1u) << 1) | (((r ^ (r >> 3)) & 1u) << 2);
}
__device__ __forceinline__ uint32_t swz_b(uint32_t r) { return ((r >> 2) & 1u) | ((((r >> 1) ^ (r >> 3)) & 1u) << 1); }

// One wave's copy of 64 pieces of 16 (4) bytes into 64 consecutive ones of LDS.
__device__ __forceinline__ void copy16(const void* from, void* lds) {
  __builtin_amdgcn_global_load_lds(from, lds, 16, 0, 0);
}

__device__ __forceinline__ void copy4(const void* from, void* lds) {
  __builtin_amdgcn_global_load_lds(from, lds, 4, 0, 0);
}

// Word d of a row's 16 scale bytes sits at position d ^ swz_s(row) where they are copied as words.
__device__ __forceinline__ uint32_t swz_s(uint32_t r) { return (r >> 3) & 3u; }

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

template <int MI, int NJ, int S, bool WIDE>
struct TileLds {
  static constexpr int BM = 64 * MI, BN = 64 * NJ;
  struct Stage {
    u32x4_m a[BM * 8];
    u32x4_m b[BN * 4];
  };
  // Scales come in chunks of four steps, one 16-byte piece per row (A's rows, then B's), in slices of
  // 64 rows that travel with the codes of the four steps before, S steps ahead of use; a buffer is
  // written again once its chunk has been read: 2 + (S - 1) / 4 of them, rounded up.  Where k / 32 is
  // a multiple of 16 (WIDE) a slice is one wave's copy of 16 bytes per row.  Else a row starts at a
  // multiple of four bytes only, and it is four waves' copies of words; an instruction of either
  // kind costs about the same (8192^3: 387 us with pieces, 445 with words).  Loading unaligned pieces
  // into registers and writing them on took longer than the words (256 x 4096 x 4224: 15.3 against
  // 11.2 us), since the compiler waits for every copy in flight before the write.
  static constexpr int kBuffers = 2 + (S + 2) / 4;
  struct Loop {
    Stage st[S];
    u32x4_m sc[kBuffers][BM + BN];
  };
  union {
    Loop loop;
    uint16_t out[4][32 * MI * 32 * NJ];   // each wave's block of C on its way out, bf16
  };
  static constexpr int kSlices = (MI + NJ + 3) / 4;                   // words: slices per step
  static constexpr int kLoads = 2 * MI + NJ + (WIDE ? 0 : kSlices);   // at least so many copies per wave and step
};

template <int P>
using Phase = std::integral_constant<int, P>;

// The first S steps' copies.
template <int S, int I = 0, typename Issue>
__device__ __forceinline__ void issue_first(Issue& issue) {
  if constexpr (I < S) {
    issue(I, Phase<(I & 3)>{});
    issue_first<S, I + 1>(issue);
  }
}

template <int MI, int NJ>
struct Frags {
  v8i_m a[MI], b[NJ];
};

// Scheduling groups: one MFMA, then up to V copies and D LDS reads, N times.
template <int N, int V, int D>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int g = 0; g < N; ++g) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (V > 0) __builtin_amdgcn_sched_group_barrier(0x020, V, 0);
    if constexpr (D > 0) __builtin_amdgcn_sched_group_barrier(0x100, D, 0);
  }
}

template <int MI, int NJ, int S, bool WIDE, bool BF16OUT>
__global__ __launch_bounds__(256) void k_gemm8_tile(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                    const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
                                                    int M, int N, int K, int tiles_m, int tiles_n,
                                                    void* __restrict__ cout) {
  using Lds = TileLds<MI, NJ, S, WIDE>;
  __shared__ Lds lds_;
  auto* st = lds_.loop.st;
  auto& sc = lds_.loop.sc;
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
  // Slice i of a chunk is 64 rows of A (i < MI) or of B.  WIDE: lane l copies row l's 16 bytes.
  // Words: wave w copies rows 16 w .., lane l word l % 4 of row l / 4 of those, to word
  // (l % 4) ^ swz_s(row) of the row's piece.  Clamped to the row's last piece or word.
  const int srow = WIDE ? lane : 16 * wave + (lane >> 2);
  const int sword = WIDE ? 0 : (lane & 3) ^ (int)swz_s((uint32_t)srow);
  auto issue_scales = [&](int chunk, int i) {
    const bool of_a = i < MI;   // uniform selects: a branch here would cut the step into pieces
    const uint8_t* from = of_a ? as : bs;
    const int row = (of_a ? m0 + 64 * i : n0 + 64 * (i - MI)) + srow, end = of_a ? M : N;
    const uint8_t* at = from + (int64_t)min(row, end - 1) * lds;
    uint32_t* to = reinterpret_cast<uint32_t*>(&sc[chunk % Lds::kBuffers][64 * i + (WIDE ? 0 : 16 * wave)]);
    if constexpr (WIDE) copy16(at + 16 * min(chunk, nk / 4 - 1), to);
    else copy4(at + 4 * min(4 * chunk + sword, nk - 1), to);
  };
  // Copies of step ks; PHASE = ks % 4 where the loop knows it (the copies of pieces need no branch
  // then, which would make the compiler move the accumulators about), else -1.
  auto issue = [&](int ks, auto phase) {
    constexpr int PHASE = decltype(phase)::value;
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
    const int chunk = (ks >> 2) + 1;   // (the last slice again where there is room for more)
    if constexpr (!WIDE) {
#pragma unroll
      for (int i = 0; i < Lds::kSlices; ++i) issue_scales(chunk, min((ks & 3) * Lds::kSlices + i, MI + NJ - 1));
    } else if constexpr (4 * PHASE < MI + NJ) {
      issue_scales(chunk, min(4 * PHASE + wave, MI + NJ - 1));
    }
  };

  // Fragment addresses: row (wave's first + 32 i + fr); sub-step u (64 K elements) takes A's
  // chunks 4 u + fh and 4 u + 2 + fh and B's chunk 2 u + fh.
  const int wm = wave & 1, wn = wave >> 1, fr = lane & 31, fh = lane >> 5;
  const uint32_t za = swz_a((uint32_t)fr), zb = swz_b((uint32_t)fr);
  const uint32_t zs = WIDE ? 0u : swz_s((uint32_t)fr);
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
    const uint32_t* c = reinterpret_cast<const uint32_t*>(sc[(ks >> 2) % Lds::kBuffers]) + ((uint32_t)(ks & 3) ^ zs);
#pragma unroll
    for (int i = 0; i < MI; ++i) wa[i] = c[(rowA + 32 * i) * 4] >> (8 * fh);
#pragma unroll
    for (int j = 0; j < NJ; ++j) wb[j] = c[(Lds::BM + rowB + 32 * j) * 4] >> (8 * fh);
  };

  v16f_m acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v16f_m{};

  // Step ks + 1 has landed once only the copies of the S - 2 steps after it are outstanding; the
  // barrier then publishes it, and the stage of step ks, all of it in registers by then, takes
  // step ks + S.
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < MI + NJ; i += 4) issue_scales(0, min(i + wave, MI + NJ - 1));
  } else {
#pragma unroll
    for (int i = 0; i < MI + NJ; ++i) issue_scales(0, i);
  }
  issue_first<S>(issue);
  wait_loads<(S - 1) * Lds::kLoads>();
  tile_barrier();
  if constexpr (MI * NJ < 16) {
    // small tiles: a whole step's fragments are read while the one before is multiplied, so a step
    // has one barrier and one LDS latency
    struct Step {
      Frags<MI, NJ> f0, f1;
      uint32_t wa[MI], wb[NJ];
    } even, odd;
    const auto fetch = [&](int ks, Step& t) {
      read(ks, 0, t.f0);
      read(ks, 1, t.f1);
      read_scales(ks, t.wa, t.wb);
    };
    const auto turn = [&](int ks, auto phase, Step& t, Step& next) {
      wait_loads<(S - 2) * Lds::kLoads>();
      tile_barrier();
      issue(ks + S, phase);
      fetch(ks + 1, next);
      __builtin_amdgcn_sched_barrier(0);   // the reads go out before the MFMAs that cover them
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mma_x8w4_lo(t.f0.a[i], t.f0.b[j], acc[i][j], t.wa[i], t.wb[j]);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mma_x8w4_hi(t.f1.a[i], t.f1.b[j], acc[i][j], t.wa[i], t.wb[j]);
      __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0, even);
    if constexpr (WIDE) {   // nk is a multiple of four
      for (int ks = 0; ks < nk; ks += 4) {
        turn(ks, Phase<S & 3>{}, even, odd);
        turn(ks + 1, Phase<(S + 1) & 3>{}, odd, even);
        turn(ks + 2, Phase<(S + 2) & 3>{}, even, odd);
        turn(ks + 3, Phase<(S + 3) & 3>{}, odd, even);
      }
    } else {
      for (int ks = 0; ks < nk; ks += 2) {
        turn(ks, Phase<-1>{}, even, odd);
        if (ks + 1 < nk) turn(ks + 1, Phase<-1>{}, odd, even);
      }
    }
  } else {
    // large tiles have no registers for that: while one sub-step's MFMAs run, the next one's
    // fragments are read, with the barrier between the two sub-steps of a step, and reads and
    // copies are dealt one by one between the MFMAs
    Frags<MI, NJ> f0, f1;
    uint32_t wa[MI], wb[NJ];
    read(0, 0, f0);
    read_scales(0, wa, wb);
    const auto turn = [&](int ks, auto phase) {
      read(ks, 1, f1);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mma_x8w4_lo(f0.a[i], f0.b[j], acc[i][j], wa[i], wb[j]);
      interleave<12, 0, 1>();
      interleave<4, 0, 0>();
      __builtin_amdgcn_sched_barrier(0);
      uint32_t va[MI], vb[NJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) va[i] = wa[i];
#pragma unroll
      for (int j = 0; j < NJ; ++j) vb[j] = wb[j];
      wait_loads<(S - 2) * Lds::kLoads>();
      tile_barrier();
      issue(ks + S, phase);
      read_scales(ks + 1, wa, wb);
      read(ks + 1, 0, f0);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mma_x8w4_hi(f1.a[i], f1.b[j], acc[i][j], va[i], vb[j]);
      interleave<12, 1, 2>();
      interleave<4, 1, 0>();
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (WIDE) {
      for (int ks = 0; ks < nk; ks += 4) {
        turn(ks, Phase<S & 3>{});
        turn(ks + 1, Phase<(S + 1) & 3>{});
        turn(ks + 2, Phase<(S + 2) & 3>{});
        turn(ks + 3, Phase<(S + 3) & 3>{});
      }
    } else {
      for (int ks = 0; ks < nk; ++ks) turn(ks, Phase<-1>{});
    }
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
    wave_lds_fence();   // the rows are read by other lanes of the wave than wrote them
    uint16_t* c16 = static_cast<uint16_t*>(cout);
    const bool vec = (N & 7) == 0;
    for (int it = 0; it < 32 * MI * LPR / 64; ++it) {
      const int row = it * (64 / LPR) + lane / LPR, c8 = (lane % LPR) * 8;
      if (br + row >= M) continue;
      uint16_t* dst = c16 + (int64_t)(br + row) * N + bc0 + c8;
      const uint16_t* src = e + row * W + c8;
      if (vec && bc0 + c8 <= N - 8) {   // (bc0 + c8 + 8 may pass 2^31)
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

constexpr int kCus = 256;   // compute units of the GPU

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
  auto kern = g.k % 512 == 0 ? k_gemm8_tile<MI, NJ, S, true, BF16OUT> : k_gemm8_tile<MI, NJ, S, false, BF16OUT>;
  kern<<<(unsigned)(tm * tn), 256, 0, g.st>>>(g.ac, g.as, g.bc, g.bs, g.m, g.n, g.k, (int)tm, (int)tn, g.c);
  return true;
}

template <int G, int NT, int WAVES, bool DIRECT, bool BF16OUT>
void run_rows(const Gemm8& g) {
  const unsigned grid = (unsigned)((g.n + (int64_t)16 * NT - 1) / (16 * NT));
  const dim3 grid2(grid, (unsigned)((g.m + 16 * G - 1) / (16 * G)));
  k_gemm8_rows<G, NT, WAVES, DIRECT, BF16OUT><<<grid2, 64 * WAVES, 0, g.st>>>(g.ac, g.as, g.bc, g.bs, g.m, g.n, g.k,
                                                                              g.c);
}

template <bool BF16OUT>
bool run(const Gemm8& g) {
  if (g.m <= 32 && g.n <= 1 << 26) {   // (a launch has at most 2^32 threads)
    // Rows of B per workgroup: 16, or 32 where the workgroups of 16 take more than a round or two
    // (us at 16 / 32: one row of A, n 4096, k 4096 4.3 / 5.4; n 8192, k 8192 10.3 / 12.0; n 11008,
    // k 4096 9.1 / 8.5; n 32768, k 8192 32.2 / 28.7; 24 rows, n 4096, k 4096 6.0 / 6.8; n 6144,
    // k 4096 9.2 / 7.4).  64 took longer than 32 (n 32768, k 8192: 31.5).
    if (g.m <= 4) {
      if (g.n >= 40 * kCus) run_rows<1, 2, 4, true, BF16OUT>(g);
      else run_rows<1, 1, 8, true, BF16OUT>(g);
    } else if (g.m <= 16) {
      if (g.n >= 40 * kCus) run_rows<1, 2, 4, false, BF16OUT>(g);
      else run_rows<1, 1, 8, false, BF16OUT>(g);
    } else {
      if (g.n > 16 * kCus) run_rows<2, 2, 4, false, BF16OUT>(g);
      else run_rows<2, 1, 8, false, BF16OUT>(g);
    }
    return true;
  }
  // 64 rows of A likewise where that is one round: a tile's one wave of copies per 64 rows of B leaves
  // CUs idle then (us, tiles / rows: 64 x 4096 x 14336 36.0 / 23.0, 64 x 4096 x 4096 9.0 / 8.2, 128 x 640
  // x 8192 13.9 / 10.4).
  if (((g.n + (int64_t)15) / 16) * ((g.m + (int64_t)63) / 64) <= kCus) {
    run_rows<4, 1, 8, false, BF16OUT>(g);
    return true;
  }
  // The tile by what a round of one tile per CU takes, in units of a 64 x 64 tile's (measured at
  // k = 4096, us for one round: 64 x 64 8.7, 64 x 128 12.0, 128 x 128 19.7 alone and 18.0 each in
  // pairs, 256 x 256 41.7), times the rounds.
  const auto cost = [&](int bm, int bn, float round) {
    const int64_t t = ((g.m + (int64_t)bm - 1) / bm) * ((g.n + (int64_t)bn - 1) / bn);
    return round * (float)((t + kCus - 1) / kCus);
  };
  const float c[4] = {cost(64, 64, 1.0f), cost(64, 128, 1.35f), cost(128, 128, 2.0f), cost(256, 256, 4.6f)};
  const bool largest = c[3] <= c[0] && c[3] <= c[1] && c[3] <= c[2];
  if (!largest && (c[2] <= c[0] && c[2] <= c[1] ? run_tile<2, 2, 2, BF16OUT>(g)
                   : c[1] <= c[0]               ? run_tile<1, 2, 4, BF16OUT>(g)
                                                : run_tile<1, 1, 4, BF16OUT>(g)))
    return true;
  return run_tile<4, 4, 2, BF16OUT>(g);   // also where the launch cannot hold the smaller tiles
}

}  // namespace

bool launch_gemm_mxfp8_mxfp4(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int64_t m,
                             int64_t n, int64_t k, bool bf16_out, void* c, hipStream_t st) {
  const Gemm8 g{ac, as, bc, bs, (int)m, (int)n, (int)k, c, st};
  return bf16_out ? run<true>(g) : run<false>(g);
}

}  // namespace fp4q
