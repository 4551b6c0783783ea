// int8 GEMM (W8A8: one scale per activation row and one per weight row) and its
// grouped form over the experts of a mixture.
//
//   C[m, n] = bf16( fp32( sum_k A[m,k] W[n,k] ) * as[m] * ws[n] )
//
// The sum is exact: int32 holds K products of two 8-bit codes up to K = 131071.
// So K may be cut anywhere (waves, groups, workgroups) without a change in the
// result.  The weight is laid out in 16-row x 64-K fragment blocks of 1 KiB, rows
// and K padded with zeros; activation bytes past K meet those zeros, so they may
// be any valid bytes of the row.
//
// LDS-tiled kernel (k_w8a8_tile), fed through direct-to-LDS loads.
#include "grouped.h"

namespace {

struct W8A8Args {
  const uint8_t* a;      // int8 codes [rows, K], lda bytes apart
  const float* as;       // [rows]
  uint32_t lda;
  const uint8_t* w;      // pre-laid-out weight(s)
  const float* wsc;      // [N], grouped: [E, N]
  size_t w_stride;       // grouped: bytes from one expert's weight to the next
  uint16_t* c;
  int64_t ldc;
  int M, N, K, KS;       // dense: rows; grouped: slots.  KS = ceil(K / 64)
  const int* offsets;    // grouped: [E + 1]
  const int* rows;       // grouped: source row of each slot, or null
  int E, Ma;             // grouped: experts, rows of a
};

// Source row of tile row i (slot r0 + i).
BS_INLINE int src_row(const W8A8Args& p, int slot) {
  const int r = p.rows != nullptr ? p.rows[slot] : slot;
  return min(max(r, 0), p.Ma - 1);
}

BS_INLINE float scaled(int acc, float sa, float sw) { return static_cast<float>(acc) * sa * sw; }

// ========================================================= many rows: LDS tiles
// A workgroup computes a BM x BN tile with WM x WN waves, each (BM/WM) x
// (BN/WN) as 32x32 sub-tiles; first MFMA operand the weight (rows = n), second
// the activation, so a lane holds four consecutive n of one m.
//
// K advances in 64-wide steps.  A step's activation codes (BM x 64 B, chunks
// swizzled by swz4) and weight codes (BN/16 fragment blocks of 1 KiB, as they
// are) go global -> LDS by direct loads into one of STAGES buffers, STAGES - 1
// steps ahead.  The steps of a turn round the stages are unrolled, so the stage
// is a constant of the code.
//
// KG > 1: that many groups of WM x WN waves share the tile, each over every
// KG-th step with buffers of its own, and their partial sums are added through
// LDS.  TAIL: K is no multiple of 64.
template <int BM, int BN, int WM, int WN, int KG, int STAGES>
struct TileCfg {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;   // of a group
  static constexpr int kTM = BM / WM / 32, kTN = BN / WN / 32;
  static constexpr int kA = BM * 64, kB = BN * 64, kStage = kA + kB;
  static constexpr int kAIters = kA / (kThreads * 16), kBIters = kB / (kThreads * 16);
  static constexpr int kDma = kAIters + kBIters;
  static constexpr int kDmaFirst = (kDma + 1) / 2;      // of them, in the half step that frees the stage
  static_assert(kA % (kThreads * 16) == 0 && kB % (kThreads * 16) == 0, "");
  static constexpr int kGroup = STAGES * kStage;         // LDS of a group
  static constexpr int kRed = (KG - 1) * BM * BN * 4;    // the other groups' partial tiles
  static constexpr int kEpi = BM * BN * 2;               // the epilogue's tile
  static constexpr int kMain = std::max(KG * kGroup, std::max(kRed, kEpi));
  static constexpr int kScales = (BM + BN) * 4;          // behind it: as of the rows, ws of the columns
  static constexpr int kScalePieces = (BM + BN) / 64, kScaleIters = (kScalePieces + kWaves * KG - 1) / (kWaves * KG);
  static constexpr int kLds = kMain + kScales;
};

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int OCC, bool GROUPED, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN * KG, OCC) void k_w8a8_tile(W8A8Args p, int group_m) {
  using C = TileCfg<BM, BN, WM, WN, KG, STAGES>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x;
  const int wg_wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int kg = wg_wave / C::kWaves, wave = wg_wave % C::kWaves;
  const int wm = wave / WN, wn = wave % WN;
  const int N = p.N, KS = p.KS, NT = (N + 15) >> 4;
  const int n_tiles = (N + BN - 1) / BN;
  // this group's steps: KG * i + kg for i < n_steps
  const int n_steps = (KS - kg + KG - 1) / KG, n_turns = (KS + KG - 1) / KG;

  int m0, nrows, nt;
  const uint8_t* w = p.w;
  const float* wsc = p.wsc;
  if constexpr (GROUPED) {
    int e, r1;
    const uint32_t id = BM >= 128 ? xcd_runs(blockIdx.x, gridDim.x, n_tiles) : blockIdx.x;
    nt = id % n_tiles;
    if (!find_tile<BM>(p.offsets, p.E, p.M, id / n_tiles, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
    wsc += static_cast<size_t>(e) * N;
  } else {
    int mt;
    xcd_tile(blockIdx.x, (p.M + BM - 1) / BM, n_tiles, group_m, mt, nt);
    m0 = mt * BM;
    nrows = min(BM, p.M - m0);
  }
  const int n0 = nt * BN, nt0 = n0 >> 4;
  uint8_t* const glds = lds + kg * C::kGroup;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(glds));

  // 32-bit source offsets of the loads from the tile's base (rows past the
  // tile's last and columns past N re-read valid ones; their results are not
  // stored).  Chunks past K re-read the row's last one (TAIL).
  const uint8_t* const a = GROUPED ? p.a : p.a + static_cast<size_t>(m0) * p.lda;
  w += static_cast<size_t>(nt0) * KS * 1024;
  uint32_t aoff[C::kAIters], aend[C::kAIters], boff[C::kBIters];
#pragma unroll
  for (int i = 0; i < C::kAIters; ++i) {
    const int q = (i * C::kWaves + wave) * 64 + l;
    const int row = q >> 2;
    int src = min(row, nrows - 1);
    if constexpr (GROUPED) src = src_row(p, m0 + src);
    aoff[i] = static_cast<uint32_t>(src) * p.lda;
    aend[i] = aoff[i] + static_cast<uint32_t>(p.K - 16);
    aoff[i] += static_cast<uint32_t>(16 * swz4(row, q & 3));
  }
#pragma unroll
  for (int i = 0; i < C::kBIters; ++i)
    boff[i] = static_cast<uint32_t>(min(nt0 + i * C::kWaves + wave, NT - 1) - nt0) * static_cast<uint32_t>(KS) * 1024u +
              static_cast<uint32_t>(l * 16);
  // the i-th load of step ks into stage st
  auto dma_one = [&](int i, int ks, int st) {
    const uint32_t base = lds0 + st * C::kStage;
    if (i < C::kAIters) {
      const uint32_t dst = base + (i * C::kWaves + wave) * 1024;
      if constexpr (TAIL) dma16(dst, a, min(aoff[i] + static_cast<uint32_t>(ks) * 64u, aend[i]));
      else dma16(dst, a + static_cast<size_t>(ks) * 64, aoff[i]);
    } else {
      dma16(base + C::kA + ((i - C::kAIters) * C::kWaves + wave) * 1024, w + static_cast<size_t>(ks) * 1024,
            boff[i - C::kAIters]);
    }
  };

  v16i acc[C::kTN][C::kTM];
#pragma unroll
  for (int i = 0; i < C::kTN; ++i)
#pragma unroll
    for (int j = 0; j < C::kTM; ++j) acc[i][j] = v16i{};

  // fragment places within a stage.  Weight sub-tile i, half hh: lane l takes
  // column l%32, K block 2hh + l/32; activation sub-tile j: row l%32, the same.
  const int nlane = (l & 15) + 16 * (l >> 5);         // within a 1 KiB block, half 0
  const int bbase = C::kA + (wn * (BN / WN / 16) + ((l >> 4) & 1)) * 1024 + nlane * 16;
  int arow[C::kTM], abase[2];
#pragma unroll
  for (int j = 0; j < C::kTM; ++j) arow[j] = wm * (BM / WM) + 32 * j + (l & 31);
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) abase[hh] = arow[0] * 64 + 16 * swz4(arow[0], 2 * hh + (l >> 5));

  struct Frag {
    v4i b[C::kTN], a[C::kTM];
  };
  constexpr int kPieces = C::kTN + C::kTM;
  // LDS read piece i of half hh of stage st: weight 0, the activations, the other weights
  auto piece = [&](int st, int hh, Frag& f, int i) {
    const uint8_t* base = glds + st * C::kStage;
    if (i == 0 || i > C::kTM) {
      const int t = i == 0 ? 0 : i - C::kTM;
      f.b[t] = *reinterpret_cast<const v4i*>(base + bbase + t * 2048 + hh * 512);
    } else {
      f.a[i - 1] = *reinterpret_cast<const v4i*>(base + abase[hh] + (i - 1) * 2048);
    }
  };
  // MFMAs of half HH of the step in stage U.  Between them: the LDS reads of the
  // next half (rf) and half of a step's loads (HH 0: the rest of step s + STAGES
  // - 1's; HH 1: the first of step s + STAGES's, whose stage has just become free).
  auto half = [&](auto uu, auto hh, const Frag& f, Frag& rf, int dks) {
    constexpr int U = decltype(uu)::value, HH = decltype(hh)::value;
    constexpr int kRead = HH == 0 ? U : (U + 1) % STAGES;
    constexpr int kN = C::kTN * C::kTM;
    constexpr int d0 = HH ? 0 : C::kDmaFirst, d1 = HH ? C::kDmaFirst : C::kDma;
    constexpr int kFill = HH ? U : (U + STAGES - 1) % STAGES;
#pragma unroll
    for (int n = 0; n < kN || n < kPieces; ++n) {
      if (n < kN) {
        const int i = n / C::kTM, j = n % C::kTM;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[i], f.a[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (n < kPieces) piece(kRead, 1 - HH, rf, n);
      // the loads, spread evenly over the half's MFMAs
#pragma unroll
      for (int d = d0; d < d1; ++d)
        if ((d - d0) * kN / (d1 - d0) == n) dma_one(d, dks, kFill);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s: first half; this wave's loads of step s+1 have landed and its LDS
  // reads are done; barrier (s+1 published, the stage of s free); second half,
  // which reads s+1's first fragments.  So a stage is filled again right behind
  // its last reads and waited for only where it is read, STAGES - 1 steps later.
  // Steps past the end re-load the last one (never used, or the same bytes).
  Frag f0, f1;
  auto step_of = [&](int ls) { return min(KG * min(ls, n_steps - 1) + kg, KS - 1); };
  {
    // scales: rows, then columns, 64 a load, straight to their place in LDS
    const uint32_t sbase = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + C::kMain;
#pragma unroll
    for (int i = 0; i < C::kScaleIters; ++i) {
      const int pc = (i * C::kWaves * KG + wg_wave) % C::kScalePieces;
      if (pc < BM / 64) {
        int src = m0 + min(pc * 64 + l, nrows - 1);
        if constexpr (GROUPED) src = src_row(p, src);
        dma4(sbase + pc * 256, p.as, static_cast<uint32_t>(src) * 4u);
      } else {
        dma4(sbase + pc * 256, wsc, static_cast<uint32_t>(min(n0 + (pc - BM / 64) * 64 + l, N - 1)) * 4u);
      }
    }
  }
  if (KG == 1 || n_steps > 0) {
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
#pragma unroll
      for (int i = 0; i < C::kDma; ++i) dma_one(i, step_of(s), s);
    }
#pragma unroll
    for (int i = 0; i < C::kDmaFirst; ++i) dma_one(i, step_of(STAGES - 1), STAGES - 1);
    wait_vm<(STAGES - 2) * C::kDma + C::kDmaFirst>();   // the scales and step 0 have landed
  } else {
    wait_vm<0>();
  }
  __syncthreads();
  if (KG == 1 || n_steps > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) piece(0, 0, f0, i);
  }
  // the group's ls-th step, in stage U (live: it exists)
  auto step = [&](auto uu, int ls, bool live) {
    if (KG == 1 || live) {
      half(uu, Int<0>{}, f0, f1, step_of(ls + STAGES - 1));
      wait_vm<(STAGES - 2) * C::kDma>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if (KG > 1 && !live) return;
    half(uu, Int<1>{}, f1, f0, step_of(ls + STAGES));
  };
  // (with one group, steps past the end are skipped; several groups meet at
  // every barrier, so those run it empty)
  for (int ls = 0; ls < n_turns; ls += STAGES) {
    step(Int<0>{}, ls, ls < n_steps);
    if (ls + 1 < n_turns) step(Int<1>{}, ls + 1, ls + 1 < n_steps);
    if (ls + 2 < n_turns) step(Int<2>{}, ls + 2, ls + 2 < n_steps);
    if constexpr (STAGES > 3)
      if (ls + 3 < n_turns) step(Int<3>{}, ls + 3, ls + 3 < n_steps);
  }
  wait_vm<0>();

  // the groups' partial sums, added by group 0.  Fragment order: element r of
  // lane l of sub-tile (i, j) at quarter r/4, 16 bytes a lane.
  if constexpr (KG > 1) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr int kWaveBytes = C::kTN * C::kTM * 4096;
    if (kg > 0) {
      uint8_t* dst = lds + ((kg - 1) * C::kWaves + wave) * kWaveBytes + l * 16;
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *reinterpret_cast<v4i*>(dst + (i * C::kTM + j) * 4096 + r * 1024) =
                v4i{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int g = 1; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < C::kTN; ++i)
#pragma unroll
          for (int j = 0; j < C::kTM; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const v4i v = *reinterpret_cast<const v4i*>(
                  lds + ((g - 1) * C::kWaves + wave) * kWaveBytes + l * 16 + (i * C::kTM + j) * 4096 + r * 1024);
#pragma unroll
              for (int u = 0; u < 4; ++u) acc[i][j][4 * r + u] += v[u];
            }
    }
  }

  // Epilogue: the tile through LDS as bf16, so that a row leaves as whole
  // 16-byte pieces side by side.  A lane's four columns are half a piece; piece
  // q of a row sits at slot q ^ (row % pieces).
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __syncthreads();       // the stages are done with
  const float* s_as = reinterpret_cast<const float*>(lds + C::kMain);
  const float* s_ws = s_as + BM;
  constexpr int kLanes = BN / 8, kRows = C::kThreads * KG / kLanes;   // pieces of a row, rows at once
  if (kg == 0) {         // (the other groups have handed their sums over)
#pragma unroll
    for (int i = 0; i < C::kTN; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int col = wn * (BN / WN) + 32 * i + 8 * r + 4 * (l >> 5);
        const float4 sw = *reinterpret_cast<const float4*>(s_ws + col);
#pragma unroll
        for (int j = 0; j < C::kTM; ++j) {
          const int row = arow[j];
          const float sa = s_as[row];
          const v16i& av = acc[i][j];
          *reinterpret_cast<uint2*>(lds + row * (BN * 2) + (((col >> 3) ^ (row % kLanes)) << 4) + 8 * (l >> 5)) =
              uint2{bf16x2_rne(scaled(av[4 * r], sa, sw.x), scaled(av[4 * r + 1], sa, sw.y)),
                    bf16x2_rne(scaled(av[4 * r + 2], sa, sw.z), scaled(av[4 * r + 3], sa, sw.w))};
        }
      }
  }
  __syncthreads();
  // rows that are 16-byte aligned leave in pieces; else, and in a last piece that
  // N cuts, value by value
  const bool wide = p.ldc % 8 == 0 && reinterpret_cast<uintptr_t>(p.c) % 16 == 0;
  const int q = tid % kLanes, cols = min(8, N - n0 - 8 * q);
  if (cols <= 0) return;
#pragma unroll 4
  for (int r = tid / kLanes; r < nrows; r += kRows) {
    const uint4 o = *reinterpret_cast<const uint4*>(lds + r * (BN * 2) + ((q ^ (r % kLanes)) << 4));
    uint16_t* dst = p.c + (m0 + r) * p.ldc + n0 + 8 * q;
    if (wide && cols == 8) {
      st_stream16(reinterpret_cast<uint4*>(dst), o);
    } else {
      const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (u < cols) dst[u] = static_cast<uint16_t>(v[u >> 1] >> (16 * (u & 1)));
    }
  }
}

// ---------------------------------------------------------------- host side
template <int BM, int BN, int WM, int WN, int KG, int STAGES, int OCC, bool GROUPED>
int launch_tile(const W8A8Args& p, int64_t wgs, hipStream_t st) {
  if (wgs > 0x7FFFFFFF) return BS_ERR_SHAPE;
  const dim3 grid(static_cast<uint32_t>(wgs)), block(64 * WM * WN * KG);
  if (p.K % 64 == 0) k_w8a8_tile<BM, BN, WM, WN, KG, STAGES, OCC, GROUPED, false><<<grid, block, 0, st>>>(p, 4);
  else k_w8a8_tile<BM, BN, WM, WN, KG, STAGES, OCC, GROUPED, true><<<grid, block, 0, st>>>(p, 4);
  return bs_launch_status();
}

int64_t tiles(int M, int N, int bm, int bn) {
  return static_cast<int64_t>((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

}  // namespace

size_t bs_w8a8_workspace(int M, int N, int K) { return 0; }

int bs_launch_w8a8(const uint8_t* a, int64_t lda, const float* as, const uint8_t* w, const float* wsc, uint16_t* c,
                   int64_t ldc, int M, int N, int K, void* ws, hipStream_t st) {
  W8A8Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.w = w;
  p.wsc = wsc;
  p.c = c;
  p.ldc = ldc;
  p.M = M;
  p.N = N;
  p.K = K;
  p.KS = (K + 63) / 64;
  if (tiles(M, N, 128, 128) >= 256) return launch_tile<128, 128, 2, 2, 1, 4, 2, false>(p, tiles(M, N, 128, 128), st);
  return launch_tile<64, 64, 2, 2, 1, 4, 4, false>(p, tiles(M, N, 64, 64), st);
}

int bs_launch_w8a8_grouped(const uint8_t* a, int64_t lda, const float* as, const int* offsets, const int* rows,
                           const uint8_t* w, size_t w_stride, const float* wsc, uint16_t* c, int64_t ldc, int S,
                           int Ma, int E, int N, int K, hipStream_t st) {
  W8A8Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.w = w;
  p.wsc = wsc;
  p.w_stride = w_stride;
  p.c = c;
  p.ldc = ldc;
  p.M = S;
  p.N = N;
  p.K = K;
  p.KS = (K + 63) / 64;
  p.offsets = offsets;
  p.rows = rows;
  p.E = E;
  p.Ma = Ma;
  if (S / E > 64)
    return launch_tile<128, 128, 2, 2, 1, 4, 2, true>(
        p, static_cast<int64_t>(tile_bound(S, E, 128)) * ((N + 127) / 128), st);
  return launch_tile<64, 64, 2, 2, 1, 4, 4, true>(p, static_cast<int64_t>(tile_bound(S, E, 64)) * ((N + 63) / 64), st);
}
