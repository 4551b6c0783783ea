// MXFP4 W4A4 GEMM (activations and weights both e2m1 with one e8m0 scale per
// 32 along K) and its grouped form over the experts of a mixture.
//
//   C[m, n] = bf16( sum_b 2^(EA[m,b]-127) 2^(EW[n,b]-127) sum_{k in b} A[m,k] W[n,k] )
//
// gfx950's scaled MFMA takes both operands and both block scales as they are
// stored and accumulates in fp32; fp4 x fp4 issues at twice the rate of the
// mixed fp8 x fp4 form (about 9.7 PFLOP/s with registers only).  The weight
// is the pre-laid-out MXFP4 weight of the W4A8 GEMM.
//
// Two kernels.  Few rows: a weight stream (k_w4a4_stream), bound by HBM (M = 8
// N = 17408 K = 5120: 11.1 to 11.7 us with the weight from HBM, 4.1 to 4.3 TB/s,
// where a large copy runs at 5.2; 9.9 from the last-level cache).  Many rows:
// LDS-tiled (k_w4a4_tile), fed through direct-to-LDS loads and bound by the matrix
// cores' power: M = 8192 N = 10240 K = 5120 takes 196 to 213 us by card (4.0 to
// 4.4 PFLOP/s), 154 us when every code is zero, and 178 us with all loads and LDS
// reads taken out of the loop.  Both have a grouped form: the slots of the sorted
// (token, expert) pairs are cut into row tiles expert by expert, and every
// workgroup finds its tile from the expert offsets on the device, so the host
// never waits for them; the activation rows are read through the sorted order
// (row gather in the loads), never copied.
#include <algorithm>
#include <cmath>

#include "grouped.h"

namespace {

struct W4A4Args {
  const uint8_t* a;      // e2m1 codes [rows, K/2], lda bytes apart
  const uint8_t* as;     // e8m0 [rows, K/32], lds bytes apart
  uint32_t lda, lds;
  const uint8_t* w;      // pre-laid-out weight(s): codes
  const uint8_t* wsc;    // and e8m0 section
  size_t w_stride;       // grouped: bytes from one expert's weight to the next
  uint16_t* c;
  int64_t ldc;
  int M, N, KS;          // dense: rows; grouped: slots.  KS = K / 128
  const int* offsets;    // grouped: [E + 1]
  const int* rows;       // grouped: source row of each slot, or null
  int E, Ma;             // grouped: experts, rows of a
  int rs;                // stream: activation rows staged per workgroup
  int iters;             // stream: K runs per workgroup
  float* slab;
  int* counters;
};

// Source row of tile row i (slot r0 + i).
BS_INLINE int src_row(const W4A4Args& p, int slot) {
  const int r = p.rows != nullptr ? p.rows[slot] : slot;
  return min(max(r, 0), p.Ma - 1);
}

// ============================================================ few rows: stream
// grid (column groups, row tiles, K splits): workgroup (x, y, z) computes
// n-tiles [x*TW*T, (x+1)*TW*T) of 16 columns for the up to 16*MB rows of row
// tile y (dense: all rows) over its run of `iters * KW * R` K steps.  Wave (tw, kw) owns T tiles over R
// steps of each KW*R; the KW partial sums of a tile are added through LDS in
// kw order, K splits through the workspace.  The activation slice (KW*R steps
// x rs rows x 64 B of codes and one scale dword per row and step) is copied to
// LDS by direct loads, shared by the TW*T tiles; the weights go straight to
// registers, all of a wave's loads at once.
template <int MB, int TW, int KW, int T, int R, bool GROUPED>
__global__ __launch_bounds__(TW * KW * 64) void k_w4a4_stream(W4A4Args p) {
  static_assert(TW * KW > 4, "the 16x16x128 scaled MFMA accumulates in ordinary registers (> 4 waves)");
  static_assert(R % 4 == 0, "one e8m0 dword per lane covers four steps");
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int last;
  constexpr int kSteps = KW * R;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tw = wave % TW, kw = wave / TW;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int KS = p.KS, RS = p.rs, KQ = (KS + 3) >> 2;
  const int ntiles = p.N >> 4;
  const int tile0 = (blockIdx.x * TW + tw) * T;

  int m0, nrows;
  const uint8_t *w = p.w, *wscb = p.wsc;
  if constexpr (GROUPED) {
    int e, r1;
    if (!find_tile<16 * MB>(p.offsets, p.E, p.M, blockIdx.y, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
    wscb += static_cast<size_t>(e) * p.w_stride;
  } else {
    m0 = 0;
    nrows = RS;
  }
  const uint32_t* wsc = reinterpret_cast<const uint32_t*>(wscb);

  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
  const int a_instr = (kSteps * RS * 4 + 63) >> 6, s_instr = (kSteps * RS + 63) >> 6;
  const uint32_t* s_sc = reinterpret_cast<const uint32_t*>(lds + a_instr * 1024);
  float* s_red = reinterpret_cast<float*>(lds);

  v4f acc[T][MB];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[t][mb] = v4f{0, 0, 0, 0};

  const int iters = GROUPED ? p.iters : 1;   // (the loop costs the dense form register copies)
  for (int it = 0; it < iters; ++it) {
    const int wg_k0 = (blockIdx.z * iters + it) * kSteps;
    if (GROUPED && wg_k0 >= KS) break;
    const int wg_steps = min(kSteps, KS - wg_k0);
    const int ks0 = wg_k0 + kw * R;
    const int klast = min(ks0 + R, KS) - 1;  // below ks0 for an idle wave
    const int nsteps = klast - ks0 + 1;      // <= 0 for an idle wave
    if (GROUPED && it) __syncthreads();      // every wave is done with the slice
    // chunk c of row i of step r sits at position (r*RS + i)*4 + swz4(i, c),
    // its scale dword at position r*RS + i; positions past the slice re-read
    // valid bytes that are never used
    for (int k = wave; k < a_instr + s_instr; k += TW * KW) {
      const bool codes = k < a_instr;
      const int q = (codes ? k : k - a_instr) * 64 + l;
      const int ri = codes ? q >> 2 : q;
      const int r = min(ri / RS, wg_steps - 1);
      const int ii = ri % RS;
      int row = m0 + min(ii, nrows - 1);
      if constexpr (GROUPED) row = src_row(p, row);
      if (codes)
        dma16(lds0 + k * 1024, p.a,
              static_cast<uint32_t>(row) * p.lda + static_cast<uint32_t>((wg_k0 + r) * 64 + swz4(ii, q & 3) * 16));
      else
        dma4(lds0 + a_instr * 1024 + (k - a_instr) * 256, p.as,
             static_cast<uint32_t>(row) * p.lds + static_cast<uint32_t>((wg_k0 + r) * 4));
    }
    v4i wf[T][R];
    uint32_t sd[T][R / 4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const size_t tile = static_cast<size_t>(min(tile0 + t, ntiles - 1));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const size_t ks = max(min(ks0 + r, klast), 0);
        const uint4 x = ld_stream16(reinterpret_cast<const uint4*>(w + (tile * KS + ks) * 1024 + l * 16));
        wf[t][r] = v4i{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
      }
#pragma unroll
      for (int qd = 0; qd < R / 4; ++qd)
        sd[t][qd] = wsc[(tile * KQ + min((ks0 >> 2) + qd, max(klast, 0) >> 2)) * 64 + l];
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<T * R + T * (R / 4)>();  // this wave's activation loads have landed
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= nsteps) break;
      v8i af[MB];
      int as[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int rc = min(16 * mb + (l & 15), RS - 1);
        const int at = (kw * R + r) * RS + rc;
        const uint4 x = *reinterpret_cast<const uint4*>(lds + at * 64 + (swz4(rc, g) << 4));
        af[mb] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        as[mb] = static_cast<int>(s_sc[at] >> (8 * g));
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int sc = static_cast<int>(sd[t][r >> 2] >> (8 * (r & 3)));
        const v8i wm = v8i{wf[t][r][0], wf[t][r][1], wf[t][r][2], wf[t][r][3], 0, 0, 0, 0};
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          acc[t][mb] =
              __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wm, af[mb], acc[t][mb], 4, 4, 0, sc, 0, as[mb]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  if constexpr (KW > 1) {   // the KW partials of a tile, in kw order
    constexpr int kPer = T * MB * 4;
    __syncthreads();
    if (kw > 0) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s_red[(((kw - 1) * TW + tw) * kPer + (t * MB + mb) * 4 + j) * 64 + l] = acc[t][mb][j];
    }
    __syncthreads();
    if (kw == 0)
#pragma unroll
      for (int u = 1; u < KW; ++u)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[t][mb][j] += s_red[(((u - 1) * TW + tw) * kPer + (t * MB + mb) * 4 + j) * 64 + l];
  }
  auto store = [&](int t, int mb, v4f v) {
    const int i = 16 * mb + (l & 15), n = (tile0 + t) * 16 + 4 * g;
    if (i < nrows && tile0 + t < ntiles)
      *reinterpret_cast<uint2*>(p.c + (m0 + i) * p.ldc + n) =
          uint2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  };
  const bool owner = kw == 0;
  const int S = gridDim.z;
  if (GROUPED || S == 1) {
    if (owner)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) store(t, mb, acc[t][mb]);
    return;
  }
  // K splits: fp32 partials in fragment order, device-scope, added by the last
  // workgroup of the tile in split order; it leaves its counter at zero.
  const int tg = blockIdx.y * gridDim.x + blockIdx.x;
  auto frag = [&](int sp, int t, int mb) {
    const size_t f =
        ((((static_cast<size_t>(sp) * gridDim.y * gridDim.x) + tg) * TW + tw) * T + t) * MB + mb;
    return p.slab + f * 256 + l;
  };
  if (owner)
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float* dst = frag(blockIdx.z, t, mb);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __hip_atomic_store(dst + j * 64, acc[t][mb][j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(&p.counters[tg], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == S - 1;
  __syncthreads();
  if (!last || !owner) return;
  constexpr int kNV = T * MB * 4;
  constexpr int kU = kNV >= 32 ? 2 : (kNV >= 16 ? 4 : 8);
  float sum[kNV];
  sum_partials<kNV, 64, kU>(sum, frag(0, 0, 0), static_cast<size_t>(gridDim.y) * gridDim.x * (TW * T * MB * 256), S);
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int v = (t * MB + mb) * 4;
      store(t, mb, v4f{sum[v], sum[v + 1], sum[v + 2], sum[v + 3]});
    }
  if (threadIdx.x == 0) __hip_atomic_store(&p.counters[tg], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ========================================================= many rows: LDS tiles
// A workgroup computes a BM x BN tile with WM x WN waves, each (BM/WM) x
// (BN/WN) as 32x32 sub-tiles; first MFMA operand the weight (rows = n), second
// the activation, so a lane holds four consecutive n of one m.
//
// K advances in 128-wide steps, four to a window.  A step's activation codes
// (BM x 64 B, chunks swizzled by swz4) and weight codes (BN/16 fragment blocks
// of 1 KiB, as they are) go global -> LDS by direct loads into one of STAGES
// buffers, STAGES - 1 steps ahead; the scales of a window (16 B per activation
// row, 256 B per 16 columns) into a window buffer during the window before.
// The steps of a window are unrolled, so the stage, the scale dword and its
// byte are constants of the code, and a window's scales are read from LDS once,
// under the last MFMAs of the window before.  (Reading and shifting a scale
// dword at every half step stalled on each: M = 8192 N = 10240 K = 5120 237 us
// instead of 201.)
//
// KG > 1: that many groups of WM x WN waves share the tile, each over every
// KG-th window with buffers of its own, and their partial sums are added
// through LDS in group order.  A step is a chain (barrier, LDS reads, MFMAs)
// that one small wave tile per SIMD cannot hide; a second chain on the same
// SIMD does, where splitting K over workgroups would send every partial tile
// through memory (M = 65 N = K = 5120: 9.3 us, 128 x 128 tiles with K split over
// workgroups 12.9).
//
// AS16: the activation scale rows are 16-byte aligned and K is a multiple of
// 512, so a row's window is one 16-byte load (rows of 16 B); otherwise it is
// four 4-byte loads (planes of BM dwords).  One 4-byte load per row and step
// touched as many cache lines per step as the codes themselves.
template <int BM, int BN, int WM, int WN, int KG, int STAGES, bool AS16>
struct TileCfg {
  static_assert(STAGES == 3 || STAGES == 4, "the waits below");
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;   // of a group
  static constexpr int kTM = BM / WM / 32, kTN = BN / WN / 32;
  static constexpr int kA = BM * 64, kB = BN * 64, kStage = kA + kB;
  static constexpr int kSB = BN * 16, kSA = BM * 16, kWin = kSB + kSA;
  static constexpr int kWin0 = STAGES * kStage;        // the window buffer follows the stages
  static constexpr int kAIters = kA / (kThreads * 16), kBIters = kB / (kThreads * 16);
  static constexpr int kSBPieces = kSB / 1024, kSAPieces = AS16 ? kSA / 1024 : kSA / 256;
  // loads per stage and per window, the same for every wave: a wave past a
  // section's last piece repeats an earlier one (same bytes, same place)
  static constexpr int kSBIters = (kSBPieces + kWaves - 1) / kWaves, kSAIters = (kSAPieces + kWaves - 1) / kWaves;
  static constexpr int kDma = kAIters + kBIters, kWinDma = kSBIters + kSAIters;
  static constexpr int kDmaFirst = (kDma + 1) / 2;      // of them, in the half step that frees the stage
  static_assert(kA % (kThreads * 16) == 0 && kB % (kThreads * 16) == 0 && kSB % 1024 == 0 && kSA % 1024 == 0, "");
  static constexpr int kGroup = kWin0 + kWin;            // LDS of a group
  static constexpr int kRed = (KG - 1) * BM * BN * 4;    // the other groups' partial tiles
  static constexpr int kEpi = BM * BN * 2;               // the epilogue's tile
  static constexpr int kLds = std::max(KG * kGroup, std::max(kRed, kEpi));
};

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int OCC, bool GROUPED, bool AS16>
__global__ __launch_bounds__(64 * WM * WN * KG, OCC) void k_w4a4_tile(W4A4Args p, int group_m) {
  using C = TileCfg<BM, BN, WM, WN, KG, STAGES, AS16>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x;
  const int wg_wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int kg = wg_wave / C::kWaves, wave = wg_wave % C::kWaves;
  const int wm = wave / WN, wn = wave % WN;
  const int N = p.N, KS = p.KS, NT = N >> 4, KQ = (KS + 3) >> 2;
  const int n_tiles = (N + BN - 1) / BN;
  // this group's windows: KG * i + kg for i < n_win
  const int n_win = (KQ - kg + KG - 1) / KG, n_turns = (KQ + KG - 1) / KG;
  auto win_of = [&](int i) { return KG * min(i, n_win - 1) + kg; };

  int m0, nrows, nt;
  const uint8_t *w = p.w, *wsc = p.wsc;
  if constexpr (GROUPED) {
    int e, r1;
    const uint32_t id = BM >= 128 ? xcd_runs(blockIdx.x, gridDim.x, n_tiles) : blockIdx.x;
    nt = id % n_tiles;
    if (!find_tile<BM>(p.offsets, p.E, p.M, id / n_tiles, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
    wsc += static_cast<size_t>(e) * p.w_stride;
  } else {
    int mt;
    xcd_tile(blockIdx.x, (p.M + BM - 1) / BM, n_tiles, group_m, mt, nt);
    m0 = mt * BM;
    nrows = min(BM, p.M - m0);
  }
  const int n0 = nt * BN, nt0 = n0 >> 4;
  uint8_t* const glds = lds + kg * C::kGroup;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(glds));

  // 32-bit source offsets of the loads (rows past the tile's last and columns
  // past N re-read valid ones; their results are not stored)
  uint32_t aoff[C::kAIters], boff_g[C::kBIters], sboff[C::kSBIters], saoff[C::kSAIters];
#pragma unroll
  for (int i = 0; i < C::kAIters; ++i) {
    const int q = (i * C::kWaves + wave) * 64 + l;
    const int row = q >> 2;
    int src = m0 + min(row, nrows - 1);
    if constexpr (GROUPED) src = src_row(p, src);
    aoff[i] = static_cast<uint32_t>(src) * p.lda + static_cast<uint32_t>(16 * swz4(row, q & 3));
  }
#pragma unroll
  for (int i = 0; i < C::kBIters; ++i)
    boff_g[i] = static_cast<uint32_t>(min(nt0 + i * C::kWaves + wave, NT - 1)) * static_cast<uint32_t>(KS) * 1024u +
                static_cast<uint32_t>(l * 16);
#pragma unroll
  for (int i = 0; i < C::kSBIters; ++i) {
    const int q = ((i * C::kWaves + wave) % C::kSBPieces) * 64 + l;
    sboff[i] = static_cast<uint32_t>(min(nt0 + (q >> 4), NT - 1)) * static_cast<uint32_t>(KQ) * 256u +
               static_cast<uint32_t>((q & 15) * 16);
  }
  // AS16: piece = 64 rows; else piece = (dword j, 64 rows), j outermost
#pragma unroll
  for (int i = 0; i < C::kSAIters; ++i) {
    const int pc = (i * C::kWaves + wave) % C::kSAPieces;
    int src = m0 + min((AS16 ? pc : pc % (BM / 64)) * 64 + l, nrows - 1);
    if constexpr (GROUPED) src = src_row(p, src);
    saoff[i] = static_cast<uint32_t>(src) * p.lds;
  }
  // the i-th load of step ks into stage st
  auto dma_one = [&](int i, int ks, int st) {
    const uint32_t base = lds0 + st * C::kStage;
    if (i < C::kAIters)
      dma16(base + (i * C::kWaves + wave) * 1024, p.a + static_cast<size_t>(ks) * 64, aoff[i]);
    else
      dma16(base + C::kA + ((i - C::kAIters) * C::kWaves + wave) * 1024, w + static_cast<size_t>(ks) * 1024,
            boff_g[i - C::kAIters]);
  };
  // the i-th load of the scales of the group's wi-th window
  auto win_one = [&](int i, int wi) {
    const int win = win_of(wi);
    const uint32_t base = lds0 + C::kWin0;
    if (i < C::kSBIters) {
      dma16(base + ((i * C::kWaves + wave) % C::kSBPieces) * 1024, wsc + static_cast<size_t>(win) * 256, sboff[i]);
    } else {
      const int j = i - C::kSBIters, pc = (j * C::kWaves + wave) % C::kSAPieces;
      if constexpr (AS16)
        dma16(base + C::kSB + pc * 1024, p.as + static_cast<size_t>(win) * 16, saoff[j]);
      else
        dma4(base + C::kSB + pc * 256, p.as + static_cast<size_t>(min(4 * win + pc / (BM / 64), KS - 1)) * 4, saoff[j]);
    }
  };

  v16f acc[C::kTN][C::kTM];
#pragma unroll
  for (int i = 0; i < C::kTN; ++i)
#pragma unroll
    for (int j = 0; j < C::kTM; ++j) acc[i][j] = v16f{};

  // fragment places within a stage.  Weight sub-tile i, half hh: lane l takes
  // column l%32, K block 2hh + l/32; activation sub-tile j: row l%32, the same.
  const int nlane = (l & 15) + 16 * (l >> 5);         // within a 1 KiB block, half 0
  const int bbase = C::kA + (wn * (BN / WN / 16) + ((l >> 4) & 1)) * 1024 + nlane * 16;
  const int sbbase = (wn * (BN / WN / 16) + ((l >> 4) & 1)) * 256 + nlane * 4;
  int arow[C::kTM], abase[2];
#pragma unroll
  for (int j = 0; j < C::kTM; ++j) arow[j] = wm * (BM / WM) + 32 * j + (l & 31);
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) abase[hh] = arow[0] * 64 + 16 * swz4(arow[0], 2 * hh + (l >> 5));
  const int sh_a = 8 * (l >> 5);   // the lane's K block of a half is byte 2hh + l/32

  struct Frag {
    v4i b[C::kTN], a[C::kTM];
  };
  struct Scale {
    int b[C::kTN][2];   // byte j: step j of the window
    int a[C::kTM][4];   // dword j: step j; byte 2hh after the shift by sh_a
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
  auto read_scale = [&](Scale& s, int i) {
    const uint8_t* base = glds + C::kWin0;
    if (i < C::kTN) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) s.b[i][hh] = *reinterpret_cast<const int*>(base + sbbase + i * 512 + hh * 128);
    } else {
      const int t = i - C::kTN;
      if constexpr (AS16) {
        const v4i v = *reinterpret_cast<const v4i*>(base + C::kSB + arow[t] * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) s.a[t][j] = v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s.a[t][j] = *reinterpret_cast<const int*>(base + C::kSB + (j * BM + arow[t]) * 4);
      }
    }
  };
  // Place of a step in the unrolled turn: U is the step's index modulo
  // lcm(4, STAGES), J = U % 4 its step of the window, U % STAGES its stage.
  // MFMAs of half HH of a step s.  Between them: the LDS reads of the next half
  // (rf), half of a step's loads (HH 0: the rest of step s + STAGES - 1's; HH 1:
  // the first of step s + STAGES's, whose stage has just become free), and in the
  // step's second half the loads of window next_win's scales (J = 0; the buffer's
  // last reads were a step before) or their reads (J = 3).
  auto half = [&](auto uu, auto hh, const Frag& f, Frag& rf, const Scale& s, int dks, int next_win, Scale& ns) {
    constexpr int U = decltype(uu)::value, HH = decltype(hh)::value, J = U % 4;
    constexpr int kRead = HH == 0 ? U % STAGES : (U + 1) % STAGES;
    constexpr int kN = C::kTN * C::kTM;
    constexpr int d0 = HH ? 0 : C::kDmaFirst, d1 = HH ? C::kDmaFirst : C::kDma;
    constexpr int kFill = HH ? U % STAGES : (U + STAGES - 1) % STAGES;
#pragma unroll
    for (int n = 0; n < kN || n < kPieces; ++n) {
      if (n < kN) {
        const int i = n / C::kTM, j = n % C::kTM;
        const v8i bw = v8i{f.b[i][0], f.b[i][1], f.b[i][2], f.b[i][3], 0, 0, 0, 0};
        const v8i aw = v8i{f.a[j][0], f.a[j][1], f.a[j][2], f.a[j][3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bw, aw, acc[i][j], 4, 4, J, s.b[i][HH], 2 * HH,
                                                                    s.a[j][J]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (n < kPieces) piece(kRead, 1 - HH, rf, n);
      // the loads, spread evenly over the half's MFMAs
#pragma unroll
      for (int d = d0; d < d1; ++d)
        if ((d - d0) * kN / (d1 - d0) == n) dma_one(d, dks, kFill);
      if (J == 0 && HH == 1 && n == kN - 1)
#pragma unroll
        for (int d = 0; d < C::kWinDma; ++d) win_one(d, next_win);
      if (J == 3 && HH == 1) {
#pragma unroll
        for (int d = 0; d < kPieces; ++d)
          if (d * kN / kPieces == n) read_scale(ns, d);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s: first half; this wave's loads of step s+1 have landed and its LDS
  // reads are done; barrier (s+1 published, the stage of s free); second half,
  // which reads s+1's first fragments.  So a stage is filled again right behind
  // its last reads and waited for only where it is read, STAGES - 1 steps later
  // (with the barrier in front of both halves, half a step is lost at each end:
  // 64 experts N = 1024 K = 5120, 4000 rows 51 us, so 41).
  // Steps and windows past the end re-load the last one (never used, or the
  // same bytes).
  Frag f0, f1;
  Scale sc, ns;
  // the ls-th step of this group, in steps of K
  auto step_of = [&](int ls) { return min(4 * win_of(ls >> 2) + (ls & 3), KS - 1); };
  if (KG == 1 || n_win > 0) {
#pragma unroll
    for (int d = 0; d < C::kWinDma; ++d) win_one(d, 0);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
#pragma unroll
      for (int i = 0; i < C::kDma; ++i) dma_one(i, step_of(s), s);
    }
#pragma unroll
    for (int i = 0; i < C::kDmaFirst; ++i) dma_one(i, step_of(STAGES - 1), STAGES - 1);
  }
  wait_vm<(STAGES - 2) * C::kDma + C::kDmaFirst>();   // the first window and step 0 have landed
  __syncthreads();
  if (KG == 1 || n_win > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) piece(0, 0, f0, i);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) read_scale(ns, i);
  }
  // step J of the group's wi-th window (live: it exists)
  auto step = [&](auto uu, int wi, bool live) {
    constexpr int U = decltype(uu)::value, J = U % 4;
    if (KG == 1 || live) {
      if constexpr (J == 0) {
#pragma unroll
        for (int t = 0; t < C::kTM; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc.a[t][j] = static_cast<int>(static_cast<uint32_t>(ns.a[t][j]) >> sh_a);
#pragma unroll
        for (int t = 0; t < C::kTN; ++t)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) sc.b[t][hh] = ns.b[t][hh];
      }
      half(uu, Int<0>{}, f0, f1, sc, step_of(4 * wi + J + STAGES - 1), wi + 1, ns);
      // loads newer than step s+1's: STAGES - 2 steps, and the window's scale
      // loads (issued behind the first of step STAGES) in steps 1 .. STAGES - 2
      wait_vm<(STAGES - 2) * C::kDma + (J >= 1 && J <= STAGES - 2 ? C::kWinDma : 0)>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if (KG > 1 && !live) return;
    half(uu, Int<1>{}, f1, f0, sc, step_of(4 * wi + J + STAGES), wi + 1, ns);
  };
  // (with one group, steps past the end are skipped; several groups meet at
  // every barrier, so those run it empty)
  auto window = [&](auto ww, int wi) {
    constexpr int W = 4 * decltype(ww)::value;
    if (wi >= n_turns) return;
    const int k0 = 4 * (KG * wi + kg);
    const bool here = wi < n_win;
    step(Int<W>{}, wi, here);
    if (KG > 1 || k0 + 1 < KS) step(Int<W + 1>{}, wi, here && k0 + 1 < KS);
    if (KG > 1 || k0 + 2 < KS) step(Int<W + 2>{}, wi, here && k0 + 2 < KS);
    if (KG > 1 || k0 + 3 < KS) step(Int<W + 3>{}, wi, here && k0 + 3 < KS);
  };
  constexpr int kTurn = STAGES == 4 ? 1 : 3;   // windows until the stages come round
  for (int wi = 0; wi < n_turns; wi += kTurn) {
    window(Int<0>{}, wi);
    if constexpr (kTurn == 3) {
      window(Int<1>{}, wi + 1);
      window(Int<2>{}, wi + 2);
    }
  }
  wait_vm<0>();

  // the groups' partial sums, added by group 0 in group order.  Fragment order:
  // element r of lane l of sub-tile (i, j) at quarter r/4, 16 bytes a lane.
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
            *reinterpret_cast<float4*>(dst + (i * C::kTM + j) * 4096 + r * 1024) = make_float4(
                acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]);
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
              const float4 v = *reinterpret_cast<const float4*>(
                  lds + ((g - 1) * C::kWaves + wave) * kWaveBytes + l * 16 + (i * C::kTM + j) * 4096 + r * 1024);
              acc[i][j][4 * r] += v.x;
              acc[i][j][4 * r + 1] += v.y;
              acc[i][j][4 * r + 2] += v.z;
              acc[i][j][4 * r + 3] += v.w;
            }
    }
  }

  // Epilogue: the tile through LDS as bf16, so that a row leaves as whole
  // 16-byte pieces side by side.  A lane's four columns are half a piece; piece
  // q of a row sits at slot q ^ (row % pieces), which leaves two rows of a write's
  // 32 on a bank (their halves swapped on every other 16 rows would leave one, and
  // is 1 to 2% slower: the reads have to swap them back).
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __syncthreads();       // the stages are done with
  constexpr int kLanes = BN / 8, kRows = C::kThreads * KG / kLanes;   // pieces of a row, rows at once
  if (kg == 0) {         // (the other groups have handed their sums over)
#pragma unroll
    for (int j = 0; j < C::kTM; ++j) {
      const int row = arow[j];
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const v16f& av = acc[i][j];
          const int q = (wn * (BN / WN) + 32 * i) / 8 + r;
          *reinterpret_cast<uint2*>(lds + row * (BN * 2) + ((q ^ (row % kLanes)) << 4) + 8 * (l >> 5)) =
              uint2{bf16x2_rne(av[4 * r], av[4 * r + 1]), bf16x2_rne(av[4 * r + 2], av[4 * r + 3])};
        }
    }
  }
  __syncthreads();
  const int q = tid % kLanes;
  if (n0 + 8 * q >= N) return;   // N % 16 == 0: eight columns are wholly inside or outside
#pragma unroll 4
  for (int r = tid / kLanes; r < nrows; r += kRows) {
    const uint4 o = *reinterpret_cast<const uint4*>(lds + r * (BN * 2) + ((q ^ (r % kLanes)) << 4));
    uint16_t* dst = p.c + (m0 + r) * p.ldc + n0 + 8 * q;
    if (p.ldc % 8 == 0) {
      st_stream16(reinterpret_cast<uint4*>(dst), o);
    } else {
      st_stream8(reinterpret_cast<uint2*>(dst), o.x, o.y);
      st_stream8(reinterpret_cast<uint2*>(dst + 4), o.z, o.w);
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr size_t kMaxStreamLds = 160 * 1024 - 256;
constexpr int kMaxSplits = 65535;   // grid z

struct StreamCfg {
  int mb, tw, kw, t, r, rs, groups, mtiles, s, iters;
};
size_t stream_lds(const StreamCfg& d) {
  const size_t pos = static_cast<size_t>(d.kw) * d.r * d.rs;
  const size_t slice = (pos * 4 + 63) / 64 * 1024 + (pos + 63) / 64 * 256;
  const size_t red = static_cast<size_t>(d.kw - 1) * d.tw * d.t * d.mb * 4 * 64 * sizeof(float);
  return std::max(slice, red);
}

// Swept at 1 to 16 rows over K = 512 .. 17408, N = 512 .. 34816, weights pooled
// past the last-level cache: a workgroup covers all of a short K with no idle
// K-wave, a longer one in runs of 40 steps (24 from K = 12288 on with wide N).
// With M = 8: K = 1024 N = 17408 6.95 us with ten K-waves, 4.4 with two; K =
// 5120 N = 5120 5.8 -> 5.4; K = 5120 N = 17408 10.9, K = 17408 N = 5120 12.1.
StreamCfg dense_stream_cfg(int M, int N, int KS) {
  StreamCfg d{};
  d.mb = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
  d.rs = M;
  d.mtiles = 1;
  const int nt = N / 16;
  auto set = [&](int tw, int kw, int t, int r) { d.tw = tw; d.kw = kw; d.t = t; d.r = r; };
  if (d.mb > 1) set(8, 1, 1, 8);
  else if (KS <= 4) set(8, 1, 1, 4);
  else if (KS <= 8) set(4, 2, 1, 4);
  else if (KS <= 16) set(2, 4, 1, 4);
  else if (nt < 256) set(1, 10, 1, 4);
  else if (KS >= 96) set(4, 3, 1, 8);
  else if (nt < 512) set(2, 5, 1, 8);
  else set(3, 5, 1, 8);
  d.groups = (nt + d.tw * d.t - 1) / (d.tw * d.t);
  d.s = (KS + d.kw * d.r - 1) / (d.kw * d.r);
  d.iters = 1;
  return d;
}

// The weight stream takes up to 16 rows (M = 16 N = K = 5120 6.3 us, tiles 8.9),
// and up to 64 where K is long and N narrow (K >= 12288, N < 8192): there its K
// splits over workgroups keep more of the GPU loading than the tiles' K groups
// (M = 48: N = 5120 K = 17408 24.4 us against 28.5; N = 7168 K = 12288, the
// border, 22.0 against 21.6).  A split has a counter for every column group and
// a grid layer for every run of K: wider N (from 786448 at K > 5120) and longer
// K (past 67 million, up to 16 rows 335 million) are left to the tiles, which
// need neither.
bool use_stream(int M, int N, int KS) {
  if (M > 16 && (M > 64 || KS < 96 || N >= 8192)) return false;
  const StreamCfg d = dense_stream_cfg(M, N, KS);
  return d.s == 1 || (d.s <= kMaxSplits && d.groups * d.mtiles <= kWsMaxCounters);
}

template <int MB, int TW, int KW, int T, int R, bool GROUPED>
int launch_stream(const StreamCfg& d, W4A4Args& p, hipStream_t st) {
  const size_t lds = stream_lds(d);
  if (lds > kMaxStreamLds || d.mtiles > 65535 || d.s > kMaxSplits) return BS_ERR_SHAPE;
  p.rs = d.rs;
  p.iters = d.iters;
  auto* fn = &k_w4a4_stream<MB, TW, KW, T, R, GROUPED>;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(kMaxStreamLds));
  if (attr != hipSuccess) return BS_ERR_LAUNCH;
  fn<<<dim3(d.groups, d.mtiles, d.s), TW * KW * 64, lds, st>>>(p);
  return bs_launch_status();
}

int run_dense_stream(W4A4Args& p, void* ws, hipStream_t st) {
  const StreamCfg d = dense_stream_cfg(p.M, p.N, p.KS);
  if (d.s > 1) {
    p.counters = static_cast<int*>(ws);
    p.slab = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
  }
  // one instantiation per configuration of dense_stream_cfg
  if (d.mb == 4) return launch_stream<4, 8, 1, 1, 8, false>(d, p, st);
  if (d.mb == 2) return launch_stream<2, 8, 1, 1, 8, false>(d, p, st);
  if (d.tw == 8) return launch_stream<1, 8, 1, 1, 4, false>(d, p, st);
  if (d.kw == 2) return launch_stream<1, 4, 2, 1, 4, false>(d, p, st);
  if (d.kw == 4) return launch_stream<1, 2, 4, 1, 4, false>(d, p, st);
  if (d.kw == 10) return launch_stream<1, 1, 10, 1, 4, false>(d, p, st);
  if (d.kw == 3) return launch_stream<1, 4, 3, 1, 8, false>(d, p, st);
  if (d.tw == 2) return launch_stream<1, 2, 5, 1, 8, false>(d, p, st);
  return launch_stream<1, 3, 5, 1, 8, false>(d, p, st);
}

// One 16-byte load per row and window of activation scales (see TileCfg).
bool scales16(const W4A4Args& p) { return p.KS % 4 == 0 && p.lds % 16 == 0 && bs_aligned(p.as, 16); }

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int OCC, bool GROUPED>
int launch_tile(const W4A4Args& p, int64_t wgs, hipStream_t st) {
  if (wgs > 0x7FFFFFFF) return BS_ERR_SHAPE;
  const dim3 grid(static_cast<uint32_t>(wgs)), block(64 * WM * WN * KG);
  // group_m 4: the raster's m-tiles that sweep n together (2 to 16 within 1%)
  if (scales16(p)) k_w4a4_tile<BM, BN, WM, WN, KG, STAGES, OCC, GROUPED, true><<<grid, block, 0, st>>>(p, 4);
  else k_w4a4_tile<BM, BN, WM, WN, KG, STAGES, OCC, GROUPED, false><<<grid, block, 0, st>>>(p, 4);
  return bs_launch_status();
}

// The dense tile shapes and what a launch of each takes, in us: with x = tiles
// / 256 (one per CU) and R = ceil(x) rounds,
//   t = start + R * (round + steps * step) + x * steps * load
// fitted over 13 row counts from 24 to 4096 at ten N x K, N = 1024 .. 17408 and
// K = 512 .. 17408, weights pooled past the last-level cache: by least squares
// (rms 12 to 18%), then moved to the least loss by the choice (the shape with
// the smallest t is the measured best or within 1% of it in 124 of the 130, at
// worst 14%).  128 x 256, whose two workgroups fill a CU's LDS, takes over
// between half a round and one of the large tiles (M = 1024 N = K = 5120 28.2
// us, 128 x 128 36.8, 256 x 256 41.0); with exactly 256 workgroups of it some
// CUs may get two and others none (M = 2048 N = 4096 K = 1024 9.0 to 15.2 us;
// 192 of them 8.9): two rounds.  Two K groups of 64 x 64 tiles pay from K =
// 2048 on (M = 24 N = K = 5120 9.3 us, one group 11.3; N = 4096 K = 1024 4.0
// and 3.8), of 64 x 128 tiles nowhere (M = 128 N = 10240 K = 5120 17.1, one 16.5).
struct TileShape {
  int bm, bn;
  float start, round, step, load;
};
constexpr TileShape kTiles[] = {
    {256, 256, 0.362f, 7.182f, 0.420f, 0.617f}, // 4 waves of 128 x 128
    {128, 256, 2.993f, 0.687f, 0.388f, 0.270f}, // 4 waves of 64 x 128, two workgroups a CU
    {128, 128, 2.326f, 0.716f, 0.265f, 0.160f}, // 4 waves of 64 x 64, two workgroups a CU
    {64, 128, 3.186f, 0.181f, 0.243f, 0.037f},  // 4 waves of 64 x 32, three workgroups a CU
    {64, 64, 2.547f, 0.465f, 0.125f, 0.056f},   // 2 K groups of 2 waves of 64 x 32, two workgroups a CU
    {64, 64, 2.425f, 0.000f, 0.207f, 0.010f},   // 4 waves of 32 x 32, four workgroups a CU
};
float tile_cost(int i, int M, int N, int KS) {
  const TileShape& t = kTiles[i];
  const int64_t tiles = static_cast<int64_t>((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
  const float x = static_cast<float>(tiles) / 256.0f;
  const float rounds = i == 1 && tiles == 256 ? 2.0f : std::ceil(x);
  return t.start + rounds * (t.round + KS * t.step) + x * KS * t.load;
}
int best_tile(int M, int N, int KS) {
  int best = 0;
  for (int i = 1; i < 6; ++i)
    if (tile_cost(i, M, N, KS) < tile_cost(best, M, N, KS)) best = i;
  return best;
}

// columns [n0, n1) of the problem as tiles of shape i
int run_tiles(int i, const W4A4Args& q, int n0, int n1, hipStream_t st) {
  W4A4Args p = q;
  const size_t nt = static_cast<size_t>(n0) / 16;
  p.w += nt * p.KS * 1024;
  p.wsc += nt * ((p.KS + 3) / 4) * 256;
  p.c += n0;
  p.N = n1 - n0;
  const int64_t wgs =
      static_cast<int64_t>((p.M + kTiles[i].bm - 1) / kTiles[i].bm) * ((p.N + kTiles[i].bn - 1) / kTiles[i].bn);
  switch (i) {
    case 0: return launch_tile<256, 256, 2, 2, 1, 4, 1, false>(p, wgs, st);
    case 1: return launch_tile<128, 256, 2, 2, 1, 3, 2, false>(p, wgs, st);
    case 2: return launch_tile<128, 128, 2, 2, 1, 4, 2, false>(p, wgs, st);
    case 3: return launch_tile<64, 128, 1, 4, 1, 4, 3, false>(p, wgs, st);
    case 4: return launch_tile<64, 64, 1, 2, 2, 4, 2, false>(p, wgs, st);
    default: return launch_tile<64, 64, 2, 2, 1, 4, 4, false>(p, wgs, st);
  }
}

// One shape for all columns; or, where the large tiles would end in a partial
// round, large tiles over as many columns as whole rounds take and the rest as
// the shape that is quickest there (the second launch costs about 1 us more).
int run_dense_tile(const W4A4Args& p, hipStream_t st) {
  const int b = best_tile(p.M, p.N, p.KS);
  const int mt = (p.M + 255) / 256, nt = (p.N + 255) / 256;
  const int rounds = mt * static_cast<int64_t>(nt) / 256;
  if (rounds >= 1) {
    const int n1 = rounds * 256 / mt * 256;   // < N unless the rounds are whole
    if (n1 > 0 && n1 < p.N) {
      const int r = best_tile(p.M, p.N - n1, p.KS);
      if (tile_cost(0, p.M, n1, p.KS) + tile_cost(r, p.M, p.N - n1, p.KS) + 1.0f < tile_cost(b, p.M, p.N, p.KS)) {
        const int rc = run_tiles(0, p, 0, n1, st);
        return rc != BS_OK ? rc : run_tiles(r, p, n1, p.N, st);
      }
    }
  }
  return run_tiles(b, p, 0, p.N, st);
}

}  // namespace

size_t bs_w4a4_workspace(int M, int N, int K) {
  if (!use_stream(M, N, K / 128)) return 0;
  const StreamCfg d = dense_stream_cfg(M, N, K / 128);
  return d.s > 1 ? kWsCounterBytes + static_cast<size_t>(d.s) * d.mtiles * d.groups * d.tw * d.t * d.mb * 1024 : 0;
}

int bs_launch_w4a4(const uint8_t* a, int64_t lda, const uint8_t* as, int64_t lds, const uint8_t* w, size_t w_scales,
                   uint16_t* c, int64_t ldc, int M, int N, int K, void* ws, hipStream_t st) {
  W4A4Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.lds = static_cast<uint32_t>(lds);
  p.w = w;
  p.wsc = w + w_scales;
  p.c = c;
  p.ldc = ldc;
  p.M = M;
  p.N = N;
  p.KS = K / 128;
  return use_stream(M, N, p.KS) ? run_dense_stream(p, ws, st) : run_dense_tile(p, st);
}

// The weight stream over tiles of 16 rows and 16 * TW * T columns, KW * R steps
// of K at a time.
template <int TW, int KW, int T, int R>
int launch_grouped_stream(W4A4Args& p, int S, hipStream_t st) {
  const StreamCfg d{1,  TW, KW, T, R, 16, (p.N / 16 + TW * T - 1) / (TW * T), tile_bound(S, p.E, 16),
                    1,  (p.KS + KW * R - 1) / (KW * R)};
  return launch_stream<1, TW, KW, T, R, true>(d, p, st);
}

// Row tiles by S / E, the rows an expert would have if they were spread evenly
// (swept at 256, 128, 64, 16 and 8 experts, S / E from 1/32 to 4096, weights
// pooled past the last-level cache):
//   - few rows (S / E < 16, from K = 1152 on < 10: at 12 rows the stream takes
//     53 to 55 us against 52.6, at 8 49.6 against 51.9): the weight stream.  A
//     workgroup of eight waves takes 256 columns with no K split, so that all
//     its waves are busy at any K (256 experts N = 2048 K = 512, 64 rows of 8:
//     22.4 us, 128 columns in two K groups 32.6; N = 1024 K = 2048, 128 rows
//     23.1 against 24.1); 128 columns in two K groups where the grid is then
//     two workgroups a CU or less, or K > 2048 (32 rows 9.9 us against 11.9; 64
//     experts N = 1024 K = 5120, 32 rows 17.9 against 25.1, 512 rows 32.5
//     against 34.8); 64 columns in four K groups where even that leaves half
//     the CUs idle (8 rows of K = 2048 5.8 us against 7.1; 8 experts, one row of
//     N = K = 4096 7.6 against 10.8);
//   - up to 32 rows of K > 1024: 64 x 128 tiles, three workgroups a CU (64
//     experts N = 1024 K = 2048: 15 rows 16.1 us, 128 x 256 16.9; 37 rows 17.8 and
//     17.4, 48 rows 21.4 and 17.6; 256 experts, 16 rows 54 us, the stream 60);
//   - else 128 x 256 tiles, two workgroups a CU, so one's stores run under the
//     other's MFMAs (256 experts N = 1024 K = 2048, 65536 rows 118 us; 128 x 128
//     144, 256 x 256 142, which gains from 2000 rows of K = 7168 on only, 7%).
int bs_launch_w4a4_grouped(const uint8_t* a, int64_t lda, const uint8_t* as, int64_t lds, const int* offsets,
                           const int* rows, const uint8_t* w, size_t w_scales, size_t w_stride, uint16_t* c,
                           int64_t ldc, int S, int Ma, int E, int N, int K, hipStream_t st) {
  W4A4Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.lds = static_cast<uint32_t>(lds);
  p.w = w;
  p.wsc = w + w_scales;
  p.w_stride = w_stride;
  p.c = c;
  p.ldc = ldc;
  p.M = S;
  p.N = N;
  p.KS = K / 128;
  p.offsets = offsets;
  p.rows = rows;
  p.E = E;
  p.Ma = Ma;
  const int avg = S / E;
  if (avg < (p.KS <= 8 ? 16 : 10)) {
    const int64_t wgs = static_cast<int64_t>(tile_bound(S, E, 16)) * ((N + 127) / 128);
    if (wgs <= 128 && p.KS > 8) return launch_grouped_stream<2, 4, 2, 4>(p, S, st);
    if (p.KS > 16 || (wgs <= 512 && p.KS > 4)) return launch_grouped_stream<4, 2, 2, 4>(p, S, st);
    return launch_grouped_stream<8, 1, 2, 4>(p, S, st);
  }
  if (p.KS > 8 && avg <= 32)
    return launch_tile<64, 128, 1, 4, 1, 4, 3, true>(p, static_cast<int64_t>(tile_bound(S, E, 64)) * ((N + 127) / 128),
                                                     st);
  return launch_tile<128, 256, 2, 2, 1, 3, 2, true>(p, static_cast<int64_t>(tile_bound(S, E, 128)) * ((N + 255) / 256),
                                                    st);
}
