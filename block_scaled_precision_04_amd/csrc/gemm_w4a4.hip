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
// Two kernels.  Few rows: a weight stream (k_w4a4_stream), bound by HBM.
// Many rows: LDS-tiled (k_w4a4_tile), bound by the matrix cores, fed through
// direct-to-LDS loads.  Both have a grouped form: the slots of the sorted
// (token, expert) pairs are cut into row tiles expert by expert, and every
// workgroup finds its tile from the expert offsets on the device, so the host
// never waits for them; the activation rows are read through the sorted order
// (row gather in the loads), never copied.
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace {

struct W4A4Args {
  const uint8_t* a;      // e2m1 codes [rows, K/2], lda bytes apart
  const uint8_t* as;     // e8m0 [rows, K/32], lds bytes apart
  uint32_t lda, lds;
  const uint8_t* w;      // pre-laid-out weight(s)
  size_t w_scales;       // byte offset of the e8m0 section
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

// The `tile`-th row tile of the grouped problem: the slots of expert e are cut
// into runs of up to BM.  Lane l looks at experts 4l .. 4l+3 of each 256; a
// wave-wide scan of their tile counts finds the tile.  Offsets are clamped to
// [0, S], so whatever they hold no slot outside the buffers is named.
// Returns false past the last tile.
template <int BM>
BS_INLINE bool find_tile(const int* __restrict__ offsets, int E, int S, int tile, int& expert, int& r0, int& r1) {
  const int l = threadIdx.x & 63;
  int run = 0;
  for (int b = 0; b < E; b += 256) {
    int o[5], cnt[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) o[i] = min(max(offsets[min(b + 4 * l + i, E)], 0), S);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cnt[i] = o[i + 1] > o[i] ? (o[i + 1] - o[i] + BM - 1) / BM : 0;
      mine += cnt[i];
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      incl += l >= d ? v : 0;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (tile < run + total) {
      int before = run + incl - mine;
      int fe = -1, f0 = 0, f1 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (tile >= before && tile < before + cnt[i]) {
          fe = b + 4 * l + i;
          f0 = o[i] + (tile - before) * BM;
          f1 = min(f0 + BM, o[i + 1]);
        }
        before += cnt[i];
      }
      const int src = __builtin_ctzll(__ballot(fe >= 0));
      expert = __builtin_amdgcn_readlane(fe, src);
      r0 = __builtin_amdgcn_readlane(f0, src);
      r1 = __builtin_amdgcn_readlane(f1, src);
      return true;
    }
    run += total;
  }
  return false;
}

// ceil(count / BM) summed over experts is largest when as many experts as
// possible hold one row: with A = min(S, E) of them, A + (S - A) / BM.
int tile_bound(int S, int E, int BM) {
  const int A = std::min(S, E);
  return A + (S - A) / BM;
}

// Source row of tile row i (slot r0 + i).
BS_INLINE int src_row(const W4A4Args& p, int slot) {
  const int r = p.rows != nullptr ? p.rows[slot] : slot;
  return min(max(r, 0), p.Ma - 1);
}

// ============================================================ few rows: stream
// 16-byte chunk swizzle of a 64-byte activation row in LDS: the 16 rows of a
// fragment read take one chunk each, four rows per 256-byte line.
BS_INLINE int swz4(int row, int chunk) { return chunk ^ ((row >> 2) & 3); }

// grid (column groups, row tiles, K splits): workgroup (x, y, z) computes
// n-tiles [x*TW*T, (x+1)*TW*T) of 16 columns for the 16*MB rows of row tile y
// over its run of `iters * KW * R` K steps.  Wave (tw, kw) owns T tiles over R
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
  const uint8_t* w = p.w;
  if constexpr (GROUPED) {
    int e, r1;
    if (!find_tile<16 * MB>(p.offsets, p.E, p.M, blockIdx.y, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
  } else {
    m0 = blockIdx.y * 16 * MB;
    nrows = min(RS, p.M - m0);
  }
  const uint32_t* wsc = reinterpret_cast<const uint32_t*>(w + p.w_scales);

  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
  const int a_instr = (kSteps * RS * 4 + 63) >> 6, s_instr = (kSteps * RS + 63) >> 6;
  const uint32_t* s_sc = reinterpret_cast<const uint32_t*>(lds + a_instr * 1024);
  float* s_red = reinterpret_cast<float*>(lds);

  v4f acc[T][MB];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[t][mb] = v4f{0, 0, 0, 0};

  for (int it = 0; it < p.iters; ++it) {
    const int wg_k0 = (blockIdx.z * p.iters + it) * kSteps;
    if (wg_k0 >= KS) break;
    const int wg_steps = min(kSteps, KS - wg_k0);
    const int ks0 = wg_k0 + kw * R;
    const int klast = min(ks0 + R, KS) - 1;  // below ks0 for an idle wave
    const int nsteps = klast - ks0 + 1;      // <= 0 for an idle wave
    if (it) __syncthreads();                 // every wave is done with the slice
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
// of 1 KiB, as they are) go global -> LDS by direct loads into one of four
// stage buffers; the scales of a window (16 B per activation row, 256 B per 16
// columns) into one of two window buffers.  The four steps of a window are
// unrolled, so the stage, the scale dword and its byte are constants of the
// code, and a window's scales are read from LDS once, ahead of the window.
//
// AS16: the activation scale rows are 16-byte aligned and K is a multiple of
// 512, so a row's window is one 16-byte load (rows of 16 B); otherwise it is
// four 4-byte loads (planes of BM dwords).  One 4-byte load per row and step
// touched as many cache lines per step as the codes themselves.
template <int BM, int BN, int WM, int WN, bool AS16>
struct TileCfg {
  static constexpr int kStages = 4;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kTM = BM / WM / 32, kTN = BN / WN / 32;
  static constexpr int kA = BM * 64, kB = BN * 64, kStage = kA + kB;
  static constexpr int kSB = BN * 16, kSA = BM * 16, kWin = kSB + kSA;
  static constexpr int kWin0 = kStages * kStage;       // the window buffers follow the stages
  static constexpr int kAIters = kA / (kThreads * 16), kBIters = kB / (kThreads * 16);
  static constexpr int kSBPieces = kSB / 1024, kSAPieces = AS16 ? kSA / 1024 : kSA / 256;
  // loads per stage and per window, the same for every wave: a wave past a
  // section's last piece repeats an earlier one (same bytes, same place)
  static constexpr int kSBIters = (kSBPieces + kWaves - 1) / kWaves, kSAIters = (kSAPieces + kWaves - 1) / kWaves;
  static constexpr int kDma = kAIters + kBIters, kWinDma = kSBIters + kSAIters;
  static_assert(kA % (kThreads * 16) == 0 && kB % (kThreads * 16) == 0 && kSB % 1024 == 0 && kSA % 1024 == 0, "");
  static constexpr int kPassN = BN < 128 ? BN : 128;   // columns staged at once by the epilogue
  static constexpr int kMain = kWin0 + 2 * kWin;
  static constexpr int kLds = kMain > BM * kPassN * 4 ? kMain : BM * kPassN * 4;
};

template <int V>
using Int = std::integral_constant<int, V>;

template <int BM, int BN, int WM, int WN, int OCC, bool GROUPED, bool SPLIT, bool AS16>
__global__ __launch_bounds__(64 * WM * WN, OCC) void k_w4a4_tile(W4A4Args p, int group_m) {
  using C = TileCfg<BM, BN, WM, WN, AS16>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int N = p.N, KS = p.KS, NT = N >> 4, KQ = (KS + 3) >> 2;
  const int n_tiles = (N + BN - 1) / BN;
  // K splits cut between windows
  const int S = SPLIT ? static_cast<int>(gridDim.y) : 1, sp = SPLIT ? static_cast<int>(blockIdx.y) : 0;
  const int w_begin = SPLIT ? KQ * sp / S : 0, w_end = SPLIT ? KQ * (sp + 1) / S : KQ;
  const int k_last = min(4 * w_end, KS) - 1;

  int m0, nrows, nt;
  const uint8_t* w = p.w;
  if constexpr (GROUPED) {
    int e, r1;
    nt = blockIdx.x % n_tiles;
    if (!find_tile<BM>(p.offsets, p.E, p.M, blockIdx.x / n_tiles, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
  } else {
    int mt;
    xcd_tile(blockIdx.x, (p.M + BM - 1) / BM, n_tiles, group_m, mt, nt);
    m0 = mt * BM;
    nrows = min(BM, p.M - m0);
  }
  const uint8_t* wsc = w + p.w_scales;
  const int n0 = nt * BN, nt0 = n0 >> 4;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));

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
  // the i-th load of window win into its buffer
  auto win_one = [&](int i, int win) {
    const uint32_t base = lds0 + C::kWin0 + (win & 1) * C::kWin;
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
    const uint8_t* base = lds + st * C::kStage;
    if (i == 0 || i > C::kTM) {
      const int t = i == 0 ? 0 : i - C::kTM;
      f.b[t] = *reinterpret_cast<const v4i*>(base + bbase + t * 2048 + hh * 512);
    } else {
      f.a[i - 1] = *reinterpret_cast<const v4i*>(base + abase[hh] + (i - 1) * 2048);
    }
  };
  auto read_scale = [&](int win, Scale& s, int i) {
    const uint8_t* base = lds + C::kWin0 + (win & 1) * C::kWin;
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
  auto shift_scale = [&](Scale& s) {
#pragma unroll
    for (int t = 0; t < C::kTM; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.a[t][j] = static_cast<int>(static_cast<uint32_t>(s.a[t][j]) >> sh_a);
  };
  // MFMAs of half HH of step J of a window.  Between them: the LDS reads of the
  // next half (rf, from stage rst, half rhh), this half's share of the loads of
  // step dks (into stage (J + 3) % 4), of the next window's scale loads (J = 0)
  // and, in the window's last half, the reads of the next window's scales.
  auto half = [&](auto jj, auto hh, const Frag& f, const Scale& s, int rst, int rhh, Frag& rf, int dks, int win,
                  int next_win, Scale& ns) {
    constexpr int J = decltype(jj)::value, HH = decltype(hh)::value;
    constexpr int kN = C::kTN * C::kTM;
    constexpr int d0 = HH * ((C::kDma + 1) / 2), d1 = HH ? C::kDma : (C::kDma + 1) / 2;
    (void)win;
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
      if (n < kPieces) piece(rst, rhh, rf, n);
      // the loads, spread evenly over the half's MFMAs
#pragma unroll
      for (int d = d0; d < d1; ++d)
        if ((d - d0) * kN / (d1 - d0) == n) dma_one(d, dks, (J + 3) & 3);
      if (J == 0 && HH == 1 && n == kN - 1)
#pragma unroll
        for (int d = 0; d < C::kWinDma; ++d) win_one(d, next_win);
      if (J == 3 && HH == 1) {
#pragma unroll
        for (int d = 0; d < kPieces; ++d)
          if (d * kN / kPieces == n) read_scale(next_win, ns, d);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s: this wave's loads of step s+1 have landed and its LDS reads are
  // done; barrier (s+1 published, the stage of s-1 free); then the two halves.
  // The loads of a step are issued three steps ahead.  Steps past the end
  // re-load the last one (never used).
  Frag f0, f1;
  Scale s0, s1;
#pragma unroll
  for (int d = 0; d < C::kWinDma; ++d) win_one(d, w_begin);
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int i = 0; i < C::kDma; ++i) dma_one(i, min(4 * w_begin + s, k_last), s);
  wait_vm<2 * C::kDma>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPieces; ++i) piece(0, 0, f0, i);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) read_scale(w_begin, s0, i);
  auto step = [&](auto jj, int win, Scale& s, Scale& ns) {
    constexpr int J = decltype(jj)::value;
    const int ks = 4 * win + J, next = min(win + 1, w_end - 1);
    // newer loads that may be outstanding: those of step s+2, and the window's
    // scale loads when they were issued after them (in step 0)
    wait_vm<C::kDma + (J == 1 ? C::kWinDma : 0)>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (J == 0) shift_scale(s);
    half(jj, Int<0>{}, f0, s, J, 1, f1, min(ks + 3, k_last), win, next, ns);
    half(jj, Int<1>{}, f1, s, (J + 1) & 3, 0, f0, min(ks + 3, k_last), win, next, ns);
  };
  // two windows per turn, so the scale sets swap without copies
  auto window = [&](int win, Scale& s, Scale& ns) {
    step(Int<0>{}, win, s, ns);
    if (4 * win + 1 <= k_last) step(Int<1>{}, win, s, ns);
    if (4 * win + 2 <= k_last) step(Int<2>{}, win, s, ns);
    if (4 * win + 3 <= k_last) step(Int<3>{}, win, s, ns);
  };
  for (int win = w_begin; win < w_end; win += 2) {
    window(win, s0, s1);
    if (win + 1 < w_end) window(win + 1, s1, s0);
  }
  wait_vm<0>();

  // K splits: partial tile in fragment order through the workspace
  if constexpr (SPLIT) {
    if (S > 1) {
      __shared__ int last;
      constexpr int kNV = C::kTN * C::kTM * 16;
      float* base = p.slab + (static_cast<size_t>(blockIdx.x) * C::kWaves + wave) * (kNV * 64) + l;
      const size_t stride = static_cast<size_t>(gridDim.x) * C::kWaves * (kNV * 64);
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            __hip_atomic_store(base + sp * stride + ((i * C::kTM + j) * 16 + r) * 64, acc[i][j][r], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
      __syncthreads();
      if (tid == 0)
        last = __hip_atomic_fetch_add(&p.counters[blockIdx.x], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == S - 1;
      __syncthreads();
      if (!last) return;
      float sum[kNV];
      sum_partials<kNV, 64, 1>(sum, base, stride, S);
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = sum[(i * C::kTM + j) * 16 + r];
      if (tid == 0) __hip_atomic_store(&p.counters[blockIdx.x], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }

  // Epilogue: fp32 through LDS, kPassN columns of the tile at a time, so that
  // each store instruction writes whole pieces of rows.  16-byte chunk q of a
  // row sits at slot q ^ (row % 16).
  constexpr int kPassN = C::kPassN, kPasses = BN / kPassN;
  constexpr int kPP = C::kTN / kPasses;             // a wave's sub-tiles per pass
  constexpr int kW = kPP * 32;                      // a wave's columns per pass
  static_assert(WN * kW == kPassN && C::kTN % kPasses == 0, "");
  constexpr int kLanes = kPassN / 8;                // lanes per row, 8 columns each
  constexpr int kRows = C::kThreads / kLanes;
  static_assert(BM % kRows == 0, "");
  const int lane8 = tid % kLanes, rsub = tid / kLanes;
#pragma unroll
  for (int h = 0; h < kPasses; ++h) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::kTM; ++j) {
      uint8_t* rowp = lds + arow[j] * (kPassN * 4);
      const int x = arow[j] & 15;
#pragma unroll
      for (int i = 0; i < kPP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const v16f& av = acc[h * kPP + i][j];
          const int q = wn * (kW / 4) + 8 * i + 2 * r + (l >> 5);
          *reinterpret_cast<float4*>(rowp + ((q ^ x) << 4)) =
              make_float4(av[4 * r], av[4 * r + 1], av[4 * r + 2], av[4 * r + 3]);
        }
    }
    __syncthreads();
    // staged column x of pass h is tile column (x / kW) * (BN / WN) + h * kW + x % kW
    const int x0 = 4 * lane8, x1 = kPassN / 2 + 4 * lane8;
    const int c0 = n0 + x0 / kW * (BN / WN) + h * kW + x0 % kW, c1 = n0 + x1 / kW * (BN / WN) + h * kW + x1 % kW;
#pragma unroll 4
    for (int r = rsub; r < BM; r += kRows) {
      const uint8_t* rp = lds + r * (kPassN * 4);
      const float4 u = *reinterpret_cast<const float4*>(rp + ((lane8 ^ (r & 15)) << 4));
      const float4 v = *reinterpret_cast<const float4*>(rp + (((lane8 + kPassN / 8) ^ (r & 15)) << 4));
      if (r < nrows) {
        uint16_t* dst = p.c + (m0 + r) * p.ldc;
        // N % 16 == 0: a piece of four columns is wholly inside or outside
        if (c0 < N) st_stream8(reinterpret_cast<uint2*>(dst + c0), bf16x2_rne(u.x, u.y), bf16x2_rne(u.z, u.w));
        if (c1 < N) st_stream8(reinterpret_cast<uint2*>(dst + c1), bf16x2_rne(v.x, v.y), bf16x2_rne(v.z, v.w));
      }
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int kStreamMaxM = 64;   // dense: up to here the weight stream runs
constexpr size_t kMaxStreamLds = 160 * 1024 - 256;

struct StreamCfg {
  int mb, tw, kw, t, r, rs, groups, mtiles, s, iters;
};
size_t stream_lds(const StreamCfg& d) {
  const size_t pos = static_cast<size_t>(d.kw) * d.r * d.rs;
  const size_t slice = (pos * 4 + 63) / 64 * 1024 + (pos + 63) / 64 * 256;
  const size_t red = static_cast<size_t>(d.kw - 1) * d.tw * d.t * d.mb * 4 * 64 * sizeof(float);
  return std::max(slice, red);
}

StreamCfg dense_stream_cfg(int M, int N, int KS) {
  StreamCfg d{};
  d.mb = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
  d.rs = std::min(M, 16 * d.mb);
  d.mtiles = (M + 16 * d.mb - 1) / (16 * d.mb);
  auto set = [&](int tw, int kw, int t, int r) { d.tw = tw; d.kw = kw; d.t = t; d.r = r; };
  if (d.mb == 1) {
    if (KS >= 96) set(4, 3, 1, 8);
    else if (M >= 5 && N / 16 >= 640) set(3, 5, 1, 8);
    else set(1, 10, 1, 4);
  } else {
    set(8, 1, 1, 8);
  }
  d.groups = (N / 16 + d.tw * d.t - 1) / (d.tw * d.t);
  d.s = (KS + d.kw * d.r - 1) / (d.kw * d.r);
  d.iters = 1;
  return d;
}

StreamCfg grouped_stream_cfg(int S, int E, int N, int KS, int mb) {
  StreamCfg d{};
  d.mb = mb;
  d.rs = 16 * mb;
  d.mtiles = tile_bound(S, E, 16 * mb);
  d.tw = mb == 1 ? 2 : 4;
  d.kw = mb == 1 ? 4 : 2;
  d.t = 1;
  d.r = 4;
  d.groups = (N / 16 + d.tw * d.t - 1) / (d.tw * d.t);
  d.s = 1;
  d.iters = (KS + d.kw * d.r - 1) / (d.kw * d.r);
  return d;
}

template <int MB, int TW, int KW, int T, int R, bool GROUPED>
int launch_stream(const StreamCfg& d, W4A4Args& p, hipStream_t st) {
  const size_t lds = stream_lds(d);
  if (lds > kMaxStreamLds || d.mtiles > 65535 || d.s > 65535) return BS_ERR_SHAPE;
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
    if (d.groups * d.mtiles > kWsMaxCounters) return BS_ERR_SHAPE;
    p.counters = static_cast<int*>(ws);
    p.slab = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
  }
  if (d.mb == 1 && d.kw == 3) return launch_stream<1, 4, 3, 1, 8, false>(d, p, st);
  if (d.mb == 1 && d.kw == 5) return launch_stream<1, 3, 5, 1, 8, false>(d, p, st);
  if (d.mb == 1) return launch_stream<1, 1, 10, 1, 4, false>(d, p, st);
  if (d.mb == 2) return launch_stream<2, 8, 1, 1, 8, false>(d, p, st);
  return launch_stream<4, 8, 1, 1, 8, false>(d, p, st);
}

// Tiles of the dense problem: 256x256 where they fill the GPU (one workgroup
// per CU), otherwise 128x128 with K split until about 256 workgroups run.
struct TilePlan {
  bool large;
  int tiles, s;
};
TilePlan tile_plan(int M, int N, int KS) {
  const int big = ((M + 255) / 256) * ((N + 255) / 256);
  if (big >= 192) return TilePlan{true, big, 1};
  const int t = ((M + 127) / 128) * ((N + 127) / 128);
  const int s = t < 256 ? std::max(1, std::min(256 / t, KS / 8)) : 1;
  return TilePlan{false, t, s};
}

// One 16-byte load per row and window of activation scales (see TileCfg).
bool scales16(const W4A4Args& p) { return p.KS % 4 == 0 && p.lds % 16 == 0 && bs_aligned(p.as, 16); }

int run_dense_tile(W4A4Args& p, void* ws, hipStream_t st) {
  const TilePlan pl = tile_plan(p.M, p.N, p.KS);
  const bool as16 = scales16(p);
  if (pl.large) {
    if (as16) k_w4a4_tile<256, 256, 2, 2, 1, false, false, true><<<dim3(pl.tiles, 1), 256, 0, st>>>(p, 4);
    else k_w4a4_tile<256, 256, 2, 2, 1, false, false, false><<<dim3(pl.tiles, 1), 256, 0, st>>>(p, 4);
    return bs_launch_status();
  }
  if (pl.s > 1) {
    p.counters = static_cast<int*>(ws);
    p.slab = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
  }
  if (as16) k_w4a4_tile<128, 128, 2, 2, 2, false, true, true><<<dim3(pl.tiles, pl.s), 256, 0, st>>>(p, 4);
  else k_w4a4_tile<128, 128, 2, 2, 2, false, true, false><<<dim3(pl.tiles, pl.s), 256, 0, st>>>(p, 4);
  return bs_launch_status();
}

}  // namespace

size_t bs_w4a4_workspace(int M, int N, int K) {
  if (M <= kStreamMaxM) {
    const StreamCfg d = dense_stream_cfg(M, N, K / 128);
    return d.s > 1 ? kWsCounterBytes + static_cast<size_t>(d.s) * d.mtiles * d.groups * d.tw * d.t * d.mb * 1024 : 0;
  }
  const TilePlan pl = tile_plan(M, N, K / 128);
  return pl.s > 1 ? kWsCounterBytes + static_cast<size_t>(pl.s) * pl.tiles * 128 * 128 * sizeof(float) : 0;
}

int bs_launch_w4a4(const uint8_t* a, int64_t lda, const uint8_t* as, int64_t lds, const uint8_t* w, size_t w_scales,
                   uint16_t* c, int64_t ldc, int M, int N, int K, void* ws, hipStream_t st) {
  W4A4Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.lds = static_cast<uint32_t>(lds);
  p.w = w;
  p.w_scales = w_scales;
  p.c = c;
  p.ldc = ldc;
  p.M = M;
  p.N = N;
  p.KS = K / 128;
  return M <= kStreamMaxM ? run_dense_stream(p, ws, st) : run_dense_tile(p, ws, st);
}

int bs_launch_w4a4_grouped(const uint8_t* a, int64_t lda, const uint8_t* as, int64_t lds, const int* offsets,
                           const int* rows, const uint8_t* w, size_t w_scales, size_t w_stride, uint16_t* c,
                           int64_t ldc, int S, int Ma, int E, int N, int K, hipStream_t st) {
  W4A4Args p{};
  p.a = a;
  p.as = as;
  p.lda = static_cast<uint32_t>(lda);
  p.lds = static_cast<uint32_t>(lds);
  p.w = w;
  p.w_scales = w_scales;
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
  const int avg = S / E;   // rows per expert if they were spread evenly
  if (avg <= 16) return launch_stream<1, 2, 4, 1, 4, true>(grouped_stream_cfg(S, E, N, p.KS, 1), p, st);
  if (avg <= 48) return launch_stream<4, 4, 2, 1, 4, true>(grouped_stream_cfg(S, E, N, p.KS, 4), p, st);
  const int64_t wgs = static_cast<int64_t>(tile_bound(S, E, 128)) * ((N + 127) / 128);
  if (wgs > 0x7FFFFFFF) return BS_ERR_SHAPE;
  if (scales16(p))
    k_w4a4_tile<128, 128, 2, 2, 2, true, false, true><<<dim3(static_cast<uint32_t>(wgs)), 256, 0, st>>>(p, 0);
  else
    k_w4a4_tile<128, 128, 2, 2, 2, true, false, false><<<dim3(static_cast<uint32_t>(wgs)), 256, 0, st>>>(p, 0);
  return bs_launch_status();
}
