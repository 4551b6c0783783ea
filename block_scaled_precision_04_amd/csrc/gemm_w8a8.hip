// int8 GEMM (W8A8: one scale per activation row and one per weight row) and its
// grouped form over the experts of a mixture.
//
//   C[m, n] = bf16( fp32( sum_k A[m,k] W[n,k] ) * as[m] * ws[n] )
//
// The sum is exact: int32 holds K products of two 8-bit codes up to K = 131071.
// So K may be cut anywhere (waves, groups, workgroups) without a change in the
// result.  The weight is laid out in 16-row x 64-K fragment blocks of 1 KiB, N
// padded with zeros to 16 and K to 128; activation bytes past K meet those zeros,
// so they may be any valid bytes of the row.
//
// Two kernels.  Few rows: a weight stream (k_w8a8_stream), bound by HBM.  Many
// rows: LDS-tiled (k_w8a8_tile), fed through direct-to-LDS loads.  Both have a
// grouped form: the slots of the sorted (token, expert) pairs are cut into row
// tiles expert by expert, and every workgroup finds its tile from the expert
// offsets on the device, so the host never waits for them; the activation rows are
// read through the sorted order (row gather in the loads), never copied.
#include <cmath>

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
  int M, N, K, KS;       // dense: rows; grouped: slots.  KS: 64-K blocks of the weight, even
  const int* offsets;    // grouped: [E + 1]
  const int* rows;       // grouped: source row of each slot, or null
  int E, Ma;             // grouped: experts, rows of a
  int tw, kw;            // stream: waves along N and along K
  int rs;                // stream: activation rows staged per workgroup
  int iters;             // stream: K runs per workgroup
  int* slab;
  int* counters;
};

// Source row of tile row i (slot r0 + i).
BS_INLINE int src_row(const W8A8Args& p, int slot) {
  const int r = p.rows != nullptr ? p.rows[slot] : slot;
  return min(max(r, 0), p.Ma - 1);
}

BS_INLINE float scaled(int acc, float sa, float sw) { return static_cast<float>(acc) * sa * sw; }

// ============================================================ few rows: stream
// grid (column groups, row tiles, K splits): workgroup (x, y, z) computes
// n-tiles [x*TW*T, (x+1)*TW*T) of 16 columns for the up to 16*MB rows of row
// tile y (dense: all rows) over its run of `iters * KW * R` K blocks.  Wave (tw,
// kw) owns T tiles over R blocks of each KW*R; the KW partial sums of a tile are
// added through LDS, K splits through the workspace.  The activation slice (KW*R
// blocks x rs rows x 64 B) is copied to LDS by direct loads, shared by the TW*T
// tiles; the weights go straight to registers, all of a wave's loads at once.
template <int MB, int T, int R, bool LOOP, bool GROUPED>
__global__ __launch_bounds__(1024) void k_w8a8_stream(W8A8Args p) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int last;
  const int TW = p.tw, KW = p.kw, kSteps = KW * R;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tw = wave % TW, kw = wave / TW;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int KS = p.KS, RS = p.rs, last_chunk = (p.K >> 4) - 1;
  const int ntiles = (p.N + 15) >> 4;
  const int tile0 = (blockIdx.x * TW + tw) * T;

  int m0, nrows;
  const uint8_t* w = p.w;
  const float* wsc = p.wsc;
  if constexpr (GROUPED) {
    int e, r1;
    if (!find_tile<16 * MB>(p.offsets, p.E, p.M, blockIdx.y, e, m0, r1)) return;
    nrows = r1 - m0;
    w += static_cast<size_t>(e) * p.w_stride;
    wsc += static_cast<size_t>(e) * p.N;
  } else {
    m0 = 0;
    nrows = RS;
  }

  // grouped: byte offset of the row that this lane loads of each row block (looked
  // up once, not anew for every load of the loop below)
  static_assert(!GROUPED || MB == 1, "16 rows a workgroup");
  uint32_t row_off = 0;
  if constexpr (GROUPED) row_off = static_cast<uint32_t>(src_row(p, m0 + min(l >> 2, nrows - 1))) * p.lda;

  // the owner's scales: its row of each row block, its four columns of each tile
  const bool owner = kw == 0;
  float sa[MB], sw[T][4];
  if (owner) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      int src = m0 + min(16 * mb + (l & 15), nrows - 1);
      if constexpr (GROUPED) src = src_row(p, src);
      sa[mb] = p.as[src];
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) sw[t][j] = wsc[min((tile0 + t) * 16 + 4 * g + j, p.N - 1)];
  }

  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
  const int a_instr = (kSteps * RS * 4 + 63) >> 6;
  int* s_red = reinterpret_cast<int*>(lds);

  v4i acc[T][MB];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[t][mb] = v4i{0, 0, 0, 0};

  const int iters = LOOP ? p.iters : 1;   // (the loop costs register copies)
  for (int it = 0; it < iters; ++it) {
    const int wg_k0 = (blockIdx.z * iters + it) * kSteps;
    if (LOOP && wg_k0 >= KS) break;
    const int wg_steps = min(kSteps, KS - wg_k0);
    const int ks0 = wg_k0 + kw * R;
    const int klast = min(ks0 + R, KS) - 1;  // below ks0 for an idle wave
    const int nsteps = klast - ks0 + 1;      // <= 0 for an idle wave
    if (LOOP && it) __syncthreads();      // every wave is done with the slice
    // chunk c of row i of block r sits at position (r*RS + i)*4 + swz4(i, c);
    // positions past the slice, and chunks past K, re-read valid bytes (the
    // weight is zero there)
    if constexpr (GROUPED) {   // (RS = 16: a load is 16 rows of a block, the lane's row always the same)
      for (int k = wave; k < a_instr; k += TW * KW) {
        const int r = min(k, wg_steps - 1);
        dma16(lds0 + k * 1024, p.a,
              row_off + static_cast<uint32_t>(min((wg_k0 + r) * 4 + swz4(l >> 2, l & 3), last_chunk) * 16));
      }
    } else {
      for (int k = wave; k < a_instr; k += TW * KW) {
        const int q = k * 64 + l;
        const int ri = q >> 2;
        const int r = min(ri / RS, wg_steps - 1);
        const int ii = ri % RS;
        const int row = m0 + min(ii, nrows - 1);
        dma16(lds0 + k * 1024, p.a,
              static_cast<uint32_t>(row) * p.lda +
                  static_cast<uint32_t>(min((wg_k0 + r) * 4 + swz4(ii, q & 3), last_chunk) * 16));
      }
    }
    v4i wf[T][R];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const size_t tile = static_cast<size_t>(min(tile0 + t, ntiles - 1));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const size_t ks = max(min(ks0 + r, klast), 0);
        const uint4 x = ld_stream16(reinterpret_cast<const uint4*>(w + (tile * KS + ks) * 1024 + l * 16));
        wf[t][r] = v4i{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<T * R>();  // this wave's activation loads have landed
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= nsteps) break;
      v4i af[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int rc = min(16 * mb + (l & 15), RS - 1);
        af[mb] = *reinterpret_cast<const v4i*>(lds + ((kw * R + r) * RS + rc) * 64 + (swz4(rc, g) << 4));
      }
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          acc[t][mb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[t][r], af[mb], acc[t][mb], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    // All of a turn's weights are waited for here; without this the compiler waits for
    // the next turn's activation loads before it issues that turn's weight loads.  With
    // row_off: 16 experts of 4096x4096, 4 tokens, 20.0 -> 18.7 us; 128 of 512x256 5.7 ->
    // 5.5; 256 of 1024x2048, 32 tokens, 53.9 -> 54.8.  Not for the dense forms: 32 rows
    // +-2%, and 64 rows, whose activation loads are 4 times as many, are better off with
    // those ahead of every wave's weights (N = K = 5120 13.8 -> 15.1 us, K = 17408 28.8
    // -> 33.5).
    if constexpr (GROUPED) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) keep_vgprs(wf[t][r]);
    }
  }

  if (KW > 1) {   // the KW partials of a tile
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
      for (int u = 1; u < KW; ++u)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[t][mb][j] += s_red[(((u - 1) * TW + tw) * kPer + (t * MB + mb) * 4 + j) * 64 + l];
  }
  const bool wide = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.c) % 8 == 0;
  auto store = [&](int t, int mb, v4i v) {
    const int i = 16 * mb + (l & 15), n = (tile0 + t) * 16 + 4 * g;
    if (i >= nrows || n >= p.N) return;
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = scaled(v[j], sa[mb], sw[t][j]);
    const uint2 o{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])};
    uint16_t* dst = p.c + (m0 + i) * p.ldc + n;
    if (wide && n + 4 <= p.N) {
      *reinterpret_cast<uint2*>(dst) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < p.N) dst[j] = static_cast<uint16_t>((j < 2 ? o.x : o.y) >> (16 * (j & 1)));
    }
  };
  const int S = gridDim.z;
  if (GROUPED || S == 1) {
    if (owner)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) store(t, mb, acc[t][mb]);
    return;
  }
  // K splits: partials in fragment order, device-scope, added by the last
  // workgroup of the tile; it leaves its counter at zero.
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
        int* dst = frag(blockIdx.z, t, mb);
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
  int sum[kNV];
  sum_partials<kNV, 64, kU>(sum, frag(0, 0, 0), static_cast<size_t>(gridDim.y) * gridDim.x * (TW * T * MB * 256), S);
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int v = (t * MB + mb) * 4;
      store(t, mb, v4i{sum[v], sum[v + 1], sum[v + 2], sum[v + 3]});
    }
  if (threadIdx.x == 0) __hip_atomic_store(&p.counters[tg], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ========================================================= many rows: LDS tiles
// A workgroup computes a BM x BN tile with WM x WN waves, each (BM/WM) x
// (BN/WN) as 32x32 sub-tiles; first MFMA operand the weight (rows = n), second
// the activation, so a lane holds four consecutive n of one m.
//
// K advances in steps of SUB blocks of 64.  A block's activation codes (BM x 64 B,
// chunks swizzled by swz4) and weight codes (BN/16 fragment blocks of 1 KiB, as
// they are) go global -> LDS by direct loads into one of STAGES buffers, STAGES - 1
// steps ahead.  The steps of a turn round the stages are unrolled, so the stage
// is a constant of the code.
//
// KG > 1: that many groups of WM x WN waves share the tile, each over every
// KG-th step with buffers of its own, and their partial sums are added through
// LDS.  SPLIT: the grid's layers share a tile, each a run of K.  TAIL: K is no multiple
// of 128.
template <int BM, int BN, int WM, int WN, int KG, int STAGES, int SUB>
struct TileCfg {
  static_assert(STAGES >= 2 && STAGES <= 4 && (SUB == 1 || SUB == 2), "the K loop");
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;   // of a group
  static constexpr int kTM = BM / WM / 32, kTN = BN / WN / 32;
  static constexpr int kA = BM * 64, kB = BN * 64, kBlock = kA + kB, kStage = SUB * kBlock;
  static constexpr int kAIters = kA / (kThreads * 16), kBIters = kB / (kThreads * 16);   // loads per 64 of K
  static constexpr int kDma = SUB * (kAIters + kBIters), kHalves = 2 * SUB;
  static constexpr int kDmaFirst = (kDma + kHalves - 1) / kHalves;   // of them, in the half that frees the stage
  static_assert(kA % (kThreads * 16) == 0 && kB % (kThreads * 16) == 0, "");
  static constexpr int kGroup = STAGES * kStage;         // LDS of a group
  static constexpr int kRed = (KG - 1) * BM * BN * 4;    // the other groups' partial tiles
  static constexpr int kEpi = BM * BN * 2;               // the epilogue's tile
  static constexpr int kMain = std::max(KG * kGroup, std::max(kRed, kEpi));
  static constexpr int kScales = (BM + BN) * 4;          // behind it: as of the rows, ws of the columns
  static constexpr int kScalePieces = (BM + BN) / 64, kScaleIters = (kScalePieces + kWaves * KG - 1) / (kWaves * KG);
  static constexpr int kLds = kMain + kScales;
};

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int SUB, int OCC, bool GROUPED, bool TAIL, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN * KG, OCC) void k_w8a8_tile(W8A8Args p, int group_m) {
  using C = TileCfg<BM, BN, WM, WN, KG, STAGES, SUB>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x;
  const int wg_wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int kg = wg_wave / C::kWaves, wave = wg_wave % C::kWaves;
  const int wm = wave / WN, wn = wave % WN;
  const int N = p.N, KS = p.KS, NT = (N + 15) >> 4;
  const int n_tiles = (N + BN - 1) / BN;
  // this group's steps of SUB blocks of K: KG * i + kg for i < n_steps
  // (SPLIT: of the workgroup's run of p.iters of them)
  static_assert(!SPLIT || (KG == 1 && !GROUPED), "K splits");
  const int s0 = SPLIT ? static_cast<int>(blockIdx.z) * p.iters : 0;
  const int SS = SPLIT ? min(p.iters, KS / SUB - s0) : KS / SUB;
  const int n_steps = (SS - kg + KG - 1) / KG, n_turns = (SS + KG - 1) / KG;

  int m0, nrows, nt, tile = 0;
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
    tile = mt * n_tiles + nt;
  }
  const int n0 = nt * BN, nt0 = n0 >> 4;
  uint8_t* const glds = lds + kg * C::kGroup;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(glds));

  // 32-bit source offsets of the loads from the tile's base (rows past the
  // tile's last and columns past N re-read valid ones; their results are not
  // stored).  Chunks past K re-read the row's last one (TAIL).
  const uint8_t* const a = GROUPED ? p.a : p.a + static_cast<size_t>(m0) * p.lda;
  w += (static_cast<size_t>(nt0) * KS + s0 * SUB) * 1024;
  uint32_t aoff[C::kAIters], aend[C::kAIters], boff[C::kBIters];
#pragma unroll
  for (int i = 0; i < C::kAIters; ++i) {
    const int q = (i * C::kWaves + wave) * 64 + l;
    const int row = q >> 2;
    int src = min(row, nrows - 1);
    if constexpr (GROUPED) src = src_row(p, m0 + src);
    aoff[i] = static_cast<uint32_t>(src) * p.lda;
    aend[i] = aoff[i] + static_cast<uint32_t>(p.K - 16);
    aoff[i] += static_cast<uint32_t>(16 * swz4(row, q & 3) + s0 * SUB * 64);
  }
#pragma unroll
  for (int i = 0; i < C::kBIters; ++i)
    boff[i] = static_cast<uint32_t>(min(nt0 + i * C::kWaves + wave, NT - 1) - nt0) * static_cast<uint32_t>(KS) * 1024u +
              static_cast<uint32_t>(l * 16);
  // the i-th load of step ss into stage st
  auto dma_one = [&](int i, int ss, int st) {
    const int sub = i / (C::kAIters + C::kBIters), j = i % (C::kAIters + C::kBIters);
    const int ks = ss * SUB + sub;
    const uint32_t base = lds0 + st * C::kStage + sub * C::kBlock;
    if (j < C::kAIters) {
      const uint32_t dst = base + (j * C::kWaves + wave) * 1024;
      if constexpr (TAIL) dma16(dst, a, min(aoff[j] + static_cast<uint32_t>(ks) * 64u, aend[j]));
      else dma16(dst, a + static_cast<size_t>(ks) * 64, aoff[j]);
    } else {
      dma16(base + C::kA + ((j - C::kAIters) * C::kWaves + wave) * 1024, w + static_cast<size_t>(ks) * 1024,
            boff[j - C::kAIters]);
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
  // LDS read piece i of half h of stage st: weight 0, the activations, the other weights
  auto piece = [&](int st, int h, Frag& f, int i) {
    const uint8_t* base = glds + st * C::kStage + (h >> 1) * C::kBlock;
    if (i == 0 || i > C::kTM) {
      const int t = i == 0 ? 0 : i - C::kTM;
      f.b[t] = *reinterpret_cast<const v4i*>(base + bbase + t * 2048 + (h & 1) * 512);
    } else {
      f.a[i - 1] = *reinterpret_cast<const v4i*>(base + abase[h & 1] + (i - 1) * 2048);
    }
  };
  // MFMAs of half H of the step in stage U.  Between them: the LDS reads of the
  // next half (rf) and a share of a step's loads (the last half: the first of step
  // s + STAGES's, whose stage has just become free; the others: the rest of step
  // s + STAGES - 1's).
  auto half = [&](auto uu, auto hh, const Frag& f, Frag& rf, int dks) {
    constexpr int U = decltype(uu)::value, H = decltype(hh)::value;
    constexpr bool kLast = H == C::kHalves - 1;
    constexpr int kRead = kLast ? (U + 1) % STAGES : U;
    constexpr int kN = C::kTN * C::kTM;
    constexpr int kRest = C::kDma - C::kDmaFirst;
    constexpr int d0 = kLast ? 0 : C::kDmaFirst + H * kRest / (C::kHalves - 1);
    constexpr int d1 = kLast ? C::kDmaFirst : C::kDmaFirst + (H + 1) * kRest / (C::kHalves - 1);
    constexpr int kFill = kLast ? U : (U + STAGES - 1) % STAGES;
#pragma unroll
    for (int n = 0; n < kN || n < kPieces; ++n) {
      if (n < kN) {
        const int i = n / C::kTM, j = n % C::kTM;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[i], f.a[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (n < kPieces) piece(kRead, kLast ? 0 : H + 1, rf, n);
      // the loads, spread evenly over the half's MFMAs
#pragma unroll
      for (int d = d0; d < d1; ++d)
        if ((d - d0) * kN / (d1 - d0) == n) dma_one(d, dks, kFill);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s: all halves but the last; this wave's loads of step s+1 have landed and
  // its LDS reads are done; barrier (s+1 published, the stage of s free); the last
  // half, which reads s+1's first fragments.  So a stage is filled again right behind
  // its last reads and waited for only where it is read, STAGES - 1 steps later.
  // Steps past the end re-load the last one (never used, or the same bytes).
  Frag f0, f1;
  auto step_of = [&](int ls) { return min(KG * min(ls, n_steps - 1) + kg, SS - 1); };
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
      const int next = step_of(ls + STAGES - 1);
      half(uu, Int<0>{}, f0, f1, next);
      if constexpr (SUB > 1) {
        half(uu, Int<1>{}, f1, f0, next);
        half(uu, Int<2>{}, f0, f1, next);
      }
      wait_vm<(STAGES - 2) * C::kDma>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if (KG > 1 && !live) return;
    half(uu, Int<C::kHalves - 1>{}, f1, f0, step_of(ls + STAGES));
  };
  // (with one group, steps past the end are skipped; several groups meet at
  // every barrier, so those run it empty)
  for (int ls = 0; ls < n_turns; ls += STAGES) {
    step(Int<0>{}, ls, ls < n_steps);
    if (ls + 1 < n_turns) step(Int<1>{}, ls + 1, ls + 1 < n_steps);
    if constexpr (STAGES > 2)
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

  // K splits: partial tiles in fragment order through the workspace, as the stream's;
  // the last workgroup of the tile, whose own sums are still in its registers, adds the
  // others' and leaves the counter at zero.  (Whole numbers: any order is the same.)
  if constexpr (SPLIT) {
    __shared__ int s_last;
    constexpr int kPart = C::kTN * C::kTM * 16 * 64;
    const int S = gridDim.z;
    const size_t stride = static_cast<size_t>(gridDim.x) * C::kWaves * kPart;
    int* const mine = p.slab + (static_cast<size_t>(tile) * C::kWaves + wave) * kPart + l;
    {
      int* dst = mine + blockIdx.z * stride;
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            __hip_atomic_store(dst + ((i * C::kTM + j) * 16 + r) * 64, acc[i][j][r], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("" ::: "memory");
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(&p.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == S - 1;
    __syncthreads();
    if (!s_last) return;
    for (int z = 0; z < S; ++z) {
      if (z == static_cast<int>(blockIdx.z)) continue;
      const int* src = mine + z * stride;
      v16i x[C::kTN][C::kTM];
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            x[i][j][r] = __hip_atomic_load(src + ((i * C::kTM + j) * 16 + r) * 64, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int i = 0; i < C::kTN; ++i)
#pragma unroll
        for (int j = 0; j < C::kTM; ++j) acc[i][j] += x[i][j];
    }
    if (tid == 0) __hip_atomic_store(&p.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // Epilogue: the tile through LDS as bf16, so that a row leaves as whole
  // 16-byte pieces side by side.  A lane's four columns are half a piece; piece
  // q of a row sits at slot q ^ (row % swap), within runs of swap pieces.
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __syncthreads();       // the stages are done with
  const float* s_as = reinterpret_cast<const float*>(lds + C::kMain);
  const float* s_ws = s_as + BM;
  constexpr int kLanes = BN / 8, kRows = C::kThreads * KG / kLanes;   // pieces of a row, rows at once
  constexpr int kSwap = kLanes & -kLanes;                             // (a power of two that divides them)
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
          *reinterpret_cast<uint2*>(lds + row * (BN * 2) + (((col >> 3) ^ (row % kSwap)) << 4) + 8 * (l >> 5)) =
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
  if (cols <= 0 || tid >= kRows * kLanes) return;
#pragma unroll 4
  for (int r = tid / kLanes; r < nrows; r += kRows) {
    const uint4 o = *reinterpret_cast<const uint4*>(lds + r * (BN * 2) + ((q ^ (r % kSwap)) << 4));
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
constexpr size_t kMaxStreamLds = 160 * 1024 - 256;
constexpr int kMaxSplits = 65535;   // grid z

struct StreamCfg {
  int mb, tw, kw, t, r;                  // row blocks, waves, tiles and K blocks a wave
  int rs, groups, mtiles, s, iters;      // rows staged, the grid, K runs a workgroup
};
size_t stream_lds(const StreamCfg& d) {
  const size_t slice = (static_cast<size_t>(d.kw) * d.r * d.rs * 4 + 63) / 64 * 1024;
  const size_t red = static_cast<size_t>(d.kw - 1) * d.tw * d.t * d.mb * 4 * 64 * sizeof(int);
  return std::max(slice, red);
}
size_t stream_slab(const StreamCfg& d) {
  return static_cast<size_t>(d.s) * d.mtiles * d.groups * d.tw * d.t * d.mb * 1024;
}

template <int MB, int T, int R, bool LOOP, bool GROUPED>
int launch_stream(const StreamCfg& d, W8A8Args& p, hipStream_t st) {
  const size_t lds = stream_lds(d);
  if (lds > kMaxStreamLds || d.tw * d.kw > 16 || d.mtiles > 65535 || d.s > kMaxSplits) return BS_ERR_SHAPE;
  p.tw = d.tw;
  p.kw = d.kw;
  p.rs = d.rs;
  p.iters = d.iters;
  auto* fn = &k_w8a8_stream<MB, T, R, LOOP, GROUPED>;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(kMaxStreamLds));
  if (attr != hipSuccess) return BS_ERR_LAUNCH;
  fn<<<dim3(d.groups, d.mtiles, d.s), d.tw * d.kw * 64, lds, st>>>(p);
  return bs_launch_status();
}

// rows M as blocks of 16, columns and K cut as (tw, kw, t, r, iters) says
StreamCfg stream_cfg(int M, int N, int KS, int mb, int tw, int kw, int t, int r, int iters) {
  const int run = kw * r * iters;
  return StreamCfg{mb, tw, kw, t, r, M, ((N + 15) / 16 + tw * t - 1) / (tw * t), 1, (KS + run - 1) / run, iters};
}

// The dense stream's cuts, from sweeps over N = 64 .. 34816 and K = 128 .. 17408
// with weights pooled past the last-level cache.
// Up to 16 rows (the choice is 2% behind the best of 22 cuts in the mean of 300
// sizes, at worst 20%): one workgroup covers a K of up to 128 blocks (K = 8192)
// with waves of eight blocks, so nothing goes through the workspace (8 rows N =
// 17408 K = 5120 17.3 us, 5.2 TB/s; in two splits of five waves 19.4); two
// column tiles a wave where 257 to 512 of them would leave a part of a second
// round (N = K = 5120 7.6 against 8.3); short K in waves of four.  Longer K, and
// 9 to 16 rows of many columns, whose slice would fill a CU's LDS alone, in runs
// of four to six waves.
// 17 to 64 rows: K in runs of a loop, so that about 256 to 512 workgroups stay (24
// rows of 42 sizes: 2% behind the best of 45 cuts in the mean, at worst 14%; N = 5120,
// K = 17408 24 us, with longer waves of fewer splits 30; N = 17408, K = 5120 24).
StreamCfg dense_stream_cfg(int M, int N, int KS) {
  const int nt = (N + 15) / 16;
  auto cut = [&](int tw, int t, int r, int kw_max) {
    const int s = (KS + r * kw_max - 1) / (r * kw_max);
    return stream_cfg(M, N, KS, 1, tw, (KS + s * r - 1) / (s * r), t, r, 1);
  };
  if (M <= 16) {
    if (KS <= 8) return cut(2, 1, 4, 4);
    if (KS <= 16) return cut(1, 1, 4, 4);
    if (KS <= 128 && !(M > 8 && nt > 512) && !(KS > 80 && nt <= 32)) return cut(1, nt > 256 && nt <= 512 ? 2 : 1, 8, 16);
    if (nt <= 32) return cut(1, 1, 8, 5);
    return M > 8 && nt >= 256 ? cut(4, 1, 8, 4) : cut(2, 1, 8, 6);
  }
  auto loop = [&](int tw, int r, int kw, int target) {
    kw = std::min(kw, (KS + r - 1) / r);
    const int runs = (KS + kw * r - 1) / (kw * r), groups = (nt + tw - 1) / tw;
    const int s = std::max(1, std::min(runs, target / groups));
    return stream_cfg(M, N, KS, M <= 32 ? 2 : 4, tw, kw, 1, r, (runs + s - 1) / s);
  };
  if (M <= 32) {
    if (KS <= 2) return loop(4, 4, 4, 256);
    if (KS <= 8) return nt <= 512 ? loop(2, 4, 2, 256) : loop(4, 8, 2, 512);
    if (KS <= 32) return nt <= 128 ? loop(1, 4, 8, 256) : (nt <= 256 ? loop(2, 4, 4, 256) : loop(2, 8, 4, 512));
    if (nt > 512) return KS >= 192 ? loop(8, 8, 1, 512) : (nt <= 768 ? loop(2, 4, 2, 1024) : loop(4, 8, 2, 1024));
    if (KS >= 192) return loop(2, 8, 4, 512);
    return nt <= 64 ? loop(2, 4, 4, 512) : loop(2, 8, 4, 256);
  }
  return nt <= 64 ? loop(2, 4, 4, 256) : (nt <= 512 ? loop(4, 4, 4, 256) : loop(8, 8, 1, 512));
}

// Up to 32 rows, and up to 64 of K > 2048 where the tiles' columns are few or K
// is long (64 rows: N = 1024 K = 17408 13.6 us, tiles 42; N = K = 5120 13.4
// against 16.8; N = 17408 K = 5120 29.5 against 28.7, left to the tiles).  A K
// split has a counter for every column group and a grid layer for every run.
bool use_stream(int M, int N, int KS) {
  if (M > 32 && (M > 64 || KS <= 32 || (N > 8192 && KS < 192))) return false;
  const StreamCfg d = dense_stream_cfg(M, N, KS);
  return d.s == 1 || (d.s <= kMaxSplits && d.groups * d.mtiles <= kWsMaxCounters);
}

int run_dense_stream(W8A8Args& p, void* ws, hipStream_t st) {
  const StreamCfg d = dense_stream_cfg(p.M, p.N, p.KS);
  if (d.s > 1) {
    p.counters = static_cast<int*>(ws);
    p.slab = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
  }
#define BS_STREAM(MB_, R_) \
  (d.iters > 1 ? launch_stream<MB_, 1, R_, true, false>(d, p, st) : launch_stream<MB_, 1, R_, false, false>(d, p, st))
  if (d.mb == 1) {
    if (d.r == 4) return launch_stream<1, 1, 4, false, false>(d, p, st);
    return d.t == 2 ? launch_stream<1, 2, 8, false, false>(d, p, st) : launch_stream<1, 1, 8, false, false>(d, p, st);
  }
  if (d.mb == 2) return d.r == 4 ? BS_STREAM(2, 4) : BS_STREAM(2, 8);
  // (eight blocks a wave: 24 runs of K or more over at most seven grid layers, always a loop)
  return d.r == 4 ? BS_STREAM(4, 4) : launch_stream<4, 1, 8, true, false>(d, p, st);
#undef BS_STREAM
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int SUB, int OCC, bool GROUPED>
int launch_tile(const W8A8Args& p, int64_t wgs, hipStream_t st) {
  if (wgs > 0x7FFFFFFF) return BS_ERR_SHAPE;
  const dim3 grid(static_cast<uint32_t>(wgs)), block(64 * WM * WN * KG);
  if (p.K % 128 == 0) k_w8a8_tile<BM, BN, WM, WN, KG, STAGES, SUB, OCC, GROUPED, false, false><<<grid, block, 0, st>>>(p, 4);
  else k_w8a8_tile<BM, BN, WM, WN, KG, STAGES, SUB, OCC, GROUPED, true, false><<<grid, block, 0, st>>>(p, 4);
  return bs_launch_status();
}
// K in runs of p.iters steps, one to a grid layer
template <int BM, int BN, int WM, int WN, int STAGES, int SUB, int OCC>
int launch_split(const W8A8Args& p, int64_t wgs, hipStream_t st) {
  const int steps = p.KS / SUB;
  const dim3 grid(static_cast<uint32_t>(wgs), 1, (steps + p.iters - 1) / p.iters), block(64 * WM * WN);
  if (p.K % 128 == 0) k_w8a8_tile<BM, BN, WM, WN, 1, STAGES, SUB, OCC, false, false, true><<<grid, block, 0, st>>>(p, 4);
  else k_w8a8_tile<BM, BN, WM, WN, 1, STAGES, SUB, OCC, false, true, true><<<grid, block, 0, st>>>(p, 4);
  return bs_launch_status();
}

// The dense tile shapes and what a launch of each takes, in us: with x = tiles
// / 256 (one per CU) and R = ceil(x) rounds,
//   t = start + R * (round + steps * step) + x * steps * load,  steps of 128 of K
// fitted over 20 row counts from 40 to 6000 at twelve N x K, N = 512 .. 34816 and
// K = 256 .. 17408, weights pooled past the last-level cache: by least squares,
// then moved a little, with the K splits' below, to the least loss by the choice: 0.4%
// behind the best in the mean of the 344 sizes of the fit, at worst 13%; on 64 sizes
// left out of it (M = 65 .. 6000, N and K drawn over the same ranges) 2.4% in the mean, at
// worst 23%, 53 of them within 3% (the others mostly K below 1000, where 128 x 256 in
// two workgroups a CU is passed over).  The four shapes with a side of 192 are there
// for the sizes whose tiles would fill little more than half of the CUs' last round
// (1024 rows, N = 10240, K = 5120: 54 us, without them 65; 512 rows 43 and 49; 128
// rows, N = 17408 34 and 40); without them the choice is 2% behind in the mean.
struct TileShape {
  int bm, bn;
  float start, round, step, load;
};
constexpr TileShape kTiles[] = {
    {256, 256, 0.000f, 7.046f, 0.966f, 0.691f},  // 8 waves of 64 x 128
    {128, 256, 1.535f, 2.757f, 0.870f, 0.140f},  // 4 waves of 64 x 128, two workgroups a CU
    {128, 256, 0.081f, 3.969f, 0.778f, 0.215f},  // 8 waves of 64 x 64
    {128, 128, 2.219f, 1.633f, 0.561f, 0.093f},  // 4 waves of 64 x 64, two workgroups a CU
    {64, 128, 2.069f, 0.579f, 0.458f, 0.000f},   // 4 waves of 64 x 32, three workgroups a CU
    {64, 128, 1.673f, 3.132f, 0.376f, 0.000f},   // 2 K groups of 2 waves of 64 x 64
    {64, 64, 2.200f, 0.859f, 0.245f, 0.000f},    // 4 waves of 32 x 32, K steps of 128, two workgroups a CU
    {192, 256, 0.000f, 6.827f, 0.944f, 0.327f},  // 4 waves of 96 x 128
    {192, 128, 2.086f, 2.045f, 0.707f, 0.091f},  // 4 waves of 96 x 64, two workgroups a CU
    {128, 192, 1.066f, 3.426f, 0.601f, 0.166f},  // 4 waves of 64 x 96
    {64, 192, 1.485f, 4.680f, 0.510f, 0.000f},   // 2 K groups of 2 waves of 64 x 96
};
constexpr int kShapes = sizeof(kTiles) / sizeof(kTiles[0]);
int64_t tiles_of(int i, int M, int N) {
  const TileShape& t = kTiles[i];
  return static_cast<int64_t>((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
}
float tile_cost(int i, int M, int N, int steps) {
  const TileShape& t = kTiles[i];
  const float x = static_cast<float>(tiles_of(i, M, N)) / 256.0f;
  return t.start + std::ceil(x) * (t.round + steps * t.step) + x * steps * t.load;
}
int best_tile(int M, int N, int steps) {
  int best = 0;
  for (int i = 1; i < kShapes; ++i)
    if (tile_cost(i, M, N, steps) < tile_cost(best, M, N, steps)) best = i;
  return best;
}

// K splits of four of the shapes, through the workspace, where the tiles are too few
// for the CUs or K is long (M = 128, N = 1024, K = 17408 14.6 us, unsplit 46; N = 5120 33
// and 49): in S runs of `per` steps a launch takes
//   scale * t(S * tiles, per steps) + add + mb * (all partials' MB) + kb * (KB that the
//   last workgroup of a tile adds)
// fitted over eleven row counts from 65 to 1500 at fourteen N x K, K = 2048 .. 17408
// (without splits the choice would be 38% behind the best in the mean of those).
struct SplitCost {
  int shape;
  float scale, add, mb, kb;
};
constexpr SplitCost kSplits[] = {{2, 1.115f, 1.905f, 0.114f, 0.0106f},
                                 {3, 1.022f, 0.750f, 0.135f, 0.0142f},
                                 {4, 0.975f, 1.373f, 0.190f, 0.0197f},
                                 {6, 1.232f, 0.000f, 0.141f, 0.0392f}};
W8A8Plan choose_tile(int M, int N, int steps) {
  W8A8Plan best{false, best_tile(M, N, steps), 0, 0};
  if (steps < 8 || tiles_of(2, M, N) > 400) return best;
  float least = tile_cost(best.shape, M, N, steps);
  for (const SplitCost& c : kSplits) {
    const TileShape& t = kTiles[c.shape];
    const int64_t tiles = tiles_of(c.shape, M, N);
    int last = 0;
    for (int s : {2, 3, 4, 5, 6, 8, 10, 12, 16, 24}) {
      const int per = (steps + s - 1) / s, S = (steps + per - 1) / per;
      if (per < 4 || S * tiles > 800) break;
      if (per == last) continue;
      last = per;
      const float x = static_cast<float>(S * tiles) / 256.0f, kb = static_cast<float>(t.bm * t.bn) * 0.004f;
      const float cost = c.scale * (t.start + std::ceil(x) * (t.round + per * t.step) + x * per * t.load) + c.add +
                         c.mb * kb * 0.001f * static_cast<float>(S * tiles) + c.kb * kb * static_cast<float>(S - 1);
      if (cost < least) {
        least = cost;
        best = W8A8Plan{false, c.shape, per, kWsCounterBytes + static_cast<size_t>(S * tiles) * t.bm * t.bn * sizeof(int)};
      }
    }
  }
  return best;
}
int run_split(const W8A8Plan& c, W8A8Args& p, void* ws, hipStream_t st) {
  p.counters = static_cast<int*>(ws);
  p.slab = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
  p.iters = c.shape == 6 ? c.per : 2 * c.per;   // (steps of 128 there, of 64 else)
  const int64_t wgs = tiles_of(c.shape, p.M, p.N);
  switch (c.shape) {
    case 2: return launch_split<128, 256, 2, 4, 4, 1, 1>(p, wgs, st);
    case 3: return launch_split<128, 128, 2, 2, 4, 1, 2>(p, wgs, st);
    case 4: return launch_split<64, 128, 1, 4, 4, 1, 3>(p, wgs, st);
    default: return launch_split<64, 64, 2, 2, 4, 2, 2>(p, wgs, st);
  }
}

// columns [n0, n1) of the problem as tiles of shape i; n0 is a multiple of 16
int run_tiles(int i, const W8A8Args& q, int n0, int n1, hipStream_t st) {
  W8A8Args p = q;
  p.w += static_cast<size_t>(n0 / 16) * p.KS * 1024;
  p.wsc += n0;
  p.c += n0;
  p.N = n1 - n0;
  const int64_t wgs = tiles_of(i, p.M, p.N);
  switch (i) {
    case 0: return launch_tile<256, 256, 4, 2, 1, 4, 1, 1, false>(p, wgs, st);
    case 1: return launch_tile<128, 256, 2, 2, 1, 3, 1, 2, false>(p, wgs, st);
    case 2: return launch_tile<128, 256, 2, 4, 1, 4, 1, 1, false>(p, wgs, st);
    case 3: return launch_tile<128, 128, 2, 2, 1, 4, 1, 2, false>(p, wgs, st);
    case 4: return launch_tile<64, 128, 1, 4, 1, 4, 1, 3, false>(p, wgs, st);
    case 5: return launch_tile<64, 128, 1, 2, 2, 4, 1, 1, false>(p, wgs, st);
    case 6: return launch_tile<64, 64, 2, 2, 1, 4, 2, 2, false>(p, wgs, st);
    case 7: return launch_tile<192, 256, 2, 2, 1, 3, 1, 1, false>(p, wgs, st);
    case 8: return launch_tile<192, 128, 2, 2, 1, 3, 1, 2, false>(p, wgs, st);
    case 9: return launch_tile<128, 192, 2, 2, 1, 4, 1, 1, false>(p, wgs, st);
    default: return launch_tile<64, 192, 1, 2, 2, 4, 1, 1, false>(p, wgs, st);
  }
}

// One shape for all columns; or, where the large tiles would end in a partial
// round, large tiles over as many columns as whole rounds take and the rest as
// the shape that is quickest there (the second launch costs about 1 us more).
int run_dense_tile(const W8A8Plan& c, W8A8Args& p, void* ws, hipStream_t st) {
  const int steps = p.KS / 2;
  if (c.per > 0) return run_split(c, p, ws, st);
  const int b = c.shape;
  const int64_t mt = (p.M + 255) / 256, nt = (p.N + 255) / 256;
  const int64_t rounds = mt * nt / 256;
  if (rounds >= 1) {
    const int n1 = static_cast<int>(rounds * 256 / mt * 256);   // < N unless the rounds are whole
    if (n1 > 0 && n1 < p.N) {
      const int r = best_tile(p.M, p.N - n1, steps);
      if (tile_cost(0, p.M, n1, steps) + tile_cost(r, p.M, p.N - n1, steps) + 1.0f < tile_cost(b, p.M, p.N, steps)) {
        const int rc = run_tiles(0, p, 0, n1, st);
        return rc != BS_OK ? rc : run_tiles(r, p, n1, p.N, st);
      }
    }
  }
  return run_tiles(b, p, 0, p.N, st);
}

}  // namespace

W8A8Plan bs_w8a8_plan(int M, int N, int K) {
  const int KS = (K + 127) / 128 * 2;
  if (!use_stream(M, N, KS)) return choose_tile(M, N, KS / 2);
  const StreamCfg d = dense_stream_cfg(M, N, KS);
  return W8A8Plan{true, 0, 0, d.s > 1 ? kWsCounterBytes + stream_slab(d) : 0};
}

int bs_launch_w8a8(const uint8_t* a, int64_t lda, const float* as, const uint8_t* w, const float* wsc, uint16_t* c,
                   int64_t ldc, int M, int N, int K, const W8A8Plan& plan, void* ws, hipStream_t st) {
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
  p.KS = (K + 127) / 128 * 2;
  return plan.stream ? run_dense_stream(p, ws, st) : run_dense_tile(plan, p, ws, st);
}

// Row tiles by S / E, the rows an expert would have if they were spread evenly
// (swept at 256, 128, 64, 32, 16 and 8 experts, S / E from 1/32 to 2048, weights
// pooled past the last-level cache; up to 512 tokens with an even load, from 1024
// tokens on with a skewed one, where about half of 256 experts get a row):
//   - less than 16 rows: the weight stream over tiles of 16 rows, waves of eight K
//     blocks.  64 columns a workgroup in two K groups (256 experts N = 1024 K =
//     2048: 128 rows 36 us, 5.9 TB/s; 2048 rows 86 us, tiles 94), 32 in four where
//     the grid is small then (8 rows 7.5 us against 8.3; 64 experts K = 5120 6 rows
//     12.0 against 15.1), one K group up to K = 512; 256 columns for K <= 256 (64
//     experts' 1024 rows of N = 512 6.4 us against 7.2);
//   - few tiles: 64 x 64 (8 experts N = K = 512, 1024 rows 5.2 us, 128 x 256 8);
//   - up to 47 rows: 64 x 128, three workgroups a CU (256 experts N = 1024 K = 2048,
//     32 rows, skewed, 61 us, 128 x 256 69; but 16 rows, even, 102, 128 x 256 95);
//   - else 128 x 256, two workgroups a CU, so one's stores run under the other's
//     MFMAs (256 experts N = 1024 K = 2048, 65536 rows, skewed, 174 us; 256 x 256 190,
//     128 x 128 229); up to K = 256 128 x 128, three a CU (128 experts N = 512, 65536
//     rows, skewed, 27.5 us against 29.8).
// 256 experts N = 1024 K = 2048 with an even load, where all 537 MB of weights are read:
// 8, 16, 32, 64, 128 and 256 rows an expert 88, 104, 103, 100, 113 and 179 us.  The
// shapes were not compared there from 32 rows on.
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
  p.KS = (K + 127) / 128 * 2;
  p.offsets = offsets;
  p.rows = rows;
  p.E = E;
  p.Ma = Ma;
  const int avg = S / E;
  auto wgs = [&](int bm, int bn) { return static_cast<int64_t>(tile_bound(S, E, bm)) * ((N + bn - 1) / bn); };
  if (avg < 16 && tile_bound(S, E, 16) <= 65535) {
    auto cut = [&](int tw, int kw, int t, int r) {
      const int run = kw * r;
      return StreamCfg{1, tw, kw, t, r, 16, ((N + 15) / 16 + tw * t - 1) / (tw * t), tile_bound(S, E, 16),
                       1, (p.KS + run - 1) / run};
    };
    if (p.KS <= 4) return launch_stream<1, 2, 4, true, true>(cut(8, 1, 2, 4), p, st);
    if (p.KS <= 8) return launch_stream<1, 1, 8, true, true>(cut(4, 1, 1, 8), p, st);
    if (p.KS > 16 && wgs(16, 64) <= 512) return launch_stream<1, 1, 8, true, true>(cut(2, 4, 1, 8), p, st);
    return launch_stream<1, 1, 8, true, true>(cut(4, 2, 1, 8), p, st);
  }
  if (wgs(64, 64) <= 512) return launch_tile<64, 64, 2, 2, 1, 4, 2, 2, true>(p, wgs(64, 64), st);
  if (avg < 48) return launch_tile<64, 128, 1, 4, 1, 4, 1, 3, true>(p, wgs(64, 128), st);
  if (p.KS <= 4) return launch_tile<128, 128, 2, 2, 1, 3, 1, 3, true>(p, wgs(128, 128), st);
  return launch_tile<128, 256, 2, 2, 1, 3, 1, 2, true>(p, wgs(128, 256), st);
}
