// Token routing of a mixture of experts: the (token, expert) pairs sorted by
// expert, token rows gathered in that order, the experts' rows combined back
// with their weights, and the gradient of that.
//
// Pair p = t * k + j is token t's j-th choice.  A stable counting sort by
// expert id gives every kept pair a slot; pairs whose id is outside [0, E)
// take no slot (pos = -1).  Everything is deterministic: counts do not depend
// on the order in which they are added up, ranks come from lane masks, and
// every sum runs in the order of j.
#include <algorithm>

#include "common.h"

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = 1024;
// Up to kOneBlockPairs one workgroup sorts the batch (E = 256: 3.6 us at 64
// pairs, 8.0 at 4096, 12.5 at 8192, where two launches of four workgroups take
// 8.6).  Beyond that a workgroup takes kBlockPairs, or as many as leave
// kMaxBlocks workgroups, since each of them reads all the others' counts
// (65536 pairs: 1024 a workgroup 9.3 us, 2048 9.5, 4096 11.4; 262144: 15.1,
// 12.4, 13.1).
constexpr int kOneBlockPairs = 4096;
constexpr int kBlockPairs = 2048;
constexpr int kMaxBlocks = 128;

int sort_chunk(int P) {
  if (P <= kOneBlockPairs) return P;
  return std::max(kBlockPairs, ((P + kMaxBlocks - 1) / kMaxBlocks + 1023) / 1024 * 1024);
}
int sort_blocks(int P) {
  const int c = sort_chunk(P);
  return (P + c - 1) / c;
}

// pairs of this wave: the workgroup's run in equal parts of whole 64s
struct Run {
  int begin, end;
};
BS_INLINE Run wave_run(int P, int chunk, int wave, int waves) {
  const int b0 = blockIdx.x * chunk, b1 = min(b0 + chunk, P);
  const int per = ((b1 - b0 + waves - 1) / waves + 63) & ~63;
  const int begin = min(b0 + wave * per, b1);
  return Run{begin, min(begin + per, b1)};
}

// counts of each workgroup's pairs: hist[block][E]
__global__ __launch_bounds__(kSortThreads) void k_moe_count(const int* __restrict__ ids, int* __restrict__ hist, int P,
                                                            int E, int chunk) {
  __shared__ int cnt[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int b0 = blockIdx.x * chunk, b1 = min(b0 + chunk, P);
  for (int p = b0 + threadIdx.x; p < b1; p += kSortThreads) {
    const int id = ids[p];
    if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[static_cast<size_t>(blockIdx.x) * E + e] = cnt[e];
}

// LDS accesses of one wave run in program order; this keeps the compiler from
// moving them.
BS_INLINE void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The sort: per-wave counts of the workgroup's own pairs, the experts' starts
// (from hist where there are several workgroups, whose counts all of them add
// up), then every wave places its pairs 64 at a time: a lane's rank among the
// lanes of its expert comes from one ballot per id bit.
// Dynamic LDS: counts [waves][E], totals [E], counts of earlier workgroups [E].
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(const int* __restrict__ ids, const int* __restrict__ hist,
                                                           int* __restrict__ rows, int* __restrict__ pos,
                                                           int* __restrict__ offsets, int P, int k, int E, int chunk,
                                                           int id_bits) {
  extern __shared__ int lds[];
  const int waves = blockDim.x >> 6;
  int* cnt = lds;                // [waves][E]: counts, then the wave's next slot
  int* tot = lds + waves * E;    // [E]: pairs of the expert, then its start
  int* pre = tot + E;            // [E]: of those, in earlier workgroups
  __shared__ int kept_total;
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  for (int i = threadIdx.x; i < (waves + 2) * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const Run r = wave_run(P, chunk, wave, waves);
  for (int p = r.begin + l; p < r.end; p += 64) {
    const int id = ids[p];
    if (id >= 0 && id < E) atomicAdd(&cnt[wave * E + id], 1);
  }
  if (hist != nullptr) {
    // the workgroups' counts, `parts` threads to an expert, four loads at once
    // (one thread per expert, a load at a time, took half the kernel)
    const int nb = gridDim.x, me = blockIdx.x, parts = max(1, static_cast<int>(blockDim.x) / E);
    for (int i = threadIdx.x; i < E * parts; i += blockDim.x) {
      const int e = i % E;
      int all = 0, run = 0;
      for (int b0 = i / E; b0 < nb; b0 += 4 * parts) {
        int c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) c[u] = hist[static_cast<size_t>(min(b0 + u * parts, nb - 1)) * E + e];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int b = b0 + u * parts;
          all += b < nb ? c[u] : 0;
          run += b < me ? c[u] : 0;
        }
      }
      atomicAdd(&tot[e], all);
      atomicAdd(&pre[e], run);
    }
  }
  __syncthreads();
  // cnt[w][e] := pairs of e in earlier workgroups and earlier waves of this one
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int run = pre[e];
    for (int w = 0; w < waves; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    if (hist == nullptr) tot[e] = run;
  }
  __syncthreads();
  if (wave == 0) {   // exclusive scan of tot: each lane a run of experts
    const int per = (E + 63) >> 6;
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += l * per + i < E ? tot[l * per + i] : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      incl += l >= o ? v : 0;
    }
    int at = incl - mine;
    for (int i = 0; i < per; ++i) {
      const int e = l * per + i;
      if (e < E) {
        const int c = tot[e];
        tot[e] = at;
        if (blockIdx.x == 0) offsets[e] = at;
        at += c;
      }
    }
    if (l == 63) {
      kept_total = incl;
      if (blockIdx.x == 0) offsets[E] = incl;
    }
  }
  __syncthreads();
  int next = r.begin + l < r.end ? ids[r.begin + l] : -1;
  for (int p0 = r.begin; p0 < r.end; p0 += 64) {
    const int p = p0 + l, id = next;
    next = p + 64 < r.end ? ids[p + 64] : -1;   // loaded under these ballots
    const bool keep = id >= 0 && id < E;
    unsigned long long same = __ballot(keep);
    for (int b = 0; b < id_bits; ++b) {
      const unsigned long long m = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? m : ~m;
    }
    if (keep) {
      const int rank = __popcll(same & ((1ull << l) - 1));
      const int slot = tot[id] + cnt[wave * E + id] + rank;
      // (counts overwritten by another call that shares ws unordered name no slot outside)
      if (static_cast<unsigned>(slot) < static_cast<unsigned>(P)) rows[slot] = p / k;
      pos[p] = slot;
      wave_lds_fence();   // every lane has read its count
      if ((same >> l) == 1) cnt[wave * E + id] += rank + 1;   // the expert's last lane
    } else if (p < r.end) {
      pos[p] = -1;
    }
    wave_lds_fence();
  }
  // slots that no pair takes
  const int b1 = min(static_cast<int>(blockIdx.x + 1) * chunk, P);
  for (int s = max(kept_total, static_cast<int>(blockIdx.x) * chunk) + threadIdx.x; s < b1; s += blockDim.x)
    rows[s] = -1;
}

// ------------------------------------------------------------------ row moves
// A thread owns 8 columns (16 bytes) of a token: chunk c of nch.
constexpr int kRT = 256;

// xs[pos[t, j]] = x[t]: the token's row is read once and written k times (8192
// tokens x 8 rows of 2048 52 us, 302 MB at 5.8 TB/s; without the streaming hint
// on the stores 60).
__global__ __launch_bounds__(kRT) void k_moe_gather(const uint4* __restrict__ x, const int* __restrict__ pos,
                                                    uint4* __restrict__ xs, uint32_t total, uint32_t nch, int k, int P) {
  const uint32_t i = blockIdx.x * kRT + threadIdx.x;
  if (i >= total) return;
  const uint32_t t = i / nch, c = i - t * nch;
  const uint4 v = x[i];
  const int* pt = pos + static_cast<size_t>(t) * k;
  for (int j = 0; j < k; ++j) {
    const int s = pt[j];
    if (s >= 0 && s < P) st_stream16(xs + static_cast<size_t>(s) * nch + c, v);
  }
}

// Expert rows whose loads are in flight together.  The gradient holds two
// addresses a row as well, in scalar registers: eight rows spill them (8192
// tokens x 8 rows of 2048: 107 us with four, 570 MB at 5.3 TB/s; 108 with eight;
// 2 rows of 5120: 68 and 72).
constexpr int kJ = 8, kJb = 4;

BS_INLINE void unpack_row(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// out[t] = sum_j w[t, j] * y[pos[t, j]], fp32, in the order of j; one rounding.
// Bound by HBM: 8192 tokens x 8 rows of 2048 53 us, 302 MB at 5.7 TB/s.
// A dropped pair's load goes to row 0 and is not added (its row may hold
// anything, NaN too).
template <bool WEIGHTED>
__global__ __launch_bounds__(kRT) void k_moe_combine(const uint4* __restrict__ y, const int* __restrict__ pos,
                                                     const float* __restrict__ w, uint4* __restrict__ out,
                                                     uint32_t total, uint32_t nch, int k, int P) {
  const uint32_t i = blockIdx.x * kRT + threadIdx.x;
  if (i >= total) return;
  const uint32_t t = i / nch, c = i - t * nch;
  const size_t p0 = static_cast<size_t>(t) * k;
  float acc[8] = {};
  for (int j0 = 0; j0 < k; j0 += kJ) {
    int s[kJ];
    float wj[kJ];
    uint4 v[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const size_t p = p0 + min(j0 + j, k - 1);
      s[j] = pos[p];
      wj[j] = WEIGHTED ? w[p] : 1.0f;
      if (j0 + j >= k || s[j] >= P) s[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (j0 + j < k) v[j] = ld_stream16(y + static_cast<size_t>(max(s[j], 0)) * nch + c);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (j0 + j >= k) break;
      float f[8];
      unpack_row(v[j], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = s[j] >= 0 ? fmaf(wj[j], f[q], acc[q]) : acc[q];
    }
  }
  out[i] = make_uint4(bf16x2_rne(acc[0], acc[1]), bf16x2_rne(acc[2], acc[3]), bf16x2_rne(acc[4], acc[5]),
                      bf16x2_rne(acc[6], acc[7]));
}

// dy[pos[t, j]] = w[t, j] * dout[t] and dw[t, j] = <dout[t], y[pos[t, j]]>.
// W waves share a token's columns (W = 1: four tokens to a workgroup); a lane's
// part of the dot product runs over its chunks in order, then the lanes and the
// waves are added in a fixed order.
template <int W>
__global__ __launch_bounds__(kRT) void k_moe_combine_bwd(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                                                         const int* __restrict__ pos, const float* __restrict__ w,
                                                         uint4* __restrict__ dy, float* __restrict__ dw, int T,
                                                         int nch, int k, int P) {
  static_assert(W == 1 || W == kRT / 64, "");
  __shared__ float part[W][kJb];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int t = W == 1 ? blockIdx.x * (kRT / 64) + wave : blockIdx.x;
  if (t >= T) return;
  const size_t p0 = static_cast<size_t>(t) * k;
  const uint4* drow = dout + static_cast<size_t>(t) * nch;
  for (int j0 = 0; j0 < k; j0 += kJb) {
    int s[kJb];
    float wj[kJb], dot[kJb];
#pragma unroll
    for (int j = 0; j < kJb; ++j) {
      const size_t p = p0 + min(j0 + j, k - 1);
      s[j] = pos[p];
      wj[j] = w[p];
      dot[j] = 0.0f;
      if (j0 + j >= k || s[j] >= P) s[j] = -1;
    }
    for (int c = W == 1 ? l : static_cast<int>(threadIdx.x); c < nch; c += 64 * W) {
      const uint4 dv = drow[c];
      uint4 v[kJb];
#pragma unroll
      for (int j = 0; j < kJb; ++j)
        if (j0 + j < k) v[j] = ld_stream16(y + static_cast<size_t>(max(s[j], 0)) * nch + c);
      float d[8];
      unpack_row(dv, d);
#pragma unroll
      for (int j = 0; j < kJb; ++j) {
        if (j0 + j >= k) break;
        float f[8];
        unpack_row(v[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) dot[j] = fmaf(d[q], f[q], dot[j]);
        if (s[j] >= 0)
          st_stream16(dy + static_cast<size_t>(s[j]) * nch + c,
                      make_uint4(bf16x2_rne(d[0] * wj[j], d[1] * wj[j]), bf16x2_rne(d[2] * wj[j], d[3] * wj[j]),
                                 bf16x2_rne(d[4] * wj[j], d[5] * wj[j]), bf16x2_rne(d[6] * wj[j], d[7] * wj[j])));
      }
    }
#pragma unroll
    for (int j = 0; j < kJb; ++j) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
    }
    if constexpr (W > 1) {
      if (j0) __syncthreads();   // part is read below
      if (l == 0)
#pragma unroll
        for (int j = 0; j < kJb; ++j) part[wave][j] = dot[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kJb; ++j) {
        dot[j] = part[0][j];
#pragma unroll
        for (int v = 1; v < W; ++v) dot[j] += part[v][j];
      }
    }
    if (W == 1 ? l == 0 : threadIdx.x == 0)
#pragma unroll
      for (int j = 0; j < kJb; ++j)
        if (j0 + j < k) dw[p0 + j0 + j] = s[j] >= 0 ? dot[j] : 0.0f;
  }
}

// Sizes the routing kernels index with 32 bits: pairs, and 8-column chunks of
// the token rows.
bool sizes_ok(int T, int k, int K) {
  return T >= 1 && k >= 1 && static_cast<int64_t>(T) * k <= (1 << 24) && K >= 8 && K % 8 == 0 && K <= 32768 &&
         static_cast<int64_t>(T) * (K / 8) < (1ll << 31);
}

}  // namespace

size_t bs_moe_sort_workspace(int T, int k, int E) {
  if (T < 1 || k < 1 || static_cast<int64_t>(T) * k > (1 << 24) || E < 1 || E > kMaxExperts) return 0;
  const int nb = sort_blocks(T * k);
  return nb > 1 ? kWsCounterBytes + static_cast<size_t>(nb) * E * sizeof(int) : 0;
}

extern "C" {

BS_API int moe_sort(const int32_t* ids, int32_t* rows, int32_t* pos, int32_t* offsets, int T, int k, int E, void* ws,
                    size_t ws_bytes, bs_stream_t stream) {
  BS_CHECK(T >= 0 && k >= 1 && E >= 1 && E <= kMaxExperts && static_cast<int64_t>(T) * k <= (1 << 24), BS_ERR_SHAPE);
  BS_CHECK(offsets && (T == 0 || (ids && rows && pos)), BS_ERR_NULL);
  BS_CHECK(bs_aligned(ids, 4) && bs_aligned(rows, 4) && bs_aligned(pos, 4) && bs_aligned(offsets, 4), BS_ERR_ALIGN);
  const int P = T * k, chunk = sort_chunk(P), nb = P ? sort_blocks(P) : 1;
  hipStream_t st = static_cast<hipStream_t>(stream);
  int* hist = nullptr;
  if (nb > 1) {
    BS_CHECK(ws && ws_bytes >= bs_moe_sort_workspace(T, k, E), BS_ERR_WORKSPACE);
    BS_CHECK(bs_aligned(ws, 256), BS_ERR_ALIGN);
    hist = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
    k_moe_count<<<nb, kSortThreads, 0, st>>>(ids, hist, P, E, chunk);
  }
  // small batches: no more waves than there are 64s of pairs, but four for the
  // passes over the experts
  const int waves = std::max(4, std::min(kSortWaves, (std::min(P, chunk) + 63) / 64));
  int id_bits = 0;
  while ((1 << id_bits) < E) ++id_bits;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&k_moe_sort), hipFuncAttributeMaxDynamicSharedMemorySize,
                          (kSortWaves + 2) * kMaxExperts * static_cast<int>(sizeof(int)));
  if (attr != hipSuccess) return BS_ERR_LAUNCH;
  k_moe_sort<<<nb, 64 * waves, static_cast<size_t>(waves + 2) * E * sizeof(int), st>>>(ids, hist, rows, pos, offsets,
                                                                                      P, k, E, chunk, id_bits);
  return bs_launch_status();
}

BS_API int moe_gather(const void* x, const int32_t* pos, void* xs, int T, int k, int K, bs_stream_t stream) {
  if (T == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(x && pos && xs, BS_ERR_NULL);
  BS_CHECK(sizes_ok(T, k, K), BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(x, 16) && bs_aligned(xs, 16) && bs_aligned(pos, 4), BS_ERR_ALIGN);
  const uint32_t nch = K / 8, total = static_cast<uint32_t>(T) * nch;
  k_moe_gather<<<(total + kRT - 1) / kRT, kRT, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint4*>(x), pos, static_cast<uint4*>(xs), total, nch, k, T * k);
  return bs_launch_status();
}

BS_API int moe_combine(const void* y, const int32_t* pos, const float* weights, void* out, int T, int k, int K,
                       bs_stream_t stream) {
  if (T == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(y && pos && out, BS_ERR_NULL);
  BS_CHECK(sizes_ok(T, k, K), BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(y, 16) && bs_aligned(out, 16) && bs_aligned(pos, 4) && bs_aligned(weights, 4), BS_ERR_ALIGN);
  const uint32_t nch = K / 8, total = static_cast<uint32_t>(T) * nch;
  const dim3 grid((total + kRT - 1) / kRT);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint4* yp = static_cast<const uint4*>(y);
  uint4* op = static_cast<uint4*>(out);
  if (weights) k_moe_combine<true><<<grid, kRT, 0, st>>>(yp, pos, weights, op, total, nch, k, T * k);
  else k_moe_combine<false><<<grid, kRT, 0, st>>>(yp, pos, weights, op, total, nch, k, T * k);
  return bs_launch_status();
}

BS_API int moe_combine_backward(const void* dout, const void* y, const int32_t* pos, const float* weights, void* dy,
                                float* dweights, int T, int k, int K, bs_stream_t stream) {
  if (T == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(dout && y && pos && weights && dy && dweights, BS_ERR_NULL);
  BS_CHECK(sizes_ok(T, k, K), BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(dout, 16) && bs_aligned(y, 16) && bs_aligned(dy, 16) && bs_aligned(pos, 4) &&
               bs_aligned(weights, 4) && bs_aligned(dweights, 4),
           BS_ERR_ALIGN);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint4 *dp = static_cast<const uint4*>(dout), *yp = static_cast<const uint4*>(y);
  uint4* dyp = static_cast<uint4*>(dy);
  // up to 1024 columns a wave takes a token alone (9 rows of 1024: 64 us against
  // 74; one row of 64: 7 against 40; 8 rows of 2048: 126 against 107)
  if (K <= 1024) k_moe_combine_bwd<1><<<(T + 3) / 4, kRT, 0, st>>>(dp, yp, pos, weights, dyp, dweights, T, K / 8, k, T * k);
  else k_moe_combine_bwd<4><<<T, kRT, 0, st>>>(dp, yp, pos, weights, dyp, dweights, T, K / 8, k, T * k);
  return bs_launch_status();
}

}  // extern "C"
