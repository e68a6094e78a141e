// bwd_tc.cuh — attention's backward on the tensor cores, bf16 in and out: of
// the full-precision bf16 attention (binattn_ref_bf16_backward) and of the
// binary one (binattn_backward_bf16).
//
// With L_ij = c <q_i, k_j> + bias[h,i,j] (binary: c alpha_q_i alpha_k_j S_ij +
// bias) and P = softmax_j(L):
//   dP = dO V^T,  D_i = sum_j P_ij dP_ij,  dL = P (dP - D)
//   dV = P^T dO,  dQ = c dL K,  dK = c dL^T Q,  dbias = sum_b dL.
// P is never written out: each kernel computes it again from the scores and the
// row's log-sum-exp.
//  - rows_kernel: one CTA per 128 query rows, twice over the keys. First pass:
//    the online max m and sum l of the row's softmax and the rescaled sum of
//    exp(.) dP, joined into LSE_i and D_i (fp32, written for the other two).
//    Second pass: dL, rounded to bf16, times K into dQ.
//  - cols_kernel: one CTA per 128 keys, once over the query rows: P^T and
//    dL^T, rounded to bf16, times dO and Q into dV and dK.
//  - dbias_kernel: one CTA per 128 query rows of one head, over the keys with
//    the batch innermost: dL summed over b in fp32 registers, rounded once.
// Every sum has one owner and one order, so there are no atomics and the same
// call gives the same bits. The price against one kernel that adds dQ with
// atomics is two more score products and exps.
//
// The three share one machine. The streamed operand (K and V, or Q and dO) comes
// in tiles of 64 rows by TMA into a ring of stages, as 64-channel panels of
// 128-byte swizzled rows: one panel serves both as the K-major operand of the
// score products and as the MN-major operand of the gradient products. The
// kept operand (128 rows) sits in tensor memory. Scores and dP of a tile are
// two 128 x 64 fp32 accumulators in one of two tensor-memory buffers; P or dL
// goes back as bf16 over its own half of the scores. 16 compute warps: eight
// per buffer (tiles alternate), four per 32-column half, one thread per row.
// LSE and D are known before any exp of the second pass, so threads need
// nothing of one another inside a tile. Warp 16 issues the MMAs, warp 17 the
// copies. Bounded waits as in fwd_tc2.cuh.
//
// Rounding: P, dL (binary: dL times the alpha of the summed side) and the
// results to bf16, half a step each; all else fp32.
#pragma once
#include <algorithm>
#include <atomic>
#include <cstring>
#include <string>

#include "fwd_tc.cuh"
#include "fwd_tc2.cuh"

namespace binattn {
namespace bt {

using namespace sm100;
using tc2::kLog2e;
using tc2::max3f;
using tc2::named_sync;

constexpr int kRows = 128;               // kept rows per CTA (MMA M, TMEM lanes)
constexpr int kCols = 64;                // streamed rows per tile (score MMA N)
constexpr int kComputeWarps = 16;
constexpr int kMmaWarp = 16, kTmaWarp = 17;
constexpr int kThreads = 18 * 32;
constexpr int kCompute = kComputeWarps * 32;
constexpr int kPanel = kCols * 128;      // bytes: 64 rows x 64 channels bf16
constexpr int kBiasBytes = kRows * kCols * 2;
constexpr int kVecBytes = 1024;          // per stage: up to four vectors of 64 floats
constexpr int kBar = 1;                  // named barrier of the compute warps
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const uint16_t* a0;  // kept operands [B,H,N,d]: q and dO (rows, dbias), k and v (cols)
  const uint16_t* a1;
  const float* aq;     // binary: c alpha_q (times log2 e without a bias), padded [BH][Npad]
  const float* ak;     // binary: alpha_k, padded [BH][Npad]
  float cs;            // bf16: factor of the scores (times log2 e without a bias)
  float out;           // factor of dQ (rows) or dK (cols)
  float* lse;          // [BH][Npad]: what logits are taken relative to (see exp2v)
  float* l2;           // [BH][Npad]: with a bias, log2 of the row's sum
  float* D;            // [BH][Npad]
  uint16_t* g0;        // rows: dQ; cols: dV; dbias: dbias
  uint16_t* g1;        // cols: dK
  float* part;         // dbias: fp32 partial sums [nsplit][H][N][N]
  int B, H, N, d, Npad, items;
  int nb, nchunks, nsplit, jsplit;  // dbias
};

// Operand descriptor of 128-byte swizzled rows (8-row groups sbo = 1024 bytes
// apart; MN-major: 64-element panels lbo apart).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// D[128 x 64] = A[128 x ch16 * 16] B[64 x ...]^T: A in tensor memory (bf16
// pairs, 8 columns per 16 channels) or shared memory (128-row panels), B a
// 64-row tile.
template <bool kSS>
__device__ __forceinline__ void issue_scores(uint32_t d_col, uint32_t a, uint32_t b, int ch16) {
  constexpr uint32_t id = idesc_bf16(kRows, kCols, false);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= ch16) break;
    const uint64_t bd = desc_sw128(b + (k >> 2) * kPanel + (k & 3) * 32, 16);
    if constexpr (kSS) mma_ss_warp(d_col, desc_sw128(a + (k >> 2) * 2 * kPanel + (k & 3) * 32, 16), bd, id, k > 0);
    else mma_ts_warp(d_col, a + k * 8, bd, id, k > 0);
  }
}
// D[128 x DP] += A[128 x 64] B[64 x DP]: A bf16 pairs in tensor memory, its two
// 32-column halves 32 columns apart; B a 64-row tile, channels along N.
__device__ __forceinline__ void issue_grad(uint32_t d_col, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    mma_ts_warp(d_col, a + (k >> 1) * 32 + (k & 1) * 8, desc_sw128(b + k * 2048, kPanel), id, accumulate || k > 0);
}

// Thread r's row of a kept operand into its TMEM lane as bf16 pairs, channels
// >= d and rows that are not valid as zeros.
__device__ __forceinline__ void stage_row(const uint16_t* row, bool valid, int d, int DP, uint32_t col) {
  for (int c = 0; c < DP; c += 16) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (valid && c + 8 * e < d) v = __ldg(reinterpret_cast<const uint4*>(row + c + 8 * e));
      w[4 * e] = v.x; w[4 * e + 1] = v.y; w[4 * e + 2] = v.z; w[4 * e + 3] = v.w;
    }
    tmem_st8(col + c / 2, w);
  }
}

// 32 TMEM columns of fp32 times f, as bf16, to row[c0 .. c0 + 32) below d.
__device__ __forceinline__ void store_row(uint32_t col, float f, uint16_t* row, bool valid, int c0, int d) {
  uint32_t v[32];
  tmem_ld32(col + c0, v);
  tmem_ld_wait();
  if (!valid) return;
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    if (c0 + e < d) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_bf16x2(__uint_as_float(v[e + 2 * k]) * f, __uint_as_float(v[e + 2 * k + 1]) * f);
      *reinterpret_cast<uint4*>(row + c0 + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Pair e of a tile's 16-byte bias units: bf16 pairs widened.
__device__ __forceinline__ float2 widen(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Logits of kN columns in place. Without a bias they are in log2 units (the
// factor log2 e is in ci), with one in natural units, so that a bias of the
// type's lowest value does not overflow. bias: the thread's columns as packed
// pairs; ak: the columns' alpha_k (binary).
template <bool kBin, bool kBias, int kN>
__device__ __forceinline__ void logits(uint32_t* s, const float* ak, float ci, const uint32_t* bias) {
  float2* x = reinterpret_cast<float2*>(s);
  const float2 c2 = make_float2(ci, ci);
#pragma unroll
  for (int e = 0; e < kN / 2; e += 2) {
    if constexpr (kBin) {
      const float4 a = *reinterpret_cast<const float4*>(ak + 2 * e);
      x[e] = __fmul2_rn(x[e], make_float2(a.x, a.y));
      x[e + 1] = __fmul2_rn(x[e + 1], make_float2(a.z, a.w));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      x[e + u] = kBias ? __ffma2_rn(x[e + u], c2, widen(bias[e + u])) : __fmul2_rn(x[e + u], c2);
  }
}
// exp of x minus `top`, x in the units of logits(). Without a bias, top is the
// max or the log-sum-exp. With one, a row may consist of masked logits of
// -1e9 or the type's lowest value, where max + log(sum) would lose the sum: top
// is the max, and the (log2 of the) sum is taken off after the subtraction, in
// the multiply-add that changes the units.
template <bool kBias>
__device__ __forceinline__ float2 exp2v(float2 x, float2 minus_top, float2 minus_l2 = make_float2(0.f, 0.f)) {
  float2 y = __fadd2_rn(x, minus_top);
  if constexpr (kBias) y = __ffma2_rn(y, make_float2(kLog2e, kLog2e), minus_l2);
  return make_float2(ex2(y.x), ex2(y.y));
}

// Shared memory: the stages, then (cols, kSS) the kept operands, then scratch.
struct Map {
  int tile, vec, stage, kept, scratch, bars, bytes;
};
__host__ __device__ inline Map smem_map(int d, bool bias, int stages, bool kept, int scratch) {
  Map m;
  const int np = d > 64 ? 2 : 1;
  m.tile = np * kPanel;                                // one streamed matrix
  m.vec = 2 * m.tile + (bias ? kBiasBytes : 0);        // vectors, after both and the bias
  m.stage = m.vec + kVecBytes;
  m.kept = stages * m.stage;
  m.scratch = m.kept + (kept ? 4 * m.tile : 0);
  m.bars = m.scratch + scratch;
  m.bytes = m.bars + 256;
  return m;
}
constexpr int kMinSmem = 120 * 1024;  // one CTA per SM: each holds all of its tensor memory

struct Bars {
  uint64_t *full, *empty, *s_full, *p_full, *a_ready, *o_done, *kept, *drain;
  uint32_t* tmem;
  volatile int* abort;
  __device__ explicit Bars(uint8_t* p) {
    uint64_t* b = reinterpret_cast<uint64_t*>(p);
    full = b;            // [4] a stage's copies landed
    empty = b + 4;       // [4] every reader is done with the stage
    s_full = b + 8;      // [2] scores and dP of the buffer's tile
    p_full = b + 10;     // [2] the 256 threads of the buffer are done with it (and wrote P / dL)
    a_ready = b + 12;    // kept operands staged, accumulators read (512 threads)
    o_done = b + 13;     // the item's last MMA
    kept = b + 14;       // kept operands in shared memory landed
    drain = b + 15;
    tmem = reinterpret_cast<uint32_t*>(b + 16);
    abort = reinterpret_cast<volatile int*>(b + 17);
  }
  __device__ void init() {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kCompute / 2);
    }
    mbar_init(a_ready, kCompute);
    mbar_init(o_done, 1);
    mbar_init(kept, 1);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
};

// This warp's index, known to be the same in all its lanes: branches on it stay
// uniform, so the issuing warp's operands live in uniform registers (measured:
// the ten score products of a tile issue in 390 cycles instead of 665).
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

// A bounded wait of a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Common start and end of the kernels.
__device__ __forceinline__ uint32_t begin(Bars& b, int warp) {
  if (threadIdx.x == 0) b.init();
  if (warp == kMmaWarp) {
    tmem_alloc(b.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  return *b.tmem;
}
__device__ __forceinline__ void end(uint32_t tmem, int warp) {
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
// The copying thread's last act: its `issued` copies have all landed (bounded).
__device__ __forceinline__ void settle(Bars& b, int issued, int stages) {
  volatile int never = 0;
  for (int g = issued > stages ? issued - stages : 0; g < issued; ++g)
    mbar_wait(&b.full[g % stages], (g / stages) & 1, &never);
}
__device__ __forceinline__ void drain_mma(Bars& b) {
  mma_commit_warp(b.drain);
  volatile int never = 0;
  mbar_wait(b.drain, 0, &never);
}

// Tensor memory of rows_kernel and dbias_kernel; cols_kernel sets its own
// accumulator columns.
constexpr int kBuf = 128;         // columns per buffer: scores [0, 64), dP [64, 128)
constexpr int kAcc = 256;
constexpr int kRowsQ = 384, kRowsDO = 448;
constexpr int kRowStages = 4;
constexpr int kRowsScratch = 3 * 4 * kRows * 4;   // [m, l, sum][warpgroup][row] floats
constexpr int kDbiasScratch = 4 * 4 * kRows * 4;  // [LSE, D, factor, log2 sum][batch entry][row]

template <bool kBin, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
rows_kernel(const Params p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_bias) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kS = kRowStages;
  const Map mp = smem_map(p.d, kBias, kS, false, kRowsScratch);
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, np = d > 64 ? 2 : 1;
  const int nkt = (N + kCols - 1) / kCols, T = 2 * nkt;
  const int nit = (N + kRows - 1) / kRows;
  const int G = static_cast<int>(gridDim.x);
  const int n_items = (p.items - static_cast<int>(blockIdx.x) + G - 1) / G;
  // items: the batch fastest, so that CTAs that share a bias tile run side by side
  auto item = [&](int it, int& bh, int& h, int& i0) {
    const int w = static_cast<int>(blockIdx.x) + it * G;
    const int b = w % p.B, qt = (w / p.B) % nit;
    h = w / (p.B * nit);
    bh = b * p.H + h;
    i0 = qt * kRows;
  };
  const uint32_t tmem = begin(bar, warp);

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      const uint32_t bytes = 2u * mp.tile + (kBias ? kBiasBytes : 0) + (kBin ? kCols * 4 : 0);
      for (int it = 0; ok && it < n_items; ++it) {
        int bh, h, i0;
        item(it, bh, h, i0);
        for (int t = 0; t < T; ++t, ++g) {
          const int s = g % kS, j0 = (t < nkt ? t : t - nkt) * kCols;
          if (g >= kS && !(ok = mbar_wait(&bar.empty[s], ((g / kS) - 1) & 1, bar.abort))) break;
          uint8_t* st = smem + s * mp.stage;
          mbar_arrive_expect_tx(&bar.full[s], bytes);
          for (int c = 0; c < np; ++c) {
            tma_load_3d(st + c * kPanel, &tm_k, 64 * c, j0, bh, &bar.full[s]);
            tma_load_3d(st + mp.tile + c * kPanel, &tm_v, 64 * c, j0, bh, &bar.full[s]);
          }
          if constexpr (kBias) tma_load_3d(st + 2 * mp.tile, &tm_bias, j0, i0, h, &bar.full[s]);
          if constexpr (kBin)
            bulk_load(st + mp.vec, p.ak + static_cast<size_t>(bh) * p.Npad + j0, kCols * 4, &bar.full[s]);
        }
      }
      settle(bar, g, kS);
    }
  } else if (warp == kMmaWarp) {
    // the whole warp runs this (see mma_ts_warp)
    const uint32_t id = idesc_bf16(kRows, DP, true);
    bool ok = true;
    for (int it = 0; ok && it < n_items; ++it) {
      if (!(ok = wait_warp(bar.a_ready, it & 1, bar.abort))) break;
      tc_fence_after();
      for (int t = 0; t < T + 2; ++t) {
        const int g = it * T + t, b = g & 1;
        if (t >= 2) {  // the tile before last: its buffer is free, its dL written
          if (!(ok = wait_warp(&bar.p_full[b], ((g - 2) >> 1) & 1, bar.abort))) break;
          tc_fence_after();
          const int s = (g - 2) % kS;
          if (t - 2 >= nkt)
            issue_grad(tmem + kAcc, tmem + b * kBuf, smem_u32(smem + s * mp.stage), id, t - 2 > nkt);
          mma_commit_warp(&bar.empty[s]);
        }
        if (t < T) {
          const int s = g % kS;
          if (!(ok = wait_warp(&bar.full[s], (g / kS) & 1, bar.abort))) break;
          const uint32_t st = smem_u32(smem + s * mp.stage);
          issue_scores<false>(tmem + b * kBuf, tmem + kRowsQ, st, DP / 16);
          issue_scores<false>(tmem + b * kBuf + 64, tmem + kRowsDO, st + mp.tile, DP / 16);
          mma_commit_warp(&bar.s_full[b]);
        }
      }
      if (ok) mma_commit_warp(bar.o_done);
    }
    drain_mma(bar);
  } else {
    const int wg = warp >> 2, buf = wg >> 1, hh = wg & 1;
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + buf * kBuf + 32 * hh, dp_col = s_col + 64;
    float* sc = reinterpret_cast<float*>(smem + mp.scratch);  // [3][4 wg][128 rows]
    bool ok = true;
    auto wait_all = [&](uint64_t* b, uint32_t parity) { return wait_warp(b, parity, bar.abort); };
    // scores, dP and the stage of tile g in registers, as logits; columns >= N
    // are -inf
    uint32_t xr[32], dp[32];
    auto tile = [&](int g, int j0, float ci) -> const uint8_t* {
      const int s = g % kS;
      ok = ok && wait_all(&bar.s_full[buf], (g >> 1) & 1) && wait_all(&bar.full[s], (g / kS) & 1);
      tc_fence_after();
      const uint8_t* st = smem + s * mp.stage;
      if (ok) {
        tmem_ld32(s_col, xr);
        tmem_ld32(dp_col, dp);
        uint32_t bias[16];
        if constexpr (kBias) {
          const uint8_t* br = st + 2 * mp.tile + r * 128;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 v = *reinterpret_cast<const uint4*>(br + (((4 * hh + u) ^ (r & 7)) << 4));
            bias[4 * u] = v.x; bias[4 * u + 1] = v.y; bias[4 * u + 2] = v.z; bias[4 * u + 3] = v.w;
          }
        }
        tmem_ld_wait();
        logits<kBin, kBias, 32>(xr, reinterpret_cast<const float*>(st + mp.vec) + 32 * hh, ci, bias);
        if (j0 + kCols > N) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (j0 + 32 * hh + e >= N) xr[e] = 0xff800000u;
        }
      }
      return st;
    };
    for (int it = 0; it < n_items; ++it) {
      int bh, h, i0;
      item(it, bh, h, i0);
      const int row = i0 + r;
      const bool valid = row < N;
      const size_t tok = static_cast<size_t>(bh) * N + (valid ? row : 0);
      if (ok && wg < 2) stage_row((wg ? p.a1 : p.a0) + tok * d, valid, d, DP, lb + (wg ? kRowsDO : kRowsQ));
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar.a_ready);
      const float ci = !kBin ? p.cs : valid ? p.aq[static_cast<size_t>(bh) * p.Npad + row] : 0.f;
      const int g0 = it * T;

      // ---- first pass: m, l and sum exp(x - m) dP of this thread's columns
      float m = -INFINITY, l = 0.f, aD = 0.f;
      int t = buf;  // T is even, so a tile's buffer is its parity in the item
      for (; t < nkt; t += 2) {
        tile(g0 + t, t * kCols, ci);
        if (!ok) continue;
        tc_fence_before();
        mbar_arrive(&bar.p_full[buf]);  // everything of the tile is in registers
        float* x = reinterpret_cast<float*>(xr);
        float a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = max3f(x[k], x[k + 4], x[k + 8]);
          a[k] = max3f(a[k], x[k + 12], x[k + 16]);
          a[k] = max3f(a[k], x[k + 20], x[k + 24]);
          a[k] = fmaxf(a[k], x[k + 28]);
        }
        const float mn = fmaxf(m, fmaxf(max3f(a[0], a[1], a[2]), a[3]));
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing but -inf so far: every exp is 0
        const float corr = exp2v<kBias>(make_float2(m, m), make_float2(-ms, -ms)).x;
        m = mn;
        float2 l2 = make_float2(0.f, 0.f), d2 = l2;
        const float2 nm = make_float2(-ms, -ms);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 ex = exp2v<kBias>(reinterpret_cast<float2*>(xr)[e], nm);
          l2 = __fadd2_rn(l2, ex);
          d2 = __ffma2_rn(ex, reinterpret_cast<float2*>(dp)[e], d2);
        }
        l = fmaf(l, corr, l2.x + l2.y);
        aD = fmaf(aD, corr, d2.x + d2.y);
      }
      // ---- the row's four partial results (two buffers, two halves) joined
      sc[wg * kRows + r] = m;
      sc[(4 + wg) * kRows + r] = l;
      sc[(8 + wg) * kRows + r] = aD;
      named_sync(kBar, kCompute);
      float M = -INFINITY, Ls = 0.f, Ds = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, sc[k * kRows + r]);
      // a row with nothing but -inf: no weights, so +inf makes every P 0
      float lse = INFINITY, l2 = 0.f, D = 0.f;
      if (M > -INFINITY) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float w = exp2v<kBias>(make_float2(sc[k * kRows + r], 0.f), make_float2(-M, -M)).x;
          Ls = fmaf(w, sc[(4 + k) * kRows + r], Ls);
          Ds = fmaf(w, sc[(8 + k) * kRows + r], Ds);
        }
        l2 = log2f(Ls);
        lse = kBias ? M : M + l2;
        D = Ds / Ls;
      }
      if (wg == 0 && row < p.Npad) {
        p.lse[static_cast<size_t>(bh) * p.Npad + row] = valid ? lse : INFINITY;
        p.D[static_cast<size_t>(bh) * p.Npad + row] = valid ? D : 0.f;
        if (kBias) p.l2[static_cast<size_t>(bh) * p.Npad + row] = valid ? l2 : 0.f;
      }
      // ---- second pass: dL (binary: times alpha_k) as bf16 over the scores
      const float2 nl = make_float2(-lse, -lse), nl2 = make_float2(-l2, -l2), nD = make_float2(-D, -D);
      for (; t < T; t += 2) {
        const int j0 = (t - nkt) * kCols;
        const uint8_t* st = tile(g0 + t, j0, ci);
        if (!ok) continue;
        const float* ak = reinterpret_cast<const float*>(st + mp.vec) + 32 * hh;
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 P = exp2v<kBias>(reinterpret_cast<float2*>(xr)[e], nl, nl2);
          float2 dl = __fmul2_rn(P, __fadd2_rn(reinterpret_cast<float2*>(dp)[e], nD));
          if constexpr (kBin) dl = __fmul2_rn(dl, *reinterpret_cast<const float2*>(ak + 2 * e));
          pk[e] = pack_bf16x2(dl.x, dl.y);
        }
        tmem_st16(s_col, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[buf]);
      }
      ok = ok && wait_all(bar.o_done, it & 1);
      tc_fence_after();
      if (ok && 32 * wg < d) store_row(lb + kAcc, p.out, p.g0 + tok * d, valid, 32 * wg, d);
    }
  }
  end(tmem, warp);
}

// kSS: the kept operands (K and V) in shared memory, for head dims whose
// operands and accumulators do not all fit in tensor memory (2 buffers of 128
// columns + 3 DP > 512).
template <bool kBin, bool kBias, bool kSS>
__global__ void __launch_bounds__(kThreads, 1)
cols_kernel(const Params p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
            const __grid_constant__ CUtensorMap tm_bias, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kS = kSS ? 3 : 4;
  const Map mp = smem_map(p.d, kBias, kS, kSS, 0);
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, np = d > 64 ? 2 : 1;
  const int T = (N + kCols - 1) / kCols;
  const int njt = (N + kRows - 1) / kRows;
  const int G = static_cast<int>(gridDim.x);
  const int n_items = (p.items - static_cast<int>(blockIdx.x) + G - 1) / G;
  const int dv_col = kAcc, dk_col = kAcc + (kSS ? 128 : DP), k_col = kAcc + 2 * DP, v_col = k_col + DP / 2;
  auto item = [&](int it, int& bh, int& h, int& j0) {
    const int w = static_cast<int>(blockIdx.x) + it * G;
    const int b = w % p.B, kt = (w / p.B) % njt;
    h = w / (p.B * njt);
    bh = b * p.H + h;
    j0 = kt * kRows;
  };
  const uint32_t tmem = begin(bar, warp);

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      int g = 0, kept = 0;  // copies of stages and of kept operands issued
      const uint32_t bytes = 2u * mp.tile + (kBias ? kBiasBytes + kCols * 4 : 0) + (kBin ? 3 : 2) * kCols * 4;
      for (int it = 0; ok && it < n_items; ++it) {
        int bh, h, j0;
        item(it, bh, h, j0);
        if constexpr (kSS) {
          if (it > 0 && !(ok = mbar_wait(bar.o_done, (it - 1) & 1, bar.abort))) break;
          ++kept;
          mbar_arrive_expect_tx(bar.kept, 4u * mp.tile);
          for (int c = 0; c < np; ++c)
            for (int u = 0; u < 2; ++u) {
              tma_load_3d(smem + mp.kept + (2 * c + u) * kPanel, &tm_k, 64 * c, j0 + 64 * u, bh, bar.kept);
              tma_load_3d(smem + mp.kept + 2 * mp.tile + (2 * c + u) * kPanel, &tm_v, 64 * c, j0 + 64 * u, bh,
                          bar.kept);
            }
        }
        for (int t = 0; t < T; ++t, ++g) {
          const int s = g % kS, i0 = t * kCols;
          if (g >= kS && !(ok = mbar_wait(&bar.empty[s], ((g / kS) - 1) & 1, bar.abort))) break;
          uint8_t* st = smem + s * mp.stage;
          mbar_arrive_expect_tx(&bar.full[s], bytes);
          for (int c = 0; c < np; ++c) {
            tma_load_3d(st + c * kPanel, &tm_q, 64 * c, i0, bh, &bar.full[s]);
            tma_load_3d(st + mp.tile + c * kPanel, &tm_do, 64 * c, i0, bh, &bar.full[s]);
          }
          if constexpr (kBias)
            for (int u = 0; u < 2; ++u)
              tma_load_3d(st + 2 * mp.tile + u * kPanel, &tm_bias, j0 + 64 * u, i0, h, &bar.full[s]);
          const size_t at = static_cast<size_t>(bh) * p.Npad + i0;
          bulk_load(st + mp.vec, p.lse + at, kCols * 4, &bar.full[s]);
          bulk_load(st + mp.vec + 256, p.D + at, kCols * 4, &bar.full[s]);
          if constexpr (kBin) bulk_load(st + mp.vec + 512, p.aq + at, kCols * 4, &bar.full[s]);
          if constexpr (kBias) bulk_load(st + mp.vec + 768, p.l2 + at, kCols * 4, &bar.full[s]);
        }
      }
      settle(bar, g, kS);
      if (kept > 0) {
        volatile int never = 0;
        mbar_wait(bar.kept, (kept - 1) & 1, &never);
      }
    }
  } else if (warp == kMmaWarp) {
    // the whole warp runs this (see mma_ts_warp)
    const uint32_t id = idesc_bf16(kRows, DP, true);
    bool ok = true;
    for (int it = 0; ok && it < n_items; ++it) {
      if (!(ok = wait_warp(bar.a_ready, it & 1, bar.abort))) break;
      if (kSS && !(ok = wait_warp(bar.kept, it & 1, bar.abort))) break;
      tc_fence_after();
      for (int t = 0; t < T + 2; ++t) {
        const int g = it * T + t, b = g & 1;
        if (t >= 2) {
          if (!(ok = wait_warp(&bar.p_full[b], ((g - 2) >> 1) & 1, bar.abort))) break;
          tc_fence_after();
          const int s = (g - 2) % kS;
          const uint32_t st = smem_u32(smem + s * mp.stage);
          issue_grad(tmem + dv_col, tmem + b * kBuf, st + mp.tile, id, t > 2);
          issue_grad(tmem + dk_col, tmem + b * kBuf + 64, st, id, t > 2);
          mma_commit_warp(&bar.empty[s]);
        }
        if (t < T) {
          const int s = g % kS;
          if (!(ok = wait_warp(&bar.full[s], (g / kS) & 1, bar.abort))) break;
          const uint32_t st = smem_u32(smem + s * mp.stage);
          const uint32_t kept = smem_u32(smem + mp.kept);
          issue_scores<kSS>(tmem + b * kBuf, kSS ? kept : tmem + k_col, st, DP / 16);
          issue_scores<kSS>(tmem + b * kBuf + 64, kSS ? kept + 2 * mp.tile : tmem + v_col, st + mp.tile, DP / 16);
          mma_commit_warp(&bar.s_full[b]);
        }
      }
      if (ok) mma_commit_warp(bar.o_done);
    }
    drain_mma(bar);
  } else {
    const int wg = warp >> 2, buf_wg = wg >> 1, hh = wg & 1;
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + buf_wg * kBuf + 32 * hh, dp_col = s_col + 64;
    // this thread's key in the bias boxes: byte offset of (query row 0, key r),
    // before the row's swizzle of its 16-byte units
    const int bkey = (r >> 6) * kPanel + (r & 7) * 2, bunit = (r & 63) >> 3;
    bool ok = true;
    auto wait_all = [&](uint64_t* b, uint32_t parity) { return wait_warp(b, parity, bar.abort); };
    for (int it = 0; it < n_items; ++it) {
      int bh, h, j0;
      item(it, bh, h, j0);
      const int key = j0 + r;
      const bool valid = key < N;
      const size_t tok = static_cast<size_t>(bh) * N + (valid ? key : 0);
      if constexpr (!kSS) {
        if (ok && wg < 2) stage_row((wg ? p.a1 : p.a0) + tok * d, valid, d, DP, lb + (wg ? v_col : k_col));
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(bar.a_ready);
      const float akj = kBin && valid ? p.ak[static_cast<size_t>(bh) * p.Npad + key] : 0.f;
      const int g0 = it * T;
      for (int t = (g0 & 1) == buf_wg ? 0 : 1; t < T; t += 2) {  // this buffer's tiles
        const int g = g0 + t, s = g % kS;
        ok = ok && wait_all(&bar.s_full[buf_wg], (g >> 1) & 1) && wait_all(&bar.full[s], (g / kS) & 1);
        if (!ok) continue;
        tc_fence_after();
        const uint8_t* st = smem + s * mp.stage;
        const float* vec = reinterpret_cast<const float*>(st + mp.vec) + 32 * hh;  // LSE, D at 64, c alpha_q at 128, log2 sum at 192
        const uint8_t* bt = st + 2 * mp.tile + bkey + 32 * hh * 128;
        uint32_t xr[32], dp[32];
        tmem_ld32(s_col, xr);
        tmem_ld32(dp_col, dp);
        tmem_ld_wait();
        uint32_t pp[16], pd[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 lse = *reinterpret_cast<const float2*>(vec + 2 * e);
          const float2 D = *reinterpret_cast<const float2*>(vec + 64 + 2 * e);
          float2 x = reinterpret_cast<float2*>(xr)[e], ci = make_float2(p.cs, p.cs);
          if constexpr (kBin) {
            ci = *reinterpret_cast<const float2*>(vec + 128 + 2 * e);
            x = __fmul2_rn(x, make_float2(akj, akj));
          }
          if constexpr (kBias) {
            float2 b;
            const int e0 = 2 * e, e1 = 2 * e + 1;
            b.x = __uint_as_float(
                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(bt + e0 * 128 + ((bunit ^ (e0 & 7)) << 4))) << 16);
            b.y = __uint_as_float(
                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(bt + e1 * 128 + ((bunit ^ (e1 & 7)) << 4))) << 16);
            x = __ffma2_rn(x, ci, b);
          } else {
            x = __fmul2_rn(x, ci);
          }
          float2 nl2 = make_float2(0.f, 0.f);
          if constexpr (kBias) {
            nl2 = *reinterpret_cast<const float2*>(vec + 192 + 2 * e);
            nl2 = make_float2(-nl2.x, -nl2.y);
          }
          const float2 P = exp2v<kBias>(x, make_float2(-lse.x, -lse.y), nl2);
          float2 dl = __fmul2_rn(P, __fadd2_rn(reinterpret_cast<float2*>(dp)[e], make_float2(-D.x, -D.y)));
          if constexpr (kBin) dl = __fmul2_rn(dl, ci);
          pp[e] = pack_bf16x2(P.x, P.y);
          pd[e] = pack_bf16x2(dl.x, dl.y);
        }
        tmem_st16(s_col, pp);
        tmem_st16(dp_col, pd);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[buf_wg]);
      }
      ok = ok && wait_all(bar.o_done, it & 1);
      tc_fence_after();
      if (ok && 32 * wg < d) {
        store_row(lb + dv_col, 1.f, p.g0 + tok * d, valid, 32 * wg, d);
        store_row(lb + dk_col, p.out, p.g1 + tok * d, valid, 32 * wg, d);
      }
    }
  }
  end(tmem, warp);
}

// Batch entries whose kept operands fit in tensor memory beside the buffers.
inline int dbias_batch(int d) {
  const int n = 256 / ((d + 15) / 16 * 16);
  return n < 4 ? n : 4;
}

// dbias of 128 query rows of one head and the key tiles of split x: per pair of
// key tiles (one per buffer) and chunk of up to p.nb batch entries, dL summed
// over the chunk in registers. With one chunk the sums are the result; with
// more, chunks are added in order in an fp32 array, and where too few CTAs
// would run, the chunks are also split over CTAs with an array each
// (dbias_sum_kernel joins them).
template <bool kBin, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
dbias_kernel(const Params p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ CUtensorMap tm_bias) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kS = kRowStages;
  const Map mp = smem_map(p.d, kBias, kS, false, kDbiasScratch);
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, np = d > 64 ? 2 : 1;
  const int nit = (N + kRows - 1) / kRows;
  const int npairs = ((N + kCols - 1) / kCols + 1) / 2;  // a last odd tile is paired with one beyond N
  const int G = static_cast<int>(gridDim.x);
  const int n_items = (p.items - static_cast<int>(blockIdx.x) + G - 1) / G;
  // items: key split, then query tile, then head, then chunk split
  struct Item {
    int h, i0, pr0, pr1, ch0, ch1, split;
  };
  auto item = [&](int it) {
    int w = static_cast<int>(blockIdx.x) + it * G;
    Item x;
    const int js = w % p.jsplit;
    w /= p.jsplit;
    x.i0 = (w % nit) * kRows;
    w /= nit;
    x.h = w % p.H;
    x.split = w / p.H;
    x.pr0 = static_cast<int>(static_cast<long long>(npairs) * js / p.jsplit);
    x.pr1 = static_cast<int>(static_cast<long long>(npairs) * (js + 1) / p.jsplit);
    x.ch0 = static_cast<int>(static_cast<long long>(p.nchunks) * x.split / p.nsplit);
    x.ch1 = static_cast<int>(static_cast<long long>(p.nchunks) * (x.split + 1) / p.nsplit);
    return x;
  };
  auto batch = [&](int ch) { return min(p.nb, p.B - ch * p.nb); };
  const uint32_t tmem = begin(bar, warp);

  // Tiles of one chunk of one item: for every key pair, for every batch entry,
  // buffer 0's tile and buffer 1's.
  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      for (int it = 0; ok && it < n_items; ++it) {
        const Item x = item(it);
        for (int ch = x.ch0; ok && ch < x.ch1; ++ch) {
          const int nb = batch(ch);
          for (int pr = x.pr0; ok && pr < x.pr1; ++pr) {
            for (int u = 0; u < 2 * nb; ++u, ++g) {
              const int s = g % kS, j0 = (2 * pr + (u & 1)) * kCols;
              const int bh = (ch * p.nb + (u >> 1)) * p.H + x.h;
              if (g >= kS && !(ok = mbar_wait(&bar.empty[s], ((g / kS) - 1) & 1, bar.abort))) break;
              const bool with_bias = kBias && u < 2;  // the first entry's tiles bring the bias
              // a tile wholly beyond N (the last pair's second) has no alpha_k
              const bool with_ak = kBin && j0 < N;
              uint8_t* st = smem + s * mp.stage;
              mbar_arrive_expect_tx(&bar.full[s], 2u * mp.tile + (with_bias ? kBiasBytes : 0) +
                                                      (with_ak ? kCols * 4 : 0));
              for (int c = 0; c < np; ++c) {
                tma_load_3d(st + c * kPanel, &tm_k, 64 * c, j0, bh, &bar.full[s]);
                tma_load_3d(st + mp.tile + c * kPanel, &tm_v, 64 * c, j0, bh, &bar.full[s]);
              }
              if (with_bias) tma_load_3d(st + 2 * mp.tile, &tm_bias, j0, x.i0, x.h, &bar.full[s]);
              if (with_ak)
                bulk_load(st + mp.vec, p.ak + static_cast<size_t>(bh) * p.Npad + j0, kCols * 4, &bar.full[s]);
            }
          }
        }
      }
      settle(bar, g, kS);
    }
  } else if (warp == kMmaWarp) {
    // the whole warp runs this (see mma_ts_warp)
    bool ok = true;
    int g0 = 0, staged = 0;
    for (int it = 0; ok && it < n_items; ++it) {
      const Item x = item(it);
      for (int ch = x.ch0; ok && ch < x.ch1; ++ch, ++staged) {
        const int nb = batch(ch), T = (x.pr1 - x.pr0) * 2 * nb;
        if (!(ok = wait_warp(bar.a_ready, staged & 1, bar.abort))) break;
        tc_fence_after();
        for (int t = 0; t < T + 2; ++t) {
          const int g = g0 + t, b = g & 1;
          if (t >= 2) {
            if (!(ok = wait_warp(&bar.p_full[b], ((g - 2) >> 1) & 1, bar.abort))) break;
            tc_fence_after();
            if (lane == 0) mbar_arrive(&bar.empty[(g - 2) % kS]);  // its MMAs were complete before the threads read them
          }
          if (t < T) {
            const int s = g % kS, e = (t >> 1) % nb;
            if (!(ok = wait_warp(&bar.full[s], (g / kS) & 1, bar.abort))) break;
            const uint32_t st = smem_u32(smem + s * mp.stage);
            issue_scores<false>(tmem + b * kBuf, tmem + kAcc + e * DP, st, DP / 16);
            issue_scores<false>(tmem + b * kBuf + 64, tmem + kAcc + e * DP + DP / 2, st + mp.tile, DP / 16);
            mma_commit_warp(&bar.s_full[b]);
          }
        }
        g0 += T;
      }
    }
    drain_mma(bar);
  } else {
    const int wg = warp >> 2, buf = wg >> 1, hh = wg & 1;
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + buf * kBuf + 32 * hh, dp_col = s_col + 64;
    float* sc = reinterpret_cast<float*>(smem + mp.scratch);  // [LSE, D, ci, log2 sum][entry of the chunk][128 rows]
    bool ok = true;
    auto wait_all = [&](uint64_t* b, uint32_t parity) { return wait_warp(b, parity, bar.abort); };
    int g = buf;
    for (int it = 0; it < n_items; ++it) {
      const Item x = item(it);
      const int row = x.i0 + r;
      const bool valid = row < N;
      for (int ch = x.ch0; ch < x.ch1; ++ch) {
        const int nb = batch(ch);
        // Every thread is past the previous chunk's tiles (their MMAs with
        // them), so the kept operands and row vectors may be replaced.
        named_sync(kBar, kCompute);
        if (ok) {
          for (int u = wg; u < 2 * nb; u += 4) {
            const size_t tok = (static_cast<size_t>(ch * p.nb + (u >> 1)) * p.H + x.h) * N + (valid ? row : 0);
            stage_row((u & 1 ? p.a1 : p.a0) + tok * d, valid, d, DP, lb + kAcc + (u >> 1) * DP + (u & 1 ? DP / 2 : 0));
          }
        }
        if (wg < nb) {
          const size_t at = (static_cast<size_t>(ch * p.nb + wg) * p.H + x.h) * p.Npad + row;
          sc[wg * kRows + r] = valid ? p.lse[at] : INFINITY;
          sc[(4 + wg) * kRows + r] = valid ? p.D[at] : 0.f;
          sc[(8 + wg) * kRows + r] = !kBin ? p.cs : valid ? p.aq[at] : 0.f;
          if (kBias) sc[(12 + wg) * kRows + r] = valid ? p.l2[at] : 0.f;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar.a_ready);
        named_sync(kBar, kCompute);  // the row vectors are in place
        const bool first = ch == x.ch0, last = ch + 1 == x.ch1;
        for (int pr = x.pr0; pr < x.pr1; ++pr) {
          const int j0 = (2 * pr + buf) * kCols + 32 * hh;  // this thread's first column
          float2 acc[16];
          uint32_t bias[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] = make_float2(0.f, 0.f);
          for (int b = 0; b < nb; ++b, g += 2) {
            const int s = g % kS;
            ok = ok && wait_all(&bar.s_full[buf], (g >> 1) & 1) && wait_all(&bar.full[s], (g / kS) & 1);
            if (!ok) continue;
            tc_fence_after();
            const uint8_t* st = smem + s * mp.stage;
            if (kBias && b == 0) {
              const uint8_t* br = st + 2 * mp.tile + r * 128;
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const uint4 v = *reinterpret_cast<const uint4*>(br + (((4 * hh + u) ^ (r & 7)) << 4));
                bias[4 * u] = v.x; bias[4 * u + 1] = v.y; bias[4 * u + 2] = v.z; bias[4 * u + 3] = v.w;
              }
            }
            const float lse = sc[b * kRows + r], D = sc[(4 + b) * kRows + r], ci = sc[(8 + b) * kRows + r];
            const float l2 = kBias ? sc[(12 + b) * kRows + r] : 0.f;
            const float* ak = reinterpret_cast<const float*>(st + mp.vec) + 32 * hh;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t xr[16], dp[16];
              tmem_ld16(s_col + 16 * q, xr);
              tmem_ld16(dp_col + 16 * q, dp);
              tmem_ld_wait();
              logits<kBin, kBias, 16>(xr, ak + 16 * q, ci, bias + 8 * q);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 P =
                    exp2v<kBias>(reinterpret_cast<float2*>(xr)[e], make_float2(-lse, -lse), make_float2(-l2, -l2));
                acc[8 * q + e] = __ffma2_rn(P, __fadd2_rn(reinterpret_cast<float2*>(dp)[e], make_float2(-D, -D)),
                                            acc[8 * q + e]);
              }
            }
            tc_fence_before();
            mbar_arrive(&bar.p_full[buf]);
          }
          if (!ok || !valid) continue;
          const size_t at = (static_cast<size_t>(x.h) * N + row) * N + j0;
          float* part = p.part ? p.part + static_cast<size_t>(x.split) * p.H * N * N + at : nullptr;
          const float* a = reinterpret_cast<const float*>(acc);
          float sum[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[e] = a[e];
          if (!first) {  // this thread's own sums of the chunks before
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (j0 + e < N) sum[e] += part[e];
          }
          if (last && p.nsplit == 1) {
            uint16_t* dst = p.g0 + at;
            if (N % 8 == 0) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                if (j0 + e < N)
                  *reinterpret_cast<uint4*>(dst + e) =
                      make_uint4(pack_bf16x2(sum[e], sum[e + 1]), pack_bf16x2(sum[e + 2], sum[e + 3]),
                                 pack_bf16x2(sum[e + 4], sum[e + 5]), pack_bf16x2(sum[e + 6], sum[e + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (j0 + e < N) dst[e] = float_to_bf16_bits(sum[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (j0 + e < N) part[e] = sum[e];
          }
        }
      }
    }
  }
  end(tmem, warp);
}

// dbias from the chunk splits' sums, added in order.
__global__ void __launch_bounds__(256) dbias_sum_kernel(const float* __restrict__ part, long long n, int nsplit,
                                                        uint16_t* __restrict__ out) {
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * 256) {
    float s = part[i];
    for (int k = 1; k < nsplit; ++k) s += part[k * n + i];
    out[i] = float_to_bf16_bits(s);
  }
}

// Binary operands of the tensor cores: the sign words as bf16 +-1 [tokens, d]
// (d % 8 == 0; one thread per 8 channels), and alpha with rows of N padded to
// Npad (zeros), times f.
__global__ void __launch_bounds__(256) expand_signs_kernel(const uint32_t* __restrict__ bits, long long chunks, int d,
                                                           uint16_t* __restrict__ out) {
  const int per = d / 8, W = words_for(d);
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < chunks;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long tok = i / per;
    const int g = static_cast<int>(i - tok * per);
    const uint32_t byte = bits[tok * W + (g >> 2)] >> (8 * (g & 3));
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)  // bf16 1.0 is 0x3F80, -1.0 is 0xBF80
      w[e] = 0xBF80BF80u ^ (((byte >> (2 * e)) & 1u) << 15) ^ (((byte >> (2 * e + 1)) & 1u) << 31);
    *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__global__ void __launch_bounds__(256) pad_alpha_kernel(const float* __restrict__ aq, const float* __restrict__ ak,
                                                        long long n, int N, int Npad, float c, float units,
                                                        float* __restrict__ oq, float* __restrict__ ok) {
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long bh = i / Npad;
    const int t = static_cast<int>(i - bh * Npad);
    const bool in = t < N;
    oq[i] = in ? __fmul_rn(__fmul_rn(c, aq[bh * N + t]), units) : 0.f;
    ok[i] = in ? ak[bh * N + t] : 0.f;
  }
}

// ------------------------------------------------------------------- host
// [BH][N][d] bf16 as boxes of 64 channels x 64 rows, or a bias [H][N][N] (rows
// ld apart) as boxes of 64 keys x box_rows rows; 128-byte swizzle, zeros
// outside.
inline bool make_map(CUtensorMap* tm, const uint16_t* base, cuuint64_t inner, cuuint64_t rows, cuuint64_t ld,
                     cuuint64_t planes, cuuint32_t box_rows, const char* what, std::string* msg) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) {
    *msg = "cuTensorMapEncodeTiled entry point unavailable";
    return false;
  }
  const cuuint32_t es[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {inner, rows, planes};
  const cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  CUresult rc = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (rc != CUDA_SUCCESS) {
    *msg = std::string("tensor map (") + what + ") rejected: " + std::to_string(rc);
    return false;
  }
  return true;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// How dbias is cut up. Chunks of nb batch entries; key splits and then chunk
// splits until about two items per SM of a 148-SM part run.
struct DbiasPlan {
  int nb, nchunks, nsplit, jsplit, items;
};
inline DbiasPlan dbias_plan(int B, int H, int N, int d) {
  DbiasPlan q;
  q.nb = dbias_batch(d);
  q.nchunks = (B + q.nb - 1) / q.nb;
  const long long nit = (N + kRows - 1) / kRows;
  const int npairs = ((N + kCols - 1) / kCols + 1) / 2;
  const long long base = nit * H;
  auto up = [](long long a, long long b) { return static_cast<int>((a + b - 1) / b); };
  q.jsplit = base >= 296 ? 1 : std::min(npairs, up(296, base));
  q.nsplit = base * q.jsplit >= 296 ? 1 : std::min(q.nchunks, up(296, base * q.jsplit));
  q.items = static_cast<int>(base * q.jsplit * q.nsplit);
  return q;
}

inline size_t r256(size_t x) { return (x + 255) / 256 * 256; }
inline int npad_for(int N) { return (N + kCols - 1) / kCols * kCols; }

// The workspace of a call, parts rounded up to 256 bytes.
struct Ws {
  size_t lse, D, l2, bias, sq, sk, aq, ak, part, total;
};
inline Ws workspace(int B, int H, int N, int d, bool bin, bool bias, bool dbias) {
  const size_t rows = static_cast<size_t>(B) * H * npad_for(N) * 4, x = static_cast<size_t>(B) * H * N * d * 2;
  const DbiasPlan q = dbias_plan(B, H, N, d);
  Ws w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += r256(bytes);
    return here;
  };
  w.lse = take(rows);
  w.D = take(rows);
  w.l2 = take(bias ? rows : 0);
  w.bias = take(bias && N % 8 ? static_cast<size_t>(H) * N * ((N + 7) / 8 * 8) * 2 : 0);
  w.sq = take(bin ? x : 0);
  w.sk = take(bin ? x : 0);
  w.aq = take(bin ? rows : 0);
  w.ak = take(bin ? rows : 0);
  w.part = take(dbias && q.nchunks > 1 ? static_cast<size_t>(q.nsplit) * H * N * N * 4 : 0);
  w.total = at;
  return w;
}

template <class K>
inline bool set_smem(K kern, int bytes, std::atomic<uint64_t>& done, std::string* msg) {
  if (!needs_setup(done)) return true;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) {
    *msg = std::string("cudaFuncSetAttribute (backward): ") + cudaGetErrorString(e);
    return false;
  }
  mark_setup(done);
  return true;
}
inline bool launched(const char* what, std::string* msg) {
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return true;
  *msg = std::string(what) + " launch: " + cudaGetErrorString(e);
  return false;
}
constexpr int kMaxSmem = 227 * 1024;

struct Maps {
  CUtensorMap q, k, v, dO, bias_rows, bias_cols;
};

template <bool kBin, bool kBias>
inline int run(Params p, const Maps& tm, const uint16_t* q, const uint16_t* k, const uint16_t* v, const uint16_t* dO,
               float c, uint16_t* dq, uint16_t* dk, uint16_t* dv, uint16_t* dbias, cudaStream_t st,
               std::string* msg) {
  const int nsm = sm_count(), nt = (p.N + kRows - 1) / kRows;
  auto grid = [&](int items) { return static_cast<unsigned>(items < nsm ? items : nsm); };
  auto bytes = [](const Map& m) { return m.bytes > kMinSmem ? m.bytes : kMinSmem; };
  {
    static std::atomic<uint64_t> done{0};
    if (!set_smem(rows_kernel<kBin, kBias>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
    Params r = p;
    r.a0 = q;
    r.a1 = dO;
    r.out = c;
    r.g0 = dq;
    r.items = p.B * p.H * nt;
    rows_kernel<kBin, kBias><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, kRowStages, false, kRowsScratch)),
                               st>>>(r, tm.k, tm.v, tm.bias_rows);
    if (!launched("rows_kernel", msg)) return BINATTN_ERR_CUDA;
  }
  {
    Params r = p;
    r.a0 = k;
    r.a1 = v;
    r.out = kBin ? (kBias ? 1.f : kLn2) : c;  // binary: c alpha_q (and log2 e) are already in dL
    r.g0 = dv;
    r.g1 = dk;
    r.items = p.B * p.H * nt;
    if (p.d <= 80) {
      static std::atomic<uint64_t> done{0};
      if (!set_smem(cols_kernel<kBin, kBias, false>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
      cols_kernel<kBin, kBias, false><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, 4, false, 0)), st>>>(
          r, tm.q, tm.dO, tm.bias_cols, tm.k, tm.v);
    } else {
      static std::atomic<uint64_t> done{0};
      if (!set_smem(cols_kernel<kBin, kBias, true>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
      cols_kernel<kBin, kBias, true><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, 3, true, 0)), st>>>(
          r, tm.q, tm.dO, tm.bias_cols, tm.k, tm.v);
    }
    if (!launched("cols_kernel", msg)) return BINATTN_ERR_CUDA;
  }
  if (dbias) {
    const DbiasPlan plan = dbias_plan(p.B, p.H, p.N, p.d);
    static std::atomic<uint64_t> done{0};
    if (!set_smem(dbias_kernel<kBin, kBias>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
    Params r = p;
    r.a0 = q;
    r.a1 = dO;
    r.g0 = dbias;
    r.items = plan.items;
    r.nb = plan.nb;
    r.nchunks = plan.nchunks;
    r.nsplit = plan.nsplit;
    r.jsplit = plan.jsplit;
    if (plan.nchunks == 1) r.part = nullptr;
    dbias_kernel<kBin, kBias><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, kRowStages, false, kDbiasScratch)),
                                st>>>(r, tm.k, tm.v, tm.bias_rows);
    if (!launched("dbias_kernel", msg)) return BINATTN_ERR_CUDA;
    if (plan.nsplit > 1) {
      const long long n = static_cast<long long>(p.H) * p.N * p.N;
      dbias_sum_kernel<<<static_cast<unsigned>(std::min<long long>((n + 255) / 256, 148 * 8)), 256, 0, st>>>(
          p.part, n, plan.nsplit, dbias);
      if (!launched("dbias_sum_kernel", msg)) return BINATTN_ERR_CUDA;
    }
  }
  return BINATTN_OK;
}

// The backward of one call. bf16: q, k; binary: qb, kb, alpha_q, alpha_k (q and
// k null). ws: workspace(...).total bytes.
inline int backward(const uint16_t* q, const uint16_t* k, const uint32_t* qb, const uint32_t* kb, const float* alpha_q,
                    const float* alpha_k, const uint16_t* bias, const uint16_t* v, const uint16_t* dO, float c, int B,
                    int H, int N, int d, uint16_t* dq, uint16_t* dk, uint16_t* dv, uint16_t* dbias, char* ws,
                    cudaStream_t st, std::string* msg) {
  const bool bin = qb != nullptr;
  const Ws w = workspace(B, H, N, d, bin, bias != nullptr, dbias != nullptr);
  const float units = bias ? 1.f : kLog2e;
  Params p;
  std::memset(&p, 0, sizeof p);
  p.B = B;
  p.H = H;
  p.N = N;
  p.d = d;
  p.Npad = npad_for(N);
  p.cs = c * units;
  p.lse = reinterpret_cast<float*>(ws + w.lse);
  p.D = reinterpret_cast<float*>(ws + w.D);
  p.l2 = reinterpret_cast<float*>(ws + w.l2);
  p.part = reinterpret_cast<float*>(ws + w.part);
  if (bin) {
    const long long chunks = static_cast<long long>(B) * H * N * (d / 8);
    const long long n = static_cast<long long>(B) * H * p.Npad;
    auto grid = [](long long k) { return static_cast<unsigned>(std::min<long long>((k + 255) / 256, 148 * 8)); };
    uint16_t* sq = reinterpret_cast<uint16_t*>(ws + w.sq);
    uint16_t* sk = reinterpret_cast<uint16_t*>(ws + w.sk);
    float* aq = reinterpret_cast<float*>(ws + w.aq);
    float* ak = reinterpret_cast<float*>(ws + w.ak);
    expand_signs_kernel<<<grid(chunks), 256, 0, st>>>(qb, chunks, d, sq);
    expand_signs_kernel<<<grid(chunks), 256, 0, st>>>(kb, chunks, d, sk);
    pad_alpha_kernel<<<grid(n), 256, 0, st>>>(alpha_q, alpha_k, n, N, p.Npad, c, units, aq, ak);
    if (!launched("expand_signs_kernel", msg)) return BINATTN_ERR_CUDA;
    q = sq;
    k = sk;
    p.aq = aq;
    p.ak = ak;
  }
  int ld = N;
  if (bias && N % 8) {
    ld = (N + 7) / 8 * 8;
    uint16_t* padded = reinterpret_cast<uint16_t*>(ws + w.bias);
    tc2::pad_bias_rows(bias, static_cast<long long>(H) * N, N, N, ld, padded, st);
    if (!launched("pad_bias_rows_kernel", msg)) return BINATTN_ERR_CUDA;
    bias = padded;
  }
  Maps tm;
  std::memset(&tm, 0, sizeof tm);
  const cuuint64_t BH = static_cast<cuuint64_t>(B) * H;
  if (!make_map(&tm.q, q, d, N, d, BH, kCols, "Q", msg) || !make_map(&tm.k, k, d, N, d, BH, kCols, "K", msg) ||
      !make_map(&tm.v, v, d, N, d, BH, kCols, "V", msg) || !make_map(&tm.dO, dO, d, N, d, BH, kCols, "dO", msg))
    return BINATTN_ERR_CUDA;
  if (bias && (!make_map(&tm.bias_rows, bias, N, N, ld, H, kRows, "bias", msg) ||
               !make_map(&tm.bias_cols, bias, N, N, ld, H, kCols, "bias", msg)))
    return BINATTN_ERR_CUDA;
  if (bin)
    return bias ? run<true, true>(p, tm, q, k, v, dO, c, dq, dk, dv, dbias, st, msg)
                : run<true, false>(p, tm, q, k, v, dO, c, dq, dk, dv, dbias, st, msg);
  return bias ? run<false, true>(p, tm, q, k, v, dO, c, dq, dk, dv, dbias, st, msg)
              : run<false, false>(p, tm, q, k, v, dO, c, dq, dk, dv, dbias, st, msg);
}

}  // namespace bt
}  // namespace binattn
