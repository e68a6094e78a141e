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
// atomics is two more score products, two more products dP and two more rounds of
// exps: 9 products instead of 5 (with dbias 11).
//
// The three share one machine. tile_kernel first lays q, k, v and dO (binary: the
// signs of q and k as +-1) out as the tensor cores take them: tiles of 64 rows,
// each a block of 8-channel groups, [group][row][8]. Such a block serves both as
// the K-major operand of the score products and as the MN-major operand of the
// gradient products, needs no padding of the head dim beyond 16, and comes into
// a ring of stages as one contiguous copy: tensor-map boxes of 144-byte rows
// (d = 72) took the copy engine 1100 cycles a tile, more than the arithmetic. The
// kept operand (128 rows) sits in tensor memory. Scores and dP of a tile are two
// 128 x 64 fp32 accumulators in one of two tensor-memory buffers, and each of
// two compute warpgroups (one thread per kept row) has a buffer of its own and
// takes every second tile. P or dL goes back as bf16, over the scores or dP or
// (rows_kernel, where they fit) into one of three slots. LSE and D are known
// before any exp of the second pass, so threads need nothing of one another
// inside a tile. Warps 8 and 10 issue the MMAs, warp 9 the copies. Bounded waits
// as in fwd_tc2.cuh.
//
// Measured on one B200 (GEMM 1614 TFLOP/s, copies 6.5 TB/s). 2 x 16 x 4096 x 72,
// bf16, without a bias: rows 485 us (five products, 797 TFLOP/s), cols 315 us
// (four, 982 TFLOP/s). The same binary with a dense bias and dbias: rows 621 us,
// cols 396 us, dbias 433 us (two products and the bias's read and dbias's write, 2.5
// TB/s). 64 x 12 x 197 x 64 with a bias: 87, 70 and 145 us. No one unit bounds
// them: a tile's exps take 512 cycles at 16 per SM and cycle and its products
// 350 (first pass) to 700 (cols), against 1000 (rows) and 1300 (cols) measured. The
// rest are the hand-overs of a tile between copies, issuer and compute warps,
// with two tiles under way per SM.
//
// Rounding: P, dL (binary: dL times the alpha of the summed side) and the
// results to bf16, half a step each; all else fp32.
#pragma once
#include <algorithm>
#include <atomic>
#include <cstring>
#include <string>
#include <type_traits>

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
constexpr int kComputeWarps = 8;         // one warpgroup per buffer, one thread per kept row
constexpr int kMmaWarp = 8, kTmaWarp = 9, kGradWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kThreadsDbias = 10 * 32;   // no gradient products, so no warp 10
constexpr int kCompute = kComputeWarps * 32;
constexpr int kGroup = kCols * 16;       // bytes of a tile's 8-channel group
constexpr int kBiasPanel = 64 * 128;     // bytes of a box of 64 rows x 64 keys of the bias
constexpr int kBiasBytes = kRows * kCols * 2;
constexpr int kVecBytes = 1024;          // per stage: up to four vectors of 64 floats
constexpr int kBar = 1;                  // named barrier of the compute warps
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const uint16_t* a0;  // kept operands, tiled: q and dO (rows, dbias), k and v (cols)
  const uint16_t* a1;
  const uint16_t* b0;  // streamed operands, tiled: k and v (rows, dbias), q and dO (cols)
  const uint16_t* b1;
  const float* aq;     // binary: c alpha_q (times log2 e without a bias), padded [BH][Npad]
  const float* ak;     // binary: alpha_k, padded [BH][Npad]
  float cs;            // bf16: factor of the scores (times log2 e without a bias)
  float out;           // factor of dQ (rows) or dK (cols)
  // Row vectors, [BH][Npad], all negated: what logits are taken relative to (see
  // exp2v), with a bias log2 of the row's sum, and D.
  float* nlse;
  float* nl2;
  float* nD;
  uint16_t* g0;        // rows: dQ; cols: dV; dbias: dbias
  uint16_t* g1;        // cols: dK
  float* part;         // dbias: fp32 partial sums [nsplit][H][N][N]
  int B, H, N, d, Npad, items;
  int nb, nchunks, nsplit, jsplit;  // dbias
};

// Descriptors of operands in 8 x 16-byte blocks without a swizzle: lbo and sbo
// are the distances of blocks in the leading and the other direction.
__device__ __forceinline__ uint64_t make_desc(uint32_t lo, uint32_t sbo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((sbo >> 4) | (1u << 14)));
  return d;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// D[128 x 64] = A[128 x 16 kCh] B[64 x 16 kCh]^T: A in tensor memory (bf16
// pairs, 8 columns per 16 channels) or shared memory ([group][128 rows][8]), B
// a tile. The channel count is a template argument: with a loop around them,
// the products issue at half the rate of the tensor cores.
template <bool kSS, int kCh>
__device__ __forceinline__ void issue_scores(uint32_t d_col, uint32_t a, uint32_t b, uint32_t lead) {
  constexpr uint32_t id = idesc_bf16(kRows, kCols, false);
  const uint32_t bl = desc_lo(b, kGroup), al = desc_lo(a, 2 * kGroup);
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    const uint64_t bd = make_desc(bl + k * (2 * kGroup >> 4), 128);
    if constexpr (kSS) mma_ss_lead(d_col, make_desc(al + k * (4 * kGroup >> 4), 128), bd, id, k > 0, lead);
    else mma_ts_lead(d_col, a + k * 8, bd, id, k > 0, lead);
  }
}
// D[128 x 16 kCh] += A[128 x 64] B[64 x 16 kCh]: A bf16 pairs in tensor memory,
// its two 32-row halves `gap` columns apart; B a tile, channels along N.
template <int kCh>
__device__ __forceinline__ void issue_grad(uint32_t d_col, uint32_t a, int gap, uint32_t b, bool accumulate,
                                           uint32_t lead) {
  constexpr uint32_t id = idesc_bf16(kRows, 16 * kCh, true);
  const uint32_t bl = desc_lo(b, 128);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    mma_ts_lead(d_col, a + (k >> 1) * gap + (k & 1) * 8, make_desc(bl + k * 16, kGroup), id, accumulate || k > 0, lead);
}
// f<kCh>() for the channel count of a call.
template <class F>
__device__ __forceinline__ bool with_channels(int ch16, F f) {
  switch (ch16) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}

// Row `row` of a tiled operand: its 16-byte group g is at [g * kCols].
__device__ __forceinline__ const uint4* tiled_row(const uint16_t* t, int bh, int nt, int row, int DP) {
  return reinterpret_cast<const uint4*>(t) + (static_cast<size_t>(bh) * nt + row / kCols) * (DP / 8) * kCols + row % kCols;
}
// A thread's row of a kept operand, all of its loads under way at once, and from
// there into its TMEM lane as bf16 pairs or into shared memory; a row that is not
// valid is zeros.
struct KeptRow {
  uint4 v[16];
};
__device__ __forceinline__ void load_row(KeptRow& k, const uint4* row, bool valid, int DP) {
#pragma unroll
  for (int g = 0; g < 16; ++g) k.v[g] = valid && g < DP / 8 ? __ldg(row + g * kCols) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void stage_row(const KeptRow& k, int DP, uint32_t col) {
#pragma unroll
  for (int g = 0; g < 16; g += 2) {
    if (g < DP / 8) {
      const uint32_t w[8] = {k.v[g].x,     k.v[g].y,     k.v[g].z,     k.v[g].w,
                             k.v[g + 1].x, k.v[g + 1].y, k.v[g + 1].z, k.v[g + 1].w};
      tmem_st8(col + 4 * g, w);
    }
  }
}
__device__ __forceinline__ void stage_row_smem(const KeptRow& k, int DP, uint8_t* dst, int r) {
#pragma unroll
  for (int g = 0; g < 16; ++g)
    if (g < DP / 8) *reinterpret_cast<uint4*>(dst + g * 2 * kGroup + r * 16) = k.v[g];
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

// Row r's bias columns of half h of a tile (half of a 128-byte swizzled row of
// the stage's box) as packed pairs.
__device__ __forceinline__ void load_bias(const uint8_t* box, int r, int h, uint32_t (&b)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 v = *reinterpret_cast<const uint4*>(box + r * 128 + (((4 * h + u) ^ (r & 7)) << 4));
    b[4 * u] = v.x; b[4 * u + 1] = v.y; b[4 * u + 2] = v.z; b[4 * u + 3] = v.w;
  }
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
// 2^y of two values (y <= 1 or so) without the special-function unit: y = n + f
// with n the nearest integer (added to 1.5 * 2^23 it stands in the low bits of
// the sum), 2^f by a polynomial fitted to the smallest relative error on [-1/2,
// 1/2] with constant term 1 (1.08e-7, in fp32 1.7e-7: no worse than ex2.approx),
// and n added to the exponent. y is cut off at -127, where f is 0 and the
// result's bits are all 0: masked pairs keep a weight of exactly 0.
__device__ __forceinline__ float2 ex2_fma(float2 y) {
  y = make_float2(fmaxf(y.x, -127.f), fmaxf(y.y, -127.f));
  const float2 t = __fadd2_rn(y, make_float2(12582912.f, 12582912.f));
  const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), y);
  float2 p = make_float2(0.00132647272f, 0.00132647272f);
  p = __ffma2_rn(p, f, make_float2(0.00967151269f, 0.00967151269f));
  p = __ffma2_rn(p, f, make_float2(0.0555073374f, 0.0555073374f));
  p = __ffma2_rn(p, f, make_float2(0.240222421f, 0.240222421f));
  p = __ffma2_rn(p, f, make_float2(0.693146978f, 0.693146978f));
  p = __ffma2_rn(p, f, make_float2(1.f, 1.f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}
// exp of x minus `top`, x in the units of logits(). Without a bias, top is the
// max or the log-sum-exp. With one, a row may consist of masked logits of
// -1e9 or the type's lowest value, where max + log(sum) would lose the sum: top
// is the max, and the (log2 of the) sum is taken off after the subtraction, in
// the multiply-add that changes the units.
// kFma takes it on the FMA pipe (below).
template <bool kBias, bool kFma = false>
__device__ __forceinline__ float2 exp2v(float2 x, float2 minus_top, float2 minus_l2 = make_float2(0.f, 0.f)) {
  float2 y = __fadd2_rn(x, minus_top);
  if constexpr (kBias) y = __ffma2_rn(y, make_float2(kLog2e, kLog2e), minus_l2);
  if constexpr (kFma) return ex2_fma(y);
  return make_float2(ex2(y.x), ex2(y.y));
}
// Without a bias every fourth pair of a row's exps runs on the FMA pipe, which has
// room there beside the special-function unit: 767 against 785 us at 2 x 16 x
// 4096 x 72 on the same inputs again and again (every second 830, every eighth 773). With a bias the FMA pipe has
// its share of the logits too, and taking none is best: 1487 against 1510 us.
template <bool kBias>
__device__ __forceinline__ constexpr bool on_fma(int pair) { return !kBias && pair % 4 == 3; }

// Shared memory: the stages, then (cols, kSS) the kept operands, then scratch.
struct Map {
  int tile, vec, stage, stages, kept, scratch, bars, bytes;
};
constexpr int kMaxSmem = 227 * 1024;
constexpr int kMaxStages = 8;
constexpr int kTileBars = 8;             // barriers of tiles in turn; more tiles are never under way than stages
static_assert(kMaxStages <= kTileBars, "a tile's barrier must be free again before its next tile has a stage");
constexpr int kBarBytes = 512;
__host__ __device__ inline Map smem_map(int d, bool bias, bool kept, int scratch) {
  Map m;
  m.tile = (d + 15) / 16 * 16 * 128;                   // one streamed matrix
  m.vec = 2 * m.tile + (bias ? kBiasBytes : 0);        // vectors, after both and the bias
  m.stage = m.vec + kVecBytes;
  // As many stages as fit: a tile holds its stage until its gradient products
  // are done, some 2500 cycles, and the next copy takes 1000 more.
  const int room = (kMaxSmem - kBarBytes - scratch - (kept ? 4 * m.tile : 0)) / m.stage;
  m.stages = room < kMaxStages ? room : kMaxStages;
  m.kept = m.stages * m.stage;
  m.scratch = m.kept + (kept ? 4 * m.tile : 0);
  m.bars = m.scratch + scratch;
  m.bytes = m.bars + kBarBytes;
  return m;
}
constexpr int kMinSmem = 120 * 1024;  // one CTA per SM: each holds all of its tensor memory

struct Bars {
  uint64_t *full, *empty, *s_full, *p_full, *r_full, *g_done, *a_ready, *o_done, *drain;
  uint32_t* tmem;
  volatile int* abort;
  __device__ explicit Bars(uint8_t* p) {
    uint64_t* b = reinterpret_cast<uint64_t*>(p);
    full = b;            // [8] a stage's copies landed
    empty = b + 8;       // [8] every reader is done with the stage
    p_full = b + 16;     // [8] tile g's 128 threads wrote its P / dL (g % 8: a tile is waited for
                         // before the eighth one after it has a stage)
    s_full = b + 24;     // [2] scores and dP of the buffer's tile
    r_full = b + 26;     // [2] its 128 threads hold the tile's scores and dP in registers
    g_done = b + 28;     // [3] the gradient products from a slot of dL (or, over the scores, from a buffer)
    a_ready = b + 31;    // kept operands staged, accumulators read (256 threads)
    o_done = b + 32;     // the item's last MMA
    drain = b + 33;      // [2] an issuing warp's last MMA
    tmem = reinterpret_cast<uint32_t*>(b + 35);
    abort = reinterpret_cast<volatile int*>(b + 36);
  }
  __device__ void init() {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kTileBars; ++i) mbar_init(&p_full[i], kCompute / 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&r_full[i], kCompute / 2);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&g_done[i], 1);
    mbar_init(a_ready, kCompute);
    mbar_init(o_done, 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort = 0;
    fence_mbar_init();
  }
};

// This warp's index, known to be the same in all its lanes: branches on it stay
// uniform, so the issuing warp's operands live in uniform registers (measured:
// the ten score products of a tile issue in 390 cycles instead of 665).
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

// A bounded wait of a whole warp, with one answer; of one barrier, or of two at
// once. What runs when a barrier is not complete yet stays out of line: the
// issuing warp passes through several waits per tile and is slowed by what it
// has to fetch.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_slow(bar, parity, abort);
}
__device__ __forceinline__ bool wait_warp(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, volatile int* abort) {
  const bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
  if (__all_sync(0xffffffffu, r0 && r1)) return true;
  return wait_slow(b0, p0, abort) && wait_slow(b1, p1, abort);
}

// A place in the ring of stages: the slot, and the parity of its round.
struct Ring {
  int n, s;
  uint32_t ph = 0;
  __device__ Ring(int stages, int first) : n(stages), s(first) {}
  __device__ void step(int k) {
    s += k;
    if (s >= n) {
      s -= n;
      ph ^= 1;
    }
  }
};

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
  for (int s = 0; s < stages && s < issued; ++s) mbar_wait(&b.full[s], ((issued - 1 - s) / stages) & 1, &never);
}
__device__ __forceinline__ void drain_mma(Bars& b, int which = 0) {
  mma_commit_lead(&b.drain[which], elect_one());
  volatile int never = 0;
  mbar_wait(&b.drain[which], 0, &never);
}

// Tensor memory of rows_kernel and dbias_kernel; cols_kernel sets its own
// accumulator columns.
constexpr int kBuf = 128;         // columns per buffer: scores [0, 64), dP [64, 128)
constexpr int kAcc = 256;
constexpr int kMaxTs = 80;        // widest head dim (rounded up to 16) whose operands leave room for slots
constexpr int kRowsScratch = 2 * 3 * 2 * kRows * 4;  // [item's parity][m, l, sum][warpgroup][row] floats
constexpr int kDbiasScratch = 4 * 4 * kRows * 4;  // [LSE, D, factor, log2 sum][batch entry][row]
constexpr int kDbiasWarp = 4096;  // a warp's 32 rows of bias; also, at half the size, its piece of the result
__host__ __device__ constexpr int dbias_scratch(bool bias) {
  return kDbiasScratch + kComputeWarps * (bias ? kDbiasWarp : kDbiasWarp / 2);
}

template <bool kBin, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
rows_kernel(const Params p, const __grid_constant__ CUtensorMap tm_bias) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const Map mp = smem_map(p.d, kBias, false, kRowsScratch);
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, nt = (N + kCols - 1) / kCols;
  const int nkt = nt, T = 2 * nkt;
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
  // tensor memory: buffers, dQ, Q and dO, then (where they fit) three slots of dL
  const int q_col = kAcc + DP, do_col = q_col + DP / 2, p_col = do_col + DP / 2;
  const uint32_t tmem = begin(bar, warp);

  if (warp == kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      Ring at_ring(mp.stages, 0);
      const uint32_t bytes = 2u * mp.tile + (kBias ? kBiasBytes : 0) + (kBin ? kCols * 4 : 0);
      for (int it = 0; ok && it < n_items; ++it) {
        int bh, h, i0;
        item(it, bh, h, i0);
        for (int t = 0; t < T; ++t, ++g, at_ring.step(1)) {
          const int s = at_ring.s, j0 = (t < nkt ? t : t - nkt) * kCols;
          if (!(ok = mbar_wait(&bar.empty[s], at_ring.ph ^ 1, bar.abort))) break;  // at once in the first round
          uint8_t* st = smem + s * mp.stage;
          mbar_arrive_expect_tx(&bar.full[s], bytes);
          const size_t at = (static_cast<size_t>(bh) * nt + j0 / kCols) * (mp.tile / 2);
          bulk_load(st, p.b0 + at, mp.tile, &bar.full[s]);
          bulk_load(st + mp.tile, p.b1 + at, mp.tile, &bar.full[s]);
          if constexpr (kBias) tma_load_3d(st + 2 * mp.tile, &tm_bias, j0, i0, h, &bar.full[s]);
          if constexpr (kBin)
            bulk_load(st + mp.vec, p.ak + static_cast<size_t>(bh) * p.Npad + j0, kCols * 4, &bar.full[s]);
        }
      }
      settle(bar, g, mp.stages);
    }
  } else if (warp == kMmaWarp || warp == kGradWarp) {
    // Whole warps run this (see mma_ts_lead). One issues the scores and dP of a
    // tile once its buffer is free (slots of dL: once the tile before is in
    // registers; dL over the scores: once its dQ products are done) and its
    // stage is full; the other a tile's dQ products once its dL is written,
    // and frees the stage.
    const uint32_t lead = elect_one();
    with_channels(DP / 16, [&](auto ch) {
      constexpr int kCh = decltype(ch)::value;
      constexpr bool kSlots = kCh * 16 <= kMaxTs;
      Ring ring(mp.stages, 0);
      for (int it = 0, g = 0; it < n_items; ++it) {
        if (warp == kMmaWarp) {
          if (!wait_warp(bar.a_ready, it & 1, bar.abort)) return false;
          for (int t = 0; t < T; ++t, ++g, ring.step(1)) {
            const int b = g & 1, s = ring.s;
            uint64_t* const full = &bar.full[s];
            const uint32_t ph = ring.ph;
            if (g < 2 ? !wait_warp(full, ph, bar.abort)
                      : !wait_warp(full, ph, kSlots ? &bar.r_full[b] : &bar.g_done[b], ((g - 2) >> 1) & 1, bar.abort))
              return false;
            tc_fence_after();
            const uint32_t st = smem_u32(smem + s * mp.stage);
            issue_scores<false, kCh>(tmem + b * kBuf, tmem + q_col, st, lead);
            issue_scores<false, kCh>(tmem + b * kBuf + 64, tmem + do_col, st + mp.tile, lead);
            mma_commit_lead(&bar.s_full[b], lead);
          }
        } else {
          for (int t = 0; t < T; ++t, ++g, ring.step(1)) {
            const int b = g & 1, s = ring.s;
            const int slot = kSlots ? (it * nkt + t - nkt) % 3 : b;  // slots: by the second pass's tiles
            if (!wait_warp(&bar.p_full[g & 7], (g >> 3) & 1, bar.abort)) return false;
            tc_fence_after();
            if (t >= nkt)
              issue_grad<kCh>(tmem + kAcc, tmem + (kSlots ? p_col + slot * 32 : b * kBuf), kSlots ? 16 : 32,
                              smem_u32(smem + s * mp.stage), t > nkt, lead);
            if (!kSlots || t >= nkt) mma_commit_lead(&bar.g_done[slot], lead);
            mma_commit_lead(&bar.empty[s], lead);
          }
          mma_commit_lead(bar.o_done, lead);
        }
      }
      return true;
    });
    drain_mma(bar, warp == kGradWarp);
  } else {
    const int wg = warp >> 2;  // also this warpgroup's buffer
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + wg * kBuf, dp_col = s_col + 64;
    bool ok = true;
    // Half h (32 columns) of the tile at j0: scores as logits (columns >= N as
    // -inf) and dP.
    uint32_t xr[32], dp[32];
    Ring ring(mp.stages, wg);  // this buffer's tiles are every second one
    auto arrived = [&](int g) {
      ok = ok && (kBias || kBin ? wait_warp(&bar.s_full[wg], (g >> 1) & 1, &bar.full[ring.s], ring.ph, bar.abort)
                                : wait_warp(&bar.s_full[wg], (g >> 1) & 1, bar.abort));
      tc_fence_after();
    };
    auto half = [&](int h, int j0, float ci) {
      const uint8_t* st = smem + ring.s * mp.stage;
      uint32_t bias[16];
      tmem_ld32(s_col + 32 * h, xr);
      tmem_ld32(dp_col + 32 * h, dp);
      if constexpr (kBias) load_bias(st + 2 * mp.tile, r, h, bias);
      tmem_ld_wait();
      if (h == 1) {
        tc_fence_before();
        mbar_arrive(&bar.r_full[wg]);
      }
      logits<kBin, kBias, 32>(xr, reinterpret_cast<const float*>(st + mp.vec) + 32 * h, ci, bias);
      if (j0 + 32 * h + 32 > N) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (j0 + 32 * h + e >= N) xr[e] = 0xff800000u;
      }
    };
    for (int it = 0; it < n_items; ++it) {
      int bh, h, i0;
      item(it, bh, h, i0);
      const int row = i0 + r;
      const bool valid = row < N;
      const size_t tok = static_cast<size_t>(bh) * N + (valid ? row : 0);
      if (ok) {
        KeptRow kept;
        load_row(kept, tiled_row(wg ? p.a1 : p.a0, bh, nt, valid ? row : 0, DP), valid, DP);
        stage_row(kept, DP, lb + (wg ? do_col : q_col));
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar.a_ready);
      const float ci = !kBin ? p.cs : valid ? p.aq[static_cast<size_t>(bh) * p.Npad + row] : 0.f;
      const int g0 = it * T;

      // ---- first pass: m, l and sum exp(x - m) dP of this warpgroup's tiles
      float m = -INFINITY, l = 0.f, aD = 0.f;
      int t = wg;  // T is even, so a tile's buffer is its parity in the item
      for (; t < nkt; t += 2, ring.step(2)) {
        arrived(g0 + t);
        if (!ok) continue;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          half(hf, t * kCols, ci);
          if (hf == 1) mbar_arrive(&bar.p_full[(g0 + t) & 7]);
          const float* x = reinterpret_cast<const float*>(xr);
          float a[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a[q] = max3f(x[q], x[q + 4], x[q + 8]);
            a[q] = max3f(a[q], x[q + 12], x[q + 16]);
            a[q] = max3f(a[q], x[q + 20], x[q + 24]);
            a[q] = fmaxf(a[q], x[q + 28]);
          }
          const float mn = fmaxf(m, fmaxf(max3f(a[0], a[1], a[2]), a[3]));
          const float ms = mn == -INFINITY ? 0.f : mn;  // nothing but -inf so far: every exp is 0
          const float corr = exp2v<kBias>(make_float2(m, m), make_float2(-ms, -ms)).x;
          m = mn;
          float2 l2 = make_float2(0.f, 0.f), d2 = l2;
          const float2 nm = make_float2(-ms, -ms);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 xe = reinterpret_cast<const float2*>(xr)[e];
            const float2 ex = on_fma<kBias>(e) ? exp2v<kBias, true>(xe, nm) : exp2v<kBias>(xe, nm);
            l2 = __fadd2_rn(l2, ex);
            d2 = __ffma2_rn(ex, reinterpret_cast<const float2*>(dp)[e], d2);
          }
          l = fmaf(l, corr, l2.x + l2.y);
          aD = fmaf(aD, corr, d2.x + d2.y);
        }
      }
      // ---- the row's two partial results (one per warpgroup) joined. Items take
      // turns on two arrays: with one key tile a warpgroup may come to the next
      // item's join while a thread of the other still reads this one's.
      float* sc = reinterpret_cast<float*>(smem + mp.scratch) + (it & 1) * 6 * kRows;  // [3][2 warpgroups][128 rows]
      sc[wg * kRows + r] = m;
      sc[(2 + wg) * kRows + r] = l;
      sc[(4 + wg) * kRows + r] = aD;
      named_sync(kBar, kCompute);
      const float M = fmaxf(sc[r], sc[kRows + r]);
      // a row with nothing but -inf: no weights, so -inf makes every P 0
      float nlse = -INFINITY, nl2 = 0.f, nD = 0.f;
      if (M > -INFINITY) {
        const float2 w = exp2v<kBias>(make_float2(sc[r], sc[kRows + r]), make_float2(-M, -M));
        const float Ls = fmaf(w.x, sc[2 * kRows + r], w.y * sc[3 * kRows + r]);
        const float Ds = fmaf(w.x, sc[4 * kRows + r], w.y * sc[5 * kRows + r]);
        nl2 = -log2f(Ls);
        nlse = kBias ? -M : nl2 - M;
        nD = -(Ds / Ls);
      }
      if (wg == 0 && row < p.Npad) {
        const size_t at = static_cast<size_t>(bh) * p.Npad + row;
        p.nlse[at] = valid ? nlse : -INFINITY;
        p.nD[at] = valid ? nD : 0.f;
        if (kBias) p.nl2[at] = valid ? nl2 : 0.f;
      }
      // ---- second pass: dL (binary: times alpha_k) as bf16 into its slot, or
      // over the scores
      const float2 nlse2 = make_float2(nlse, nlse), nl22 = make_float2(nl2, nl2), nD2 = make_float2(nD, nD);
      for (; t < T; t += 2, ring.step(2)) {
        const int g = g0 + t;
        arrived(g);
        if (!ok) continue;
        const float* ak = reinterpret_cast<const float*>(smem + ring.s * mp.stage + mp.vec);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          half(hf, (t - nkt) * kCols, ci);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 xe = reinterpret_cast<const float2*>(xr)[e];
            const float2 P = on_fma<kBias>(e) ? exp2v<kBias, true>(xe, nlse2, nl22) : exp2v<kBias>(xe, nlse2, nl22);
            float2 dl = __fmul2_rn(P, __fadd2_rn(reinterpret_cast<const float2*>(dp)[e], nD2));
            if constexpr (kBin) dl = __fmul2_rn(dl, *reinterpret_cast<const float2*>(ak + 32 * hf + 2 * e));
            pk[e] = pack_bf16x2(dl.x, dl.y);
          }
          if (DP <= kMaxTs) {
            // The slot's last dQ products, those of tile n - 3 of the second
            // passes, are done with it. (Tile n - 6's are: two tiles ago this
            // warpgroup waited for tile n - 5's, so the parity tells the two apart.)
            const int n = it * nkt + t - nkt;
            if (hf == 0 && n >= 3) {
              if (!(ok = wait_warp(&bar.g_done[n % 3], (n / 3 - 1) & 1, bar.abort))) break;
              tc_fence_after();
            }
            tmem_st16(lb + p_col + (n % 3) * 32 + 16 * hf, pk);
          } else {
            tmem_st16(s_col + 32 * hf, pk);
          }
        }
        if (!ok) continue;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[g & 7]);
      }
      ok = ok && wait_warp(bar.o_done, it & 1, bar.abort);
      tc_fence_after();
      for (int c0 = 32 * wg; ok && c0 < d; c0 += 64) store_row(lb + kAcc, p.out, p.g0 + tok * d, valid, c0, d);
    }
  }
  end(tmem, warp);
}

// kSS: the kept operands (K and V) in shared memory, for head dims whose
// operands and accumulators do not all fit in tensor memory (2 buffers of 128
// columns + 3 DP > 512).
template <bool kBin, bool kBias, bool kSS>
__global__ void __launch_bounds__(kThreads, 1)
cols_kernel(const Params p, const __grid_constant__ CUtensorMap tm_bias) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const Map mp = smem_map(p.d, kBias, kSS, 0);
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, nt = (N + kCols - 1) / kCols;
  const int T = nt;
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
      int g = 0;
      Ring at_ring(mp.stages, 0);
      const uint32_t bytes = 2u * mp.tile + (kBias ? kBiasBytes + kCols * 4 : 0) + (kBin ? 3 : 2) * kCols * 4;
      for (int it = 0; ok && it < n_items; ++it) {
        int bh, h, j0;
        item(it, bh, h, j0);
        for (int t = 0; t < T; ++t, ++g, at_ring.step(1)) {
          const int s = at_ring.s, i0 = t * kCols;
          if (!(ok = mbar_wait(&bar.empty[s], at_ring.ph ^ 1, bar.abort))) break;  // at once in the first round
          uint8_t* st = smem + s * mp.stage;
          mbar_arrive_expect_tx(&bar.full[s], bytes);
          const size_t tl = (static_cast<size_t>(bh) * nt + t) * (mp.tile / 2);
          bulk_load(st, p.b0 + tl, mp.tile, &bar.full[s]);
          bulk_load(st + mp.tile, p.b1 + tl, mp.tile, &bar.full[s]);
          if constexpr (kBias)
            for (int u = 0; u < 2; ++u)
              tma_load_3d(st + 2 * mp.tile + u * kBiasPanel, &tm_bias, j0 + 64 * u, i0, h, &bar.full[s]);
          const size_t at = static_cast<size_t>(bh) * p.Npad + i0;
          bulk_load(st + mp.vec, p.nlse + at, kCols * 4, &bar.full[s]);
          bulk_load(st + mp.vec + 256, p.nD + at, kCols * 4, &bar.full[s]);
          if constexpr (kBin) bulk_load(st + mp.vec + 512, p.aq + at, kCols * 4, &bar.full[s]);
          if constexpr (kBias) bulk_load(st + mp.vec + 768, p.nl2 + at, kCols * 4, &bar.full[s]);
        }
      }
      settle(bar, g, mp.stages);
    }
  } else if (warp == kMmaWarp) {
    // the whole warp runs this (see mma_ts_lead)
    const uint32_t lead = elect_one();
    with_channels(DP / 16, [&](auto ch) {
      constexpr int kCh = decltype(ch)::value;
      if constexpr (kSS == (kCh * 16 > kMaxTs)) {
        const uint32_t kept = smem_u32(smem + mp.kept);
        Ring ring(mp.stages, 0), last(mp.stages, 0);  // the scores' stage, the gradient products'
        for (int it = 0; it < n_items; ++it) {
          if (!wait_warp(bar.a_ready, it & 1, bar.abort)) return false;
          tc_fence_after();
          for (int t = 0; t < T + 2; ++t) {
            const int g = it * T + t, b = g & 1;
            // stage full, and P and dL of the tile before last written
            uint64_t* const full = &bar.full[ring.s];
            uint64_t* const prev = &bar.p_full[(g - 2) & 7];
            const uint32_t ph = ring.ph, pp = ((g - 2) >> 3) & 1;
            if (t < 2       ? t < T && !wait_warp(full, ph, bar.abort)
                : t < T     ? !wait_warp(full, ph, prev, pp, bar.abort)
                            : !wait_warp(prev, pp, bar.abort))
              return false;
            tc_fence_after();
            if (t >= 2) {
              const uint32_t st = smem_u32(smem + last.s * mp.stage);
              issue_grad<kCh>(tmem + dv_col, tmem + b * kBuf, 32, st + mp.tile, t > 2, lead);
              issue_grad<kCh>(tmem + dk_col, tmem + b * kBuf + 64, 32, st, t > 2, lead);
              mma_commit_lead(&bar.empty[last.s], lead);
              last.step(1);
            }
            if (t < T) {
              const uint32_t st = smem_u32(smem + ring.s * mp.stage);
              issue_scores<kSS, kCh>(tmem + b * kBuf, kSS ? kept : tmem + k_col, st, lead);
              issue_scores<kSS, kCh>(tmem + b * kBuf + 64, kSS ? kept + 2 * mp.tile : tmem + v_col, st + mp.tile, lead);
              mma_commit_lead(&bar.s_full[b], lead);
              ring.step(1);
            }
          }
          mma_commit_lead(bar.o_done, lead);
        }
      }
      return true;
    });
    drain_mma(bar);
  } else if (warp < kComputeWarps) {
    const int wg = warp >> 2;  // also this warpgroup's buffer
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + wg * kBuf, dp_col = s_col + 64;
    // this thread's key in the bias boxes: byte offset of (query row 0, key r),
    // before the row's swizzle of its 16-byte units
    const int bkey = (r >> 6) * kBiasPanel + (r & 7) * 2, bunit = (r & 63) >> 3;
    bool ok = true;
    Ring ring(mp.stages, wg);  // this buffer's tiles are every second one
    for (int it = 0; it < n_items; ++it) {
      int bh, h, j0;
      item(it, bh, h, j0);
      const int key = j0 + r;
      const bool valid = key < N;
      const size_t tok = static_cast<size_t>(bh) * N + (valid ? key : 0);
      if (ok) {
        KeptRow kept;
        load_row(kept, tiled_row(wg ? p.a1 : p.a0, bh, nt, valid ? key : 0, DP), valid, DP);
        if constexpr (kSS) stage_row_smem(kept, DP, smem + mp.kept + wg * 2 * mp.tile, r);
        else stage_row(kept, DP, lb + (wg ? v_col : k_col));
      }
      if constexpr (kSS) fence_proxy_async_smem();
      else tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar.a_ready);
      const float akj = kBin && valid ? p.ak[static_cast<size_t>(bh) * p.Npad + key] : 0.f;
      const int g0 = it * T;
      for (int t = (g0 & 1) == wg ? 0 : 1; t < T; t += 2, ring.step(2)) {  // this buffer's tiles
        const int g = g0 + t;
        ok = ok && wait_warp(&bar.s_full[wg], (g >> 1) & 1, &bar.full[ring.s], ring.ph, bar.abort);
        if (!ok) continue;
        tc_fence_after();
        const uint8_t* st = smem + ring.s * mp.stage;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // -LSE; -D 64 floats on, c alpha_q 128, -log2 sum 192
          const float* vec = reinterpret_cast<const float*>(st + mp.vec) + 32 * hf;
          const uint8_t* bt = st + 2 * mp.tile + bkey + 32 * hf * 128;
          uint32_t xr[32], dp[32];
          tmem_ld32(s_col + 32 * hf, xr);
          tmem_ld32(dp_col + 32 * hf, dp);
          tmem_ld_wait();
          uint32_t pp[16], pd[16];
#pragma unroll
          for (int e2 = 0; e2 < 8; ++e2) {
            auto four = [&](int at) { return *reinterpret_cast<const float4*>(vec + at + 4 * e2); };
            const float4 nlse4 = four(0), nD4 = four(64);
            float4 ci4 = make_float4(p.cs, p.cs, p.cs, p.cs), nl24 = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (kBin) ci4 = four(128);
            if constexpr (kBias) nl24 = four(192);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int e = 2 * e2 + q;
              auto two = [&](const float4& v) { return q ? make_float2(v.z, v.w) : make_float2(v.x, v.y); };
              const float2 ci = two(ci4);
              float2 x = reinterpret_cast<float2*>(xr)[e];
              if constexpr (kBin) x = __fmul2_rn(x, make_float2(akj, akj));
              if constexpr (kBias) {
                auto at = [&](int i) {  // bias of query row i of the half, this thread's key
                  return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(
                                             bt + i * 128 + ((bunit ^ (i & 7)) << 4))) << 16);
                };
                x = __ffma2_rn(x, ci, make_float2(at(2 * e), at(2 * e + 1)));
              } else {
                x = __fmul2_rn(x, ci);
              }
              const float2 P = on_fma<kBias>(e) ? exp2v<kBias, true>(x, two(nlse4), two(nl24))
                                         : exp2v<kBias>(x, two(nlse4), two(nl24));
              float2 dl = __fmul2_rn(P, __fadd2_rn(reinterpret_cast<float2*>(dp)[e], two(nD4)));
              if constexpr (kBin) dl = __fmul2_rn(dl, ci);
              pp[e] = pack_bf16x2(P.x, P.y);
              pd[e] = pack_bf16x2(dl.x, dl.y);
            }
          }
          tmem_st16(s_col + 32 * hf, pp);
          tmem_st16(dp_col + 32 * hf, pd);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[g & 7]);
      }
      ok = ok && wait_warp(bar.o_done, it & 1, bar.abort);
      tc_fence_after();
      for (int c0 = 32 * wg; ok && c0 < d; c0 += 64) {
        store_row(lb + dv_col, 1.f, p.g0 + tok * d, valid, c0, d);
        store_row(lb + dk_col, p.out, p.g1 + tok * d, valid, c0, d);
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
__global__ void __launch_bounds__(kThreadsDbias, 1)
dbias_kernel(const Params p, const __grid_constant__ CUtensorMap tm_bias) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const Map mp = smem_map(p.d, kBias, false, dbias_scratch(kBias));
  Bars bar(smem + mp.bars);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int N = p.N, d = p.d, DP = (d + 15) / 16 * 16, nt = (N + kCols - 1) / kCols;
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
      Ring at_ring(mp.stages, 0);
      for (int it = 0; ok && it < n_items; ++it) {
        const Item x = item(it);
        for (int ch = x.ch0; ok && ch < x.ch1; ++ch) {
          const int nb = batch(ch);
          for (int pr = x.pr0; ok && pr < x.pr1; ++pr) {
            for (int u = 0; u < 2 * nb; ++u, ++g, at_ring.step(1)) {
              const int s = at_ring.s, j0 = (2 * pr + (u & 1)) * kCols;
              const int bh = (ch * p.nb + (u >> 1)) * p.H + x.h;
              if (!(ok = mbar_wait(&bar.empty[s], at_ring.ph ^ 1, bar.abort))) break;  // at once in the first round
              const bool with_bias = kBias && u < 2;  // the first entry's tiles bring the bias
              // a tile wholly beyond N (the last pair's second) is not there: the
              // stage keeps what it held, and what comes of it is not stored
              const bool in = j0 < N;
              uint8_t* st = smem + s * mp.stage;
              const uint32_t bytes = (in ? 2u * mp.tile + (kBin ? kCols * 4 : 0) : 0) + (with_bias ? kBiasBytes : 0);
              if (bytes) mbar_arrive_expect_tx(&bar.full[s], bytes);
              else mbar_arrive(&bar.full[s]);
              if (in) {
                const size_t at = (static_cast<size_t>(bh) * nt + j0 / kCols) * (mp.tile / 2);
                bulk_load(st, p.b0 + at, mp.tile, &bar.full[s]);
                bulk_load(st + mp.tile, p.b1 + at, mp.tile, &bar.full[s]);
                if constexpr (kBin)
                  bulk_load(st + mp.vec, p.ak + static_cast<size_t>(bh) * p.Npad + j0, kCols * 4, &bar.full[s]);
              }
              if (with_bias) tma_load_3d(st + 2 * mp.tile, &tm_bias, j0, x.i0, x.h, &bar.full[s]);
            }
          }
        }
      }
      settle(bar, g, mp.stages);
    }
  } else if (warp == kMmaWarp) {
    // the whole warp runs this (see mma_ts_lead)
    const uint32_t lead = elect_one();
    with_channels(DP / 16, [&](auto ch16) {
      constexpr int kCh = decltype(ch16)::value;
      int g0 = 0, staged = 0;
      Ring ring(mp.stages, 0), last(mp.stages, 0);
      for (int it = 0; it < n_items; ++it) {
        const Item x = item(it);
        for (int ch = x.ch0; ch < x.ch1; ++ch, ++staged) {
          const int nb = batch(ch), T = (x.pr1 - x.pr0) * 2 * nb;
          if (!wait_warp(bar.a_ready, staged & 1, bar.abort)) return false;
          tc_fence_after();
          int e = 0;  // batch entry of the chunk
          for (int t = 0; t < T + 2; ++t) {
            const int g = g0 + t, b = g & 1;
            uint64_t* const full = &bar.full[ring.s];
            uint64_t* const prev = &bar.p_full[(g - 2) & 7];
            const uint32_t ph = ring.ph, pp = ((g - 2) >> 3) & 1;
            if (t < 2       ? t < T && !wait_warp(full, ph, bar.abort)
                : t < T     ? !wait_warp(full, ph, prev, pp, bar.abort)
                            : !wait_warp(prev, pp, bar.abort))
              return false;
            tc_fence_after();
            if (t >= 2) {
              // its MMAs were complete before the threads read them
              if (lane == 0) mbar_arrive(&bar.empty[last.s]);
              last.step(1);
            }
            if (t < T) {
              const uint32_t st = smem_u32(smem + ring.s * mp.stage);
              issue_scores<false, kCh>(tmem + b * kBuf, tmem + kAcc + e * DP, st, lead);
              issue_scores<false, kCh>(tmem + b * kBuf + 64, tmem + kAcc + e * DP + DP / 2, st + mp.tile, lead);
              mma_commit_lead(&bar.s_full[b], lead);
              ring.step(1);
              if (b == 1) e = e + 1 == nb ? 0 : e + 1;
            }
          }
          g0 += T;
        }
      }
      return true;
    });
    drain_mma(bar);
  } else if (warp < kComputeWarps) {
    const int wg = warp >> 2;  // also this warpgroup's buffer
    const int r = ((warp & 3) << 5) | lane;
    const uint32_t lb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lb + wg * kBuf, dp_col = s_col + 64;
    float* sc = reinterpret_cast<float*>(smem + mp.scratch);  // [-LSE, -D, ci, -log2 sum][entry of the chunk][row]
    uint8_t* const stg = smem + mp.scratch + kDbiasScratch + warp * (kBias ? kDbiasWarp : kDbiasWarp / 2);
    uint8_t* const own = stg + lane * 16;  // this thread's bias: 16-byte units 512 apart
    bool ok = true;
    int g = wg;
    Ring ring(mp.stages, wg);
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
          // warpgroup 0 the chunk's rows of q, 1 those of dO: half a row of two
          // entries at a time
          for (int e = 0; e < nb; e += 2) {
            for (int g0 = 0; g0 < DP / 8; g0 += 8) {
              uint4 v[2][8];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint4* src = tiled_row(wg ? p.a1 : p.a0, (ch * p.nb + e + k) * p.H + x.h, nt, row, DP);
#pragma unroll
                for (int g = 0; g < 8; ++g)
                  v[k][g] = valid && e + k < nb && g0 + g < DP / 8 ? __ldg(src + (g0 + g) * kCols) : make_uint4(0, 0, 0, 0);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int g = 0; g < 8; g += 2)
                  if (e + k < nb && g0 + g < DP / 8) {
                    const uint32_t w[8] = {v[k][g].x,     v[k][g].y,     v[k][g].z,     v[k][g].w,
                                           v[k][g + 1].x, v[k][g + 1].y, v[k][g + 1].z, v[k][g + 1].w};
                    tmem_st8(lb + kAcc + (e + k) * DP + (wg ? DP / 2 : 0) + 4 * (g0 + g), w);
                  }
            }
          }
        }
        for (int u = wg; u < nb; u += 2) {
          const size_t at = (static_cast<size_t>(ch * p.nb + u) * p.H + x.h) * p.Npad + row;
          sc[u * kRows + r] = valid ? p.nlse[at] : -INFINITY;
          sc[(4 + u) * kRows + r] = valid ? p.nD[at] : 0.f;
          sc[(8 + u) * kRows + r] = !kBin ? p.cs : valid ? p.aq[at] : 0.f;
          if (kBias) sc[(12 + u) * kRows + r] = valid ? p.nl2[at] : 0.f;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar.a_ready);
        named_sync(kBar, kCompute);  // the row vectors are in place
        const bool first = ch == x.ch0, last = ch + 1 == x.ch1;
        for (int pr = x.pr0; pr < x.pr1; ++pr) {
          float2 acc[2][16];
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = make_float2(0.f, 0.f);
          for (int b = 0; b < nb; ++b, g += 2, ring.step(2)) {
            ok = ok && wait_warp(&bar.s_full[wg], (g >> 1) & 1, &bar.full[ring.s], ring.ph, bar.abort);
            if (!ok) continue;
            tc_fence_after();
            const uint8_t* st = smem + ring.s * mp.stage;
            if (kBias && b == 0) {
              // kept for the other entries; in registers it would spill
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<uint4*>(own + u * 512) =
                    *reinterpret_cast<const uint4*>(st + 2 * mp.tile + r * 128 + ((u ^ (r & 7)) << 4));
            }
            const float nlse = sc[b * kRows + r], nD = sc[(4 + b) * kRows + r], ci = sc[(8 + b) * kRows + r];
            const float nl2 = kBias ? sc[(12 + b) * kRows + r] : 0.f;
            const float* ak = reinterpret_cast<const float*>(st + mp.vec);
#pragma unroll
            for (int q = 0; q < 8; ++q) {  // 8 columns
              uint32_t xr[8], dp[8];
              tc2::tmem_ld8(s_col + 8 * q, xr);
              tc2::tmem_ld8(dp_col + 8 * q, dp);
              tmem_ld_wait();
              uint4 bias = make_uint4(0, 0, 0, 0);
              if constexpr (kBias) bias = *reinterpret_cast<const uint4*>(own + q * 512);
              const uint32_t b8[4] = {bias.x, bias.y, bias.z, bias.w};
              logits<kBin, kBias, 8>(xr, ak + 8 * q, ci, b8);
              if (q == 7) {  // all of the tile is in registers
                tc_fence_before();
                mbar_arrive(&bar.p_full[g & 7]);
              }
              float2* to = acc[q >> 2] + 4 * (q & 3);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 P =
                    exp2v<kBias>(reinterpret_cast<float2*>(xr)[e], make_float2(nlse, nlse), make_float2(nl2, nl2));
                to[e] = __ffma2_rn(P, __fadd2_rn(reinterpret_cast<float2*>(dp)[e], make_float2(nD, nD)), to[e]);
              }
            }
          }
          if (!ok) continue;
          __syncwarp();  // the lanes are done with their bias
          // A warp's 32 rows of 64 bytes go through shared memory (2 KB,
          // 16-byte units swizzled by the row), so that a store writes whole
          // 64-byte pieces of a few rows instead of 16 bytes of 32 rows.
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float* sum = reinterpret_cast<const float*>(acc[q]);
            const int j0 = (2 * pr + wg) * kCols + 32 * q;  // the half's first column
            auto unit = [&](int row, int u) { return stg + row * 64 + ((u ^ ((row >> 1) & 3)) << 4); };
            const int r0 = x.i0 + (warp & 3) * 32;
            const size_t base = (static_cast<size_t>(x.h) * N + r0) * N + j0;  // of the warp's first row
            if (first && last && p.nsplit == 1) {
  #pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(unit(lane, k)) =
                    make_uint4(pack_bf16x2(sum[8 * k], sum[8 * k + 1]), pack_bf16x2(sum[8 * k + 2], sum[8 * k + 3]),
                               pack_bf16x2(sum[8 * k + 4], sum[8 * k + 5]), pack_bf16x2(sum[8 * k + 6], sum[8 * k + 7]));
              __syncwarp();
              if (N % 8 == 0) {
                const int u = lane & 3;
  #pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int row = 8 * k + (lane >> 2);
                  if (r0 + row < N && j0 + 8 * u < N)
                    *reinterpret_cast<uint4*>(p.g0 + base + static_cast<size_t>(row) * N + 8 * u) =
                        *reinterpret_cast<const uint4*>(unit(row, u));
                }
              } else {
                for (int row = 0; row < 32 && r0 + row < N; ++row)
                  if (j0 + lane < N)
                    p.g0[base + static_cast<size_t>(row) * N + lane] =
                        reinterpret_cast<const uint16_t*>(unit(row, lane >> 3))[lane & 7];
              }
              __syncwarp();
              continue;
            }
            // fp32 sums over chunks, 16 columns at a time; each element is read,
            // added to and written by the same thread in every chunk
            float* part = p.part + static_cast<size_t>(x.split) * p.H * N * N + base;
            const bool round = last && p.nsplit == 1;
  #pragma unroll
            for (int h = 0; h < 2; ++h) {
  #pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(unit(lane, k)) = make_float4(sum[16 * h + 4 * k], sum[16 * h + 4 * k + 1],
                                                                        sum[16 * h + 4 * k + 2], sum[16 * h + 4 * k + 3]);
              __syncwarp();
              const int c0 = 16 * h + (lane & 15);
  #pragma unroll 4
              for (int k = 0; k < 16; ++k) {
                const int row = 2 * k + (lane >> 4);
                if (r0 + row < N && j0 + c0 < N) {
                  const size_t at = static_cast<size_t>(row) * N + c0;
                  float v = reinterpret_cast<const float*>(unit(row, (lane & 15) >> 2))[lane & 3];
                  if (!first) v += part[at];
                  if (round) p.g0[base + at] = float_to_bf16_bits(v);
                  else part[at] = v;
                }
              }
              __syncwarp();
            }
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

// Lays [BH][N][d] tensors out in tiles, [BH][nt][DP / 8 groups][64 rows][8
// channels] with zeros for rows >= N and channels >= d; blockIdx.y: which of
// four. A tensor comes as bf16 rows or, sign words, as +-1. Eight rows of four
// groups per warp, so that both sides move 64 bytes or more at a time.
struct TileArgs {
  const uint16_t* rows[4];   // null: bits
  const uint32_t* bits[4];
  uint16_t* out[4];
};
__global__ void __launch_bounds__(256) tile_kernel(const TileArgs a, int N, int d, int nt, long long units) {
  const int y = blockIdx.y, groups = (d + 15) / 16 * 2, quads = (groups + 3) / 4;
  const uint16_t* rows = a.rows[y];
  const uint32_t* bits = a.bits[y];
  uint4* out = reinterpret_cast<uint4*>(a.out[y]);
  const int lane = threadIdx.x & 31, W = words_for(d);
  // a unit: eight rows of four groups
  for (long long u = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += gridDim.x * 8ll) {
    const int gq = static_cast<int>(u % quads);
    const long long ro = u / quads;  // eight rows
    const long long tile = ro / (kCols / 8);
    const int r = static_cast<int>(ro % (kCols / 8)) * 8 + (lane & 7), g = 4 * gq + (lane >> 3);
    const long long bh = tile / nt;
    const int n = static_cast<int>(tile % nt) * kCols + r;
    if (g >= groups) continue;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n < N && 8 * g < d) {
      const size_t tok = static_cast<size_t>(bh) * N + n;
      if (rows) {
        v = __ldg(reinterpret_cast<const uint4*>(rows + tok * d) + g);
      } else {
        const uint32_t byte = __ldg(bits + tok * W + (g >> 2)) >> (8 * (g & 3));
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // bf16 1.0 is 0x3F80, -1.0 is 0xBF80
          w[e] = 0xBF80BF80u ^ (((byte >> (2 * e)) & 1u) << 15) ^ (((byte >> (2 * e + 1)) & 1u) << 31);
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    out[(tile * groups + g) * kCols + r] = v;
  }
}
// alpha with rows of N padded to Npad (zeros): alpha_q times c and the units.
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
// A bias [H][N][N] (rows ld apart) as boxes of 64 keys x box_rows rows; 128-byte
// swizzle, zeros outside.
inline bool make_bias_map(CUtensorMap* tm, const uint16_t* base, cuuint64_t N, cuuint64_t ld, cuuint64_t H,
                          cuuint32_t box_rows, std::string* msg) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) {
    *msg = "cuTensorMapEncodeTiled entry point unavailable";
    return false;
  }
  const cuuint32_t es[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {N, N, H};
  const cuuint64_t strides[2] = {ld * 2, N * ld * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  CUresult rc = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (rc != CUDA_SUCCESS) {
    *msg = "tensor map (bias) rejected: " + std::to_string(rc);
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

// How dbias is cut up: the batch in chunks of nb entries; then the key splits and
// chunk splits whose slowest CTA of a 148-SM part has the least to do, counted in
// tiles: 2 nb per pair of key tiles and chunk, about 4 nb for staging a chunk's
// operands, 8 for an item. A chunk split costs an fp32 array written and read, so
// it has to gain a tenth.
struct DbiasPlan {
  int nb, nchunks, nsplit, jsplit, items;
};
inline DbiasPlan dbias_plan(int B, int H, int N, int d) {
  DbiasPlan q{};
  q.nb = dbias_batch(d) < B ? dbias_batch(d) : B;
  q.nchunks = (B + q.nb - 1) / q.nb;
  const long long base = static_cast<long long>((N + kRows - 1) / kRows) * H;
  const int npairs = ((N + kCols - 1) / kCols + 1) / 2;
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  double best = 0;
  for (int ns = 1; ns <= q.nchunks && ns <= 16; ++ns) {
    for (int js = 1; js <= npairs && js <= 32; ++js) {
      const long long item = up(q.nchunks, ns) * q.nb * (2 * up(npairs, js) + 4) + 8;
      const double cost = static_cast<double>(up(base * ns * js, 148) * item) * (ns > 1 ? 1.1 + 0.01 * ns : 1.0);
      if (q.items == 0 || cost < best) {
        best = cost;
        q.nsplit = ns;
        q.jsplit = js;
        q.items = static_cast<int>(base * ns * js);
      }
    }
  }
  return q;
}

inline size_t r256(size_t x) { return (x + 255) / 256 * 256; }
inline int npad_for(int N) { return (N + kCols - 1) / kCols * kCols; }

// The workspace of a call, parts rounded up to 256 bytes.
struct Ws {
  size_t nlse, nD, nl2, bias, tiled[4], aq, ak, part, total;
};
inline Ws workspace(int B, int H, int N, int d, bool bin, bool bias, bool dbias) {
  const size_t rows = static_cast<size_t>(B) * H * npad_for(N) * 4, 
               x = static_cast<size_t>(B) * H * npad_for(N) * ((d + 15) / 16 * 16) * 2;
  const DbiasPlan q = dbias ? dbias_plan(B, H, N, d) : DbiasPlan{};
  Ws w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += r256(bytes);
    return here;
  };
  w.nlse = take(rows);
  w.nD = take(rows);
  w.nl2 = take(bias ? rows : 0);
  w.bias = take(bias && N % 8 ? static_cast<size_t>(H) * N * ((N + 7) / 8 * 8) * 2 : 0);
  for (size_t& t : w.tiled) t = take(x);
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
template <bool kBin, bool kBias>
inline int run(Params p, const CUtensorMap& bias_rows, const CUtensorMap& bias_cols, uint16_t* const (&tiled)[4], float c,
               uint16_t* dq, uint16_t* dk, uint16_t* dv, uint16_t* dbias, cudaStream_t st,
               std::string* msg) {
  const int nsm = sm_count(), nt = (p.N + kRows - 1) / kRows;
  auto grid = [&](int items) { return static_cast<unsigned>(items < nsm ? items : nsm); };
  auto bytes = [](const Map& m) { return m.bytes > kMinSmem ? m.bytes : kMinSmem; };
  {
    static std::atomic<uint64_t> done{0};
    if (!set_smem(rows_kernel<kBin, kBias>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
    Params r = p;
    r.a0 = tiled[0];  // q, k, v, dO
    r.a1 = tiled[3];
    r.b0 = tiled[1];
    r.b1 = tiled[2];
    r.out = c;
    r.g0 = dq;
    r.items = p.B * p.H * nt;
    rows_kernel<kBin, kBias><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, false, kRowsScratch)),
                               st>>>(r, bias_rows);
    if (!launched("rows_kernel", msg)) return BINATTN_ERR_CUDA;
  }
  {
    Params r = p;
    r.a0 = tiled[1];
    r.a1 = tiled[2];
    r.b0 = tiled[0];
    r.b1 = tiled[3];
    r.out = kBin ? (kBias ? 1.f : kLn2) : c;  // binary: c alpha_q (and log2 e) are already in dL
    r.g0 = dv;
    r.g1 = dk;
    r.items = p.B * p.H * nt;
    if (p.d <= kMaxTs) {
      static std::atomic<uint64_t> done{0};
      if (!set_smem(cols_kernel<kBin, kBias, false>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
      cols_kernel<kBin, kBias, false><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, false, 0)), st>>>(r, bias_cols);
    } else {
      static std::atomic<uint64_t> done{0};
      if (!set_smem(cols_kernel<kBin, kBias, true>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
      cols_kernel<kBin, kBias, true><<<grid(r.items), kThreads, bytes(smem_map(p.d, kBias, true, 0)), st>>>(r, bias_cols);
    }
    if (!launched("cols_kernel", msg)) return BINATTN_ERR_CUDA;
  }
  if (dbias) {
    const DbiasPlan plan = dbias_plan(p.B, p.H, p.N, p.d);
    static std::atomic<uint64_t> done{0};
    if (!set_smem(dbias_kernel<kBin, kBias>, kMaxSmem, done, msg)) return BINATTN_ERR_CUDA;
    Params r = p;
    r.a0 = tiled[0];  // q, k, v, dO
    r.a1 = tiled[3];
    r.b0 = tiled[1];
    r.b1 = tiled[2];
    r.g0 = dbias;
    r.items = plan.items;
    r.nb = plan.nb;
    r.nchunks = plan.nchunks;
    r.nsplit = plan.nsplit;
    r.jsplit = plan.jsplit;
    if (plan.nchunks == 1) r.part = nullptr;
    dbias_kernel<kBin, kBias><<<grid(r.items), kThreadsDbias, bytes(smem_map(p.d, kBias, false, dbias_scratch(kBias))),
                                st>>>(r, bias_rows);
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
  const float units_of_logits = bias ? 1.f : kLog2e;
  Params p;
  std::memset(&p, 0, sizeof p);
  p.B = B;
  p.H = H;
  p.N = N;
  p.d = d;
  p.Npad = npad_for(N);
  p.cs = c * units_of_logits;
  p.nlse = reinterpret_cast<float*>(ws + w.nlse);
  p.nD = reinterpret_cast<float*>(ws + w.nD);
  p.nl2 = reinterpret_cast<float*>(ws + w.nl2);
  p.part = reinterpret_cast<float*>(ws + w.part);
  auto grid = [](long long threads) { return static_cast<unsigned>(std::min<long long>((threads + 255) / 256, 148 * 8)); };
  const int nt = p.Npad / kCols;
  uint16_t* tiled[4];
  for (int i = 0; i < 4; ++i) tiled[i] = reinterpret_cast<uint16_t*>(ws + w.tiled[i]);
  const long long units = static_cast<long long>(B) * H * nt * (kCols / 8) * (((d + 15) / 16 * 2 + 3) / 4);
  const TileArgs ta{{q, k, v, dO}, {qb, kb, nullptr, nullptr}, {tiled[0], tiled[1], tiled[2], tiled[3]}};
  tile_kernel<<<dim3(grid(units * 32), 4), 256, 0, st>>>(ta, N, d, nt, units);
  if (!launched("tile_kernel", msg)) return BINATTN_ERR_CUDA;
  if (bin) {
    const long long n = static_cast<long long>(B) * H * p.Npad;
    float* aq = reinterpret_cast<float*>(ws + w.aq);
    float* ak = reinterpret_cast<float*>(ws + w.ak);
    pad_alpha_kernel<<<grid(n), 256, 0, st>>>(alpha_q, alpha_k, n, N, p.Npad, c, units_of_logits, aq, ak);
    if (!launched("pad_alpha_kernel", msg)) return BINATTN_ERR_CUDA;
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
  CUtensorMap bias_rows, bias_cols;
  std::memset(&bias_rows, 0, sizeof bias_rows);
  std::memset(&bias_cols, 0, sizeof bias_cols);
  if (bias && (!make_bias_map(&bias_rows, bias, N, ld, H, kRows, msg) ||
               !make_bias_map(&bias_cols, bias, N, ld, H, kCols, msg)))
    return BINATTN_ERR_CUDA;
  if (bin)
    return bias ? run<true, true>(p, bias_rows, bias_cols, tiled, c, dq, dk, dv, dbias, st, msg)
                : run<true, false>(p, bias_rows, bias_cols, tiled, c, dq, dk, dv, dbias, st, msg);
  return bias ? run<false, true>(p, bias_rows, bias_cols, tiled, c, dq, dk, dv, dbias, st, msg)
              : run<false, false>(p, bias_rows, bias_cols, tiled, c, dq, dk, dv, dbias, st, msg);
}

}  // namespace bt
}  // namespace binattn
