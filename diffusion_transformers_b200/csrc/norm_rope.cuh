// norm_rope.cuh — what stands between a block's Q/K projection and its
// attention: the RMS norm of every head's query and key and the rotation of
// their channel pairs by the token's position, in one pass over the
// projection's output (any token, head and batch strides); the same pass ended
// in sign bits and alpha, binattn_pack's output; and its gradient.
//
// Per row x (one token of one head, d channels), weight w and the token's
// tables cos_p, sin_p, p < R / 2:
//   r = 1 / sqrt(mean x^2 + eps),  y_c = r x_c w_c
//   z_a = y_a cos_p - y_b sin_p,  z_b = y_a sin_p + y_b cos_p
// for the pair (a, b) = (p, p + R / 2) or, interleaved, (2p, 2p + 1), and
// z_c = y_c for c >= R. Its gradient, with dz = dLoss / dz:
//   dy = dz turned back (sin -> -sin),  dw_c = sum over rows of dy_c r x_c
//   g = dy w,  dx = r (g - r x mean(g r x)).
// fp32 throughout; each result is rounded once, when it is stored.
//
// The pass is bound by memory, so the mapping keeps loads wide and the work per
// row small. A row is d / 8 chunks of 8 channels; a chunk is two quads of 4 (8
// bytes of bf16, 16 of fp32) chosen so that both members of its four pairs are in
// it. A lane has kC chunks (the largest of 3, 2, 1 that divides their number), so
// L = d / 8 / kC lanes share a row and 32 / L rows a warp. A lane's channels are
// the same in every row, so the sums of dw stay in registers. One thread
// per row, as pack_bf16_rows_kernel has it, would cost a strided view 32 cache
// lines per load. Rows are numbered (batch, token, head) with the head fastest:
// the rows a block works on share a few tokens' tables. Shapes outside d % 8 ==
// 0, R % 8 == 0 and 4-element alignment take one warp per row and scalar loads.
//
// Measured on one B200 (copies 6.5 TB/s) on the device (replayed graphs, inputs
// above L2), 2 x 16 x 4096 x 72 with R = 72, q and k: bf16 29 us, 2.6 TB/s; fp32 36 us,
// 4.2 TB/s; the gradient in bf16 52 us, 6 of them the sums of dw over the blocks, in
// fp32 85 us. Sign bits at 8 x 16 x 1024 x 72, bf16, interleaved: 37 us (770
// instructions per warp for ten rows, half of the issue slots used), against 40 for
// the norm and rotation followed by two packs; fp32 47 against 74, but bf16 in split
// pairs 40 against 39. What bounds it is issue and latency with 16 warps per SM
// (128 registers for three chunks and their angles); held to 80 registers, for
// three blocks per SM, it gained nothing. The gradient spills at three chunks (24 to
// 220 bytes a thread). The scalar kernel (rot = 36 of 72): 111 us, sign bits 122,
// gradient 150. One token of 16 heads: 2.2 us, a launch.
#pragma once
#include "common.cuh"

namespace binattn {
namespace nr {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 148 * 3;  // per tensor of a launch (blocks_for)

// Both tensors (index 0: q, 1: k; blockIdx.y) of one call. Strides in elements.
struct Params {
  const void* x[2];
  long long xb[2], xh[2], xn[2];
  const float* w[2];  // null: ones
  const float* cosv;
  const float* sinv;
  int R, per_batch;
  float eps;
  int B, H, N, d;
  void* out[2];        // norm_rope: [B,H,N,d]; backward: dx, strided
  long long ob[2], oh[2], on[2];
  uint32_t* bits[2];   // pack
  float* alpha[2];
  const void* dz[2];   // backward: [B,H,N,d]
  float* dwpart;       // backward: [2][blocks][d] partial sums, or null
};

constexpr int kOpOut = 0, kOpPack = 1, kOpBwd = 2;

__device__ __forceinline__ float ldf(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ldf(const uint16_t* p) { return bf16_bits_to_float(__ldg(p)); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }
__device__ __forceinline__ void stf(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }

// Four channels at once, as they lie in memory and widened.
template <typename T> struct Quad;
template <> struct Quad<float> {
  float4 v;
  __device__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <> struct Quad<uint16_t> {
  uint2 v;
  __device__ void load(const uint16_t* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
};
__device__ __forceinline__ void ld4(const float* p, float (&f)[4]) {
  Quad<float> q;
  q.load(p);
  q.get(f);
}
__device__ __forceinline__ void st4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void st4(uint16_t* p, float a, float b, float c, float d) {
  uint2 v;
  v.x = float_to_bf16_bits(a) | static_cast<uint32_t>(float_to_bf16_bits(b)) << 16;
  v.y = float_to_bf16_bits(c) | static_cast<uint32_t>(float_to_bf16_bits(d)) << 16;
  *reinterpret_cast<uint2*>(p) = v;
}

// The sign of z, since r > 0, is that of p1 - p2 with p1 = xa wa c and p2 = xb wb
// s. Their fp32 difference t is off by at most 2^-23 (|p1| + |p2|) and 2^-24 |t|
// from the two or three roundings, so its sign is right beyond 1e-6 (|p1| +
// |p2|) (and above the range where products underflow); closer to zero it is
// decided exactly. A product of three fp32 numbers has up to 72 bits: x w fits
// in 64-bit arithmetic, times c it is a rounded product and its rounding error,
// both exact (their lowest bit is no lower than 2^-447). Rounding is monotone, so
// the rounded products decide unless they are equal, and then the errors do.
// Equal products give zero, which counts as not negative.
__device__ __forceinline__ bool clear(float t, float p1, float p2) {
  return fabsf(t) > fmaf(1e-6f, fabsf(p1) + fabsf(p2), 1e-30f);
}
__device__ __forceinline__ bool nonneg_exact(float xa, float wa, float c, float xb, float wb, float s) {
  const double u = __dmul_rn(static_cast<double>(xa), static_cast<double>(wa)), cd = static_cast<double>(c);
  const double v = __dmul_rn(static_cast<double>(xb), static_cast<double>(wb)), sd = static_cast<double>(s);
  const double a = __dmul_rn(u, cd), b = __dmul_rn(v, sd);
  return a != b ? a > b : __fma_rn(u, cd, -a) >= __fma_rn(v, sd, -b);
}

// The token of row i (batch, token, head with the head fastest). Callers hold B * H
// and N to 65535, so every row, and a round's step beyond the last, fits 32 bits.
static_assert(65535ull * 65535 + kMaxBlocks * kWarps * 32ull <= 0xffffffffull, "rows are numbered in 32 bits");
struct Row {
  int b, h, n;
};
__device__ __forceinline__ Row row_of(unsigned i, int H, int N) {
  Row w;
  const unsigned tk = i / static_cast<unsigned>(H);  // batch * N + token
  w.h = static_cast<int>(i - tk * static_cast<unsigned>(H));
  w.b = static_cast<int>(tk / static_cast<unsigned>(N));
  w.n = static_cast<int>(tk - static_cast<unsigned>(w.b) * static_cast<unsigned>(N));
  return w;
}

// Sum over the L lanes of this lane's row (pos: its place in the row, base: the
// row's first lane), to all of them, in a fixed order.
__device__ __forceinline__ float row_sum(float v, int L, int pos, int base, bool pow2) {
  if (pow2) {
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  for (int o = 1; o < L; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, o);
    if (pos + o < L) v += u;
  }
  return __shfl_sync(0xffffffffu, v, base);
}

// T: x's type, G: dz's (backward). kInter: pairs (2p, 2p + 1). kC: chunks per lane.
template <typename T, typename G, int kOp, bool kInter, int kC>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_rows_kernel(const Params p) {
  const int t = blockIdx.y;
  const int d = p.d, H = p.H, N = p.N, half = p.R / 2, R8 = p.R / 8;
  const int L = d / 8 / kC, rpw = 32 / L;  // lanes per row, rows per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / L, pos = lane - grp * L, base = grp * L;
  const bool pow2 = (L & (L - 1)) == 0;
  const bool live = grp < rpw;  // lanes past the last whole row idle
  const T* x = static_cast<const T*>(p.x[t]);
  T* out = kOp == kOpPack ? nullptr : static_cast<T*>(p.out[t]);
  // Chunk k of this lane is chunk j = pos + k L of the row: its two quads are the
  // first and second members of four pairs, or eight consecutive channels
  // (interleaved, or not rotated).
  auto quads = [&](int k, int& ca, int& cb) {
    const int j = pos + k * L;
    const bool split = !kInter && j < R8;
    ca = split ? 4 * j : 8 * j;
    cb = split ? half + 4 * j : 8 * j + 4;
  };
  // first and second members of a chunk's four pairs
  auto members = [&](const auto& qa, const auto& qb, float (&f)[4], float (&s)[4]) {
    float a[4], b[4];
    qa.get(a);
    qb.get(b);
    if (kInter) {
      f[0] = a[0]; s[0] = a[1]; f[1] = a[2]; s[1] = a[3];
      f[2] = b[0]; s[2] = b[1]; f[3] = b[2]; s[3] = b[3];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = a[e], s[e] = b[e];
    }
  };
  // w in shared memory: it is read once per row, and registers are short
  __shared__ float4 wsm[32];
  if (threadIdx.x < d) reinterpret_cast<float*>(wsm)[threadIdx.x] = p.w[t] ? p.w[t][threadIdx.x] : 1.f;
  __syncthreads();
  auto weights = [&](int k, float (&f)[4], float (&s)[4]) {
    int ca, cb;
    quads(k, ca, cb);
    members(Quad<float>{wsm[ca / 4]}, Quad<float>{wsm[cb / 4]}, f, s);
  };
  float dwf[kC][4], dws[kC][4];
#pragma unroll
  for (int k = 0; k < kC; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) dwf[k][e] = dws[k][e] = 0.f;

  const unsigned rows = static_cast<unsigned>(p.B) * H * N;
  const float inv_d = 1.f / static_cast<float>(d);
  const unsigned step = gridDim.x * kWarps * rpw;  // rows per round
  const Row by = row_of(step, H, N);               // ... as batch entries, tokens, heads
  unsigned i = (blockIdx.x * kWarps + warp) * rpw + grp;
  Row w = row_of(i, H, N);
  // A row's x (and dz) are loaded, as they lie in memory, while the row before is
  // worked on: the bytes that are under way bound the pass.
  Quad<T> xq[2 * kC];
  Quad<G> zq[kOp == kOpBwd ? 2 * kC : 1];
  auto fetch = [&](const Row& w) {
    const T* src = x + w.b * p.xb[t] + w.h * p.xh[t] + w.n * p.xn[t];
    const G* gz = kOp == kOpBwd ? static_cast<const G*>(p.dz[t]) + ((static_cast<size_t>(w.b) * H + w.h) * N + w.n) * d : nullptr;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      int ca, cb;
      quads(k, ca, cb);
      xq[2 * k].load(src + ca);
      xq[2 * k + 1].load(src + cb);
      if constexpr (kOp == kOpBwd) {
        zq[2 * k].load(gz + ca);
        zq[2 * k + 1].load(gz + cb);
      }
    }
  };
  if (live && i < rows) fetch(w);
  // the trip count is warp-uniform: by the warp's first row
  for (unsigned i0 = i - grp; i0 < rows; i0 += step, i += step) {
    const bool in = live && i < rows;
    float xf[kC][4], xs[kC][4], cs[kC][4], sn[kC][4], zf[kC][4], zs[kC][4];
    const size_t row = (static_cast<size_t>(w.b) * H + w.h) * N + w.n;
    const size_t tok = (p.per_batch ? static_cast<size_t>(w.b) * N : 0) + w.n;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) xf[k][e] = xs[k][e] = zf[k][e] = zs[k][e] = sn[k][e] = 0.f, cs[k][e] = 1.f;
      if (in) {
        if (pos + k * L < R8) {
          ld4(p.cosv + tok * half + 4 * (pos + k * L), cs[k]);
          ld4(p.sinv + tok * half + 4 * (pos + k * L), sn[k]);
        }
        members(xq[2 * k], xq[2 * k + 1], xf[k], xs[k]);
        if constexpr (kOp == kOpBwd) {  // dz turned back
          members(zq[2 * k], zq[2 * k + 1], zf[k], zs[k]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = zf[k][e] * cs[k][e] + zs[k][e] * sn[k][e];
            zs[k][e] = zs[k][e] * cs[k][e] - zf[k][e] * sn[k][e];
            zf[k][e] = y;
          }
        }
      }
    }
    Row next = w;  // the row `step` further on
    next.h += by.h;
    next.n += by.n;
    next.b += by.b;
    if (next.h >= H) next.h -= H, ++next.n;
    if (next.n >= N) next.n -= N, ++next.b;
    if (live && i + step < rows) fetch(next);
#pragma unroll
    for (int k = 0; k < kC; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(xf[k][e], xf[k][e], fmaf(xs[k][e], xs[k][e], ss));
    const float r = rsqrtf(row_sum(ss, L, pos, base, pow2) * inv_d + p.eps);
    if constexpr (kOp == kOpBwd) {
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        float wf[4], ws[4];
        weights(k, wf, ws);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xf[k][e] *= r;
          xs[k][e] *= r;
          dwf[k][e] = fmaf(zf[k][e], xf[k][e], dwf[k][e]);
          dws[k][e] = fmaf(zs[k][e], xs[k][e], dws[k][e]);
          zf[k][e] *= wf[e];
          zs[k][e] *= ws[e];
          dot = fmaf(zf[k][e], xf[k][e], fmaf(zs[k][e], xs[k][e], dot));
        }
      }
      const float mean = row_sum(dot, L, pos, base, pow2) * inv_d;
#pragma unroll
      for (int k = 0; k < kC; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          zf[k][e] = r * (zf[k][e] - xf[k][e] * mean);
          zs[k][e] = r * (zs[k][e] - xs[k][e] * mean);
        }
    }
    if constexpr (kOp == kOpPack) {
      float sum = 0.f;
      uint32_t bits[kC];  // per chunk: the first members' signs, then the second ones'
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        bool sure = true;
        uint32_t b = 0;
        float wf[4], ws[4];
        weights(k, wf, ws);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float uf = xf[k][e] * wf[e], us = xs[k][e] * ws[e];
          const float p1 = uf * cs[k][e], p2 = us * sn[k][e], p3 = us * cs[k][e], p4 = uf * sn[k][e];
          const float tf = p1 - p2, ts = p3 + p4;
          sum += fabsf(tf) + fabsf(ts);
          sure = sure && clear(tf, p1, p2) && clear(ts, p3, p4);
          b |= (tf > 0.f ? 1u : 0u) << e | (ts > 0.f ? 16u : 0u) << e;
        }
        if (in && !sure) {  // seldom: some value of the chunk is next to zero
          b = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            b |= (nonneg_exact(xf[k][e], wf[e], cs[k][e], xs[k][e], ws[e], sn[k][e]) ? 1u : 0u) << e;
            b |= (nonneg_exact(xs[k][e], ws[e], cs[k][e], xf[k][e], wf[e], -sn[k][e]) ? 16u : 0u) << e;
          }
        }
        bits[k] = b;
      }
      const float alpha = row_sum(sum, L, pos, base, pow2) * r * inv_d;
      const int wb = 4 * words_for(d);  // bytes per row, the last ones padding
      uint8_t* dst = reinterpret_cast<uint8_t*>(p.bits[t]) + row * wb;
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        // byte j of the row's sign words: channels 8 j .. 8 j + 7
        const int j = pos + k * L;
        uint32_t byte;
        if (kInter) {
          byte = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) byte |= ((bits[k] >> e) & 1u) << (2 * e) | ((bits[k] >> (4 + e)) & 1u) << (2 * e + 1);
        } else {
          // quad q of the row is half a byte: the lower half of the chunk that has
          // it as first members, or the upper half of the one that has it second
          auto nibble = [&](int q) {
            const bool first = q < R8, second = !first && q < 2 * R8;
            const int c = first ? q : second ? q - R8 : q / 2;  // chunk
            const int ck = c / L;
            uint32_t v = 0;
#pragma unroll
            for (int kk = 0; kk < kC; ++kk) {
              const uint32_t got = __shfl_sync(0xffffffffu, bits[kk], base + c - ck * L);
              if (kk == ck) v = got;
            }
            return (first ? v : second ? v >> 4 : v >> (4 * (q & 1))) & 0xFu;
          };
          byte = nibble(2 * j) | nibble(2 * j + 1) << 4;
        }
        if (in) dst[j] = static_cast<uint8_t>(byte);
      }
      if (in && pos == 0) {
        for (int b = d / 8; b < wb; ++b) dst[b] = 0;
        p.alpha[t][row] = alpha;
      }
    } else if (in) {
      T* to = out + w.b * p.ob[t] + w.h * p.oh[t] + w.n * p.on[t];
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        float(&f)[4] = zf[k];
        float(&s)[4] = zs[k];
        if constexpr (kOp == kOpOut) {
          float wf[4], ws[4];
          weights(k, wf, ws);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float yf = xf[k][e] * r * wf[e], ys = xs[k][e] * r * ws[e];
            f[e] = yf * cs[k][e] - ys * sn[k][e];
            s[e] = yf * sn[k][e] + ys * cs[k][e];
          }
        }
        int ca, cb;
        quads(k, ca, cb);
        if (kInter) {
          st4(to + ca, f[0], s[0], f[1], s[1]);
          st4(to + cb, f[2], s[2], f[3], s[3]);
        } else {
          st4(to + ca, f[0], f[1], f[2], f[3]);
          st4(to + cb, s[0], s[1], s[2], s[3]);
        }
      }
    }
    w = next;
  }
  if constexpr (kOp == kOpBwd) {
    // the block's sums of dw: every lane group's registers, added in group order
    if (!p.dwpart) return;
    __shared__ float red[kThreads * 8 * kC];  // [group][d]: at most kThreads / L groups of 8 kC L channels
    if (live) {
      float* mine = red + (warp * rpw + grp) * d;
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        int ca, cb;
        quads(k, ca, cb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mine[kInter ? ca + 2 * e : ca + e] = dwf[k][e];
          mine[kInter ? ca + 2 * e + 1 : cb + e] = dws[k][e];
        }
      }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < d; ch += kThreads) {
      float s = 0.f;
      for (int g = 0; g < kWarps * rpw; ++g) s += red[g * d + ch];
      p.dwpart[(static_cast<size_t>(t) * gridDim.x + blockIdx.x) * d + ch] = s;
    }
  }
}

// Any d <= 128, R and alignment: one warp per row, lane l has channels l + 32 i.
template <typename T, typename G, int kOp>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const Params p, int inter) {
  const int t = blockIdx.y;
  const int d = p.d, H = p.H, N = p.N, R = p.R, half = p.R / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(p.x[t]);
  const float* wt = p.w[t];
  const unsigned rows = static_cast<unsigned>(p.B) * H * N;
  const float inv_d = 1.f / static_cast<float>(d);
  float dw[4] = {0.f, 0.f, 0.f, 0.f};
  auto all_sum = [](float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  for (unsigned i = blockIdx.x * kWarps + warp; i < rows; i += gridDim.x * kWarps) {
    const Row w = row_of(i, H, N);
    const T* src = x + w.b * p.xb[t] + w.h * p.xh[t] + w.n * p.xn[t];
    const size_t row = (static_cast<size_t>(w.b) * H + w.h) * N + w.n;
    const size_t tok = (p.per_batch ? static_cast<size_t>(w.b) * N : 0) + w.n;
    const G* gz = kOp == kOpBwd ? static_cast<const G*>(p.dz[t]) + row * d : nullptr;
    float xv[4], ss = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = lane + 32 * k;
      xv[k] = ch < d ? ldf(src + ch) : 0.f;
      ss = fmaf(xv[k], xv[k], ss);
    }
    const float r = rsqrtf(all_sum(ss) * inv_d + p.eps);
    float z[4] = {0.f, 0.f, 0.f, 0.f}, g[4] = {0.f, 0.f, 0.f, 0.f}, acc = 0.f;
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = lane + 32 * k;
      bool on = false;
      if (ch < d) {
        const float wc = wt ? __ldg(wt + ch) : 1.f;
        // the pair partner, and the angle with the sign this member takes it in:
        // z_c = y_c cos - y_partner sgn
        int pc = ch;
        float cs = 1.f, sg = 0.f;
        if (ch < R) {
          const bool first = inter ? !(ch & 1) : ch < half;
          const int pr = inter ? ch >> 1 : first ? ch : ch - half;
          pc = inter ? ch ^ 1 : first ? ch + half : ch - half;
          cs = __ldg(p.cosv + tok * half + pr);
          sg = __ldg(p.sinv + tok * half + pr);
          if (!first) sg = -sg;
        }
        if constexpr (kOp == kOpBwd) {
          // turned back: dy_c = dz_c cos + dz_partner sgn
          const float dy = ldf(gz + ch) * cs + ldf(gz + pc) * sg;
          const float xh = xv[k] * r;
          dw[k] = fmaf(dy, xh, dw[k]);
          g[k] = dy * wc;
          acc = fmaf(g[k], xh, acc);
        } else {
          const float xp = ldf(src + pc), wp = wt ? __ldg(wt + pc) : 1.f;
          const float p1 = xv[k] * wc * cs, p2 = xp * wp * sg;
          const float tv = p1 - p2;
          if constexpr (kOp == kOpPack) {
            acc += fabsf(tv);
            on = clear(tv, p1, p2) ? tv > 0.f : nonneg_exact(xv[k], wc, cs, xp, wp, sg);
          } else {
            z[k] = tv * r;
          }
        }
      }
      if constexpr (kOp == kOpPack) {
        const uint32_t b = __ballot_sync(0xffffffffu, on);
        if (lane == k) word = b;
      }
    }
    if constexpr (kOp == kOpPack) {
      const float alpha = all_sum(acc) * r * inv_d;
      const int W = words_for(d);
      if (lane < W) p.bits[t][row * W + lane] = word;
      if (lane == 0) p.alpha[t][row] = alpha;
    } else {
      if constexpr (kOp == kOpBwd) {
        const float mean = all_sum(acc) * inv_d;
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = r * (g[k] - xv[k] * r * mean);
      }
      T* dst = static_cast<T*>(p.out[t]) + w.b * p.ob[t] + w.h * p.oh[t] + w.n * p.on[t];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < d) stf(dst + lane + 32 * k, z[k]);
    }
  }
  if constexpr (kOp == kOpBwd) {
    if (!p.dwpart) return;
    __shared__ float red[kWarps][128];
#pragma unroll
    for (int k = 0; k < 4; ++k) red[warp][lane + 32 * k] = dw[k];
    __syncthreads();
    for (int ch = threadIdx.x; ch < d; ch += kThreads) {
      float s = 0.f;
      for (int g = 0; g < kWarps; ++g) s += red[g][ch];
      p.dwpart[(static_cast<size_t>(t) * gridDim.x + blockIdx.x) * d + ch] = s;
    }
  }
}

// dw of q (blockIdx.x 0) and k (1) from the blocks' partial sums, 8 channels per
// block: 32 slices of the partial sums per channel, each added in order, then the
// slices in order.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* __restrict__ part, int blocks, int d,
                                                           float* dwq, float* dwk) {
  __shared__ float red[32][8];
  const int c = threadIdx.x & 7, ch = blockIdx.y * 8 + c, slice = threadIdx.x >> 3;
  const float* src = part + static_cast<size_t>(blockIdx.x) * blocks * d;
  float s = 0.f;
  if (ch < d) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32) s += __ldg(src + static_cast<size_t>(b) * d + ch);
  }
  red[slice][c] = s;
  __syncthreads();
  float* out = blockIdx.x ? dwk : dwq;
  if (slice == 0 && ch < d && out) {
    for (int g = 1; g < 32; ++g) s += red[g][c];
    out[ch] = s;
  }
}

// Blocks per tensor of a launch: one round of rows, at most 3 blocks per SM of a
// 148-SM part and tensor (the kernels stride over the rest; the backward writes
// one row of partial sums per block).
inline int blocks_for(unsigned long long rows, int rows_per_block) {
  const unsigned long long b = (rows + rows_per_block - 1) / rows_per_block;
  return b < kMaxBlocks ? static_cast<int>(b) : kMaxBlocks;
}

// Whether the vector kernel takes the call: see the head of this file.
inline bool vec_ok(const Params& p, int es, int gs, bool bwd) {
  if (p.d % 8 || p.R % 8) return false;
  for (int t = 0; t < 2; ++t) {
    if (reinterpret_cast<uintptr_t>(p.x[t]) % (4 * es) || p.xb[t] % 4 || p.xh[t] % 4 || p.xn[t] % 4) return false;
    if (p.out[t] && (reinterpret_cast<uintptr_t>(p.out[t]) % (4 * es) || p.ob[t] % 4 || p.oh[t] % 4 || p.on[t] % 4))
      return false;
    if (bwd && reinterpret_cast<uintptr_t>(p.dz[t]) % (4 * gs)) return false;
  }
  return true;
}

template <typename T, typename G, int kOp, int kC>
inline int launch_rows(const Params& p, bool inter, cudaStream_t st) {
  const unsigned long long rows = static_cast<unsigned long long>(p.B) * p.H * p.N;
  const int blocks = blocks_for(rows, kWarps * (32 / (p.d / 8 / kC)));
  if (inter) norm_rope_rows_kernel<T, G, kOp, true, kC><<<dim3(blocks, 2), kThreads, 0, st>>>(p);
  else norm_rope_rows_kernel<T, G, kOp, false, kC><<<dim3(blocks, 2), kThreads, 0, st>>>(p);
  return blocks;
}
template <typename T, typename G, int kOp>
inline int launch(const Params& p, bool inter, bool vec, cudaStream_t st) {
  if (vec) {
    const int chunks = p.d / 8;
    if (chunks % 3 == 0) return launch_rows<T, G, kOp, 3>(p, inter, st);
    if (chunks % 2 == 0) return launch_rows<T, G, kOp, 2>(p, inter, st);
    return launch_rows<T, G, kOp, 1>(p, inter, st);
  }
  const unsigned long long rows = static_cast<unsigned long long>(p.B) * p.H * p.N;
  const int blocks = blocks_for(rows, kWarps);
  norm_rope_any_kernel<T, G, kOp><<<dim3(blocks, 2), kThreads, 0, st>>>(p, inter);
  return blocks;
}

}  // namespace nr
}  // namespace binattn
