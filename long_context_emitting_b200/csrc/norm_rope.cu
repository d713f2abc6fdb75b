// RMS norm of query and key heads and the rotation by position, in one pass.
//
// For a head row x of 128 channels, weight w and position p:
//   y = x * rsqrt(mean(x^2) + eps) * w        (y = x without a weight)
//   pair i of 64: angle a = p * inv_freq[i];  (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a)
// with j = i + 64 (half split), or channels (2i, 2i+1) (interleaved).  All of it
// is fp32 in registers, rounded once when the row is stored.
//
// The angle.  p * inv_freq in fp32 is off by p * 2^-24 radians (0.008 at a
// position of 131072), so it is formed in 64 bits as turns, reduced to
// [-1/2, 1/2] there, and only then handed to sincospif in fp32.  It is the same
// for every head of a token: a block computes its tokens' 64 pairs once, into
// shared memory, and all its heads read them.
//
// What bounds it: memory (a row is read and written once, 4 bytes per channel
// in all).  A row is 8 lanes x two 16-byte chunks, channels 8j.. and 64 + 8j..,
// so both halves of a half-split pair are in one lane and nothing is exchanged
// but the sum of squares; the lane's eight cosines and sines stay in registers
// over all heads, and the next rows are on their way while some are worked on.
// Measured on one B200: 16384 tokens x 40 heads, bfloat16 with norms, 61.5 us,
// 5.46 TB/s (83% of a plain copy's rate).  Four tokens per block: with eight the
// same, with sixteen 82 us (too few blocks); two passes of rows ahead 67 us.
// One token of 16 sequences takes 3.3 us, little more than an empty launch.
#include "common.cuh"
#include "internal.h"
#include "q4.cuh"

namespace kascade {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = kThreads / 8;  // rows a block works on at a time

struct RopeArgs {
  const uint16_t* x[2];  // q, k
  uint16_t* y[2];
  const uint16_t* w[2];  // weights, or NULL
  kascade_strides xs[2], ys[2];
  const int32_t* pos;
  const float* inv_freq;
  float eps;
  int N, Hq, H;          // tokens per sequence; query heads; all heads
  int tiles;             // token tiles per sequence
  int heads_per_block;
};

// TOK tokens x kRows / TOK heads at a time.
template <int TOK, bool F16, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  overlap_launches();
  __shared__ float2 cs[TOK][kHeadDim / 2];
  const int b = blockIdx.x / a.tiles;
  const int n0 = (blockIdx.x - b * a.tiles) * TOK;
  for (int e = threadIdx.x; e < TOK * (kHeadDim / 2); e += kThreads) {
    const int t = e / (kHeadDim / 2), i = e % (kHeadDim / 2);
    const int n = min(n0 + t, a.N - 1);
    constexpr double kInvTwoPi = 0.15915494309189533577;
    const double turns = (double)a.pos[(int64_t)b * a.N + n] * (double)a.inv_freq[i] * kInvTwoPi;
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[t][i] = make_float2(c, s);
  }
  __syncthreads();

  const int row = threadIdx.x / 8, j = threadIdx.x % 8;
  const int t = row % TOK, n = min(n0 + t, a.N - 1);
  const int h_lo = blockIdx.y * a.heads_per_block, h_hi = min(a.H, h_lo + a.heads_per_block);
  constexpr int kStep = kRows / TOK;
  float2 turn[8];  // this lane's pairs
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = cs[t][!INTER ? 8 * j + i : i < 4 ? 4 * j + i : 32 + 4 * j + i - 4];
  // The query heads of the block, then its key heads; the next rows are on their way while some are
  // worked on.  Rows past the end compute on the last one and store nothing.
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const int first = part ? max(h_lo, a.Hq) - a.Hq : h_lo, end = part ? h_hi - a.Hq : min(h_hi, a.Hq);
    if (first >= end) continue;
    const kascade_strides &xs = a.xs[part], &ys = a.ys[part];
    const uint16_t* x = a.x[part] + (int64_t)b * xs.b + (int64_t)n * xs.n + 8 * j;
    uint16_t* y = a.y[part] + (int64_t)b * ys.b + (int64_t)n * ys.n + 8 * j;
    const bool norm = a.w[part] != nullptr;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (norm) {
      w0 = ldg16(a.w[part] + 8 * j);
      w1 = ldg16(a.w[part] + 64 + 8 * j);
    }
    int h = first + row / TOK;
    const uint16_t* x0 = x + (int64_t)min(h, end - 1) * xs.h;
    uint4 c0 = load16(x0), c1 = load16(x0 + 64);
    for (int hh = first; hh < end; hh += kStep, h += kStep) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unpack2<F16>(word_of(c0, i), v[2 * i], v[2 * i + 1]);
        unpack2<F16>(word_of(c1, i), v[8 + 2 * i], v[8 + 2 * i + 1]);
      }
      if (hh + kStep < end) {
        const uint16_t* x1 = x + (int64_t)min(h + kStep, end - 1) * xs.h;
        c0 = load16(x1);
        c1 = load16(x1 + 64);
      }
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss += v[i] * v[i];
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        ss += __shfl_xor_sync(0xffffffffu, ss, 4);
        const float r = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          unpack2<F16>(word_of(w0, i), lo, hi);
          v[2 * i] *= r * lo;
          v[2 * i + 1] *= r * hi;
          unpack2<F16>(word_of(w1, i), lo, hi);
          v[8 + 2 * i] *= r * lo;
          v[8 + 2 * i + 1] *= r * hi;
        }
      }
      float o[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (INTER) {  // pairs (2i, 2i+1) of chunk 0, then of chunk 1
          const float2 r = turn[i];
          o[2 * i] = v[2 * i] * r.x - v[2 * i + 1] * r.y;
          o[2 * i + 1] = v[2 * i + 1] * r.x + v[2 * i] * r.y;
        } else {                // channel 8j + i with 64 + 8j + i
          const float2 r = turn[i];
          o[i] = v[i] * r.x - v[8 + i] * r.y;
          o[8 + i] = v[8 + i] * r.x + v[i] * r.y;
        }
      }
      if (h < end && n0 + t < a.N) {
        uint16_t* d = y + (int64_t)h * ys.h;
        *reinterpret_cast<uint4*>(d) = make_uint4(pack_x2<F16>(o[0], o[1]), pack_x2<F16>(o[2], o[3]),
                                                  pack_x2<F16>(o[4], o[5]), pack_x2<F16>(o[6], o[7]));
        *reinterpret_cast<uint4*>(d + 64) = make_uint4(pack_x2<F16>(o[8], o[9]), pack_x2<F16>(o[10], o[11]),
                                                       pack_x2<F16>(o[12], o[13]), pack_x2<F16>(o[14], o[15]));
      }
    }
  }
}

template <int TOK>
cudaError_t launch_tok(RopeArgs& a, int B, bool f16, bool interleaved, cudaStream_t st) {
  a.tiles = (a.N + TOK - 1) / TOK;
  const int64_t blocks = (int64_t)B * a.tiles;
  // Few tokens: the heads go to several blocks, until there are about four blocks per SM.
  constexpr int kStep = kRows / TOK;
  const int steps = (a.H + kStep - 1) / kStep;
  int split = (int)((4 * 148 + blocks - 1) / blocks);
  if (split > steps) split = steps;
  a.heads_per_block = (steps + split - 1) / split * kStep;
  const dim3 grid((unsigned)blocks, (a.H + a.heads_per_block - 1) / a.heads_per_block);
  auto kern = f16 ? (interleaved ? qk_norm_rope_kernel<TOK, true, true> : qk_norm_rope_kernel<TOK, true, false>)
                  : (interleaved ? qk_norm_rope_kernel<TOK, false, true> : qk_norm_rope_kernel<TOK, false, false>);
  return launch_overlapped(kern, grid, kThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  RopeArgs a;
  a.x[0] = p.q; a.x[1] = p.k; a.y[0] = p.q_out; a.y[1] = p.k_out;
  a.w[0] = p.q_weight; a.w[1] = p.k_weight;
  a.xs[0] = p.q_strides; a.xs[1] = p.k_strides; a.ys[0] = p.q_out_strides; a.ys[1] = p.k_out_strides;
  a.pos = p.positions; a.inv_freq = p.inv_freq; a.eps = p.eps;
  a.N = p.N; a.Hq = p.Hq; a.H = p.Hq + p.Hkv;
  // Four tokens per block share their pairs' cosines with four heads at a time; with fewer tokens
  // per sequence that many lanes would idle, so each block takes one token and 16 heads at a time.
  return p.N >= 4 ? launch_tok<4>(a, p.B, p.f16, p.interleaved, st) : launch_tok<1>(a, p.B, p.f16, p.interleaved, st);
}

}  // namespace kascade
