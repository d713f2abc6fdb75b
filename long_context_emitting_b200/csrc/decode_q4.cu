// Decode attention over the 4-bit paged cache (row format in q4.cuh): the anchor
// (every token, pooled probabilities) and the reuse layer (selected tokens).
//
// With V, K = minimum + scale * code per row and group, for each query head:
//   s_t = scale · q · K_t;  out = sum_t softmax(s)_t V_t;  lse = log sum_t exp(s_t)
//
// A warp takes one token at a time: lane l holds channels 4l .. 4l + 3, so its
// four K codes are one half word, its four V codes another, and both belong to
// scale group l / 8.  All arithmetic is fp32.  The anchor's splits go through
// the workspace and a combine kernel; a reuse row is one block.
#include "common.cuh"
#include "internal.h"
#include "q4.cuh"

#include <cmath>

namespace kascade {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLn2 = 0.6931471805599453f;

struct Q4Args {
  const uint16_t* q;
  const uint8_t* pages;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  const int32_t* seq_len;
  const int32_t* idx;
  const int32_t* idx_k;
  const int32_t* head_map;
  int k_max;
  int Hq, Hkv, max_T;
  int tok_per_warp, nsplit;
  float scale_log2;
  float* logits;   // anchor: [B, Hkv, max_T, G] base-2 scaled logits
  float* part_ml;  // [B*Hkv, nsplit, G, 2]
  float* part_o;   // [B*Hkv, nsplit, G, 128]
  uint16_t* out;   // reuse
  float* lse;
  unsigned* status;
};

// What exponentials are taken relative to: the maximum, or 0 where there is no finite score yet
// (exp2(-inf - 0) is then 0).  A maximum ignores NaN; the sum of the exponentials keeps it, so a
// NaN score reaches the results whether or not it is alone.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float lse2_of(float m, float l) { return l == 0.f ? -INFINITY : finite_max(m) + __log2f(l); }

template <int G, bool GATHER, bool F16>
__global__ void __launch_bounds__(kThreads) decode_q4_kernel(const Q4Args a) {
  __shared__ float sm_o[kWarps][G][kHeadDim];
  __shared__ float sm_m[kWarps][G], sm_l[kWarps][G];
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t bh = (int64_t)b * a.Hkv + h;

  int T = a.seq_len[b];
  bool ok = T >= 0 && T <= a.max_T;
  int n_items = T;
  const int32_t* rows = nullptr;
  if (GATHER && ok) {
    const int am = a.head_map[h];
    ok = am >= 0 && am < a.Hkv;
    if (ok) {
      rows = a.idx + ((int64_t)b * a.Hkv + am) * a.k_max;
      n_items = a.idx_k[b * a.Hkv + am];
      ok = n_items >= 0 && n_items <= a.k_max;
    }
    if (T == 0) n_items = 0;
  }
  if (!ok) {
    if (threadIdx.x == 0 && split == 0) flag_status(a.status, kStatusBadIndex);
    n_items = 0;
  }
  const int i_begin = (split * kWarps + warp) * a.tok_per_warp;
  const int i_end = min((int64_t)i_begin + a.tok_per_warp, (int64_t)n_items);

  float q[G][4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint2 w = *reinterpret_cast<const uint2*>(a.q + ((int64_t)b * a.Hq + h * G + g) * kHeadDim + 4 * lane);
    unpack2<F16>(w.x, q[g][0], q[g][1]);
    unpack2<F16>(w.y, q[g][2], q[g][3]);
  }
  float m[G], l[G], o[G][4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    o[g][0] = o[g][1] = o[g][2] = o[g][3] = 0.f;
  }
  const int grp = lane >> 3, r = lane & 7;
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
  for (int i = i_begin; i < i_end; ++i) {
    const int t = GATHER ? __ldg(rows + i) : i;
    int64_t off = -1;
    if (t >= 0 && t < T) off = q4_row(table, t, a.page_size, a.num_pages, a.Hkv, h);
    if (off < 0) {
      if (lane == 0) flag_status(a.status, kStatusBadIndex);
      if (!GATHER && lane < G) a.logits[(bh * a.max_T + i) * G + lane] = -INFINITY;
      continue;
    }
    const uint8_t* row = a.pages + off;
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(row + 4 * (4 * (r >> 1) + grp) + 2 * (r & 1));
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(row + kQ4V + 4 * (2 * r + (grp >> 1)) + 2 * (grp & 1));
    const uint16_t* tail = reinterpret_cast<const uint16_t*>(row + kQ4Tail);
    const float ks = bf16_lo(tail[grp]), km = bf16_lo(tail[4 + grp]);
    const float vs = bf16_lo(tail[8 + grp]), vm = bf16_lo(tail[12 + grp]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) s += q[g][c] * fmaf(ks, (float)((kc >> (4 * c)) & 15u), km);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= a.scale_log2;
      if (!GATHER && lane == 0) a.logits[(bh * a.max_T + i) * G + g] = s;
      const float mn = fmaxf(m[g], s);
      const float base = finite_max(mn);
      const float al = fast_exp2(m[g] - base), p = fast_exp2(s - base);
      m[g] = mn;
      l[g] = l[g] * al + p;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[g][c] = o[g][c] * al + p * fmaf(vs, (float)((vc >> (4 * c)) & 15u), vm);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int c = 0; c < 4; ++c) sm_o[warp][g][4 * lane + c] = o[g][c];
    if (lane == 0) {
      sm_m[warp][g] = m[g];
      sm_l[warp][g] = l[g];
    }
  }
  __syncthreads();
  const int d = threadIdx.x;  // kThreads == kHeadDim
  for (int g = 0; g < G; ++g) {
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][g]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = fast_exp2(sm_m[w][g] - finite_max(M));
      acc += f * sm_o[w][g][d];
      L += f * sm_l[w][g];
    }
    if (GATHER) {
      a.out[((int64_t)b * a.Hq + h * G + g) * kHeadDim + d] = to_bits<F16>(L == 0.f ? 0.f : acc / L);
      if (a.lse && d == 0) a.lse[(int64_t)b * a.Hq + h * G + g] = lse2_of(M, L) * kLn2;
    } else {
      const int64_t slot = (bh * a.nsplit + split) * G + g;
      a.part_o[slot * kHeadDim + d] = acc;
      if (d == 0) {
        a.part_ml[slot * 2] = M;
        a.part_ml[slot * 2 + 1] = L;
      }
    }
  }
}

struct CombineArgs {
  const int32_t* seq_len;
  int Hq, Hkv, G, max_T, nsplit;
  const float* part_ml;
  const float* part_o;
  const float* logits;
  float* pooled;
  int64_t ld_pooled;
  uint16_t* out;
  float* lse;
};

constexpr int kCombineThreads = 256;
constexpr int kPoolChunk = 2048;  // tokens per block

// Second kernel of the anchor: every block merges the splits' maxima and sums of its (b, h); the
// first also their outputs; each turns its chunk of logits into pooled probabilities.
template <bool F16>
__global__ void __launch_bounds__(kCombineThreads) decode_q4_combine_kernel(const CombineArgs a) {
  __shared__ float s_M[8], s_L[8], s_lse2[8];
  const int b = blockIdx.z, h = blockIdx.y, chunk = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G;
  const int64_t bh = (int64_t)b * a.Hkv + h;
  const float* ml = a.part_ml + bh * a.nsplit * G * 2;
  if (warp < G) {
    float M = -INFINITY, L = 0.f;
    for (int s = lane; s < a.nsplit; s += 32) M = fmaxf(M, ml[(s * G + warp) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int s = lane; s < a.nsplit; s += 32)
      L += fast_exp2(ml[(s * G + warp) * 2] - finite_max(M)) * ml[(s * G + warp) * 2 + 1];
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) {
      s_M[warp] = finite_max(M);
      s_L[warp] = L;
      s_lse2[warp] = lse2_of(M, L);
    }
  }
  __syncthreads();
  if (chunk == 0) {
    const float* po = a.part_o + bh * a.nsplit * G * kHeadDim;
    for (int e = threadIdx.x; e < G * kHeadDim; e += kCombineThreads) {
      const int g = e / kHeadDim, d = e % kHeadDim;
      float acc = 0.f;
      for (int s = 0; s < a.nsplit; ++s)
        acc += fast_exp2(ml[(s * G + g) * 2] - s_M[g]) * po[((int64_t)s * G + g) * kHeadDim + d];
      a.out[((int64_t)b * a.Hq + h * G + g) * kHeadDim + d] = to_bits<F16>(s_L[g] == 0.f ? 0.f : acc / s_L[g]);
    }
    if (a.lse && threadIdx.x < G) a.lse[(int64_t)b * a.Hq + h * G + threadIdx.x] = s_lse2[threadIdx.x] * kLn2;
  }
  int T = a.seq_len[b];
  if (T < 0 || T > a.max_T) T = 0;
  const int t_hi = (int)min((int64_t)(chunk + 1) * kPoolChunk, (int64_t)T);
  const float* lrow = a.logits + bh * a.max_T * G;
  float* prow = a.pooled + bh * a.ld_pooled;
  const float invG = 1.f / (float)G;
  for (int t = chunk * kPoolChunk + threadIdx.x; t < t_hi; t += kCombineThreads) {
    float acc = 0.f;
    // no finite score at all (every page entry bad): relative to 0 the probabilities are 0
    for (int g = 0; g < G; ++g) acc += fast_exp2(lrow[(int64_t)t * G + g] - finite_max(s_lse2[g]));
    prow[t] = acc * invG;
  }
}

struct WsLayout {
  size_t logits, part_ml, part_o, total;
};
WsLayout ws_layout(int B, int Hkv, int G, int max_T, int nsplit) {
  WsLayout w;
  size_t off = 0;
  w.logits = off;
  off = align_up(off + (size_t)B * Hkv * max_T * G * sizeof(float), 256);
  w.part_ml = off;
  off = align_up(off + (size_t)B * Hkv * nsplit * G * 2 * sizeof(float), 256);
  w.part_o = off;
  w.total = align_up(off + (size_t)B * Hkv * nsplit * G * kHeadDim * sizeof(float), 256);
  return w;
}

template <bool GATHER, bool F16>
void launch_g(const Q4Args& a, int G, dim3 grid, cudaStream_t st) {
  if (G == 1) decode_q4_kernel<1, GATHER, F16><<<grid, kThreads, 0, st>>>(a);
  else if (G == 2) decode_q4_kernel<2, GATHER, F16><<<grid, kThreads, 0, st>>>(a);
  else if (G == 4) decode_q4_kernel<4, GATHER, F16><<<grid, kThreads, 0, st>>>(a);
  else decode_q4_kernel<8, GATHER, F16><<<grid, kThreads, 0, st>>>(a);
}

Q4Args common_args(const DecodeQ4Params& p) {
  Q4Args a = {};
  a.q = p.q; a.pages = p.kv_pages; a.block_table = p.block_table;
  a.max_pages = p.max_pages; a.page_size = p.page_size; a.num_pages = p.num_pages;
  a.seq_len = p.seq_len; a.idx = p.idx; a.idx_k = p.idx_k; a.head_map = p.head_map; a.k_max = p.k_max;
  a.Hq = p.Hq; a.Hkv = p.Hkv; a.max_T = p.max_T;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.out = p.out; a.lse = p.lse; a.status = p.status;
  return a;
}

}  // namespace

size_t decode_q4_workspace_bytes(int B, int Hkv, int G, int max_T) {
  return ws_layout(B, Hkv, G, max_T, decode_split_for(B * Hkv, max_T, false).nsplit).total;
}

cudaError_t launch_decode_anchor_q4(const DecodeQ4Params& p, cudaStream_t st) {
  const DecodeSplit sp = decode_split_for(p.B * p.Hkv, p.max_T, false);
  const WsLayout w = ws_layout(p.B, p.Hkv, p.G, p.max_T, sp.nsplit);
  char* ws = static_cast<char*>(p.ws);
  Q4Args a = common_args(p);
  a.tok_per_warp = sp.tok_per_warp;
  a.nsplit = sp.nsplit;
  a.logits = reinterpret_cast<float*>(ws + w.logits);
  a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  const dim3 grid(sp.nsplit, p.Hkv, p.B);
  if (p.f16) launch_g<false, true>(a, p.G, grid, st);
  else launch_g<false, false>(a, p.G, grid, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CombineArgs c;
  c.seq_len = p.seq_len;
  c.Hq = p.Hq; c.Hkv = p.Hkv; c.G = p.G; c.max_T = p.max_T; c.nsplit = sp.nsplit;
  c.part_ml = a.part_ml; c.part_o = a.part_o; c.logits = a.logits;
  c.pooled = p.pooled; c.ld_pooled = p.ld_pooled; c.out = p.out; c.lse = p.lse;
  const dim3 cgrid(p.max_T > 0 ? (p.max_T + kPoolChunk - 1) / kPoolChunk : 1, p.Hkv, p.B);
  if (p.f16) decode_q4_combine_kernel<true><<<cgrid, kCombineThreads, 0, st>>>(c);
  else decode_q4_combine_kernel<false><<<cgrid, kCombineThreads, 0, st>>>(c);
  return cudaGetLastError();
}

cudaError_t launch_decode_reuse_q4(const DecodeQ4Params& p, cudaStream_t st) {
  Q4Args a = common_args(p);
  a.nsplit = 1;
  a.tok_per_warp = (p.k_max + kWarps - 1) / kWarps;
  const dim3 grid(1, p.Hkv, p.B);
  if (p.f16) launch_g<true, true>(a, p.G, grid, st);
  else launch_g<true, false>(a, p.G, grid, st);
  return cudaGetLastError();
}

}  // namespace kascade
