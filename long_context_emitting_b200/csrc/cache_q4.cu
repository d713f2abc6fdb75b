// Quantising K/V rows to 4 bits as they are written into pages, and reading
// them back in 16 bits.  The row format is in q4.cuh.
//
// Quantisation of a group of 32 channels x (asymmetric, so that channels with
// an offset keep their resolution; exact in the sense that the codes are those
// of real arithmetic on the stored scale and minimum):
//   m = the largest bfloat16 <= min(x)
//   s = the smallest bfloat16 >= (max(x) - m) / 15      (so no value clips)
//   n = (x - m) / s rounded to nearest, half to even, in 0..15 (0 when s = 0)
//   value = m + s n
// m and s are rounded outward with the directed roundings of fp32 and one
// truncation, which is exact because every bfloat16 bound is also an fp32
// number.  For n, fp32 division is monotone and cannot round a quotient that
// is not half-way onto a half-way point; only the subtraction x - m may, when
// it is inexact, and then its rounding error (two-sum) says to which side the
// value lies.
//
// What bounds both kernels: memory, 512 bytes of 16-bit rows against 160 bytes
// of cache row per token and key head.  Half a warp handles one row: a lane
// holds 8 channels of K and of V (one 16-byte load or store each), a group is
// four lanes, and one exchange with the lane four further puts the V halves of
// two groups into one word.
#include "common.cuh"
#include "internal.h"
#include "q4.cuh"

#include <math_constants.h>

namespace kascade {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;  // rows per block

struct CacheArgs {
  const uint16_t* k;  // write: source rows
  const uint16_t* v;
  kascade_strides ks, vs;
  uint16_t* k_out;    // read: destination [B, Hkv, N, 128]
  uint16_t* v_out;
  uint8_t* pages;
  const int32_t* block_table;
  const int32_t* start;
  const int32_t* count;  // NULL: N tokens of every sequence
  int num_pages, max_pages, page_size;
  int N, Hkv, tiles;
  unsigned* status;
};

// bfloat16 bits of x rounded toward -inf / +inf (x finite).
__device__ __forceinline__ uint32_t bf16_down(float x) {
  const uint32_t u = __float_as_uint(x);
  return ((x < 0.f && (u & 0xffffu)) ? u + 0x10000u : u) >> 16;
}
__device__ __forceinline__ uint32_t bf16_up_pos(float x) {  // x >= 0
  const uint32_t u = __float_as_uint(x);
  return ((u & 0xffffu) ? u + 0x10000u : u) >> 16;
}

struct Group {
  uint32_t words;  // 8 codes of this lane
  uint32_t s, m;   // bfloat16 bits of the group's scale and minimum
  bool bad;        // a value is not finite, or the range is not
};

// Codes of this lane's 8 values; lanes 4g .. 4g+3 of the half warp are one group.
__device__ __forceinline__ Group quantise(const float (&x)[8]) {
  float lo = x[0], hi = x[0];
  bool fin = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    fin = fin && (fabsf(x[i]) < CUDART_INF_F);  // false for NaN too
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    fin = __shfl_xor_sync(0xffffffffu, (int)fin, o) && fin;
  }
  Group g;
  g.m = bf16_down(lo);
  const float m = __uint_as_float(g.m << 16);
  g.s = bf16_up_pos(__fdiv_ru(__fadd_ru(hi, -m), 15.f));
  const float s = __uint_as_float(g.s << 16);
  g.bad = !(fin && s < CUDART_INF_F && fabsf(m) < CUDART_INF_F);
  g.words = 0;
  if (g.bad) {  // reads back as NaN: the loss shows
    g.s = 0;
    g.m = 0x7fc0u;
    return g;
  }
  if (s == 0.f) return g;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fadd_rn(x[i], -m);
    const float q = __fdiv_rn(d, s);
    float n = rintf(q);
    const float f = floorf(q);
    if (q - f == 0.5f) {  // half-way: the rounding error of d, if any, decides
      const float bb = __fadd_rn(d, -x[i]);
      const float err = __fadd_rn(__fadd_rn(x[i], -__fadd_rn(d, -bb)), __fadd_rn(-m, -bb));
      if (err > 0.f) n = f + 1.f;
      if (err < 0.f) n = f;
    }
    g.words |= (uint32_t)(int)fminf(fmaxf(n, 0.f), 15.f) << (4 * i);
  }
  return g;
}

// The token and head of this half warp: TOK tokens x kRows / TOK heads per block.
template <int TOK>
struct Place {
  int b, n, h;
  __device__ __forceinline__ Place(const CacheArgs& a) {
    const int row = threadIdx.x / 16;
    b = blockIdx.x / a.tiles;
    n = (blockIdx.x - b * a.tiles) * TOK + row % TOK;
    h = blockIdx.y * (kRows / TOK) + row / TOK;
  }
};

// Byte offset of the row in the page store, or -1 where nothing is to be done.
__device__ __forceinline__ int64_t row_of(const CacheArgs& a, int b, int n, int h, bool first) {
  if (n >= a.N || h >= a.Hkv) return -1;
  const int start = a.start[b], count = a.count ? a.count[b] : a.N;
  // positions stay below 2^30, the longest sequence the decode calls take
  const int64_t end = (int64_t)start + count, limit = min((int64_t)a.max_pages * a.page_size, (int64_t)1 << 30);
  if (start < 0 || count < 0 || count > a.N || end > limit) {
    if (first) flag_status(a.status, kStatusBadIndex);
    return -1;
  }
  if (n >= count) return -1;
  const int64_t o =
      q4_row(a.block_table + (int64_t)b * a.max_pages, start + n, a.page_size, a.num_pages, a.Hkv, h);
  if (o < 0 && first) flag_status(a.status, kStatusBadIndex);
  return o;
}

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheArgs a) {
  const Place<TOK> p(a);
  const int l = threadIdx.x % 16;
  const int64_t o = row_of(a, p.b, p.n, p.h, l == 0);
  float xk[8], xv[8];
  uint4 ck = make_uint4(0, 0, 0, 0), cv = ck;
  if (o >= 0) {
    ck = ldg16(a.k + (int64_t)p.b * a.ks.b + (int64_t)p.n * a.ks.n + (int64_t)p.h * a.ks.h + 8 * l);
    cv = ldg16(a.v + (int64_t)p.b * a.vs.b + (int64_t)p.n * a.vs.n + (int64_t)p.h * a.vs.h + 8 * l);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpack2<F16>(word_of(ck, i), xk[2 * i], xk[2 * i + 1]);
    unpack2<F16>(word_of(cv, i), xv[2 * i], xv[2 * i + 1]);
  }
  const Group gk = quantise(xk), gv = quantise(xv);
  // lane (g, j) holds channels 32g + 8j ..: V half words of lane groups r = 2j and 2j + 1.  Even g
  // builds the word of r = 2j (halves g, g + 1), odd g that of r = 2j + 1.
  const int g = l >> 2, j = l & 3;
  const bool odd = g & 1;
  const uint32_t give = odd ? gv.words & 0xffffu : gv.words >> 16;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
  const uint32_t vword = odd ? (got | (gv.words & 0xffff0000u)) : ((gv.words & 0xffffu) | (got << 16));
  // bfloat16 number l of the tail: K scales, K minima, V scales, V minima, by groups
  const int src = (threadIdx.x & 16) + 4 * (l & 3);
  const uint32_t tk = __shfl_sync(0xffffffffu, gk.s | (gk.m << 16), src);
  const uint32_t tv = __shfl_sync(0xffffffffu, gv.s | (gv.m << 16), src);
  const uint32_t tw = l < 8 ? tk : tv;
  if (o < 0) return;
  if (gk.bad || gv.bad) flag_status(a.status, kStatusNonFinite);
  uint8_t* dst = a.pages + o;
  reinterpret_cast<uint32_t*>(dst)[4 * j + g] = gk.words;
  reinterpret_cast<uint32_t*>(dst + kQ4V)[2 * (2 * j + (int)odd) + (g >> 1)] = vword;
  reinterpret_cast<uint16_t*>(dst + kQ4Tail)[l] = (uint16_t)((l & 4) ? tw >> 16 : tw);
}

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  const Place<TOK> p(a);
  const int l = threadIdx.x % 16;
  const int g = l >> 2, j = l & 3;
  const bool odd = g & 1;
  const int64_t o = row_of(a, p.b, p.n, p.h, l == 0);
  uint32_t kw = 0, vw = 0, tail = 0;
  if (o >= 0) {
    const uint8_t* src = a.pages + o;
    kw = __ldg(reinterpret_cast<const uint32_t*>(src) + 4 * j + g);
    vw = __ldg(reinterpret_cast<const uint32_t*>(src + kQ4V) + 2 * (2 * j + (int)odd) + (g >> 1));
    tail = __ldg(reinterpret_cast<const uint16_t*>(src + kQ4Tail) + l);
  }
  const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? vw & 0xffffu : vw >> 16, 4);
  vw = odd ? (got | (vw & 0xffff0000u)) : ((vw & 0xffffu) | (got << 16));
  const int base = threadIdx.x & 16;
  float f[4];  // K scale, K minimum, V scale, V minimum of this lane's group
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__shfl_sync(0xffffffffu, tail, base + 4 * i + g) << 16);
  if (o < 0) return;
  uint32_t ok[4], ov[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ok[i] = pack_x2<F16>(fmaf(f[0], (float)((kw >> (8 * i)) & 15u), f[1]),
                         fmaf(f[0], (float)((kw >> (8 * i + 4)) & 15u), f[1]));
    ov[i] = pack_x2<F16>(fmaf(f[2], (float)((vw >> (8 * i)) & 15u), f[3]),
                         fmaf(f[2], (float)((vw >> (8 * i + 4)) & 15u), f[3]));
  }
  const int64_t dst = (((int64_t)p.b * a.Hkv + p.h) * a.N + p.n) * kHeadDim + 8 * l;
  *reinterpret_cast<uint4*>(a.k_out + dst) = make_uint4(ok[0], ok[1], ok[2], ok[3]);
  *reinterpret_cast<uint4*>(a.v_out + dst) = make_uint4(ov[0], ov[1], ov[2], ov[3]);
}

template <int TOK>
cudaError_t launch_tok(CacheArgs& a, int B, bool f16, bool write, cudaStream_t st) {
  a.tiles = (a.N + TOK - 1) / TOK;
  constexpr int kHeads = kRows / TOK;
  const dim3 grid((unsigned)((int64_t)B * a.tiles), (a.Hkv + kHeads - 1) / kHeads);
  auto kern = write ? (f16 ? cache_write_kernel<TOK, true> : cache_write_kernel<TOK, false>)
                    : (f16 ? cache_read_kernel<TOK, true> : cache_read_kernel<TOK, false>);
  kern<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_q4(const CacheQ4Params& p, bool write, cudaStream_t st) {
  CacheArgs a;
  a.k = p.k; a.v = p.v; a.ks = p.k_strides; a.vs = p.v_strides;
  a.k_out = p.k_out; a.v_out = p.v_out;
  a.pages = p.kv_pages; a.block_table = p.block_table; a.start = p.start; a.count = p.count;
  a.num_pages = p.num_pages; a.max_pages = p.max_pages; a.page_size = p.page_size;
  a.N = p.N; a.Hkv = p.Hkv; a.status = p.status;
  // Four tokens x four heads per block; with fewer tokens per sequence, one token x 16 heads.
  return p.N >= 4 ? launch_tok<4>(a, p.B, p.f16, write, st) : launch_tok<1>(a, p.B, p.f16, write, st);
}

}  // namespace kascade
