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
// number.  n comes from one multiplication by 1 / s, off by less than 2^-17, and
// is certain unless the quotient lies within 2^-16 of a half-way point (or s is
// so small that 1 / s is not a normal number).  Those lanes divide: fp32 division
// is monotone and cannot round a quotient that is not half-way onto a half-way
// point; only the subtraction x - m may, when it is inexact, and then its
// rounding error (two-sum) says to which side the value lies.
//
// What bounds both kernels: memory, 512 bytes of 16-bit rows against 160 bytes
// of cache row per token and key head.  Half a warp handles one row: a lane
// holds 8 channels of K and of V (one 16-byte load or store each), a group is
// four lanes, and one exchange with the lane four further puts the V halves of
// two groups into one word.  A block takes 16 tokens (fewer when there are few)
// through several heads, so that a token's page is looked up once and the next
// head's rows are on their way while one head's are worked on.
#include "common.cuh"
#include "internal.h"
#include "q4.cuh"

#include <algorithm>
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
  int N, Hkv, tiles, heads_per_block;
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

// Minima (or maxima) of the halves of two words, in the data's type; a NaN loses.
template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (F16) {
    const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r =
        __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return min2<F16>(a ^ 0x80008000u, b ^ 0x80008000u) ^ 0x80008000u;
}

// The code of x by division, for values next to a half-way point.
__device__ __noinline__ uint32_t exact_code(float x, float m, float s) {
  const float d = __fadd_rn(x, -m);
  const float q = __fdiv_rn(d, s);
  float n = rintf(q);
  const float f = floorf(q);
  if (q - f == 0.5f) {  // half-way: the rounding error of d, if any, decides
    const float bb = __fadd_rn(d, -x);
    const float err = __fadd_rn(__fadd_rn(x, -__fadd_rn(d, -bb)), __fadd_rn(-m, -bb));
    if (err > 0.f) n = f + 1.f;
    if (err < 0.f) n = f;
  }
  return (uint32_t)(int)fminf(fmaxf(n, 0.f), 15.f);
}

// Codes of this lane's 8 values; lanes 4g .. 4g+3 of the half warp are one group.
template <bool F16>
__device__ __forceinline__ Group quantise(const uint4& w) {
  float x[8];
  float none = 0.f;  // NaN as soon as a value is not finite
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpack2<F16>(word_of(w, i), x[2 * i], x[2 * i + 1]);
    none = fmaf(x[2 * i], 0.f, fmaf(x[2 * i + 1], 0.f, none));
  }
  const uint32_t lo2 = min2<F16>(min2<F16>(w.x, w.y), min2<F16>(w.z, w.w));
  const uint32_t hi2 = max2<F16>(max2<F16>(w.x, w.y), max2<F16>(w.z, w.w)) ^ 0x80008000u;
  // (minimum, minus maximum) in one word
  uint32_t ends = min2<F16>(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
  ends = min2<F16>(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
  ends = min2<F16>(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
  float lo, hi;
  unpack2<F16>(ends, lo, hi);
  hi = -hi;
  const uint32_t odd = __ballot_sync(0xffffffffu, !(none == 0.f));
  Group g;
  g.m = bf16_down(lo);
  const float m = __uint_as_float(g.m << 16);
  g.s = bf16_up_pos(__fdiv_ru(__fadd_ru(hi, -m), 15.f));
  const float s = __uint_as_float(g.s << 16);
  g.bad = ((odd >> (threadIdx.x & 28)) & 15u) || !(s < CUDART_INF_F && fabsf(m) < CUDART_INF_F);
  g.words = 0;
  if (g.bad) {  // reads back as NaN: the loss shows
    g.s = 0;
    g.m = 0x7fc0u;
    return g;
  }
  if (s == 0.f) return g;
  const float inv = __frcp_rn(s);
  float near = s < 0x1p-100f ? 1.f : 0.f;  // distance to the code, at most 1/2
  float n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = x[i] - m;
    n[i] = fmaf(d, inv, 0x1.8p23f) - 0x1.8p23f;  // rounds to an integer
    near = fmaxf(near, fabsf(fmaf(d, inv, -n[i])));
  }
  // four codes in 16 bits: exact in fp32, and read off the low bits after adding 2^23
  const float a = fmaf(n[3], 4096.f, fmaf(n[2], 256.f, fmaf(n[1], 16.f, n[0]))) + 0x1p23f;
  const float b = fmaf(n[7], 4096.f, fmaf(n[6], 256.f, fmaf(n[5], 16.f, n[4]))) + 0x1p23f;
  g.words = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
  if (near > 0.5f - 0x1p-16f) {
    g.words = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) g.words |= exact_code(x[i], m, s) << (4 * i);
  }
  return g;
}

// Where a half warp works: one token of a tile of TOK, through heads h, h + kRows / TOK, ... < h_end.
template <int TOK>
struct Place {
  int b, n, h, h_end;
  int64_t row;  // of head 0 in the page store, or -1 where nothing is to be done
  __device__ __forceinline__ Place(const CacheArgs& a) {
    const int r = threadIdx.x / 16;
    b = blockIdx.x / a.tiles;
    n = (blockIdx.x - b * a.tiles) * TOK + r % TOK;
    h = blockIdx.y * a.heads_per_block + r / TOK;
    h_end = min(a.Hkv, (int)(blockIdx.y + 1) * a.heads_per_block);
    row = row_of(a);
  }
  __device__ __forceinline__ int64_t row_of(const CacheArgs& a) const {
    const bool first = threadIdx.x % 16 == 0 && h < h_end;  // one lane reports
    if (n >= a.N) return -1;
    const int start = a.start[b], count = a.count ? a.count[b] : a.N;
    // positions stay below 2^30, the longest sequence the decode calls take
    const int64_t end = (int64_t)start + count, limit = min((int64_t)a.max_pages * a.page_size, (int64_t)1 << 30);
    if (start < 0 || count < 0 || count > a.N || end > limit) {
      if (first) flag_status(a.status, kStatusBadIndex);
      return -1;
    }
    if (n >= count) return -1;
    const int t = start + n, pi = t / a.page_size;
    const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + pi);
    if (page < 0 || page >= a.num_pages) {
      if (first) flag_status(a.status, kStatusBadIndex);
      return -1;
    }
    return (int64_t)page * a.Hkv * a.page_size + (t - pi * a.page_size);
  }
};

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheArgs a) {
  const Place<TOK> p(a);
  // whole warps leave together: a tile past the end of its sequence costs nothing more
  if (!__any_sync(0xffffffffu, p.row >= 0)) return;
  const int l = threadIdx.x % 16;
  const int g = l >> 2, j = l & 3;
  const bool odd = g & 1;
  constexpr int kStep = kRows / TOK;
  const uint16_t* k = a.k + (int64_t)p.b * a.ks.b + (int64_t)p.n * a.ks.n + (int64_t)p.h * a.ks.h + 8 * l;
  const uint16_t* v = a.v + (int64_t)p.b * a.vs.b + (int64_t)p.n * a.vs.n + (int64_t)p.h * a.vs.h + 8 * l;
  uint8_t* dst = a.pages + (p.row + (int64_t)p.h * a.page_size) * kQ4Row;
  bool bad = false;
  uint4 ck = make_uint4(0, 0, 0, 0), cv = ck;
  if (p.row >= 0 && p.h < p.h_end) {
    ck = ldg16(k);
    cv = ldg16(v);
  }
  const int passes = (p.h_end - (int)blockIdx.y * a.heads_per_block + kStep - 1) / kStep;  // of the block
  for (int i = 0, h = p.h; i < passes; ++i, h += kStep) {
    const bool live = p.row >= 0 && h < p.h_end;
    uint4 nk = make_uint4(0, 0, 0, 0), nv = nk;
    k += (int64_t)kStep * a.ks.h;
    v += (int64_t)kStep * a.vs.h;
    if (p.row >= 0 && h + kStep < p.h_end) {
      nk = ldg16(k);
      nv = ldg16(v);
    }
    const Group gk = quantise<F16>(ck), gv = quantise<F16>(cv);
    // lane (g, j) holds channels 32g + 8j ..: V half words of lane groups r = 2j and 2j + 1.  Even g
    // builds the word of r = 2j (halves g, g + 1), odd g that of r = 2j + 1.
    const uint32_t give = odd ? gv.words & 0xffffu : gv.words >> 16;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
    const uint32_t vword = odd ? (got | (gv.words & 0xffff0000u)) : ((gv.words & 0xffffu) | (got << 16));
    // bfloat16 number l of the tail: K scales, K minima, V scales, V minima, by groups
    const int src = (threadIdx.x & 16) + 4 * (l & 3);
    const uint32_t tk = __shfl_sync(0xffffffffu, gk.s | (gk.m << 16), src);
    const uint32_t tv = __shfl_sync(0xffffffffu, gv.s | (gv.m << 16), src);
    const uint32_t tw = l < 8 ? tk : tv;
    if (live) {
      bad |= gk.bad || gv.bad;
      reinterpret_cast<uint32_t*>(dst)[4 * j + g] = gk.words;
      reinterpret_cast<uint32_t*>(dst + kQ4V)[2 * (2 * j + (int)odd) + (g >> 1)] = vword;
      reinterpret_cast<uint16_t*>(dst + kQ4Tail)[l] = (uint16_t)((l & 4) ? tw >> 16 : tw);
    }
    dst += (int64_t)kStep * a.page_size * kQ4Row;
    ck = nk;
    cv = nv;
  }
  if (bad) flag_status(a.status, kStatusNonFinite);
}

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  const Place<TOK> p(a);
  if (!__any_sync(0xffffffffu, p.row >= 0)) return;
  const int l = threadIdx.x % 16;
  const int g = l >> 2, j = l & 3;
  const bool odd = g & 1;
  constexpr int kStep = kRows / TOK;
  const uint8_t* src = a.pages + (p.row + (int64_t)p.h * a.page_size) * kQ4Row;
  uint32_t kw = 0, vw = 0, tail = 0;
  auto load = [&](uint32_t& k, uint32_t& v, uint32_t& t) {
    k = __ldg(reinterpret_cast<const uint32_t*>(src) + 4 * j + g);
    v = __ldg(reinterpret_cast<const uint32_t*>(src + kQ4V) + 2 * (2 * j + (int)odd) + (g >> 1));
    t = __ldg(reinterpret_cast<const uint16_t*>(src + kQ4Tail) + l);
  };
  if (p.row >= 0 && p.h < p.h_end) load(kw, vw, tail);
  const int base = threadIdx.x & 16;
  int64_t dst = (((int64_t)p.b * a.Hkv + p.h) * a.N + p.n) * kHeadDim + 8 * l;
  const int passes = (p.h_end - (int)blockIdx.y * a.heads_per_block + kStep - 1) / kStep;
  for (int i = 0, h = p.h; i < passes; ++i, h += kStep) {
    uint32_t nk = 0, nv = 0, nt = 0;
    src += (int64_t)kStep * a.page_size * kQ4Row;
    if (p.row >= 0 && h + kStep < p.h_end) load(nk, nv, nt);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? vw & 0xffffu : vw >> 16, 4);
    vw = odd ? (got | (vw & 0xffff0000u)) : ((vw & 0xffffu) | (got << 16));
    float f[4];  // K scale, K minimum, V scale, V minimum of this lane's group
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = __uint_as_float(__shfl_sync(0xffffffffu, tail, base + 4 * u + g) << 16);
    if (p.row >= 0 && h < p.h_end) {
      uint32_t ok[4], ov[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ok[u] = pack_x2<F16>(fmaf(f[0], (float)((kw >> (8 * u)) & 15u), f[1]),
                             fmaf(f[0], (float)((kw >> (8 * u + 4)) & 15u), f[1]));
        ov[u] = pack_x2<F16>(fmaf(f[2], (float)((vw >> (8 * u)) & 15u), f[3]),
                             fmaf(f[2], (float)((vw >> (8 * u + 4)) & 15u), f[3]));
      }
      *reinterpret_cast<uint4*>(a.k_out + dst) = make_uint4(ok[0], ok[1], ok[2], ok[3]);
      *reinterpret_cast<uint4*>(a.v_out + dst) = make_uint4(ov[0], ov[1], ov[2], ov[3]);
    }
    dst += (int64_t)kStep * a.N * kHeadDim;
    kw = nk;
    vw = nv;
    tail = nt;
  }
}

template <int TOK>
cudaError_t launch_tok(CacheArgs& a, int B, bool f16, bool write, cudaStream_t st) {
  a.tiles = (a.N + TOK - 1) / TOK;
  const int64_t blocks = (int64_t)B * a.tiles;
  // Few tiles: the heads go to several blocks, until there are about eight blocks per SM.
  constexpr int kStep = kRows / TOK;
  const int steps = (a.Hkv + kStep - 1) / kStep;
  const int split = (int)std::min<int64_t>((8 * 148 + blocks - 1) / blocks, steps);
  a.heads_per_block = (steps + split - 1) / split * kStep;
  const dim3 grid((unsigned)blocks, (a.Hkv + a.heads_per_block - 1) / a.heads_per_block);
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
  // Sixteen tokens of one head at a time; with fewer tokens per sequence, that many heads instead.
  if (p.N >= 16) return launch_tok<16>(a, p.B, p.f16, write, st);
  return p.N >= 4 ? launch_tok<4>(a, p.B, p.f16, write, st) : launch_tok<1>(a, p.B, p.f16, write, st);
}

}  // namespace kascade
