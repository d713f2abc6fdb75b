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
// m and s are rounded outward.  s is a product with a little less than 1/15,
// rounded up to bfloat16 and moved up once more if 15 s is still below the
// range: 15 s is an fp32 number, so that is decided exactly.  n comes from a
// product with an approximate 1 / s.  Its remainder r = (x - m) - n s is exact
// in fp32, and where r is not clearly below s / 2 the code is settled by r and,
// where x - m was inexact, by its rounding error (two-sum).  Half-way points are
// common (a 16-bit value on an 8-bit grid), so that path is short too.
//
// What bounds both kernels: memory, 512 bytes of 16-bit rows against 160 bytes
// of cache row per token and key head.  Half a warp handles one row: a lane
// holds 8 channels of K and of V (one 16-byte load or store each), a group is
// four lanes, and one exchange with the lane four further puts the V halves of
// two groups into one word.  A block takes 16 tokens (fewer when there are few)
// through several heads, so that a token's page is looked up once and the next
// head's rows are on their way while one head's are worked on.
// Measured on one B200, 26162 tokens x 8 heads: write 45 us in half precision and 47
// in bfloat16 (3.0 to 3.1 TB/s; 313 warp instructions per two rows, so the issue
// slots, 73% busy, come before memory; 64 registers with 8 bytes spilled), read back
// 28 to 30 us (4.7 to 5.0 TB/s).
#include "common.cuh"
#include "f32x2.cuh"
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

// Minima and maxima of the halves of two words, in the data's type; a NaN stays.
template <bool F16, bool MAX>
__device__ __forceinline__ uint32_t ends2(uint32_t a, uint32_t b) {
  if constexpr (F16) {
    const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&b);
    const __half2 r = MAX ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a), y = *reinterpret_cast<const __nv_bfloat162*>(&b);
    const __nv_bfloat162 r = MAX ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

__device__ __forceinline__ float approx_rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Minimum and minus maximum of the group's values, packed in the data's type.
template <bool F16>
__device__ __forceinline__ uint32_t group_ends(const uint4& w) {
  const uint32_t lo = ends2<F16, false>(ends2<F16, false>(w.x, w.y), ends2<F16, false>(w.z, w.w));
  const uint32_t hi = ends2<F16, true>(ends2<F16, true>(w.x, w.y), ends2<F16, true>(w.z, w.w)) ^ 0x80008000u;
  uint32_t ends = ends2<F16, false>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
  ends = ends2<F16, false>(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
  return ends2<F16, false>(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
}

struct Scale {
  float s, m, inv;
  bool bad;  // a value is not finite, or the range is not
};
template <bool F16>
__device__ __forceinline__ Scale group_scale(uint32_t ends) {
  float lo, hi;
  unpack2<F16>(ends, lo, hi);
  Scale g;
  g.m = __uint_as_float(bf16_down(lo) << 16);
  const float range = __fadd_ru(-hi, -g.m);
  uint32_t s = bf16_up_pos(range * 0x1.11110cp-4f);  // 1/15 less 2^-22 of it
  if (fmaf(__uint_as_float(s << 16), 15.f, -range) < 0.f) ++s;
  g.s = __uint_as_float(s << 16);
  g.inv = approx_rcp(fmaxf(g.s, 0x1p-120f));
  g.bad = !(range < CUDART_INF_F);
  return g;
}

// Codes of this lane's 8 values; lanes 4g .. 4g+3 of the half warp are one group.
template <bool F16>
__device__ __forceinline__ uint32_t codes(const uint4& w, float s, float m, float inv) {
  float x[8], n[8], r[8];
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2<F16>(word_of(w, i), x[2 * i], x[2 * i + 1]);
  // two channels per instruction
  const uint64_t minus_m = f2_pack(-m, -m), inv2 = f2_pack(inv, inv), minus_s = f2_pack(-s, -s);
  const uint64_t magic = f2_pack(0x1.8p23f, 0x1.8p23f), minus_magic = f2_pack(-0x1.8p23f, -0x1.8p23f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t d = f2_add(f2_pack(x[i], x[i + 1]), minus_m);
    const uint64_t whole = f2_add(f2_fma(d, inv2, magic), minus_magic);  // rounds to integers
    f2_unpack(whole, n[i], n[i + 1]);
    f2_unpack(f2_fma(whole, minus_s, d), r[i], r[i + 1]);
    most = fmax3(most, fabsf(r[i]), fabsf(r[i + 1]));
  }
  if (most >= s * (0.5f - 0x1p-15f) && s > 0.f) {  // without a range all codes are 0
    if (s < 0x1p-120f) {  // 1 / s is out of range: quotients of scaled numbers
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = rintf(((x[i] - m) * 0x1p64f) / (s * 0x1p64f));
        r[i] = fmaf(-n[i], s, x[i] - m);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(r[i]) >= s * (0.5f - 0x1p-15f)) {
        const float d = x[i] - m, back = d - x[i];
        const float lost = (x[i] - (d - back)) + (-m - back);  // x - m is d + lost
        const float side = copysignf(1.f, r[i]);
        const float over = fmaf(2.f * lost, side, fmaf(2.f, fabsf(r[i]), -s));
        const bool odd = __float_as_uint(n[i] + 0x1p23f) & 1u;
        if (over > 0.f || (over == 0.f && odd)) n[i] += side;
      }
    }
  }
  // four codes in 16 bits: exact in fp32, and read off the low bits after adding 2^23
  const float a = fmaf(n[3], 4096.f, fmaf(n[2], 256.f, fmaf(n[1], 16.f, n[0]))) + 0x1p23f;
  const float b = fmaf(n[7], 4096.f, fmaf(n[6], 256.f, fmaf(n[5], 16.f, n[4]))) + 0x1p23f;
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
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
    const int page = a.block_table[(int64_t)b * a.max_pages + pi];
    if (page < 0 || page >= a.num_pages) {
      if (first) flag_status(a.status, kStatusBadIndex);
      return -1;
    }
    return (int64_t)page * a.Hkv * a.page_size + (t - pi * a.page_size);
  }
};

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const CacheArgs a) {
  overlap_launches();
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
    ck = load16(k);
    cv = load16(v);
  }
  const int passes = (p.h_end - (int)blockIdx.y * a.heads_per_block + kStep - 1) / kStep;  // of the block
  for (int i = 0, h = p.h; i < passes; ++i, h += kStep) {
    const bool live = p.row >= 0 && h < p.h_end;
    uint4 nk = make_uint4(0, 0, 0, 0), nv = nk;
    k += (int64_t)kStep * a.ks.h;
    v += (int64_t)kStep * a.vs.h;
    if (p.row >= 0 && h + kStep < p.h_end) {
      nk = load16(k);
      nv = load16(v);
    }
    // even lanes work out K's scale of their group, odd lanes V's
    const uint32_t ek = group_ends<F16>(ck), ev = group_ends<F16>(cv);
    Scale mine = group_scale<F16>((l & 1) ? ev : ek);
    const uint32_t bits = mine.bad ? 0x7fc00000u : (__float_as_uint(mine.m) | (__float_as_uint(mine.s) >> 16));
    const int lk = threadIdx.x & 30, lv = lk + 1;
    const uint32_t tk = __shfl_sync(0xffffffffu, bits, lk), tv = __shfl_sync(0xffffffffu, bits, lv);
    const float ik = __shfl_sync(0xffffffffu, mine.inv, lk), iv = __shfl_sync(0xffffffffu, mine.inv, lv);
    // a group that is not finite reads back as NaN: scale 0, minimum NaN (its codes are any)
    const uint32_t kwords = codes<F16>(ck, bf16_lo(tk), bf16_hi(tk), ik);
    const uint32_t vwords = codes<F16>(cv, bf16_lo(tv), bf16_hi(tv), iv);
    // lane (g, j) holds channels 32g + 8j ..: V half words of lane groups r = 2j and 2j + 1.  Even g
    // builds the word of r = 2j (halves g, g + 1), odd g that of r = 2j + 1.
    const uint32_t give = odd ? vwords & 0xffffu : vwords >> 16;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
    const uint32_t vword = odd ? (got | (vwords & 0xffff0000u)) : ((vwords & 0xffffu) | (got << 16));
    // bfloat16 number l of the tail: K scales, K minima, V scales, V minima, by groups
    const int src = (threadIdx.x & 16) + 4 * (l & 3);
    const uint32_t wk = __shfl_sync(0xffffffffu, tk, src), wv = __shfl_sync(0xffffffffu, tv, src);
    const uint32_t tw = l < 8 ? wk : wv;
    if (live) {
      bad |= mine.bad;
      reinterpret_cast<uint32_t*>(dst)[4 * j + g] = kwords;
      reinterpret_cast<uint32_t*>(dst + kQ4V)[2 * (2 * j + (int)odd) + (g >> 1)] = vword;
      reinterpret_cast<uint16_t*>(dst + kQ4Tail)[l] = (uint16_t)((l & 4) ? tw >> 16 : tw);
    }
    dst += (int64_t)kStep * a.page_size * kQ4Row;
    ck = nk;
    cv = nv;
  }
  if (bad) flag_status(a.status, kStatusNonFinite);
}

// minimum + scale * code of the 8 codes in a word, in 16 bits.  A nibble at bit 4i, put below the
// exponent of 2^23, is that number plus code · 16^i: nothing is shifted or converted.
template <bool F16>
__device__ __forceinline__ uint4 values(uint32_t w, float s, float m) {
  float v[8];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t h = half ? w >> 16 : w;
    float unit = s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float n = __uint_as_float((h & (15u << (4 * i))) | 0x4b000000u) - 0x1p23f;
      v[4 * half + i] = fmaf(unit, n, m);
      unit *= 0.0625f;
    }
  }
  return make_uint4(pack_x2<F16>(v[0], v[1]), pack_x2<F16>(v[2], v[3]), pack_x2<F16>(v[4], v[5]),
                    pack_x2<F16>(v[6], v[7]));
}

template <int TOK, bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  overlap_launches();
  const Place<TOK> p(a);
  if (!__any_sync(0xffffffffu, p.row >= 0)) return;
  const int l = threadIdx.x % 16;
  const int g = l >> 2, j = l & 3;
  const bool odd = g & 1;
  constexpr int kStep = kRows / TOK;
  const uint8_t* src = a.pages + (p.row + (int64_t)p.h * a.page_size) * kQ4Row;
  uint32_t kw = 0, vw = 0, tail = 0;
  auto load = [&](uint32_t& k, uint32_t& v, uint32_t& t) {
    k = reinterpret_cast<const uint32_t*>(src)[4 * j + g];
    v = reinterpret_cast<const uint32_t*>(src + kQ4V)[2 * (2 * j + (int)odd) + (g >> 1)];
    t = reinterpret_cast<const uint16_t*>(src + kQ4Tail)[l];
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
      const uint4 ok = values<F16>(kw, f[0], f[1]), ov = values<F16>(vw, f[2], f[3]);
      *reinterpret_cast<uint4*>(a.k_out + dst) = ok;
      *reinterpret_cast<uint4*>(a.v_out + dst) = ov;
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
  return launch_overlapped(kern, grid, kThreads, 0, st, a);
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
