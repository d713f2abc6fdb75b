// Decode attention over the 4-bit paged cache (row format in q4.cuh): the anchor
// (every token, pooled probabilities) and the reuse layer (selected tokens).
//
// With K, V = minimum + scale * code per row and group, for each query head:
//   s_t = scale · q · K_t;  out = sum_t softmax(s)_t V_t;  lse = log sum_t exp(s_t)
//
// The codes are never turned into values.  A group's scale and minimum are the
// same for its 32 channels, so
//   q · K_t    = sum_g [ ks_{t,g} (q_g · n_{t,g}) + km_{t,g} sum(q_g) ]
//   out_d      = sum_t (p_t vs_{t,g}) n_{t,d}  +  sum_t p_t vm_{t,g}      (d in group g)
// and mma.sync multiplies the codes n themselves: a nibble in bits 4..7 of a half
// word (K) or in bits 6..9 (V) is the half-precision subnormal n · 2^-20 or n · 2^-18,
// exact.  (tcgen05 would want the codes unpacked into shared or tensor memory first:
// 512 bytes written and read again per row of 160.)  The other operand carries the
// powers of two: q (scaled per head so that its largest element is near 2^14; a
// bfloat16 or half q is then exact in half precision down to 2^-28 of that) and
// p · vs (below).
//   * S^T[16 tokens x 8 heads]: two m16n8k16 per scale group, whose fp32 sums
//     the row's scales weight; the minima come in by one more mma, bfloat16
//     minima against sum(q_g) split into three bfloat16 terms (24 bits).
//   * O^T[128 channels x 8 heads]: per group the weights p · vs are the B operand,
//     in two half-precision terms (22 bits).  One alone left outputs 4e-4 off before
//     their own rounding, which shows (bfloat16, 16 x 32K: 1.71e-3 from 64 bits
//     instead of 1.67e-3); the second costs 5% there (147 to 154.6 us) and 14% with
//     8 heads.  Weights of different tokens may differ by any power of two, so each
//     head and group has its own factor c, a power of two: the first weights, and any
//     that would pass 2^15, are put near 2^8, where weights 2^22 times smaller still
//     keep 11 bits.  When the running maximum moves, c takes up the change and the
//     sums stay.  The minima are summed in fp32 (8 sums per lane).
//   * The running maximum moves only when a score exceeds it by 8 (weights then
//     reach 2^8 instead of 1), so most stages need one vote instead of a
//     reduction and a rescale of the sums.  V up to 2^116 / T and K up to 2^100 are
//     safe from overflow on the way.
//   * Up to 4 heads fill half the columns.  The other half then serves the second
//     16 rows of a stage (scores) or the weights' second terms (values).
//
// What bounds it, on one B200 (16 sequences of 32K, 32 heads on 8, bfloat16): the
// first kernel reads 671 MB in 144 to 155 us (by box), 4.3 to 4.7 TB/s; loads and
// scores alone take 115 us, which is memory.  No unit is full beside it (issue
// slots 62%, logic pipe 56%, tensor pipe 23%): it is the latency of 730 warp
// instructions per 32 rows at 12 warps per SM, first stall a fixed-latency wait.
// 168 registers suffice for up to 4 heads; the variants for more spill (anchor 48
// bytes stored and 68 loaded, reuse 8 and 8).  A warp owns a run of rows and a ring
// of two 32-row stages in shared memory that bulk copies fill: a half stage is 2560
// adjacent bytes.  No registers hold data in flight, and three blocks of four warps
// per SM leave each thread 168: with four blocks and 128 registers it was 10%
// slower, with a third stage no faster.
// A reuse stage is 32 rows of 160 bytes by 16-byte copies, two lanes to a sector;
// one bulk copy per row took half as long again.  Rows lie 160 bytes apart, which is
// 8 banks mod 32; the fragment rows are taken in the order 0 6 1 7 2 4 3 5 so
// that the 16-byte K reads (pairs of rows) and the 8-byte V reads (every second
// fragment row) both meet different banks.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "q4.cuh"
#include "tcgen05.cuh"

#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>

namespace kascade {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStageRows = 32;
constexpr int kStages = 2;
constexpr int kCtasPerSm = 3;
constexpr uint32_t kStageBytes = kStageRows * kQ4Row;
constexpr uint32_t kRingBytes = kWarps * kStages * kStageBytes;
constexpr uint32_t kSmemBytes = kRingBytes + 128;
constexpr int kSlots = kCtasPerSm * 148;  // resident blocks
constexpr int kNoToken = -2147483647 - 1;  // lanes past the end
constexpr float kLn2 = 0.6931471805599453f;
static_assert(kRingBytes >= kWarps * 8 * kHeadDim * sizeof(float), "the merge overlays the rings");

struct Q4Args {
  const uint16_t* q;
  const uint8_t* pages;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  uint32_t page_mul, page_shift;  // t / page_size = umulhi(t, page_mul) >> page_shift, 0 <= t < 2^31
  const int32_t* seq_len;
  const int32_t* idx;
  const int32_t* idx_k;
  const int32_t* head_map;
  int k_max;
  int Hq, Hkv, G, max_T;
  int B;
  int give_up;     // anchor: the block that gives up before its first copy (self-test), or -1
  float scale_log2;
  float* logits;   // anchor: [B, Hkv, max_T, G] base-2 scaled logits
  int2* parts;     // [B*Hkv]: first and last block of a unit
  float* part_ml;  // [blocks + B*Hkv, G, 2]
  float* part_o;   // [blocks + B*Hkv, G, 128]
  uint16_t* out;   // reuse
  float* lse;
  unsigned* status;
};

// What exponentials are taken relative to: the maximum, or 0 where there is no finite score yet
// (exp2(-inf - 0) is then 0).  A maximum ignores NaN; the sum of the exponentials keeps it, so a
// NaN score reaches the results whether or not it is alone.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float lse2_of(float m, float l) { return l == 0.f ? -INFINITY : finite_max(m) + __log2f(l); }

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

// Read once: these lines leave L2 first, so that the logits find room there until they are pooled.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// Untiled copy of `bytes` (a multiple of 16, both ends 16-byte aligned) that completes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// Asynchronous copy of 16 bytes (zeros where src_bytes is 0).  The 64-byte hint is for rows of 160 bytes:
// without it whole 128-byte lines come from memory, 256 bytes a row instead of 192 (105 against 80 MB for
// 16 sequences of 32K; 26.6 against 26.2 us, ragged 44.45 against 44.15).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::64B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(src_bytes), "l"(policy)
               : "memory");
}

// d = a b: a product that starts a sum (the sums' registers need no zeros first).
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// bfloat16 number g of two words.
__device__ __forceinline__ float tail_at(uint32_t w01, uint32_t w23, int g) {
  const uint32_t w = g < 2 ? w01 : w23;
  return (g & 1) ? bf16_hi(w) : bf16_lo(w);
}

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The query operand: heads are the 8 columns, head gid of a lane's fragments.  With PAIR there are
// two of them, for the first and the second 16 rows of a stage: the heads in columns 0..3 and zeros
// in the others, and zeros there and the heads in columns 4..7.  Both products go to one sum, which
// then holds the scores of 32 rows.
template <bool PAIR>
struct Query {
  uint32_t b[PAIR ? 2 : 1][4][4];  // per scale group: the two k16 steps' b0, b1
  uint32_t s[PAIR ? 2 : 1][2];     // sum(q_g) against the minima
  float f0, f1;                    // factors of heads 2 tig, 2 tig + 1 to base-2 logits (times 2^20)
};

// The lane's query words: 8 channels of each scale group, of head gid (PAIR: gid & 3).
template <bool PAIR>
__device__ __forceinline__ void fetch_query(uint4 (&w)[4], const uint16_t* q, int G, int gid, int tig) {
  const int head = PAIR ? gid & 3 : gid;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    // columns past the last head are padding: load a valid row and zero it
    w[g] = load16(q + (head < G ? head : G - 1) * kHeadDim + 32 * g + 8 * tig);
    if (head >= G) w[g] = make_uint4(0, 0, 0, 0);
  }
}

template <bool PAIR, bool F16>
__device__ __forceinline__ void build_query(Query<PAIR>& x, const uint4 (&w)[4], float scale_log2, int gid, int tig) {
  float v[4][8];
  float top = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack2<F16>(word_of(w[g], i), v[g][2 * i], v[g][2 * i + 1]);
      top = fmaxf(top, fmaxf(fabsf(v[g][2 * i]), fabsf(v[g][2 * i + 1])));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // q' = q 2^-e with its largest element in [2^14, 2^15); e = 0 for a zero or non-finite head
  int e = (int)(__float_as_uint(top) >> 23) - 127 - 14;
  if (!(top > 0.f) || e > 127 - 14) e = 0;
  e = max(e, -120);
  const float down = pow2i(-e);
  float sum[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    sum[g] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[g][i] *= down;
      sum[g] += v[g][i];
    }
    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
    sum[g] *= 0x1p-20f;  // the codes' unit
#pragma unroll
    for (int i = 0; i < 4; ++i) x.b[0][g][i] = pack_f16x2(v[g][i], v[g][i + 4]);  // code j of a word is in half j / 4
  }
  // k = 0..3: leading term of sum_g against minimum g, 4..7: second, 8..11: third, 12..15: nothing
  const float u0 = (tig & 1) ? sum[2] : sum[0], u1 = (tig & 1) ? sum[3] : sum[1];
  const uint32_t hi = pack_bf16x2(u0, u1);
  const float r0 = u0 - bf16_lo(hi), r1 = u1 - bf16_hi(hi);
  const uint32_t mid = pack_bf16x2(r0, r1);
  const uint32_t lo = pack_bf16x2(r0 - bf16_lo(mid), r1 - bf16_hi(mid));
  x.s[0][0] = tig < 2 ? hi : mid;
  x.s[0][1] = tig < 2 ? lo : 0u;
  if constexpr (PAIR) {
    const uint32_t m = gid < 4 ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t& q0 = x.b[0][i >> 2][i & 3];
      q0 &= m;
      // lanes gid and gid ^ 4 change places (a mask instead would be applied anew in every stage)
      x.b[1][i >> 2][i & 3] = __shfl_xor_sync(0xffffffffu, q0, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x.s[0][i] &= m;
      x.s[1][i] = __shfl_xor_sync(0xffffffffu, x.s[0][i], 16);
    }
  }
  const float f = scale_log2 * pow2i(e);
  x.f0 = __shfl_sync(0xffffffffu, f, 8 * tig);
  x.f1 = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
}

// Bytes 1 and 3 of w as two half words.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t w) { return __byte_perm(w, 0u, 0x4341); }

// Products of the codes in words wa and wb (of a lane's rows a and b) with the query.  Every nibble is
// brought to bits 4..7 of its half word: the matrix unit lines products up by the operands' exponents,
// which for a subnormal number say nothing of its leading zeros, and so many bits the sum then lacks.
// (With half of the nibbles at bits 0..3 the log-sum-exp was off by 2e-7 instead of 5e-8.)
template <bool FIRST>
__device__ __forceinline__ void score_codes(float (&d)[4], uint32_t wa, uint32_t wb, const uint32_t (&q)[4]) {
  constexpr uint32_t kNibble = 0x00f000f0u;
  const uint32_t la = (wa << 4) & kNibble, lb = (wb << 4) & kNibble;
  if constexpr (FIRST) mma_f16_first(d, la, lb, wa & kNibble, wb & kNibble, q[0], q[1]);
  else mma_f16_16816(d, la, lb, wa & kNibble, wb & kNibble, q[0], q[1]);
  const uint32_t ua = upper_bytes(wa), ub = upper_bytes(wb);
  mma_f16_16816(d, (ua << 4) & kNibble, (ub << 4) & kNibble, ua & kNibble, ub & kNibble, q[2], q[3]);
}

// Scores of 16 (PAIR: 32) rows at shared address `rows`, in units of 2^-20: c[0], c[1] are the lane's
// two heads of its row a, c[2], c[3] of row b = a + 8.  `mine` is the address of the lane's own row a.
template <bool PAIR>
__device__ __forceinline__ void scores(const Query<PAIR>& x, uint32_t rows, uint32_t row_a, uint32_t mine, int tig,
                                       float (&c)[4]) {
  constexpr int kSets = PAIR ? 2 : 1;
  const uint2 sa = lds64(mine + kQ4Tail), sb = lds64(mine + 8 * kQ4Row + kQ4Tail);
  uint4 ka[kSets], kb[kSets];
#pragma unroll
  for (int u = 0; u < kSets; ++u) {
    const uint32_t a = rows + 16 * u * kQ4Row + row_a, b = a + 8 * kQ4Row;
    ka[u] = lds128(a + 16 * tig);
    kb[u] = lds128(b + 16 * tig);
    const uint32_t ma = lds32(a + kQ4Tail + 8 + 4 * (tig & 1)), mb = lds32(b + kQ4Tail + 8 + 4 * (tig & 1));
    if (u == 0) mma_bf16_first(c, ma, mb, ma, mb, x.s[u][0], x.s[u][1]);
    else mma_bf16_16816(c, ma, mb, ma, mb, x.s[u][0], x.s[u][1]);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float d[4];
    score_codes<true>(d, word_of(ka[0], g), word_of(kb[0], g), x.b[0][g]);
    if constexpr (PAIR) score_codes<false>(d, word_of(ka[1], g), word_of(kb[1], g), x.b[1][g]);
    const float fa = tail_at(sa.x, sa.y, g), fb = tail_at(sb.x, sb.y, g);
    c[0] = fmaf(fa, d[0], c[0]);
    c[1] = fmaf(fa, d[1], c[1]);
    c[2] = fmaf(fb, d[2], c[2]);
    c[3] = fmaf(fb, d[3], c[3]);
  }
}

// Running state of a warp.  A lane's heads are 2 tig, 2 tig + 1 (PAIR: 2 (tig & 1) and the next).
struct State {
  float m0, m1, l0, l1;
  // [group][channel pair]: rows gid = channel 4 gid + 2 pair + 16 times the next one, gid + 8 = the latter
  float o[4][2][4];
  float z[4][2];     // sums of p · vm, this lane's rows
  float c[4][2];     // [group][head]: the sums o and the weights that enter them are times this power of two
};

constexpr int kMaxC = 127 + 100;  // largest c that a sum starts from, 2^100, as a biased exponent

// Over the lanes that hold the same head (tig), with PAIR also those of the other 16 rows.
template <bool PAIR>
__device__ __forceinline__ float head_max(float x) {
  if constexpr (PAIR) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  return warp_max_xor_gid(x);
}
template <bool PAIR>
__device__ __forceinline__ float head_sum(float x) {
  if constexpr (PAIR) x += __shfl_xor_sync(0xffffffffu, x, 2);
  return warp_sum_xor_gid(x);
}

__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23); }  // x >= 0
__device__ __forceinline__ float biased_pow2(int e) { return __int_as_float(max(e, 0) << 23); }

__device__ __forceinline__ void scale_sums(State& w, int g, int h, float f) {
  w.o[g][0][h] *= f;
  w.o[g][0][2 + h] *= f;
  w.o[g][1][h] *= f;
  w.o[g][1][2 + h] *= f;
}

// The weights' unit of head h has grown by 1 / al, 0 <= al <= 1 (NaN: the head is lost anyway): c
// takes up the power of two, as far as it may, and the sums what is left.
__device__ __forceinline__ void rebase(State& w, int h, float al) {
  const bool some = al > 0.f;
  const int up = some ? 127 - exponent_of(al) : 512;
  const float rest = some ? __uint_as_float((__float_as_uint(al) & 0x7fffffu) | 0x3f800000u) : 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int e = exponent_of(w.c[g][h]) + up, n = min(e, kMaxC);
    w.c[g][h] = biased_pow2(n);
    scale_sums(w, g, h, rest * biased_pow2(127 + n - e));
    w.z[g][h] *= al;
  }
}

// A stage's weights as the B operands of the value products, [block of 16 rows][group]: rounded to half
// precision, and what that rounding left.  With PAIR the latter stands in the columns that have no head
// (second[] is not used): columns 0..3 of block 0 hold the weights and 4..7 the rest, of block 1 the
// other way round; the merge adds the two.
struct Weights {
  uint32_t first[2][4][2], second[2][4][2];
};

// p: exponentials of the lane's rows a and b (layout of scores), of each set of rows.  `tail` is the
// address of the first row a's V scales.  Also adds the minima's sums.
template <bool PAIR>
__device__ __forceinline__ void weights(State& w, uint32_t tail, const float (&p)[PAIR ? 1 : 2][4], int tig,
                                        Weights& out) {
  constexpr int kSets = PAIR ? 1 : 2;
  uint4 t[kSets][2];
#pragma unroll
  for (int u = 0; u < 2 * kSets; ++u) t[u >> 1][u & 1] = lds128(tail + 8 * u * kQ4Row);
  uint32_t hi[kSets][4][2], lo[kSets][4][2], top = 0;
  auto pack = [&](int g) {
#pragma unroll
    for (int u = 0; u < 2 * kSets; ++u) {
      const float f = tail_at(t[u >> 1][u & 1].x, t[u >> 1][u & 1].y, g);
      const float* q = &p[u >> 1][2 * (u & 1)];
      float w0, w1;
      f2_unpack(f2_mul(f2_pack(q[0], q[1]), f2_pack(w.c[g][0], w.c[g][1])), w0, w1);
      w0 *= f;
      w1 *= f;
      const uint32_t h = pack_f16x2(w0, w1);
      hi[u >> 1][g][u & 1] = h;
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
      lo[u >> 1][g][u & 1] = pack_f16x2(w0 - back.x, w1 - back.y);
    }
  };
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    pack(g);
#pragma unroll
    for (int u = 0; u < kSets; ++u) top = __vimax3_u16x2(top, hi[u][g][0], hi[u][g][1]);  // not negative: as integers
  }
  if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7800u || top >= 0x78000000u)) {
    // A weight has reached 2^15: factors that put the largest weight of such a head and group in
    // [2^7, 2^8).  A weight that is not finite spoils its own sums and moves no factor.
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < 2 * kSets; ++u) {
          const float y = p[u >> 1][2 * (u & 1) + h] * tail_at(t[u >> 1][u & 1].x, t[u >> 1][u & 1].y, g);
          x = fmaxf(x, y < INFINITY ? y : 0.f);
        }
        x = head_max<PAIR>(x);
        if (x * w.c[g][h] >= 0x1p15f) {
          const int n = 127 + 7 + 127 - max(exponent_of(x), 27);  // c stays within 2^107
          scale_sums(w, g, h, biased_pow2(127 + n - exponent_of(w.c[g][h])));
          w.c[g][h] = biased_pow2(n);
        }
      }
      pack(g);
    }
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int u = 0; u < kSets; ++u) {
      const float za = tail_at(t[u][0].z, t[u][0].w, g), zb = tail_at(t[u][1].z, t[u][1].w, g);
      w.z[g][0] = fmaf(p[u][0], za, fmaf(p[u][2], zb, w.z[g][0]));
      w.z[g][1] = fmaf(p[u][1], za, fmaf(p[u][3], zb, w.z[g][1]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (PAIR) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, lo[0][g][i], 2);
        out.first[0][g][i] = movmatrix_trans(tig < 2 ? hi[0][g][i] : other);
        out.first[1][g][i] = movmatrix_trans(tig < 2 ? other : hi[0][g][i]);
      } else {
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
          out.first[u][g][i] = movmatrix_trans(hi[u][g][i]);
          out.second[u][g][i] = movmatrix_trans(lo[u][g][i]);
        }
      }
    }
  }
}

__device__ __forceinline__ void add2(float& x, float& y, float dx, float dy) {
  f2_unpack(f2_add(f2_pack(x, y), f2_pack(dx, dy)), x, y);
}

// O += V P for the 32 rows at `rows`.  The products of a stage start from zero and are added to the
// sums in fp32: the matrix unit cuts each product off at the last bit of the sum that it joins, always
// toward zero, and 2000 products of one sign would be 2^-15 short, which the minima, summed apart,
// would not be (at 128K tokens 0.5% of the output).  Codes stand two bits higher than the bytes they are
// taken from, in bits 6..9 of a half word: the unit lines products up by the operands' exponents, so every
// bit in front of a subnormal code is one less for its products.  In bits 4..7 outputs were 7e-5 off
// before their rounding (2.17e-4 instead of 2.10e-4 in half precision), now 2e-5; 159 instead of 154.6 us.
template <bool PAIR>
__device__ __forceinline__ void values(State& w, uint32_t rows, int gid, int tig, const Weights& b) {
  uint2 e[2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    // V rows of this lane's k pairs: fragment rows 2 tig, 2 tig + 1 and those + 8
    const uint32_t v0 = rows + (uint32_t)(16 * u + tig) * kQ4Row + kQ4V + 8 * gid;
    const uint32_t v1 = rows + (uint32_t)(16 * u + 4 + (tig ^ 2)) * kQ4Row + kQ4V + 8 * gid;
    e[u][0] = lds64(v0);
    e[u][1] = lds64(v1);
    e[u][2] = lds64(v0 + 8 * kQ4Row);
    e[u][3] = lds64(v1 + 8 * kQ4Row);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    constexpr uint32_t kHigh = 0x03c003c0u;        // high nibbles of the shifted bytes
    const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;  // half g % 2 of both rows' words
    float d[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // whole bytes, and their high nibbles: the merge takes the difference of the two sums
      const uint32_t x = __byte_perm(g < 2 ? e[u][0].x : e[u][0].y, g < 2 ? e[u][1].x : e[u][1].y, sel);
      const uint32_t y = __byte_perm(g < 2 ? e[u][2].x : e[u][2].y, g < 2 ? e[u][3].x : e[u][3].y, sel);
      const uint32_t a0 = (x & 0x00ff00ffu) << 2, a1 = a0 & kHigh, a2 = (y & 0x00ff00ffu) << 2, a3 = a2 & kHigh;
      const uint32_t b0 = upper_bytes(x) << 2, b1 = b0 & kHigh, b2 = upper_bytes(y) << 2, b3 = b2 & kHigh;
      if (u == 0) {
        mma_f16_first(d[0], a0, a1, a2, a3, b.first[u][g][0], b.first[u][g][1]);
        mma_f16_first(d[1], b0, b1, b2, b3, b.first[u][g][0], b.first[u][g][1]);
      } else {
        mma_f16_16816(d[0], a0, a1, a2, a3, b.first[u][g][0], b.first[u][g][1]);
        mma_f16_16816(d[1], b0, b1, b2, b3, b.first[u][g][0], b.first[u][g][1]);
      }
      if constexpr (!PAIR) {
        mma_f16_16816(d[0], a0, a1, a2, a3, b.second[u][g][0], b.second[u][g][1]);
        mma_f16_16816(d[1], b0, b1, b2, b3, b.second[u][g][0], b.second[u][g][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      add2(w.o[g][0][i], w.o[g][0][i + 1], d[0][i], d[0][i + 1]);
      add2(w.o[g][1][i], w.o[g][1][i + 1], d[1][i], d[1][i + 1]);
    }
  }
}

// The anchor's work is the stages (32 tokens) of all (sequence, key head) units, one after the other,
// and each block takes an equal share of them: the lengths are known on the device alone, and a
// batch of one long and many short sequences then keeps every SM busy to the end.  Starting and
// merging a unit costs a block about as much as kUnitCost stages, so a unit is that much longer on
// the line.  A block's part of unit u goes to slot block + u of the partial results: both only ever
// grow along the line, so no two parts meet, and a unit's slots follow one another.
// Measured with 4, 8, 12, 16 and 24: 65536 ... 0 tokens (8 sequences, 8 heads, half) 50.1, 34.8, 33.2, 33.2, 33.5 us;
// one of 64K beside 31 of 300 45.7, 42.4, 43.2, 44.2, 46.4; 64 of 200 to 2153 48.3, 45.9, 46.1, 46.7, 48.1.
constexpr int kUnitCost = 12;
__device__ __forceinline__ int stages_of(int T, int max_T) {
  return T > 0 && T <= max_T ? (T + kStageRows - 1) / kStageRows : 0;
}
__device__ __forceinline__ int length_of(int T, int max_T) {  // on the line
  const int n = stages_of(T, max_T);
  return n ? n + kUnitCost : 0;
}
// Length of all sequences, for one key head.  `mine` is the length of sequence `lane`, loaded before.
__device__ __forceinline__ int64_t line_length(const int32_t* seq_len, int B, int max_T, int mine) {
  const int lane = threadIdx.x & 31;
  int64_t total = __reduce_add_sync(0xffffffffu, (unsigned)length_of(mine, max_T));
#pragma unroll 4
  for (int i = 32; i < B; i += 32)
    total += __reduce_add_sync(0xffffffffu, (unsigned)(i + lane < B ? length_of(seq_len[i + lane], max_T) : 0));
  return total;
}
// Blocks that take part: each has some of the line, each warp has a stage where there are enough.
__device__ __forceinline__ int working_blocks(int64_t length, int blocks) {
  return (int)min((int64_t)blocks, (length + kWarps - 1) / kWarps);
}

// PAIR: at most 4 query heads per key head.  The scores of a stage's first 16 rows are in columns 0..3
// and those of the second in 4..7 (see Query), so exponentials, weights and minima cost half.
template <bool GATHER, bool PAIR, bool F16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_q4_kernel(const Q4Args a) {
  // (clusters of the next reuse call, were they let in early, would leave some SMs to fewer of its blocks)
  if (!GATHER) allow_dependents_launch();
  grid_dependency_wait();
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float sm_m[kWarps][8], sm_l[kWarps][8];
  __shared__ float sm_po[8][kHeadDim], sm_pm[8], sm_pl[8];  // reuse: this block's part for the cluster's merge
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // known to be the same in all lanes
  const int lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int G = a.G;

  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * kStages * kStageBytes;
  const uint32_t bar = smem_u32(&bars[warp][0]);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 2);
    mbar_fence_init();
  }
  __syncwarp();

  int b, h, T, i_begin, i_end, token_0 = 0;
  const int step = GATHER ? (int)gridDim.x * kWarps * kStageRows : kStageRows;  // from one stage of a warp to its next
  const int32_t* sel = nullptr;
  int64_t left = 0;  // anchor: what this block still has of the line
  int at = 0;        // and where in its unit that starts
  if constexpr (GATHER) {
    b = blockIdx.z;
    h = blockIdx.y;
    T = a.seq_len[b];
    const int am = a.head_map[h], row = b * a.Hkv + min(max(am, 0), a.Hkv - 1);
    int n_items = a.idx_k[row];
    const bool ok = T >= 0 && T <= a.max_T && am >= 0 && am < a.Hkv && n_items >= 0 && n_items <= a.k_max;
    sel = a.idx + (int64_t)row * a.k_max;
    if (!ok && threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, kStatusBadIndex);
    if (!ok || T == 0) n_items = 0;  // nothing to gather from an empty sequence
    // the cluster's warps take the row's stages in turn: even shares, whatever its length
    i_begin = ((int)blockIdx.x * kWarps + warp) * kStageRows;
    i_end = n_items;
    // the first indices do not wait for the row's length
    token_0 = i_begin + lane < a.k_max ? sel[i_begin + lane] : 0;
  } else {
    const int mine = lane < a.B ? a.seq_len[lane] : 0;
    const int64_t total = line_length(a.seq_len, a.B, a.max_T, mine) * a.Hkv;
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < a.B; i += kThreads)
        if (a.seq_len[i] < 0 || a.seq_len[i] > a.max_T) flag_status(a.status, kStatusBadIndex);
    const int blocks = working_blocks(total, gridDim.x);
    if ((int)blockIdx.x >= blocks) return;
    const int64_t lo = total * blockIdx.x / blocks;
    left = total * (blockIdx.x + 1) / blocks - lo;
    b = h = T = 0;
    int64_t base = 0;
    for (int i = 0; i < a.B; i += 32) {  // the sequence that holds lo
      const int len = i == 0 ? mine : i + lane < a.B ? a.seq_len[i + lane] : 0, n = length_of(len, a.max_T);
      int64_t end = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += x;
      }
      end = (end + base) * a.Hkv;
      const uint32_t past = __ballot_sync(0xffffffffu, end > lo);
      if (past) {
        const int l = __ffs(past) - 1;
        const int64_t in = lo - (__shfl_sync(0xffffffffu, end, l) - (int64_t)__shfl_sync(0xffffffffu, n, l) * a.Hkv);
        const int per = __shfl_sync(0xffffffffu, n, l);
        T = __shfl_sync(0xffffffffu, len, l);
        b = i + l;
        h = (int)(in / per);
        at = (int)(in - (int64_t)h * per);
        break;
      }
      base = __shfl_sync(0xffffffffu, end, 31) / a.Hkv;
    }
  }
  const int tok_a = (gid & 1) ? 4 + ((gid >> 1) ^ 2) : gid >> 1;  // token of fragment row gid
  const uint32_t row_a = (uint32_t)tok_a * kQ4Row;
  // PAIR: this lane's rows of a stage are the first 16 or, from tig 2 on, the second
  const uint32_t half = PAIR && tig >= 2 ? 16 : 0;
  const int col = PAIR ? 2 * (tig & 1) : 2 * tig;  // the lane's first head
  const uint64_t policy = read_once_policy();
  int st = 0, phase = 0;
  bool bad = false;  // an index or page out of range was met
  // A block whose wait for a copy gave up copies no more, but goes on along its share: each part that it
  // owes has the sum NaN, which the second kernel hands to all results of that unit.  (Without that they
  // would be made of an earlier call's parts, as far as the workspace holds some.)
  bool alive = GATHER || (int)blockIdx.x != a.give_up;

  while (true) {
    if constexpr (!GATHER) {
      const int n = stages_of(T, a.max_T), end = (int)min((int64_t)at + left, (int64_t)(n + kUnitCost));
      if (end <= max(at, kUnitCost)) return;  // nothing left, or no stage of the last unit
      left -= end - at;
      const int s0 = max(at - kUnitCost, 0), ns = end - kUnitCost - s0;
      if (threadIdx.x == 0) {
        int2* parts = a.parts + ((int64_t)b * a.Hkv + h);
        if (s0 == 0) parts->x = (int)blockIdx.x;
        if (s0 + ns == n) parts->y = (int)blockIdx.x;
        if (!alive) flag_status(a.status, kStatusTimeout);
      }
      i_begin = (s0 + (int)((int64_t)ns * warp / kWarps)) * kStageRows;
      i_end = min((s0 + (int)((int64_t)ns * (warp + 1) / kWarps)) * kStageRows, T);
    }
    const int64_t bh = (int64_t)b * a.Hkv + h;
    const int n_iter = alive && i_end > i_begin ? (i_end - i_begin + step - 1) / step : 0;
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;

    // Row addresses run ahead of the copies: the selected token is loaded two stages early, its page one,
    // and neither is looked at before the next stage's turn.  The anchor needs one row per half stage: 16
    // tokens that start at a multiple of 16 lie in one page, one behind the other.
    auto load_token = [&](int it) -> int {
      const int i = i_begin + step * it + (GATHER ? lane : lane & 16);
      if (i >= i_end) return kNoToken;
      return GATHER ? sel[i] : i;
    };
    // the first token (reuse) or page (anchor) is on its way while q is
    int token_2 = !GATHER ? load_token(0) : i_begin + lane < i_end ? token_0 : kNoToken, token_1 = kNoToken, page_1 = 0,
        page_index = 0;
    auto load_page = [&](int it) {  // of stage it, whose tokens have been loaded; then the tokens of it + 1
      token_1 = token_2;
      if (GATHER && (token_1 < 0 || token_1 >= T)) {
        bad |= i_begin + step * it + lane < i_end;
        token_1 = kNoToken;
      }
      if (token_1 != kNoToken) {
        page_index = (int)(__umulhi((uint32_t)token_1, a.page_mul) >> a.page_shift);
        page_1 = table[page_index];
      }
      token_2 = load_token(it + 1);
    };
    if (!GATHER) load_page(0);
    uint32_t masks[kStages];  // rows present, stage by stage in order of use
    auto issue = [&](int it, int st, uint32_t& mask) {
      // in the page store; of no meaning (and so unsigned) unless the token and its page are good
      const int place = (int)(((uint32_t)page_1 * (uint32_t)a.Hkv + (uint32_t)h) * (uint32_t)a.page_size +
                              ((uint32_t)token_1 - (uint32_t)page_index * (uint32_t)a.page_size));
      const bool here = token_1 != kNoToken, good = (unsigned)page_1 < (unsigned)a.num_pages;
      bad |= here && !good;
      const uint32_t dst = ring + (uint32_t)st * kStageBytes;
      if constexpr (GATHER) {
        const int row = here && good ? place : -1;
        load_page(it + 1);
        mask = __ballot_sync(0xffffffffu, row >= 0);
        // 320 chunks of 16 bytes, ten to a row; the two of a 32-byte sector go to neighbouring lanes
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const int u = lane + 2 * i, r = (u * 205) >> 11;  // (lane + 32 i) / 10 = r + 3 i
          const int pl = __shfl_sync(0xffffffffu, row, r + 3 * i);
          copy16(dst + 16 * lane + 512 * i, a.pages + ((int64_t)max(pl, 0) * kQ4Row + 16 * (u - 10 * r)),
                 pl >= 0 ? 16 : 0, policy);
        }
      } else {
        const int rows = here && good ? min(i_end - token_1, 16) : 0;
        load_page(it + 1);
        mask = __ballot_sync(0xffffffffu, (lane & 15) < rows);
        if ((lane & 15) == 0) {  // two copies, each announced by its own lane (of no bytes, where there are no rows)
          mbar_expect_tx(bar + 8 * st, (uint32_t)rows * kQ4Row);
          if (rows) bulk_load(dst + (uint32_t)lane * kQ4Row, a.pages + (int64_t)place * kQ4Row, (uint32_t)rows * kQ4Row,
                              bar + 8 * st, policy);
        }
      }
    };

    uint4 query[4];
    fetch_query<PAIR>(query, a.q + ((int64_t)b * a.Hq + (int64_t)h * G) * kHeadDim, G, gid, tig);
    if (GATHER) load_page(0);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (s < n_iter) issue(s, (st + s) % kStages, masks[s]);
      if constexpr (GATHER) cp_async_commit();
    }
    Query<PAIR> qx;
    build_query<PAIR, F16>(qx, query, a.scale_log2, gid, tig);
    State w;
    w.m0 = w.m1 = -INFINITY;
    w.l0 = w.l1 = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      w.z[g][0] = w.z[g][1] = 0.f;
      w.c[g][0] = w.c[g][1] = biased_pow2(kMaxC);
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[g][0][i] = w.o[g][1][i] = 0.f;
    }
    float* lrow = a.logits + (bh * a.max_T + i_begin + (int)half + tok_a) * G + col;
    const int64_t eight = 8 * G;  // logits of 8 tokens
    float base0 = 0.f, base1 = 0.f;  // finite_max of the maxima

    int st_in = (st + kStages - 1) % kStages;
    int it = 0;
    for (; it < n_iter; ++it) {
      if (it + kStages - 1 < n_iter) issue(it + kStages - 1, st_in, masks[kStages - 1]);
      if (++st_in == kStages) st_in = 0;
      if constexpr (GATHER) {
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        __syncwarp();
      } else {
        alive = __all_sync(0xffffffffu, mbar_wait(bar + 8 * st, (uint32_t)phase, a.status));
        if (!alive) break;
      }
      const uint32_t rows = ring + (uint32_t)st * kStageBytes;
      const uint32_t mask = masks[0];
      const bool full = mask == 0xffffffffu;
      if (!GATHER && !full) {
        // Rows that are not there become zeros (the reuse's copies have seen to that): whatever stands there
        // would meet weights of 0 and columns of zeros, and 0 times a stray NaN is not 0.
        for (int i = lane; i < (int)kStageBytes / 16; i += 32)
          if (!((mask >> (i / 10)) & 1u)) sts128(rows + 16 * i, make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();  // copies come to the same place later
        __syncwarp();
      }
      constexpr int kSets = PAIR ? 1 : 2;  // sets of 16 rows that a lane works on
      const uint32_t mine = rows + half * kQ4Row + row_a;
      float s[kSets][4];
      scores<PAIR>(qx, rows, row_a, mine, tig, s[0]);
      if constexpr (!PAIR) scores<PAIR>(qx, rows + 16 * kQ4Row, row_a, mine + 16 * kQ4Row, tig, s[1]);
#pragma unroll
      for (int u = 0; u < kSets; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] = s[u][i] * 0x1p20f * ((i & 1) ? qx.f1 : qx.f0);
      if (!full) {
#pragma unroll
        for (int u = 0; u < 2 * kSets; ++u)
          if (!((mask >> (8 * u + half + tok_a)) & 1u)) s[u >> 1][2 * (u & 1)] = s[u >> 1][2 * (u & 1) + 1] = -INFINITY;
      }
      if constexpr (!GATHER) {
        if (full && !(G & 1)) {
          if (col < G) {
#pragma unroll
            for (int u = 0; u < 2 * kSets; ++u) {
              const float* x = &s[u >> 1][2 * (u & 1)];
              *reinterpret_cast<float2*>(lrow + u * eight) = make_float2(x[0], x[1]);
            }
          }
        } else {
          const int rest = i_end - (i_begin + kStageRows * it + (int)half + tok_a);
#pragma unroll
          for (int u = 0; u < 2 * kSets; ++u) {
            if (rest > 8 * u) {
              if (col < G) lrow[u * eight] = s[u >> 1][2 * (u & 1)];
              if (col + 1 < G) lrow[u * eight + 1] = s[u >> 1][2 * (u & 1) + 1];
            }
          }
        }
        lrow += 4 * eight;
      }
      float x0 = fmaxf(s[0][0], s[0][2]), x1 = fmaxf(s[0][1], s[0][3]);
      if constexpr (!PAIR) {
        x0 = fmaxf(x0, fmaxf(s[1][0], s[1][2]));
        x1 = fmaxf(x1, fmaxf(s[1][1], s[1][3]));
      }
      if (__any_sync(0xffffffffu, x0 > w.m0 + 8.f || x1 > w.m1 + 8.f)) {
        const float n0 = fmaxf(w.m0, head_max<PAIR>(x0)), n1 = fmaxf(w.m1, head_max<PAIR>(x1));
        base0 = finite_max(n0);
        base1 = finite_max(n1);
        const float al0 = fast_exp2(w.m0 - base0), al1 = fast_exp2(w.m1 - base1);
        w.m0 = n0;
        w.m1 = n1;
        w.l0 *= al0;
        w.l1 *= al1;
        rebase(w, 0, al0);
        rebase(w, 1, al1);
      }
#pragma unroll
      for (int u = 0; u < kSets; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] = fast_exp2(s[u][i] - ((i & 1) ? base1 : base0));
        w.l0 += s[u][0] + s[u][2];
        w.l1 += s[u][1] + s[u][3];
      }
      Weights wt;
      weights<PAIR>(w, mine + kQ4Tail + 16, s, tig, wt);
      values<PAIR>(w, rows, gid, tig, wt);
      __syncwarp();  // the stage is read: it may be refilled
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) masks[i] = masks[i + 1];
      if (++st == kStages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (!alive) {  // gave up on a copy: wait, with the same bound, for the others in flight
      for (int k = 1; k < kStages && it + k < n_iter; ++k) {
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
        mbar_wait(bar + 8 * st, (uint32_t)phase, a.status);
      }
    }

    if (bad) flag_status(a.status, kStatusBadIndex);
    bad = false;

    // ---- merge the four warps; the rings are free once all are here ------------
    const float l0 = head_sum<PAIR>(w.l0), l1 = head_sum<PAIR>(w.l1);
    if constexpr (GATHER) __syncthreads();
    else alive = __syncthreads_and(alive);
    float (*sm_o)[8][kHeadDim] = reinterpret_cast<float (*)[8][kHeadDim]>(smem);
    const bool owner = !PAIR || tig < 2;
    if constexpr (PAIR) {  // columns 4..7 hold the weights' second terms
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float& o = w.o[i >> 3][(i >> 2) & 1][i & 3];
        o += __shfl_xor_sync(0xffffffffu, o, 2);
      }
    }
    if (gid == 0 && owner) {
      sm_m[warp][col] = w.m0;
      sm_m[warp][col + 1] = w.m1;
      sm_l[warp][col] = l0;
      sm_l[warp][col + 1] = l1;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float up0 = 0x1p10f / w.c[g][0], up1 = 0x1p10f / w.c[g][1];  // sums are in 2^-22 c
      const float z0 = head_sum<PAIR>(w.z[g][0]), z1 = head_sum<PAIR>(w.z[g][1]);
      if (!owner) continue;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int d = 32 * g + 4 * gid + 2 * u;
        const float* o = w.o[g][u];
        *reinterpret_cast<float2*>(&sm_o[warp][col][d]) =
            make_float2(fmaf((o[0] - o[2]) * 0x1p12f, up0, z0), fmaf(o[2] * 0x1p8f, up0, z0));
        *reinterpret_cast<float2*>(&sm_o[warp][col + 1][d]) =
            make_float2(fmaf((o[1] - o[3]) * 0x1p12f, up1, z1), fmaf(o[3] * 0x1p8f, up1, z1));
      }
    }
    __syncthreads();
    const int d = threadIdx.x;  // kThreads == kHeadDim
    for (int g = 0; g < G; ++g) {
      float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm_m[i][g]);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float f = fast_exp2(sm_m[i][g] - finite_max(M));
        acc += f * sm_o[i][g][d];
        L += f * sm_l[i][g];
      }
      if constexpr (GATHER) {
        sm_po[g][d] = acc;
        if (d == 0) {
          sm_pm[g] = M;
          sm_pl[g] = L;
        }
      } else {
        const int64_t slot = ((int64_t)blockIdx.x + bh) * G + g;
        a.part_o[slot * kHeadDim + d] = acc;
        if (d == 0) {
          a.part_ml[slot * 2] = M;
          a.part_ml[slot * 2 + 1] = alive ? L : CUDART_NAN_F;
        }
      }
    }
    if constexpr (GATHER) {
      // the splits of (b, h) are one cluster: they merge through distributed shared memory
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      const int ns = (int)cluster.num_blocks();
      for (int g = (int)cluster.block_rank(); g < G; g += ns) {  // the blocks share the heads
        float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll 4
        for (int r = 0; r < ns; ++r) M = fmaxf(M, *cluster.map_shared_rank(&sm_pm[g], r));
#pragma unroll 4
        for (int r = 0; r < ns; ++r) {
          const float f = fast_exp2(*cluster.map_shared_rank(&sm_pm[g], r) - finite_max(M));
          L += f * *cluster.map_shared_rank(&sm_pl[g], r);
          acc += f * *cluster.map_shared_rank(&sm_po[g][d], r);
        }
        a.out[((int64_t)b * a.Hq + h * G + g) * kHeadDim + d] = to_bits<F16>(L == 0.f ? 0.f : acc / L);
        if (a.lse && d == 0) a.lse[(int64_t)b * a.Hq + h * G + g] = lse2_of(M, L) * kLn2;
      }
      cluster.sync();  // peers keep their shared memory until all have read it
      return;
    }
    // the next unit
    fence_proxy_async_smem();  // the merge wrote where the next copies go
    __syncthreads();
    if (left <= 0) return;
    at = 0;
    if (++h == a.Hkv) {
      h = 0;
      do {
        if (++b == a.B) return;
        T = a.seq_len[b];
      } while (stages_of(T, a.max_T) == 0);
    }
  }
}

struct CombineArgs {
  const int32_t* seq_len;
  int Hq, Hkv, G, max_T, blocks, chunk;  // blocks: grid of the first kernel
  const int2* parts;
  const float* part_ml;
  const float* part_o;
  const float* logits;
  float* pooled;
  int64_t ld_pooled;
  uint16_t* out;
  float* lse;
};

constexpr int kCombineThreads = 256;
constexpr int kPoolBatch = 1024;  // tokens of a block in flight; a block has some batches (chunk tokens)

// Second kernel of the anchor.  Blocks x < G merge the outputs of one head over the splits, eight
// splits at a time; the others turn a chunk of logits into pooled probabilities.  Each works out the
// maxima and sums that it needs from the splits'; a chunk's logits are loaded before that.  V: float4
// per token of the logits (G = 4 V), 0 for other G.
template <bool F16, int V>
__global__ void __launch_bounds__(kCombineThreads) decode_q4_combine_kernel(const CombineArgs a) {
  overlap_launches();
  __shared__ float s_L[8];
  __shared__ __align__(16) float s_M[8], s_inv[8];
  __shared__ float4 s_o[kCombineThreads / 32][kHeadDim / 4];
  const int b = blockIdx.z, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G;
  const int64_t bh = (int64_t)b * a.Hkv + h;
  int T = a.seq_len[b];
  const int2 part = a.parts[bh];  // of no meaning for an empty sequence
  if (T < 0 || T > a.max_T) T = 0;
  const bool merge = blockIdx.x < G;
  const int64_t t_lo = merge ? 0 : (int64_t)((int)blockIdx.x - G) * a.chunk;
  if (!merge && t_lo >= T) return;
  const int t_hi = (int)min(t_lo + a.chunk, (int64_t)T);
  const float* lrow = a.logits + bh * a.max_T * G;
  constexpr int kPer = kPoolBatch / kCombineThreads / (V > 1 ? V : 1);  // tokens per thread and batch
  constexpr int kBatch = kPer * kCombineThreads;
  float4 x[V > 0 ? kPer : 1][V > 0 ? V : 1];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + i * kCombineThreads + threadIdx.x;
#pragma unroll
      for (int j = 0; j < V; ++j)
        x[i][j] = t < t_hi ? reinterpret_cast<const float4*>(lrow)[(int64_t)t * V + j]
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  if (V > 0 && !merge) load((int)t_lo);
  // the slots of this unit: those of the blocks that hold its first stage to its last
  int c0 = 0, ns = 0;
  if (T > 0) {
    // the first kernel has written both for every unit with tokens; the bounds are for lengths that
    // someone changes between the two kernels
    if (part.x >= 0 && part.x <= part.y && part.y < a.blocks) {
      c0 = part.x;
      ns = part.y - part.x + 1;
    }
  }
  const float* ml = a.part_ml + (c0 + bh) * G * 2;
  if (merge ? warp == 0 : warp < G) {
    const int g = merge ? (int)blockIdx.x : warp;
    float M = -INFINITY, L = 0.f;
    for (int s = lane; s < ns; s += 32) M = fmaxf(M, ml[(s * G + g) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int s = lane; s < ns; s += 32) L += fast_exp2(ml[(s * G + g) * 2] - finite_max(M)) * ml[(s * G + g) * 2 + 1];
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) {
      s_M[g] = finite_max(M);
      s_L[g] = L;
      // probabilities are exp2(s - M) / L: a log-sum-exp is off by half its last bit, which all would share
      s_inv[g] = L == 0.f ? 0.f : 1.f / (L * (float)G);  // no score at all: probabilities 0
    }
  }
  __syncthreads();
  if (merge) {
    const int g = (int)blockIdx.x;
    const float4* po = reinterpret_cast<const float4*>(a.part_o + (c0 + bh) * G * kHeadDim) + g * 32 + lane;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = warp; s < ns; s += kCombineThreads / 32) {
      const float f = fast_exp2(ml[(s * G + g) * 2] - s_M[g]);
      const float4 v = po[(int64_t)s * G * 32];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    s_o[warp][lane] = acc;
    __syncthreads();
    if (threadIdx.x < kHeadDim) {
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < kCombineThreads / 32; ++i) o += reinterpret_cast<const float*>(s_o[i])[threadIdx.x];
      a.out[((int64_t)b * a.Hq + h * G + g) * kHeadDim + threadIdx.x] = to_bits<F16>(s_L[g] == 0.f ? 0.f : o / s_L[g]);
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[(int64_t)b * a.Hq + h * G + g] = lse2_of(s_L[g] == 0.f ? -INFINITY : s_M[g], s_L[g]) * kLn2;
    return;
  }
  float* prow = a.pooled + bh * a.ld_pooled;
  if constexpr (V > 0) {
    float4 m[V], f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      m[j] = *reinterpret_cast<const float4*>(&s_M[4 * j]);
      f[j] = *reinterpret_cast<const float4*>(&s_inv[4 * j]);
    }
    for (int t0 = (int)t_lo; t0 < t_hi; t0 += kBatch) {
      float p[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        p[i] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
          p[i] += (fast_exp2(x[i][j].x - m[j].x) * f[j].x + fast_exp2(x[i][j].y - m[j].y) * f[j].y) +
                  (fast_exp2(x[i][j].z - m[j].z) * f[j].z + fast_exp2(x[i][j].w - m[j].w) * f[j].w);
      }
      load(t0 + kBatch);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = t0 + i * kCombineThreads + threadIdx.x;
        if (t < t_hi) prow[t] = p[i];
      }
    }
  } else {
    for (int t = (int)t_lo + threadIdx.x; t < t_hi; t += kCombineThreads) {
      float acc = 0.f;
      for (int g = 0; g < G; ++g) acc += fast_exp2(lrow[(int64_t)t * G + g] - s_M[g]) * s_inv[g];
      prow[t] = acc;
    }
  }
}

// Blocks of the anchor's first kernel: one wave, or fewer where the warps would have no stage.
int anchor_blocks(int64_t units, int max_T) {
  const int64_t stages = units * ((max_T + kStageRows - 1) / kStageRows + kUnitCost);
  return (int)std::max<int64_t>(1, std::min<int64_t>(kSlots, (stages + kWarps - 1) / kWarps));
}

// Blocks (one cluster) per reuse row: one wave, at least a stage per warp.
int reuse_split(int64_t units, int k_max) {
  const int64_t n = std::min<int64_t>(std::min<int64_t>(16, std::max<int64_t>(1, kSlots / units)),
                                      ((int64_t)k_max + kWarps * kStageRows - 1) / (kWarps * kStageRows));
  return (int)std::max<int64_t>(1, n);
}

struct WsLayout {
  size_t logits, parts, part_ml, part_o, total;
};
WsLayout ws_layout(int B, int Hkv, int G, int max_T) {
  WsLayout w;
  const size_t slots = (size_t)B * Hkv + anchor_blocks((int64_t)B * Hkv, max_T);
  size_t off = 0;
  w.logits = off;
  off = align_up(off + (size_t)B * Hkv * max_T * G * sizeof(float), 256);
  w.parts = off;
  off = align_up(off + (size_t)B * Hkv * sizeof(int2), 256);
  w.part_ml = off;
  off = align_up(off + slots * G * 2 * sizeof(float), 256);
  w.part_o = off;
  w.total = align_up(off + slots * G * kHeadDim * sizeof(float), 256);
  return w;
}

Q4Args common_args(const DecodeQ4Params& p) {
  Q4Args a = {};
  a.q = p.q; a.pages = p.kv_pages; a.block_table = p.block_table;
  a.max_pages = p.max_pages; a.page_size = p.page_size; a.num_pages = p.num_pages;
  // with 2^(s+1) >= page_size > 2^s and mul = floor(2^(32+s) / page_size) + 1 the product is too
  // large by at most t 2^(s+1) < 2^(32+s): never enough to reach the next quotient
  while (((int64_t)2 << a.page_shift) < p.page_size) ++a.page_shift;
  a.page_mul = (uint32_t)(((uint64_t)1 << (32 + a.page_shift)) / (uint64_t)p.page_size + 1);
  a.seq_len = p.seq_len; a.idx = p.idx; a.idx_k = p.idx_k; a.head_map = p.head_map; a.k_max = p.k_max;
  a.B = p.B; a.Hq = p.Hq; a.Hkv = p.Hkv; a.G = p.G; a.max_T = p.max_T;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.out = p.out; a.lse = p.lse; a.status = p.status;
  a.give_up = p.give_up;
  return a;
}

auto pick_combine(int G, bool f16) {
  if (G == 4) return f16 ? decode_q4_combine_kernel<true, 1> : decode_q4_combine_kernel<false, 1>;
  if (G == 8) return f16 ? decode_q4_combine_kernel<true, 2> : decode_q4_combine_kernel<false, 2>;
  return f16 ? decode_q4_combine_kernel<true, 0> : decode_q4_combine_kernel<false, 0>;
}

template <bool GATHER>
auto pick_kernel(bool pair, bool f16) {
  return pair ? (f16 ? decode_q4_kernel<GATHER, true, true> : decode_q4_kernel<GATHER, true, false>)
              : (f16 ? decode_q4_kernel<GATHER, false, true> : decode_q4_kernel<GATHER, false, false>);
}

}  // namespace

size_t decode_q4_workspace_bytes(int B, int Hkv, int G, int max_T) {
  return ws_layout(B, Hkv, G, max_T).total;
}

cudaError_t launch_decode_anchor_q4(const DecodeQ4Params& p, cudaStream_t st) {
  const int blocks = anchor_blocks((int64_t)p.B * p.Hkv, p.max_T);
  const WsLayout w = ws_layout(p.B, p.Hkv, p.G, p.max_T);
  char* ws = static_cast<char*>(p.ws);
  Q4Args a = common_args(p);
  a.logits = reinterpret_cast<float*>(ws + w.logits);
  a.parts = reinterpret_cast<int2*>(ws + w.parts);
  a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  auto kern = pick_kernel<false>(p.G <= 4, p.f16);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(kern, blocks, kThreads, kSmemBytes, st, a);
  if (e != cudaSuccess) return e;
  CombineArgs c;
  c.seq_len = p.seq_len;
  c.Hq = p.Hq; c.Hkv = p.Hkv; c.G = p.G; c.max_T = p.max_T; c.blocks = blocks;
  c.parts = a.parts;
  c.part_ml = a.part_ml; c.part_o = a.part_o; c.logits = a.logits;
  c.pooled = p.pooled; c.ld_pooled = p.ld_pooled; c.out = p.out; c.lse = p.lse;
  // As many batches per block as leave about eight blocks per SM.
  const int batch = p.G == 8 ? kPoolBatch / 2 : kPoolBatch;
  const int64_t batches = ((int64_t)p.max_T + batch - 1) / batch * p.B * p.Hkv;
  c.chunk = batch * (int)std::min<int64_t>(16, std::max<int64_t>(1, batches / (8 * 148)));
  const dim3 cgrid(p.G + (p.max_T + c.chunk - 1) / c.chunk, p.Hkv, p.B);
  return launch_overlapped(pick_combine(p.G, p.f16), cgrid, kCombineThreads, 0, st, c);
}

cudaError_t launch_decode_reuse_q4(const DecodeQ4Params& p, cudaStream_t st) {
  const int nsplit = reuse_split((int64_t)p.B * p.Hkv, p.k_max);
  Q4Args a = common_args(p);
  auto kern = pick_kernel<true>(p.G <= 4, p.f16);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  if (nsplit > 8) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nsplit, p.Hkv, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[1] = pdl_attribute();
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nsplit;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace kascade
