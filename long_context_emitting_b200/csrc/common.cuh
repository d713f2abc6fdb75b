// Device helpers shared by the Kascade kernels (sm_100a).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kascade {

constexpr int kHeadDim = 128;

// Bits of the sticky device status word (see kascade_get_device_status).
constexpr unsigned kStatusBadIndex = 1u;
constexpr unsigned kStatusNonFinite = 2u;
constexpr unsigned kStatusTimeout = 4u;  // a bounded wait gave up

// Programmatic dependent launch.  The decode reuse (gather) kernel is launched
// with the programmatic stream-serialization attribute, so its CTAs can be
// scheduled while the previous kernel of the stream (often the previous
// layer's gather) finishes.  grid_dependency_wait() blocks until that kernel
// has completed and its writes are visible (a no-op without the attribute);
// the kernel calls it before its first global-memory access, so the stream's
// order of effects is unchanged.  allow_dependents_launch() lets the next such
// kernel start launching once every CTA of this grid has called it or exited.
// (Giving the attribute to the 16-bit decode anchor's split and combine kernels
// and to Top-k as well made the 32-layer step 20% slower, so of those only the
// gather kernel takes it.  The kernels around the 4-bit cache do, through
// launch_overlapped(): 570 instead of 580 us for a captured step of 8 layers.)
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The launch attribute of programmatic dependent launch.
inline cudaLaunchAttribute pdl_attribute();

// Launch of a kernel that starts with overlap_launches(): its blocks may take their places while the
// stream's previous kernel drains, and the next such kernel's while this one does.
template <typename... K, typename... A>
cudaError_t launch_overlapped(void (*kern)(K...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
// First statement of such a kernel, in every thread: nothing is read or written before the previous
// kernel's effects are there, and so none completes before those in front of it.
__device__ __forceinline__ void overlap_launches() {
  allow_dependents_launch();
  grid_dependency_wait();
}

inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}

__device__ __forceinline__ void flag_status(unsigned* status, unsigned bit) {
  if (status) atomicOr(status, bit);
}

// 16-byte streaming load that bypasses L1 and asks L2 to fetch 256-byte lines.
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
  uint4 r;
  asm("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "l"(p));
  return r;
}

__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 r;
  asm("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "l"(p));
  return r;
}

// 16 bytes by an ordinary load.  A kernel that is launched early (grid_dependency_wait) may be resident
// while kernels two or three places ahead of it still run: allow_dependents_launch() at a kernel's start
// lets in its successor, and that one the next.  What those write changes during this kernel's lifetime,
// so it may not be read through the non-coherent path (ld.global.nc, __ldg), which wants it constant for
// all of that time; such a kernel keeps that path for what no kernel writes (weights).
__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }

__device__ __forceinline__ uint32_t word_of(const uint4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

// D(16x8 f32) += A(16x16 bf16, row) * B(16x8 bf16, col)
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held one row-pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 2^x on the SFU (ex2.approx; flushes subnormal results to zero).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint16_t to_bf16_bits(float x) {
  __nv_bfloat16 v = __float2bfloat16_rn(x);
  return *reinterpret_cast<uint16_t*>(&v);
}

// fp16 counterparts (the f16 entry points: same kernels, half-precision data)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint16_t to_f16_bits(float x) {
  __half v = __float2half_rn(x);
  return *reinterpret_cast<uint16_t*>(&v);
}
// element-type dispatch: F16 = half precision, else bfloat16
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16) mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
  else mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_x2(float lo, float hi) {
  if constexpr (F16) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ uint16_t to_bits(float x) {
  if constexpr (F16) return to_f16_bits(x);
  else return to_bf16_bits(x);
}

__device__ __forceinline__ float warp_max_xor_gid(float v) {
  // reduce over the 8 lanes that share (lane & 3): xor 4, 8, 16
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
  return v;
}

__device__ __forceinline__ float warp_sum_xor_gid(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  return v;
}

}  // namespace kascade
