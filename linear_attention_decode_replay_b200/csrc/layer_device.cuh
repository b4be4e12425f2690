// Device helpers of the operators around the decode step: 16-byte vectors of inputs as
// floats, the rows that packed sequences own, and programmatic dependent launch.
#pragma once

#include "layer_params.h"
#include "replay_device.cuh"

namespace replay {

constexpr int32_t kErrSeqs = 1 << 4;  // a bad or repeated row id, or sequence bounds out of order

// Blackwell's packed FP32: two products, sums or FMAs an instruction, each rounded to nearest
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(f32x2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A vector of inputs, 16 bytes: 4 floats or 8 BF16; or 4 BF16 in 8 bytes.
__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void bf16_unpack2(uint32_t w, float* f) {  // a BF16 is the upper half of its FP32
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xFFFF0000u);
}
template <typename IO, int N = 16 / sizeof(IO)>
struct Vec;
template <>
struct Vec<float, 4> {
  static constexpr int n = 4;
  using raw = uint4;
  __device__ __forceinline__ static void unpack(uint4 u, float* f) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ __forceinline__ static uint4 zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  static constexpr int n = 8;
  using raw = uint4;
  __device__ __forceinline__ static void unpack(uint4 u, float* f) {
    bf16_unpack2(u.x, f);
    bf16_unpack2(u.y, f + 2);
    bf16_unpack2(u.z, f + 4);
    bf16_unpack2(u.w, f + 6);
  }
  __device__ __forceinline__ static uint32_t pack2(float lo, float hi) { return bf16_pack2(lo, hi); }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  __device__ __forceinline__ static uint4 zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Vec<__nv_bfloat16, 4> {
  static constexpr int n = 4;
  using raw = uint2;
  __device__ __forceinline__ static void unpack(uint2 u, float* f) {
    bf16_unpack2(u.x, f);
    bf16_unpack2(u.y, f + 2);
  }
  __device__ __forceinline__ static uint2 pack(const float* f) {
    return make_uint2(bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3]));
  }
  __device__ __forceinline__ static uint2 zero() { return make_uint2(0u, 0u); }
};
// x sigmoid(x). For BF16 results the hardware's exponential and reciprocal: each is within a
// few units of 2^-23, and x log2(e), rounded before the exponential, adds |x| 2^-24 (so that
// the result is within 2^-19 for |x| < 16, and its own rounding is 2^-8); results under 2^-119
// may become 0. For FP32 results the accurate exponential and a division within 2 steps
// (results under 2^-119 may become 0).
template <typename IO>
__device__ __forceinline__ float silu(float x) {
  if constexpr (sizeof(IO) == 2) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return x * r;
  }
  return __fdividef(x, 1.f + expf(-x));
}
template <typename IO>
__device__ __forceinline__ f32x2 silu2(f32x2 x) {
  float a, b;
  if constexpr (sizeof(IO) == 2) {
    unpair(mul2(x, pair(-1.4426950408889634f, -1.4426950408889634f)), a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    unpair(add2(pair(a, b), pair(1.f, 1.f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return mul2(x, pair(a, b));
  }
  unpair(x, a, b);
  return pair(silu<IO>(a), silu<IO>(b));
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Let the next kernel on the stream be scheduled, and wait until the one before it has
// completed: nothing in global memory is touched before this returns.
__device__ __forceinline__ void pdl_enter() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Tokens [begin, end) of sequence s; false (recorded in the status word) where its bounds
// are out of order or outside the packed tokens.
__device__ __forceinline__ bool seq_bounds(const Packed& pk, int s, int64_t& begin, int64_t& end) {
  begin = pk.cu[s];
  end = pk.cu[s + 1];
  const bool ok = begin >= 0 && end >= begin && end <= pk.tokens;
  if (!ok && pk.status) atomicOr(pk.status, kErrSeqs);
  return ok;
}

// The state row of sequence s, by a whole warp; -1 for a padding entry (a negative id),
// and (recorded in the status word) for an id past the batch or one that an earlier
// sequence has: the first of equal ids is served.
__device__ __forceinline__ int seq_row(const Packed& pk, int s) {
  if (!pk.seqs) return s;  // the host checked n_seqs <= batch
  const int row = pk.seqs[s];
  if (row < 0) return -1;
  bool bad = row >= pk.batch;
  for (int e = threadIdx.x & 31; e < s; e += 32) bad |= pk.seqs[e] == row;
  bad = __any_sync(0xffffffffu, bad);
  if (bad && pk.status && (threadIdx.x & 31) == 0) atomicOr(pk.status, kErrSeqs);
  return bad ? -1 : row;
}

// Launches `kern` so that its blocks may be scheduled while the previous kernel on the
// stream drains (pdl_enter waits for it).
template <typename P>
cudaError_t pdl_launch(void (*kern)(const P), dim3 grid, int threads, int smem, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace replay
