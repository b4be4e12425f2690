// Gated norm of a layer's outputs: u = (y + D v) z sigmoid(z), out = u w / sqrt(mean(u^2) +
// eps), the mean over each of `groups` equal parts of a row. One pass: u stays in registers
// between the sum and the scaling, so the kernel is bound by memory bandwidth. The sum of
// squares and the scaling are FP32; the result is rounded once, to the layer's io type.
#include "layer_device.cuh"

namespace replay {

namespace {

template <typename IO>
__device__ __forceinline__ float gate(float z) {
  if constexpr (sizeof(IO) == 2) return __fdividef(z, 1.f + __expf(-z));
  return z / (1.f + expf(-z));
}

// V consecutive values of y (FP32 or io) as floats
template <typename Y, int V>
__device__ __forceinline__ void load_y(const void* y, size_t i, float* f) {
  constexpr int n = Vec<Y>::n;
#pragma unroll
  for (int j = 0; j < V; j += n)
    Vec<Y>::unpack(*reinterpret_cast<const uint4*>(static_cast<const Y*>(y) + i + j), f + j);
}

// u of the V elements from column c of row r
template <typename IO, typename Y>
__device__ __forceinline__ void gated(const NormParams& p, int64_t r, int c, float* u) {
  constexpr int V = Vec<IO>::n;
  const size_t at = (size_t)r * p.H * p.P + c;
  float z[V];
  load_y<Y, V>(p.y, at, u);
  Vec<IO>::unpack(*reinterpret_cast<const uint4*>(static_cast<const IO*>(p.z) + (size_t)r * p.ldz + c), z);
  if (p.v) {
    float v[V];
    Vec<IO>::unpack(*reinterpret_cast<const uint4*>(static_cast<const IO*>(p.v) + at), v);
    const float skip = p.D[c / p.P];  // P is a multiple of 8: one head per vector
#pragma unroll
    for (int j = 0; j < V; ++j) u[j] = fmaf(skip, v[j], u[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) u[j] *= gate<IO>(z[j]);
}

template <typename IO>
__device__ __forceinline__ void scale_store(const NormParams& p, int64_t r, int c, const float* u, float inv) {
  constexpr int V = Vec<IO>::n;
  float o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = u[j] * inv * p.weight[c + j];
  *reinterpret_cast<uint4*>(static_cast<IO*>(p.out) + (size_t)r * p.H * p.P + c) = Vec<IO>::pack(o);
}

constexpr int kNormVecs = 4;  // vectors of u that a thread keeps

}  // namespace

// T threads take one part of one row; a block of `blockDim.x` threads takes several parts
// where T is less. Parts wider than T * kNormVecs vectors read their inputs a second time.
template <typename IO, typename Y, int T>
__global__ void __launch_bounds__(T > 256 ? T : 256) gated_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = Vec<IO>::n, NV = kNormVecs;
  constexpr int kPer = (T > 256 ? T : 256) / T;
  pdl_enter();
  __shared__ float part[T > 32 ? kPer * (T / 32) : 1];
  const int width = p.H * p.P / p.groups;
  const int tid = threadIdx.x % T, sub = threadIdx.x / T;
  const int64_t unit = (int64_t)blockIdx.x * kPer + sub;
  const bool on = unit < p.rows * p.groups;
  const int64_t r = on ? unit / p.groups : 0;
  const int c0 = on ? (int)(unit - r * p.groups) * width : 0;

  float u[NV][V];
  float sum = 0.f;
  if (on) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + tid) * V;
      if (c < width) {
        gated<IO, Y>(p, r, c0 + c, u[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(u[i][j], u[i][j], sum);
      }
    }
    for (int c = (NV * T + tid) * V; c < width; c += T * V) {
      float x[V];
      gated<IO, Y>(p, r, c0 + c, x);
#pragma unroll
      for (int j = 0; j < V; ++j) sum = fmaf(x[j], x[j], sum);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if constexpr (T > 32) {
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) sum += part[sub * (T / 32) + i];
  }
  if (!on) return;
  const float inv = 1.f / sqrtf(sum / (float)width + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + tid) * V;
    if (c < width) scale_store<IO>(p, r, c0 + c, u[i], inv);
  }
  for (int c = (NV * T + tid) * V; c < width; c += T * V) {
    float x[V];
    gated<IO, Y>(p, r, c0 + c, x);
    scale_store<IO>(p, r, c0 + c, x, inv);
  }
}

namespace {

template <typename IO, typename Y>
cudaError_t norm_io(const NormParams& p, cudaStream_t s) {
  const int vecs = p.H * p.P / p.groups / Vec<IO>::n;
  const int64_t units = p.rows * p.groups;
  if (vecs <= 32 * kNormVecs) return pdl_launch(gated_norm_kernel<IO, Y, 32>, dim3((unsigned)((units + 7) / 8)), 256, 0, s, p);
  if (vecs <= 128 * kNormVecs)
    return pdl_launch(gated_norm_kernel<IO, Y, 128>, dim3((unsigned)((units + 1) / 2)), 256, 0, s, p);
  return pdl_launch(gated_norm_kernel<IO, Y, 512>, dim3((unsigned)units), 512, 0, s, p);
}

}  // namespace

cudaError_t launch_gated_norm(const NormParams& p, int io, int y_io, int num_sms, cudaStream_t s) {
  if (io == 1) return y_io == 1 ? norm_io<__nv_bfloat16, __nv_bfloat16>(p, s) : norm_io<__nv_bfloat16, float>(p, s);
  return norm_io<float, float>(p, s);
}

}  // namespace replay
