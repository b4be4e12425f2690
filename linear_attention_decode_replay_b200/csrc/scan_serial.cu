// The scan of packed prompts, token by token:
//   S <- a_t S + Delta_t v_t k_t^T,   y_t = S q_t.
// A block holds a block of state rows of one head of one sequence in registers and walks
// the sequence's tokens; a thread holds kRows rows of kCols columns. All arithmetic is
// FP32. It serves every size and type; 3 P N FMAs per token and head bound it.
#include "layer_device.cuh"

namespace replay {

namespace {

constexpr int kSerialThreads = 128;
constexpr int kSerialTokens = 16;  // tokens staged in shared memory together
constexpr int kRows = 2, kCols = 16;

template <int N>
constexpr int serial_rows() {  // state rows of one block
  return kSerialThreads / (N / kCols) * kRows;
}

}  // namespace

template <typename IO, int N>
__global__ void __launch_bounds__(kSerialThreads) scan_serial_kernel(const __grid_constant__ ScanParams p) {
  constexpr int TPR = N / kCols;  // lanes that share a row
  constexpr int RB = serial_rows<N>();
  constexpr int TC = kSerialTokens, V = Vec<IO>::n;
  __shared__ __align__(16) float sk[TC][N], sq[TC][N], sv[TC][RB];
  __shared__ float2 sda[TC];  // Delta, a
  __shared__ __align__(16) float sy[TC][RB];
  pdl_enter();
  const int row_blocks = (p.P + RB - 1) / RB;
  const int s = blockIdx.x / (p.H * row_blocks);
  const int h = blockIdx.x / row_blocks % p.H, g = h / (p.H / p.G);
  const int p0 = blockIdx.x % row_blocks * RB;
  const int rows = p.P - p0 < RB ? p.P - p0 : RB;
  int64_t begin, end;
  if (!seq_bounds(p.pk, s, begin, end)) return;
  const int row = seq_row(p.pk, s);
  if (row < 0) return;

  const int lane = threadIdx.x % TPR;  // columns 4 (lane + TPR i) + 0..3
  const int r0 = threadIdx.x / TPR * kRows;
  float* Sg = p.S + (((size_t)row * p.H + h) * p.P + p0) * N;
  float S[kRows][kCols];
  const bool res = p.pk.resume && p.pk.resume[s];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (res && r0 + r < rows) x = *reinterpret_cast<const float4*>(Sg + (size_t)(r0 + r) * N + 4 * (lane + TPR * i));
      S[r][4 * i] = x.x, S[r][4 * i + 1] = x.y, S[r][4 * i + 2] = x.z, S[r][4 * i + 3] = x.w;
    }

  const IO* q = static_cast<const IO*>(p.q);
  const IO* k = static_cast<const IO*>(p.k);
  const IO* v = static_cast<const IO*>(p.v);
  for (int64_t t0 = begin; t0 < end; t0 += TC) {
    const int n = end - t0 < TC ? (int)(end - t0) : TC;
    __syncthreads();  // the last tokens' reads are done
    for (int i = threadIdx.x; i < n * (N / V); i += kSerialThreads) {
      const int t = i / (N / V), c = i % (N / V) * V;
      const size_t at = ((size_t)(t0 + t) * p.G + g) * N + c;
      Vec<IO>::unpack(*reinterpret_cast<const uint4*>(k + at), &sk[t][c]);
      Vec<IO>::unpack(*reinterpret_cast<const uint4*>(q + at), &sq[t][c]);
    }
    const int vr = rows / V;
    for (int i = threadIdx.x; i < n * vr; i += kSerialThreads) {
      const int t = i / vr, c = i % vr * V;
      Vec<IO>::unpack(*reinterpret_cast<const uint4*>(v + ((size_t)(t0 + t) * p.H + h) * p.P + p0 + c), &sv[t][c]);
    }
    if (threadIdx.x < n) {
      const size_t at = (size_t)(t0 + threadIdx.x) * p.H + h;
      sda[threadIdx.x] = make_float2(p.dt[at], p.a[at]);
    }
    __syncthreads();
    if ((int)(threadIdx.x & ~31u) / TPR * kRows < rows) {  // the warp holds a row of the head
      for (int t = 0; t < n; ++t) {
        const float2 da = sda[t];
        float y[kRows], w[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          y[r] = 0.f;
          w[r] = da.x * sv[t][r0 + r];
        }
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const float4 kk = *reinterpret_cast<const float4*>(&sk[t][4 * (lane + TPR * i)]);
          const float4 qq = *reinterpret_cast<const float4*>(&sq[t][4 * (lane + TPR * i)]);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            float* x = &S[r][4 * i];
            x[0] = fmaf(w[r], kk.x, da.y * x[0]);
            x[1] = fmaf(w[r], kk.y, da.y * x[1]);
            x[2] = fmaf(w[r], kk.z, da.y * x[2]);
            x[3] = fmaf(w[r], kk.w, da.y * x[3]);
            y[r] = fmaf(x[0], qq.x, y[r]);
            y[r] = fmaf(x[1], qq.y, y[r]);
            y[r] = fmaf(x[2], qq.z, y[r]);
            y[r] = fmaf(x[3], qq.w, y[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
          for (int off = TPR / 2; off >= 1; off >>= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], off);
          if (lane == 0) sy[t][r0 + r] = y[r];
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * vr; i += kSerialThreads) {
      const int t = i / vr, c = i % vr * V;
      *reinterpret_cast<uint4*>(static_cast<IO*>(p.y) + ((size_t)(t0 + t) * p.H + h) * p.P + p0 + c) =
          Vec<IO>::pack(&sy[t][c]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      if (r0 + r < rows)
        *reinterpret_cast<float4*>(Sg + (size_t)(r0 + r) * N + 4 * (lane + TPR * i)) =
            make_float4(S[r][4 * i], S[r][4 * i + 1], S[r][4 * i + 2], S[r][4 * i + 3]);
  if (p.counts && h == 0 && p0 == 0 && threadIdx.x == 0) p.counts[row] = 0;
}

namespace {

template <typename IO, int N>
cudaError_t serial_n(const ScanParams& p, cudaStream_t s) {
  const int64_t blocks = (int64_t)p.pk.n_seqs * p.H * ((p.P + serial_rows<N>() - 1) / serial_rows<N>());
  return pdl_launch(scan_serial_kernel<IO, N>, dim3((unsigned)blocks), kSerialThreads, 0, s, p);
}
template <typename IO>
cudaError_t serial_io(const ScanParams& p, cudaStream_t s) {
  switch (p.N) {
    case 16: return serial_n<IO, 16>(p, s);
    case 32: return serial_n<IO, 32>(p, s);
    case 64: return serial_n<IO, 64>(p, s);
    case 128: return serial_n<IO, 128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_scan_serial(const ScanParams& p, int io, cudaStream_t s) {
  return io == 1 ? serial_io<__nv_bfloat16>(p, s) : serial_io<float>(p, s);
}

}  // namespace replay
