// The scan of packed prompts, token by token:
//   S <- a_t S + Delta_t v_t k_t^T,   y_t = S q_t.
// A block holds a block of state rows of one head of one sequence in registers and walks
// the sequence's tokens; a thread holds kRows rows of kCols columns. All arithmetic is
// FP32, as packed pairs (three instructions for two elements a token). It serves every size
// and type. Handing k and q to the threads loads the shared-memory pipe about as much as the
// FMAs load theirs: four rows of 8 columns a thread read half of what two of 16 do. Four
// prompts of 2050 FP32 tokens in all, 64 heads of 64 x 128: 206 us (two rows: 223 us, that pipe
// 84 % busy; now 63 %, the FMA pipe 59 %). What is left there is few warps (11 % of an SM's)
// and blocks of unequal length; where there are few blocks, a token's chain.
#include "layer_device.cuh"
#include "tcgen05.cuh"

namespace replay {

namespace {

constexpr int kSerialThreads = 128;
constexpr int kRows = 4, kCols = 8;

// Tokens staged in shared memory together, and tokens whose sums over a row's lanes are taken
// together: short BF16 sequences want little staging and many blocks an SM (256 sequences of
// one token: 194 us; with two rows a thread 209 us, and 305 us with 16 and 8), FP32 prompts few
// barriers and sums (four of 2050 in all: 206 us with 16 and 8, 218 us with 16 and 4).
template <typename IO, int N>
constexpr int serial_tokens() {
  return sizeof(IO) == 2 || N == 16 ? 8 : 16;
}
template <typename IO>
constexpr int serial_batch() {
  return sizeof(IO) == 2 ? 4 : 8;
}
template <int N>
constexpr int serial_rows() {  // state rows of one block
  return kSerialThreads / (N / kCols) * kRows;
}

}  // namespace

template <typename IO, int N>
__global__ void __launch_bounds__(kSerialThreads, sizeof(IO) == 2 ? 4 : 1) scan_serial_kernel(const __grid_constant__ ScanParams p) {
  constexpr int TPR = N / kCols;  // lanes that share a row
  constexpr int RB = serial_rows<N>();
  constexpr int TC = serial_tokens<IO, N>(), kBatch = serial_batch<IO>(), V = Vec<IO>::n;
  // two stages: one is filled and its outputs drained while the other is computed
  __shared__ __align__(16) float sk[2][TC][N], sq[2][TC][N], sv[2][TC][RB], sy[2][TC][RB];
  __shared__ float2 sda[2][TC];  // Delta, a
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
  f32x2 S[kRows][kCols / 2];
  const bool res = p.pk.resume && p.pk.resume[s];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      ulonglong2 x = make_ulonglong2(0, 0);
      if (res && r0 + r < rows)
        x = *reinterpret_cast<const ulonglong2*>(Sg + (size_t)(r0 + r) * N + 4 * (lane + TPR * i));
      S[r][2 * i] = x.x, S[r][2 * i + 1] = x.y;
    }

  // the next stage's values on their way: vectors of k and q, of v, and one token's Delta, a
  constexpr int KV = (TC * N / V + kSerialThreads - 1) / kSerialThreads;
  constexpr int VV = (TC * RB / V + kSerialThreads - 1) / kSerialThreads;
  const IO* q = static_cast<const IO*>(p.q) + (size_t)g * N;
  const IO* k = static_cast<const IO*>(p.k) + (size_t)g * N;
  const IO* v = static_cast<const IO*>(p.v) + (size_t)h * p.P + p0;
  uint4 fk[KV], fq[KV], fv[VV];
  float2 fda;
  auto fetch = [&](int64_t t0) {  // past the sequence: zeros, and no decay
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      const int i = u * kSerialThreads + threadIdx.x, t = i / (N / V), c = i % (N / V) * V;
      const bool in = t < TC && t0 + t < end;
      fk[u] = in ? *reinterpret_cast<const uint4*>(k + (size_t)(t0 + t) * p.G * N + c) : Vec<IO>::zero();
      fq[u] = in ? *reinterpret_cast<const uint4*>(q + (size_t)(t0 + t) * p.G * N + c) : Vec<IO>::zero();
    }
#pragma unroll
    for (int u = 0; u < VV; ++u) {
      const int i = u * kSerialThreads + threadIdx.x, t = i / (RB / V), c = i % (RB / V) * V;
      const bool in = t < TC && t0 + t < end && c < rows;
      fv[u] = in ? *reinterpret_cast<const uint4*>(v + (size_t)(t0 + t) * p.H * p.P + c) : Vec<IO>::zero();
    }
    fda = make_float2(0.f, 1.f);
    if (threadIdx.x < TC && t0 + threadIdx.x < end) {
      const size_t at = (size_t)(t0 + threadIdx.x) * p.H + h;
      fda = make_float2(p.dt[at], p.a[at]);
    }
  };
  auto store_y = [&](int64_t t0, int b) {
    for (int i = threadIdx.x; i < TC * (RB / V); i += kSerialThreads) {
      const int t = i / (RB / V), c = i % (RB / V) * V;
      if (t0 + t < end && c < rows)
        *reinterpret_cast<uint4*>(static_cast<IO*>(p.y) + ((size_t)(t0 + t) * p.H + h) * p.P + p0 + c) =
            Vec<IO>::pack(&sy[b][t][c]);
    }
  };

  int b = 0;
  if (begin < end) fetch(begin);
  for (int64_t t0 = begin; t0 < end; t0 += TC, b ^= 1) {
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      const int i = u * kSerialThreads + threadIdx.x, t = i / (N / V), c = i % (N / V) * V;
      if (t < TC) {
        Vec<IO>::unpack(fk[u], &sk[b][t][c]);
        Vec<IO>::unpack(fq[u], &sq[b][t][c]);
      }
    }
#pragma unroll
    for (int u = 0; u < VV; ++u) {
      const int i = u * kSerialThreads + threadIdx.x, t = i / (RB / V), c = i % (RB / V) * V;
      if (t < TC) Vec<IO>::unpack(fv[u], &sv[b][t][c]);
    }
    if (threadIdx.x < TC) sda[b][threadIdx.x] = fda;
    __syncthreads();  // this stage is there; the last one's outputs are, and its inputs are read
    if (t0 + TC < end) fetch(t0 + TC);
    if (t0 > begin) store_y(t0 - TC, b ^ 1);
    if ((int)(threadIdx.x & ~31u) / TPR * kRows >= rows) continue;  // the warp holds no row of the head
#pragma unroll 1
    for (int tb = 0; tb < TC && t0 + tb < end; tb += kBatch) {
      float y[kBatch * kRows];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float2 da = sda[b][tb + u];
        const float4 vv = *reinterpret_cast<const float4*>(&sv[b][tb + u][r0]);
        const f32x2 a2 = pair(da.y, da.y);
        const f32x2 w2[kRows] = {pair(da.x * vv.x, da.x * vv.x), pair(da.x * vv.y, da.x * vv.y),
                                 pair(da.x * vv.z, da.x * vv.z), pair(da.x * vv.w, da.x * vv.w)};
        f32x2 y2[kRows] = {};
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(&sk[b][tb + u][4 * (lane + TPR * i)]);
          const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(&sq[b][tb + u][4 * (lane + TPR * i)]);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            f32x2* x = &S[r][2 * i];
            x[0] = fma2(w2[r], kk.x, mul2(a2, x[0]));
            x[1] = fma2(w2[r], kk.y, mul2(a2, x[1]));
            y2[r] = fma2(x[0], qq.x, y2[r]);
            y2[r] = fma2(x[1], qq.y, y2[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float lo, hi;
          unpair(y2[r], lo, hi);
          y[u * kRows + r] = lo + hi;
        }
      }
      // sums over the row's lanes, transposed: each lane ends with some tokens' rows
      int base;
      using Red = SegReduce<kBatch * kRows, TPR>;
      Red::run(y, threadIdx.x & 31, base);
#pragma unroll
      for (int e = 0; e < Red::kHeld; ++e)
        sy[b][tb + (base + e) / kRows][r0 + (base + e) % kRows] = y[e];
    }
  }
  __syncthreads();
  if (begin < end) store_y(begin + (end - begin - 1) / TC * TC, b ^ 1);
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      if (r0 + r < rows)
        *reinterpret_cast<ulonglong2*>(Sg + (size_t)(r0 + r) * N + 4 * (lane + TPR * i)) =
            make_ulonglong2(S[r][2 * i], S[r][2 * i + 1]);
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
