// A layer's inputs from its projection's rows, for packed prompts and for single tokens:
//   c_t = bias + sum_i w[i] x[t - (width - 1) + i]   (within the sequence; before its first
//                                                    token: the stored rows, or zero)
//   v | k | q = c_t sigmoid(c_t),   Delta = softplus(raw + dt_bias),   a = exp(-Delta A).
// One pass: every channel is read once and written once, so both kernels are bound by
// memory bandwidth. Sums are FP32; q, k and v are rounded once, to the layer's io type.
#include "layer_device.cuh"

namespace replay {

namespace {

constexpr int kThreadsIn = 128;

// x sigmoid(x). BF16 results take the fast exponential and division (relative error about
// 2^-21, against the result's own rounding of 2^-9); FP32 results the accurate ones.
template <typename IO>
__device__ __forceinline__ float silu(float x) {
  if constexpr (sizeof(IO) == 2) return __fdividef(x, 1.f + __expf(-x));
  return x / (1.f + expf(-x));
}

// Delta and a of one head from the raw step size; softplus(x) = max(x, 0) + log1p(e^-|x|)
// holds for every x.
__device__ __forceinline__ void step_size(float x, float A, float& dt, float& a) {
  dt = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
  if (x != x) dt = x;
  a = expf(-dt * A);
}

template <typename IO, int W>
struct Filter {
  static constexpr int V = Vec<IO>::n;
  float w[W][V], b[V];
  __device__ __forceinline__ void load(const InputsParams& p, int c0) {
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = p.bias ? p.bias[c0 + j] : 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) w[i][j] = p.w[(size_t)i * p.D + c0 + j];
  }
  // the output of `x` after the rows `hist`, which it then joins
  __device__ __forceinline__ uint4 step(float (*hist)[V], uint4 xu) const {
    float x[V], o[V];
    Vec<IO>::unpack(xu, x);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float acc = b[j];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) acc = fmaf(w[i][j], hist[i][j], acc);
      o[j] = silu<IO>(fmaf(w[W - 1][j], x[j], acc));
#pragma unroll
      for (int i = 0; i + 1 < W - 1; ++i) hist[i][j] = hist[i + 1][j];
      hist[W - 2][j] = x[j];
    }
    return Vec<IO>::pack(o);
  }
};

// Where the vector of channels [c0, c0 + V) goes: v, k or q (a vector never straddles two:
// P and N are multiples of 8).
struct Dest {
  uint8_t* base;
  size_t stride;  // bytes from token to token
};
template <typename IO>
__device__ __forceinline__ Dest dest_of(const InputsParams& p, int c0) {
  const int hp = p.H * p.P, gn = p.G * p.N;
  if (c0 < hp) return {static_cast<uint8_t*>(p.v) + (size_t)c0 * sizeof(IO), hp * sizeof(IO)};
  if (c0 < hp + gn) return {static_cast<uint8_t*>(p.k) + (size_t)(c0 - hp) * sizeof(IO), gn * sizeof(IO)};
  return {static_cast<uint8_t*>(p.q) + (size_t)(c0 - hp - gn) * sizeof(IO), gn * sizeof(IO)};
}

}  // namespace

// Packed prompts. A block takes a tile of tokens and kThreadsIn vectors of channels (the
// last row of blocks: the tile's step sizes); a thread walks its tokens with the filter's
// rows in registers. The tile that holds a sequence's first token also takes the
// width - 2 tokens after it, wherever they lie, and writes the sequence's new state, so
// that the thread that writes a state element is the only one that reads it.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreadsIn) prompt_inputs_kernel(const __grid_constant__ InputsParams p) {
  constexpr int V = Vec<IO>::n, K = W - 1;
  constexpr int U = 4;  // tokens whose loads are in flight together
  pdl_enter();
  const Packed& pk = p.pk;
  const int64_t t0 = (int64_t)blockIdx.x * p.tile;
  const bool last = blockIdx.x == gridDim.x - 1;
  const int64_t t1 = last ? pk.tokens : t0 + p.tile;
  const bool steps = blockIdx.y == gridDim.y - 1;
  const int c0 = ((int)blockIdx.y * kThreadsIn + (int)threadIdx.x) * V;
  const bool on = !steps && c0 < p.D;

  Filter<IO, W> f;
  Dest d = {nullptr, 0};
  if (on) {
    f.load(p, c0);
    d = dest_of<IO>(p, c0);
  }
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + (size_t)c0 * sizeof(IO);
  const size_t xs = (size_t)p.ldx * sizeof(IO);
  auto x_at = [&](int64_t t) { return __ldg(reinterpret_cast<const uint4*>(x + (size_t)t * xs)); };

  // the first sequence that starts in this tile or after it
  int lo = 0, hi = pk.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pk.cu[mid] < t0) lo = mid + 1;
    else hi = mid;
  }
  for (int s = lo > 0 ? lo - 1 : 0; s < pk.n_seqs; ++s) {
    const bool owner = s >= lo;
    if (owner && !(pk.cu[s] < t1 || last)) break;
    int64_t begin, end;
    if (!seq_bounds(pk, s, begin, end)) continue;
    const int64_t ta = owner ? begin : (t0 > begin + K ? t0 : begin + K);
    const int64_t to = !owner || t1 > begin + K ? t1 : begin + K;
    const int64_t tb = end < to ? end : to;
    if (!owner && ta >= tb) continue;
    const int row = seq_row(pk, s);
    if (row < 0) continue;
    if (steps) {
      const int64_t n = (tb - ta) * p.H;
      for (int64_t i = threadIdx.x; i < n; i += kThreadsIn) {
        const int64_t t = ta + i / p.H;
        const int h = (int)(i % p.H);
        const float raw = to_float(static_cast<const IO*>(p.raw)[(size_t)t * p.ldr + h]);
        step_size(raw + (p.dt_bias ? p.dt_bias[h] : 0.f), p.A[h], p.dt[(size_t)t * p.H + h], p.a[(size_t)t * p.H + h]);
      }
      continue;
    }
    if (!on) continue;
    float hist[K][V];
    if (owner) {
      uint4 old[K];
      uint4* st = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.conv) + ((size_t)row * K * p.D + c0) * sizeof(IO));
      const size_t ss = (size_t)p.D * sizeof(IO) / 16;
      const bool res = pk.resume && pk.resume[s];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        old[i] = res ? st[i * ss] : make_uint4(0u, 0u, 0u, 0u);
        Vec<IO>::unpack(old[i], hist[i]);
      }
      const int64_t n = end - begin;
#pragma unroll
      for (int i = 0; i < K; ++i) {  // the last K of the rows [old | x]
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (n + i >= K) {
          u = x_at(begin + n + i - K);
        } else {
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (j == n + i) u = old[j];
        }
        st[i * ss] = u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) Vec<IO>::unpack(x_at(ta - K + i), hist[i]);
    }
    int64_t t = ta;
    for (; t + U <= tb; t += U) {
      uint4 xu[U];
#pragma unroll
      for (int u = 0; u < U; ++u) xu[u] = x_at(t + u);
#pragma unroll
      for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(d.base + (size_t)(t + u) * d.stride) = f.step(hist, xu[u]);
    }
    for (; t < tb; ++t) *reinterpret_cast<uint4*>(d.base + (size_t)t * d.stride) = f.step(hist, x_at(t));
  }
}

// One token of each row. A block takes a few rows and kThreadsIn vectors of channels (the
// last row of blocks: their step sizes), so that the filter is loaded once for
// several rows. Into a decode layer (ring not null), v, k, Delta and a go to the record
// that the row's next entry takes, (start + count) mod cap.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreadsIn) token_inputs_kernel(const __grid_constant__ InputsParams p) {
  constexpr int V = Vec<IO>::n, K = W - 1;
  pdl_enter();
  const Packed& pk = p.pk;
  const bool steps = blockIdx.y == gridDim.y - 1;
  const int c0 = ((int)blockIdx.y * kThreadsIn + (int)threadIdx.x) * V;
  const bool on = !steps && c0 < p.D;
  const int r0 = (int)blockIdx.x * p.tile;
  const int r1 = r0 + p.tile < pk.n_seqs ? r0 + p.tile : pk.n_seqs;
  const int hp = p.H * p.P, gn = p.G * p.N;

  Filter<IO, W> f;
  if (on) f.load(p, c0);
  for (int r = r0; r < r1; ++r) {
    const int row = seq_row(pk, r);
    if (row < 0) continue;
    int slot = 0;
    if (p.ring) {
      const int32_t word = p.counts[row];
      const int start = word >> 16, c = word & 0xFFFF;
      if (word < 0 || c > p.L || start >= p.cap) {
        if (pk.status && threadIdx.x == 0) atomicOr(pk.status, kErrPointer);
        continue;
      }
      slot = start + c < p.cap ? start + c : start + c - p.cap;
    }
    if (steps) {
      for (int h = threadIdx.x; h < p.H; h += kThreadsIn) {
        const float raw = to_float(static_cast<const IO*>(p.raw)[(size_t)r * p.ldr + h]);
        float dt, a;
        step_size(raw + (p.dt_bias ? p.dt_bias[h] : 0.f), p.A[h], dt, a);
        if (p.dt) p.dt[(size_t)r * p.H + h] = dt;
        if (p.a) p.a[(size_t)r * p.H + h] = a;
        if (p.ring) {
          float* e = reinterpret_cast<float*>(p.ring + (((size_t)row * p.H + h) * p.cap + slot) * p.rec_bytes +
                                              p.P * sizeof(IO));
          e[0] = dt;
          e[1] = a;
        }
      }
      continue;
    }
    if (!on) continue;
    const uint4 xu = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) +
                                                     ((size_t)r * p.ldx + c0) * sizeof(IO));
    uint4* st = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.conv) + ((size_t)row * K * p.D + c0) * sizeof(IO));
    const size_t ss = (size_t)p.D * sizeof(IO) / 16;
    float hist[K][V];
    uint4 old[K];
#pragma unroll
    for (int i = 0; i < K; ++i) old[i] = st[i * ss];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      Vec<IO>::unpack(old[i], hist[i]);
      st[i * ss] = i + 1 < K ? old[i + 1 < K ? i + 1 : i] : xu;
    }
    const uint4 o = f.step(hist, xu);
    const size_t at = (size_t)c0 * sizeof(IO);
    if (c0 < hp) {
      if (p.v) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v) + (size_t)r * hp * sizeof(IO) + at) = o;
      if (p.ring) {
        const int h = c0 / p.P;
        *reinterpret_cast<uint4*>(p.ring + (((size_t)row * p.H + h) * p.cap + slot) * p.rec_bytes +
                                  (size_t)(c0 - h * p.P) * sizeof(IO)) = o;
      }
    } else if (c0 < hp + gn) {
      const int ck = c0 - hp;
      if (p.k) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k) + ((size_t)r * gn + ck) * sizeof(IO)) = o;
      if (p.ring) {
        const int g = ck / p.N;
        *reinterpret_cast<uint4*>(p.ring_k + (((size_t)row * p.G + g) * p.cap + slot) * p.rec_k_bytes +
                                  (size_t)(ck - g * p.N) * sizeof(IO)) = o;
      }
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.q) + ((size_t)r * gn + c0 - hp - gn) * sizeof(IO)) = o;
    }
  }
}

namespace {

template <typename IO>
cudaError_t prompt_io(const InputsParams& p, dim3 grid, cudaStream_t s) {
  switch (p.width) {
    case 2: return pdl_launch(prompt_inputs_kernel<IO, 2>, grid, kThreadsIn, 0, s, p);
    case 3: return pdl_launch(prompt_inputs_kernel<IO, 3>, grid, kThreadsIn, 0, s, p);
    case 4: return pdl_launch(prompt_inputs_kernel<IO, 4>, grid, kThreadsIn, 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}
template <typename IO>
cudaError_t token_io(const InputsParams& p, dim3 grid, cudaStream_t s) {
  switch (p.width) {
    case 2: return pdl_launch(token_inputs_kernel<IO, 2>, grid, kThreadsIn, 0, s, p);
    case 3: return pdl_launch(token_inputs_kernel<IO, 3>, grid, kThreadsIn, 0, s, p);
    case 4: return pdl_launch(token_inputs_kernel<IO, 4>, grid, kThreadsIn, 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}
int channel_blocks(const InputsParams& p, int io) {
  const int v = io == 1 ? 8 : 4;
  return (p.D / v + kThreadsIn - 1) / kThreadsIn;
}

}  // namespace

cudaError_t launch_prompt_inputs(const InputsParams& in, int io, int num_sms, cudaStream_t s) {
  InputsParams p = in;
  const int cb = channel_blocks(p, io);
  p.tile = 32;
  const int64_t tiles = p.pk.tokens > 0 ? (p.pk.tokens + p.tile - 1) / p.tile : 1;
  const dim3 grid((unsigned)tiles, cb + 1);
  return io == 1 ? prompt_io<__nv_bfloat16>(p, grid, s) : prompt_io<float>(p, grid, s);
}

cudaError_t launch_token_inputs(const InputsParams& in, int io, int num_sms, cudaStream_t s) {
  InputsParams p = in;
  const int cb = channel_blocks(p, io);
  p.tile = 1;
  const dim3 grid((unsigned)((p.pk.n_seqs + p.tile - 1) / p.tile), cb + 1);
  return io == 1 ? token_io<__nv_bfloat16>(p, grid, s) : token_io<float>(p, grid, s);
}

}  // namespace replay
