// A layer's inputs from its projection's rows, for packed prompts and for single tokens:
//   c_t = bias + sum_i w[i] x[t - (width - 1) + i]   (within the sequence; before its first
//                                                    token: the stored rows, or zero)
//   v | k | q = c_t sigmoid(c_t),   Delta = softplus(raw + dt_bias),   a = exp(-Delta A).
// One pass: every channel is read once and written once, so memory bandwidth bounds both
// kernels; the exponential and the reciprocal of each output keep the special function
// unit 61 % busy. Sums are FP32; q, k and v are rounded once, to the
// layer's io type. 8192 tokens of 20480 BF16 channels: 137 us, 77 % of the measured copy
// bandwidth; one token of 256 such rows: 18 us, 74 %.
#include "layer_device.cuh"

namespace replay {

namespace {

constexpr int kThreadsIn = 128;

// Delta and a of one head from the raw step size; softplus(x) = max(x, 0) + log1p(e^-|x|)
// holds for every x.
__device__ __forceinline__ void step_size(float x, float A, float& dt, float& a) {
  dt = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
  if (x != x) dt = x;
  a = expf(-dt * A);
}

// Channels of one thread: four, so that a block's loads in flight need few registers.
constexpr int kChannels = 4;

template <typename IO, int W>
struct Filter {  // pairs of channels, for packed FMAs
  using Vc = Vec<IO, kChannels>;
  using Row = f32x2[kChannels / 2];
  Row w[W], b;
  __device__ __forceinline__ void load(const InputsParams& p, int c0) {
    const ulonglong2 bb = p.bias ? *reinterpret_cast<const ulonglong2*>(p.bias + c0) : make_ulonglong2(0, 0);
    b[0] = bb.x, b[1] = bb.y;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(p.w + (size_t)i * p.D + c0);
      w[i][0] = ww.x, w[i][1] = ww.y;
    }
  }
  __device__ __forceinline__ static void unpack(typename Vc::raw u, Row& r) {
    float f[kChannels];
    Vc::unpack(u, f);
    r[0] = pair(f[0], f[1]), r[1] = pair(f[2], f[3]);
  }
  // the output of `x` after the rows `hist`, which it then joins
  __device__ __forceinline__ typename Vc::raw step(Row* hist, typename Vc::raw xu) const {
    Row x;
    unpack(xu, x);
    float o[kChannels];
#pragma unroll
    for (int j = 0; j < kChannels / 2; ++j) {
      f32x2 acc = b[j];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) acc = fma2(w[i][j], hist[i][j], acc);
      unpair(silu2<IO>(fma2(w[W - 1][j], x[j], acc)), o[2 * j], o[2 * j + 1]);
#pragma unroll
      for (int i = 0; i + 1 < W - 1; ++i) hist[i][j] = hist[i + 1][j];
      hist[W - 2][j] = x[j];
    }
    return Vc::pack(o);
  }
};

// a vector of inputs into shared memory, on its way until its group is waited for
__device__ __forceinline__ void copy_async(uint2* dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async(uint4* dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

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

// Packed prompts. A block takes a tile of tokens and kThreadsIn vectors of channels (the last
// one of a tile: its step sizes); a thread walks its tokens with the filter's rows in
// registers, and the tokens ahead on their way into shared memory (in registers they cost
// warps: 143 against 134 us). The tile that holds a sequence's first token also takes the
// width - 2 tokens after it, wherever they lie, and writes the sequence's new state, so
// that the thread that writes a state element is the only one that reads it.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreadsIn, sizeof(IO) == 2 ? 6 : 4) prompt_inputs_kernel(const __grid_constant__ InputsParams p) {
  using Vc = Vec<IO, kChannels>;
  using Raw = typename Vc::raw;
  constexpr int V = kChannels, K = W - 1;
  constexpr int U = 4;  // tokens of a group; the groups of a ring are in flight together
  constexpr int kRing = 4;
  __shared__ Raw ring[kRing][U][kThreadsIn];  // each thread's own: no barriers
  pdl_enter();
  const Packed& pk = p.pk;
  // blocks of the same tokens are neighbours, so that the rows are read as a whole
  const int cols = p.col_blocks;
  const int tile = blockIdx.x / cols, col = blockIdx.x % cols;
  const int64_t t0 = (int64_t)tile * p.tile;
  const bool last = blockIdx.x >= gridDim.x - cols;
  const int64_t t1 = last ? pk.tokens : t0 + p.tile;
  const bool steps = col == cols - 1;
  const int c0 = (col * kThreadsIn + (int)threadIdx.x) * V;
  const bool on = !steps && c0 < p.D;

  Filter<IO, W> f;
  Dest d = {nullptr, 0};
  if (on) {
    f.load(p, c0);
    d = dest_of<IO>(p, c0);
  }
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + (size_t)c0 * sizeof(IO);
  const size_t xs = (size_t)p.ldx * sizeof(IO);
  auto x_at = [&](int64_t t) { return __ldg(reinterpret_cast<const Raw*>(x + (size_t)t * xs)); };

  // Bounds that fall mislead the search below, so that a sequence may be passed over: one block
  // looks for them, so that they are always reported.
  if (tile == 0 && steps) {
    bool falls = false;
    for (int i = threadIdx.x; i < pk.n_seqs; i += kThreadsIn) falls |= pk.cu[i] > pk.cu[i + 1];
    if (falls && pk.status) atomicOr(pk.status, kErrSeqs);
  }
  // the first sequence that starts in this tile or after it: 32 bounds at a time
  int lo = 0, hi = pk.n_seqs;
  while (lo < hi) {
    const int hop = (hi - lo + 31) / 32, at = lo + (int)(threadIdx.x & 31) * hop;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(pk.cu + (at < hi ? at : lo)) < t0));
    if (hop == 1) {
      lo += n;
      break;
    }
    if (n == 0) break;
    hi = lo + n * hop < hi ? lo + n * hop : hi;
    lo += (n - 1) * hop + 1;
  }
  for (int s = lo > 0 ? lo - 1 : 0; s < pk.n_seqs; ++s) {
    if (s >= lo && !(pk.cu[s] < t1 || last)) break;
    int64_t begin, end;
    const bool res = s >= lo && pk.resume && pk.resume[s];  // on its way with the bounds and the row
    if (!seq_bounds(pk, s, begin, end)) continue;
    const bool owner = s >= lo && begin >= t0;  // it starts in this tile, and so in no other's, whatever the order
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
    const uint8_t* xt = x + (size_t)ta * xs;
    uint8_t* yt = d.base + (size_t)ta * d.stride;
    const int count = (int)(tb - ta);
    int asked = 0;  // tokens whose copies were issued
    auto fetch = [&](int g) {  // the next U tokens into the ring's group g, as far as there are any
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (asked + u < count) copy_async(&ring[g][u][threadIdx.x], xt + u * xs);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asked += U;
      xt += U * xs;
    };
#pragma unroll
    for (int g = 0; g < kRing - 1; ++g) fetch(g);
    typename Filter<IO, W>::Row hist[K];
    if (owner) {
      Raw old[K];
      Raw* st = reinterpret_cast<Raw*>(static_cast<uint8_t*>(p.conv) + ((size_t)row * K * p.D + c0) * sizeof(IO));
      const size_t ss = (size_t)p.D / V;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        old[i] = res ? st[i * ss] : Vc::zero();
        f.unpack(old[i], hist[i]);
      }
      const int64_t n = end - begin;
#pragma unroll
      for (int i = 0; i < K; ++i) {  // the last K of the rows [old | x]
        Raw u = Vc::zero();
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
      for (int i = 0; i < K; ++i) f.unpack(x_at(ta - K + i), hist[i]);
    }
    int g = 0;
    for (int t = 0; t < count; t += U) {
      fetch(g == 0 ? kRing - 1 : g - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < count) *reinterpret_cast<Raw*>(yt + u * d.stride) = f.step(hist, ring[g][u][threadIdx.x]);
      yt += U * d.stride;
      g = g == kRing - 1 ? 0 : g + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

// One token of each row. A block takes a few rows and kThreadsIn vectors of channels (the
// last one of them: their step sizes), so that the filter is loaded once for
// several rows. Into a decode layer (ring not null), v, k, Delta and a go to the record
// that the row's next entry takes, (start + count) mod cap.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreadsIn) token_inputs_kernel(const __grid_constant__ InputsParams p) {
  using Vc = Vec<IO, kChannels>;
  using Raw = typename Vc::raw;
  constexpr int V = kChannels, K = W - 1;
  constexpr int R = 4;  // rows whose loads are in flight together
  pdl_enter();
  const Packed& pk = p.pk;
  const int cols = p.col_blocks, col = blockIdx.x % cols;
  const bool steps = col == cols - 1;
  const int c0 = (col * kThreadsIn + (int)threadIdx.x) * V;
  const bool on = !steps && c0 < p.D;
  const int r0 = (int)(blockIdx.x / cols) * p.tile;
  const int r1 = r0 + p.tile < pk.n_seqs ? r0 + p.tile : pk.n_seqs;
  const int hp = p.H * p.P, gn = p.G * p.N;
  // what the vector belongs to: v of a head, k of a group or q; and its place in a ring record
  const int kind = c0 < hp ? 0 : c0 < hp + gn ? 1 : 2;
  const int ck = c0 - (kind == 0 ? 0 : kind == 1 ? hp : hp + gn);
  uint8_t* out = static_cast<uint8_t*>(kind == 0 ? p.v : kind == 1 ? p.k : p.q);
  const size_t out_row = (size_t)(kind == 0 ? hp : gn) * sizeof(IO);
  const int unit = kind == 0 ? p.P : p.N, of = kind == 0 ? p.H : p.G, nth = ck / unit;
  uint8_t* ring = kind == 2 || !p.ring ? nullptr : kind == 0 ? p.ring : p.ring_k;
  const int rec = kind == 0 ? p.rec_bytes : p.rec_k_bytes;

  Filter<IO, W> f;
  if (on) f.load(p, c0);
  const size_t ss = (size_t)p.D / V;
  for (int rb = r0; rb < r1; rb += R) {
    int row[R], slot[R];
    Raw xu[R], old[R][K];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      row[u] = rb + u < r1 ? seq_row(pk, rb + u) : -1;
      slot[u] = 0;
      if (p.ring && row[u] >= 0) {
        const int32_t word = p.counts[row[u]];
        const int start = word >> 16, c = word & 0xFFFF;
        if (word < 0 || c > p.L || start >= p.cap) {
          if (pk.status && threadIdx.x == 0) atomicOr(pk.status, kErrPointer);
          row[u] = -1;
        }
        slot[u] = start + c < p.cap ? start + c : start + c - p.cap;
      }
      if (on && row[u] >= 0) {
        xu[u] = *reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p.x) + ((size_t)(rb + u) * p.ldx + c0) * sizeof(IO));
        const Raw* st = reinterpret_cast<const Raw*>(static_cast<uint8_t*>(p.conv) + ((size_t)row[u] * K * p.D + c0) * sizeof(IO));
#pragma unroll
        for (int i = 0; i < K; ++i) old[u][i] = st[i * ss];
      }
    }
    if (steps) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (row[u] < 0) continue;
        const int r = rb + u;
        for (int h = threadIdx.x; h < p.H; h += kThreadsIn) {
          const float raw = to_float(static_cast<const IO*>(p.raw)[(size_t)r * p.ldr + h]);
          float dt, a;
          step_size(raw + (p.dt_bias ? p.dt_bias[h] : 0.f), p.A[h], dt, a);
          if (p.dt) p.dt[(size_t)r * p.H + h] = dt;
          if (p.a) p.a[(size_t)r * p.H + h] = a;
          if (p.ring) {
            float* e = reinterpret_cast<float*>(p.ring + (((size_t)row[u] * p.H + h) * p.cap + slot[u]) * p.rec_bytes +
                                                p.P * sizeof(IO));
            e[0] = dt;
            e[1] = a;
          }
        }
      }
      continue;
    }
    if (!on) continue;
#pragma unroll
    for (int u = 0; u < R; ++u) {
      if (row[u] < 0) continue;
      typename Filter<IO, W>::Row hist[K];
      Raw* st = reinterpret_cast<Raw*>(static_cast<uint8_t*>(p.conv) + ((size_t)row[u] * K * p.D + c0) * sizeof(IO));
#pragma unroll
      for (int i = 0; i < K; ++i) {
        f.unpack(old[u][i], hist[i]);
        st[i * ss] = i + 1 < K ? old[u][i + 1 < K ? i + 1 : i] : xu[u];
      }
      const Raw o = f.step(hist, xu[u]);
      if (out) *reinterpret_cast<Raw*>(out + (size_t)(rb + u) * out_row + (size_t)ck * sizeof(IO)) = o;
      if (ring)
        *reinterpret_cast<Raw*>(ring + (((size_t)row[u] * of + nth) * p.cap + slot[u]) * rec +
                                (size_t)(ck - nth * unit) * sizeof(IO)) = o;
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
int channel_blocks(const InputsParams& p) { return (p.D / kChannels + kThreadsIn - 1) / kThreadsIn; }

}  // namespace

cudaError_t launch_prompt_inputs(const InputsParams& in, int io, int num_sms, cudaStream_t s) {
  InputsParams p = in;
  const int cb = channel_blocks(p);
  // A block starts with a search and the rows before its tile: long tiles, but enough blocks
  // to fill the SMs, and few sequences behind one another in a tile where they are short.
  p.tile = 64;
  while (p.tile > 8 && (p.pk.tokens / p.tile * cb < 8 * num_sms || p.pk.tokens < (int64_t)p.tile * p.pk.n_seqs / 2))
    p.tile /= 2;
  const int64_t tiles = p.pk.tokens > 0 ? (p.pk.tokens + p.tile - 1) / p.tile : 1;
  p.col_blocks = cb + 1;
  const dim3 grid((unsigned)(tiles * p.col_blocks));
  return io == 1 ? prompt_io<__nv_bfloat16>(p, grid, s) : prompt_io<float>(p, grid, s);
}

cudaError_t launch_token_inputs(const InputsParams& in, int io, int num_sms, cudaStream_t s) {
  InputsParams p = in;
  const int cb = channel_blocks(p);
  p.tile = 4;  // rows of a block: the filter is loaded once for them
  while (p.tile > 1 && (int64_t)p.pk.n_seqs * cb < (int64_t)4 * num_sms * p.tile) p.tile /= 2;
  p.col_blocks = cb + 1;
  const dim3 grid((unsigned)((int64_t)(p.pk.n_seqs + p.tile - 1) / p.tile * p.col_blocks));
  return io == 1 ? token_io<__nv_bfloat16>(p, grid, s) : token_io<float>(p, grid, s);
}

}  // namespace replay
