// The scan of packed prompts on the tensor cores, for BF16 inputs. A chunk of Q = 128 tokens
// of one head is four products, with r_ij = prod_{j < l <= i} a_l:
//   C  = Q K^T                          y_i  = abar_i Y2_i + Y1_i,   abar_i = prod_{l <= i} a_l
//   Y1 = P V,  P_ij = C_ij r_ij Delta_j (j <= i)
//   Y2 = Q S^T                          S   <- abar_Q S + dS
//   dS = U^T K, U_j = (Delta_j prod_{l > j} a_l) v_j
// A block walks one head of one sequence (64 of its P rows). q, k and v come by TMA into
// 128-byte swizzled tiles; C, Y1, Y2 and dS are tensor-memory accumulators; S stays in
// registers, one state column n a thread. FP32 factors enter the products as sums of BF16
// parts: U in three (remainder 2^-24: the state keeps FP32 accuracy), S and P in two
// (remainder 2^-17, under the outputs' own rounding of 2^-9). dS is summed apart from S,
// since the accumulators do not round to nearest and S may hold thousands of tokens.
// Decays are products, never exponentials of differences: a = 0 and any sign are exact.
#include "layer_device.cuh"
#include "tcgen05.cuh"

namespace replay {

namespace {

constexpr int kChunk = 128;
constexpr int kPT = 64;  // state rows of one block
constexpr int kTcThreads = 320;
// warps 0-3 (rows of C: P and the outputs), 4-7 (U and the state), 8 (TMA), 9 (MMA)

struct alignas(64) ScanTcParams {
  CUtensorMap q, k, v;
  ScanParams s;
};

// tensor memory columns
constexpr uint32_t kColC = 0, kColPhi = 128, kColPlo = 192, kColY1 = 256, kColY2 = 320, kColDS = 384;

struct TcBars {
  uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t c_full, p_full, y_full, y_free, u_full, ds_full, s_full, tot_full, da_full[2], drain;
  uint32_t tmem, abort;
  float total[2][4];  // the four warps' products of a
  int bad[2];         // the chunk holds a v that is not finite
};

template <int NT>
struct TcLayout {  // bytes from the 1024-byte aligned base
  static constexpr int kTile = kChunk * 128;  // 128 rows of 64 BF16
  static constexpr int kQK = NT / 64 * kTile;
  static constexpr int kSop = NT * 128;  // one part of the state operand: NT rows of 64 BF16
  static constexpr int q = 0, k = kQK, v = k + 2 * kQK, u = v + 2 * kTile, s = u + 3 * kTile;
  static constexpr int da = s + 2 * kSop;                      // float2 [2][128]: a_{j+1}, Delta_j
  static constexpr int abar = da + 2 * kChunk * 8;             // float [2][128]
  static constexpr int bars = abar + 2 * kChunk * 4;
  static constexpr int bytes = bars + (int)sizeof(TcBars) + 1024;
};

// two floats' BF16 parts packed (a in the low half), and what remains of them
__device__ __forceinline__ uint32_t take_part(float& a, float& b) {
  const uint32_t w = Vec<__nv_bfloat16>::pack2(a, b);
  a -= __uint_as_float(w << 16);
  b -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(kTcThreads, 1) scan_tc_kernel(const __grid_constant__ ScanTcParams tp) {
  using Lay = TcLayout<NT>;
  constexpr int kTile = Lay::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  TcBars* bars = reinterpret_cast<TcBars*>(smem + Lay::bars);
  float2* da = reinterpret_cast<float2*>(smem + Lay::da);
  float* abar = reinterpret_cast<float*>(smem + Lay::abar);
  const ScanParams& p = tp.s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1), mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], 1), mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], 1), mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->da_full[i], 128);
      bars->bad[i] = 0;
    }
    mbar_init(&bars->c_full, 1), mbar_init(&bars->p_full, 128);
    mbar_init(&bars->y_full, 1), mbar_init(&bars->y_free, 128);
    mbar_init(&bars->u_full, 128), mbar_init(&bars->ds_full, 1), mbar_init(&bars->s_full, 128);
    mbar_init(&bars->tot_full, 128), mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the block's unit: sequence, head, block of 64 state rows
  const int ptiles = (p.P + kPT - 1) / kPT;
  const int unit = blockIdx.x;
  const int s = unit / (p.H * ptiles);
  const int h = unit / ptiles % p.H, g = h / (p.H / p.G);
  const int p0 = unit % ptiles * kPT;
  int64_t begin, end;
  if (!seq_bounds(p.pk, s, begin, end)) return;
  const int row = seq_row(p.pk, s);
  if (row < 0) return;
  const int chunks = (int)((end - begin + kChunk - 1) / kChunk);

  if (warp == 9) tmem_alloc(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t* abort = &bars->abort;

  // waits for a phase; false once any wait of the block has run out
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    const uint32_t parity = phase & 1;
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*abort) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        *abort = 1;
        if (p.pk.status) atomicOr(p.pk.status, kErrWaitTimeout);
        return false;
      }
    }
  };

  // the same for a whole warp: every lane goes on, or none
  auto wait_warp = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    if (lane == 0) {
      int c = 0, nq = 0, nk = 0, nv = 0;  // tiles issued
      for (; c < chunks; ++c) {
        const int b = c & 1;
        const int t = (int)(begin + (int64_t)c * kChunk);
        if (c >= 2 && !wait(&bars->k_empty[b], (c >> 1) - 1)) break;
        mbar_arrive_expect_tx(&bars->k_full[b], Lay::kQK);
        for (int i = 0; i < NT / 64; ++i)
          tma_load3(smem + Lay::k + b * Lay::kQK + i * kTile, &tp.k, 64 * i, g, t, &bars->k_full[b]);
        ++nk;
        if (c >= 1 && !wait(&bars->q_empty, c - 1)) break;
        mbar_arrive_expect_tx(&bars->q_full, Lay::kQK);
        for (int i = 0; i < NT / 64; ++i)
          tma_load3(smem + Lay::q + i * kTile, &tp.q, 64 * i, g, t, &bars->q_full);
        ++nq;
        if (c >= 2 && !wait(&bars->v_empty[b], (c >> 1) - 1)) break;
        mbar_arrive_expect_tx(&bars->v_full[b], kTile);
        tma_load3(smem + Lay::v + b * kTile, &tp.v, p0, h, t, &bars->v_full[b]);
        ++nv;
      }
      if (*abort) {  // no copy may land after the block has gone
        if (nq) mbar_wait_bounded(&bars->q_full, (nq - 1) & 1);
        for (int b = 0; b < 2; ++b) {
          if (nk > b) mbar_wait_bounded(&bars->k_full[b], ((nk - 1 - b) >> 1) & 1);
          if (nv > b) mbar_wait_bounded(&bars->v_full[b], ((nv - 1 - b) >> 1) & 1);
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      const uint32_t sq = smem_u32(smem + Lay::q), su = smem_u32(smem + Lay::u), ss = smem_u32(smem + Lay::s);
      constexpr uint32_t kC = mma_idesc(128, 128, 0, 0), kY1 = mma_idesc(128, kPT, 0, 1);
      constexpr uint32_t kDS2 = mma_idesc(128, 2 * kPT, 1, 1), kDS1 = mma_idesc(128, kPT, 1, 1);
      for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        const uint32_t sk = smem_u32(smem + Lay::k + b * Lay::kQK), sv = smem_u32(smem + Lay::v + b * kTile);
        // C = Q K^T, once the last chunk's C has been read
        if (!wait(&bars->q_full, c) || !wait(&bars->k_full[b], c >> 1)) break;
        tc_fence_after();
        for (int i = 0; i < NT / 16; ++i) {
          const uint32_t at = i / 4 * kTile + i % 4 * 32;
          mma_ss(tmem + kColC, smem_desc(sq + at, 16), smem_desc(sk + at, 16), kC, i > 0);
        }
        mma_commit(&bars->c_full);
        // Y2 = Q S^T, once the last chunk's outputs have been read
        if (!wait(&bars->s_full, c) || (c >= 1 && !wait(&bars->y_free, c - 1))) break;
        tc_fence_after();
        for (int part = 0; part < 2; ++part)
          for (int i = 0; i < NT / 16; ++i)
            mma_ss(tmem + kColY2, smem_desc(sq + i / 4 * kTile + i % 4 * 32, 16),
                   smem_desc(ss + part * Lay::kSop + i * 2048, 16), kY1, part + i > 0);
        mma_commit(&bars->q_empty);
        // dS = K^T U: the two larger parts side by side, the third onto the second
        if (!wait(&bars->u_full, c)) break;
        tc_fence_after();
        for (int i = 0; i < kChunk / 16; ++i)
          mma_ss(tmem + kColDS, smem_desc(sk + i * 2048, kTile), smem_desc(su + i * 2048, kTile), kDS2, i > 0);
        for (int i = 0; i < kChunk / 16; ++i)
          mma_ss(tmem + kColDS + kPT, smem_desc(sk + i * 2048, kTile), smem_desc(su + 2 * kTile + i * 2048, 16), kDS1,
                 true);
        mma_commit(&bars->ds_full);
        mma_commit(&bars->k_empty[b]);
        // Y1 = P V
        if (!wait(&bars->p_full, c) || !wait(&bars->v_full[b], c >> 1)) break;
        tc_fence_after();
        for (int part = 0; part < 2; ++part)
          for (int i = 0; i < kChunk / 16; ++i)
            mma_ts(tmem + kColY1, tmem + (part ? kColPlo : kColPhi) + i * 8, smem_desc(sv + i * 2048, 16), kY1,
                   part + i > 0);
        mma_commit(&bars->y_full);
        mma_commit(&bars->v_empty[b]);
      }
      if (*abort) {  // nothing may still run on the tensor memory when it is freed
        mma_commit(&bars->drain);
        mbar_wait_bounded(&bars->drain, 0);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ P and the outputs: row i of the chunk
    const int i = threadIdx.x;
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t zero[16] = {0};
    for (int cb = warp + 1; cb < 4; ++cb) {  // columns past the diagonal block stay zero
      tmem_st16(tl + kColPhi + 16 * cb, zero);
      tmem_st16(tl + kColPlo + 16 * cb, zero);
    }
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      const int64_t t = begin + (int64_t)c * kChunk + i;
      if (!wait_warp(&bars->da_full[b], c >> 1) || !wait_warp(&bars->c_full, c)) break;
      tc_fence_after();
      const float4* dab = reinterpret_cast<const float4*>(da + b * kChunk);
      float r = 0.f;
      for (int cb = warp; cb >= 0; --cb) {
        uint32_t x[32], hi[16], lo[16];
        tmem_ld32(tl + kColC + 32 * cb, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int jj = 30; jj >= 0; jj -= 2) {
          const float4 d = dab[(32 * cb + jj) / 2];  // a_{j+1}, Delta_j, a_{j+2}, Delta_{j+1}
          float p1, p0v;
          if (cb == warp) {  // the diagonal block: r starts at j = i
            r = jj + 1 == lane ? 1.f : r * d.z;
            p1 = jj + 1 <= lane ? __uint_as_float(x[jj + 1]) * (r * d.w) : 0.f;
            r = jj == lane ? 1.f : r * d.x;
            p0v = jj <= lane ? __uint_as_float(x[jj]) * (r * d.y) : 0.f;
          } else {
            r *= d.z;
            p1 = __uint_as_float(x[jj + 1]) * (r * d.w);
            r *= d.x;
            p0v = __uint_as_float(x[jj]) * (r * d.y);
          }
          hi[jj / 2] = take_part(p0v, p1);
          lo[jj / 2] = Vec<__nv_bfloat16>::pack2(p0v, p1);
        }
        tmem_st16(tl + kColPhi + 16 * cb, hi);
        tmem_st16(tl + kColPlo + 16 * cb, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->p_full);

      if (!wait_warp(&bars->y_full, c)) break;
      tc_fence_after();
      const float ab = abar[b * kChunk + i];
      const bool bad = bars->bad[b] != 0;
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + ((size_t)t * p.H + h) * p.P + p0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t y1[32], y2[32];
        tmem_ld32(tl + kColY1 + 32 * half, y1);
        tmem_ld32(tl + kColY2 + 32 * half, y2);
        tmem_wait_ld(y1);
        tmem_wait_ld(y2);
        if (half == 1) {
          tc_fence_before();
          mbar_arrive(&bars->y_free);
        }
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = fmaf(ab, __uint_as_float(y2[j]), __uint_as_float(y1[j]));
        if (t < end) {
          if (bad) {  // the products saw zeros in place of what is not finite in v: it reaches every later row
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + p0 + 32 * half;
            for (int j = 0; j <= i; ++j) {
              const __nv_bfloat16* vj = v + ((size_t)(t - i + j) * p.H + h) * p.P;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (p0 + 32 * half + e < p.P) o[e] = fmaf(__bfloat162float(vj[e]), 0.f, o[e]);
            }
          }
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            if (p0 + 32 * half + j < p.P)
              *reinterpret_cast<uint4*>(y + 32 * half + j) = Vec<__nv_bfloat16>::pack(o + j);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ U and the state: token j, then column n
    const int j = threadIdx.x - 128, w4 = warp - 4;
    const uint32_t tl = tmem + ((uint32_t)(w4 * 32) << 16);
    const int n = j;
    float S[kPT];
    float* Sg = p.S + ((size_t)row * p.H + h) * p.P * p.N + n;
    const bool res = p.pk.resume && p.pk.resume[s];
#pragma unroll
    for (int e = 0; e < kPT; ++e) S[e] = res && n < p.N && p0 + e < p.P ? Sg[(size_t)(p0 + e) * p.N] : 0.f;
    // the state's two BF16 parts as an operand: row n, chunk x at x ^ (n % 8)
    auto put_state = [&] {
      if (n < NT) {
        uint8_t* dst = smem + Lay::s + n * 128;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f0 = S[8 * x + 2 * e], f1 = S[8 * x + 2 * e + 1];
            hi[e] = take_part(f0, f1);
            lo[e] = Vec<__nv_bfloat16>::pack2(f0, f1);
          }
          uint8_t* at = dst + ((x ^ (n & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + Lay::kSop) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
      mbar_arrive(&bars->s_full);
    };
    float a = 1.f, dt = 0.f;
    auto load_da = [&](int c) {  // this thread's token of chunk c; past the sequence: no decay, no step
      const int64_t t = begin + (int64_t)c * kChunk + j;
      const bool in = c < chunks && t < end;
      a = in ? p.a[(size_t)t * p.H + h] : 1.f;
      dt = in ? p.dt[(size_t)t * p.H + h] : 0.f;
    };
    load_da(0);
    if (chunks > 0) put_state();
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      const int len = (int)(end - begin - (int64_t)c * kChunk < kChunk ? end - begin - (int64_t)c * kChunk : kChunk);
      // products of the decays up to and after this token
      float pre = a, suf = a;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, pre, off), d = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane >= off) pre *= u;
        if (lane + off < 32) suf *= d;
      }
      if (lane == 31) bars->total[b][w4] = pre;
      suf = __shfl_down_sync(0xffffffffu, suf, 1);
      if (lane == 31) suf = 1.f;
      if (j == 0) bars->bad[b] = 0;
      mbar_arrive(&bars->tot_full);
      if (!wait_warp(&bars->tot_full, c)) break;
      float all = 1.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float tx = bars->total[b][x];
        all *= tx;
        if (x < w4) pre *= tx;
        if (x > w4) suf *= tx;
      }
      da[b * kChunk + j].y = dt;
      if (j > 0) da[b * kChunk + j - 1].x = a;
      if (j == kChunk - 1) da[b * kChunk + j].x = 1.f;
      abar[b * kChunk + j] = pre;
      mbar_arrive(&bars->da_full[b]);
      const float wj = dt * suf;
      load_da(c + 1);

      if (!wait_warp(&bars->v_full[b], c >> 1)) break;
      uint8_t* vrow = smem + Lay::v + b * kTile + j * 128;
      uint8_t* urow = smem + Lay::u + j * 128;
      float check = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int at = (x ^ (j & 7)) << 4;
        float f[8];
        Vec<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(vrow + at), f);
        uint32_t u1[4], u2[4], u3[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          check = fmaf(f[2 * e], 0.f, check);
          check = fmaf(f[2 * e + 1], 0.f, check);
          float f0 = j < len ? wj * f[2 * e] : 0.f, f1 = j < len ? wj * f[2 * e + 1] : 0.f;
          u1[e] = take_part(f0, f1);
          u2[e] = take_part(f0, f1);
          u3[e] = Vec<__nv_bfloat16>::pack2(f0, f1);
        }
        *reinterpret_cast<uint4*>(urow + at) = make_uint4(u1[0], u1[1], u1[2], u1[3]);
        *reinterpret_cast<uint4*>(urow + kTile + at) = make_uint4(u2[0], u2[1], u2[2], u2[3]);
        *reinterpret_cast<uint4*>(urow + 2 * kTile + at) = make_uint4(u3[0], u3[1], u3[2], u3[3]);
      }
      if (len < kChunk && !wait_warp(&bars->k_full[b], c >> 1)) break;
      if (j >= len) {
        // another sequence's tokens: zeros in v and k (0 times its NaN would be NaN)
        for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(vrow + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
        for (int i = 0; i < NT / 64; ++i)
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4*>(smem + Lay::k + b * Lay::kQK + i * kTile + j * 128 + 16 * x) =
                make_uint4(0u, 0u, 0u, 0u);
      } else if (check != check) {
        // what is not finite must not meet the zeros of the earlier tokens' rows of P
        for (int x = 0; x < 64; ++x) {
          uint16_t* e = reinterpret_cast<uint16_t*>(vrow) + x;
          if ((*e & 0x7F80) == 0x7F80) *e = 0;
        }
        bars->bad[b] = 1;
      }
      fence_async_smem();
      mbar_arrive(&bars->u_full);

      if (!wait_warp(&bars->ds_full, c)) break;
      tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t d1[32], d2[32];
        tmem_ld32(tl + kColDS + 32 * half, d1);
        tmem_ld32(tl + kColDS + kPT + 32 * half, d2);
        tmem_wait_ld(d1);
        tmem_wait_ld(d2);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[32 * half + e] = fmaf(all, S[32 * half + e], __uint_as_float(d1[e]) + __uint_as_float(d2[e]));
      }
      tc_fence_before();
      if (c + 1 < chunks) {
        if (!wait_warp(&bars->q_empty, c)) break;  // Y2 has read the state before
        put_state();
      }
    }
    if (!*abort) {
#pragma unroll
      for (int e = 0; e < kPT; ++e)
        if (n < p.N && p0 + e < p.P) Sg[(size_t)(p0 + e) * p.N] = S[e];
      if (p.counts && h == 0 && p0 == 0 && j == 0) p.counts[row] = 0;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// [tokens][heads][width] BF16 in tiles of 128 tokens by 64 values of one head; what lies
// past the tokens or the width reads as zero
bool tile_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int width) {
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * heads * 2};
  const cuuint32_t box[3] = {64, 1, kChunk}, step[3] = {1, 1, 1};
  EncodeFn f = encode_fn();
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch_tc(const ScanTcParams& tp, int64_t units, cudaStream_t s) {
  constexpr int smem = TcLayout<NT>::bytes;
  static bool configured[64] = {false};  // per device; setting it twice does no harm
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(scan_tc_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  return pdl_launch(scan_tc_kernel<NT>, dim3((unsigned)units), kTcThreads, smem, s, tp);
}

}  // namespace

cudaError_t launch_scan_tc(const ScanParams& p, int num_sms, cudaStream_t s) {
  ScanTcParams tp;
  tp.s = p;
  if (!tile_map(&tp.q, p.q, p.pk.tokens, p.G, p.N) || !tile_map(&tp.k, p.k, p.pk.tokens, p.G, p.N) ||
      !tile_map(&tp.v, p.v, p.pk.tokens, p.H, p.P))
    return cudaErrorInvalidValue;
  const int64_t units = (int64_t)p.pk.n_seqs * p.H * ((p.P + kPT - 1) / kPT);
  return p.N > 64 ? launch_tc<128>(tp, units, s) : launch_tc<64>(tp, units, s);
}

}  // namespace replay
