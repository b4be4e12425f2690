// The scan of packed prompts on the tensor cores, for BF16 inputs. A chunk of Q = 128 tokens
// of one head is four products, with r_ij = prod_{j < l <= i} a_l:
//   C  = Q K^T                          y_i  = abar_i Y2_i + Y1_i,   abar_i = prod_{l <= i} a_l
//   Y1 = P V,  P_ij = C_ij r_ij Delta_j (j <= i)
//   Y2 = Q S^T                          S   <- abar_Q S + dS
//   dS = U^T K, U_j = (Delta_j prod_{l > j} a_l) v_j
// A block walks units, a head of a sequence (64 of its P rows) each, longest sequences first.
// q, k and v come by TMA into 128-byte swizzled tiles; C, Y1, Y2 and dS are accumulators in
// tensor memory; S stays in registers, half a state column n a thread. FP32 factors enter the
// products as sums of BF16 parts: U in three (what is left is under 2^-24 of it, so that the
// state keeps FP32 accuracy), S and P in two (2^-16, under the outputs' own rounding of 2^-8).
// dS is summed apart from S, since the accumulators do not round to nearest and S may hold
// thousands of tokens. Decays are products, never exponentials of differences: a = 0 and any
// sign need no care, and magnitudes above 1 only that no run of them overflows. A few long sequences are cut into segments: the segments' own states first
// (LOCAL: k and v only), then the states that they start from, then all segments at once.
//
// What bounds it: a chunk of one head at N = 128 takes an SM about 4900 cycles. Its products
// are 2300 of them (tensor pipe 47 % active), its wavefronts in the shared-memory pipe 3000, its
// instructions 2600 a scheduler; the chain C - P - Y1 within a chunk, whose P lies where the
// next C will, keeps them from overlapping further. (The parts of Y2 and dS lie side by side
// and fill tensor memory. Summed onto one another, S's second part and U's third would free the
// 128 columns of a second C, for narrower products; not tried.) 8192 tokens of the 64-head layer
// (G = 64): 109 us, 60 % of the measured copy bandwidth; 32768 tokens of one sequence (G = 8):
// 511 us, of which a third the segments' own states. Both at 1965 MHz: run for a second on end they
// meet the power limit, and at 1590 and 1657 MHz take 126 and 582 us. One part each for P and
// S gained 3 to 5 % and raised the outputs' error from 1.7e-3 to 2.3e-3: left at two.
#include <atomic>

#include "layer_device.cuh"
#include "tcgen05.cuh"

namespace replay {

namespace {

constexpr int kChunk = 128;
constexpr int kPT = 64;        // state rows of one block
constexpr int kSplitSms = 148;  // the SMs that a split aims to fill
constexpr int kTcThreads = 896;
// Seven warpgroups: 0 and 1 (rows of C: P and the outputs), 2 and 3 (tokens: decays and U),
// 4 and 5 (columns of the state), each pair sharing the work by columns, and 6 (plan, TMA
// and MMA). At 72 registers a thread at launch, 2, 3 and 6 give up what the state needs.
constexpr int kWarpU = 8, kWarpS = 16, kWarpTma = 24, kWarpMmaQ = 25, kWarpMmaU = 26, kWarpPlan = 27;
constexpr int kRegsLaunch = 72, kRegsTokens = 64, kRegsState = 88, kRegsCopy = 56;
static_assert(2 * (kRegsLaunch + kRegsTokens + kRegsState) + kRegsCopy <= 7 * kRegsLaunch, "registers moved, not made");
constexpr int kSlots = 5;  // chunks whose decays are held: who writes one knows that the fifth before it is done with

struct alignas(64) ScanTcParams {
  CUtensorMap q, k, v;
  ScanParams s;
  int wide_y;  // rows of y start on 32-byte boundaries
  int units;   // sequences (or segments) x heads x blocks of 64 rows; block b takes b, b + grid, ..
};

// Tensor memory columns. P lies over C: the two BF16 parts of 16 columns of P take the 16
// columns that held C's. (LOCAL: two buffers of dS alone.)
constexpr uint32_t kColC = 0, kColY1 = 128, kColY2 = 192, kColDS = 320;

// A block's next unit: tokens [begin, begin + len) of one sequence, 64 state rows from p0 of
// one head. len < 0: there is none.
struct Unit {
  int begin, len, h, g, p0, row, id;
  int from, to;  // the state that it starts from and leaves: 0 zero / nowhere, 1 the caller's, 2 the segment's
};
constexpr int kSortSeqs = 64;  // up to as many sequences are taken longest first

struct TcBars {
  uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t c_full, p_full, y_full, y_free, u_full[2], ds_full[2], ds_free[2], s_full, da_full[kSlots], drain[2];
  uint64_t unit_full[2], unit_empty[2];
  uint32_t tmem, abort;
  int seg_tokens;  // of a segment, or more than any sequence has
  Unit unit[2];
  int order[kSortSeqs];
};
// the decays of one chunk; "block" is 32 tokens
struct alignas(16) Decays {
  float2 da[kChunk];  // a_{j+1}, Delta_j
  float g[kChunk];    // Delta_j times the a after j in its block
  float pre[kChunk];  // the a up to i in its block
  float total[4];     // each block's product
  int bad;            // the chunk holds a v that is not finite
};

template <int NT, bool LOCAL>
struct TcLayout {  // bytes from the 1024-byte aligned base
  static constexpr int kTile = kChunk * 128;  // 128 rows of 64 BF16
  static constexpr int kQK = NT / 64 * kTile;
  static constexpr int kSop = NT * 128;     // one part of the state operand: NT rows of 64 BF16
  static constexpr int kU = LOCAL ? 2 : 1;  // buffers of U and of dS
  static constexpr int q = 0, k = LOCAL ? 0 : kQK, v = k + 2 * kQK, u = v + 2 * kTile, s = u + kU * 3 * kTile;
  static constexpr int dec = s + (LOCAL ? 0 : 2 * kSop);
  static constexpr int bars = dec + kSlots * (int)sizeof(Decays);
  static_assert(dec % 16 == 0 && bars % 8 == 0, "vector reads of the decays, 8-byte barriers");
  static constexpr int bytes = bars + (int)sizeof(TcBars) + 1024;
};

// two floats' BF16 parts packed (the first in the low half), and what remains of them
__device__ __forceinline__ uint32_t take_part(f32x2& x) {
  float a, b;
  unpair(x, a, b);
  const uint32_t w = Vec<__nv_bfloat16>::pack2(a, b);
  x = fma2(pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), pair(-1.f, -1.f), x);
  return w;
}
__device__ __forceinline__ uint32_t last_part(f32x2 x) {
  float a, b;
  unpair(x, a, b);
  return Vec<__nv_bfloat16>::pack2(a, b);
}

// two registers of a load from tensor memory as a pair
__device__ __forceinline__ f32x2 reg_pair(const uint32_t* r) {
  return pair(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// 32 bytes, a whole sector, in one store (the address 32-byte aligned)
__device__ __forceinline__ void store_sector(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

}  // namespace

// The segments of sequence s (one, where its bounds are bad).
__device__ __forceinline__ int segments_of(const Packed& pk, int seg_tokens, int s) {
  const int64_t len = (int64_t)pk.cu[s + 1] - pk.cu[s];
  return len > seg_tokens && len <= pk.tokens ? (int)((len + seg_tokens - 1) / seg_tokens) : 1;
}

// Whether all segments have their place, by a whole warp. Sequences that share tokens, where
// bounds fall, can have more than the tokens allow; then every sequence is taken whole.
__device__ __forceinline__ bool segments_fit(const Packed& pk, int seg_tokens, int max_segs) {
  int n = 0;
#pragma unroll 1
  for (int s = threadIdx.x & 31; s < pk.n_seqs; s += 32) n = min(n + segments_of(pk, seg_tokens, s), 1 << 25);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
  return n <= max_segs;
}

// Segment number `seg` of the packed sequences' segments: its sequence, its place among the
// sequence's, and how many those are. Whole warps; false past the last segment.
__device__ __forceinline__ bool find_segment(const Packed& pk, int seg_tokens, int seg, int& s, int& m, int& of) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int s0 = 0; s0 < pk.n_seqs; s0 += 32) {
    const int n = s0 + lane < pk.n_seqs ? segments_of(pk, seg_tokens, s0 + lane) : 0;
    int upto = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > seg);
    if (hit) {
      const int l = __ffs(hit) - 1;
      s = s0 + l;
      of = __shfl_sync(0xffffffffu, n, l);
      m = seg - (before + __shfl_sync(0xffffffffu, upto - n, l));
      return s < pk.n_seqs;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

__device__ __forceinline__ bool takes_longest_first(const ScanParams& p) {
  return !p.seg_tokens && p.pk.n_seqs <= kSortSeqs;
}

// Unit number `id`, by a whole warp; false if there is nothing to do for it.
template <bool LOCAL>
__device__ __forceinline__ bool unit_of(const ScanTcParams& tp, TcBars* bars, int id, Unit& u) {
  const ScanParams& p = tp.s;
  const int ptiles = (p.P + kPT - 1) / kPT;
  int s = id / (p.H * ptiles), seg = 0, segs = 1;
  // the length of a segment is read where it is needed: a register of it would spill
  if (p.seg_tokens && !find_segment(p.pk, *const_cast<volatile int*>(&bars->seg_tokens), s, s, seg, segs)) return false;
  if (LOCAL && seg == segs - 1) return false;
  if (takes_longest_first(p)) s = bars->order[s];
  int64_t begin, end;
  if (!seq_bounds(p.pk, s, begin, end)) return false;
  if (segs > 1) {
    begin += (int64_t)seg * p.seg_tokens;
    if (seg < segs - 1) end = begin + p.seg_tokens;
  }
  u.row = seq_row(p.pk, s);
  if (u.row < 0) return false;
  u.begin = (int)begin, u.len = (int)(end - begin);
  u.h = id / ptiles % p.H, u.g = u.h / (p.H / p.G), u.p0 = id % ptiles * kPT;
  u.id = id;
  u.from = LOCAL ? 0 : segs > 1 ? 2 : p.pk.resume && p.pk.resume[s] ? 1 : 0;
  u.to = LOCAL ? 2 : seg == segs - 1 ? 1 : 0;
  return true;
}

// A block's unit of a round. After the first round the blocks take units in turned order: long
// ones go with short ones.
__device__ __forceinline__ int id_of(int round) {
  return round * gridDim.x + (round == 0 ? blockIdx.x : gridDim.x - 1 - blockIdx.x);
}

// After a wait that gave up: NaN over the outputs and states that the block was to make, by
// warps 0 to 7, so that the failure shows where the caller looks at no status word.
template <bool LOCAL>
__device__ __forceinline__ void spoil(const ScanTcParams& tp, TcBars* bars) {
  const ScanParams& p = tp.s;
  const int lane = threadIdx.x & 31;
  const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
  for (int round = threadIdx.x / 32; round * (int64_t)gridDim.x < tp.units; round += kWarpU) {
    const int id = id_of(round);
    Unit u;
    if (id >= tp.units || !unit_of<LOCAL>(tp, bars, id, u)) continue;
    const int rows = p.P - u.p0 < kPT ? p.P - u.p0 : kPT;
    float* state = LOCAL ? p.seg_state + (size_t)id * kPT * p.N : p.S + (((size_t)u.row * p.H + u.h) * p.P + u.p0) * p.N;
    if (u.to)
#pragma unroll 1
      for (int i = lane; i < rows * p.N; i += 32) state[i] = nan;
    if (LOCAL) {
      if (lane == 0) p.seg_decay[id] = nan;
      continue;
    }
    const int vecs = rows / 8;  // P is a multiple of 8
#pragma unroll 1
    for (int64_t i = lane; i < (int64_t)u.len * vecs; i += 32) {
      const int64_t t = u.begin + i / vecs;
      uint16_t* y = static_cast<uint16_t*>(p.y) + ((size_t)t * p.H + u.h) * p.P + u.p0 + i % vecs * 8;
      *reinterpret_cast<uint4*>(y) = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    }
  }
}

// LOCAL: only the segments' own states, from zero, for those with a segment behind them.
template <int NT, bool LOCAL>
__global__ void __launch_bounds__(kTcThreads, 1) scan_tc_kernel(const __grid_constant__ ScanTcParams tp) {
  using Lay = TcLayout<NT, LOCAL>;
  constexpr int kTile = Lay::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  TcBars* bars = reinterpret_cast<TcBars*>(smem + Lay::bars);
  Decays* dec = reinterpret_cast<Decays*>(smem + Lay::dec);
  const ScanParams& p = tp.s;
  // values of the whole warp, told so to the compiler
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1), mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], 1), mbar_init(&bars->k_empty[i], LOCAL ? 1 : 2);
      mbar_init(&bars->v_full[i], 1), mbar_init(&bars->v_empty[i], LOCAL ? 256 : 1);
    }
    mbar_init(&bars->c_full, 1), mbar_init(&bars->p_full, 256);
    mbar_init(&bars->y_full, 1), mbar_init(&bars->y_free, 256);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->u_full[i], 256);
    mbar_init(&bars->s_full, 256);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->ds_full[i], 1), mbar_init(&bars->ds_free[i], 256);
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars->da_full[i], 128);
    mbar_init(&bars->drain[0], 1), mbar_init(&bars->drain[1], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->unit_full[i], 1), mbar_init(&bars->unit_empty[i], LOCAL ? 18 : 27);
    bars->abort = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kWarpTma) tmem_alloc(&bars->tmem, 512);
  if (warp == kWarpPlan) {
    const bool fit = !p.seg_tokens || segments_fit(p.pk, p.seg_tokens, p.max_segs);
    if (lane == 0) bars->seg_tokens = fit ? p.seg_tokens : INT32_MAX;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(bars->tmem);
  volatile uint32_t* abort = &bars->abort;

  // waits for a phase; false if it takes too long (the block then winds down: every other
  // wait of its ends within the same time)
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    int left = kPollLimit;
#pragma unroll 1
    while (!mbar_poll(bar, phase & 1)) {
      if (--left == 0) {
        *abort = 1;
        return false;
      }
    }
    return true;
  };
  // two phases, tested together
  auto wait2 = [&](uint64_t* bar0, int phase0, uint64_t* bar1, int phase1) -> bool {
    const bool b0 = mbar_poll(bar0, phase0 & 1), b1 = mbar_poll(bar1, phase1 & 1);
    return (b0 || wait(bar0, phase0)) && (b1 || wait(bar1, phase1));
  };
  // the same for a whole warp: every lane goes on, or none
  auto wait_warp = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
  auto wait2_warp = [&](uint64_t* bar0, int phase0, uint64_t* bar1, int phase1) {
    return __all_sync(0xffffffffu, wait2(bar0, phase0, bar1, phase1)) != 0;
  };

  // the k-th unit (by a lane of its own, or a whole warp); its chunks, < 0 if there is none
  auto take_unit = [&](Unit& u, int k) -> int {
    if (!wait(&bars->unit_full[k & 1], k >> 1)) return -1;
    u = bars->unit[k & 1];
    mbar_arrive(&bars->unit_empty[k & 1]);
    return u.len < 0 ? -1 : (u.len + kChunk - 1) / kChunk;
  };
  auto take_unit_warp = [&](Unit& u, int k) -> int {
    if (!wait_warp(&bars->unit_full[k & 1], k >> 1)) return -1;
    u = bars->unit[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->unit_empty[k & 1]);
    return uniform(u.len < 0 ? -1 : (u.len + kChunk - 1) / kChunk);
  };
  auto ds_col = [](int n) { return LOCAL ? (uint32_t)(n & 1) * 256 : kColDS; };
  // Every role walks the block's units and their chunks; n counts the chunks, over all units,
  // and gives the phases of the barriers.

  if (warp >= kWarpTma) {
    regs_down<kRegsCopy>();
    // ------------------------------------------------------------ plan
    if (warp == kWarpPlan) {
      if (takes_longest_first(p)) {
        for (int s = lane; s < p.pk.n_seqs; s += 32) {
          const int len = p.pk.cu[s + 1] - p.pk.cu[s];
          int rank = 0;
          for (int e = 0; e < p.pk.n_seqs; ++e) {
            const int other = p.pk.cu[e + 1] - p.pk.cu[e];
            rank += other > len || (other == len && e < s);
          }
          bars->order[rank] = s;
        }
        __syncwarp();
      }
      int k = 0;
      bool more = true;
#pragma unroll 1
      for (int round = 0; more; ++round) {
        const int id = id_of(round);
        Unit u;
        u.len = -1;
        more = round * (int64_t)gridDim.x < tp.units;
        if (more) {
          if (id >= tp.units || !unit_of<LOCAL>(tp, bars, id, u)) continue;
          if (u.from && lane == 0)  // the state that it starts from into L2
            prefetch_l2(u.from == 2 ? p.seg_state + (size_t)id * kPT * p.N
                                    : p.S + (((size_t)u.row * p.H + u.h) * p.P + u.p0) * p.N,
                        (p.P - u.p0 < kPT ? p.P - u.p0 : kPT) * p.N * 4);
        }
        if (k >= 2 && !wait_warp(&bars->unit_empty[k & 1], (k >> 1) - 1)) break;
        if (lane == 0) {
          bars->unit[k & 1] = u;
          mbar_arrive(&bars->unit_full[k & 1]);
        }
        ++k;
      }
    }
    // ------------------------------------------------------------ TMA
    if (warp == kWarpTma && lane == 0) {
      // q of a chunk, then k and v of the next: the order in which their tiles fall free. The q
      // first, and then the look for the next chunk: behind units without any it comes only once
      // every role has gone on to them.
      int n = 0, nq = 0;  // tiles of k and v, and of q, issued
      Unit u;
      int chunks = 0, c = 0, tq = -1, gq = 0;  // the chunk whose q is due: its first token and group
#pragma unroll 1
      for (int k = 0; chunks >= 0;) {
        if (!LOCAL && tq >= 0) {
          if (nq >= 1 && !wait(&bars->q_empty, nq - 1)) break;
          mbar_arrive_expect_tx(&bars->q_full, Lay::kQK);
#pragma unroll 1
          for (int i = 0; i < NT / 64; ++i) tma_load3(smem + Lay::q + i * kTile, &tp.q, 64 * i, gq, tq, &bars->q_full);
          ++nq;
        }
        while (chunks >= 0 && c >= chunks) chunks = take_unit(u, k++), c = 0;
        if (chunks < 0) break;
        const int t = u.begin + c * kChunk;
        if (!LOCAL && tq >= 0) {  // q has one tile, so its next load starts late: from L2
#pragma unroll 1
          for (int i = 0; i < NT / 64; ++i) tma_prefetch3(&tp.q, 64 * i, u.g, t);
        }
        const int b = n & 1;
        if (n >= 2 && !wait(&bars->k_empty[b], (n >> 1) - 1)) break;
        mbar_arrive_expect_tx(&bars->k_full[b], Lay::kQK);
#pragma unroll 1
        for (int i = 0; i < NT / 64; ++i)
          tma_load3(smem + Lay::k + b * Lay::kQK + i * kTile, &tp.k, 64 * i, u.g, t, &bars->k_full[b]);
        if (n >= 2 && !wait(&bars->v_empty[b], (n >> 1) - 1)) {
          mbar_wait_bounded(&bars->k_full[b], (n >> 1) & 1);
          break;
        }
        mbar_arrive_expect_tx(&bars->v_full[b], kTile);
        tma_load3(smem + Lay::v + b * kTile, &tp.v, u.p0, u.h, t, &bars->v_full[b]);
        if (c + 1 < chunks) {  // the next tiles' loads start late too
          tma_prefetch3(&tp.v, u.p0, u.h, t + kChunk);
#pragma unroll 1
          for (int i = 0; i < NT / 64; ++i) tma_prefetch3(&tp.k, 64 * i, u.g, t + kChunk);
        }
        ++n, ++c;
        tq = t, gq = u.g;
      }
      if (*abort) {  // no copy may land after the block has gone
        if (nq) mbar_wait_bounded(&bars->q_full, (nq - 1) & 1);
        for (int b = 0; b < 2; ++b) {
          if (n > b) mbar_wait_bounded(&bars->k_full[b], ((n - 1 - b) >> 1) & 1);
          if (n > b) mbar_wait_bounded(&bars->v_full[b], ((n - 1 - b) >> 1) & 1);
        }
      }
    }
    // ------------------------------------------------------------ MMA
    // Two warps, since one that has issued a product goes on only once the product runs: with
    // two the tensor cores have the next product at hand.
    constexpr uint32_t kC = mma_idesc(128, 128, 0, 0), kY1 = mma_idesc(128, kPT, 0, 1);
    constexpr uint32_t kY2 = mma_idesc(128, 2 * kPT, 0, 1), kDS = mma_idesc(128, 3 * kPT, 1, 1);
    // operand tiles; a step of 16 of K is 32 bytes along a K-major row, 16 rows of an MN-major tile
    if (!LOCAL && warp == kWarpMmaQ) {
      const uint64_t dq = smem_desc(smem_u32(smem + Lay::q), 16);
      const uint64_t ds = smem_desc(smem_u32(smem + Lay::s), Lay::kSop);
      Unit u;
      int n = 0, chunks;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok && (chunks = take_unit_warp(u, k)) >= 0; ++k) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, ++n) {
          const int b = n & 1;
          const uint64_t dk = smem_desc(smem_u32(smem + Lay::k + b * Lay::kQK), 16);
          // C = Q K^T, once Y1 is done with the last chunk's P in the same columns
          if (!(ok = wait2_warp(&bars->q_full, n, &bars->k_full[b], n >> 1))) break;
          if (n >= 1 && !(ok = wait_warp(&bars->y_full, n - 1))) break;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll 2
            for (int i = 0; i < NT / 16; ++i) {
              const int at = (i / 4 * kTile + i % 4 * 32) >> 4;
              mma_ss(tmem + kColC, dq + at, dk + at, kC, i > 0);
            }
            mma_commit(&bars->c_full);
          }
          // Y2 = Q S^T, the state's two parts side by side, once the last chunk's outputs have been read
          if (!(ok = wait_warp(&bars->s_full, n) && (n == 0 || wait_warp(&bars->y_free, n - 1)))) break;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll 2
            for (int i = 0; i < NT / 16; ++i)
              mma_ss(tmem + kColY2, dq + ((i / 4 * kTile + i % 4 * 32) >> 4), ds + i * 128, kY2, i > 0);
            mma_commit(&bars->q_empty);
            mma_commit(&bars->k_empty[b]);
          }
        }
      }
    } else if (warp == kWarpMmaU) {
      const uint64_t du = smem_desc(smem_u32(smem + Lay::u), kTile);
      Unit u;
      int n = 0, chunks;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok && (chunks = take_unit_warp(u, k)) >= 0; ++k) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, ++n) {
          const int b = n & 1;
          const uint64_t dk = smem_desc(smem_u32(smem + Lay::k + b * Lay::kQK), kTile);
          const uint64_t dv = smem_desc(smem_u32(smem + Lay::v + b * kTile), 16);
          // dS = K^T U, the three parts side by side, behind C, which the rows wait for
          if (!(ok = wait2_warp(&bars->u_full[n % Lay::kU], n / Lay::kU, &bars->k_full[b], n >> 1))) break;
          if (n >= Lay::kU && !(ok = wait_warp(&bars->ds_free[n % Lay::kU], n / Lay::kU - 1))) break;
          if (!LOCAL && !(ok = wait_warp(&bars->c_full, n))) break;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll 2
            for (int i = 0; i < kChunk / 16; ++i) mma_ss(tmem + ds_col(n), dk + i * 128, du + (n % Lay::kU * 3 * kTile >> 4) + i * 128, kDS, i > 0);
            mma_commit(&bars->ds_full[n % Lay::kU]);
            mma_commit(&bars->k_empty[b]);
          }
          if (LOCAL) continue;
          // Y1 = P V
          if (!(ok = wait2_warp(&bars->p_full, n, &bars->v_full[b], n >> 1))) break;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll 2
            for (int i = 0; i < kChunk / 16; ++i) {
              const uint32_t pa = tmem + kColC + i * 16;
              mma_ts(tmem + kColY1, pa, dv + i * 128, kY1, i > 0);
              mma_ts(tmem + kColY1, pa + 8, dv + i * 128, kY1, true);
            }
            mma_commit(&bars->y_full);
            mma_commit(&bars->v_empty[b]);
          }
        }
      }
    }
    if (*abort && (warp == kWarpMmaQ || warp == kWarpMmaU)) {  // nothing may still run when the memory is freed
      if (elect_lane()) mma_commit(&bars->drain[warp - kWarpMmaQ]);
      mbar_wait_bounded(&bars->drain[warp - kWarpMmaQ], 0);
    }
  } else if (warp < kWarpU) {
    // ------------------------------------------------------------ P and the outputs: row i of the chunk
    const int w4 = warp & 3, half = warp >> 2;
    const int i = w4 * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(w4 * 32) << 16);
    Unit u;
    int n = 0, chunks;
    bool ok = !LOCAL;
#pragma unroll 1
    for (int k = 0; ok && (chunks = take_unit_warp(u, k)) >= 0; ++k) {
      const int64_t end = (int64_t)u.begin + u.len;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++n) {
        const Decays& d = dec[n % kSlots];
        if (!(ok = wait2_warp(&bars->da_full[n % kSlots], n / kSlots, &bars->c_full, n))) break;
        tc_fence_after();
        const float pre = d.pre[i];
        // Half 0 takes the diagonal block of 32 columns, half 1 those before it. The loops stay
        // small: the roles share an instruction cache, and unrolled they waited for instructions.
        if (half == 0) {
          const float4* da = reinterpret_cast<const float4*>(d.da + 32 * w4);
          float rd = 0.f;
#pragma unroll 1
          for (int j0 = 16; j0 >= 0; j0 -= 16) {  // products from j = i down
            uint32_t x[16], hi[8], lo[8];
            tmem_ld16(tl + kColC + 32 * w4 + j0, x);
            tmem_wait_ld16(x);
#pragma unroll
            for (int j = 14; j >= 0; j -= 2) {
              const float4 w = da[(j0 + j) / 2];  // a_{j+1}, Delta_j, a_{j+2}, Delta_{j+1}
              rd = j + 1 == lane - j0 ? 1.f : rd * w.z;
              const float f1 = j + 1 <= lane - j0 ? __uint_as_float(x[j + 1]) * (rd * w.w) : 0.f;
              rd = j == lane - j0 ? 1.f : rd * w.x;
              const float f0 = j <= lane - j0 ? __uint_as_float(x[j]) * (rd * w.y) : 0.f;
              f32x2 f = pair(f0, f1);
              hi[j / 2] = take_part(f);
              lo[j / 2] = last_part(f);
            }
            tmem_st8(tl + kColC + 32 * w4 + j0, hi);
            tmem_st8(tl + kColC + 32 * w4 + j0 + 8, lo);
          }
        } else {
          const uint32_t zero[8] = {0};
#pragma unroll 1
          for (int x = 32 * (w4 + 1); x < kChunk; x += 8) tmem_st8(tl + kColC + x, zero);  // later tokens
        }
        float r = pre;  // from the block's end up to i
#pragma unroll 1
        for (int cb = half == 0 ? -1 : w4 - 1; cb >= 0; --cb) {
          uint32_t x[32];
          tmem_ld32(tl + kColC + 32 * cb, x);
          const ulonglong2* gv = reinterpret_cast<const ulonglong2*>(d.g + 32 * cb);
          const f32x2 rr = pair(r, r);
          r *= d.total[cb];
          tmem_wait_ld32(x);
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const ulonglong2 e = gv[(j0 + j) / 4];
              f32x2 f = mul2(pair(__uint_as_float(x[j0 + j]), __uint_as_float(x[j0 + j + 1])), mul2(rr, e.x));
              hi[j / 2] = take_part(f);
              lo[j / 2] = last_part(f);
              f = mul2(pair(__uint_as_float(x[j0 + j + 2]), __uint_as_float(x[j0 + j + 3])), mul2(rr, e.y));
              hi[j / 2 + 1] = take_part(f);
              lo[j / 2 + 1] = last_part(f);
            }
            tmem_st8(tl + kColC + 32 * cb + j0, hi);
            tmem_st8(tl + kColC + 32 * cb + j0 + 8, lo);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full);

        float abar = pre;
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (x < w4) abar *= d.total[x];
        if (!(ok = wait2_warp(&bars->y_full, n, &bars->q_empty, n))) break;
        tc_fence_after();
        const bool bad = d.bad != 0;
        const int64_t t = u.begin + (int64_t)c * kChunk + i;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + ((size_t)t * p.H + u.h) * p.P + u.p0 + 32 * half;
        const f32x2 ab = pair(abar, abar);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          uint32_t y1[16], y2[16], y3[16], o[8];
          tmem_ld16(tl + kColY1 + 32 * half + 16 * part, y1);
          tmem_ld16(tl + kColY2 + 32 * half + 16 * part, y2);
          tmem_ld16(tl + kColY2 + kPT + 32 * half + 16 * part, y3);
          tmem_wait_ld16(y1);
          tmem_wait_ld16(y2);
          tmem_wait_ld16(y3);
          if (part == 1) {
            tc_fence_before();
            mbar_arrive(&bars->y_free);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            o[j / 2] = last_part(fma2(ab, add2(reg_pair(y2 + j), reg_pair(y3 + j)), reg_pair(y1 + j)));
          const int left = t < end ? p.P - (u.p0 + 32 * half + 16 * part) : 0;  // of the head's rows p
          if (left >= 16 && tp.wide_y) {
            store_sector(y + 16 * part, o);
          } else {
            if (left > 0) *reinterpret_cast<uint4*>(y + 16 * part) = make_uint4(o[0], o[1], o[2], o[3]);
            if (left > 8) *reinterpret_cast<uint4*>(y + 16 * part + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        if (bad) {
          // the products saw zeros in place of what is not finite in v: it reaches every later row
          const uint16_t* v = static_cast<const uint16_t*>(p.v) + (size_t)u.h * p.P + u.p0 + 32 * half;
#pragma unroll 1
          for (int e = 0; e < 32 && u.p0 + 32 * half + e < p.P; ++e) {
            int first = kChunk;
#pragma unroll 1
            for (int r0 = 0; r0 < kChunk && first == kChunk; r0 += 32) {
              const int64_t tr = t - i + r0 + lane;
              const uint16_t x = tr < end ? v[(size_t)tr * p.H * p.P + e] : 0;
              const unsigned hit = __ballot_sync(0xffffffffu, (x & 0x7F80) == 0x7F80);
              if (hit) first = r0 + __ffs(hit) - 1;
            }
            if (t < end && first <= i) reinterpret_cast<uint16_t*>(y)[e] = 0x7FC0;
          }
        }
      }
    }
  } else if (warp < kWarpS) {
    // ------------------------------------------------------------ decays and U: token j of the chunk
    regs_down<kRegsTokens>();
    const int j = (threadIdx.x - 32 * kWarpU) & 127, w4 = warp & 3, half = (warp - kWarpU) >> 2;
    float a = 1.f, dt = 0.f;
    Unit u;
    int n = 0, chunks;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok && (chunks = take_unit_warp(u, k)) >= 0; ++k) {
      const int64_t end = (int64_t)u.begin + u.len;
      auto load_da = [&](int c) {  // this thread's token of chunk c; past the sequence: no decay, no step
        const int64_t t = u.begin + (int64_t)c * kChunk + j;
        const bool in = c < chunks && t < end;
        a = in ? p.a[(size_t)t * p.H + u.h] : 1.f;
        dt = in ? p.dt[(size_t)t * p.H + u.h] : 0.f;
      };
      if (half == 0) load_da(0);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++n) {
        const int b = n & 1;
        Decays& d = dec[n % kSlots];
        const int len = u.len - c * kChunk < kChunk ? u.len - c * kChunk : kChunk;
        if (half == 0) {
          // products of the decays up to and after this token, in its block and then over the chunk
          float pre = a, suf = a;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const float e = __shfl_up_sync(0xffffffffu, pre, off), f = __shfl_down_sync(0xffffffffu, suf, off);
            if (lane >= off) pre *= e;
            if (lane + off < 32) suf *= f;
          }
          suf = __shfl_down_sync(0xffffffffu, suf, 1);
          if (lane == 31) suf = 1.f;
          if (lane == 31) d.total[w4] = pre;
          if (j == 0) d.bad = 0;
          d.pre[j] = pre;
          d.g[j] = dt * suf;
          d.da[j].y = dt;
          if (j > 0) d.da[j - 1].x = a;
          if (j == kChunk - 1) d.da[j].x = 1.f;
          mbar_arrive(&bars->da_full[n % kSlots]);
          load_da(c + 1);
        }
        if (!(ok = wait_warp(&bars->da_full[n % kSlots], n / kSlots))) break;
        float wj = d.g[j];
#pragma unroll
        for (int x = 1; x < 4; ++x)
          if (x > w4) wj *= d.total[x];

        if (!(ok = wait_warp(&bars->v_full[b], n >> 1))) break;
        // the buffer's last values have been read
        if (n >= Lay::kU && !(ok = wait_warp(&bars->ds_full[n % Lay::kU], n / Lay::kU - 1))) break;
        uint8_t* vrow = smem + Lay::v + b * kTile + j * 128;
        uint8_t* urow = smem + Lay::u + n % Lay::kU * 3 * kTile + j * 128;
        if (len < kChunk && !(ok = wait_warp(&bars->k_full[b], n >> 1))) break;
        if (j >= len) {
          // another sequence's tokens: zeros in v and k (0 times its NaN would be NaN)
          for (int x = 4 * half; x < 4 * half + 4; ++x)
            *reinterpret_cast<uint4*>(vrow + ((x ^ (j & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          for (int i = half; i < NT / 64; i += 2)
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4*>(smem + Lay::k + b * Lay::kQK + i * kTile + j * 128 + 16 * x) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        const f32x2 ww = pair(wj, wj);
        f32x2 check[2] = {0, 0};  // 0 times what is not finite is NaN
#pragma unroll 2
        for (int x = 4 * half; x < 4 * half + 4; ++x) {
          const int at = (x ^ (j & 7)) << 4;
          const uint4 vu = *reinterpret_cast<const uint4*>(vrow + at);
          float f[8];
          Vec<__nv_bfloat16>::unpack(vu, f);
          uint32_t u1[4], u2[4], u3[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x2 v2 = pair(f[2 * e], f[2 * e + 1]);
            check[e & 1] = fma2(v2, 0, check[e & 1]);
            f32x2 part = mul2(v2, ww);
            u1[e] = take_part(part);
            u2[e] = take_part(part);
            u3[e] = last_part(part);
          }
          *reinterpret_cast<uint4*>(urow + at) = make_uint4(u1[0], u1[1], u1[2], u1[3]);
          *reinterpret_cast<uint4*>(urow + kTile + at) = make_uint4(u2[0], u2[1], u2[2], u2[3]);
          *reinterpret_cast<uint4*>(urow + 2 * kTile + at) = make_uint4(u3[0], u3[1], u3[2], u3[3]);
        }
        float c0, c1;
        unpair(add2(check[0], check[1]), c0, c1);
        if (!LOCAL && c0 + c1 != 0.f) {
          // what is not finite must not meet the zeros of the earlier tokens' rows of P
#pragma unroll 1
          for (int x = 32 * half; x < 32 * half + 32; ++x) {
            uint16_t* e = reinterpret_cast<uint16_t*>(vrow + (((x >> 3) ^ (j & 7)) << 4)) + (x & 7);
            if ((*e & 0x7F80) == 0x7F80) *e = 0;
          }
          d.bad = 1;
        }
        fence_async_smem();
        mbar_arrive(&bars->u_full[n % Lay::kU]);
        if (LOCAL) mbar_arrive(&bars->v_empty[b]);
      }
    }
  } else if (warp < kWarpTma) {
    // ------------------------------------------------------------ the state: column n
    regs_up<kRegsState>();
    const int sn = (threadIdx.x - 32 * kWarpS) & 127, w4 = warp & 3, half = (warp - kWarpS) >> 2;  // column n, half of p
    const uint32_t tl = tmem + ((uint32_t)(w4 * 32) << 16);
    f32x2 S[kPT / 4];
    // 16 rows p of the state's two BF16 parts as an operand: row n, chunk x at x ^ (n % 8)
    uint8_t* dst = smem + Lay::s + sn * 128;
    auto put_state = [&](int part) {
#pragma unroll
      for (int x = 2 * part; x < 2 * part + 2; ++x) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x2 f = S[4 * x + e];
          hi[e] = take_part(f);
          lo[e] = last_part(f);
        }
        uint8_t* at = dst + (((4 * half + x) ^ (sn & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + Lay::kSop) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    };
    Unit u;
    int n = 0, chunks;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok && (chunks = take_unit_warp(u, k)) >= 0; ++k) {
      // rows p of the state that it starts from: the caller's, a segment's, or zero
      float* Sg = p.S + (((size_t)u.row * p.H + u.h) * p.P + u.p0 + 32 * half) * p.N + sn;
      float* Eg = p.seg_state + ((size_t)u.id * kPT + 32 * half) * p.N + sn;
      const int rows = sn < p.N ? p.P - u.p0 - 32 * half : 0;  // P is a multiple of 8
      const float* from = u.from == 2 ? Eg : Sg;
#pragma unroll
      for (int e = 0; e < kPT / 2; e += 2)
        S[e / 2] = u.from && e < rows ? pair(from[(size_t)e * p.N], from[(size_t)(e + 1) * p.N]) : 0;
      float decay = 1.f;
      if (!LOCAL && chunks > 0) {  // the last chunk's Y2 has read the operand
        if (sn < NT) {
#pragma unroll
          for (int part = 0; part < 2; ++part) put_state(part);
        }
        fence_async_smem();
        mbar_arrive(&bars->s_full);
      }
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++n) {
        // dS is there, and Y2 has read the state's operand
        if (!(ok = LOCAL ? wait_warp(&bars->ds_full[n % Lay::kU], n / Lay::kU) : wait2_warp(&bars->ds_full[0], n, &bars->q_empty, n))) break;
        tc_fence_after();
        const float* tot = dec[n % kSlots].total;
        const float all = (tot[0] * tot[1]) * (tot[2] * tot[3]);
        const f32x2 all2 = pair(all, all);
        if (LOCAL) decay *= all;
        const bool put = !LOCAL && c + 1 < chunks;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t d1[16], d2[16], d3[16];
          const uint32_t at = tl + ds_col(n) + 32 * half + 16 * part;
          tmem_ld16(at, d1);
          tmem_ld16(at + kPT, d2);
          tmem_ld16(at + 2 * kPT, d3);
          tmem_wait_ld16(d1);
          tmem_wait_ld16(d2);
          tmem_wait_ld16(d3);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            f32x2& x = S[8 * part + e / 2];
            x = fma2(all2, x, add2(reg_pair(d1 + e), add2(reg_pair(d2 + e), reg_pair(d3 + e))));
          }
          if (put && sn < NT) put_state(part);
        }
        tc_fence_before();
        mbar_arrive(&bars->ds_free[n % Lay::kU]);
        if (put) {
          fence_async_smem();
          mbar_arrive(&bars->s_full);
        }
      }
      if (!ok || !u.to) continue;
      float* to = u.to == 2 ? Eg : Sg;
#pragma unroll
      for (int e = 0; e < kPT / 2; e += 2) {
        float s0, s1;
        unpair(S[e / 2], s0, s1);
        if (e < rows) {
          to[(size_t)e * p.N] = s0;
          to[(size_t)(e + 1) * p.N] = s1;
        }
      }
      if (LOCAL && sn == 0 && half == 0) p.seg_decay[u.id] = decay;
      if (!LOCAL && p.counts && u.h == 0 && u.p0 == 0 && sn == 0 && half == 0) p.counts[u.row] = 0;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpTma) tmem_free(tmem, 512);
  if (*abort && threadIdx.x < 32 * kWarpU) {  // the warps that kept the registers of the launch
    if (p.pk.status && threadIdx.x == 0) atomicOr(p.pk.status, kErrWaitTimeout);
    spoil<LOCAL>(tp, bars);
  }
}

constexpr int kCarryAhead = 8;  // segments whose loads are in flight together

// The state that each segment starts from, in place of the segments' own: for the sequences
// of more than one segment, from the caller's row (or zero) on, S <- decay S + own. A block
// takes one sequence's head, a thread four columns of a row.
__global__ void __launch_bounds__(256) scan_carry_kernel(const __grid_constant__ ScanParams p) {
  pdl_enter();
  const int h = blockIdx.x % p.H;
  const int s = blockIdx.x / p.H;
  int64_t begin, end;
  if (!seq_bounds(p.pk, s, begin, end)) return;
  const int segs = (int)((end - begin + p.seg_tokens - 1) / p.seg_tokens);
  if (segs <= 1) return;
  const int row = seq_row(p.pk, s);
  if (row < 0) return;
  if (!segments_fit(p.pk, p.seg_tokens, p.max_segs)) return;
  // segments before this sequence's
  int first = 0;
  for (int e = threadIdx.x & 31; e < s; e += 32) first += segments_of(p.pk, p.seg_tokens, e);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) first += __shfl_xor_sync(0xffffffffu, first, off);
  const int ptiles = (p.P + kPT - 1) / kPT;
  const bool res = p.pk.resume && p.pk.resume[s];
  const int vecs = p.P * p.N / 4;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < vecs; i += gridDim.y * 256) {
    const int r = i * 4 / p.N, col = i * 4 % p.N;
    const int pt = r / kPT;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (res) S = *reinterpret_cast<const float4*>(p.S + (((size_t)row * p.H + h) * p.P + r) * p.N + col);
    const size_t step = (size_t)p.H * ptiles;
    const size_t unit0 = ((size_t)first * p.H + h) * ptiles + pt;
    float4* at = reinterpret_cast<float4*>(p.seg_state + (unit0 * kPT + r % kPT) * p.N + col);
    const size_t hop = step * kPT * p.N / 4;
    for (int m0 = 0; m0 < segs; m0 += kCarryAhead) {
      float4 own[kCarryAhead];
      float d[kCarryAhead];
#pragma unroll
      for (int u = 0; u < kCarryAhead; ++u) {
        const bool in = m0 + u < segs - 1;  // the last segment's own state is not needed
        own[u] = in ? at[(m0 + u) * hop] : make_float4(0.f, 0.f, 0.f, 0.f);
        d[u] = in ? p.seg_decay[unit0 + (m0 + u) * step] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kCarryAhead; ++u) {
        if (m0 + u < segs) at[(m0 + u) * hop] = S;
        S = make_float4(fmaf(d[u], S.x, own[u].x), fmaf(d[u], S.y, own[u].y), fmaf(d[u], S.z, own[u].z),
                        fmaf(d[u], S.w, own[u].w));
      }
    }
  }
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

template <int NT, bool LOCAL>
cudaError_t launch_tc(ScanTcParams& tp, int64_t units, int num_sms, cudaStream_t s) {
  constexpr int smem = TcLayout<NT, LOCAL>::bytes;
  static std::atomic<bool> configured[64];  // per device; two threads may both set the attribute, to the same
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(scan_tc_kernel<NT, LOCAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  tp.units = (int)units;
  return pdl_launch(scan_tc_kernel<NT, LOCAL>, dim3((unsigned)(units < num_sms ? units : num_sms)), kTcThreads, smem, s, tp);
}

template <int NT>
cudaError_t launch_scan_nt(ScanTcParams& tp, int num_sms, cudaStream_t s) {
  const ScanParams& p = tp.s;
  const int64_t heads = (int64_t)p.H * ((p.P + kPT - 1) / kPT);
  if (!p.seg_tokens) return launch_tc<NT, false>(tp, p.pk.n_seqs * heads, num_sms, s);
  cudaError_t e = launch_tc<NT, true>(tp, p.max_segs * heads, num_sms, s);
  if (e != cudaSuccess) return e;
  e = pdl_launch(scan_carry_kernel, dim3((unsigned)((int64_t)p.pk.n_seqs * p.H), (p.P * p.N / 4 + 255) / 256), 256, 0, s,
                 tp.s);
  return e != cudaSuccess ? e : launch_tc<NT, false>(tp, p.max_segs * heads, num_sms, s);
}

}  // namespace

ScanSplit scan_split(int64_t tokens, int32_t n_seqs, int64_t max_len, int H, int P) {
  if (tokens <= 0 || n_seqs <= 0) return {0, 0};
  const int64_t heads = (int64_t)H * ((P + kPT - 1) / kPT);
  const int64_t chunks = tokens / kChunk + n_seqs;  // about
  const int64_t longest = ((max_len > 0 && max_len < tokens ? max_len : tokens) + kChunk - 1) / kChunk;
  // Times in chunks of one block. Whole sequences: the SMs' share and, since the blocks do not
  // end together, half of the longest. Segments of n chunks: waves of n and a block's start
  // (2) each, 1.5 times for the segments' own states, and the launches (6).
  const int64_t whole = 2 * (chunks * heads / kSplitSms) + longest + 4;
  int64_t best = 0, seg = 0;
  for (int64_t n = 2; n < longest; n += n < 32 ? 1 : n / 16) {
    const int64_t units = (tokens / (n * kChunk) + n_seqs) * heads;
    if (units > INT32_MAX / 4) continue;
    const int64_t cost = 3 * ((units + kSplitSms - 1) / kSplitSms) * (n + 2) + 12;
    if (!seg || cost < best) best = cost, seg = n;
  }
  if (!seg || whole <= best) return {0, 0};
  return {(int32_t)(seg * kChunk), (int32_t)(tokens / (seg * kChunk) + n_seqs)};
}

cudaError_t launch_scan_tc(const ScanParams& p, int num_sms, cudaStream_t s) {
  ScanTcParams tp;
  tp.s = p;
  tp.wide_y = p.P % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 32 == 0;
  if (!tile_map(&tp.q, p.q, p.pk.tokens, p.G, p.N) || !tile_map(&tp.k, p.k, p.pk.tokens, p.G, p.N) ||
      !tile_map(&tp.v, p.v, p.pk.tokens, p.H, p.P))
    return cudaErrorInvalidValue;
  return p.N > 64 ? launch_scan_nt<128>(tp, num_sms, s) : launch_scan_nt<64>(tp, num_sms, s);
}

}  // namespace replay
