// What a prefill into a decode layer needs besides the scan: the mask of the resumed rows
// (whose buffered entries are folded first) and the refreshed read copy.
#include "layer_device.cuh"
#include "replay_kparams.h"

namespace replay {

namespace {

struct MaskParams {
  Packed pk;
  uint8_t* mask;
};
struct RefreshParams {
  Packed pk;
  int32_t H, P, ckpt;
  const float* S;
  uint8_t* codes;
  float* scale;
};

}  // namespace

// Only the rows that the scan then serves: a sequence with bad bounds is skipped, its row's
// buffered entries stay where they are. (The scan reports it.)
__global__ void resume_mask_kernel(const __grid_constant__ MaskParams p) {
  pdl_enter();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.pk.batch) return;
  int s = b;
  if (p.pk.seqs)
    for (s = 0; s < p.pk.n_seqs; ++s)
      if (p.pk.seqs[s] == b) break;  // the first of equal ids is served
  bool on = false;
  if (s < p.pk.n_seqs) {
    const int begin = p.pk.cu[s], end = p.pk.cu[s + 1];
    on = p.pk.resume[s] && begin >= 0 && end >= begin && end <= p.pk.tokens;
  }
  p.mask[b] = on;
}

// One block per (sequence, head): the head's rows requantised with the arithmetic of the
// row quantisers, N / 4 lanes a row.
template <int N>
__global__ void __launch_bounds__(256) refresh_copy_kernel(const __grid_constant__ RefreshParams p) {
  constexpr int TPR = N / 4, RPB = 256 / TPR;
  pdl_enter();
  const int s = blockIdx.x / p.H, h = blockIdx.x % p.H;
  int64_t begin, end;
  if (!seq_bounds(p.pk, s, begin, end)) return;
  const int row = seq_row(p.pk, s);
  if (row < 0) return;
  const size_t r0 = ((size_t)row * p.H + h) * p.P;
  const int col = (threadIdx.x % TPR) * 4;
  for (int i = 0; i < p.P; i += RPB) {
    const int r = i + (int)threadIdx.x / TPR;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < p.P) v = *reinterpret_cast<const float4*>(p.S + (r0 + r) * N + col);
    const float am = seg_allmax<TPR>(amax4(v));
    if (r >= p.P) continue;
    float sc, inv;
    if (p.ckpt == kCkptFp4) {
      e2m1_row_scale(am, sc, inv);
      *reinterpret_cast<unsigned short*>(p.codes + (r0 + r) * (N / 2) + col / 2) =
          static_cast<unsigned short>(quant4_e2m1(v, inv));
    } else {
      e4m3_row_scale(am, sc, inv);
      *reinterpret_cast<uint32_t*>(p.codes + (r0 + r) * N + col) = quant4_e4m3(v, inv);
    }
    if (col == 0) p.scale[r0 + r] = sc;
  }
}

cudaError_t launch_resume_mask(const Packed& pk, uint8_t* mask, cudaStream_t s) {
  const MaskParams p{pk, mask};
  return pdl_launch(resume_mask_kernel, dim3((pk.batch + 255) / 256), 256, 0, s, p);
}

cudaError_t launch_refresh_copy(const Packed& pk, int H, int P, int N, int ckpt, const float* S, uint8_t* codes,
                                float* scale, cudaStream_t s) {
  const RefreshParams p{pk, H, P, ckpt, S, codes, scale};
  const dim3 grid((unsigned)((int64_t)pk.n_seqs * H));
  switch (N) {
    case 16: return pdl_launch(refresh_copy_kernel<16>, grid, 256, 0, s, p);
    case 32: return pdl_launch(refresh_copy_kernel<32>, grid, 256, 0, s, p);
    case 64: return pdl_launch(refresh_copy_kernel<64>, grid, 256, 0, s, p);
    case 128: return pdl_launch(refresh_copy_kernel<128>, grid, 256, 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace replay
