// Launch parameters of the operators around the decode step (the layer's inputs, the scan
// of prompts, the gated norm), shared by the host entry points and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace replay {

// Packed sequences: sequence s holds tokens [cu[s], cu[s + 1]) and owns row seqs[s] of the
// caller's state (row s where seqs is null).
struct Packed {
  const int32_t* cu;      // [n_seqs + 1]
  const int32_t* seqs;    // [n_seqs] or null
  const uint8_t* resume;  // [n_seqs] or null: 1 = continue from the state, 0 = from zero
  int32_t n_seqs, batch;  // batch: rows of the state
  int64_t tokens;
  int32_t* status;        // device error word or null
};

// The layer's inputs: convolution, SiLU, split, step sizes and decays.
struct InputsParams {
  Packed pk;  // token form: cu and resume are null, n_seqs rows of one token each
  int32_t H, G, P, N, D, width;
  int32_t tile;     // prompts: tokens of a block; token form: rows of a block
  int32_t col_blocks;  // blocks of a tile: its channels', and one for the step sizes
  const void* x;    // [tokens] rows of D channels (v | k | q), ldx elements apart
  const void* raw;  // [tokens] rows of H raw step sizes, ldr elements apart
  int64_t ldx, ldr;
  const float *w, *bias, *dt_bias, *A;  // [width][D], [D] or null, [H] or null, [H]
  void* conv;                           // [batch][width - 1][D]: each row's last raw inputs, oldest first
  void *q, *k, *v;                      // [tokens][G][N], [tokens][G][N], [tokens][H][P]; token form: k, v may be null
  float *dt, *a;                        // [tokens][H]; token form: may be null
  // token form into a decode layer: each row's entry goes to its next ring record
  uint8_t *ring, *ring_k;
  const int32_t* counts;
  int32_t L, cap, rec_bytes, rec_k_bytes;
};

// The scan of packed prompts.
struct ScanParams {
  Packed pk;
  int32_t H, G, P, N;
  const void *q, *k, *v;
  const float *dt, *a;
  void* y;
  float* S;         // [batch][H][P][N]
  int32_t* counts;  // a decode layer's pointer words (set empty for the served rows), or null
  // long sequences in segments of seg_tokens (0: whole): [segment][head][block of 64 rows p]
  // states of 64 x N floats, each segment's own and then the one it starts from, and decays
  int32_t seg_tokens, max_segs;
  float *seg_state, *seg_decay;
};

// How the tensor-core scan splits its work: tokens of a segment (0 = sequences whole) and the
// most segments there can be.
struct ScanSplit {
  int32_t seg_tokens, max_segs;
};
ScanSplit scan_split(int64_t tokens, int32_t n_seqs, int64_t max_len, int H, int P);

struct NormParams {
  int64_t rows;
  int32_t H, P, groups;
  const void* y;  // [rows][H * P], FP32 or io
  const void* z;  // rows of H * P, ldz elements apart
  int64_t ldz;
  const void* v;  // [rows][H * P] io, or null (no skip term)
  const float *D, *weight;
  float eps;
  void* out;  // [rows][H * P] io
  uint32_t head_magic;  // 2^32 / (P / 8) rounded up: the head of column c is (c / 8) head_magic / 2^32
};

// io: 0 = FP32, 1 = BF16
cudaError_t launch_prompt_inputs(const InputsParams& p, int io, int num_sms, cudaStream_t s);
cudaError_t launch_token_inputs(const InputsParams& p, int io, int num_sms, cudaStream_t s);
cudaError_t launch_scan_serial(const ScanParams& p, int io, cudaStream_t s);
cudaError_t launch_scan_tc(const ScanParams& p, int num_sms, cudaStream_t s);  // BF16, tokens > 0
// a decode layer's prefill: mask[b] = 1 where a sequence resumes row b; the read copy of
// the served rows requantised from their checkpoints
cudaError_t launch_resume_mask(const Packed& pk, uint8_t* mask, cudaStream_t s);
cudaError_t launch_refresh_copy(const Packed& pk, int H, int P, int N, int ckpt, const float* S, uint8_t* codes,
                                float* scale, cudaStream_t s);
cudaError_t launch_gated_norm(const NormParams& p, int io, int y_io, int num_sms, cudaStream_t s);

}  // namespace replay
