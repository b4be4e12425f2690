// Host side of the operators around the decode step (include/replay.h): argument checks
// and launches on the caller's stream. No device memory is allocated.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/replay.h"
#include "layer_params.h"
#include "replay_ctx.h"

using replay::aligned;
using replay::InputsParams;
using replay::NormParams;
using replay::Packed;
using replay::ScanParams;

namespace {

constexpr int kMaxWidth = 4;
constexpr int64_t kMaxTokens = INT32_MAX;  // cu_seqlens is int32

inline int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }
inline cudaStream_t stream_of(replay_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline int io_bytes(const replay_config& c) { return c.io == REPLAY_BF16 ? 2 : 4; }
inline int launched(cudaError_t e) { return e == cudaSuccess ? REPLAY_OK : REPLAY_ECUDA; }

// SMs of the current device, asked for once per device.
int sm_count(int* out) {
  static std::mutex mu;
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return REPLAY_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= 64) return cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? REPLAY_OK : REPLAY_ECUDA;
  if (!known[dev] && cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return REPLAY_ECUDA;
  *out = known[dev];
  return REPLAY_OK;
}

int packed(Packed* pk, const replay_config& c, int64_t tokens, const int32_t* cu, const int32_t* seqs,
           const uint8_t* resume, int32_t n_seqs, int32_t* status) {
  if (tokens < 0 || tokens > kMaxTokens || n_seqs < 0) return REPLAY_EINVAL;
  if (n_seqs > 0 && !cu) return REPLAY_EINVAL;
  if (!seqs && n_seqs > c.batch) return REPLAY_EINVAL;
  if (!aligned(cu, 4) || !aligned(seqs, 4) || !aligned(status, 4)) return REPLAY_EALIGN;
  *pk = Packed{cu, seqs, resume, n_seqs, c.batch, tokens, status};
  return REPLAY_OK;
}

// Checks and parameters that the three forms of the layer's inputs share.
int inputs_params(InputsParams* p, const replay_config& c, int32_t width, int64_t rows, const void* x, int64_t ldx,
                  const void* raw, int64_t ldr, const float* w, const float* bias, const float* dt_bias,
                  const float* A, void* conv) {
  if (width < 2 || width > kMaxWidth) return REPLAY_EINVAL;
  const int64_t D = (int64_t)c.heads * c.P + 2 * (int64_t)c.groups * c.N;
  if (D > INT32_MAX / 8) return REPLAY_EINVAL;
  if ((rows / 8 + 1) * (D / 512 + 2) > INT32_MAX) return REPLAY_EINVAL;  // blocks of one launch
  if (!w || !A || !conv || (rows > 0 && (!x || !raw))) return REPLAY_EINVAL;
  if (ldx < D || ldr < c.heads) return REPLAY_EINVAL;
  const int s = io_bytes(c);
  if (!aligned(x, 16) || (ldx * s) % 16 || !aligned(conv, 16) || !aligned(raw, s)) return REPLAY_EALIGN;
  if (!aligned(w, 16) || !aligned(bias, 16) || !aligned(dt_bias, 4) || !aligned(A, 4)) return REPLAY_EALIGN;
  *p = InputsParams{};
  p->H = c.heads, p->G = c.groups, p->P = c.P, p->N = c.N, p->D = (int32_t)D, p->width = width;
  p->x = x, p->ldx = ldx, p->raw = raw, p->ldr = ldr;
  p->w = w, p->bias = bias, p->dt_bias = dt_bias, p->A = A, p->conv = conv;
  return REPLAY_OK;
}

int scan_params(ScanParams* p, const replay_config& c, int64_t tokens, const void* q, const void* k, const void* v,
                const float* dt, const float* a, float* S, void* y) {
  if ((int64_t)p->pk.n_seqs * c.heads > INT32_MAX / 4) return REPLAY_EINVAL;  // blocks of one launch
  if (!S || (tokens > 0 && (!q || !k || !v || !dt || !a || !y))) return REPLAY_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(y, 16) || !aligned(S, 16))
    return REPLAY_EALIGN;
  if (!aligned(dt, 4) || !aligned(a, 4)) return REPLAY_EALIGN;
  p->H = c.heads, p->G = c.groups, p->P = c.P, p->N = c.N;
  p->q = q, p->k = k, p->v = v, p->dt = dt, p->a = a, p->S = S, p->y = y;
  p->counts = nullptr;
  p->seg_tokens = p->max_segs = 0;
  p->seg_state = p->seg_decay = nullptr;
  return REPLAY_OK;
}

int check_scratch(const void* scratch, int64_t have, int64_t need) {
  if (need > 0 && (!scratch || have < need)) return REPLAY_EINVAL;
  return aligned(scratch, 256) ? REPLAY_OK : REPLAY_EALIGN;
}

// The serial kernel takes FP32 inputs, and BF16 sequences of few tokens, where the tensor
// cores' chunks of 128 are mostly empty: a chunk of one head takes an SM about 6 us with its
// state, a token of the serial kernel 0.27 us in each of a few blocks an SM. 256 sequences of
// the 64-head layer of 64 x 128: 16 tokens each 380 against 672 us, 24 tokens 526 against 668,
// 32 tokens 689 against 673; of 32 heads of 128 x 128 the same within 3 %. The rule is N = 128's:
// at N = 64 (8 heads of 64 x 64) the serial kernel still leads at 40 tokens, 58 against 90 us.
bool on_tensor_cores(const replay_config& c, int64_t tokens, int32_t n_seqs, int64_t max_len) {
  if (c.io != REPLAY_BF16 || tokens == 0) return false;
  constexpr int64_t kFew = 30;
  if (tokens > kFew * n_seqs) return true;
  const int64_t longest = max_len > 0 && max_len < tokens ? max_len : tokens;
  const int64_t units = (int64_t)n_seqs * c.heads * ((c.P + 63) / 64);
  return longest > kFew && longest * 148 > kFew * units;  // one of them is long, and the others hide it not
}
int64_t segment_units(const replay_config& c, const replay::ScanSplit& sp) {
  return (int64_t)sp.max_segs * c.heads * ((c.P + 63) / 64);
}
// The scratch of one scan: the segments' states, then their decays.
int64_t scan_scratch(const replay_config& c, int64_t tokens, int32_t n_seqs, int64_t max_len) {
  if (!on_tensor_cores(c, tokens, n_seqs, max_len)) return 0;
  const replay::ScanSplit sp = replay::scan_split(tokens, n_seqs, max_len, c.heads, c.P);
  const int64_t units = sp.seg_tokens ? segment_units(c, sp) : 0;
  return round256(units * 64 * c.N * 4) + round256(units * 4);
}

int launch_scan(ScanParams& p, const replay_config& c, int64_t max_len, void* scratch, cudaStream_t s) {
  if (!on_tensor_cores(c, p.pk.tokens, p.pk.n_seqs, max_len)) return launched(replay::launch_scan_serial(p, c.io, s));
  const replay::ScanSplit sp = replay::scan_split(p.pk.tokens, p.pk.n_seqs, max_len, c.heads, c.P);
  p.seg_tokens = sp.seg_tokens, p.max_segs = sp.max_segs;
  p.seg_state = static_cast<float*>(scratch);
  p.seg_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + round256(segment_units(c, sp) * 64 * c.N * 4));
  int sms, rc;
  if ((rc = sm_count(&sms))) return rc;
  return launched(replay::launch_scan_tc(p, sms, s));
}

}  // namespace

extern "C" {

int replay_prompt_inputs(const replay_config* cfg, int32_t width, int64_t tokens, const void* x, int64_t ldx,
                         const void* raw, int64_t ldr, const float* w, const float* bias, const float* dt_bias,
                         const float* A, const int32_t* cu_seqlens, const int32_t* seqs, const uint8_t* resume,
                         int32_t n_seqs, void* conv, void* q, void* k, void* v, float* dt, float* a,
                         int32_t* status, replay_stream_t stream) {
  int rc = replay::validate_config(cfg, false);
  if (rc) return rc;
  Packed pk;
  if ((rc = packed(&pk, *cfg, tokens, cu_seqlens, seqs, resume, n_seqs, status))) return rc;
  InputsParams p;
  if ((rc = inputs_params(&p, *cfg, width, tokens, x, ldx, raw, ldr, w, bias, dt_bias, A, conv))) return rc;
  if (tokens > 0 && (!q || !k || !v || !dt || !a)) return REPLAY_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dt, 4) || !aligned(a, 4)) return REPLAY_EALIGN;
  p.pk = pk;
  p.q = q, p.k = k, p.v = v, p.dt = dt, p.a = a;
  if (n_seqs == 0) return REPLAY_OK;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  return launched(replay::launch_prompt_inputs(p, cfg->io, sms, stream_of(stream)));
}

int replay_token_inputs(const replay_config* cfg, int32_t width, int32_t n, const void* x, int64_t ldx,
                        const void* raw, int64_t ldr, const float* w, const float* bias, const float* dt_bias,
                        const float* A, const int32_t* seqs, void* conv, void* q, void* k, void* v, float* dt,
                        float* a, int32_t* status, replay_stream_t stream) {
  int rc = replay::validate_config(cfg, false);
  if (rc) return rc;
  if (n < 0 || (!seqs && n > cfg->batch)) return REPLAY_EINVAL;
  InputsParams p;
  if ((rc = inputs_params(&p, *cfg, width, n, x, ldx, raw, ldr, w, bias, dt_bias, A, conv))) return rc;
  if (n > 0 && (!q || !k || !v || !dt || !a)) return REPLAY_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dt, 4) || !aligned(a, 4)) return REPLAY_EALIGN;
  if (!aligned(seqs, 4) || !aligned(status, 4)) return REPLAY_EALIGN;
  p.pk = Packed{nullptr, seqs, nullptr, n, cfg->batch, n, status};
  p.q = q, p.k = k, p.v = v, p.dt = dt, p.a = a;
  if (n == 0) return REPLAY_OK;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  return launched(replay::launch_token_inputs(p, cfg->io, sms, stream_of(stream)));
}

int replay_append_inputs(replay_ctx* ctx, int32_t width, const void* x, int64_t ldx, const void* raw, int64_t ldr,
                         const float* w, const float* bias, const float* dt_bias, const float* A, void* conv,
                         void* q, void* v, replay_stream_t stream) {
  if (!ctx) return REPLAY_EINVAL;
  if (ctx->pending) return REPLAY_EPENDING;
  const replay_config& c = ctx->cfg;
  InputsParams p;
  const int rc = inputs_params(&p, c, width, c.batch, x, ldx, raw, ldr, w, bias, dt_bias, A, conv);
  if (rc) return rc;
  if (!q) return REPLAY_EINVAL;
  if (!aligned(q, 16) || !aligned(v, 16)) return REPLAY_EALIGN;
  p.pk = Packed{nullptr, nullptr, nullptr, c.batch, c.batch, c.batch, ctx->bufs.status};
  p.q = q, p.v = v;
  p.ring = static_cast<uint8_t*>(ctx->bufs.ring), p.ring_k = static_cast<uint8_t*>(ctx->bufs.ring_k);
  p.counts = ctx->bufs.counts + (size_t)ctx->parity * c.batch;
  p.L = c.L, p.cap = ctx->cap;
  p.rec_bytes = replay::record_bytes(c), p.rec_k_bytes = replay::record_k_bytes(c);
  return launched(replay::launch_token_inputs(p, c.io, ctx->num_sms, stream_of(stream)));
}

int64_t replay_prompt_scan_scratch(const replay_config* cfg, int64_t tokens, int32_t n_seqs, int64_t max_len) {
  const int rc = replay::validate_config(cfg, false);
  if (rc) return rc;
  if (tokens < 0 || tokens > kMaxTokens || n_seqs < 0 || max_len < 0) return REPLAY_EINVAL;
  if ((int64_t)n_seqs * cfg->heads > INT32_MAX / 4) return REPLAY_EINVAL;
  return scan_scratch(*cfg, tokens, n_seqs, max_len);
}

int replay_prompt_scan(const replay_config* cfg, int64_t tokens, const void* q, const void* k, const void* v,
                       const float* dt, const float* a, const int32_t* cu_seqlens, const int32_t* seqs,
                       const uint8_t* resume, int32_t n_seqs, int64_t max_len, float* S, void* y, void* scratch,
                       int64_t scratch_bytes, int32_t* status, replay_stream_t stream) {
  int rc = replay::validate_config(cfg, false);
  if (rc) return rc;
  ScanParams p;
  if ((rc = packed(&p.pk, *cfg, tokens, cu_seqlens, seqs, resume, n_seqs, status))) return rc;
  if ((rc = scan_params(&p, *cfg, tokens, q, k, v, dt, a, S, y))) return rc;
  const int64_t need = replay_prompt_scan_scratch(cfg, tokens, n_seqs, max_len);
  if (need < 0) return (int)need;
  if ((rc = check_scratch(scratch, scratch_bytes, need))) return rc;
  if (n_seqs == 0) return REPLAY_OK;
  return launch_scan(p, *cfg, max_len, scratch, stream_of(stream));
}

int64_t replay_prefill_scratch(const replay_ctx* ctx, int64_t tokens, int32_t n_seqs, int64_t max_len) {
  if (!ctx) return REPLAY_EINVAL;
  const int64_t n = replay_prompt_scan_scratch(&ctx->cfg, tokens, n_seqs, max_len);
  return n < 0 ? n : round256(ctx->cfg.batch) + n;
}

int replay_prefill(replay_ctx* ctx, int64_t tokens, const void* q, const void* k, const void* v, const float* dt,
                   const float* a, const int32_t* cu_seqlens, const int32_t* seqs, const uint8_t* resume,
                   int32_t n_seqs, int64_t max_len, void* y, void* scratch, int64_t scratch_bytes,
                   replay_stream_t stream) {
  if (!ctx) return REPLAY_EINVAL;
  if (ctx->pending) return REPLAY_EPENDING;
  const replay_config& c = ctx->cfg;
  cudaStream_t s = stream_of(stream);
  ScanParams p;
  int rc = packed(&p.pk, c, tokens, cu_seqlens, seqs, resume, n_seqs, ctx->bufs.status);
  if (rc) return rc;
  if ((rc = scan_params(&p, c, tokens, q, k, v, dt, a, ctx->bufs.S0, y))) return rc;
  const int64_t need = replay_prefill_scratch(ctx, tokens, n_seqs, max_len);
  if (need < 0) return (int)need;
  if ((rc = check_scratch(scratch, scratch_bytes, need))) return rc;
  if (n_seqs == 0) return REPLAY_OK;
  if (resume) {  // the resumed sequences' buffered entries into their checkpoints
    uint8_t* mask = static_cast<uint8_t*>(scratch);
    if (replay::launch_resume_mask(p.pk, mask, s) != cudaSuccess) return REPLAY_ECUDA;
    if ((rc = replay_flush(ctx, mask, stream))) return rc;
  }
  p.counts = ctx->bufs.counts + (size_t)ctx->parity * c.batch;
  if ((rc = launch_scan(p, c, max_len, static_cast<uint8_t*>(scratch) + round256(c.batch), s))) return rc;
  if (c.ckpt != REPLAY_CKPT_F32)
    return launched(replay::launch_refresh_copy(p.pk, c.heads, c.P, c.N, replay::ckpt_kind(c.ckpt), ctx->bufs.S0,
                                                ctx->bufs.S0_codes, ctx->bufs.S0_scale, s));
  return REPLAY_OK;
}

int replay_gated_norm(const replay_config* cfg, int64_t rows, const void* y, int32_t y_type, const void* z,
                      int64_t ldz, const void* v, const float* D, const float* weight, int32_t norm_groups,
                      float eps, void* out, replay_stream_t stream) {
  int rc = replay::validate_config(cfg, false);
  if (rc) return rc;
  const int64_t width = (int64_t)cfg->heads * cfg->P;
  if (rows < 0 || width > INT32_MAX || norm_groups < 1 || width % norm_groups || (width / norm_groups) % 8)
    return REPLAY_EINVAL;
  if (width / 8 * (cfg->P / 8) >= INT32_MAX || rows > INT32_MAX / norm_groups) return REPLAY_EINVAL;
  if (y_type != REPLAY_F32 && y_type != cfg->io) return REPLAY_EINVAL;
  if (!weight || ldz < width || !(eps >= 0.f)) return REPLAY_EINVAL;
  if (rows > 0 && (!y || !z || !out || (!v) != (!D))) return REPLAY_EINVAL;  // no rows: their pointers may be null
  if (!aligned(y, 16) || !aligned(z, 16) || (ldz * io_bytes(*cfg)) % 16 || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(D, 4) || !aligned(weight, 16))
    return REPLAY_EALIGN;
  if (rows == 0) return REPLAY_OK;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  NormParams p{rows, cfg->heads, cfg->P, norm_groups, y, z, ldz, v, D, weight, eps, out, 0u};
  return launched(replay::launch_gated_norm(p, cfg->io, y_type, sms, stream_of(stream)));
}

}  // extern "C"
