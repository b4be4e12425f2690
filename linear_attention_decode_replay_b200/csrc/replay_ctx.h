// The host context and the checks that the C ABI's entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/replay.h"
#include "replay_device.cuh"
#include "replay_kparams.h"

struct replay_ctx {
  replay_config cfg;
  replay_buffers bufs;
  int cap;
  int parity;   // which half of counts holds the current pointer words
  int pending;  // n_pos of an unresolved verify, 0 if none
  int device;
  int num_sms;
  replay::KParams kp_step, kp_verify, kp_flush;  // prebuilt launch layouts (pointers filled per call)
  int verify_ok;                          // kp_verify was built (max_pos > 1)
  int smem_optin;                         // the device's per-block shared-memory limit
  replay::KParams kp_static[replay::kMaxPos + 1]; // replay_verify_static_scratch layouts, by n_pos
  int kp_static_ok[replay::kMaxPos + 1];  // ... built on first use
};

namespace replay {

inline int round_up(int x, int m) { return (x + m - 1) / m * m; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int validate_config(const replay_config* c, bool needs_window) {
  if (!c) return REPLAY_EINVAL;
  if (c->batch < 1 || c->heads < 1 || c->groups < 1 || c->heads % c->groups) return REPLAY_EINVAL;
  if (c->P < 8 || c->P > 256 || c->P % 8) return REPLAY_EINVAL;
  if (c->N != 16 && c->N != 32 && c->N != 64 && c->N != 128) return REPLAY_EINVAL;
  if ((int64_t)c->P * c->N * 4 > 65536) return REPLAY_EINVAL;
  if (c->io != REPLAY_F32 && c->io != REPLAY_BF16) return REPLAY_EINVAL;
  if ((int64_t)c->batch * c->heads > INT32_MAX / 2) return REPLAY_EINVAL;
  if (needs_window) {
    if (c->L < 1 || c->L > kMaxWindow) return REPLAY_EINVAL;
    if (c->max_pos < 1 || c->max_pos > kMaxPos || c->max_pos > c->L) return REPLAY_EINVAL;
    if (c->ckpt != REPLAY_CKPT_F32 && c->ckpt != REPLAY_CKPT_F32_FP8READ && c->ckpt != REPLAY_CKPT_F32_FP4READ)
      return REPLAY_EINVAL;
  }
  return REPLAY_OK;
}

inline int ring_capacity(const replay_config& c) { return c.L + c.max_pos; }
// head record: v (P io values), Delta, a; k record: k (N io values)
inline int record_bytes(const replay_config& c) {
  const int s_io = c.io == REPLAY_BF16 ? 2 : 4;
  return round_up(c.P * s_io + 8, 16);
}
// k record: k (N io values), then 16 bytes of padding. The padding staggers consecutive
// records by four shared-memory banks once a unit's records sit in a stage, so that the
// lanes that read several entries' k at once (one entry per lane pair or quarter) spread
// over all 32 banks; without it every record starts on the same bank.
inline int record_k_bytes(const replay_config& c) { return c.N * (c.io == REPLAY_BF16 ? 2 : 4) + 16; }
inline int ckpt_kind(int ckpt) {
  return ckpt == REPLAY_CKPT_F32_FP8READ ? kCkptFp8 : ckpt == REPLAY_CKPT_F32_FP4READ ? kCkptFp4
                                                                                              : kCkptF32;
}

struct DeviceInfo {
  int device, num_sms, smem_optin;
};

inline int device_info(DeviceInfo* d) {
  if (cudaGetDevice(&d->device) != cudaSuccess) return REPLAY_ECUDA;
  if (cudaDeviceGetAttribute(&d->num_sms, cudaDevAttrMultiProcessorCount, d->device) != cudaSuccess)
    return REPLAY_ECUDA;
  if (cudaDeviceGetAttribute(&d->smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d->device) != cudaSuccess)
    return REPLAY_ECUDA;
  return REPLAY_OK;
}

}  // namespace replay
