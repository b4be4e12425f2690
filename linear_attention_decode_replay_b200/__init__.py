"""ReplaySSM decode path for scalar-decay (Mamba-2-style) SSM layers on B200.

A thin Python binding over the C ABI of ``include/replay.h`` (``libreplay.so``): every
step of the path runs in the library's CUDA kernels; this module only checks tensor
shapes and dtypes and passes device pointers and the current CUDA stream. PyTorch
provides device memory and streams.

    cfg = Config(batch=256, heads=64, groups=64, P=64, N=128, L=16)
    bufs = alloc_buffers(cfg, "cuda")          # caller-owned device buffers
    bufs["S0"].copy_(initial_checkpoint)
    r = Replay(cfg, bufs)
    y = r.step(q, k, v, dt, a)                 # one decode token per sequence
    y = r.verify(q5, k5, v5, dt5, a5)          # 5 speculative positions, output-only
    r.rollback(n_keep)                         # keep n_keep[b] of them (pointer move)
    r.flush()                                  # fold every buffer into the checkpoint

Around the step, from the rows of a layer's projection (gate | v k q channels | step
sizes) to the rows of its output projection:

    x, raw, z = proj[:, HP:HP + D], proj[:, HP + D:], proj[:, :HP]
    q, k, v, dt, a = prompt_inputs(cfg, conv, x, raw, w, A, cu_seqlens)  # prompts, packed
    y = r.prefill(q, k, v, dt, a, cu_seqlens)  # their outputs; their states into the layer
    o = gated_norm(cfg, y, z, weight, v=v, D=D_skip)
    q, v = r.append_inputs(conv, x1, raw1, w, A)  # one token: its entry into the ring
    o = gated_norm(cfg, r.step_resident(q), z1, weight, v=v, D=D_skip)

Small batches are bound by the host's launch rate; an even number of ``step`` calls on
fixed input and output tensors can be captured in a CUDA graph once one call has run
outside the capture (the conditions are in ``include/replay.h``). Each call flips which
half of the pointer words is current, so capture two windows when L is odd:

    r.step(q[0], k[0], v[0], dt[0], a[0], y=y[0])   # one call outside the capture
    n = cfg.L if cfg.L % 2 == 0 else 2 * cfg.L      # an even number of calls
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t in range(n):
            r.step(q[t % cfg.L], k[t % cfg.L], v[t % cfg.L], dt[t % cfg.L], a[t % cfg.L], y=y[t % cfg.L])
    g.replay()                                       # n decode steps, one graph launch
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _abi
from ._abi import (  # noqa: F401
    DEV_POINTER,
    DEV_ROLLBACK,
    DEV_SEQS,
    DEV_SNAPSHOT,
    DEV_WAIT_TIMEOUT,
    ReplayError,
    check,
    load,
    strerror,
)

__all__ = ["Config", "Replay", "alloc_buffers", "ring_capacity", "ring_record_bytes", "ring_k_record_bytes",
           "code_shape", "snapshot_bytes", "eager_step", "eager_step_fp8", "quantize_rows_e4m3", "quantize_rows_e2m1",
           "prompt_inputs", "token_inputs", "prompt_scan", "gated_norm", "ReplayError", "load", "strerror"]


_CKPT = {"f32": _abi.REPLAY_CKPT_F32, "f32_fp8read": _abi.REPLAY_CKPT_F32_FP8READ,
         "f32_fp4read": _abi.REPLAY_CKPT_F32_FP4READ}


class _Kept:
    __slots__ = ("_kept",)  # what a Config works out once: in a slot, it is no part of vars() or of pickles


@dataclass(frozen=True)
class Config(_Kept):
    """Sizes of one decode layer (see replay_config in include/replay.h)."""

    batch: int
    heads: int
    groups: int
    P: int
    N: int
    L: int
    max_pos: int = 1
    io: str = "bf16"  # "bf16" or "f32": dtype of q, k, v
    ckpt: str = "f32"  # "f32", "f32_fp8read" or "f32_fp4read"

    def c(self) -> _abi.CConfig:
        return _abi.CConfig(self.batch, self.heads, self.groups, self.P, self.N, self.L, self.max_pos,
                            _abi.REPLAY_BF16 if self.io == "bf16" else _abi.REPLAY_F32,
                            _CKPT[self.ckpt])

    @property
    def io_dtype(self) -> torch.dtype:
        return torch.bfloat16 if self.io == "bf16" else torch.float32

    def __getstate__(self):
        return dict(vars(self))  # the fields: pickled and copied as before any use

    @property
    def _layer(self):
        """What the calls around the step need of it: the C config by reference, the io
        dtype, the channels and the shapes of one token's q (k), v and dt (a)."""
        try:
            return self._kept
        except AttributeError:
            H, G, P, N = self.heads, self.groups, self.P, self.N
            kept = ctypes.byref(self.c()), self.io_dtype, H * P + 2 * G * N, (G, N), (H, P), (H,)
            object.__setattr__(self, "_kept", kept)
            return kept


def ring_capacity(cfg: Config) -> int:
    cap = load().replay_ring_capacity(ctypes.byref(cfg.c()))
    if cap < 0:
        raise ReplayError(cap, "replay_ring_capacity")
    return cap


def ring_record_bytes(cfg: Config) -> int:
    """Bytes of one head record of the ring (v, Delta, a)."""
    r = load().replay_ring_record_bytes(ctypes.byref(cfg.c()))
    if r < 0:
        raise ReplayError(r, "replay_ring_record_bytes")
    return r


def ring_k_record_bytes(cfg: Config) -> int:
    """Bytes of one k record of the ring (one per k/q group)."""
    r = load().replay_ring_k_record_bytes(ctypes.byref(cfg.c()))
    if r < 0:
        raise ReplayError(r, "replay_ring_k_record_bytes")
    return r


def code_shape(cfg: Config):
    """Shape of the read copy's codes (uint8): FP8 one byte per value, FP4 two values per byte."""
    n = cfg.N // 2 if cfg.ckpt == "f32_fp4read" else cfg.N
    return (cfg.batch, cfg.heads, cfg.P, n)


def snapshot_bytes(cfg: Config) -> int:
    """Bytes of one sequence's snapshot (replay_export / replay_import)."""
    r = load().replay_snapshot_bytes(ctypes.byref(cfg.c()))
    if r < 0:
        raise ReplayError(r, "replay_snapshot_bytes")
    return r


def alloc_buffers(cfg: Config, device="cuda") -> dict:
    """Allocates the caller-owned device buffers of one layer (S0 left uninitialised)."""
    cap = ring_capacity(cfg)
    rec = ring_record_bytes(cfg)
    rk = ring_k_record_bytes(cfg)
    B, H, G, P, N = cfg.batch, cfg.heads, cfg.groups, cfg.P, cfg.N
    bufs = {
        "S0": torch.empty(B, H, P, N, device=device, dtype=torch.float32),
        "ring_k": torch.zeros(B, G, cap, rk, device=device, dtype=torch.uint8),
        "ring": torch.zeros(B, H, cap, rec, device=device, dtype=torch.uint8),
        "counts": torch.zeros(2, B, device=device, dtype=torch.int32),
        "status": torch.zeros(1, device=device, dtype=torch.int32),
    }
    if cfg.max_pos > 1:
        bufs["qpack"] = torch.empty(B, G, cfg.max_pos, N, device=device, dtype=cfg.io_dtype)
    if cfg.ckpt != "f32":
        bufs["S0_codes"] = torch.empty(code_shape(cfg), device=device, dtype=torch.uint8)
        bufs["S0_scale"] = torch.empty(B, H, P, device=device, dtype=torch.float32)
    return bufs


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t, shape=None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


# The calls around the step are short beside what Python spends on their arguments, so their
# checks are one expression a tensor, and say what is wrong only where something is.
def _arg(t, shape, dtype, name, dev):
    """Address of a dense tensor of this shape and dtype on CUDA device `dev` (None: none)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _ptr(t, shape, dtype, name)
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _rows(t, n, width, dtype, name, dev):
    """Address and row stride (elements) of a 2-D tensor whose rows may lie apart."""
    try:
        if t.dtype is dtype and t.shape == (n, width) and t.get_device() == dev:
            row, col = t.stride()
            if col == 1 or width == 1:  # the stride of a single row says nothing
                return t.data_ptr(), row if n > 1 else (width + 7) // 8 * 8
            raise ValueError(f"{name} must have contiguous rows")
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {(n, width)}, got {tuple(t.shape)}")


def _device_of(t, name):
    """Index of the CUDA device that a call's tensors must be on: its first tensor's."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


# The current device and a device's current stream, by torch's short forms, or, where a torch
# has none, by its public calls.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(dev, stream, body):
    """body(raw stream) with device `dev` current and `stream` (None: its current one) the
    stream of the allocations in it, so that none is handed to another stream's work early."""
    if stream is None and _current_device() == dev:
        return body(_raw_stream(dev))
    with torch.cuda.device(dev):
        if stream is None:
            return body(_raw_stream(dev))
        with torch.cuda.stream(stream):
            return body(stream.cuda_stream)


def _width(cfg, w):
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError(f"w must be a tensor of shape (width, {cfg._layer[2]})")
    return w.shape[0]


def _filter_args(cfg, conv, w, A, bias, dt_bias, dev):
    """width, and the addresses of w, bias, dt_bias, A and conv."""
    _, t, D, _, _, hs = cfg._layer
    width, f32 = _width(cfg, w), torch.float32
    return (width, _arg(w, (width, D), f32, "w", dev), _arg(bias, (D,), f32, "bias", dev),
            _arg(dt_bias, hs, f32, "dt_bias", dev), _arg(A, hs, f32, "A", dev),
            _arg(conv, (cfg.batch, width - 1, D), t, "conv", dev))


def _n_seqs(cu_seqlens):
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor of n_seqs + 1 offsets")
    return cu_seqlens.shape[0] - 1


def _packed_args(cu_seqlens, seqs, resume, dev):
    """n_seqs, and the addresses of cu_seqlens, seqs and resume."""
    n = _n_seqs(cu_seqlens)
    return (n, _arg(cu_seqlens, (n + 1,), torch.int32, "cu_seqlens", dev), _arg(seqs, (n,), torch.int32, "seqs", dev),
            _arg(resume, (n,), torch.uint8, "resume", dev))


def _input_outs(cfg, n, like, out, dev):
    """q, k, v, dt, a of n tokens, `out` checked or new tensors, and their addresses."""
    _, t, _, qs, vs, hs = cfg._layer
    if out is None:
        q, v, dt = like.new_empty((n, *qs)), like.new_empty((n, *vs)), like.new_empty((n, *hs), dtype=torch.float32)
        k, a = torch.empty_like(q), torch.empty_like(dt)
        return (q, k, v, dt, a), (q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), a.data_ptr())
    q, k, v, dt, a = out
    f32 = torch.float32
    return out, (_arg(q, (n, *qs), t, "q", dev), _arg(k, (n, *qs), t, "k", dev), _arg(v, (n, *vs), t, "v", dev),
                 _arg(dt, (n, *hs), f32, "dt", dev), _arg(a, (n, *hs), f32, "a", dev))


class Replay:
    """One decode layer's checkpoint + buffer state, over caller-owned device buffers."""

    def __init__(self, cfg: Config, buffers: dict, stream=None):
        self.cfg = cfg
        self.buffers = buffers
        lib = load()
        B, H, G, P, N = cfg.batch, cfg.heads, cfg.groups, cfg.P, cfg.N
        cap = ring_capacity(cfg)
        copy = cfg.ckpt != "f32"
        rec = ring_record_bytes(cfg)
        rk = ring_k_record_bytes(cfg)
        cb = _abi.CBuffers(
            _ptr(buffers["S0"], (B, H, P, N), torch.float32, "S0"),
            _ptr(buffers.get("S0_codes"), code_shape(cfg), torch.uint8, "S0_codes") if copy else None,
            _ptr(buffers.get("S0_scale"), (B, H, P), torch.float32, "S0_scale") if copy else None,
            _ptr(buffers["ring_k"], (B, G, cap, rk), torch.uint8, "ring_k"),
            _ptr(buffers["ring"], (B, H, cap, rec), torch.uint8, "ring"),
            _ptr(buffers.get("qpack"), (B, G, cfg.max_pos, N), cfg.io_dtype, "qpack") if cfg.max_pos > 1 else None,
            _ptr(buffers["counts"], (2, B), torch.int32, "counts"),
            _ptr(buffers["status"], (1,), torch.int32, "status"),
        )
        self._ctx = ctypes.c_void_p()
        check(lib.replay_init(ctypes.byref(cfg.c()), ctypes.byref(cb), _stream(stream),
                              ctypes.byref(self._ctx)), "replay_init")
        self._lib = lib

    def _token_shapes(self, n_pos):
        B, H, G, P, N = self.cfg.batch, self.cfg.heads, self.cfg.groups, self.cfg.P, self.cfg.N
        lead = (B,) if n_pos is None else (B, n_pos)
        return (*lead, G, N), (*lead, H, P), (*lead, H)

    def step(self, q, k, v, dt, a, y=None, flushed=None, stream=None):
        """One decode token per sequence; returns y [B][H][P] FP32."""
        qs, vs, ds = self._token_shapes(None)
        t = self.cfg.io_dtype
        if y is None:
            y = torch.empty(vs, device=q.device, dtype=torch.float32)
        check(self._lib.replay_step(self._ctx, _ptr(q, qs, t, "q"), _ptr(k, qs, t, "k"), _ptr(v, vs, t, "v"),
                                    _ptr(dt, ds, torch.float32, "dt"), _ptr(a, ds, torch.float32, "a"),
                                    _ptr(y, vs, torch.float32, "y"),
                                    _ptr(flushed, (self.cfg.batch,), torch.uint8, "flushed"), _stream(stream)),
              "replay_step")
        return y

    def verify(self, q, k, v, dt, a, y=None, flushed=None, stream=None):
        """Output-only scoring of n_pos = q.shape[1] positions; returns y [B][n_pos][H][P]."""
        n_pos = q.shape[1]
        qs, vs, ds = self._token_shapes(n_pos)
        t = self.cfg.io_dtype
        if y is None:
            y = torch.empty(vs, device=q.device, dtype=torch.float32)
        check(self._lib.replay_verify(self._ctx, n_pos, _ptr(q, qs, t, "q"), _ptr(k, qs, t, "k"),
                                      _ptr(v, vs, t, "v"), _ptr(dt, ds, torch.float32, "dt"),
                                      _ptr(a, ds, torch.float32, "a"), _ptr(y, vs, torch.float32, "y"),
                                      _ptr(flushed, (self.cfg.batch,), torch.uint8, "flushed"), _stream(stream)),
              "replay_verify")
        return y

    def verify_static_scratch(self, q, k, v, dt, a, y=None, flushed=None, stream=None):
        """verify() for callers that cannot allocate device memory: the queries are packed
        into the library's fixed 32 MiB device array instead of the qpack buffer, so the
        layer needs no qpack (max_pos = 1 works; n_pos above max_pos first folds the
        buffers too full to take the new entries). Calls that overlap on the GPU share
        that array and race. Pass `y` to keep this binding from allocating the output."""
        n_pos = q.shape[1]
        qs, vs, ds = self._token_shapes(n_pos)
        t = self.cfg.io_dtype
        if y is None:
            y = torch.empty(vs, device=q.device, dtype=torch.float32)
        check(self._lib.replay_verify_static_scratch(
            self._ctx, n_pos, _ptr(q, qs, t, "q"), _ptr(k, qs, t, "k"), _ptr(v, vs, t, "v"),
            _ptr(dt, ds, torch.float32, "dt"), _ptr(a, ds, torch.float32, "a"), _ptr(y, vs, torch.float32, "y"),
            _ptr(flushed, (self.cfg.batch,), torch.uint8, "flushed"), _stream(stream)),
            "replay_verify_static_scratch")
        return y

    def append_slots(self, slots=None, stream=None):
        """Ring record of every sequence's next entry (int32 [B] on the device, written on
        the stream): position s of head h of sequence b goes to record (slots[b] + s) % cap
        of ring[b][h]. For callers that write the entries there themselves and then call
        step_resident / verify_resident."""
        if slots is None:
            slots = torch.empty(self.cfg.batch, device=self.buffers["counts"].device, dtype=torch.int32)
        check(self._lib.replay_append_slots(self._ctx, _ptr(slots, (self.cfg.batch,), torch.int32, "slots"),
                                            _stream(stream)), "replay_append_slots")
        return slots

    def step_resident(self, q, y=None, flushed=None, stream=None):
        """step() whose entry the caller already wrote into the ring at append_slots()."""
        qs, vs, _ = self._token_shapes(None)
        if y is None:
            y = torch.empty(vs, device=q.device, dtype=torch.float32)
        check(self._lib.replay_step_resident(self._ctx, _ptr(q, qs, self.cfg.io_dtype, "q"),
                                             _ptr(y, vs, torch.float32, "y"),
                                             _ptr(flushed, (self.cfg.batch,), torch.uint8, "flushed"),
                                             _stream(stream)), "replay_step_resident")
        return y

    def verify_resident(self, q, y=None, flushed=None, stream=None):
        """verify() whose n_pos = q.shape[1] entries the caller already wrote into the ring."""
        n_pos = q.shape[1]
        qs, vs, _ = self._token_shapes(n_pos)
        if y is None:
            y = torch.empty(vs, device=q.device, dtype=torch.float32)
        check(self._lib.replay_verify_resident(self._ctx, n_pos, _ptr(q, qs, self.cfg.io_dtype, "q"),
                                               _ptr(y, vs, torch.float32, "y"),
                                               _ptr(flushed, (self.cfg.batch,), torch.uint8, "flushed"),
                                               _stream(stream)), "replay_verify_resident")
        return y

    def export(self, seqs, dst=None, stream=None):
        """Snapshots of the sequences seqs (int32 [n] on the device) into dst (uint8 [n,
        snapshot_bytes] on the device, allocated here if None); returns dst."""
        n = seqs.shape[0]
        nb = snapshot_bytes(self.cfg)
        if dst is None:
            dst = torch.empty(n, nb, device=seqs.device, dtype=torch.uint8)
        check(self._lib.replay_export(self._ctx, _ptr(seqs, (n,), torch.int32, "seqs"), n,
                                      _ptr(dst, (n, nb), torch.uint8, "dst"), _stream(stream)), "replay_export")
        return dst

    def import_(self, seqs, src, stream=None):
        """Restores snapshot i of src (uint8 [n, snapshot_bytes]) into sequence seqs[i]."""
        n = seqs.shape[0]
        check(self._lib.replay_import(self._ctx, _ptr(seqs, (n,), torch.int32, "seqs"), n,
                                      _ptr(src, (n, snapshot_bytes(self.cfg)), torch.uint8, "src"), _stream(stream)),
              "replay_import")

    def append_inputs(self, conv, x, raw, w, A, bias=None, dt_bias=None, q=None, v=None, stream=None):
        """token_inputs() of every sequence, its entry written straight into the ring; returns
        q for step_resident(), which must come next, and v (for gated_norm's skip term)."""
        cfg, B = self.cfg, self.cfg.batch
        _, t, D, qs, vs, _ = cfg._layer
        dev = self.buffers["S0"].get_device()
        width, *ptrs = _filter_args(cfg, conv, w, A, bias, dt_bias, dev)
        xp, ldx = _rows(x, B, D, t, "x", dev)
        rp, ldr = _rows(raw, B, cfg.heads, t, "raw", dev)

        def body(st):
            q1 = x.new_empty((B, *qs)) if q is None else q
            v1 = x.new_empty((B, *vs)) if v is None else v
            check(self._lib.replay_append_inputs(self._ctx, width, xp, ldx, rp, ldr, *ptrs,
                                                 _arg(q1, (B, *qs), t, "q", dev), _arg(v1, (B, *vs), t, "v", dev), st),
                  "replay_append_inputs")
            return q1, v1

        return _on(dev, stream, body)

    def prefill(self, q, k, v, dt, a, cu_seqlens, seqs=None, resume=None, y=None, max_len=0, scratch=None, stream=None):
        """prompt_scan() into the layer: packed prompts become the states that step() decodes
        on from. Sequence i is the layer's sequence seqs[i]; where resume[i], it continues
        from that sequence's checkpoint and buffered entries. Returns y [T][H][P] io."""
        if not isinstance(q, torch.Tensor):
            raise TypeError("q must be a torch.Tensor")
        dev, T = self.buffers["S0"].get_device(), q.shape[0]
        n, cu, sp, rp = _packed_args(cu_seqlens, seqs, resume, dev)
        ptrs, y_shape = _scan_args(self.cfg, T, q, k, v, dt, a, dev)

        def body(st):
            y1 = v.new_empty(y_shape) if y is None else y
            need = self._lib.replay_prefill_scratch(self._ctx, T, n, max_len)
            check(min(need, 0), "replay_prefill_scratch")
            sc = v.new_empty(need, dtype=torch.uint8) if scratch is None else scratch
            check(self._lib.replay_prefill(self._ctx, T, *ptrs, cu, sp, rp, n, max_len,
                                           _arg(y1, y_shape, v.dtype, "y", dev),
                                           _arg(sc, sc.shape, torch.uint8, "scratch", dev), sc.numel(), st),
                  "replay_prefill")
            return y1

        return _on(dev, stream, body)

    def rollback(self, n_keep, stream=None):
        """Keep n_keep[b] (int32 [B] on the device) of the pending verify's positions."""
        check(self._lib.replay_rollback(self._ctx, _ptr(n_keep, (self.cfg.batch,), torch.int32, "n_keep"),
                                        _stream(stream)), "replay_rollback")

    def flush(self, mask=None, stream=None):
        """Fold the buffers of the sequences with mask[b] != 0 (uint8 [B]; None = all)."""
        check(self._lib.replay_flush(self._ctx, _ptr(mask, (self.cfg.batch,), torch.uint8, "mask"),
                                     _stream(stream)), "replay_flush")

    def read_counts(self, stream=None):
        """Committed entries per sequence (synchronises the stream)."""
        out = (ctypes.c_int32 * self.cfg.batch)()
        check(self._lib.replay_read_counts(self._ctx, ctypes.cast(out, ctypes.c_void_p), _stream(stream)),
              "replay_read_counts")
        return list(out)

    def check_status(self, stream=None) -> int:
        """Device error bits (0 = none); synchronises the stream."""
        bits = ctypes.c_int32(0)
        rc = self._lib.replay_check_status(self._ctx, ctypes.byref(bits), _stream(stream))
        if rc not in (_abi.REPLAY_OK, _abi.REPLAY_EDEVICE):
            raise ReplayError(rc, "replay_check_status")
        return bits.value

    def close(self):
        if getattr(self, "_ctx", None) and self._ctx.value:
            self._lib.replay_destroy(self._ctx)
            self._ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


def eager_step(cfg: Config, S, q, k, v, dt, a, y=None, stream=None):
    """Baseline eager step: S <- a S + dt v k^T (in place), y = S q."""
    B, H, G, P, N = cfg.batch, cfg.heads, cfg.groups, cfg.P, cfg.N
    t = cfg.io_dtype
    if y is None:
        y = torch.empty(B, H, P, device=S.device, dtype=torch.float32)
    check(load().eager_step(ctypes.byref(cfg.c()), _ptr(S, (B, H, P, N), torch.float32, "S"),
                            _ptr(q, (B, G, N), t, "q"), _ptr(k, (B, G, N), t, "k"), _ptr(v, (B, H, P), t, "v"),
                            _ptr(dt, (B, H), torch.float32, "dt"), _ptr(a, (B, H), torch.float32, "a"),
                            _ptr(y, (B, H, P), torch.float32, "y"), _stream(stream)), "eager_step")
    return y


def eager_step_fp8(cfg: Config, S8, scale, q, k, v, dt, a, y=None, stream=None):
    """Baseline eager step on a shared FP8 e4m3 state with per-row scales (in place)."""
    B, H, G, P, N = cfg.batch, cfg.heads, cfg.groups, cfg.P, cfg.N
    t = cfg.io_dtype
    if y is None:
        y = torch.empty(B, H, P, device=S8.device, dtype=torch.float32)
    check(load().eager_step_fp8(ctypes.byref(cfg.c()), _ptr(S8, (B, H, P, N), torch.uint8, "S8"),
                                _ptr(scale, (B, H, P), torch.float32, "scale"), _ptr(q, (B, G, N), t, "q"),
                                _ptr(k, (B, G, N), t, "k"), _ptr(v, (B, H, P), t, "v"),
                                _ptr(dt, (B, H), torch.float32, "dt"), _ptr(a, (B, H), torch.float32, "a"),
                                _ptr(y, (B, H, P), torch.float32, "y"), _stream(stream)), "eager_step_fp8")
    return y


def quantize_rows_e2m1(x, codes=None, scale=None, stream=None):
    """Per-row e2m1 codes (two per byte, element 2i in the low nibble) and FP32 scales of
    x [..., n] (FP32, n in 16/32/64/128)."""
    n = x.shape[-1]
    rows = x.numel() // n
    cshape = (*x.shape[:-1], n // 2)
    if codes is None:
        codes = torch.empty(cshape, device=x.device, dtype=torch.uint8)
    if scale is None:
        scale = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    check(load().replay_quantize_rows_e2m1(_ptr(x, None, torch.float32, "x"), rows, n,
                                           _ptr(codes, cshape, torch.uint8, "codes"),
                                           _ptr(scale, x.shape[:-1], torch.float32, "scale"), _stream(stream)),
          "replay_quantize_rows_e2m1")
    return codes, scale


def quantize_rows_e4m3(x, codes=None, scale=None, stream=None):
    """Per-row e4m3 codes and FP32 scales of x [..., n] (FP32, n in 16/32/64/128)."""
    n = x.shape[-1]
    rows = x.numel() // n
    if codes is None:
        codes = torch.empty(x.shape, device=x.device, dtype=torch.uint8)
    if scale is None:
        scale = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    check(load().replay_quantize_rows_e4m3(_ptr(x, None, torch.float32, "x"), rows, n,
                                           _ptr(codes, x.shape, torch.uint8, "codes"),
                                           _ptr(scale, x.shape[:-1], torch.float32, "scale"), _stream(stream)),
          "replay_quantize_rows_e4m3")
    return codes, scale


def prompt_inputs(cfg: Config, conv, x, raw, w, A, cu_seqlens, bias=None, dt_bias=None, seqs=None, resume=None,
                  out=None, status=None, stream=None):
    """The inputs of packed prompts from the projection's rows: causal convolution with SiLU
    of the channels x [T][D] (v | k | q; rows may be slices of wider ones), split, and
    Delta = softplus(raw + dt_bias), a = exp(-Delta A) of the raw step sizes [T][H]. conv
    [batch][width - 1][D] (io) holds each row's last raw inputs: read where resume[s],
    always updated. w [width][D], bias [D], dt_bias, A [H] are FP32; cu_seqlens int32
    [n + 1], seqs int32 [n] (rows; None = 0..n-1), resume uint8 [n] (None = none).
    Returns (q, k, v, dt, a)."""
    dev, T = _device_of(x, "x"), x.shape[0]
    c, t, D, *_ = cfg._layer
    width, wp, bp, dbp, Ap, cp = _filter_args(cfg, conv, w, A, bias, dt_bias, dev)
    n, cu, sp, rp = _packed_args(cu_seqlens, seqs, resume, dev)
    xp, ldx = _rows(x, T, D, t, "x", dev)
    rawp, ldr = _rows(raw, T, cfg.heads, t, "raw", dev)
    stp = _arg(status, (1,), torch.int32, "status", dev)

    def body(st):
        o, ptrs = _input_outs(cfg, T, x, out, dev)
        check(load().replay_prompt_inputs(c, width, T, xp, ldx, rawp, ldr, wp, bp, dbp, Ap, cu, sp, rp, n, cp, *ptrs, stp,
                                          st), "replay_prompt_inputs")
        return o

    return _on(dev, stream, body)


def token_inputs(cfg: Config, conv, x, raw, w, A, bias=None, dt_bias=None, seqs=None, out=None, status=None,
                 stream=None):
    """prompt_inputs() for one decode token of each of n rows, from and to the state: row i
    of x belongs to row seqs[i] of conv (None = i; a negative id is padding)."""
    _width(cfg, w)
    dev, n = _device_of(x, "x"), x.shape[0]
    c, t, D, *_ = cfg._layer
    width, wp, bp, dbp, Ap, cp = _filter_args(cfg, conv, w, A, bias, dt_bias, dev)
    xp, ldx = _rows(x, n, D, t, "x", dev)
    rawp, ldr = _rows(raw, n, cfg.heads, t, "raw", dev)
    sp = _arg(seqs, (n,), torch.int32, "seqs", dev)
    stp = _arg(status, (1,), torch.int32, "status", dev)

    def body(st):
        o, ptrs = _input_outs(cfg, n, x, out, dev)
        check(load().replay_token_inputs(c, width, n, xp, ldx, rawp, ldr, wp, bp, dbp, Ap, sp, cp, *ptrs, stp, st),
              "replay_token_inputs")
        return o

    return _on(dev, stream, body)


def _scan_args(cfg, T, q, k, v, dt, a, dev):
    """Addresses of q, k, v, dt, a of T packed tokens, and the shape of y."""
    _, t, _, qs, vs, hs = cfg._layer
    kn, hp, h, f32 = (T, *qs), (T, *vs), (T, *hs), torch.float32
    return (_arg(q, kn, t, "q", dev), _arg(k, kn, t, "k", dev), _arg(v, hp, t, "v", dev), _arg(dt, h, f32, "dt", dev),
            _arg(a, h, f32, "a", dev)), hp


def prompt_scan(cfg: Config, S, q, k, v, dt, a, cu_seqlens, seqs=None, resume=None, y=None, max_len=0, scratch=None,
                status=None, stream=None):
    """The selective scan of packed prompts: S <- a S + dt v k^T, y = S q token by token, from
    row seqs[s] of S [batch][H][P][N] (FP32) where resume[s], else from zero; the final
    states go back to S. q, k [T][G][N], v [T][H][P] (io), dt, a [T][H] (FP32), cu_seqlens
    int32 [n + 1], seqs int32 [n], resume uint8 [n]. max_len, if known, steers how the work
    is split. Returns y [T][H][P] (io). A scan that fails on the device (its wait gave up,
    DEV_WAIT_TIMEOUT in status) leaves NaN in place of what it could not make."""
    _n_seqs(cu_seqlens)
    dev, T = _device_of(q, "q"), q.shape[0]
    c = cfg._layer[0]
    n, cu, sp, rp = _packed_args(cu_seqlens, seqs, resume, dev)
    ptrs, y_shape = _scan_args(cfg, T, q, k, v, dt, a, dev)
    Sp = _arg(S, (cfg.batch, cfg.heads, cfg.P, cfg.N), torch.float32, "S", dev)
    stp = _arg(status, (1,), torch.int32, "status", dev)
    lib = load()

    def body(st):
        y1 = v.new_empty(y_shape) if y is None else y
        sc = scratch
        if sc is None:
            need = lib.replay_prompt_scan_scratch(c, T, n, max_len)
            check(min(need, 0), "replay_prompt_scan_scratch")
            if need:
                sc = v.new_empty(need, dtype=torch.uint8)
        scp, sb = (None, 0) if sc is None else (_arg(sc, sc.shape, torch.uint8, "scratch", dev), sc.numel())
        check(lib.replay_prompt_scan(c, T, *ptrs, cu, sp, rp, n, max_len, Sp, _arg(y1, y_shape, v.dtype, "y", dev), scp, sb,
                                     stp, st), "replay_prompt_scan")
        return y1

    return _on(dev, stream, body)


def gated_norm(cfg: Config, y, z, weight, v=None, D=None, norm_groups=1, eps=1e-5, out=None, stream=None):
    """The gated norm of a layer's outputs: u = (y + D v) silu(z), out = u weight /
    sqrt(mean(u^2) + eps), the mean over each of norm_groups equal parts of a row. y
    [T][H][P] (FP32 or io), z [T][H*P] (io; rows may be slices of wider ones), weight
    [H*P] FP32; v [T][H][P] (io) and D [H] (FP32) for the skip term. Returns [T][H*P] io."""
    c, t, _, _, vs, hs = cfg._layer
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a torch.Tensor")
    if y.dtype is not torch.float32 and y.dtype is not t:
        raise ValueError(f"y must have dtype {torch.float32} or {t}, got {y.dtype}")
    dev, T = _device_of(z, "z"), y.shape[0]
    width, hp = cfg.heads * cfg.P, (T, *vs)
    y_type = _abi.REPLAY_F32 if y.dtype is torch.float32 else _abi.REPLAY_BF16
    yp, wp = _arg(y, hp, y.dtype, "y", dev), _arg(weight, (width,), torch.float32, "weight", dev)
    zp, ldz = _rows(z, T, width, t, "z", dev)
    vp, Dp = _arg(v, hp, t, "v", dev), _arg(D, hs, torch.float32, "D", dev)

    def body(st):
        o = z.new_empty((T, width)) if out is None else out
        check(load().replay_gated_norm(c, T, yp, y_type, zp, ldz, vp, Dp, wp, norm_groups, eps,
                                       _arg(o, (T, width), t, "out", dev), st), "replay_gated_norm")
        return o

    return _on(dev, stream, body)
