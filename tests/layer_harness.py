"""Seeded inputs of the operators around the decode step, for their GPU tests, and the
rounding steps their tolerances count."""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

import linear_attention_decode_replay_b200 as lar
from workloads import gen

U32 = 2.0 ** -24  # half a step of FP32, relative
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the io type, relative
TINY = 2.0 ** -126


@dataclass(frozen=True)
class Case:
    name: str
    H: int
    G: int
    P: int
    N: int
    lens: tuple
    io: str = "bf16"
    width: int = 4
    resume: str = "none"  # "none", "all" or "some"
    rows: int = 0         # rows of the state; 0: one a sequence, in order, no ids passed
    lead: int = 0         # tokens before the first sequence
    tail: int = 0         # ... and behind the last
    seed: int = 0

    @property
    def T(self):
        return self.lead + sum(self.lens) + self.tail

    @property
    def D(self):
        return self.H * self.P + 2 * self.G * self.N

    @property
    def batch(self):
        return self.rows or len(self.lens)

    @property
    def dtype(self):
        return torch.bfloat16 if self.io == "bf16" else torch.float32

    def cfg(self, **kw):
        return lar.Config(batch=self.batch, heads=self.H, groups=self.G, P=self.P, N=self.N, L=1, io=self.io, **kw)


def packed(case, device="cuda"):
    """cu_seqlens, seqs, resume of a case (device tensors; seqs and resume may be None)."""
    g = torch.Generator().manual_seed(case.seed + 5)
    cu = torch.tensor([case.lead] + (case.lead + np.cumsum(case.lens)).tolist(), dtype=torch.int32)
    n = len(case.lens)
    seqs = torch.randperm(case.rows, generator=g)[:n].to(torch.int32) if case.rows else None
    resume = {"none": None, "all": torch.ones(n, dtype=torch.uint8),
              "some": (torch.arange(n) % 2 == 0).to(torch.uint8)}[case.resume]
    return tuple(None if t is None else t.to(device) for t in (cu, seqs, resume))


def scan_inputs(case, decay=None, device="cuda"):
    """q, k, v, dt, a, S. decay: None (step sizes of fast and slow heads) or a constant a."""
    g = torch.Generator(device=device).manual_seed(case.seed + 11)
    randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    T, H = case.T, case.H
    q, k = randn(T, case.G, case.N), randn(T, case.G, case.N)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    v = randn(T, H, case.P)
    rate = torch.exp(torch.linspace(-5.0, 0.0, H, device=device)) if H > 1 else torch.full((1,), 0.1, device=device)
    dt = torch.nn.functional.softplus(randn(T, H)) * rate
    a = torch.exp(-dt) if decay is None else torch.full_like(dt, decay)
    S = 0.1 * randn(case.batch, H, case.P, case.N)
    return [q.to(case.dtype), k.to(case.dtype), v.to(case.dtype), dt, a, S]


def layer_rows(case, n=None, device="cuda"):
    """The projection's rows (gate | channels | step sizes), the filter and the state."""
    g = torch.Generator(device=device).manual_seed(case.seed + 23)
    randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    n = case.T if n is None else n
    hp = case.H * case.P
    proj = randn(n, hp + case.D + case.H + (-case.H) % 8).to(case.dtype)
    f = {"w": 0.5 * randn(case.width, case.D), "bias": 0.2 * randn(case.D), "dt_bias": randn(case.H),
         "A": 0.5 + torch.rand(case.H, generator=g, device=device)}
    conv = randn(case.batch, case.width - 1, case.D).to(case.dtype)
    return {"proj": proj, "z": proj[:, :hp], "x": proj[:, hp:hp + case.D],
            "raw": proj[:, hp + case.D:hp + case.D + case.H], "conv": conv, **f}


def f64(t):
    return None if t is None else gen.to_numpy64(t)


def assert_within(got, want, bound, what):
    """Elementwise |got - want| <= bound wherever want is finite; the same infinities and NaN."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), f"{what}: other elements are finite"
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(bound, want.shape)[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max():.3e} over its bound"
