"""CPU checks of the operators around the decode step: the float64 oracle against torch and
the decode oracle, and the argument checks of the C ABI (no compute calls)."""

import copy
import ctypes
import dataclasses
import pickle

import numpy as np
import pytest
import torch

import linear_attention_decode_replay_b200 as lar
from linear_attention_decode_replay_b200 import _abi
from oracle import layer_oracle as lo
from oracle import replay_oracle as ro


def test_convolution_is_torchs():
    g = np.random.default_rng(0)
    T, D, W, H = 9, 6, 4, 2
    x, raw, w, b, dtb, A = (g.standard_normal(s) for s in ((T, D), (T, H), (W, D), (D,), (H,), (H,)))
    conv = g.standard_normal((3, W - 1, D))
    cu, seqs, resume = [0, 2, 2, 9], [2, 0, 1], [1, 1, 0]
    y, dt, a, new, _ = lo.prompt_inputs(x, raw, w, b, dtb, A, conv, cu, seqs, resume)
    t = torch.from_numpy
    for s in range(3):
        old = conv[seqs[s]] if resume[s] else np.zeros((W - 1, D))
        seen = np.concatenate([old, x[cu[s]:cu[s + 1]]])
        assert np.array_equal(new[seqs[s]], seen[len(seen) - W + 1:])
        if cu[s + 1] > cu[s]:
            ref = torch.nn.functional.conv1d(t(seen.T[None].copy()), t(w.T[:, None].copy()), t(b), groups=D)[0].T
            np.testing.assert_allclose(y[cu[s]:cu[s + 1]], torch.nn.functional.silu(ref).numpy(), rtol=1e-12)
    sp = torch.nn.functional.softplus(t(raw + dtb), threshold=1e9)
    np.testing.assert_allclose(dt, sp.numpy(), rtol=1e-12)
    np.testing.assert_allclose(a, np.exp(-dt * A), rtol=1e-12)


def test_scan_is_the_eager_recurrence():
    g = np.random.default_rng(1)
    T, H, G, P, N = 7, 4, 2, 8, 16
    q, k, v = (g.standard_normal(s) for s in ((T, G, N), (T, G, N), (T, H, P)))
    dt, a = g.random((T, H)), g.random((T, H))
    S0 = g.standard_normal((2, H, P, N))
    cu, resume = [0, 3, 7], [1, 0]
    y, S = lo.prompt_scan(q, k, v, dt, a, S0, cu, None, resume)
    for s in range(2):
        X = (S0[s:s + 1] if resume[s] else np.zeros_like(S0[:1])).copy()
        for t in range(cu[s], cu[s + 1]):
            X, yt = ro.eager_batch_step(X, q[t:t + 1], k[t:t + 1], v[t:t + 1], dt[t:t + 1], a[t:t + 1], G)
            np.testing.assert_allclose(y[t], yt[0], rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(S[s], X[0], rtol=1e-12)


def test_norm_is_torchs():
    g = np.random.default_rng(2)
    y, v = g.standard_normal((3, 4, 8)), g.standard_normal((3, 4, 8))
    z, w, D = g.standard_normal((3, 32)), g.standard_normal(32), g.standard_normal(4)
    out = lo.gated_norm(y, z, w, v, D, groups=2, eps=1e-3)
    t = torch.from_numpy
    u = t((y + D[:, None] * v).reshape(3, 32)) * torch.nn.functional.silu(t(z))
    ref = torch.nn.functional.rms_norm(u.reshape(3, 2, 16), (16,), eps=1e-3).reshape(3, 32) * t(w)
    np.testing.assert_allclose(out, ref.numpy(), rtol=1e-12)


def test_rows_served():
    assert lo.rows_served([0, 1, 2, 3, 4], [1, -1, 1, 7], 2) == [(0, 0, 1, 1)]


# ------------------------------------------------------------------- the C ABI's refusals
P0 = ctypes.c_void_p(0x10000)  # never read: every call below is refused on the host
ODD = ctypes.c_void_p(0x10004)


def _cfg(**kw):
    base = dict(batch=2, heads=4, groups=2, P=16, N=16, L=1, max_pos=1, io=_abi.REPLAY_BF16, ckpt=0)
    return ctypes.byref(_abi.CConfig(**{**base, **kw}))


D = 4 * 16 + 2 * 2 * 16  # channels of that layer


def _prompt_inputs(cfg=None, **kw):
    a = dict(width=4, tokens=8, x=P0, ldx=D, raw=P0, ldr=4, w=P0, bias=None, dt_bias=None, A=P0, cu=P0, seqs=None,
             resume=None, n=2, conv=P0, q=P0, k=P0, v=P0, dt=P0, a=P0, status=None, stream=None)
    a.update(kw)
    return _abi.load().replay_prompt_inputs(cfg or _cfg(), *a.values())


def _token_inputs(cfg=None, **kw):
    a = dict(width=4, n=2, x=P0, ldx=D, raw=P0, ldr=4, w=P0, bias=None, dt_bias=None, A=P0, seqs=None, conv=P0, q=P0,
             k=P0, v=P0, dt=P0, a=P0, status=None, stream=None)
    a.update(kw)
    return _abi.load().replay_token_inputs(cfg or _cfg(), *a.values())


def _scan(cfg=None, **kw):
    a = dict(tokens=8, q=P0, k=P0, v=P0, dt=P0, a=P0, cu=P0, seqs=None, resume=None, n=2, max_len=0, S=P0, y=P0,
             scratch=None, scratch_bytes=0, status=None, stream=None)
    a.update(kw)
    return _abi.load().replay_prompt_scan(cfg or _cfg(), *a.values())


def _norm(cfg=None, **kw):
    a = dict(rows=3, y=P0, y_type=_abi.REPLAY_BF16, z=P0, ldz=64, v=None, D=None, weight=P0, groups=1, eps=1e-5, out=P0,
             stream=None)
    a.update(kw)
    return _abi.load().replay_gated_norm(cfg or _cfg(), *a.values())


@pytest.mark.parametrize("bad", [dict(cfg=_cfg(N=48)), dict(width=1), dict(width=5), dict(tokens=-1),
                                 dict(tokens=2**31), dict(x=None), dict(raw=None), dict(w=None), dict(A=None),
                                 dict(conv=None), dict(q=None), dict(dt=None), dict(cu=None), dict(n=-1), dict(n=3),
                                 dict(ldx=D - 8), dict(ldr=3)], ids=str)
def test_prompt_inputs_refuses(bad):
    assert _prompt_inputs(**bad) == _abi.REPLAY_EINVAL


@pytest.mark.parametrize("bad", [dict(x=ODD), dict(ldx=D + 4), dict(conv=ODD), dict(q=ODD), dict(v=ODD),
                                 dict(raw=ctypes.c_void_p(0x10001)), dict(w=ctypes.c_void_p(0x10002)),
                                 dict(cu=ctypes.c_void_p(0x10002)), dict(status=ctypes.c_void_p(0x10002))], ids=str)
def test_prompt_inputs_refuses_alignments(bad):
    assert _prompt_inputs(**bad) == _abi.REPLAY_EALIGN


def test_calls_with_nothing_to_do():
    assert _prompt_inputs(n=0, cu=None) == _abi.REPLAY_OK
    assert _token_inputs(n=0, x=None, raw=None, q=None, k=None, v=None, dt=None, a=None) == _abi.REPLAY_OK
    assert _scan(n=0, cu=None) == _abi.REPLAY_OK
    assert _norm(rows=0, y=None, z=None, out=None) == _abi.REPLAY_OK


@pytest.mark.parametrize("bad", [dict(cfg=_cfg(P=12)), dict(width=0), dict(n=-1), dict(n=3), dict(x=None),
                                 dict(raw=None), dict(conv=None), dict(k=None), dict(a=None), dict(ldx=8)], ids=str)
def test_token_inputs_refuses(bad):
    assert _token_inputs(**bad) == _abi.REPLAY_EINVAL
    assert _token_inputs(seqs=ctypes.c_void_p(0x10002)) == _abi.REPLAY_EALIGN


@pytest.mark.parametrize("bad", [dict(cfg=_cfg(groups=3)), dict(tokens=-1), dict(tokens=2**31), dict(q=None),
                                 dict(a=None), dict(S=None), dict(y=None), dict(cu=None), dict(n=3), dict(n=-1),
                                 dict(max_len=-1), dict(seqs=P0, n=2**30)], ids=str)
def test_prompt_scan_refuses(bad):
    assert _scan(**bad) == _abi.REPLAY_EINVAL
    for name in "qkvy":
        assert _scan(**{name: ODD}) == _abi.REPLAY_EALIGN
    assert _scan(S=ODD) == _abi.REPLAY_EALIGN and _scan(scratch=ODD) == _abi.REPLAY_EALIGN


def test_scan_scratch_and_its_check():
    lib = _abi.load()
    assert lib.replay_prompt_scan_scratch(_cfg(N=20), 8, 2, 0) == _abi.REPLAY_EINVAL
    assert lib.replay_prompt_scan_scratch(_cfg(), -1, 2, 0) == _abi.REPLAY_EINVAL
    assert lib.replay_prompt_scan_scratch(_cfg(), 8, -2, 0) == _abi.REPLAY_EINVAL
    assert lib.replay_prompt_scan_scratch(_cfg(), 0, 0, 0) == 0
    for tokens, n, longest in ((8, 2, 0), (100000, 1, 0), (100000, 2, 99000), (2**31 - 1, 2, 0)):
        need = lib.replay_prompt_scan_scratch(_cfg(), tokens, n, longest)
        assert need >= 0 and need % 256 == 0
        if need:
            assert _scan(tokens=tokens, n=n, max_len=longest) == _abi.REPLAY_EINVAL
            assert _scan(tokens=tokens, n=n, max_len=longest, scratch=P0, scratch_bytes=need - 1) == _abi.REPLAY_EINVAL


@pytest.mark.parametrize("bad", [dict(cfg=_cfg(N=20)), dict(rows=-1), dict(y=None), dict(z=None), dict(out=None),
                                 dict(weight=None), dict(v=P0), dict(D=P0), dict(groups=0), dict(groups=3),
                                 dict(groups=16), dict(ldz=56), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(y_type=5), dict(rows=2**31)], ids=str)
def test_gated_norm_refuses(bad):
    assert _norm(**bad) == _abi.REPLAY_EINVAL
    for name in ("y", "z", "out"):
        assert _norm(**{name: ODD}) == _abi.REPLAY_EALIGN
    assert _norm(ldz=68) == _abi.REPLAY_EALIGN


def test_layer_calls_on_a_null_context_are_refused():
    lib = _abi.load()
    p = P0
    assert lib.replay_append_inputs(None, 4, p, D, p, 4, p, None, None, p, p, p, None, None) == _abi.REPLAY_EINVAL
    assert lib.replay_prefill(None, 8, p, p, p, p, p, p, None, None, 2, 0, p, p, 256, None) == _abi.REPLAY_EINVAL
    assert lib.replay_prefill_scratch(None, 8, 2, 0) == _abi.REPLAY_EINVAL


def test_the_binding_refuses_other_tensors():
    cfg = lar.Config(batch=2, heads=4, groups=2, P=16, N=16, L=1)
    x = torch.zeros(3, D, dtype=torch.bfloat16)
    conv = torch.zeros(2, 3, D, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    f = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        lar.prompt_inputs(cfg, conv, x, f(3, 4), f(4, D), f(4), cu)
    with pytest.raises(ValueError, match="CUDA"):
        lar.token_inputs(cfg, conv, x, f(3, 4), f(4, D), f(4))
    with pytest.raises(ValueError, match="CUDA"):
        lar.prompt_scan(cfg, f(2, 4, 16, 16), f(3, 2, 16), f(3, 2, 16), f(3, 4, 16), f(3, 4), f(3, 4), cu)
    with pytest.raises(ValueError, match="CUDA"):
        lar.gated_norm(cfg, f(3, 4, 16), f(3, 64).bfloat16(), f(64))
    with pytest.raises(ValueError, match="dtype"):
        lar.gated_norm(cfg, f(3, 4, 16).double(), f(3, 64).bfloat16(), f(64))
    with pytest.raises(ValueError, match="width"):
        lar.token_inputs(cfg, conv, x, f(3, 4), f(4), f(4))
    with pytest.raises(ValueError, match="cu_seqlens"):
        lar.prompt_scan(cfg, f(2, 4, 16, 16), f(3, 2, 16), f(3, 2, 16), f(3, 4, 16), f(3, 4), f(3, 4), cu[:0])


def test_the_binding_refuses_what_is_no_tensor():
    cfg = lar.Config(batch=2, heads=4, groups=2, P=16, N=16, L=1)
    f, cu = torch.zeros, torch.tensor([0, 3], dtype=torch.int32)
    layer = object.__new__(lar.Replay)  # no context: the argument is refused before one is used
    layer.cfg, layer.buffers, layer._ctx = cfg, {"S0": f(2, 4, 16, 16)}, None
    with pytest.raises(TypeError, match="y must be"):
        lar.gated_norm(cfg, [1.0], f(3, 64).bfloat16(), f(64))
    with pytest.raises(TypeError, match="q must be"):
        layer.prefill([1.0], f(3, 2, 16), f(3, 4, 16), f(3, 4), f(3, 4), cu)


def test_a_norm_of_no_rows_with_the_skip_term():
    """Without rows v, like y, z and out, has no address; D has its own."""
    assert _norm(rows=0, y=None, z=None, out=None, v=None, D=P0) == _abi.REPLAY_OK
    assert _norm(rows=1, v=None, D=P0) == _abi.REPLAY_EINVAL


@pytest.mark.parametrize("again", [lambda c: pickle.loads(pickle.dumps(c)), copy.copy, copy.deepcopy,
                                   lambda c: lar.Config(**vars(c)), lambda c: dataclasses.replace(c)],
                         ids=["pickle", "copy", "deepcopy", "vars", "replace"])
def test_a_config_that_was_used_is_copied_like_a_new_one(again):
    cfg = lar.Config(batch=2, heads=4, groups=2, P=16, N=16, L=1)
    fields = dict(vars(cfg))
    with pytest.raises(ValueError, match="CUDA"):
        lar.gated_norm(cfg, torch.zeros(3, 4, 16), torch.zeros(3, 64).bfloat16(), torch.zeros(64))
    other = again(cfg)
    assert other == cfg and hash(other) == hash(cfg) and vars(cfg) == fields == vars(other)
    with pytest.raises(ValueError, match="CUDA"):
        lar.gated_norm(other, torch.zeros(3, 4, 16), torch.zeros(3, 64).bfloat16(), torch.zeros(64))


def test_the_binding_needs_no_private_call_of_torch(monkeypatch):
    """Loaded with a torch that lacks its short forms, it takes the public calls."""
    import importlib.util

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.find_spec(lar.__name__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: type("S", (), {"cuda_stream": 40 + dev}))
    monkeypatch.setattr(other, "_current_device", lambda: 3)
    assert other._on(3, None, lambda raw: raw) == 43
