"""The layer's inputs and the gated norm against the float64 oracle, and a layer's whole
path: prompt inputs, prefill, decode steps from token inputs, and the norm.

Bounds. The convolution sums width products and a bias in FP32: the error of its sum is at
most (width + 2) 2^-24 of the terms' magnitudes; sigmoid(c) c has a slope of at most 1.1,
and its own evaluation is within 8 units of 2^-24 (accurate exponential, sum, division),
or, for results rounded to BF16, 2^-19 (the fast exponential is within 2 + |c| 1.2 steps of
2^-23 of the result, |c| < 12 here). Rounding to the io type adds half a step. Step sizes
and decays: the sum, exponential, logarithm and sum each within 2 steps of 2^-23 (8 units
of 2^-24); a = exp(-Delta A) turns Delta's relative error into |Delta A| of it."""

import numpy as np
import pytest
import torch

import linear_attention_decode_replay_b200 as lar
from linear_attention_decode_replay_b200 import _abi
from layer_harness import HALF, U32, Case, assert_within, f64, layer_rows, packed
from oracle import layer_oracle as lo
from oracle import replay_oracle as ro

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

CASES = [
    Case("tiny", 2, 2, 16, 16, (37,), "f32"),
    Case("one", 1, 1, 8, 16, (1,), "bf16", resume="all"),
    Case("short", 3, 1, 24, 32, (1, 2, 3, 0, 4, 5), "bf16", resume="some", rows=9),
    Case("w2", 4, 2, 64, 64, (65, 1, 31), "bf16", 2, resume="all"),
    Case("w3", 2, 1, 40, 128, (33, 32, 2, 30), "f32", 3, resume="some", rows=4, lead=2, tail=7),
    Case("w4", 8, 8, 64, 128, (95, 97, 1), "bf16", 4, resume="some"),
    Case("starts", 2, 1, 64, 128, (31, 1, 1, 1, 30, 64, 63, 2, 31), "bf16", 4, resume="all", rows=12, lead=1),
    Case("pieces", 8, 2, 64, 128, (5,) * 60, "bf16", 4, resume="all"),
    Case("wide", 64, 8, 64, 128, (150,), "bf16", 4),
]


def split(case, y):
    return lo.split(y, case.H, case.G, case.P, case.N)


def check_inputs(case, got, want, live=None):
    y, dt, a, conv, mag = want
    live = ~np.isnan(dt[:, 0]) if live is None else live
    q, k, v, gdt, ga, gconv = got
    by = 1.1 * (case.width + 2) * U32 * mag + np.abs(y) * ((2.0 ** -19 if case.io == "bf16" else 8 * U32) + HALF[case.io])
    for name, g, w, b in zip("qkv", (q, k, v), split(case, y), split(case, by)):
        assert_within(f64(g)[live], w[live], b[live] + 1e-37, f"{case.name}: {name}")
    return live, gdt, ga, gconv


@pytest.mark.parametrize("case", CASES, ids=[c.name for c in CASES])
@pytest.mark.parametrize("plain", [False, True], ids=["bias", "no_bias"])
def test_prompt_inputs_match_the_oracle(case, plain):
    r = layer_rows(case)
    cu, seqs, resume = packed(case)
    bias, dt_bias = (None, None) if plain else (r["bias"], r["dt_bias"])
    conv = r["conv"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = case.dtype
    out = tuple(torch.full(s, 7.0, device="cuda", dtype=d) for s, d in
                (((case.T, case.G, case.N), t), ((case.T, case.G, case.N), t), ((case.T, case.H, case.P), t),
                 ((case.T, case.H), torch.float32), ((case.T, case.H), torch.float32)))
    q, k, v, dt, a = lar.prompt_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"], cu, bias=bias,
                                       dt_bias=dt_bias, seqs=seqs, resume=resume, out=out, status=status)
    assert q is out[0] and status.item() == 0
    want = lo.prompt_inputs(f64(r["x"]), f64(r["raw"]), f64(r["w"]), f64(bias), f64(dt_bias), f64(r["A"]),
                            f64(r["conv"]), f64(cu), f64(seqs), f64(resume))
    live, *_ = check_inputs(case, (q, k, v, dt, a, conv), want)
    x_mag = np.abs(f64(r["raw"])) + (0 if plain else np.abs(f64(dt_bias)))
    bdt = 8 * U32 * want[1] + U32 * x_mag  # the sum's rounding moves softplus by as much at most
    ba = want[2] * (4 * U32 + f64(r["A"]) * (bdt + U32 * want[1])) + 1e-37
    assert_within(f64(dt)[live], want[1][live], bdt[live], "dt")
    assert_within(f64(a)[live], want[2][live], ba[live], "a")
    assert np.array_equal(f64(conv), want[3])
    for o in out:
        assert (o[torch.from_numpy(~live).cuda()] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("n", [1, 2, 7, 40])
def test_token_inputs_are_prompts_of_one_token(io, width, n):
    """Bit for bit the packed form's outputs and states for sequences of length one."""
    case = Case("tok", 6, 3, 24, 32, (1,) * n, io, width, resume="all", rows=n + 3, seed=n)
    r = layer_rows(case)
    cu, seqs, resume = packed(case)
    c0, c1 = r["conv"].clone(), r["conv"].clone()
    want = lar.prompt_inputs(case.cfg(), c0, r["x"], r["raw"], r["w"], r["A"], cu, r["bias"], r["dt_bias"], seqs, resume)
    got = lar.token_inputs(case.cfg(), c1, r["x"], r["raw"], r["w"], r["A"], r["bias"], r["dt_bias"], seqs)
    for w, g in zip(want, got):
        assert torch.equal(w, g)
    assert torch.equal(c0, c1)


def test_token_padding_and_bad_ids():
    case = Case("ids", 2, 1, 32, 32, (1,) * 5, "bf16", rows=4)
    r = layer_rows(case)
    seqs = torch.tensor([2, -1, 2, 9, 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    conv = r["conv"].clone()
    t = case.dtype
    out = tuple(torch.full(s, 7.0, device="cuda", dtype=d) for s, d in
                (((5, 1, 32), t), ((5, 1, 32), t), ((5, 2, 32), t), ((5, 2), torch.float32), ((5, 2), torch.float32)))
    lar.token_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"], seqs=seqs, out=out, status=status)
    assert status.item() == _abi.DEV_SEQS
    for o in out:
        assert (o[1:4] == 7).all() and not (o[[0, 4]] == 7).all()
    assert torch.equal(conv[[1, 3]], r["conv"][[1, 3]])
    assert torch.equal(conv[0, :2], r["conv"][0, 1:]) and torch.equal(conv[0, 2], r["x"][4])
    conv2 = r["conv"].clone()
    lar.prompt_inputs(case.cfg(), conv2, r["x"], r["raw"], r["w"], r["A"],
                      torch.arange(6, dtype=torch.int32, device="cuda"), seqs=seqs,
                      resume=torch.ones(5, dtype=torch.uint8, device="cuda"), status=status.zero_())
    assert status.item() == _abi.DEV_SEQS and torch.equal(conv, conv2)


def test_extreme_step_sizes():
    """Raw step sizes far out: softplus neither overflows nor loses its tail."""
    case = Case("steps", 4, 1, 8, 16, (8,), "f32")
    r = layer_rows(case)
    raw = torch.tensor([-200.0, -90.0, -20.0, -1e-4, 0.0, 20.0, 90.0, 3e4], device="cuda")[:, None].repeat(1, 4)
    cu, *_ = packed(case)
    *_, dt, a = lar.prompt_inputs(case.cfg(), r["conv"], r["x"], raw.contiguous(), r["w"], r["A"], cu)
    want = lo.softplus(f64(raw))
    assert_within(dt, want, 8 * U32 * want + 1e-37, "dt")
    wa = np.exp(-want * f64(r["A"]))
    assert_within(a, wa, wa * (4 * U32 + 10 * U32 * want * f64(r["A"])) + 1e-37, "a")


@pytest.mark.parametrize("T,H,P,groups", [(1, 1, 8, 1), (3, 2, 16, 2), (37, 8, 64, 1), (5, 64, 64, 8), (9, 64, 64, 1),
                                          (4, 5, 24, 1), (2, 64, 256, 1), (3, 130, 64, 1), (300, 4, 32, 4)])
@pytest.mark.parametrize("io,y_type", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("skip", [False, True])
def test_gated_norm_matches_the_oracle(T, H, P, groups, io, y_type, skip):
    """Bound: u carries the gate's error and three roundings (each 2^-24; the fast gate 2^-19
    where the result is BF16); the mean's is half of 2 u's plus the sum's (positive terms:
    width / 512 + 16 roundings), so the result's relative error is at most twice u's and the
    sum's, plus 4, plus half a step. The skip term's sum counts against its terms' magnitudes."""
    case = Case("norm", H, 1, P, 16, (T,), io, seed=T + H)
    r = layer_rows(case)
    g = torch.Generator(device="cuda").manual_seed(T)
    y = torch.randn(T, H, P, generator=g, device="cuda").to(torch.bfloat16 if y_type == "bf16" else torch.float32)
    v = torch.randn(T, H, P, generator=g, device="cuda").to(case.dtype) if skip else None
    D = torch.randn(H, generator=g, device="cuda") if skip else None
    w = torch.randn(H * P, generator=g, device="cuda")
    out = lar.gated_norm(case.cfg(), y, r["z"], w, v=v, D=D, norm_groups=groups)
    fy, fv, fD, fz = f64(y), f64(v), f64(D), f64(r["z"])
    want = lo.gated_norm(fy, fz, f64(w), fv, fD, groups)
    mag = np.abs(fy) + (np.abs(fD)[None, :, None] * np.abs(fv) if skip else 0)
    u = (fy + (fD[None, :, None] * fv if skip else 0)).reshape(T, groups, -1) * lo.silu(fz).reshape(T, groups, -1)
    rms = np.sqrt((u * u).mean(-1, keepdims=True) + 1e-5)
    term = (mag.reshape(T, -1) * np.abs(lo.silu(fz))).reshape(T, groups, -1) / rms
    fast = 2.0 ** -19 if io == "bf16" else 8 * U32
    width = H * P // groups
    # the mean's relative error: u's error against u, in norms over the part
    mean = fast + U32 * (3 * np.sqrt((term * term).mean(-1, keepdims=True)) + width / 512 + 16)
    b = ((fast + 3 * U32) * term + np.abs(u / rms) * (mean + 4 * U32)).reshape(T, -1) * np.abs(f64(w))
    assert_within(out, want, b + HALF[io] * np.abs(want) + 1e-37, "out")


def test_gated_norm_of_zero_rows_and_in_place():
    case = Case("z", 4, 1, 64, 16, (6,), "bf16")
    r = layer_rows(case)
    y = torch.randn(6, 4, 64, device="cuda").bfloat16()
    y[2] = 0
    w = torch.ones(256, device="cuda")
    want = lar.gated_norm(case.cfg(), y, r["z"], w)
    assert (want[2] == 0).all()  # eps holds the division
    lar.gated_norm(case.cfg(), y, r["z"], w, out=y.view(6, 256))
    assert torch.equal(y.view(6, 256), want)
    assert lar.gated_norm(case.cfg(), y[:0], r["z"][:0], w).shape == (0, 256)


def test_no_tokens_and_no_sequences():
    case = Case("none", 2, 1, 32, 32, (0, 0), "bf16", resume="some")
    r = layer_rows(case)
    cu, _, resume = packed(case)
    conv = r["conv"].clone()
    q, *_ = lar.prompt_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"], cu, resume=resume)
    assert q.shape[0] == 0 and torch.equal(conv[0], r["conv"][0]) and (conv[1] == 0).all()
    conv = r["conv"].clone()
    lar.prompt_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"], cu[:1])
    lar.token_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"])
    assert torch.equal(conv, r["conv"])


def test_inputs_in_a_graph_and_on_another_stream():
    case = Case("graph", 4, 2, 64, 128, (90, 33, 2), "bf16", resume="all")
    r = layer_rows(case)
    cu, _, resume = packed(case)
    conv = r["conv"].clone()
    call = lambda c, **kw: lar.prompt_inputs(case.cfg(), c, r["x"], r["raw"], r["w"], r["A"], cu, r["bias"],  # noqa: E731
                                             r["dt_bias"], resume=resume, **kw)
    want = call(conv)
    side = torch.cuda.Stream()
    c1 = r["conv"].clone()
    torch.cuda.synchronize()
    got = call(c1, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and torch.equal(c1, conv)
    c2 = r["conv"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(c2)
        o = lar.gated_norm(case.cfg(), out[2], r["z"], r["w"][0, :case.H * case.P].contiguous())
    for _ in range(2):
        c2.copy_(r["conv"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out)) and torch.equal(c2, conv)
        assert torch.equal(o, lar.gated_norm(case.cfg(), want[2], r["z"], r["w"][0, :case.H * case.P].contiguous()))


@pytest.mark.parametrize("ckpt", ["f32", "f32_fp8read", "f32_fp4read"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_layer_from_prompt_to_decode(ckpt, io):
    """Two rows of a layer of four get prompts, decode a few tokens, one of them takes a second
    piece of prompt on top of its buffered entries, and decode goes on: outputs, states and
    counts against the oracle fed the same inputs token by token."""
    H, G, P, N, L, B = 4, 2, 24, 32, 5, 4
    cfg = lar.Config(batch=B, heads=H, groups=G, P=P, N=N, L=L, io=io, ckpt=ckpt)
    bufs = lar.alloc_buffers(cfg, "cuda")
    bufs["S0"].normal_(0, 0.1)
    layer = lar.Replay(cfg, bufs)
    ref = ro.ReplayBatch(f64(bufs["S0"]).copy(), G, L, ckpt=ckpt)
    tol = 1e-4 if ckpt == "f32" else 1e-2  # the bars of the decode parity tests

    def prompt(lens, rows, resume, seed):
        case = Case("p", H, G, P, N, lens, io, rows=B, seed=seed)
        r = layer_rows(case)
        cu = packed(case)[0]
        seqs = torch.tensor(rows, dtype=torch.int32, device="cuda")
        res = None if resume is None else torch.tensor(resume, dtype=torch.uint8, device="cuda")
        q, k, v, dt, a = lar.prompt_inputs(cfg, conv, r["x"], r["raw"], w, A, cu, seqs=seqs, resume=res)
        for i, b in enumerate(rows):
            if resume and resume[i]:
                ref.seqs[b].fold()
        S0 = ref.checkpoints()
        y = layer.prefill(q, k, v, dt, a, cu, seqs=seqs, resume=res)
        args = [f64(t) for t in (q, k, v, dt, a)]
        want, S = lo.prompt_scan(*args, S0, f64(cu), rows, resume)
        mag, _ = lo.prompt_scan_magnitude(*args, S0, f64(cu), rows, resume)
        # test_gpu_scan's bound; the folded checkpoint that a piece resumes from is within 1e-5
        assert_within(y, want, ((2 * max(lens) + N + 8) * U32 + 1e-5) * mag + HALF[io] * np.abs(want)
                      + (2.0 ** -14 * mag if io == "bf16" else 0), "prefill y")
        for b in rows:
            ref.seqs[b] = ro.ReplaySeq(S[b], G, L, ckpt=ckpt)
        o = lar.gated_norm(cfg, y, r["z"], torch.ones(H * P, device="cuda"), v=v, D=torch.ones(H, device="cuda"))
        assert torch.isfinite(o).all()

    def decode(n, seed):
        for t in range(n):
            case = Case("d", H, G, P, N, (1,) * B, io, seed=seed + t)
            r = layer_rows(case)
            c0 = conv.clone()
            q1, k1, v1, dt1, a1 = lar.token_inputs(cfg, c0, r["x"], r["raw"], w, A)
            q, v = layer.append_inputs(conv, r["x"], r["raw"], w, A)
            assert torch.equal(q, q1) and torch.equal(v, v1) and torch.equal(conv, c0)
            y = layer.step_resident(q)
            want, _ = ref.step(*[f64(x) for x in (q1, k1, v1, dt1, a1)])
            assert ro.relative_error(f64(y), want) <= tol
            o = lar.gated_norm(cfg, y, r["z"], torch.ones(H * P, device="cuda"), v=v, D=torch.ones(H, device="cuda"))
            assert torch.isfinite(o).all()
        assert layer.read_counts() == list(ref.counts)

    case = Case("f", H, G, P, N, (1,) * B, io, seed=99)
    f = layer_rows(case)
    conv, w, A = f["conv"], f["w"], f["A"]
    decode(3, 100)
    prompt((140, 7), [2, 0], None, 1)
    decode(7, 200)
    prompt((20, 0, 33), [2, 1, 3], [1, 1, 0], 2)
    decode(6, 300)
    assert layer.check_status() == 0


def test_a_prefill_in_a_graph():
    """A prompt into a layer and two steps, captured: every replay gives what the calls give."""
    H, G, P, N, B = 4, 2, 24, 32, 2
    cfg = lar.Config(batch=B, heads=H, groups=G, P=P, N=N, L=3)
    case = Case("g", H, G, P, N, (140, 70), "bf16", rows=B)
    r = layer_rows(case)
    cu = packed(case)[0]
    ins = lar.prompt_inputs(cfg, r["conv"].clone(), r["x"], r["raw"], r["w"], r["A"], cu)
    token = [t[:B].contiguous() for t in ins]

    def calls(layer):
        return [layer.prefill(*ins, cu), layer.step(*token), layer.step(*token)]

    first = lar.Replay(cfg, lar.alloc_buffers(cfg, "cuda"))
    want = [t.clone() for t in calls(first)]
    layer = lar.Replay(cfg, lar.alloc_buffers(cfg, "cuda"))
    calls(layer)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(layer)
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert torch.equal(layer.buffers["S0"], first.buffers["S0"])
    assert layer.read_counts() == first.read_counts() and layer.check_status() == 0


def good_sequences(bounds, T):
    """The sequences whose own bounds are good, and how many of them hold each token."""
    good = [s for s in range(len(bounds) - 1) if 0 <= bounds[s] <= bounds[s + 1] <= T]
    held = np.zeros(T, int)
    for s in good:
        held[bounds[s]:bounds[s + 1]] += 1
    return good, held


BAD_BOUNDS = {
    "falls": (60, [0, 10, 5, 60]),
    "falls_far": (100, [0, 100, 40, 60]),
    "falls_outside": (60, [0, 10, 500, 30, 60]),
    "all_down": (60, [60, 40, 20, 0]),
    # the mistake behind what one look of the search sees
    "falls_late": (900, [3 * i for i in range(280)] + [100, 850, 900]),
    "before": (60, [-4, 10, 30, 60]),
    "all_before": (60, [-9, -4, 0, 60]),
    "past": (60, [0, 10, 30, 61]),
    "far_past": (60, [0, 10, 10, 2 ** 31 - 1, 2 ** 31 - 1]),
}


@pytest.mark.parametrize("resume", ["none", "all"])
@pytest.mark.parametrize("name", BAD_BOUNDS)
def test_inputs_with_bad_bounds(name, resume):
    """Sequences with bad bounds are skipped and reported. Where no bounds fall the others have
    their outputs and states; where some do, every state is the old one or the right one, and
    every token that one sequence alone holds has its outputs or those it had."""
    T, bounds = BAD_BOUNDS[name]
    n = len(bounds) - 1
    falls = any(b < a for a, b in zip(bounds, bounds[1:]))
    case = Case(name, 3, 1, 24, 32, (T,), "bf16", rows=n + 2)
    r = layer_rows(case)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    seqs = torch.arange(n, 0, -1, dtype=torch.int32, device="cuda")
    on = torch.ones(n, dtype=torch.uint8, device="cuda") if resume == "all" else None
    conv, status = r["conv"].clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v, dt, a = out = tuple(torch.full(s, 7.0, device="cuda", dtype=d) for s, d in
                                 (((T, 1, 32), case.dtype), ((T, 1, 32), case.dtype), ((T, 3, 24), case.dtype),
                                  ((T, 3), torch.float32), ((T, 3), torch.float32)))
    lar.prompt_inputs(case.cfg(), conv, r["x"], r["raw"], r["w"], r["A"], cu, seqs=seqs, resume=on, out=out,
                      status=status)
    assert status.item() == _abi.DEV_SEQS
    good, held = good_sequences(bounds, T)
    old, new = f64(r["conv"]), f64(conv)
    same = lambda x: f64((x == 7).flatten(1).all(1)).astype(bool)  # noqa: E731
    untouched = [same(x) for x in out]
    for x in untouched:
        assert x[held == 0].all()
    if not falls:
        assert not any(x[held > 0].any() for x in untouched)
    written = ~np.any(untouched[:3], axis=0)  # some columns' block may pass over a token that another's serves
    for s in range(n):
        row = n - s
        if s not in good:
            assert np.array_equal(new[row], old[row])
            continue
        want = lo.prompt_inputs(f64(r["x"]), f64(r["raw"]), f64(r["w"]), None, None, f64(r["A"]), old,
                                bounds[s:s + 2], [row], None if on is None else [1])
        check_inputs(case, (q, k, v, dt, a, conv), want, np.isfinite(want[1][:, 0]) & (held == 1) & written)
        right = np.array_equal(new[row], want[3][row])
        assert right or (falls and np.array_equal(new[row], old[row]))
    assert np.array_equal(new[[0, n + 1]], old[[0, n + 1]])


def test_the_whole_path_without_tokens():
    """A step of a serving loop that has no prompt: every call takes it, and nothing changes."""
    case = Case("empty", 4, 2, 24, 32, (0,), "bf16", rows=3)
    cfg = case.cfg()
    layer = lar.Replay(cfg, lar.alloc_buffers(cfg, "cuda"))
    layer.buffers["S0"].normal_()
    r = layer_rows(case)
    S0, conv = layer.buffers["S0"].clone(), r["conv"].clone()
    cu, seqs, _ = packed(case)
    for n in (1, 0):  # a sequence without tokens (it keeps its state), and no sequence
        on = torch.ones(n, dtype=torch.uint8, device="cuda")
        q, k, v, dt, a = lar.prompt_inputs(cfg, conv, r["x"], r["raw"], r["w"], r["A"], cu[:n + 1], seqs=seqs[:n], resume=on)
        y = layer.prefill(q, k, v, dt, a, cu[:n + 1], seqs=seqs[:n], resume=on)
        o = lar.gated_norm(cfg, y, r["z"], torch.ones(case.H * case.P, device="cuda"), v=v,
                           D=torch.ones(case.H, device="cuda"))
        assert o.shape == (0, case.H * case.P) and o.dtype == case.dtype
    assert torch.equal(layer.buffers["S0"], S0) and torch.equal(conv, r["conv"]) and layer.check_status() == 0


@pytest.mark.parametrize("bounds", [[0, 10, 30, 61], [0, 10, 60, 30], [-1, 10, 30, 60]])
@pytest.mark.parametrize("ids", [True, False])
def test_a_prefill_that_skips_a_sequence_leaves_its_row(bounds, ids):
    """A continued sequence with bad bounds: its row's checkpoint, count and buffered entries
    stay, and decode goes on from them; the others' entries are folded."""
    case = Case("skip", 4, 2, 24, 32, (60,), "bf16", rows=3)
    cfg = lar.Config(batch=3, heads=4, groups=2, P=24, N=32, L=5)
    r = layer_rows(case)
    on = torch.ones(3, dtype=torch.uint8, device="cuda")
    bad = next(s for s in range(3) if not 0 <= bounds[s] <= bounds[s + 1] <= 60)
    rows = [2, 0, 1] if ids else [0, 1, 2]
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    seqs = torch.tensor(rows, dtype=torch.int32, device="cuda") if ids else None
    whole = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    q, k, v, dt, a = lar.prompt_inputs(cfg, r["conv"].clone(), r["x"], r["raw"], r["w"], r["A"], whole)
    token = [t[:3].contiguous() for t in (q, k, v, dt, a)]
    layers = []
    for _ in range(2):
        layer = lar.Replay(cfg, lar.alloc_buffers(cfg, "cuda"))
        layer.buffers["S0"].copy_(torch.linspace(-1, 1, layer.buffers["S0"].numel(), device="cuda").view_as(layer.buffers["S0"]))
        layer.step(*token)
        layer.step(*token)
        layers.append(layer)
    first, plain = layers
    first.prefill(q, k, v, dt, a, cu, seqs=seqs, resume=on)
    row = rows[bad]
    assert first.read_counts() == [2 if b == row else 0 for b in range(3)]
    assert torch.equal(first.buffers["S0"][row], plain.buffers["S0"][row])
    assert torch.equal(first.step(*token)[row], plain.step(*token)[row])


def test_the_inputs_of_a_verify_round_that_keeps_some_positions():
    """The rollback knows nothing of the convolution's state: put back, and brought forward by the
    kept positions alone, it is what those tokens leave one by one, and decoding goes on as if
    the others had never been."""
    H, G, P, N, B, n = 4, 2, 24, 32, 4, 5
    keep = [0, 2, 5, 1]
    cfg = lar.Config(batch=B, heads=H, groups=G, P=P, N=N, L=8, max_pos=n, io="f32")
    case = Case("verify", H, G, P, N, (n,) * B, "f32", rows=B)
    r = layer_rows(case)
    x, raw, w, A, conv = r["x"], r["raw"], r["w"], r["A"], r["conv"].clone()
    layer = lar.Replay(cfg, lar.alloc_buffers(cfg, "cuda"))
    S0 = 0.1 * torch.randn(B, H, P, N, device="cuda")
    layer.buffers["S0"].copy_(S0)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    on = torch.ones(2 * B, dtype=torch.uint8, device="cuda")
    before = conv.clone()
    ins = lar.prompt_inputs(cfg, conv, x, raw, w, A, i32([n * b for b in range(B + 1)]), resume=on[:B])
    layer.verify(*(t.unflatten(0, (B, n)) for t in ins))
    layer.rollback(i32(keep))
    moved = conv.clone()
    conv.copy_(before)
    cu = [0]
    for b in range(B):
        cu += [n * b + keep[b], n * (b + 1)]
    lar.prompt_inputs(cfg, conv, x, raw, w, A, i32(cu), seqs=i32([s for b in range(B) for s in (b, -1)]), resume=on)
    # the same tokens one by one, each sequence in a layer of its own
    one = lar.Config(batch=1, heads=H, groups=G, P=P, N=N, L=8, io="f32")
    last = layer_rows(Case("last", H, G, P, N, (1,) * B, "f32", seed=8))
    want = []
    for b in range(B):
        c, single = r["conv"][b:b + 1].clone(), lar.Replay(one, lar.alloc_buffers(one, "cuda"))
        single.buffers["S0"].copy_(S0[b:b + 1])
        for t in range(keep[b]):
            single.step_resident(single.append_inputs(c, x[n * b + t][None], raw[n * b + t][None], w, A)[0])
        assert torch.equal(conv[b], c[0])
        assert torch.equal(moved[b], c[0]) == (keep[b] == n)
        want.append(single.step_resident(single.append_inputs(c, last["x"][b:b + 1], last["raw"][b:b + 1], w, A)[0]))
    y = layer.step_resident(layer.append_inputs(conv, last["x"], last["raw"], w, A)[0])
    assert ro.relative_error(f64(y), f64(torch.cat(want))) <= 1e-5  # FP32, the same entries in other launches
    assert layer.read_counts() == [k + 1 for k in keep] and layer.check_status() == 0
