"""The scan of packed prompts against the float64 oracle.

Bound. Every output is a sum of terms Delta v k q times decays. The scan of the operands'
magnitudes, M, is the sum of the terms' magnitudes. In FP32 arithmetic a term passes at
most 2 roundings a token that it decays through (the product and the sum it joins) and
N + 8 for its own products and the dot product with q, so
    |error| <= (2 T + N + 8) 2^-24 M
for T tokens of a sequence. BF16 outputs add half a step of the result. A kernel that
feeds tensor cores splits an FP32 factor x into BF16 parts with a remainder of at most
2^-16 |x| (two parts) or 2^-23 |x| (three); outputs that are themselves rounded to BF16
are given 2^-14 M for their two factors so split."""

import dataclasses

import numpy as np
import pytest
import torch

import linear_attention_decode_replay_b200 as lar
from linear_attention_decode_replay_b200 import _abi
from layer_harness import HALF, U32, Case, assert_within, f64, packed, scan_inputs
from oracle import layer_oracle as lo

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

CASES = [
    Case("one_token", 2, 2, 16, 16, (1,), "f32"),
    Case("tiny", 2, 2, 16, 16, (37,), "f32"),
    Case("p8", 3, 1, 8, 16, (5, 130), "bf16"),
    Case("n32_odd", 6, 2, 24, 32, (7, 0, 129, 1), "bf16", resume="some", rows=6, lead=3, tail=5),
    Case("n64", 4, 4, 64, 64, (127, 128, 129), "bf16", resume="all"),
    Case("n64_p256", 2, 1, 256, 64, (70, 200), "bf16", resume="some"),
    Case("n128_p64", 8, 4, 64, 128, (300, 64, 256), "bf16", resume="some", rows=4),
    Case("n128_p64_shared", 8, 1, 64, 128, (1000,), "bf16", resume="all"),
    Case("n128_p80", 5, 5, 80, 128, (255, 2, 257), "bf16", resume="all", tail=200),
    Case("n128_p128", 4, 2, 128, 128, (640, 3), "bf16"),
    Case("f32_n128", 4, 2, 64, 128, (200, 0, 77), "f32", resume="some", rows=5, lead=1),
    Case("f32_p128", 2, 2, 128, 128, (140,), "f32", resume="all"),
    Case("f32_n64_p40", 2, 1, 40, 64, (33, 131), "f32"),
    Case("many_short", 4, 2, 64, 128, tuple(1 + i % 5 for i in range(70)), "bf16", resume="some", rows=80),
    Case("long", 2, 1, 64, 128, (5003,), "bf16", resume="all"),
    # more units than SMs: a block takes several, of sorted and of unsorted sequences
    Case("many_units", 16, 4, 64, 128, tuple(37 * i % 300 for i in range(40)), "bf16", resume="some", rows=41),
    Case("many_units_n32", 8, 8, 80, 32, tuple(1 + 53 * i % 290 for i in range(70)), "bf16", resume="some", rows=75),
    Case("long_several", 2, 2, 128, 128, (2900, 0, 1, 2561, 256, 129), "bf16", resume="some", rows=9, lead=4, tail=9),
    Case("long_n64", 3, 1, 24, 64, (1, 2000, 3333), "bf16", resume="some", rows=3),
    Case("long_f32", 1, 1, 32, 64, (3001, 40), "f32"),
]


def check(case, ins, got_y, got_S, want, mag, cu, seqs, resume):
    (y, S), (my, mS) = want, mag
    T = max(max(case.lens), 1)
    roundings = (2 * T + case.N + 8) * U32
    by = roundings * my + (HALF["bf16"] * np.abs(y) + 2.0 ** -14 * my if case.io == "bf16" else 0) + 1e-37
    live = np.zeros(case.T, bool)
    for _, t0, t1, _ in lo.rows_served(f64(cu), f64(seqs), case.batch):
        live[t0:t1] = True
    assert_within(f64(got_y)[live], y[live], by[live], f"{case.name}: y")
    assert_within(got_S, S, roundings * mS + 1e-37, f"{case.name}: S")
    return live


def run(case, ins, max_len=0, **kw):
    q, k, v, dt, a, S = ins
    cu, seqs, resume = packed(case)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S = S.clone()
    y = torch.full((case.T, case.H, case.P), 7.0, device="cuda", dtype=case.dtype)
    out = lar.prompt_scan(case.cfg(), S, q, k, v, dt, a, cu, seqs=seqs, resume=resume, y=y, max_len=max_len,
                          status=status, **kw)
    assert out is y and status.item() == 0
    return y, S, cu, seqs, resume


def oracle(ins, cu, seqs, resume):
    args = [f64(t) for t in ins] + [f64(cu), f64(seqs), f64(resume)]
    return lo.prompt_scan(*args), lo.prompt_scan_magnitude(*args)


@pytest.mark.parametrize("case", CASES, ids=[c.name for c in CASES])
def test_scan_matches_the_oracle(case):
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins)
    want, mag = oracle(ins, cu, seqs, resume)
    live = check(case, ins, y, S, want, mag, cu, seqs, resume)
    assert (y[torch.from_numpy(~live).cuda()] == 7).all()  # tokens outside every sequence
    y2, S2, *_ = run(case, ins, max_len=max(case.lens))
    check(case, ins, y2, S2, want, mag, cu, seqs, resume)
    y3, S3, *_ = run(case, ins)  # bit for bit the same again
    assert torch.equal(y, y3) and torch.equal(S, S3)


@pytest.mark.parametrize("decay", [0.0, 1.0, 0.999, -0.5, 1e-30])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_with_constant_decay(decay, io):
    """Forgetting everything (a = 0: no logarithm of it may be taken), nothing, and decays of
    either sign; products that underflow."""
    case = Case("decay", 2, 1, 64, 128, (300, 20), io, resume="all")
    ins = scan_inputs(case, decay=decay)
    ins[3] = ins[3].clone()
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


def test_steps_of_zero_and_mixed_decays():
    case = Case("mixed", 3, 3, 64, 64, (400,), "bf16", resume="all", seed=4)
    ins = scan_inputs(case)
    dt, a = ins[3], ins[4]
    dt[::7] = 0
    a[5::50] = 0
    a[::3] = 1
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "dt", "a"])
def test_bad_values_reach_only_what_follows_them(io, bad, what):
    """A NaN or an infinity at one token leaves the tokens before it, the other sequences and
    the other heads as they were."""
    case = Case("bad", 2, 2, 64, 128, (150, 200, 130), io, resume="all", seed=2)
    ins = scan_inputs(case)
    y0, S0, cu, seqs, resume = run(case, ins)
    t = 150 + 77  # token 77 of sequence 1, head 0
    x = [t_.clone() for t_ in ins]
    x["q k v dt a".split().index(what)][(t, 0, 5) if what in "qkv" else (t, 0)] = bad
    y1, S1, *_ = run(case, x)
    same = torch.ones(case.T, case.H, dtype=torch.bool, device="cuda")
    same[t:350, 0] = False
    assert torch.equal(y0[same], y1[same])
    assert torch.equal(S0[[0, 2]], S1[[0, 2]]) and torch.equal(S0[1, 1], S1[1, 1])
    want, _ = lo.prompt_scan(*[f64(i) for i in x], f64(cu), f64(seqs), f64(resume))
    got = f64(y1)
    assert np.array_equal(np.isfinite(got[t:350, 0]), np.isfinite(want[t:350, 0]))


def test_values_not_finite_everywhere_in_v():
    """Many of them, in every column and chunk: each output that one reaches is not finite, and
    no other changes."""
    case = Case("nan_v", 2, 1, 64, 128, (300,), "bf16", seed=9)
    ins = scan_inputs(case)
    y0, S0, cu, seqs, resume = run(case, ins)
    x = [t.clone() for t in ins]
    g = torch.Generator().manual_seed(1)
    first = torch.randint(0, 400, (case.H, case.P), generator=g)  # from this token on
    bad = torch.arange(case.T)[:, None, None] >= first[None]
    x[2][bad.cuda()] = float("nan")
    y1, S1, *_ = run(case, x)
    assert torch.equal(torch.isfinite(y1).cpu(), ~bad)
    assert torch.equal(y1[~bad.cuda()], y0[~bad.cuda()])
    assert torch.equal(torch.isfinite(S1[0]).all(-1).cpu(), first >= case.T)


def test_padding_and_bad_ids_are_skipped():
    case = Case("ids", 2, 1, 32, 32, (10, 20, 30, 40, 50), "bf16", resume="all")
    q, k, v, dt, a, S = ins = scan_inputs(case)
    cu, _, resume = packed(case)
    seqs = torch.tensor([3, -1, 3, 99, 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((case.T, case.H, case.P), 7.0, device="cuda", dtype=case.dtype)
    S1 = S.clone()
    lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, seqs=seqs, resume=resume, y=y, status=status)
    assert status.item() == _abi.DEV_SEQS
    live = check(case, ins, y, S1, *oracle(ins, cu, seqs, resume), cu, seqs, resume)
    assert live.sum() == 60 and (y[torch.from_numpy(~live).cuda()] == 7).all()
    status.zero_()
    lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, seqs=torch.tensor([3, -1, -1, 1, 0], dtype=torch.int32,
                                                                          device="cuda"), status=status)
    assert status.item() == 0  # padding alone is no error


def test_bad_bounds_are_skipped():
    case = Case("bounds", 2, 1, 32, 32, (10, 20, 30), "bf16")
    q, k, v, dt, a, S = scan_inputs(case)
    for bounds in ([0, 10, 5, 60], [-4, 10, 30, 60], [0, 10, 30, 61]):
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        S1 = S.clone()
        y = lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, status=status)
        assert status.item() == _abi.DEV_SEQS
        bad = [i for i in range(3) if bounds[i] < 0 or bounds[i + 1] < bounds[i] or bounds[i + 1] > case.T]
        for i in range(3):
            assert torch.equal(S1[i], S[i]) == (i in bad)
        assert y.shape == (case.T, case.H, case.P)


def test_no_tokens_and_no_sequences():
    case = Case("none", 2, 1, 32, 32, (0, 0), "bf16", resume="some")
    q, k, v, dt, a, S = scan_inputs(case)
    cu, seqs, resume = packed(case)
    S1 = S.clone()
    y = lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, resume=resume)
    assert y.shape[0] == 0 and torch.equal(S1[0], S[0]) and (S1[1] == 0).all()
    S1 = S.clone()
    lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu[:1])
    assert torch.equal(S1, S)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_prompt_in_pieces_is_the_prompt(io):
    """Fed in pieces through the state, a prompt ends where it ends fed at once: each way
    within its bound of the oracle."""
    whole = Case("whole", 4, 2, 64, 128, (700,), io)
    ins = scan_inputs(whole)
    q, k, v, dt, a, S = ins
    S = S.clone()
    on = torch.ones(1, dtype=torch.uint8, device="cuda")
    ys, at = [], 0
    for i, n in enumerate((300, 1, 128, 271)):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        part = [t[at:at + n].contiguous() for t in (q, k, v, dt, a)]
        ys.append(lar.prompt_scan(whole.cfg(), S, *part, cu, resume=on if i else None))
        at += n
    cu, seqs, resume = packed(whole)
    check(whole, ins, torch.cat(ys), S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


def test_scan_on_another_stream_and_in_a_graph():
    case = Case("graph", 4, 2, 64, 128, (900, 33), "bf16", resume="all")
    q, k, v, dt, a, S = ins = scan_inputs(case)
    y0, S0, cu, seqs, resume = run(case, ins)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    S1 = S.clone()
    torch.cuda.synchronize()
    y1 = lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, resume=resume, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(S0, S1)
    # two captured calls, replayed twice on new contents, with an eager call between
    graphs, outs = [], []
    Sg = [S.clone(), S.clone()]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lar.prompt_scan(case.cfg(), Sg[i], q, k, v, dt, a, cu, resume=resume))
        graphs.append(g)
    for _ in range(2):
        for i in range(2):
            Sg[i].copy_(S)
        graphs[0].replay()
        y2, S2, *_ = run(case, ins)
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], y0) and torch.equal(Sg[i], S0)
        assert torch.equal(y2, y0) and torch.equal(S2, S0)
    # other lengths in the same buffers
    other = dataclasses.replace(case, lens=(33, 900))
    cu.copy_(packed(other)[0])
    Sg[0].copy_(S)
    graphs[0].replay()
    torch.cuda.synchronize()
    want, mag = oracle(ins, cu, None, resume)
    check(other, ins, outs[0], Sg[0], want, mag, cu, None, resume)


@pytest.mark.parametrize("P", [8, 40])
@pytest.mark.parametrize("length", [1, 29, 30, 31, 32])
def test_lengths_on_both_sides_of_the_choice_of_kernel(length, P):
    """Short BF16 sequences go token by token, longer ones in chunks: the same bounds for both."""
    case = Case("choice", 4, 2, P, 128, (length,) * 3, "bf16", resume="some", seed=length)
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


@pytest.mark.parametrize("max_len", [1, 128, 10 ** 9])
def test_a_wrong_longest_length_only_steers(max_len):
    case = Case("estimate", 2, 1, 64, 128, (1500, 3), "bf16", resume="all")
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins, max_len=max_len)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


@pytest.mark.parametrize("resume", ["none", "all"])
@pytest.mark.parametrize("bounds", [[0, 5000, 100, 4900, 5000], [0, 2500, 0, 5000, 7000, 5000], [5000, 0, 5000, 0, 5000]])
def test_long_sequences_beside_bad_bounds(bounds, resume):
    """Long sequences are cut into segments, and sequences that share tokens have more of them
    than the tokens allow: each sequence with good bounds still ends in its own state."""
    n = len(bounds) - 1
    case = Case("fall", 2, 1, 64, 128, (5000,), "bf16", rows=n)
    q, k, v, dt, a, S = ins = scan_inputs(case)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    on = torch.ones(n, dtype=torch.uint8, device="cuda") if resume == "all" else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S1 = S.clone()
    y = lar.prompt_scan(case.cfg(), S1, q, k, v, dt, a, cu, resume=on, status=status)
    assert status.item() == _abi.DEV_SEQS
    good = [s for s in range(n) if 0 <= bounds[s] <= bounds[s + 1] <= case.T]
    held = sum(((np.arange(case.T) >= bounds[s]) & (np.arange(case.T) < bounds[s + 1])).astype(int) for s in good)
    for s in range(n):
        if s not in good:
            assert torch.equal(S1[s], S[s])
            continue
        args = [f64(t) for t in ins] + [bounds[s:s + 2], [s], None if on is None else [1]]
        (wy, wS), (my, mS) = lo.prompt_scan(*args), lo.prompt_scan_magnitude(*args)
        roundings = (2 * (bounds[s + 1] - bounds[s]) + case.N + 8) * U32
        assert_within(S1[s], wS[s], roundings * mS[s] + 1e-37, f"S of {s}")
        alone = np.isfinite(wy[:, 0, 0]) & (held == 1)
        by = (roundings + 2.0 ** -14) * my + HALF["bf16"] * np.abs(wy) + 1e-37
        assert_within(f64(y)[alone], wy[alone], by[alone], f"y of {s}")


def token_by_token(case, ins, S):
    """Whether a BF16 scan with final states S went token by token: then its states are bit for
    bit those of the FP32 scan (which always does) of the same values. Chunks sum otherwise."""
    wide = dataclasses.replace(case, io="f32")
    x = [t.float() for t in ins]
    return torch.equal(run(wide, x)[1], S)


@pytest.mark.parametrize("P", [8, 40, 64, 128])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [(7,), (8, 8, 8), (9, 1, 0, 8, 17), (30, 29, 16, 15, 24, 25)], ids=str)
def test_short_bf16_sequences_token_by_token(N, P, lens):
    """Around the stages of 8 tokens and the batches of 4, with state rows that fill the blocks of
    32 to 256 and that do not. Everything is FP32 until the outputs are rounded."""
    case = Case("short", 4, 2, P, N, lens, "bf16", resume="some", rows=len(lens) + 2, seed=N + P, lead=1, tail=3)
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins, max_len=max(lens))
    assert token_by_token(case, ins, S)
    want, mag = oracle(ins, cu, seqs, resume)
    live = check(case, ins, y, S, want, mag, cu, seqs, resume)
    by = (2 * max(lens) + N + 8) * U32 * mag[0] + HALF["bf16"] * np.abs(want[0]) + 1e-37  # no parts
    assert_within(f64(y)[live], want[0][live], by[live], "y")
    assert (y[torch.from_numpy(~live).cuda()] == 7).all()


@pytest.mark.parametrize("N", [16, 64, 128])
@pytest.mark.parametrize("length,serial", [(1, True), (29, True), (30, True), (31, False), (32, False)])
def test_the_choice_of_kernel_by_the_longest_length(N, length, serial):
    case = Case("side", 4, 2, 40, N, (length,) * 3, "bf16", resume="some", seed=length)
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins, max_len=length)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)
    assert token_by_token(case, ins, S) == serial


@pytest.mark.parametrize("lens,decay", [((300, 20), 1.2), ((300, 20), -1.1), ((100, 120), 2.0), ((128, 129), 1.9),
                                        ((3000,), 1.01), ((3000, 17), -1.02)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_with_decays_above_one(io, lens, decay):
    """States that grow, up to 2^124 of what came in: the products of a chunk's and a segment's
    decays stay inside FP32's range, and the bounds are those of any decay."""
    case = Case("grow", 2, 1, 64, 128, lens, io, resume="all")
    ins = scan_inputs(case, decay=decay)
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


def test_scan_with_decays_on_both_sides_of_one():
    case = Case("both", 4, 2, 40, 64, (2900, 300), "bf16", resume="some", rows=3)
    ins = scan_inputs(case)
    g = torch.Generator(device="cuda").manual_seed(6)
    ins[4] = 0.6 + 0.7 * torch.rand(ins[4].shape, generator=g, device="cuda")
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "dt", "a"])
@pytest.mark.parametrize("at", [0, 1000, 4000, 5002])
def test_bad_values_in_a_sequence_of_segments(bad, what, at):
    """As in a short sequence: the tokens before, the other sequence and the other head stay as
    they were, and the same outputs and state elements are finite as in the definition."""
    case = Case("bad_long", 2, 2, 64, 128, (5003, 40), "bf16", resume="all", seed=3)
    ins = scan_inputs(case)
    y0, S0, cu, seqs, resume = run(case, ins)
    x = [t.clone() for t in ins]
    x["q k v dt a".split().index(what)][(at, 0, 5) if what in "qkv" else (at, 0)] = bad
    y1, S1, *_ = run(case, x)
    same = torch.ones(case.T, case.H, dtype=torch.bool, device="cuda")
    same[at:5003, 0] = False
    assert torch.equal(y0[same], y1[same])
    assert torch.equal(S0[1], S1[1]) and torch.equal(S0[0, 1], S1[0, 1])
    want, wS = lo.prompt_scan(*[f64(i) for i in x], f64(cu), f64(seqs), f64(resume))
    assert np.array_equal(np.isfinite(f64(y1)), np.isfinite(want))
    assert np.array_equal(np.isfinite(f64(S1)), np.isfinite(wS))


@pytest.mark.parametrize("case", [
    Case("one_of_many", 16, 4, 64, 128, (300,) + (0,) * 63, "bf16", resume="some", rows=64),
    Case("every_fifth", 16, 4, 64, 128, tuple(0 if i % 5 else 50 + i for i in range(100)), "bf16", resume="some", rows=101),
    Case("every_third", 16, 2, 128, 64, tuple(0 if i % 3 else 150 for i in range(48)), "bf16", resume="all", rows=48),
    Case("few_tokens", 6, 2, 256, 16, (3, 3, 1, 5, 0, 17, 0, 0, 2, 0, 2, 0, 1, 56, 1, 2, 6, 11, 0, 2, 1, 2, 8, 0, 1), "bf16",
         resume="some", lead=26),
    Case("long_and_empty", 2, 1, 64, 128, (3000,) + (0,) * 40, "bf16", resume="some", rows=41),
], ids=lambda c: c.name)
def test_many_sequences_without_tokens(case):
    """A batch's empty places: a block takes several units without a chunk one after another, and
    goes on; empty sequences keep their rows or make them zero."""
    ins = scan_inputs(case)
    y, S, cu, seqs, resume = run(case, ins)
    check(case, ins, y, S, *oracle(ins, cu, seqs, resume), cu, seqs, resume)
    again, S2, *_ = run(case, ins, max_len=max(case.lens))
    check(case, ins, again, S2, *oracle(ins, cu, seqs, resume), cu, seqs, resume)
