"""The measured calls of a layer's operators around the decode path: what a prompt goes
through before its first decode step, and what a single token needs around that step.

* ``inputs``: the short causal convolution with SiLU over the projection's rows, split
  into v, k and q, and the step sizes and decays (Delta, a), for packed prompts.
* ``token``: the same for one token per sequence, from and to the convolution's state.
* ``scan``: the selective state space scan over packed prompts, outputs and final states.
* ``norm``: skip term, gate and grouped RMS norm of a layer's outputs.

``run`` computes them in elementary torch operations, or, with ``own`` set, through the
package's entry points. Sizes are the decode layer's (64 heads of 64 x 128 with 64 or 8
k/q groups, 32 heads of 128 x 128, the tiny 16 x 16 layer) and the batches it is run at.
"""

import math

import torch

own = False

DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # the tiny layer on one short prompt: a call's fixed cost
        dict(name="scan_tiny", op="scan", io="f32", seqs=1, tokens=37, H=2, G=2, P=16, N=16, resume=False),
        # a serving batch of eight prompts of unequal length into the 64-head layer
        dict(name="scan_prompts", op="scan", io="bf16", seqs=8, tokens=8192, H=64, G=64, P=64, N=128, resume=False),
        # one long document into the layer whose heads share k and q by eights
        dict(name="scan_long", op="scan", io="bf16", seqs=1, tokens=32768, H=64, G=8, P=64, N=128, resume=False),
        # prompts continued from their states (a prompt fed in pieces), tall heads, an odd total
        dict(name="scan_resumed", op="scan", io="bf16", seqs=5, tokens=5003, H=32, G=32, P=128, N=128, resume=True),
        # FP32 inputs, heads sharing k and q
        dict(name="scan_f32", op="scan", io="f32", seqs=4, tokens=2050, H=64, G=8, P=64, N=128, resume=True),
        # the convolution over the same serving batch, every channel of the 64-group layer
        dict(name="inputs_prompts", op="inputs", io="bf16", seqs=8, tokens=8192, H=64, G=64, P=64, N=128, width=4, resume=False),
        # a verify round's five positions of 256 sequences: short pieces, each from its state
        dict(name="inputs_pieces", op="inputs", io="bf16", seqs=256, tokens=1280, H=64, G=8, P=64, N=128, width=4, resume=True),
        # FP32 rows, a shorter filter, an odd total
        dict(name="inputs_f32", op="inputs", io="f32", seqs=3, tokens=1999, H=32, G=8, P=128, N=128, width=3, resume=True),
        # one decode token of the serving batch
        dict(name="token_b256", op="token", io="bf16", seqs=256, H=64, G=64, P=64, N=128, width=4),
        # one decode token of one sequence: a call's fixed cost
        dict(name="token_b1", op="token", io="bf16", seqs=1, H=64, G=8, P=64, N=128, width=4),
        # the outputs of a prompt batch, normed over the whole row
        dict(name="norm_prompts", op="norm", io="bf16", y="bf16", tokens=16384, H=64, P=64, groups=1, skip=True),
        # a decode step's FP32 outputs, normed over eight groups
        dict(name="norm_b256", op="norm", io="bf16", y="f32", tokens=256, H=64, P=64, groups=8, skip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _fit(c):
    """The drawn case, cut to no more than the largest listed one's work."""
    while work(c)["bytes"] > 5e8:
        c.update({n: (c[n] + 1) // 2 for n in ("tokens", "seqs") if n in c})
    return c


def draw(rng):
    op = rng.choice(["scan", "scan", "inputs", "token", "norm"])
    P, N = rng.choice([(64, 128), (64, 128), (128, 128), (64, 64), (32, 32), (16, 16), (8, 128), (24, 64), (80, 128), (256, 64)])
    H = rng.choice([1, 2, 5, 8, 16, 20, 32, 64])
    G = rng.choice([g for g in (1, 2, 4, 5, 8, 16, 20, 32, 64) if H % g == 0])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        P = rng.choice([8, 16, 32, 64, 128])
        groups = rng.choice([g for g in (1, 2, 4, 8, H) if H % g == 0])
        return _fit(dict(op=op, io=io, y=rng.choice(["f32", io]), tokens=_log(rng, 1, 12000), H=H, P=P, groups=groups, skip=rng.random() < 0.7))
    if op == "token":
        return _fit(dict(op=op, io=io, seqs=_log(rng, 1, 300), H=H, G=G, P=P, N=N, width=rng.choice([2, 3, 4, 4])))
    most = 16000 if op == "scan" else 8000
    tokens = _log(rng, 1, most)
    seqs = min(_log(rng, 1, 64), tokens)
    c = dict(op=op, io=io, seqs=seqs, tokens=tokens, H=H, G=G, P=P, N=N, resume=rng.random() < 0.5)
    if op == "inputs":
        c["width"] = rng.choice([2, 3, 4, 4])
    return _fit(c)


def _lengths(case, g):
    """Lengths of the packed sequences: unequal shares of the tokens, or, where there are
    only a few tokens a sequence, equal ones."""
    S, T = case["seqs"], case["tokens"]
    if T <= 8 * S:
        return [T // S + (1 if s < T % S else 0) for s in range(S)]
    share = torch.rand(S, generator=g) + 0.25
    cuts = (torch.cumsum(share, 0) / share.sum() * T).round().long().tolist()
    cuts[-1] = T
    return [b - a for a, b in zip([0] + cuts[:-1], cuts)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    t = IO[case["io"]]
    op, H, P = case["op"], case["H"], case["P"]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": case}
    if op == "norm":
        T = case["tokens"]
        s["y"] = randn(T, H, P).to(IO[case["y"]])
        s["proj"] = randn(T, H * P + 64).to(t)  # the gate is a slice of the projection's rows
        s["weight"] = 1 + 0.1 * randn(H * P)
        s["v"] = randn(T, H, P).to(t) if case["skip"] else None
        s["D"] = 1 + 0.1 * randn(H) if case["skip"] else None
        return s
    S, G, N = case["seqs"], case["G"], case["N"]
    s["A"] = 0.5 + 1.5 * rand(H)
    # step sizes from 0.002 to about 1, as trained layers hold them: slow and fast heads
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(math.log(0.002) + rand(H) * (math.log(0.8) - math.log(0.002)))))
    if op != "token":
        cpu = torch.Generator().manual_seed(int(seed))
        s["lens"] = _lengths(case, cpu)
        cu = [0]
        cu.extend(torch.tensor(s["lens"]).cumsum(0).tolist())
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["rows"] = torch.randperm(S, generator=cpu).to(torch.int32).to(DEV)  # sequence i owns row rows[i] of the state
        s["resume"] = torch.ones(S, dtype=torch.uint8, device=DEV) if case["resume"] else None
    if op == "scan":
        T = case["tokens"]
        q, k = randn(T, G, N), randn(T, G, N)
        s["q"], s["k"] = (q / q.norm(dim=-1, keepdim=True)).to(t), (k / k.norm(dim=-1, keepdim=True)).to(t)
        s["v"] = randn(T, H, P).to(t)
        s["dt"] = torch.nn.functional.softplus(randn(T, H) + s["dt_bias"])
        s["a"] = torch.exp(-s["dt"] * s["A"])
        s["S"] = 0.1 * randn(S, H, P, N)
        return s
    rows = case["tokens"] if op == "inputs" else S
    D = H * P + 2 * G * N
    # the projection's rows: gate | v k q channels | step sizes, padded to whole 16 bytes
    width = H * P + D + H + (-H) % 8
    s["proj"] = randn(rows, width).to(t)
    s["w"] = (rand(case["width"], D) - 0.5) * (2 / math.sqrt(case["width"]))
    s["bias"] = 0.1 * randn(D)
    s["conv"] = randn(S, case["width"] - 1, D).to(t)
    return s


def _channels(s):
    """The convolution's channels and the raw step sizes, as views of the projection's rows."""
    c = s["case"]
    at = c["H"] * c["P"]
    D = at + 2 * c["G"] * c["N"]
    return s["proj"][:, at : at + D], s["proj"][:, at + D : at + D + c["H"]]


def _split(c, x):
    """Convolved rows [T][D] into q, k [T][G][N] and v [T][H][P]."""
    at, kn = c["H"] * c["P"], c["G"] * c["N"]
    q, k, v = x[:, at + kn :], x[:, at : at + kn], x[:, :at]
    return q.reshape(-1, c["G"], c["N"]), k.reshape(-1, c["G"], c["N"]), v.reshape(-1, c["H"], c["P"])


def _layer(c, **kw):
    import linear_attention_decode_replay_b200 as lar

    return lar, lar.Config(batch=c.get("seqs", 1), heads=c["H"], groups=c.get("G", 1), P=c["P"], N=c.get("N", 16), L=1, io=c["io"], **kw)


# ------------------------------------------------------------------------ the operators
def _steps(raw, s):
    """Delta = softplus(raw + bias) and a = exp(-Delta A)."""
    x = raw.float() + s["dt_bias"]
    dt = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    return dt, torch.exp(-dt * s["A"])


def _taps(s, x):
    """Rows that the filter's taps reach from each token, as indexes into the stacked rows
    [x | state | zero], and those of the new state."""
    c, cu = s["case"], s["cu"].long()
    T, S, K = c["tokens"], c["seqs"], c["width"] - 1
    ids = torch.arange(S, device=DEV)
    seq = torch.repeat_interleave(ids, cu[1:] - cu[:-1], output_size=T)
    start, row = cu[:-1], s["rows"].long()

    def at(pos, seq):  # the stacked row of position `pos` [.., taps] of sequence `seq`
        back = pos - start[seq][:, None]
        old = T + row[seq][:, None] * K + (back + K) if s["resume"] is not None else torch.full_like(pos, T + S * K)
        return torch.where(back >= 0, pos, old)

    taps = at(torch.arange(T, device=DEV)[:, None] + torch.arange(-K, 1, device=DEV), seq)
    new = at(cu[1:][:, None] + torch.arange(-K, 0, device=DEV), ids)
    return taps, new, row


def _inputs(s):
    c = s["case"]
    x, raw = _channels(s)
    taps, new, row = _taps(s, x)
    stacked = torch.cat([x, s["conv"].reshape(-1, x.shape[1]), torch.zeros_like(x[:1])])
    acc = sum(stacked[taps[:, i]].float() * s["w"][i] for i in range(c["width"])) + s["bias"]
    y = (acc / (1 + torch.exp(-acc))).to(x.dtype)
    s["conv"][row] = stacked[new]
    return *_split(c, y), *_steps(raw, s), s["conv"]


def _token(s):
    c = s["case"]
    x, raw = _channels(s)
    seen = torch.cat([s["conv"], x[:, None]], 1)
    acc = (seen.float() * s["w"]).sum(1) + s["bias"]
    y = (acc / (1 + torch.exp(-acc))).to(x.dtype)
    s["conv"].copy_(seen[:, 1:])
    return *_split(c, y), *_steps(raw, s), s["conv"]


def _scan(s, Q=64):
    """The scan in chunks of Q tokens: products within a chunk, and a weighted sum of the
    chunks before it. Decays are differences of summed logarithms, held in 64 bits."""
    c = s["case"]
    T, H, G, P, N = c["tokens"], c["H"], c["G"], c["P"], c["N"]
    lens = torch.tensor(s["lens"], device=DEV)
    chunks = (lens + Q - 1) // Q
    C = sum((n + Q - 1) // Q for n in s["lens"])
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device=DEV), chunks, output_size=C)
    nth = torch.arange(C, device=DEV) - (torch.cumsum(chunks, 0) - chunks)[seq]
    pos = nth[:, None] * Q + torch.arange(Q, device=DEV)
    live = pos < lens[seq][:, None]
    tok = torch.where(live, s["cu"].long()[seq][:, None] + pos, T)  # token T: a row of zeros
    pad = lambda x: torch.cat([x.float(), torch.zeros_like(x[:1]).float()])[tok]  # noqa: E731
    q, k, v, dt = pad(s["q"]), pad(s["k"]), pad(s["v"]), pad(s["dt"])
    la = torch.cat([torch.log(s["a"].double()), torch.zeros(1, H, device=DEV, dtype=torch.float64)])[tok]
    cum = torch.cumsum(la, 1).permute(2, 0, 1)  # [H][C][Q]
    total = cum[:, :, -1]
    w = dt.permute(2, 0, 1)
    causal = torch.ones(Q, Q, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp((cum[:, :, :, None] - cum[:, :, None, :]).masked_fill(~causal, -math.inf)).float()
    qk = torch.einsum("cign,cjgn->gcij", q, k).repeat_interleave(H // G, 0)
    vh = v.permute(2, 0, 1, 3)  # [H][C][Q][P]
    kh = k.permute(2, 0, 1, 3).repeat_interleave(H // G, 0)
    qh = q.permute(2, 0, 1, 3).repeat_interleave(H // G, 0)
    y = torch.matmul(qk * decay * w[:, :, None, :], vh)
    to_end = (torch.exp(total[:, :, None] - cum).float() * w)[..., None]
    local = torch.matmul((vh * to_end).transpose(2, 3), kh)  # [H][C][P][N]: each chunk's own state
    # chunk d reaches chunk e > d of its sequence through the decays of the chunks between
    upto = torch.cumsum(total, 1)
    before = (seq[:, None] == seq[None, :]) & (torch.arange(C, device=DEV)[:, None] > torch.arange(C, device=DEV)[None, :])
    reach = torch.exp((upto[:, :, None] - total[:, :, None] - upto[:, None, :]).masked_fill(~before, -math.inf)).float()
    came = torch.matmul(reach, local.reshape(H, C, P * N)).reshape(H, C, P, N)
    row = s["rows"].long()
    if s["resume"] is not None:
        first = torch.cumsum(chunks, 0) - chunks
        since = torch.exp(upto - total - (upto - total)[:, first[seq]]).float()
        came = came + since[..., None, None] * s["S"][row[seq]].transpose(0, 1)
    y = y + torch.exp(cum).float()[..., None] * torch.matmul(qh, came.transpose(2, 3))
    out = torch.empty(T, H, P, device=DEV)
    out[tok[live]] = y.permute(1, 2, 0, 3)[live]
    last = torch.cumsum(chunks, 0) - 1
    s["S"][row] = (torch.exp(total)[..., None, None].float() * came + local)[:, last].transpose(0, 1)
    return out.to(s["v"].dtype), s["S"]


def _norm(s):
    c = s["case"]
    T, H, P = c["tokens"], c["H"], c["P"]
    z = s["proj"][:, : H * P].float()
    y = s["y"].float()
    if c["skip"]:
        y = y + s["D"][:, None] * s["v"].float()
    u = y.reshape(T, H * P) * (z / (1 + torch.exp(-z)))
    u = u.reshape(T, c["groups"], -1)
    u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
    return (u.reshape(T, H * P) * s["weight"]).to(s["proj"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"inputs": _inputs, "token": _token, "scan": _scan, "norm": _norm}[c["op"]](s)
    lar, cfg = _layer(c)
    if c["op"] == "norm":
        return lar.gated_norm(cfg, s["y"], s["proj"][:, : c["H"] * c["P"]], s["weight"], v=s["v"], D=s["D"], norm_groups=c["groups"], eps=EPS)
    if c["op"] == "scan":
        y = lar.prompt_scan(cfg, s["S"], s["q"], s["k"], s["v"], s["dt"], s["a"], s["cu"], seqs=s["rows"], resume=s["resume"], max_len=max(s["lens"]))
        return y, s["S"]
    x, raw = _channels(s)
    if c["op"] == "token":
        return *lar.token_inputs(cfg, s["conv"], x, raw, s["w"], s["A"], bias=s["bias"], dt_bias=s["dt_bias"]), s["conv"]
    return *lar.prompt_inputs(cfg, s["conv"], x, raw, s["w"], s["A"], s["cu"], bias=s["bias"], dt_bias=s["dt_bias"], seqs=s["rows"], resume=s["resume"]), s["conv"]


def work(case):
    c = case
    b = 2 if c["io"] == "bf16" else 4
    H, P = c["H"], c["P"]
    if c["op"] == "norm":
        n = c["tokens"] * H * P
        return {"bytes": n * ((2 if c["y"] == "bf16" else 4) + b * (3 if c["skip"] else 2)) + 4 * H * P, "flops": n * 10}
    S, G, N = c["seqs"], c["G"], c["N"]
    if c["op"] == "scan":
        T = c["tokens"]
        state = S * H * P * N * 4 * (2 if c["resume"] else 1)
        return {"bytes": T * (2 * G * N * b + 2 * H * P * b + 8 * H) + state, "flops": T * H * 5 * P * N}
    D, K = H * P + 2 * G * N, c["width"] - 1
    rows = S if c["op"] == "token" else c["tokens"]
    state = S * K * D * b * (2 if c["op"] == "token" or c["resume"] else 1)
    return {"bytes": rows * (2 * D * b + H * (b + 8)) + state + 4 * D * (K + 2), "flops": rows * (D * (2 * c["width"] + 4) + 10 * H)}


# ------------------------------------------------------------------- the definitions
def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    c = case
    H, P = c["H"], c["P"]
    if c["op"] == "norm":
        y = f["y"] + (f["D"].view(1, H, 1) * f["v"] if c["skip"] else 0)
        u = y.flatten(1) * torch.nn.functional.silu(f["proj"][:, : H * P])
        u = torch.stack([torch.nn.functional.rms_norm(x, x.shape[-1:], eps=EPS) for x in u.chunk(c["groups"], 1)], 1)
        return u.flatten(1) * f["weight"]
    if c["op"] == "scan":
        return _exact_scan(c, f)
    G, N, K = c["G"], c["N"], c["width"] - 1
    D = H * P + 2 * G * N
    x, raw = f["proj"][:, H * P : H * P + D], f["proj"][:, H * P + D : H * P + D + H]
    conv = f["conv"].clone()
    lens = s["lens"] if c["op"] == "inputs" else [1] * c["seqs"]
    rows = s["rows"].tolist() if c["op"] == "inputs" else list(range(c["seqs"]))
    out, at = [], 0
    for n, r in zip(lens, rows):
        old = conv[r] if c["op"] == "token" or c["resume"] else torch.zeros_like(conv[r])
        full = torch.cat([old, x[at : at + n]])
        acc = torch.nn.functional.conv1d(full.t()[None], f["w"].t()[:, None], f["bias"], groups=D)[0].t()
        out.append(torch.nn.functional.silu(acc))
        conv[r] = full[n:]
        at += n
    y = torch.cat(out)
    dt = torch.logaddexp(raw + f["dt_bias"], torch.zeros((), device=DEV, dtype=torch.float64))
    v, k, q = y.split([H * P, G * N, G * N], 1)
    return q.reshape(-1, G, N), k.reshape(-1, G, N), v.reshape(-1, H, P), dt, torch.exp(-dt * f["A"]), conv


def _exact_scan(c, f):
    H, G, P, N, S = c["H"], c["G"], c["P"], c["N"], c["seqs"]
    longest = max(f["lens"])
    if longest * S * H * P * N > 2e11:
        return None  # tens of thousands of steps over many states: longer than it is worth
    cu, rows = f["cu"].long(), f["rows"].long()
    lens = cu[1:] - cu[:-1]
    state = f["S"][rows].clone() if c["resume"] else torch.zeros(S, H, P, N, device=DEV, dtype=torch.float64)
    y = torch.zeros(c["tokens"] + 1, H, P, device=DEV, dtype=torch.float64)
    # token t of every sequence at once; a sequence that has ended neither decays nor adds
    zero = lambda x: torch.cat([x, torch.zeros_like(x[:1])])  # noqa: E731
    q, k, v, dt, a = zero(f["q"]), zero(f["k"]), zero(f["v"]), zero(f["dt"]), f["a"]
    a = torch.cat([a, torch.ones_like(a[:1])])
    for t in range(longest):
        i = torch.where(t < lens, cu[:-1] + t, c["tokens"])
        kt, qt = k[i].repeat_interleave(H // G, 1), q[i].repeat_interleave(H // G, 1)
        state.mul_(a[i][..., None, None]).addcmul_((dt[i][..., None] * v[i])[..., None], kt[:, :, None, :])
        y[i] = torch.matmul(state, qt[..., None])[..., 0]
    out = f["S"].clone()
    out[rows] = state
    return y[:-1], out
