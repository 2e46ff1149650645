"""Measured cases of the operators around the recurrent layer's serving and training paths.

Four calls, each in its plain form (elementary torch operations in 32 bits) and through the package:

* ``ssm_fwd``: selective state space scan over packed prompts,
      S_t = exp(dt_t a) S_{t-1} + dt_t B_t x_t^T,   y_t = S_t^T C_t + d x_t
  with dt = softplus(dt_raw + bias) and one fp32 state S [128, P] per sequence and head;
* ``ssm_step``: the same recurrence for 1 to 8 token slots of each sequence behind the short causal
  convolution, the two states in place and committed through an accepted prefix;
* ``draft_verify``: speculative acceptance of drafted tokens against the target's probabilities, and the
  next token by an exponential race, all random numbers given;
* ``block_norm_fwd`` / ``block_norm_bwd``: the norm after a block with its gate and residual scale, the
  residual sum and the norm before the next block, and the gradients.
"""
import torch

own = False

N_STATE = 128


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one long prompt at the head count of the repository's model shape: prefill, and the memory-side limit of the scan
        dict(name="ssm prompt 32768", op="ssm_fwd", dtype="bf16", lens="32768", heads=96, head_dim=64, groups=8, h0=False),
        # a prefill batch of unlike prompts that continue cached states: empty, one token, ends inside every tile size
        dict(name="ssm packed prompts", op="ssm_fwd", dtype="bf16", lens="4097,1,0,3000,129,2048,63,5501", heads=96, head_dim=64, groups=1, h0=True),
        # one prompt for a slice of the heads, 128-wide: less (sequence, head) work items than the GPU has room for
        dict(name="ssm few heads", op="ssm_fwd", dtype="bf16", lens="4096", heads=12, head_dim=128, groups=1, h0=True),
        # fp32 parity size, a short prompt
        dict(name="ssm short fp32", op="ssm_fwd", dtype="f32", lens="512", heads=2, head_dim=128, groups=2, h0=True),
        # draft verification for a full decode batch: 4 slots, padding and accepted prefixes drawn, paged states
        dict(name="step 256 x 4", op="ssm_step", dtype="bf16", seqs=256, slots=4, heads=96, head_dim=64, groups=8, paged=True, verify=True),
        # one token of one sequence: the latency of a call
        dict(name="step 1 x 1", op="ssm_step", dtype="bf16", seqs=1, slots=1, heads=24, head_dim=64, groups=1, paged=False, verify=False),
        # a decode batch's drafts against fp32 probabilities over a large vocabulary
        dict(name="verify 256 x 3", op="verify", dtype="f32", seqs=256, drafts=3, vocab=131072, drafter=True, ragged=False),
        # one sequence, bf16 probabilities, an odd vocabulary
        dict(name="verify 1 x 4", op="verify", dtype="bf16", seqs=1, drafts=4, vocab=32003, drafter=True, ragged=False),
        # a training block's boundary at the hidden size of the repository's benchmark
        dict(name="norm fwd 32768 x 7168", op="norm_fwd", dtype="bf16", rows=32768, dim=7168, post=True, gate="silu", residual=True, scale=True, pre=True),
        # and its gradients
        dict(name="norm bwd 16384 x 7168", op="norm_bwd", dtype="bf16", rows=16384, dim=7168, post=True, gate="silu", residual=True, scale=True, pre=True),
        # the recurrent core's output norm: one row per token and head, gated, no residual
        dict(name="norm per head", op="norm_fwd", dtype="bf16", rows=4096 * 96, dim=128, post=True, gate="sigmoid", residual=False, scale=False, pre=False),
        # fp32 gradients of an odd shape, no gate
        dict(name="norm bwd 1001 x 1544 fp32", op="norm_bwd", dtype="f32", rows=1001, dim=1544, post=True, gate="off", residual=True, scale=True, pre=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["ssm_fwd", "ssm_fwd", "ssm_step", "verify", "norm_fwd", "norm_bwd"])
    if op == "ssm_fwd":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        head_dim = rng.choice([64, 64, 128])
        groups = rng.choice([1, 2, 4, 8])
        heads = groups * rng.randint(1, 96 // groups)
        # fp32 prompts are parity and tuning runs: a hundredth of the serving work
        most = max(2, min(32768, int((2e6 if dtype == "bf16" else 1e5) / heads * 64 / head_dim)))
        total = _log_int(rng, 1, most)
        n = rng.choice([1, 1, 2, 3, 8])
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return dict(op=op, dtype=dtype, lens=",".join(map(str, lens)), heads=heads, head_dim=head_dim, groups=groups, h0=rng.random() < 0.5)
    if op == "ssm_step":
        groups = rng.choice([1, 2, 8])
        head_dim = rng.choice([64, 64, 128])
        heads = groups * rng.randint(1, 96 // groups)
        seqs = _log_int(rng, 1, max(1, min(256, 24576 * 64 // head_dim // heads)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=seqs, slots=rng.randint(1, 8 if seqs < 128 else 4), heads=heads, head_dim=head_dim,
                    groups=groups, paged=rng.random() < 0.5, verify=rng.random() < 0.5)
    if op == "verify":
        seqs, drafts = _log_int(rng, 1, 256), rng.randint(1, 8)
        vocab = _log_int(rng, 1000, max(1000, min(200000, int(2.6e8 / seqs / (2 * drafts + 2)))))
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), seqs=seqs, drafts=drafts, vocab=vocab, drafter=rng.random() < 0.7, ragged=rng.random() < 0.5)
    dim = 8 * _log_int(rng, 8, 1024)
    rows = _log_int(rng, 1, int((2e8 if op == "norm_fwd" else 1e8) / dim))
    post = rng.random() < 0.8
    pre = rng.random() < 0.7 if post else True
    residual = rng.random() < 0.7 if post else True
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, dim=dim, post=post, gate=rng.choice(["off", "silu", "sigmoid"]), residual=residual,
                scale=rng.random() < 0.6, pre=pre)


# ------------------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def prepare(case, seed):
    gen = _generator(seed)
    make = {"ssm_fwd": _prepare_ssm_fwd, "ssm_step": _prepare_ssm_step, "verify": _prepare_verify,
            "norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm}[case["op"]]
    state = make(case, gen)
    state["case"] = case
    return state


def _randn(gen, *shape, dtype=torch.float32):
    # bf16 tensors are drawn in bf16, which bounds the memory of the large ones
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _uniform(gen, lo, hi, *shape):
    return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo


def _scan_constants(case, gen):
    H = case["heads"]
    # step sizes around 0.01 .. 0.3 and decay rates in -1 .. -16 per unit of step: memory of one to some hundred tokens
    return dict(a=-_uniform(gen, 1.0, 16.0, H), dt_bias=_uniform(gen, -4.5, -1.5, H), d_skip=_uniform(gen, 0.5, 1.5, H))


def _prepare_ssm_fwd(case, gen):
    lens = [int(v) for v in case["lens"].split(",")]
    T, H, P, G = sum(lens), case["heads"], case["head_dim"], case["groups"]
    # rows as the short convolution with SiLU leaves them: x, B and C side by side
    rows = torch.nn.functional.silu(_randn(gen, T, H * P + 2 * G * N_STATE, dtype=_dtype(case)))
    offsets = [sum(lens[:i]) for i in range(len(lens) + 1)]
    s = dict(rows=rows, lens=lens, cu=torch.tensor(offsets, dtype=torch.int32, device="cuda"), dt=_randn(gen, T, H),
             h0=_randn(gen, len(lens), H, N_STATE, P) * 0.2 if case["h0"] else None)
    s.update(_scan_constants(case, gen))
    return s


def _prepare_ssm_step(case, gen):
    N, L, H, P, G = case["seqs"], case["slots"], case["heads"], case["head_dim"], case["groups"]
    C, W, io = H * P + 2 * G * N_STATE, 4, _dtype(case)
    pool = N + 5 if case["paged"] else N
    s = dict(rows=_randn(gen, N, L, C, dtype=io), dt=_randn(gen, N, L, H), weight=_randn(gen, C, W) * 0.5, bias=_randn(gen, C) * 0.1,
             conv_state=_randn(gen, pool, W - 1, C, dtype=io), state=_randn(gen, pool, H, N_STATE, P) * 0.2,
             y=torch.zeros(N, L, H * P, dtype=io, device="cuda").view(N, L, H, P), slots=None, accept=None, first=None)
    if case["paged"]:
        s["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:N].to(torch.int32)
    if case["verify"]:
        s["accept"] = torch.randint(0, L + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
        s["first"] = torch.randint(0, min(L, 3), (N,), generator=gen, device="cuda", dtype=torch.int32)
    s.update(_scan_constants(case, gen))
    return s


def _prepare_verify(case, gen):
    N, L, V, io = case["seqs"], case["drafts"], case["vocab"], _dtype(case)
    # the draft model is near the target: its logits plus noise; drafts are drawn from it by a race of their own
    logits = _randn(gen, N, L + 1, V) * 2.0
    p = torch.softmax(logits, -1).to(io)
    if case["drafter"]:
        q = torch.softmax(logits[:, :L] + 0.5 * _randn(gen, N, L, V), -1).to(io)
    else:
        q = None
    race = (p[:, :L] if q is None else q).float() / torch.empty(N, L, V, device="cuda").exponential_(generator=gen)
    draft = race.argmax(-1).to(torch.int32)
    return dict(p=p, q=q, draft=draft, u=torch.rand(N, L, generator=gen, device="cuda"), noise=torch.empty(N, V, device="cuda").exponential_(generator=gen),
                draft_len=torch.randint(0, L + 1, (N,), generator=gen, device="cuda", dtype=torch.int32) if case["ragged"] else None)


def _prepare_norm(case, gen):
    R, d, io = case["rows"], case["dim"], _dtype(case)
    some = lambda on, scale=1.0: _randn(gen, R, d, dtype=io) * scale if on else None
    back = case["op"] == "norm_bwd"
    s = dict(u=some(True, 1.7), gate=some(case["gate"] != "off"), residual=some(case["residual"], 3.0),
                w_post=1.0 + 0.1 * _randn(gen, d) if case["post"] else None, w_pre=1.0 + 0.1 * _randn(gen, d) if case["pre"] else None,
                scale=_uniform(gen, 0.1, 0.9, d) if case["scale"] else None,
                d_out=some(back), d_normed=some(back and case["pre"]), stats=None, case=case)
    if back:  # the forward of the same training step has left them
        s["stats"] = _plain_norm_fwd(s)[2]
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"ssm_fwd": _own_ssm_fwd, "ssm_step": _own_ssm_step, "verify": _own_verify, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd}[op](state)
    return {"ssm_fwd": _plain_ssm_fwd, "ssm_step": _plain_ssm_step, "verify": _plain_verify, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](state)


def _split(case, rows):
    """x [.., H, P], B and C [.., G, 128] of rows [.., H P + 2 G 128], as views."""
    H, P, G = case["heads"], case["head_dim"], case["groups"]
    x, b, c = torch.split(rows, [H * P, G * N_STATE, G * N_STATE], -1)
    return x.unflatten(-1, (H, P)), b.unflatten(-1, (G, N_STATE)), c.unflatten(-1, (G, N_STATE))


# the framework's calls
def _own_ssm_fwd(s):
    import gated_delta_rule_chunked_gb300 as kda
    x, b, c = _split(s["case"], s["rows"])
    return kda.ssm_fwd(x, s["dt"], s["a"], b, c, s["cu"], s["h0"], d_skip=s["d_skip"], dt_bias=s["dt_bias"], dt_softplus=True)


def _own_ssm_step(s):
    import gated_delta_rule_chunked_gb300 as kda
    y = kda.ssm_step(s["rows"], s["dt"], s["a"], s["weight"], s["bias"], s["conv_state"], s["state"], s["accept"], groups=s["case"]["groups"], activation="silu",
                     d_skip=s["d_skip"], dt_bias=s["dt_bias"], dt_softplus=True, state_indices=s["slots"], first_slot=s["first"], out=s["y"])
    return y, s["state"], s["conv_state"]


def _own_verify(s):
    import gated_delta_rule_chunked_gb300 as kda
    return kda.draft_verify(s["p"], s["q"], s["draft"], s["u"], s["noise"], s["draft_len"])


def _gate(s):
    return {} if s["gate"] is None else dict(gate=s["gate"], gate_act=s["case"]["gate"])


def _own_norm_fwd(s):
    import gated_delta_rule_chunked_gb300 as kda
    out, normed, stats = kda.block_norm_fwd(s["u"], s["w_post"], residual=s["residual"], scale=s["scale"], w_pre=s["w_pre"], eps=1e-6, **_gate(s))
    return out, normed, stats


def _own_norm_bwd(s):
    import gated_delta_rule_chunked_gb300 as kda
    return kda.block_norm_bwd(s["u"], s["w_post"], s["stats"], s["d_out"], s["d_normed"], residual=s["residual"], scale=s["scale"], w_pre=s["w_pre"], eps=1e-6,
                              **_gate(s))


# the plain forms
def _segment_sums(v):
    """v [.., n] -> [.., n, n]: the sum of v over j < k <= i where i >= j, -inf elsewhere. Summed apart for each j, without differences."""
    n = v.shape[-1]
    i, j = torch.arange(n, device=v.device)[:, None], torch.arange(n, device=v.device)[None, :]
    w = torch.where(i > j, v[..., :, None], 0.0).cumsum(-2)
    return torch.where(i >= j, w, -torch.inf)


def _step_sizes(s, dt):
    return torch.log1p(torch.exp(-(dt + s["dt_bias"]).abs())) + (dt + s["dt_bias"]).clamp(min=0.0)


def _plain_ssm_fwd(s, chunk=64):
    case, lens, Q = s["case"], s["lens"], chunk
    x, b, c = _split(case, s["rows"])
    T, H, P = x.shape
    G, N, dev = b.shape[1], len(lens), x.device
    # every sequence is padded to whole chunks; a padded token has a step size of zero
    n = torch.tensor(lens)
    chunks = (n + Q - 1) // Q
    total = int(chunks.sum())
    first = torch.cumsum(chunks, 0) - chunks
    seq = torch.repeat_interleave(torch.arange(N), n)
    at = (first[seq] * Q + torch.arange(T) - (torch.cumsum(n, 0) - n)[seq]).to(dev)

    def padded(v):
        w = torch.zeros((total * Q,) + v.shape[1:], dtype=torch.float32, device=dev)
        w[at] = v.float()
        return w.unflatten(0, (total, Q))

    X, B, C, dt = padded(x), padded(b), padded(c), padded(_step_sizes(s, s["dt"]))
    seg = _segment_sums((dt * s["a"]).permute(0, 2, 1))  # [chunk, H, Q, Q]
    decay = torch.exp(seg)
    total_decay = seg[:, :, -1, 0] + (dt * s["a"])[:, 0]  # log decay over a chunk [chunk, H]
    to_row = torch.exp(seg[:, :, :, 0] + (dt * s["a"])[:, :1].permute(0, 2, 1))  # from the chunk's start through row i
    scores = torch.einsum("nigk,njgk->ngij", C, B)
    weights = (scores[:, :, None] * decay.unflatten(1, (G, H // G))).flatten(1, 2)
    Xd = X * dt[..., None]
    y = torch.einsum("nhij,njhp->nihp", weights, Xd)
    R = H // G
    to_end = decay[:, :, -1]  # [chunk, H, Q]
    Xe = (Xd * to_end.permute(0, 2, 1)[..., None]).unflatten(2, (G, R))
    ends = torch.einsum("njgk,njgrp->ngrkp", B, Xe).flatten(1, 2)  # [chunk, H, 128, P]
    # nodes: a start (the initial state), the chunks and an end for every sequence; states entering each node
    node_of = (torch.arange(total) + 2 * torch.repeat_interleave(torch.arange(N), chunks) + 1).to(dev)
    starts = (first + 2 * torch.arange(N)).to(dev)
    stops = (first + 2 * torch.arange(N) + chunks + 1).to(dev)
    nodes = total + 2 * N
    logs = torch.zeros(nodes, H, device=dev)
    logs[node_of] = total_decay
    given = torch.zeros((nodes, H, N_STATE, P), device=dev)
    given[node_of] = ends
    if s["h0"] is not None:
        given[starts] = s["h0"]
    owner = torch.repeat_interleave(torch.arange(N), chunks + 2).to(dev)
    between = torch.exp(_segment_sums(logs.t()))  # [H, i, j]: decay over j < k <= i
    between = between * (owner[:, None] == owner[None, :])
    entering = torch.zeros_like(given)
    if nodes > 1:
        entering[1:] = torch.einsum("hij,jhkp->ihkp", between[:, :-1, :], given)
    starting = entering[node_of].unflatten(1, (G, R))
    y = y + torch.einsum("nigk,ngrkp->nigrp", C, starting).flatten(2, 3) * to_row.permute(0, 2, 1)[..., None]
    y = y + X * s["d_skip"][:, None]
    return y.flatten(0, 1)[at].to(x.dtype), entering[stops]


def _plain_ssm_step(s):
    case, rows = s["case"], s["rows"]
    N, L, Cc = rows.shape
    W, G, H, P = s["weight"].shape[1], case["groups"], case["heads"], case["head_dim"]
    dev = rows.device
    slots = torch.arange(N, device=dev) if s["slots"] is None else s["slots"].long()
    first = torch.zeros(N, dtype=torch.long, device=dev) if s["first"] is None else s["first"].long()
    accept = torch.full((N,), L, dtype=torch.long, device=dev) if s["accept"] is None else s["accept"].long()
    keep = (accept - first).clamp(min=0)  # committed tokens
    line = torch.cat([s["conv_state"][slots], rows], 1)  # W - 1 earlier inputs, then the slots
    place = lambda v: torch.where(v < W - 1, v, (v + first.reshape((-1,) + (1,) * (v.dim() - 1))).clamp(max=W - 2 + L))
    tap = torch.arange(L, device=dev)[None, :, None] - first[:, None, None] + torch.arange(W, device=dev)[None, None, :]
    tap = place(tap.clamp(min=0))  # [N, L, W]
    window = line[torch.arange(N, device=dev)[:, None, None], tap].float()  # [N, L, W, C]
    z = torch.einsum("nlwc,cw->nlc", window, s["weight"]) + s["bias"]
    z = z / (1.0 + torch.exp(-z))
    x, b, c = _split(case, z)
    live = torch.arange(L, device=dev)[None, :] >= first[:, None]
    dt = _step_sizes(s, s["dt"]) * live[..., None]
    seg = _segment_sums((dt * s["a"]).permute(0, 2, 1))  # [N, H, L, L]
    to_row = seg[..., 0] + (dt * s["a"])[:, :1].permute(0, 2, 1)  # [N, H, L]
    decay = torch.exp(seg)
    S = s["state"][slots]  # [N, H, 128, P]
    scores = torch.einsum("nigk,njgk->ngij", c, b).repeat_interleave(H // G, 1)
    xd = x * dt[..., None]
    y = torch.einsum("nhij,njhp->nihp", scores * decay, xd)
    y = y + torch.einsum("nigk,ngrkp->nigrp", c, S.unflatten(1, (G, H // G))).flatten(2, 3) * torch.exp(to_row).permute(0, 2, 1)[..., None]
    y = y + x * s["d_skip"][:, None]
    s["y"].copy_(torch.where(live[..., None, None], y.to(rows.dtype), s["y"]))
    # the state after the committed slots
    last = (accept - 1).clamp(min=0)
    pick = torch.arange(N, device=dev)
    w = decay[pick, :, last] * (torch.arange(L, device=dev)[None, None, :] < accept[:, None, None])  # [N, H, L]
    grown = torch.einsum("njgk,njgrp->ngrkp", b, (xd * w.permute(0, 2, 1)[..., None]).unflatten(2, (G, H // G))).flatten(1, 2)
    kept = torch.exp(to_row[pick, :, last]) * (accept > 0)[:, None] + (accept == 0)[:, None]
    s["state"][slots] = S * kept[..., None, None] + grown
    after = place(keep[:, None] + torch.arange(W - 1, device=dev)[None, :])
    s["conv_state"][slots] = line[pick[:, None], after]
    return s["y"], s["state"], s["conv_state"]


def _plain_verify(s):
    p, q, draft = s["p"], s["q"], s["draft"].long()
    N, L1, V = p.shape
    L, dev = L1 - 1, p.device
    inside = (draft >= 0) & (draft < V)
    if s["draft_len"] is not None:
        inside = inside & (torch.arange(L, device=dev)[None, :] < s["draft_len"][:, None])
    drafted = inside.long().cumprod(1).sum(1)
    token = draft.clamp(0, V - 1)[..., None]
    px = p[:, :L].gather(2, token)[..., 0].float()
    qx = torch.ones_like(px) if q is None else q.gather(2, token)[..., 0].float()
    ok = (s["u"] * qx < px) & (torch.arange(L, device=dev)[None, :] < drafted[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    pick = torch.arange(N, device=dev)
    row = p[pick, accepted].float()
    at = accepted.clamp(max=L - 1)
    if q is None:
        less = (torch.arange(V, device=dev)[None, :] == draft[pick, at][:, None]).float()
    else:
        less = q[pick, at].float()
    left = torch.where((accepted < drafted)[:, None], row - less, row)
    race = lambda v: torch.nan_to_num(torch.where(v > 0, v / s["noise"], 0.0), nan=0.0, posinf=torch.inf)
    score = race(left)
    best = score.amax(1, keepdim=True)
    second = race(row)
    score = torch.where(best > 0, score, second)
    best = torch.where(best > 0, best, second.amax(1, keepdim=True))
    index = torch.arange(V, device=dev)[None, :]
    chosen = torch.where((score == best) & (best > 0), index, V).amin(1)
    chosen = torch.where(chosen == V, -1, chosen)
    place = torch.arange(L1, device=dev)[None, :]
    tokens = torch.where(place < accepted[:, None], torch.cat([draft, draft[:, :1]], 1), torch.where(place == accepted[:, None], chosen[:, None], -1))
    return accepted.to(torch.int32), (L - accepted).to(torch.int32), tokens.to(torch.int32)


def _branch(s, eps=1e-6):
    """The block's normalised and gated output in fp32, and what the gradients need of it."""
    u = s["u"].float()
    if s["w_post"] is None:
        ru = None
    elif s["stats"] is not None:
        ru = s["stats"][0][:, None]
    else:
        ru = torch.rsqrt((u * u).mean(-1, keepdim=True) + eps)
    hat = u if ru is None else u * ru
    w = 1.0 if s["w_post"] is None else s["w_post"]
    if s["gate"] is None:
        g = dg = None
    else:
        z = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        g, dg = (sig, sig * (1.0 - sig)) if s["case"]["gate"] == "sigmoid" else (z * sig, sig * (1.0 + z * (1.0 - sig)))
    m = hat * w if g is None else hat * w * g
    return hat, ru, w, g, dg, m


def _summed(s, m):
    x = m if s["scale"] is None else m * s["scale"]
    return x if s["residual"] is None else s["residual"].float() + x


def _plain_norm_fwd(s, eps=1e-6):
    hat, ru, w, g, dg, m = _branch(s, eps)
    del hat, g, dg
    x = _summed(s, m)
    rx = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    normed = None if s["w_pre"] is None else (x * rx * s["w_pre"]).to(s["u"].dtype)
    stats = (None if ru is None else ru[:, 0], None if s["w_pre"] is None else rx[:, 0])
    return x.to(s["u"].dtype), normed, stats


def _plain_norm_bwd(s, eps=1e-6):
    hat, ru, w, g, dg, m = _branch(s, eps)
    x = _summed(s, m)
    dx = s["d_out"].float()
    grads = dict(du=None, dgate=None, dresidual=None, dw_post=None, dscale=None, dw_pre=None)
    if s["w_pre"] is not None:
        rx = s["stats"][1][:, None]
        e = s["d_normed"].float()
        grads["dw_pre"] = (e * x * rx).sum(0)
        e = e * s["w_pre"]
        dx = dx + rx * (e - x * rx * rx * (e * x).mean(-1, keepdim=True))
    io = s["u"].dtype
    if s["residual"] is not None:
        grads["dresidual"] = dx.to(io)
    if s["scale"] is not None:
        grads["dscale"] = (dx * m).sum(0)
        dx = dx * s["scale"]
    if g is not None:
        grads["dgate"] = (dx * hat * w * dg).to(io)
        dx = dx * g
    if s["w_post"] is not None:
        grads["dw_post"] = (dx * hat).sum(0)
        dx = dx * w
        dx = ru * (dx - hat * (dx * hat).mean(-1, keepdim=True))
    grads["du"] = dx.to(io)
    return grads


# ------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ssm_fwd":
        lens = [int(v) for v in case["lens"].split(",")]
        T, H, P, G = sum(lens), case["heads"], case["head_dim"], case["groups"]
        states = len(lens) * H * N_STATE * P * 4
        # x in, y out, B and C, the step sizes, final states (and initial ones); decay, update and read-out of the state per token
        return {"bytes": e * T * (2 * H * P + 2 * G * N_STATE) + 4 * T * H + states * (2 if case["h0"] else 1), "flops": 5.0 * T * H * N_STATE * P}
    if case["op"] == "ssm_step":
        N, L, H, P, G = case["seqs"], case["slots"], case["heads"], case["head_dim"], case["groups"]
        C = H * P + 2 * G * N_STATE
        states = 2.0 * N * H * N_STATE * P * 4  # read and written
        return {"bytes": states + e * N * (L * (C + H * P) + 2 * 3 * C) + 4 * N * L * H + 4 * C * 5, "flops": 5.0 * N * L * H * N_STATE * P + 8.0 * N * L * C}
    if case["op"] == "verify":
        N, L, V = case["seqs"], case["drafts"], case["vocab"]
        # one row of the target's, one of the drafter's and the race's numbers for each sequence
        return {"bytes": N * V * (e * (2 if case["drafter"] else 1) + 4) + N * L * 16 + N * (L + 3) * 4, "flops": 3.0 * N * V}
    R, d = case["rows"], case["dim"]
    gate, res, pre = case["gate"] != "off", case["residual"], case["pre"]
    if case["op"] == "norm_fwd":
        return {"bytes": e * R * d * (2 + gate + res + pre) + 4 * d * 3, "flops": 12.0 * R * d}
    return {"bytes": e * R * d * (3 + 2 * gate + 2 * res + pre) + 4 * d * 6, "flops": 30.0 * R * d}


# ------------------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"ssm_fwd": _exact_ssm_fwd, "ssm_step": _exact_ssm_step, "verify": _exact_verify, "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd}[case["op"]](case, s)


def _exact_scan(a, d, step, x, b, c, S, write):
    """Token by token: step [n, l, H], x [n, l, H, P], b, c [n, l, G, 128], S [n, H, 128, P]; write(t, y, S) after each token."""
    R = x.shape[2] // b.shape[2]
    for t in range(x.shape[1]):
        bt, ct = b[:, t].double().repeat_interleave(R, 1), c[:, t].double().repeat_interleave(R, 1)
        xt, h = x[:, t].double(), step[:, t]
        S = S * torch.exp(h * a)[..., None, None]
        S = S + bt[..., :, None] * (h[..., None] * xt)[..., None, :]
        write(t, torch.matmul(ct[..., None, :], S)[..., 0, :] + d[:, None] * xt, S)
    return S


def _exact_ssm_fwd(case, s):
    lens = s["lens"]
    H, P, N, longest = case["heads"], case["head_dim"], len(lens), max(lens)
    if longest * (4e-5 + N * H * N_STATE * P * 8 * 8 / 5e12) > 15.0:
        return None
    x, b, c = _split(case, s["rows"])
    idx = torch.tensor([[min(sum(lens[:i]) + t, max(x.shape[0] - 1, 0)) for t in range(longest)] for i in range(N)], device="cuda")
    alive = torch.tensor([[t < n for t in range(longest)] for n in lens], device="cuda")
    step = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=60.0)
    S = torch.zeros(N, H, N_STATE, P, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    y = torch.empty(N, longest, H, P, dtype=torch.float64, device="cuda")

    def write(t, v, _):
        y[:, t] = v

    S = _exact_scan(s["a"].double(), s["d_skip"].double(), step[idx] * alive[..., None], x[idx], b[idx], c[idx], S, write)
    return y[alive], S


def _exact_ssm_step(case, s):
    N, L = case["seqs"], case["slots"]
    Cc, W = s["weight"].shape
    slots = range(N) if s["slots"] is None else s["slots"].tolist()
    y, state, conv = s["y"].double(), s["state"].double(), s["conv_state"].clone()
    first = [0] * N if s["first"] is None else s["first"].tolist()
    accept = [L] * N if s["accept"] is None else s["accept"].tolist()
    for i, slot in enumerate(slots):
        line = torch.cat([s["conv_state"][slot], s["rows"][i, first[i]:]], 0).double()
        n = L - first[i]
        z = torch.stack([(line[t:t + W] * s["weight"].double().t()).sum(0) + s["bias"].double() for t in range(n)])
        x, b, c = _split(case, torch.nn.functional.silu(z)[None])
        step = torch.nn.functional.softplus(s["dt"][i, first[i]:].double() + s["dt_bias"].double(), threshold=60.0)[None]
        kept = accept[i] - first[i]

        def write(t, v, S):
            y[i, first[i] + t] = v[0]
            if t + 1 == kept:
                state[slot] = S[0]

        _exact_scan(s["a"].double(), s["d_skip"].double(), step, x, b, c, s["state"][slot].double()[None], write)
        if kept > 0:
            conv[slot] = torch.cat([s["conv_state"][slot], s["rows"][i, first[i]:]], 0)[kept:kept + W - 1]
    return y, state, conv.double()


def _exact_verify(case, s):
    return None  # whole numbers only


def _exact_norm(case, s):
    """The forward as a function of its fp64 inputs; a dict of them that need gradients."""
    v = {k: None if s[k] is None else s[k].double().requires_grad_(case["op"] == "norm_bwd") for k in ("u", "gate", "residual", "w_post", "w_pre", "scale")}
    rms = lambda t: (t.square().mean(-1) + 1e-6).pow(-0.5)
    m, ru, rx, normed = v["u"], None, None, None
    if v["w_post"] is not None:
        ru = rms(m)
        m = m * ru[:, None] * v["w_post"]
    if v["gate"] is not None:
        m = m * (torch.sigmoid(v["gate"]) if case["gate"] == "sigmoid" else torch.nn.functional.silu(v["gate"]))
    if v["scale"] is not None:
        m = m * v["scale"]
    out = m if v["residual"] is None else v["residual"] + m
    if v["w_pre"] is not None:
        rx = rms(out)
        normed = out * rx[:, None] * v["w_pre"]
    return v, out, normed, (ru, rx)


def _exact_norm_fwd(case, s):
    with torch.no_grad():
        _, out, normed, stats = _exact_norm(case, s)
    return out, normed, stats


def _exact_norm_bwd(case, s):
    v, out, normed, _ = _exact_norm(case, s)
    ends, seeds = ([out], [s["d_out"].double()]) if normed is None else ([out, normed], [s["d_out"].double(), s["d_normed"].double()])
    torch.autograd.backward(ends, seeds)
    return {"d" + k: None if t is None else t.grad for k, t in v.items()}
