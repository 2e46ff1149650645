"""GPU parity of the selective scan (prompts and the decode step) against its fp64 form.

Tolerances, as a share of the largest value: bf16 outputs round once at 2^-9 and their scores
once more, so 1e-2 (the library's bound for bf16 I/O); fp32 results sum at most 128 products and
decay, each rounding at 2^-24, so 128 * 2^-24 < 1e-5 of the summed magnitudes, doubled."""
import numpy as np
import pytest
import torch

import block_fp64 as ref

pytestmark = pytest.mark.gpu
TOL = {"bf16": 1e-2, "f32": 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_chunked_gb300 as m
    m.library()
    return m


def case(lens, H, G, P, io, seed, h0=True, strength=1.0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rows = torch.nn.functional.silu(torch.randn(T, H * P + 2 * G * 128, generator=gen)).to(DT[io])
    return dict(rows=rows, dt=torch.randn(T, H, generator=gen), a=-torch.rand(H, generator=gen) * 15 * strength - 0.1,
                dt_bias=torch.rand(H, generator=gen) * 3 - 4.5, d_skip=torch.randn(H, generator=gen),
                h0=torch.randn(N, H, 128, P, generator=gen) * 0.3 if h0 else None,
                cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32))


def split(rows, H, G, P):
    T = rows.shape[0]
    x, b, c = torch.split(rows, [H * P, G * 128, G * 128], 1)
    return x.unflatten(1, (H, P)), b.unflatten(1, (G, 128)), c.unflatten(1, (G, 128))


def cuda(t):
    return None if t is None else t.cuda()


def check(kda, lens, H, G, P, io, seed, h0=True, strength=1.0, views=True, **opts):
    s = case(lens, H, G, P, io, seed, h0, strength)
    x, b, c = split(s["rows"].cuda(), H, G, P)
    if not views:
        x, b, c = x.contiguous(), b.contiguous(), c.contiguous()
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, s["cu"], cuda(s["h0"]), d_skip=s["d_skip"].cuda(),
                        dt_bias=s["dt_bias"].cuda(), **opts)
    torch.cuda.synchronize()
    y_ref, h_ref = ref.scan(*[t for t in (x, s["dt"], s["a"], b, c)], lens, s["h0"], s["d_skip"], s["dt_bias"])
    assert ref.rel(y.float(), y_ref) <= TOL[io]
    assert ref.rel(hT, h_ref) <= TOL["f32"]
    return y, hT


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,G,P", [
    ([1], 1, 1, 64), ([2, 0, 7], 2, 1, 128), ([127, 128, 129], 2, 2, 64), ([8, 9, 63, 64, 65], 3, 1, 64),
    ([300], 4, 2, 128), ([255, 1, 257], 2, 1, 128), ([700], 1, 1, 64),
])
def test_prompts(kda, io, lens, H, G, P):
    check(kda, lens, H, G, P, io, seed=sum(lens) + H)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_no_initial_state_and_contiguous_inputs(kda, io):
    check(kda, [130, 5], 2, 1, 64, io, seed=3, h0=False)
    check(kda, [130, 5], 4, 4, 64, io, seed=4, views=False)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strong_and_absent_decay(kda, io):
    check(kda, [260], 3, 1, 64, io, seed=5, strength=40.0)     # most decays underflow to zero
    s = case([200], 2, 1, 64, io, 6)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), torch.zeros(2).cuda(), b, c, None, None)   # a = 0: prefix sums
    y_ref, h_ref = ref.scan(x, s["dt"], torch.zeros(2), b, c, [200])
    assert ref.rel(y.float(), y_ref) <= TOL[io] and ref.rel(hT, h_ref) <= TOL["f32"]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_raw_steps_equal_sequences_and_no_final_state(kda, io):
    s = case([140, 140], 2, 1, 64, io, 7)
    h = torch.rand(280, 2) * 0.2
    h[::3] = 0.0                                               # a step of zero leaves the state as it is
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    y, hT = kda.ssm_fwd(x, h.cuda(), s["a"].cuda(), b, c, None, s["h0"].cuda(), dt_softplus=False, n_seqs=2,
                        final_state=False)
    y_ref, _ = ref.scan(x, h, s["a"], b, c, [140, 140], s["h0"], softplus=False)
    assert hT is None and ref.rel(y.float(), y_ref) <= TOL[io]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sequences_are_apart(kda, io):
    """Rows of one sequence that are not finite stay out of its neighbours."""
    lens = [70, 131, 40, 129]
    s = case(lens, 2, 1, 64, io, 8)
    rows = s["rows"].cuda()
    bad = rows.clone()
    bad[70:201] = float("nan")
    bad[241:] = float("inf")
    args = (s["dt"].cuda(), s["a"].cuda())
    run = lambda r: kda.ssm_fwd(split(r, 2, 1, 64)[0], *args, *split(r, 2, 1, 64)[1:], s["cu"].cuda(), s["h0"].cuda())
    (y0, h0), (y1, h1) = run(rows), run(bad)
    for lo, hi, i in ((0, 70, 0), (201, 241, 2)):
        assert torch.equal(y0[lo:hi], y1[lo:hi]) and torch.equal(h0[i], h1[i])


def test_chained_calls_match_one(kda):
    """A prompt cut anywhere and continued from its state gives the same states."""
    s = case([403], 2, 1, 64, "bf16", 9)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    dt, a = s["dt"].cuda(), s["a"].cuda()
    y, hT = kda.ssm_fwd(x, dt, a, b, c, None, s["h0"].cuda())
    h, ys = s["h0"].cuda(), []
    for lo, hi in ((0, 1), (1, 130), (130, 403)):
        yy, h = kda.ssm_fwd(x[lo:hi], dt[lo:hi], a, b[lo:hi], c[lo:hi], None, h)
        ys.append(yy)
    assert ref.rel(h, hT) <= TOL["f32"] and ref.rel(torch.cat(ys).float(), y.float()) <= TOL["bf16"]


def test_same_call_same_bits(kda):
    s = case([500, 77], 3, 1, 64, "bf16", 10)
    x, b, c = split(s["rows"].cuda(), 3, 1, 64)
    run = lambda: kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, s["cu"].cuda(), s["h0"].cuda())
    (y0, h0), (y1, h1) = run(), run()
    assert torch.equal(y0, y1) and torch.equal(h0, h1)


def test_other_stream(kda):
    s = case([333], 2, 1, 64, "bf16", 11)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    dt, a = s["dt"].cuda(), s["a"].cuda()
    y0, h0 = kda.ssm_fwd(x, dt, a, b, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, h1 = kda.ssm_fwd(x, dt, a, b, c)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)


def test_no_tokens(kda):
    h0 = torch.randn(2, 1, 128, 64).cuda()
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    y, hT = kda.ssm_fwd(e(0, 1, 64), torch.empty(0, 1).cuda(), -torch.ones(1).cuda(), e(0, 1, 128), e(0, 1, 128),
                        torch.zeros(3, dtype=torch.int32), h0)
    assert y.shape == (0, 1, 64) and torch.equal(hT, h0)


def test_refusals(kda):
    s = case([16], 4, 2, 64, "bf16", 12)
    x, b, c = split(s["rows"].cuda(), 4, 2, 64)
    dt, a = s["dt"].cuda(), s["a"].cuda()
    with pytest.raises(kda.KdaError):
        kda.ssm_fwd(x[:, :3].contiguous(), dt[:, :3].contiguous(), a[:3], b, c)          # 2 groups, 3 heads
    with pytest.raises(kda.KdaError):
        kda.ssm_fwd(x.reshape(16, 8, 32), dt.repeat(1, 2), a.repeat(2), b, c)            # head_dim 32
    with pytest.raises(ValueError):
        kda.ssm_fwd(x.transpose(1, 2), dt, a, b, c)
    with pytest.raises(ValueError):
        kda.ssm_fwd(x, dt[:8], a, b, c)
    with pytest.raises(TypeError):
        kda.ssm_fwd(x, dt.double(), a, b, c)
    with pytest.raises(TypeError):
        kda.ssm_fwd(x, dt, a, b.float(), c)
    with pytest.raises(kda.KdaError):
        kda.ssm_fwd(x, dt, a, b, c, n_seqs=3)                                            # 16 tokens in 3 equal parts
    with pytest.raises(kda.KdaError):                                                    # row stride 4 * 64 + 4
        rows = torch.zeros(16, 260, dtype=torch.bfloat16, device="cuda")
        kda.ssm_fwd(rows[:, :256].unflatten(1, (4, 64)), dt, a, b, c)


@pytest.mark.parametrize("lens,H,G,P", [([2500], 1, 1, 64), ([2049, 1900], 1, 1, 128), ([3000, 0, 2, 2900], 1, 1, 64)])
def test_long_prompts_in_segments(kda, lens, H, G, P):
    """Few (sequence, head) pairs and many chunks: the sequences run in segments, folded from their own states."""
    import ctypes as C
    from gated_delta_rule_chunked_gb300 import _lib
    a = _lib.SsmArgs()
    a.n_seqs, a.total_tokens, a.heads, a.groups, a.head_dim, a.d_state = len(lens), sum(lens), H, G, P, 128
    a.cu_seqlens = a.x = a.b = a.c = a.dt = a.a = a.y = 1 << 40
    a.ldx, a.ldb, a.ldc = H * P, G * 128, G * 128
    assert kda.library().kda_ssm_fwd_workspace_size(C.byref(a)) > 0          # a workspace is what segments need
    check(kda, lens, H, G, P, "bf16", seed=sum(lens), strength=0.05)         # slow decay: the state crosses segments
    check(kda, lens, H, G, P, "bf16", seed=sum(lens) + 1, h0=False)


def test_many_sequences(kda):
    """More sequences than are put in order of length, and more pairs than a wave."""
    gen = torch.Generator().manual_seed(20)
    lens = torch.randint(0, 12, (300,), generator=gen).tolist()
    check(kda, lens, 2, 1, 64, "bf16", seed=21)
    lens = torch.randint(0, 200, (40,), generator=gen).tolist()
    check(kda, lens, 8, 4, 64, "bf16", seed=22)


@pytest.mark.parametrize("N,H,P", [(1, 40, 128), (9, 5, 128), (3, 1, 64)])
def test_fp32_slices(kda, N, H, P):
    """fp32 prompts in slices of 64 and of 16 value columns."""
    check(kda, [17] * N, H, 1, P, "f32", seed=N + H)


@pytest.mark.parametrize("off", [8, 24])
def test_rows_at_any_16_byte_offset(kda, off):
    """x, B and C inside a wider row, at offsets that are multiples of 8 elements only."""
    s = case([150], 2, 1, 64, "bf16", 30)
    wide = torch.full((150, 384 + off + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, off:off + 384] = s["rows"].cuda()
    x, b, c = split(wide[:, off:off + 384], 2, 1, 64)
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, None, s["h0"].cuda())
    y_ref, h_ref = ref.scan(x, s["dt"], s["a"], b, c, [150], s["h0"])
    assert ref.rel(y.float(), y_ref) <= TOL["bf16"] and ref.rel(hT, h_ref) <= TOL["f32"]


def test_status_stays_clear(kda):
    s = case([900, 300], 2, 1, 64, "bf16", 31)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, s["cu"].cuda(), dev_status=status)
    assert int(status) == 0


# ------------------------------------------------------------------------------------------ step
def step_case(N, L, H, G, P, W, io, seed, pool=None):
    gen = torch.Generator().manual_seed(seed)
    Cc, S = H * P + 2 * G * 128, pool or N
    return dict(xbc=torch.randn(N, L, Cc, generator=gen).to(DT[io]), dt=torch.randn(N, L, H, generator=gen),
                a=-torch.rand(H, generator=gen) * 8, weight=torch.randn(Cc, W, generator=gen) / W ** 0.5,
                bias=torch.randn(Cc, generator=gen) * 0.1, conv_state=torch.randn(S, W - 1, Cc, generator=gen).to(DT[io]),
                state=torch.randn(S, H, 128, P, generator=gen) * 0.3, d_skip=torch.randn(H, generator=gen),
                dt_bias=torch.randn(H, generator=gen) - 2)


def run_step(kda, s, G, act="silu", accept=None, slots=None, first=None, bias=True, skip=True):
    g = {k: v.cuda() for k, v in s.items()}
    N, L, _ = s["xbc"].shape
    H, P = s["state"].shape[1], s["state"].shape[3]
    out = torch.full((N, L, H, P), 7.0, dtype=s["xbc"].dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.ssm_step(g["xbc"], g["dt"], g["a"], g["weight"], g["bias"] if bias else None, g["conv_state"], g["state"],
                 cuda(accept), groups=G, d_skip=g["d_skip"] if skip else None, dt_bias=g["dt_bias"] if bias else None,
                 activation=act, state_indices=cuda(slots), first_slot=cuda(first), out=out, dev_status=status)
    torch.cuda.synchronize()
    ys, pool, cpool = ref.step(s["xbc"], s["dt"], s["a"], s["weight"], s["bias"] if bias else None, s["conv_state"],
                               s["state"], G, accept, slots, first, s["d_skip"] if skip else None,
                               s["dt_bias"] if bias else None, act=act)
    io = "bf16" if s["xbc"].dtype == torch.bfloat16 else "f32"
    seen = torch.zeros(N, L, dtype=torch.bool)
    got, want = [], []
    for (i, t), y in ys.items():
        seen[i, t] = True
        got.append(out[i, t].float().cpu())
        want.append(y)
    if got:
        assert ref.rel(torch.stack(got), torch.stack(want)) <= TOL[io]
    assert (out.cpu()[~seen] == 7.0).all()                     # padding and skipped sequences are not written
    assert ref.rel(g["state"], pool) <= TOL["f32"]
    if cpool is not None:
        assert torch.equal(g["conv_state"].cpu(), cpool)
    return int(status)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,H,G,P,W", [(1, 1, 1, 1, 64, 4), (3, 4, 4, 2, 64, 4), (2, 8, 2, 1, 128, 3), (5, 2, 3, 3, 64, 2), (2, 3, 2, 1, 64, 1)])
def test_step(kda, io, N, L, H, G, P, W):
    s = step_case(N, L, H, G, P, W, io, seed=N * 10 + L)
    assert run_step(kda, s, G) == 0
    assert run_step(kda, s, G, act="none", bias=False, skip=False) == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_step_accept_padding_and_pool(kda, io):
    N, L = 9, 5
    s = step_case(N, L, 2, 1, 64, 4, io, seed=2, pool=14)
    slots = torch.tensor([13, 0, 4, 7, 2, 9, 1, 11, 5], dtype=torch.int32)
    accept = torch.tensor([0, 1, 5, 2, 3, 5, 4, 9, -1], dtype=torch.int32)    # the last two are clamped
    first = torch.tensor([0, 1, 0, 3, 2, 5, 3, 1, 0], dtype=torch.int32)      # 5: all padding
    assert run_step(kda, s, 1, accept=accept, slots=slots, first=first) == 0


def test_step_bad_slot(kda):
    s = step_case(3, 2, 2, 1, 64, 4, "bf16", seed=3, pool=4)
    assert run_step(kda, s, 1, slots=torch.tensor([1, 4, 0], dtype=torch.int32)) == 1
    assert run_step(kda, s, 1, slots=torch.tensor([-1, -1, 9], dtype=torch.int32)) == 1


def test_more_sequences_than_a_wave(kda):
    s = step_case(40, 3, 24, 4, 64, 4, "bf16", seed=4)
    accept = torch.arange(40, dtype=torch.int32) % 4
    assert run_step(kda, s, 4, accept=accept) == 0


def test_tokens_one_by_one_match_a_prompt(kda):
    """The step over a prompt's raw rows reaches the states of convolution + scan in fp32."""
    gen = torch.Generator().manual_seed(5)
    T, H, G, P, W = 21, 2, 1, 64, 4
    Cc = H * P + 2 * G * 128
    s = step_case(1, T, H, G, P, W, "f32", seed=6)
    rows = s["xbc"][0].cuda()
    w, bias = s["weight"].cuda(), s["bias"].cuda()
    dt, a, skip, tb = s["dt"][0].cuda(), s["a"].cuda(), s["d_skip"].cuda(), s["dt_bias"].cuda()
    conv, tail = kda.conv_fwd(rows, w, bias, None, s["conv_state"].cuda())
    y, hT = kda.ssm_fwd(*split(conv, H, G, P)[:1], dt, a, *split(conv, H, G, P)[1:], None, s["state"].cuda(), d_skip=skip, dt_bias=tb)
    cs, st = s["conv_state"].cuda(), s["state"].cuda()
    ys, t = [], 0
    while t < T:
        n = min(int(torch.randint(1, 9, (1,), generator=gen)), T - t)
        ys.append(kda.ssm_step(rows[None, t:t + n].contiguous(), dt[None, t:t + n].contiguous(), a, w, bias, cs, st, groups=G,
                               d_skip=skip, dt_bias=tb)[0])
        t += n
    assert ref.rel(torch.cat(ys), y) <= TOL["f32"] and ref.rel(st, hT) <= TOL["f32"] and torch.equal(cs, tail)


def test_step_refusals(kda):
    s = {k: v.cuda() for k, v in step_case(2, 9, 2, 1, 64, 4, "bf16", seed=7).items()}
    call = lambda xbc, dt, **kw: kda.ssm_step(xbc, dt, s["a"], s["weight"], s["bias"], s["conv_state"], s["state"], **kw)
    with pytest.raises(kda.KdaError):
        call(s["xbc"], s["dt"])                                                     # 9 slots
    x, dt = s["xbc"][:, :2].contiguous(), s["dt"][:, :2].contiguous()
    with pytest.raises(ValueError):
        call(x, dt, groups=2)                                                       # channels do not add up
    with pytest.raises(ValueError):
        call(x[:1].contiguous(), dt[:1].contiguous())                               # pool of 2, no indices
    with pytest.raises(ValueError):
        call(s["xbc"][:, :2], dt)                                                   # not contiguous
    with pytest.raises(TypeError):
        call(x, dt.half())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 5, 100, 127, 200])
def test_after_a_token_that_forgets_everything(kda, io, at):
    # exp(h a) of one token is zero by a wide margin; what the tokens after it keep of one another is not touched by it
    s = case([300], 2, 1, 64, io, 71)
    s["a"] = torch.tensor([-0.5, -16.0])
    s["dt"][at] = 1e5
    s["rows"][at, :128] = 0   # its x
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, s["cu"], s["h0"].cuda(), d_skip=s["d_skip"].cuda(),
                        dt_bias=s["dt_bias"].cuda())
    y_ref, h_ref = ref.scan(x, s["dt"], s["a"], b, c, [300], s["h0"], s["d_skip"], s["dt_bias"])
    for h in range(2):
        assert ref.rel(y[at:, h].float(), torch.as_tensor(y_ref)[at:, h]) <= TOL[io]
        assert ref.rel(hT[:, h], torch.as_tensor(h_ref)[:, h]) <= TOL["f32"]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_offsets_outside_the_tokens(kda, io):
    # offsets past the last row end there; a falling pair is an empty sequence
    s = case([40, 60, 30], 2, 1, 64, io, 72)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    call = lambda cu: kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                  s["h0"].cuda(), d_skip=s["d_skip"].cuda(), dt_bias=s["dt_bias"].cuda())
    y, hT = call([0, 40, 100, 130])
    y1, hT1 = call([0, 40, 100, 500])
    assert torch.equal(y, y1) and torch.equal(hT, hT1)
    y2, hT2 = call([0, 40, 20, 130])   # the second is empty, the third starts at 20
    assert torch.equal(hT2[1], s["h0"][1].cuda()) and torch.equal(hT2[0], hT[0])


@pytest.mark.parametrize("lens,H,G,P", [([260], 1, 1, 64), ([900], 2, 1, 128), ([700, 0, 3, 650], 3, 1, 64), ([301, 300], 2, 2, 128), ([2048], 24, 1, 64)])
def test_fp32_prompts_in_segments(kda, lens, H, G, P):
    # few heads: the walk is cut, here into several segments, some of them empty
    check(kda, lens, H, G, P, "f32", seed=31 + sum(lens))
    check(kda, lens, H, G, P, "f32", seed=32 + sum(lens), h0=False, strength=0.01)   # what a segment holds reaches far into the next


def test_fp32_segments_and_steps_agree(kda):
    s = case([515], 2, 1, 64, "f32", 77, strength=0.02)
    x, b, c = split(s["rows"].cuda(), 2, 1, 64)
    kw = dict(d_skip=s["d_skip"].cuda(), dt_bias=s["dt_bias"].cuda())
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, None, s["h0"].cuda(), **kw)
    h, parts = s["h0"].cuda(), []
    for t0 in range(0, 515, 30):   # pieces too short for a second segment
        e = min(t0 + 30, 515)
        yp, h = kda.ssm_fwd(x[t0:e], s["dt"][t0:e].cuda(), s["a"].cuda(), b[t0:e], c[t0:e], None, h, **kw)
        parts.append(yp)
    assert ref.rel(torch.cat(parts).cpu(), y.cpu().double()) <= 2 * TOL["f32"]
    assert ref.rel(h.cpu(), hT.cpu().double()) <= 2 * TOL["f32"]


@pytest.mark.parametrize("lens,H,P", [([4100], 1, 64), ([2000, 1, 2100], 1, 128)])
def test_segments_that_remember(kda, lens, H, P):
    # hardly any decay: a state holds thousands of tokens, and what the first segment adds reaches the last
    s = case(lens, H, 1, P, "bf16", 41)
    x, b, c = split(s["rows"].cuda(), H, 1, P)
    a = torch.full((H,), -1e-4)
    y, hT = kda.ssm_fwd(x, s["dt"].cuda(), a.cuda(), b, c, s["cu"], s["h0"].cuda(), d_skip=s["d_skip"].cuda(), dt_bias=s["dt_bias"].cuda())
    y_ref, h_ref = ref.scan(x, s["dt"], a, b, c, lens, s["h0"], s["d_skip"], s["dt_bias"])
    assert ref.rel(y.float(), y_ref) <= TOL["bf16"] and ref.rel(hT, h_ref) <= TOL["f32"]


def test_long_sums_keep_fp32(kda):
    # all terms of one sign and no decay, 32768 of them: the tensor cores cut off up to 2^-23 of a sum at each of a chunk's 8 steps, on
    # average half, and the chunks are added with rounding: below 4 * 2^-23 + 16 * 2^-24 < 2e-6 of the largest value, doubled
    T, H = 32768, 40
    gen = torch.Generator(device="cuda").manual_seed(5)
    f = lambda *s: torch.rand(*s, generator=gen, device="cuda")
    x, b, c, dt = f(T, H, 64).bfloat16(), f(T, 1, 128).bfloat16(), f(T, 1, 128).bfloat16(), f(T, H) * 0.1 + 0.01
    a = torch.full((H,), -1e-7, device="cuda")
    _, hT = kda.ssm_fwd(x, dt, a, b, c, dt_softplus=False)
    ha = dt.double() * a.double()
    w = torch.exp(ha.flip(0).cumsum(0).flip(0) - ha) * dt.double()
    for h in (0, 17, 39):
        want = b[:, 0].double().t() @ (w[:, h, None] * x[:, h].double())
        assert ref.rel(hT[0, h], want) <= 4e-6


@pytest.mark.parametrize("n,H,P,h0", [(90, 4, 64, True), (45, 3, 128, True), (270, 1, 64, False)])
def test_many_short_prompts(kda, n, H, P, h0):
    # more (sequence, head) pairs than SMs, of a chunk or two: CTAs go on from one to the next, past empty ones and short last chunks
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 300, (n,), generator=gen).tolist()
    lens[3] = lens[4] = lens[n - 1] = 0
    lens[5], lens[6], lens[7] = 1, 128, 256
    check(kda, lens, H, 1, P, "bf16", seed=n, h0=h0)


def test_many_short_prompts_twice(kda):
    lens = [129, 1, 127, 0, 64] * 24
    s = case(lens, 3, 1, 64, "bf16", 12)
    x, b, c = split(s["rows"].cuda(), 3, 1, 64)
    call = lambda: kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, s["cu"], s["h0"].cuda(), d_skip=s["d_skip"].cuda())
    (y, hT), (y1, hT1) = call(), call()
    assert torch.equal(y, y1) and torch.equal(hT, hT1)


def test_step_activation_in_fp32_entry_by_entry(kda):
    """With zero B rows and states, one tap of one and d_skip = 1, y is silu(x). In fp32 z / (1 + e^-z): the exponential within a unit in
    the last place (2^-23), the sum and the quotient rounded (2^-24 each): 2^-22 = 2.4e-7 of every entry, at any z with a finite e^-z."""
    H, P, G = 4, 64, 1
    z = torch.linspace(-85.0, 85.0, 40 * 8 * H * P).view(40, 8, H * P).cuda()
    xbc = torch.zeros(40, 8, H * P + 256, device="cuda")
    xbc[..., :H * P] = z
    C = H * P + 256
    y = kda.ssm_step(xbc, torch.zeros(40, 8, H).cuda(), -torch.ones(H).cuda(), torch.ones(C, 1).cuda(), None, None,
                     torch.zeros(40, H, 128, P).cuda(), d_skip=torch.ones(H).cuda())
    want = z.double() / (1.0 + torch.exp(-z.double()))
    err = (y.view_as(z).double() - want).abs() / want.abs()
    assert err.max().item() <= 2.5e-7


@pytest.mark.parametrize("n,H", [(6, 2), (200, 1), (60, 3), (256, 2)])
def test_packed_prompts_between_rows_of_nobody(kda, n, H):
    """Sequences taken by length, one CTA each or going on from one to the next: the lengths are put in order in the shared memory where
    the first tile arrives. The rows before the first and after the last sequence are not finite and stay out; twenty calls
    give the same bits."""
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 280, (n,), generator=gen).tolist()
    lens[0], lens[n // 2], lens[n - 1] = 130, 0, 3
    before, after, T = 77, 150, sum(lens)
    s = case([before] + lens + [after], H, 1, 64, "bf16", 13)
    rows = s["rows"].clone()
    rows[:before], rows[before + T:] = float("nan"), float("inf")
    cu, h0 = s["cu"][1:-1].cuda(), s["h0"][1:-1].cuda()
    x, b, c = split(rows.cuda(), H, 1, 64)
    call = lambda: kda.ssm_fwd(x, s["dt"].cuda(), s["a"].cuda(), b, c, cu, h0, d_skip=s["d_skip"].cuda())
    y, hT = call()
    inside = slice(before, before + T)
    y_ref, h_ref = ref.scan(x[inside], s["dt"][inside], s["a"], b[inside], c[inside], lens, h0, s["d_skip"])
    assert ref.rel(y[inside].float(), y_ref) <= TOL["bf16"] and ref.rel(hT, h_ref) <= TOL["f32"]
    for _ in range(20):
        y1, hT1 = call()
        assert torch.equal(y[inside], y1[inside]) and torch.equal(hT, hT1)
