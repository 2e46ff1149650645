"""GPU draft verification against the entry-by-entry definition: whole numbers, so no tolerance."""
import pytest
import torch

import block_fp64 as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_chunked_gb300 as m
    m.library()
    return m


def case(N, L, V, io, seed, drafter=True, near=0.5):
    gen = torch.Generator().manual_seed(seed)
    logits = torch.randn(N, L + 1, V, generator=gen) * 2
    p = torch.softmax(logits, -1).to(DT[io])
    q = torch.softmax(logits[:, :L] + near * torch.randn(N, L, V, generator=gen), -1).to(DT[io]) if drafter else None
    source = p[:, :L] if q is None else q
    draft = torch.multinomial(source.float().reshape(-1, V), 1, generator=gen).reshape(N, L).to(torch.int32)
    return p, q, draft, torch.rand(N, L, generator=gen), torch.empty(N, V).exponential_(generator=gen)


def cuda(t):
    return None if t is None else t.cuda()


def check(kda, p, q, draft, u, noise, lens=None):
    got = kda.draft_verify(cuda(p), cuda(q), cuda(draft), cuda(u), cuda(noise), cuda(lens))
    torch.cuda.synchronize()
    want = ref.verify(p, q, draft, u, noise, lens)
    for g, w in zip(got, want):
        assert g.dtype == torch.int32 and (g.cpu().numpy() == w).all()
    return want


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,V,drafter", [(1, 1, 1, True), (3, 4, 17, True), (5, 8, 1000, True), (4, 3, 4096, False), (2, 2, 9999, True), (17, 4, 256, False), (1, 4, 40009, True)])
def test_verify(kda, io, N, L, V, drafter):
    check(kda, *case(N, L, V, io, seed=N + L + V, drafter=drafter))


@pytest.mark.parametrize("V", [64, 65])
def test_every_outcome_occurs(kda, V):
    a, _, _ = check(kda, *case(64, 3, V, "f32", seed=1))
    assert set(a.tolist()) == {0, 1, 2, 3}


def test_all_stand_and_none_stands(kda):
    p, q, draft, u, noise = case(4, 3, 100, "f32", seed=2)
    a, _, _ = check(kda, p, q, draft, torch.zeros_like(u), noise)          # 0 < p
    assert (a == 3).all()
    same = p[:, :3].contiguous()
    a, _, _ = check(kda, p, same, draft, u, noise)                         # q = p, u < 1: u q < p
    assert (a == 3).all()
    p[0, 0, draft[0, 0]] = 0.0
    a, _, _ = check(kda, p, q, draft, torch.zeros_like(u), noise)          # a token of probability zero never stands
    assert a[0] == 0


def test_ragged_and_outside_drafts(kda):
    p, q, draft, u, noise = case(8, 4, 50, "bf16", seed=3)
    u.zero_()
    draft[3, 1], draft[4, 0], draft[5, 3] = -1, 50, 2 ** 31 - 1
    lens = torch.tensor([0, 1, 4, 4, 4, 4, 9, -3], dtype=torch.int32)
    a, _, t = check(kda, p, q, draft, u, noise, lens)
    assert a.tolist() == [0, 1, 4, 1, 0, 3, 4, 0]


@pytest.mark.parametrize("V", [8, 24, 33])
def test_empty_rows_ties_and_values_that_are_not_finite(kda, V):
    p, q, draft, u, noise = case(7, 1, V, "f32", seed=4)
    draft.zero_()
    u.fill_(0.99)
    p[:, 0, 0], q[:, 0, 0] = 0.0, 1.0                                      # rejected at once
    p[0, 0] = 0.0                                                          # nothing to draw from: -1
    p[1, 0], q[1, 0] = 0.1, 0.2                                            # r empty: the race over p
    p[1, 0, 0] = 0.0
    p[2, 0], q[2, 0], noise[2] = 0.25, 0.0, 1.0                            # all equal: the lowest index that is open
    p[2, 0, 0], q[2, 0, 0] = 0.0, 1.0
    p[3, 0, V - 1], noise[3, V // 2] = float("nan"), float("nan")
    p[4, 0] = float("nan")
    noise[5, V - 1] = 0.0                                                  # an infinite score
    p[5, 0, V - 1], q[5, 0, V - 1] = 0.5, 0.0
    p[6, 0, 2], q[6, 0, 2] = float("inf"), 0.0
    a, _, t = check(kda, p, q, draft, u, noise)
    assert (a == 0).all() and t[0, 0] == -1 and t[1, 0] > 0 and t[2, 0] == 1 and t[4, 0] == -1 and t[5, 0] == V - 1


def test_draws_follow_the_distribution(kda):
    """20000 sequences share one row; the next tokens' frequencies stay within five standard errors."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    N, V = 20000, 8
    row = torch.tensor([0.3, 0.05, 0.2, 0.05, 0.1, 0.1, 0.15, 0.05], device="cuda")
    p = row.expand(N, 2, V).contiguous()
    noise = torch.empty(N, V, device="cuda").exponential_(generator=gen)
    drafts = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    _, _, tokens = kda.draft_verify(p, None, drafts, torch.zeros(N, 1, device="cuda"), noise)
    freq = torch.bincount(tokens[:, 1].long(), minlength=V) / N
    assert ((freq - row).abs() <= 5 * torch.sqrt(row * (1 - row) / N)).all()
    # rejection: u just under 1 keeps 0.3 of the certain drafts; token 0 is left out of the rest
    u = torch.rand(N, 1, generator=gen, device="cuda")
    a, _, tokens = kda.draft_verify(p, None, drafts, u, noise)
    assert abs(a.float().mean().item() - 0.3) <= 5 * (0.3 * 0.7 / N) ** 0.5
    assert (tokens[a == 0][:, 0] > 0).all()
    first = torch.bincount(tokens[:, 0].long(), minlength=V) / N           # the sampled token is a draw from p itself
    assert ((first - row).abs() <= 5 * torch.sqrt(row * (1 - row) / N)).all()


def test_feeds_the_step(kda):
    """first_slot and accept_len go into a replay as they are."""
    p, q, draft, u, noise = case(6, 3, 64, "f32", seed=6)
    accept, first, tokens = kda.draft_verify(p.cuda(), q.cuda(), draft.cuda(), u.cuda(), noise.cuda())
    assert torch.equal(first + accept, torch.full_like(first, 3))
    assert ((tokens >= 0).sum(1) == accept + 1).all()


def test_refusals(kda):
    p, q, draft, u, noise = [cuda(t) for t in case(2, 3, 32, "f32", seed=7)]
    with pytest.raises(TypeError):
        kda.draft_verify(p, q.bfloat16(), draft, u, noise)
    with pytest.raises(TypeError):
        kda.draft_verify(p, q, draft.long(), u, noise)
    with pytest.raises(ValueError):
        kda.draft_verify(p, q[:, :2].contiguous(), draft, u, noise)
    with pytest.raises(ValueError):
        kda.draft_verify(p.transpose(0, 1), q, draft, u, noise)
    with pytest.raises(kda.KdaError):
        kda.draft_verify(p[:, :1].contiguous(), None, draft[:, :0].contiguous(), u[:, :0].contiguous(), noise)   # no drafts
    with pytest.raises(TypeError):
        kda.draft_verify(p.double(), q.double(), draft, u, noise)


def accepted(kda):
    """Eight sequences of four drafts: draft_verify's accept_len and first_slot, every count among them."""
    p, q, draft, _, noise = case(8, 4, 32, "f32", seed=9)
    u = torch.zeros(8, 4)
    for i, n in enumerate((0, 1, 2, 3, 4, 2, 1, 4)):
        if n < 4:
            p[i, n, draft[i, n]] = 0.0                                     # draft n falls
    accept, first, _ = kda.draft_verify(p.cuda(), q.cuda(), draft.cuda(), u.cuda(), noise.cuda())
    assert accept.tolist() == [0, 1, 2, 3, 4, 2, 1, 4]
    return accept, first


def commit(kda, op, rows, state, accept=None, first=None):
    """One call of a recurrent step over `rows` (slots on axis 1); the states after it."""
    state = [t.clone() for t in state]
    if op == "kda":
        kda.kda_step(*rows, state[0], accept, scale=128 ** -0.5, first_slot=first)
    elif op == "conv":
        kda.conv_step(rows[0], rows[1][0, 0], None, state[0], accept, first_slot=first)
    else:
        kda.ssm_step(rows[0], rows[1], -torch.ones(2, device="cuda"), rows[2][0, 0], None, state[1], state[0], accept, first_slot=first)
    return state


def step_inputs(op):
    """Rows [8, 4, ...] of fp32 inputs (a weight is one for all slots) and the states of eight sequences."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    if op == "kda":
        return [r(8, 4, 2, 128), r(8, 4, 2, 128), r(8, 4, 2, 128), torch.sigmoid(r(8, 4, 2)), -torch.rand(8, 4, 2, 128, device="cuda", generator=gen)], \
            [r(8, 2, 128, 128)]
    channels = 64 if op == "conv" else 2 * 64 + 256
    weight = r(channels, 4)[None, None].expand(8, 4, -1, -1)
    if op == "conv":
        return [r(8, 4, channels), weight], [r(8, 3, channels)]
    return [r(8, 4, channels), r(8, 4, 2), weight], [r(8, 2, 128, 64), r(8, 3, channels)]


@pytest.mark.parametrize("by", ["accept_len", "first_slot"])
@pytest.mark.parametrize("op", ["kda", "conv", "ssm"])
def test_accepted_drafts_reach_the_states(kda, op, by):
    """Either output of draft_verify, as documented, commits exactly the accepted prefix: the states are those of a call over that
    prefix alone. fp32 sums of at most 128 products over at most 4 tokens, twice: 2 * 4 * 128 * 2^-24 < 1e-4 of the largest value; the
    convolution's state holds copies."""
    accept, first = accepted(kda)
    rows, state = step_inputs(op)
    if by == "accept_len":
        got = commit(kda, op, rows, state, accept=accept)
    else:                                                                  # draft j moves to slot first_slot + j
        moved = [torch.full_like(t, 7.0) if t.stride(0) else t for t in rows]   # padding is not read
        for new, t in zip(moved, rows):
            for i, n in enumerate(accept.tolist()):
                if t.stride(0):
                    new[i, 4 - n:] = t[i, :n]
        got = commit(kda, op, moved, state, first=first)
    for i, n in enumerate(accept.tolist()):
        before = [t[i:i + 1] for t in state]
        want = commit(kda, op, [t[i:i + 1, :n].contiguous() if t.stride(0) else t[i:i + 1, :n] for t in rows], before) if n else before
        for g, w in zip(got, want):
            exact = n == 0 or g.dim() == 3
            assert torch.equal(g[i:i + 1], w) if exact else ref.rel(g[i:i + 1], w) <= 1e-4


@pytest.mark.parametrize("op", ["kda", "conv", "ssm"])
def test_both_outputs_together_commit_less(kda, op):
    """accept_len counts from slot 0: with first_slot = L - accept_len beside it, up to half of the drafts commit nothing."""
    accept, first = accepted(kda)
    rows, state = step_inputs(op)
    got = commit(kda, op, rows, state, accept=accept, first=first)
    for i, n in enumerate(accept.tolist()):
        if 2 * n <= 4:
            assert all(torch.equal(g[i], s[i]) for g, s in zip(got, state))


@pytest.mark.parametrize("V", [1000, 1001])
def test_captured_in_a_graph(kda, V):
    """Captured on one set of inputs and replayed on others in their place."""
    first, second = ([cuda(t) for t in case(9, 3, V, "f32", seed=s)] for s in (21, 22))
    args = [t.clone() for t in first]
    kda.draft_verify(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.draft_verify(*args)
    for values in (first, second):
        for a, v in zip(args, values):
            a.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.verify(*[t.cpu() for t in values])
        assert all((g.cpu().numpy() == w).all() for g, w in zip(got, want))
