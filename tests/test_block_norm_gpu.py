"""GPU parity of the block norm and its gradients against the fp64 formula and against differences.

Tolerances as a share of the largest value: bf16 results round once (2^-9 of a value), 5e-3 with the
gradient's own cancellation; fp32 results carry sums of up to 16384 terms held pairwise in 512
threads (about 40 roundings deep) and the gate's exponential (2^-21), 2e-5; gradients of the weights
sum over rows in fp32 as well."""
import pytest
import torch

import block_fp64 as ref

pytestmark = pytest.mark.gpu
TOL = {"bf16": 5e-3, "f32": 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ALL = dict(post=True, gate="silu", residual=True, scale=True, pre=True)


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_chunked_gb300 as m
    m.library()
    return m


def case(rows, dim, io, seed, post=True, gate="silu", residual=True, scale=True, pre=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda on, k=1.0: (torch.randn(rows, dim, generator=gen) * k).to(DT[io]) if on else None
    v = lambda on, lo, hi: torch.rand(dim, generator=gen) * (hi - lo) + lo if on else None
    return dict(u=r(True, 2.0), gate=r(gate is not None, 2.0), residual=r(residual, 3.0), w_post=v(post, 0.5, 1.5),
                scale=v(scale, -1.0, 1.0), w_pre=v(pre, 0.5, 1.5)), dict(d_out=r(True), d_normed=r(pre)), gate or "silu"


def cuda(t):
    return None if t is None else t.cuda()


def kernel(kda, s, act, fwd=True, grads=None):
    g = {k: cuda(v) for k, v in s.items()}
    kw = dict(gate=g["gate"], gate_act=act, residual=g["residual"], scale=g["scale"], w_pre=g["w_pre"], eps=1e-5)
    out, normed, stats = kda.block_norm_fwd(g["u"], g["w_post"], **kw)
    back = kda.block_norm_bwd(g["u"], g["w_post"], stats, cuda(grads["d_out"]), cuda(grads["d_normed"]), **kw) if grads else None
    torch.cuda.synchronize()
    return out, normed, stats, back


def check(kda, rows, dim, io, seed, **opts):
    s, grads, act = case(rows, dim, io, seed, **opts)
    out, normed, stats, back = kernel(kda, s, act, grads=grads)
    v = {k: None if t is None else t.double().requires_grad_() for k, t in s.items()}
    o_ref, n_ref = ref.block_norm(v["u"], v["w_post"], v["gate"], act, v["residual"], v["scale"], v["w_pre"], 1e-5)
    errs = {"out": ref.rel(out.float(), o_ref)}
    loss = (o_ref * grads["d_out"].double()).sum()
    if n_ref is not None:
        errs["normed"] = ref.rel(normed.float(), n_ref)
        loss = loss + (n_ref * grads["d_normed"].double()).sum()
    else:
        assert normed is None
    loss.backward()
    bad = {k: e for k, e in errs.items() if not e <= TOL[io]}
    for k, name in (("u", "du"), ("gate", "dgate"), ("residual", "dresidual"), ("w_post", "dw_post"), ("scale", "dscale"), ("w_pre", "dw_pre")):
        if v[k] is None:
            assert back[name] is None
            continue
        e = ref.rel(back[name].float(), v[k].grad)
        if not e <= (TOL[io] if k in ("u", "gate", "residual") else TOL["f32"]):
            bad[name] = e
    assert not bad, bad


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 16), (130, 24), (77, 64), (1000, 128), (65, 200), (33, 256), (9, 264), (5, 1000),
                                      (7, 2048), (4, 2056), (3, 7168), (700, 1544), (2, 8192), (3, 8200), (2, 16384)])
def test_shapes(kda, io, rows, dim):
    check(kda, rows, dim, io, rows + dim, **ALL)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [128, 520, 3080])
@pytest.mark.parametrize("opts", [
    dict(ALL, gate=None), dict(ALL, gate="sigmoid"), dict(ALL, scale=False), dict(ALL, residual=False), dict(ALL, pre=False),
    dict(ALL, post=False), dict(ALL, post=False, gate=None, scale=False), dict(post=True, gate="sigmoid", residual=False, scale=False, pre=False),
    dict(post=True, gate=None, residual=False, scale=False, pre=False), dict(post=False, gate="silu", residual=True, scale=False, pre=False),
])
def test_parts(kda, io, dim, opts):
    check(kda, 37, dim, io, dim, **opts)


def test_more_rows_than_a_wave(kda):
    check(kda, 3001, 264, "f32", 1, **ALL)
    check(kda, 20001, 40, "f32", 2, **ALL)


@pytest.mark.parametrize("dim", [128, 2056])
def test_absent_gradients_are_zero(kda, dim):
    s, grads, act = case(21, dim, "f32", 3)
    for part in ("d_out", "d_normed"):
        zero = dict(grads, **{part: torch.zeros_like(grads[part])})
        none = dict(grads, **{part: None})
        a, b = kernel(kda, s, act, grads=zero)[3], kernel(kda, s, act, grads=none)[3]
        for k in a:
            assert ref.rel(b[k], a[k]) <= 1e-6, (part, k)


@pytest.mark.parametrize("dim", [64, 1544])
def test_gradient_against_differences(kda, dim):
    """The gradient along a direction is the fp64 forward's central difference, for every input."""
    s, grads, act = case(6, dim, "f32", 4)
    back = kernel(kda, s, act, grads=grads)[3]
    gen = torch.Generator().manual_seed(5)

    def loss(v):
        out, normed = ref.block_norm(v["u"], v["w_post"], v["gate"], act, v["residual"], v["scale"], v["w_pre"], 1e-5)
        return ((out * grads["d_out"].double()).sum() + (normed * grads["d_normed"].double()).sum()).item()

    base = {k: t.double() for k, t in s.items()}
    for k, name in (("u", "du"), ("gate", "dgate"), ("residual", "dresidual"), ("w_post", "dw_post"), ("scale", "dscale"), ("w_pre", "dw_pre")):
        e = torch.randn(s[k].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss(dict(base, **{k: base[k] + h * e})) - loss(dict(base, **{k: base[k] - h * e}))) / (2 * h)
        got = (back[name].double().cpu() * e).sum().item()
        scale = (back[name].double().cpu().norm() * e.norm()).item()     # differences err by h^2, sums by 2^-24
        assert abs(got - diff) <= 1e-5 * scale, (name, got, diff)


@pytest.mark.parametrize("dim", [128, 1000])
def test_rows_of_zeros_and_large_values(kda, dim):
    s, grads, act = case(5, dim, "f32", 6)
    s["u"][1] = 0.0
    s["residual"][1] = 0.0                                     # out = 0 too: normed = 0, not NaN
    s["u"][2] *= 1e15
    s["gate"][3] = -100.0                                      # a shut gate
    s["gate"][4] = 100.0
    out, normed, stats, back = kernel(kda, s, act, grads=grads)
    for t in (out, normed, *stats, *back.values()):
        assert torch.isfinite(t).all()
    assert (out[1] == 0).all() and (normed[1] == 0).all()


def test_status_stays_clear_and_streams(kda):
    s, grads, act = case(1500, 4096, "bf16", 9)
    g = {k: cuda(v) for k, v in s.items()}
    kw = dict(gate=g["gate"], gate_act=act, residual=g["residual"], scale=g["scale"], w_pre=g["w_pre"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    do, dn = cuda(grads["d_out"]), cuda(grads["d_normed"])
    _, _, stats = kda.block_norm_fwd(g["u"], g["w_post"], **kw)
    a = kda.block_norm_bwd(g["u"], g["w_post"], stats, do, dn, dev_status=status, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = kda.block_norm_bwd(g["u"], g["w_post"], stats, do, dn, dev_status=status, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert int(status) == 0 and all(torch.equal(a[k], b[k]) for k in a)


def test_captured_in_a_graph(kda):
    s, grads, act = case(40, 1544, "bf16", 10)
    g = {k: cuda(v) for k, v in s.items()}
    kw = dict(gate=g["gate"], gate_act=act, residual=g["residual"], scale=g["scale"], w_pre=g["w_pre"])
    do, dn = cuda(grads["d_out"]), cuda(grads["d_normed"])
    run = lambda: (lambda f: (f, kda.block_norm_bwd(g["u"], g["w_post"], f[2], do, dn, **kw)))(kda.block_norm_fwd(g["u"], g["w_post"], **kw))
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], want[0][0]) and all(torch.equal(got[1][k], want[1][k]) for k in want[1])


def test_same_call_same_bits(kda):
    s, grads, act = case(999, 1544, "bf16", 7)
    a, b = kernel(kda, s, act, grads=grads), kernel(kda, s, act, grads=grads)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[3][k], b[3][k]) for k in a[3])


def test_no_rows(kda):
    s, grads, act = case(0, 128, "bf16", 8)
    out, normed, stats, back = kernel(kda, s, act, grads=grads)
    assert out.shape == (0, 128) and (back["dw_post"] == 0).all() and (back["dw_pre"] == 0).all() and (back["dscale"] == 0).all()


def test_heads_as_rows(kda):
    """The output norm of a recurrent core: u [T, H, d] with a gate of the same shape."""
    u, z = torch.randn(11, 3, 128).cuda(), torch.randn(11, 3, 128).cuda()
    w = torch.rand(128).cuda()
    out, _, _ = kda.block_norm_fwd(u, w, gate=z, gate_act="sigmoid")
    want, _ = ref.block_norm(u.double().cpu(), w.double().cpu(), z.double().cpu(), "sigmoid", None, None, None, 1e-6)
    assert out.shape == u.shape and ref.rel(out, want) <= TOL["f32"]


def test_refusals(kda):
    u, w = torch.randn(4, 128).cuda(), torch.ones(128).cuda()
    with pytest.raises(kda.KdaError):
        kda.block_norm_fwd(torch.randn(4, 100).cuda(), torch.ones(100).cuda())
    with pytest.raises(kda.KdaError):
        kda.block_norm_fwd(u, w, eps=0.0)
    with pytest.raises(ValueError):
        kda.block_norm_fwd(u.t(), w)
    with pytest.raises(ValueError):
        kda.block_norm_fwd(u, w[:64])
    with pytest.raises(TypeError):
        kda.block_norm_fwd(u, w, gate=u.bfloat16())
    with pytest.raises(TypeError):
        kda.block_norm_fwd(u.half(), w)
    with pytest.raises(KeyError):
        kda.block_norm_fwd(u, w, gate=u, gate_act="relu")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sizes_in_turn(kda, io):
    # the sizes share kernels but not their shared memory: small ones between large ones change nothing
    for dim in (7168, 2056, 16384, 264, 7168, 16384, 128, 2056):
        check(kda, 5, dim, io, dim, **ALL)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dim", [128, 264, 1544, 2056])
def test_gate_in_fp32_entry_by_entry(kda, act, dim):
    """Without norms and sums out = u act(z), du = D act(z) and dgate = D u act'(z), entry by entry. In units of 2^-24 of a value: the
    exponential 2, the sum and the reciprocal 1 each, so 4 of the sigmoid s, 5 of g = z s, and 6 of each product with them. The
    slopes s + g - g s and s - s s end 12 off the sum of their terms' sizes, counting the products with D and u. Half a unit is
    left for the second order."""
    gen = torch.Generator().manual_seed(dim)
    rows = 50
    z = torch.linspace(-85.0, 85.0, rows * dim)[torch.randperm(rows * dim, generator=gen)].view(rows, dim)
    u, D = (torch.rand(rows, dim, generator=gen) + 0.5 for _ in range(2))
    out, _, stats = kda.block_norm_fwd(u.cuda(), None, gate=z.cuda(), gate_act=act)
    back = kda.block_norm_bwd(u.cuda(), None, stats, D.cuda(), gate=z.cuda(), gate_act=act)
    u, z, D = u.double(), z.double(), D.double()
    s = 1.0 / (1.0 + torch.exp(-z))
    g = s if act == "sigmoid" else z * s
    slope = s * (1.0 - s) if act == "sigmoid" else s + g * (1.0 - s)
    size = s + s * s if act == "sigmoid" else s + g.abs() + g.abs() * s
    errs = {name: ((got.cpu().double() - want).abs() / size).max().item() * 2 ** 24 for name, got, want, size in (
        ("out", out, u * g, u * g.abs()), ("du", back["du"], D * g, D * g.abs()), ("dgate", back["dgate"], D * u * slope, D * u * size))}
    assert errs["out"] <= 6.5 and errs["du"] <= 6.5 and errs["dgate"] <= 12.5, errs


@pytest.mark.parametrize("io,rows,dim", [("f32", 2900, 1544), ("f32", 2100, 2048), ("f32", 700, 8192), ("bf16", 1500, 7168), ("f32", 457, 16384),
                                         ("bf16", 2600, 1032)])
def test_rows_round_the_ring(kda, io, rows, dim):
    """Rings of three buffers (fp32 of 1544, 2048 and 8192 columns) and more, each filled several times over."""
    check(kda, rows, dim, io, dim, **ALL)
