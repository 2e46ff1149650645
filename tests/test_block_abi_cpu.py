"""CPU checks of the entry points around the recurrent core: struct layouts, and refusals before
anything touches a GPU."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # well-aligned, never dereferenced: validation fails first
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_chunked_gb300 import build, _lib
    build.build()
    return _lib.load()


def structs():
    from gated_delta_rule_chunked_gb300 import _lib
    return (("kda_ssm_args", _lib.SsmArgs), ("kda_ssm_step_args", _lib.SsmStepArgs),
            ("kda_draft_verify_args", _lib.DraftVerifyArgs), ("kda_block_norm_args", _lib.BlockNormArgs),
            ("kda_block_norm_bwd_args", _lib.BlockNormBwdArgs))


def test_struct_layout_matches_c(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kda.h"', "int main(void){"]
    for name, cls in structs():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "probe.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                           str(tmp_path / "probe.c"), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, cls in structs():
        assert int(got[name]) == C.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f"{name}.{f}"


def ssm(**over):
    from gated_delta_rule_chunked_gb300 import _lib
    a = _lib.SsmArgs()
    a.n_seqs, a.total_tokens, a.heads, a.groups, a.head_dim, a.d_state = 2, 64, 4, 2, 64, 128
    a.ldx, a.ldb, a.ldc = 256, 256, 256
    a.x = a.b = a.c = a.dt = a.a = a.y = FAKE
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(head_dim=32), UNSUPPORTED), (dict(d_state=64), UNSUPPORTED), (dict(io_dtype=3), UNSUPPORTED),
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(heads=0), INVALID), (dict(n_seqs=-1), INVALID),
    (dict(n_seqs=0), INVALID), (dict(total_tokens=63), INVALID), (dict(total_tokens=1 << 31), INVALID),
    (dict(ldx=248), INVALID), (dict(ldb=260), INVALID), (dict(x=None), INVALID), (dict(y=FAKE + 8), INVALID),
    (dict(dt=None), INVALID), (dict(a=None), INVALID), (dict(h0=FAKE + 4), INVALID), (dict(cu_seqlens=FAKE + 2), INVALID),
])
def test_ssm_validation(lib, over, status):
    assert lib.kda_ssm_fwd(C.byref(ssm(**over)), None) == status
    assert lib.kda_last_error().startswith(b"kda_ssm_fwd: ")


@pytest.mark.parametrize("io", [0, 1])
def test_ssm_item_limit(lib, io):
    """What the launch cannot number is refused with the other arguments, not as a CUDA error."""
    over = dict(io_dtype=io, n_seqs=32768, total_tokens=0, heads=65536, head_dim=64, ldx=65536 * 64)     # 2^31 items
    few = dict(over, n_seqs=16383, a=None)                                                               # just below 2^30
    if io == 0:
        over["n_seqs"] = 16384                                                                           # 2^30
    assert lib.kda_ssm_fwd(C.byref(ssm(**over)), None) == UNSUPPORTED
    assert b"must be below 2^30" in lib.kda_last_error()
    assert lib.kda_ssm_fwd_workspace_size(C.byref(ssm(**over))) == 0
    assert lib.kda_ssm_fwd(C.byref(ssm(**few)), None) == INVALID and b"a is NULL" in lib.kda_last_error()      # past that check


def step(**over):
    from gated_delta_rule_chunked_gb300 import _lib
    a = _lib.SsmStepArgs()
    a.n_seqs, a.steps, a.heads, a.groups, a.head_dim, a.d_state, a.width, a.activation = 2, 4, 4, 2, 64, 128, 4, 1
    a.xbc = a.conv_weight = a.conv_state = a.dt = a.a = a.state = a.y = a.workspace = FAKE
    a.workspace_bytes = 2 * 4 * (256 + 512) * 4
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(steps=9), INVALID), (dict(steps=0), INVALID), (dict(width=5), UNSUPPORTED), (dict(activation=4), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(groups=3), INVALID), (dict(state=None), INVALID), (dict(conv_state=None), INVALID),
    (dict(xbc=FAKE + 2), INVALID), (dict(state_indices=FAKE, n_slots=0), INVALID), (dict(workspace_bytes=24575), INVALID),
    (dict(workspace=None), INVALID), (dict(accept_len=FAKE + 1), INVALID), (dict(n_seqs=65536), INVALID),
])
def test_step_validation(lib, over, status):
    assert lib.kda_ssm_step_workspace_size(C.byref(step())) == 24576
    assert lib.kda_ssm_step(C.byref(step(**over)), None) == status


def verify(**over):
    from gated_delta_rule_chunked_gb300 import _lib
    a = _lib.DraftVerifyArgs()
    a.n_seqs, a.drafts, a.vocab, a.io_dtype = 2, 3, 100, 1
    a.p = a.draft = a.u = a.noise = a.accept_len = a.tokens = FAKE
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(drafts=0), INVALID), (dict(drafts=9), INVALID), (dict(vocab=0), INVALID), (dict(io_dtype=2), UNSUPPORTED),
    (dict(p=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(noise=None), INVALID), (dict(tokens=None), INVALID),
    (dict(draft=FAKE + 2), INVALID), (dict(first_slot=FAKE + 1), INVALID), (dict(n_seqs=-1), INVALID),
])
def test_verify_validation(lib, over, status):
    assert lib.kda_draft_verify(C.byref(verify(**over)), None) == status


def norm(**over):
    from gated_delta_rule_chunked_gb300 import _lib
    a = _lib.BlockNormArgs()
    a.rows, a.dim, a.eps = 4, 128, 1e-6
    a.u = a.out = a.normed = a.w_post = a.w_pre = a.rstd_post = a.rstd_pre = FAKE
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(dim=100), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(dim=16392), UNSUPPORTED), (dict(io_dtype=5), UNSUPPORTED),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rows=-1), INVALID), (dict(u=None), INVALID),
    (dict(gate=FAKE, gate_act=2), INVALID), (dict(residual=FAKE + 8), INVALID), (dict(rstd_post=None), INVALID),
    (dict(normed=None), INVALID), (dict(out=FAKE + 2), INVALID),
])
def test_norm_validation(lib, over, status):
    from gated_delta_rule_chunked_gb300 import _lib
    assert lib.kda_block_norm_fwd(C.byref(norm(**over)), None) == status
    b = _lib.BlockNormBwdArgs()
    b.fwd = norm()
    b.d_out = b.du = b.dw_post = b.dw_pre = FAKE
    assert lib.kda_block_norm_bwd(C.byref(b), None) == INVALID          # no workspace
    b.fwd = norm(dim=100)
    assert lib.kda_block_norm_bwd_workspace_size(C.byref(b)) == 0


def test_null_arguments(lib):
    for name in ("kda_ssm_fwd", "kda_ssm_step", "kda_draft_verify", "kda_block_norm_fwd", "kda_block_norm_bwd"):
        assert getattr(lib, name)(None, None) == INVALID


def test_tensors_on_another_device_are_refused(monkeypatch):
    """The library launches on the current device: a stream is only handed out for tensors that live there."""
    import torch
    import gated_delta_rule_chunked_gb300 as kda
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(kda, "_raw_stream", lambda index: 40 + index)
    assert kda._stream_of(torch.device("cuda", 0)) == 40
    with pytest.raises(ValueError, match="cuda:1"):
        kda._stream_of(torch.device("cuda", 1))
