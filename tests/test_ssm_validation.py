"""The short convolution and the selective scan: every refusal, by the C entry points (fake
addresses, nothing is launched) and by the Python binding (host tensors: a call that passed
every check stops at the device check), and the scan's plan. CPU only."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import chunkwise_delta_rule_kda_amd as kda
from oracle import selective_scan_fp64, short_conv_fp64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(not os.path.exists(kda.lib_path()),
                                reason="libkda.so not built (run __graft_entry__.build())")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
GB = 1 << 30
at = lambda i: BASE + i * GB


def conv_args(T=200, B=1, C=264, N=None, varlen=False, pool=False, **kw):
    N = (3 if varlen else B) if N is None else N
    d = dict(x=at(0), weight=at(1), bias=at(2), state_in=at(3), out=at(4), state_out=at(5), B=B,
             T=T, C=C, N=N, flags=1)
    if varlen:
        d["cu_seqlens"] = at(6)
    if pool:
        d.update(ssm_state_indices=at(7), state_pool_slots=9, state_out=None)
    d.update(kw)
    return kda.make_short_conv_args(**d)


def conv(*a, **kw):
    return kda.kda_short_conv_check(conv_args(*a, **kw))


def scan_args(T=200, B=1, D=192, N=None, varlen=False, pool=False, **kw):
    N = (3 if varlen else B) if N is None else N
    d = dict(u=at(0), delta=at(1), z=at(2), B_in=at(3), C_in=at(4), A=at(5), D_skip=at(6),
             delta_bias=at(7), state_in=at(8), out=at(9), state_out=at(10), workspace=at(11),
             workspace_bytes=GB, B=B, T=T, D=D, N=N, flags=1)
    if varlen:
        d["cu_seqlens"] = at(12)
    if pool:
        d.update(ssm_state_indices=at(13), state_pool_slots=9, state_out=None)
    d.update(kw)
    return kda.make_selective_scan_args(**d)


def scan(*a, **kw):
    return kda.kda_selective_scan_check(scan_args(*a, **kw))


def test_struct_sizes_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "kda.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu",'
                   'sizeof(kda_short_conv_args),sizeof(kda_selective_scan_args),'
                   'sizeof(kda_selective_scan_plan_info));return 0;}\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    from chunkwise_delta_rule_kda_amd.scan import kda_selective_scan_plan_info

    assert [int(x) for x in out] == [ctypes.sizeof(c) for c in (
        kda.kda_short_conv_args, kda.kda_selective_scan_args, kda_selective_scan_plan_info)]


def test_valid_calls_pass():
    assert conv() == 0 and conv(varlen=True) == 0 and conv(pool=True) == 0
    assert conv(bias=None, state_in=None, state_out=None, flags=0) == 0
    assert conv(state_out=at(3)) == 0 and conv(T=0, x=None, out=None) == 0
    assert conv(W=2, io_dtype=1, state_dtype=1) == 0 and conv(x_stride=(0, 0)) == 0
    assert conv(pool=True, state_out_indices=at(8), state_slot_pitch=800) == 0
    assert scan() == 0 and scan(varlen=True) == 0 and scan(pool=True) == 0
    assert scan(z=None, D_skip=None, delta_bias=None, state_in=None, state_out=None) == 0
    assert scan(state_out=at(8)) == 0 and scan(G=3) == 0 and scan(G=6) == 0
    assert scan(T=0, u=None, delta=None, z=None, B_in=None, C_in=None, out=None) == 0
    assert scan(T=8, workspace=None, workspace_bytes=0) == 0
    assert scan(segment_tokens=-1, workspace=None, workspace_bytes=0) == 0
    assert scan(S=8, io_dtype=1, state_dtype=1) == 0 and scan(D=8) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(weight=None), 1),
    (dict(C=0), 2), (dict(C=260), 2), (dict(C=(1 << 22) + 8), 2), (dict(W=1), 2), (dict(W=5), 2),
    (dict(B=0), 2), (dict(T=-1), 2), (dict(N=2), 2), (dict(T=(1 << 36) + 1), 2),
    (dict(T=1 << 36, C=1 << 22), 2), (dict(T=1 << 36), 2), (dict(B=1 << 31, N=1 << 31), 2),
    (dict(io_dtype=2), 3), (dict(state_dtype=-1), 3), (dict(flags=2), 4),
    (dict(x_stride=(0, -8)), 2), (dict(x_stride=(4, 264)), 2), (dict(x_stride=(0, (1 << 22) + 8)), 2),
    (dict(varlen=True, B=2), 2), (dict(varlen=True, N=0), 2),
    (dict(pool=True, state_in=None), 10), (dict(pool=True, state_pool_slots=0), 10),
    (dict(pool=True, state_slot_pitch=784), 10), (dict(pool=True, state_slot_pitch=796), 10),
    (dict(state_out_indices=at(8)), 10), (dict(pool=True, state_out=at(5)), 6),
    (dict(x=at(0) + 8), 2), (dict(weight=at(1) + 4), 2), (dict(state_in=at(3) + 8), 2),
    (dict(varlen=True, cu_seqlens=at(6) + 4), 2), (dict(pool=True, ssm_state_indices=at(7) + 2), 2),
    (dict(out=at(0)), 6), (dict(out=at(0) + 4096), 6), (dict(out=at(1)), 6), (dict(out=at(3)), 6),
    (dict(state_out=at(3) + 64), 6), (dict(state_out=at(0)), 6), (dict(state_out=at(4)), 6),
    (dict(pool=True, ssm_state_indices=at(3) + 256), 6),
])
def test_conv_refusals(kw, code):
    assert conv(**kw) == code, kda.kda_last_error()
    assert kda.kda_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(u=None), 1), (dict(delta=None), 1), (dict(B_in=None), 1), (dict(C_in=None), 1),
    (dict(A=None), 1), (dict(out=None), 1),
    (dict(D=0), 2), (dict(D=100), 2), (dict(D=(1 << 22) + 8), 2), (dict(S=4), 2), (dict(S=24), 2),
    (dict(S=128), 2), (dict(G=0), 2), (dict(G=5), 2), (dict(G=4), 2), (dict(G=-1), 2),
    (dict(B=0), 2), (dict(T=-1), 2), (dict(N=2), 2), (dict(T=(1 << 36) + 1), 2),
    (dict(T=1 << 36, D=1 << 16), 2), (dict(T=1 << 36, segment_tokens=64), 2),
    (dict(B=1 << 31, N=1 << 31), 2), (dict(B=1 << 25, N=1 << 25, T=4), 2),
    (dict(io_dtype=2), 3), (dict(state_dtype=-1), 3), (dict(flags=2), 4),
    (dict(segment_tokens=32), 10), (dict(segment_tokens=(1 << 40) + 64), 10),
    (dict(u_stride=(0, -8)), 2), (dict(delta_stride=(4, 192)), 2),
    (dict(z_stride=(0, (1 << 22) + 8)), 2), (dict(B_stride=(0, 16, 4)), 2),
    (dict(C_stride=(-8, 16, 16)), 2),
    (dict(varlen=True, B=2), 2), (dict(varlen=True, N=0), 2),
    (dict(pool=True, state_in=None), 10), (dict(pool=True, state_pool_slots=0), 10),
    (dict(pool=True, state_slot_pitch=64), 10), (dict(state_out_indices=at(14)), 10),
    (dict(pool=True, state_out=at(10)), 6),
    (dict(u=at(0) + 8), 2), (dict(A=at(5) + 4), 2), (dict(D_skip=at(6) + 2), 2),
    (dict(B_in=at(3) + 8), 2), (dict(state_in=at(8) + 8), 2),
    (dict(out=at(0)), 6), (dict(out=at(2) + 4096), 6), (dict(out=at(5)), 6), (dict(out=at(7)), 6),
    (dict(state_out=at(8) + 64), 6), (dict(state_out=at(4)), 6), (dict(state_out=at(9)), 6),
    (dict(pool=True, ssm_state_indices=at(8) + 256), 6),
    (dict(segment_tokens=64, workspace=None), 7), (dict(segment_tokens=64, workspace=at(11) + 64), 7),
    (dict(segment_tokens=64, workspace_bytes=1000), 7), (dict(segment_tokens=64, workspace=at(9)), 6),
])
def test_scan_refusals(kw, code):
    assert scan(**kw) == code, kda.kda_last_error()
    assert kda.kda_last_error() != ""


def test_null_arguments_and_launches_refuse_before_any_launch():
    lib = kda.load_library()
    assert lib.kda_short_conv_check(None) == 1 and lib.kda_short_conv(None, None) == 1
    assert lib.kda_selective_scan_check(None) == 1 and lib.kda_selective_scan(None, None) == 1
    assert lib.kda_selective_scan_plan(ctypes.byref(scan_args()), None) == 1
    assert lib.kda_selective_scan_workspace_bytes(ctypes.byref(scan_args()), None) == 1
    assert lib.kda_short_conv(ctypes.byref(conv_args(W=5)), None) == 2
    assert lib.kda_selective_scan(ctypes.byref(scan_args(S=4)), None) == 2


def test_scan_plan():
    plan = lambda **kw: kda.kda_selective_scan_plan(scan_args(**kw))
    p = plan(T=8)
    assert p["decode"] == 1 and p["workspace_bytes"] == 0 and p["segment_tokens"] == 0
    p = plan(T=8, segment_tokens=-1)
    assert p["decode"] == 0 and p["segment_tokens"] == 0 and p["workgroups"] == 6
    # few channels and a long prompt: segments; a wide layer fills the card without
    p = plan(T=8192, D=1536)
    assert 64 <= p["segment_tokens"] <= 1024 and p["segment_tokens"] % 64 == 0
    segs = -(-8192 // p["segment_tokens"])
    assert p["segments_bound"] == segs and p["workgroups"] == 48 * segs
    states = 1536 * 16 * 4
    need = segs * states + segs * 1536 * 4 + states
    assert need <= p["workspace_bytes"] <= need + 1024
    assert kda.kda_selective_scan_workspace_bytes(scan_args(T=8192, D=1536)) == p["workspace_bytes"]
    assert plan(T=8192, D=8192)["segment_tokens"] == 0
    assert plan(T=300, segment_tokens=128)["segments_bound"] == 3
    assert plan(T=300, segment_tokens=320)["segment_tokens"] == 0
    p = plan(T=300, segment_tokens=64, varlen=True, N=5)
    assert p["segments_bound"] == 300 // 64 + 5
    assert plan(T=6000, D=1536, varlen=True, N=1)["segment_tokens"] > 0
    assert plan(T=6000, D=1536, varlen=True, N=200)["segment_tokens"] == 0


# ---------------------------------------------------------------- the Python binding


def expect(code, text, fn, *a, **kw):
    with pytest.raises(kda.KdaError) as e:
        fn(*a, **kw)
    assert e.value.status == code and text in str(e.value), str(e.value)


def test_conv_binding():
    x, w, b = torch.zeros(2, 20, 64, dtype=torch.bfloat16), torch.zeros(64, 4), torch.zeros(64)
    go = lambda code, text, x=x, w=w, b=b, st=None, cu=None, **kw: expect(
        code, text, kda.kda_short_conv, x, w, b, st, cu, **kw)
    state = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    go(2, "CUDA tensor")
    go(2, "CUDA tensor", st=state)
    go(2, "must be a tensor", x=None)
    go(2, "must be a tensor", w=None)
    go(2, "three axes", x=x[0])
    go(3, "unsupported dtype", x=x.half())
    go(2, "last axis", x=x.transpose(1, 2).contiguous().transpose(1, 2))
    go(3, "weight", w=w.bfloat16())
    go(2, "weight must be", w=w[:32])
    go(2, "weight must be", w=torch.zeros(4, 64).t())
    go(2, "5 taps", w=torch.zeros(64, 5))
    go(2, "bias", b=b[:8])
    go(3, "bias", b=b.bfloat16())
    go(4, "activation", activation="relu")
    go(3, "cu_seqlens", cu=torch.zeros(3, dtype=torch.int32))
    go(2, "B = 1", cu=torch.zeros(3, dtype=torch.int64))
    go(2, "N + 1", cu=torch.zeros(1, dtype=torch.int64))
    go(2, "state_in has shape", st=state[:1])
    go(2, "state_in must be contiguous", st=torch.zeros(2, 64, 3, dtype=torch.bfloat16).transpose(1, 2))
    go(3, "state dtype is", st=state, state_dtype=torch.float32)
    go(3, "state dtype", state_dtype=torch.float16)
    go(2, "state_out has shape", state_out=state[:1])
    go(2, "must be a tensor", state_out=3)
    go(2, "out must be", out=x.float())
    ids = torch.zeros(2, dtype=torch.int32)
    go(10, "needs state_in", ssm_state_indices=ids)
    go(10, "needs ssm_state_indices", state_out_indices=ids)
    pool = torch.zeros(5, 3, 64, dtype=torch.bfloat16)
    go(2, "CUDA tensor", st=pool, ssm_state_indices=ids, state_out_indices=ids)
    go(10, "less than a slot", st=pool[:1].expand(5, 3, 64), ssm_state_indices=ids)
    go(2, "multiple of 8", st=torch.zeros(5, 196, dtype=torch.bfloat16)[:, :192].unflatten(1, (3, 64)),
       ssm_state_indices=ids)
    go(2, "slot must be contiguous", st=torch.zeros(5, 64, 3, dtype=torch.bfloat16).transpose(1, 2),
       ssm_state_indices=ids)
    go(3, "ssm_state_indices", st=pool, ssm_state_indices=ids.long())
    go(2, "state_out_indices", st=pool, ssm_state_indices=ids, state_out_indices=ids[:1])
    go(6, "with a state pool", st=pool, ssm_state_indices=ids, state_out=pool.clone())


def test_scan_binding():
    bf = torch.bfloat16
    u, A = torch.zeros(2, 20, 64, dtype=bf), torch.zeros(64, 16)
    B, D = torch.zeros(2, 20, 16, dtype=bf), torch.zeros(64)
    go = lambda code, text, u=u, delta=u, A=A, B=B, C=B, D=D, z=u, st=None, cu=None, **kw: expect(
        code, text, kda.kda_selective_scan, u, delta, A, B, C, D, z, st, cu, **kw)
    go(2, "CUDA tensor")
    go(2, "CUDA tensor", B=torch.zeros(2, 20, 2, 16, dtype=bf), C=torch.zeros(2, 20, 2, 16, dtype=bf))
    go(2, "must be a tensor", u=None)
    go(2, "must be a tensor", delta=None)
    go(2, "must be a tensor", B=None)
    go(2, "three axes", u=u[0])
    go(3, "unsupported dtype", u=u.half())
    go(3, "delta is", delta=u.float())
    go(2, "delta has shape", delta=u[:, :3])
    go(2, "z has shape", z=u[:1])
    go(3, "z is", z=u.float())
    go(2, "last axis of u", u=u.transpose(1, 2).contiguous().transpose(1, 2))
    go(3, "A is", A=A.bfloat16())
    go(2, "A must be", A=A[:8])
    go(2, "A must be", A=torch.zeros(16, 64).t())
    go(2, "B and C have shapes", C=B[:, :, :8])
    go(2, "B and C have shapes", B=torch.zeros(2, 20, 2, 16, dtype=bf))
    go(3, "C is", C=B.float())
    go(2, "last axis of B", B=torch.zeros(2, 16, 20, dtype=bf).transpose(1, 2))
    three = torch.zeros(2, 20, 3, 16, dtype=bf)
    go(2, "do not divide", B=three, C=three)
    go(2, "D must be", D=D[:3])
    go(3, "delta_bias", delta_bias=D.double())
    go(3, "cu_seqlens", cu=torch.zeros(3, dtype=torch.int32))
    go(2, "B = 1", cu=torch.zeros(3, dtype=torch.int64))
    go(2, "state_in has shape", st=torch.zeros(2, 16, 64))
    go(2, "out must be", out=u.float())
    go(2, "workspace", workspace=torch.zeros(100)[::2])
    ids = torch.zeros(2, dtype=torch.int32)
    go(10, "needs state_in", ssm_state_indices=ids)
    pool = torch.zeros(5, 64, 16)
    go(2, "CUDA tensor", st=pool, ssm_state_indices=ids)
    go(6, "with a state pool", st=pool, ssm_state_indices=ids, state_out=pool.clone())


# ---------------------------------------------------------------- the oracles


def test_oracles_against_written_out_sums():
    """The convolution as numpy's; one channel and state of the scan as the sum it stands for."""
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(1, 11, 3)), rng.normal(size=(3, 4))
    y, s, err = short_conv_fp64(x, w, silu=False)
    for c in range(3):
        want = np.convolve(x[0, :, c], w[c, ::-1])[:11]
        assert np.allclose(y[0, :, c], want, atol=1e-12)
    assert np.array_equal(s[0], x[0, -3:]) and np.all(err > 0)
    u, d = rng.normal(size=(1, 6, 1)), rng.uniform(0.1, 1, size=(1, 6, 1))
    A, B, C = -rng.uniform(0.1, 1, size=(1, 1)), rng.normal(size=(1, 6, 1, 1)), rng.normal(size=(1, 6, 1, 1))
    y, s, _, _ = selective_scan_fp64(u, d, A, B, C, softplus=False, state0=np.full((1, 1, 1), 2.0))
    for t in range(6):
        through = lambda j: np.exp(A[0, 0] * d[0, j:t + 1, 0].sum())
        h = 2.0 * through(0) + sum(through(j + 1) * d[0, j, 0] * u[0, j, 0] * B[0, j, 0, 0]
                                   for j in range(t + 1))
        assert np.isclose(y[0, t, 0], C[0, t, 0, 0] * h, atol=1e-12)
    assert np.isclose(s[0, 0, 0], h, atol=1e-12)
