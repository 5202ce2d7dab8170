"""Linear attention with one decay per head, the pool's slot operations and the gated norm:
every refusal, by the C entry points (fake addresses, nothing is launched) and by the Python
binding (host tensors: a call that passed every check stops at the device check). CPU only."""

import ctypes
import os
import subprocess

import pytest

import chunkwise_delta_rule_kda_amd as kda

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(not os.path.exists(kda.lib_path()),
                                reason="libkda.so not built (run __graft_entry__.build())")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
GB = 1 << 30
at = lambda i: BASE + i * GB


def lin(T=200, B=1, H=4, N=None, varlen=False, pool=False, **kw):
    N = (3 if varlen else B) if N is None else N
    d = dict(q=at(0), k=at(1), v=at(2), g=at(3), log_decay=at(4), state_in=at(5), o=at(6),
             state_out=at(7), workspace=at(8), workspace_bytes=GB, B=B, T=T, H=H, N=N)
    if varlen:
        d["cu_seqlens"] = at(9)
    if pool:
        d.update(ssm_state_indices=at(10), state_pool_slots=9, state_out=None)
    d.update(kw)
    return kda.make_linear_args(**d)


def status(*a, **kw):
    return kda.kda_linear_check(lin(*a, **kw))


def test_struct_sizes_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "kda.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu %zu %zu %zu",'
                   'sizeof(kda_linear_args),sizeof(kda_linear_plan_info),sizeof(kda_pool),'
                   'sizeof(kda_pool_copy_args),sizeof(kda_pool_compact_args),'
                   'sizeof(kda_gated_norm_args));return 0;}\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    from chunkwise_delta_rule_kda_amd.linear import kda_linear_plan_info

    assert [int(x) for x in out] == [ctypes.sizeof(c) for c in (
        kda.kda_linear_args, kda_linear_plan_info, kda.kda_pool, kda.kda_pool_copy_args,
        kda.kda_pool_compact_args, kda.kda_gated_norm_args)]


def test_valid_calls_pass():
    assert status() == 0 and status(varlen=True) == 0 and status(pool=True) == 0
    assert status(pool=True, state_out_indices=at(11)) == 0
    assert status(g=None, log_decay=None, state_in=None, state_out=None) == 0
    assert status(state_out=at(5)) == 0
    assert status(K=64, V=512, Hk=2, io_dtype=1, state_dtype=1, g_dtype=0) == 0
    assert status(T=0, q=None, k=None, v=None, o=None) == 0
    assert status(T=4, workspace=None, workspace_bytes=0) == 0
    assert status(q_stride=(0, 0, 0), k_stride=(1 << 30, 1 << 22, 1 << 12)) in (0, 6)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1),
    (dict(K=96), 2), (dict(K=256), 2), (dict(V=32), 2), (dict(V=100), 2), (dict(V=576), 2),
    (dict(H=0, Hk=1), 2), (dict(Hk=3), 2), (dict(Hk=8), 2), (dict(Hk=-1), 2), (dict(T=-1), 2),
    (dict(B=0), 2), (dict(N=2), 2), (dict(T=(1 << 36) + 1), 2), (dict(H=70000), 2),
    (dict(T=1 << 36, H=30000), 2), (dict(H=1 << 33), 2), (dict(B=1 << 31, N=1 << 31), 2),
    (dict(io_dtype=2), 3), (dict(state_dtype=-1), 3), (dict(g_dtype=5), 3),
    (dict(scale=float("nan")), 5), (dict(scale=-1.0), 5),
    (dict(segment_tokens=63), 10), (dict(segment_tokens=1 << 41), 10),
    (dict(q_stride=(0, -8, 128)), 2), (dict(k_stride=(0, 132, 128)), 2),
    (dict(v_stride=(0, (1 << 22) + 8, 128)), 2),
    (dict(varlen=True, B=2), 2), (dict(varlen=True, N=0), 2),
    (dict(pool=True, state_in=None), 10), (dict(pool=True, state_pool_slots=0), 10),
    (dict(pool=True, state_slot_pitch=64), 10),
    (dict(pool=True, state_slot_pitch=4 * 128 * 128 + 4), 10),
    (dict(state_out_indices=at(11)), 10),
    (dict(pool=True, state_out=at(7)), 6),
    (dict(q=at(0) + 8), 2), (dict(state_in=at(5) + 8), 2), (dict(g=at(3) + 2), 2),
    (dict(o=at(0)), 6), (dict(o=at(2) + 4096), 6), (dict(o=at(3)), 6), (dict(o=at(4)), 6),
    (dict(state_out=at(5) + 64), 6), (dict(state_out=at(1)), 6), (dict(state_out=at(6)), 6),
    (dict(pool=True, ssm_state_indices=at(5) + 256), 6),
    (dict(segment_tokens=64, workspace=None), 7), (dict(segment_tokens=64, workspace=at(8) + 64), 7),
    (dict(segment_tokens=64, workspace_bytes=1000), 7), (dict(segment_tokens=64, workspace=at(6)), 6),
    (dict(T=8), 0), (dict(T=8, segment_tokens=-1), 0),
])
def test_linear_refusals(kw, code):
    assert status(**kw) == code, kda.kda_last_error()
    assert (kda.kda_last_error() == "") == (code == 0)


def test_linear_null_and_launch_refuse_before_any_launch():
    lib = kda.load_library()
    assert lib.kda_linear_check(None) == 1 and lib.kda_linear(None, None) == 1
    assert lib.kda_linear_plan(ctypes.byref(lin()), None) == 1
    assert lib.kda_linear_workspace_bytes(ctypes.byref(lin()), None) == 1
    assert lib.kda_linear(ctypes.byref(lin(K=96)), None) == 2
    assert lib.kda_pool_copy(None, None) == 1 and lib.kda_pool_compact(None, None) == 1
    assert lib.kda_gated_norm(None, None) == 1


def test_sizes_past_one_launch_are_refused():
    # H * V wraps to 0 in 64 bits; a launch of 2^32 threads is past what HIP takes
    assert status(H=1 << 57) == 2 and status(H=(1 << 22) + 1) == 2
    tokens = dict(T=1, H=16, io_dtype=1, state_dtype=1, g=None, log_decay=None, state_in=None,
                  state_out=None, workspace=None, workspace_bytes=0, q=at(0), k=at(200),
                  v=at(400), o=at(900))
    assert status(B=(1 << 17) - 1, **tokens) == 0      # 8 workgroups of 256 threads per head
    assert status(B=1 << 17, **tokens) == 2
    wide = dict(x=at(0), out=at(200), gate=None, res=None, w=None, nw=None, nxt=None, G=1,
                D=16384, xs=(16384, 16384))
    assert norm(M=(1 << 22) - 1, **wide) == 0 and norm(M=(1 << 23), **wide) == 2
    narrow = dict(wide, D=64, xs=(64, 64))
    assert norm(M=(1 << 29) - 64, **narrow) == 0 and norm(M=1 << 29, **narrow) == 2
    assert copy(src=pool(slots=1 << 25, elems=8), dst=pool(9, slots=1 << 25, elems=8),
                si=at(20), di=at(21), pairs=1 << 24) == 2


def test_linear_plan():
    plan = lambda **kw: kda.kda_linear_plan(lin(**kw))
    for T in (1, 8):
        p = plan(T=T)
        assert p["decode"] == 1 and p["workspace_bytes"] == 0 and p["segment_tokens"] == 0
    assert plan(T=9)["decode"] == 0 and plan(T=8, segment_tokens=-1)["decode"] == 0
    assert plan(T=8, varlen=True)["decode"] == 0
    p = plan(T=1000, segment_tokens=128)
    assert p["segment_tokens"] == 128 and p["segments_bound"] == 8
    assert p["workspace_bytes"] >= 8 * 4 * (128 * 128 * 4 + 4)
    p = plan(T=1000, segment_tokens=128, varlen=True)
    assert p["segments_bound"] == 1000 // 128 + 3
    assert plan(T=1000, segment_tokens=-1)["workspace_bytes"] == 0
    # a segment as long as the call is none
    assert plan(T=128, segment_tokens=128)["segment_tokens"] == 0


def pool(i=0, slots=9, layers=1, elems=1024, pitch=None, layer=None, dtype=0):
    pitch = elems if pitch is None else pitch
    return kda.kda_pool(at(i), slots, layers, elems, pitch,
                        slots * pitch if layer is None else layer, dtype)


def copy(src=None, dst=None, si=at(3), di=at(4), pairs=5):
    a = kda.kda_pool_copy_args(src or pool(), dst or pool(1), si, di, pairs)
    return kda.load_library().kda_pool_copy_check(ctypes.byref(a))


def test_pool_copy_refusals():
    assert copy() == 0 and copy(dst=pool(0)) == 0 and copy(pairs=0, si=None, di=None) == 0
    assert copy(src=pool(layers=3), dst=pool(1, layers=3, dtype=1)) == 0
    assert copy(src=pool(layers=3, pitch=4096, layer=1024), dst=pool(1, layers=3)) == 0
    assert copy(src=pool(dtype=2)) == 3
    for bad in (dict(slots=0), dict(layers=0), dict(elems=0), dict(elems=1028),
                dict(slots=(1 << 31) + 1), dict(elems=1 << 41)):
        assert copy(src=pool(**bad)) == 2, bad
    for bad in (dict(pitch=1016), dict(pitch=1028), dict(layers=2, layer=512),
                dict(layers=3, pitch=2048, layer=1024), dict(layer=-8)):
        assert copy(src=pool(**bad)) == 10, bad
    assert copy(src=pool(elems=2048)) == 2 and copy(src=pool(layers=2)) == 2
    assert copy(pairs=-1) == 2 and copy(pairs=(1 << 31) + 1) == 2
    assert copy(si=None) == 1 and copy(di=None) == 1 and copy(si=at(3) + 2) == 2
    n = pool()
    n.base = None
    assert copy(src=n) == 1
    n.base = at(0) + 8
    assert copy(src=n) == 2
    n.base = at(1) + 2048          # inside dst, but another pool
    assert copy(src=n) == 6
    assert copy(src=pool(1, dtype=1)) == 6      # dst's memory as another type
    assert copy(di=at(1) + 64) == 6 and copy(si=at(1)) == 6
    big = dict(slots=100000, elems=1 << 30)
    assert copy(src=pool(**big), dst=pool(1, **big), pairs=1 << 20) in (2, 6)


def compact(p=None, idx=at(3), new=at(4), count=at(5), n=5, ws=at(6), size=4096):
    a = kda.kda_pool_compact_args(p or pool(), idx, new, count, n, ws, size)
    return kda.load_library().kda_pool_compact_check(ctypes.byref(a))


def test_pool_compact_refusals():
    assert compact() == 0 and compact(new=at(3)) == 0 and compact(n=0, idx=None, new=None) == 0
    assert compact(p=pool(slots=kda.KDA_POOL_COMPACT_SLOTS + 1)) == 2
    assert compact(idx=None) == 1 and compact(new=None) == 1 and compact(count=None) == 1
    assert compact(n=-1) == 2 and compact(idx=at(3) + 1) == 2
    assert compact(ws=None) == 7 and compact(size=40) == 7 and compact(ws=at(6) + 16) == 7
    assert compact(new=at(3) + 4) == 6 and compact(count=at(4)) == 6 and compact(idx=at(0)) == 6
    assert compact(ws=at(0)) == 6 and compact(count=at(6)) == 6
    n = ctypes.c_size_t()
    a = kda.kda_pool_compact_args(pool(), None, None, None, 5, None, 0)
    assert kda.load_library().kda_pool_compact_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value >= 4 * 11


def norm(x=at(0), gate=at(1), res=at(2), w=at(3), nw=at(4), out=at(5), nxt=at(6), M=4, G=2, D=128,
         xs=(256, 128), gs=(256, 128), rs=(256, 128), io=0, act=0, eps=1e-6, scale=1.0):
    a = kda.kda_gated_norm_args(x, gate, res, w, nw, out, nxt, M, G, D, *xs, *gs, *rs, io, act, eps,
                                scale)
    return kda.load_library().kda_gated_norm_check(ctypes.byref(a))


def test_gated_norm_refusals():
    assert norm() == 0 and norm(out=at(0)) == 0 and norm(out=at(1)) == 0 and norm(out=at(2)) == 0
    assert norm(M=0, x=None, out=None) == 0 and norm(nw=None, nxt=None) == 0
    for D in (0, 4, 100, 16392):
        assert norm(D=D) == 2, D
    assert norm(M=-1) == 2 and norm(G=0) == 2 and norm(M=1 << 31) == 2
    assert norm(io=2) == 3 and norm(act=2) == 4
    assert norm(eps=-1.0) == 5 and norm(eps=float("nan")) == 5 and norm(scale=float("inf")) == 5
    assert norm(x=None) == 1 and norm(out=None) == 1 and norm(nxt=None) == 1
    assert norm(gate=at(1) + 8) == 2 and norm(w=at(3) + 4) == 2
    assert norm(gs=(256, -8)) == 2 and norm(xs=(260, 128)) == 2
    assert norm(out=at(0), xs=(512, 128)) == 6       # in place needs a contiguous x
    assert norm(out=at(0) + 256) == 6 and norm(nxt=at(1)) == 6 and norm(nxt=at(5)) == 6
    assert norm(out=at(3)) == 6 and norm(nxt=at(4)) == 6


# ---------------------------------------------------------------- the Python binding


def expect(code, text, fn, *a, **kw):
    with pytest.raises(kda.KdaError) as e:
        fn(*a, **kw)
    assert e.value.status == code and text in str(e.value), str(e.value)


def test_linear_binding():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    q, k, v = z(2, 20, 2, 64), z(2, 20, 2, 64), z(2, 20, 4, 128)
    go = lambda code, text, q=q, k=k, v=v, g=None, st=None, cu=None, **kw: expect(
        code, text, kda.kda_linear, q, k, v, g, st, cu, **kw)
    go(2, "CUDA tensor")
    go(2, "four axes", q=z(20, 2, 64))
    go(2, "must be a tensor", k=None)
    go(2, "k has shape", k=z(2, 20, 1, 64))
    go(2, "v has shape", v=z(2, 19, 4, 128))
    go(3, "unsupported dtype", q=q.half(), k=k.half(), v=v.half())
    go(3, "q, k, v are", k=k.float())
    go(2, "do not divide", v=z(2, 20, 3, 128))
    go(2, "contiguous", q=z(2, 20, 64, 2).transpose(2, 3))
    go(3, "cu_seqlens", cu=torch.zeros(3, dtype=torch.int32))
    go(2, "B = 1", cu=torch.zeros(3, dtype=torch.int64))
    go(2, "N + 1", cu=torch.zeros(1, dtype=torch.int64))
    go(2, "g has shape", g=z(2, 20, 2))
    go(3, "unsupported dtype", g=z(2, 20, 4, dt=torch.float64))
    go(3, "g is", g=z(2, 20, 4), q=q.float(), k=k.float(), v=v.float())
    go(2, "log_decay", log_decay=z(2, dt=torch.float32))
    go(3, "log_decay", log_decay=z(4))
    go(2, "state_in has shape", st=z(2, 4, 64, 128))
    go(2, "state_in must be contiguous", st=z(2, 4, 64, 128).transpose(2, 3))
    go(3, "the state dtype", st=z(2, 4, 128, 64), state_dtype=torch.float32)
    go(3, "state dtype", state_dtype=torch.float16)
    go(2, "state_out has shape", state_out=z(1, 4, 128, 64))
    go(2, "o must be", o=z(2, 20, 4, 128, dt=torch.float32))
    ids = torch.zeros(2, dtype=torch.int32)
    go(10, "needs state_in", ssm_state_indices=ids)
    go(10, "needs ssm_state_indices", state_out_indices=ids)
    pool = z(5, 4, 128, 64)
    go(2, "CUDA tensor", st=pool, ssm_state_indices=ids, state_out_indices=ids)
    go(2, "contiguous", st=pool.transpose(2, 3).contiguous().transpose(2, 3), ssm_state_indices=ids)
    go(3, "ssm_state_indices", st=pool, ssm_state_indices=ids.long())
    go(2, "state_out_indices", st=pool, ssm_state_indices=ids, state_out_indices=ids[:1])
    go(6, "with a state pool", st=pool, ssm_state_indices=ids, state_out=pool.clone())


def test_pool_binding():
    pool = torch.zeros(5, 2, 64, 64)
    i = torch.zeros(3, dtype=torch.int32)
    go = lambda code, text, pool=pool, src=i, dst=i, **kw: expect(
        code, text, kda.kda_pool_copy, pool, src, dst, **kw)
    go(2, "CUDA tensor")
    go(3, "unsupported dtype", pool=pool.half())
    go(2, "must be [", pool=torch.zeros(5))
    go(2, "must be contiguous", pool=pool.transpose(2, 3)[:, :, :32])
    go(2, "empty", pool=torch.zeros(0, 64))
    go(2, "differ", source=torch.zeros(5, 2, 64, 32))
    go(2, "differ", pool=pool[None], source=torch.zeros(2, 5, 2, 64, 64), layered=True)
    go(3, "src", src=i.long())
    go(2, "ids, dst", dst=i[:2])
    go(2, "dst must be", dst=torch.zeros(6, dtype=torch.int32)[::2])
    go = lambda code, text, pool=pool, slots=i, **kw: expect(
        code, text, kda.kda_pool_compact, pool, slots, **kw)
    go(2, "CUDA tensor")
    go(3, "slots", slots=i.float())
    go(2, "entries", new_slots=i[:2])
    go(2, "one entry", count=i)


def test_norm_binding():
    x = torch.zeros(3, 4, 128)
    go = lambda code, text, x=x, *a, **kw: expect(code, text, kda.kda_gated_norm, x, *a, **kw)
    go(2, "CUDA tensor")
    go(3, "unsupported", x.double())
    go(4, "gate_act", gate_act="relu")
    go(2, "gate has shape", x, x[:, :3])
    go(3, "gate is", x, x.bfloat16())
    go(2, "weight", x, None, torch.zeros(64))
    go(3, "weight", x, None, torch.zeros(128).bfloat16())
    go(2, "out must be", out=torch.zeros(3, 128, 4).transpose(1, 2))
    go(2, "last axis", x, torch.zeros(3, 4, 256)[..., ::2])
    go(2, "cannot be seen as one", torch.zeros(3, 2, 4, 128),
       torch.zeros(3, 5, 4, 128)[:, :2])


def test_linear_pool_slots_must_not_overlap():
    """A pool whose slots lie on one another (one state expanded) or within one another."""
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, v = z(2, 20, 2, 64), z(2, 20, 4, 128)
    ids = torch.zeros(2, dtype=torch.int32)
    go = lambda code, text, pool: expect(code, text, kda.kda_linear, q, q, v, None, pool,
                                         ssm_state_indices=ids)
    one = z(1, 4, 128, 64)
    go(10, "slot pitch", one.expand(5, 4, 128, 64))
    go(10, "slot pitch", z(9, 4, 128, 64).as_strided((5, 4, 128, 64), (128 * 64, 128 * 64, 64, 1)))
    # one slot: its stride says nothing
    go(2, "CUDA tensor", one.expand(1, 4, 128, 64))
    go(2, "CUDA tensor", one.as_strided((1, 4, 128, 64), (0, 128 * 64, 64, 1)))
    go(2, "CUDA tensor", z(5, 5, 128, 64)[:, :4])  # padded


def test_linear_plan_of_128_row_workgroups():
    """The segments' state launch has 64 value rows per workgroup whatever the outputs have."""
    for kw in (dict(H=200, T=256, segment_tokens=64), dict(H=200, T=1000, V=256, segment_tokens=128),
               dict(H=40, T=8192)):
        p = kda.kda_linear_plan(lin(**kw))
        assert p["value_block"] == 128 and p["segment_tokens"] > 0, (kw, p)
        heads = kw["H"] * p["segments_bound"]
        assert p["workgroups"] == heads * kw.get("V", 128) // 128
        assert p["state_workgroups"] == heads * kw.get("V", 128) // 64
    p = kda.kda_linear_plan(lin(H=6, T=8192))
    assert p["value_block"] == 64 and p["state_workgroups"] == p["workgroups"] > 0
    p = kda.kda_linear_plan(lin(H=200, T=256, segment_tokens=-1))
    assert p["value_block"] == 128 and p["state_workgroups"] == 0


def test_segments_past_one_state_launch_are_refused():
    """128-row workgroups for the outputs, twice as many of 64 rows for the segments' states:
    the larger launch has to stay below 2^32 threads, 2^22 (segment, head) pairs of V = 128."""
    far = dict(H=256, V=128, g=None, log_decay=None, state_in=None, state_out=None, q=at(0), k=at(500),
               v=at(1000), o=at(1500), workspace=at(2000), workspace_bytes=1 << 40, segment_tokens=64)
    most = (1 << 14) - 1  # segments of 256 heads, with the launch's rounding up
    p = kda.kda_linear_plan(lin(T=64 * most, **far))
    assert p["value_block"] == 128 and p["segment_tokens"] == 64
    assert p["state_workgroups"] * 512 < 1 << 32
    assert status(T=64 * most, **far) == 0, kda.kda_last_error()
    for T in (64 * (most + 1), 64 * 20000, 64 * 32000):
        assert status(T=T, **far) == 2, T
        assert "one launch" in kda.kda_last_error()


def test_arguments_that_are_no_tensors_are_refused():
    """With a KdaError, as every other argument that is not what it should be."""
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, v, pool = z(2, 20, 2, 64), z(2, 20, 4, 128), z(5, 4, 128, 64)
    ids = torch.zeros(2, dtype=torch.int32)
    for bad in (3, [1.0], "state"):
        for kw in (dict(state_in=bad), dict(state_in=bad, ssm_state_indices=ids),
                   dict(state_out=bad), dict(state_in=pool, ssm_state_indices=ids, state_out=bad),
                   dict(workspace=bad), dict(g=bad), dict(log_decay=bad), dict(cu_seqlens=bad),
                   dict(o=bad), dict(state_in=pool, ssm_state_indices=bad),
                   dict(state_in=pool, ssm_state_indices=ids, state_out_indices=bad)):
            expect(2, "must be a tensor", kda.kda_linear, q, q, v, **kw)
        for kw in (dict(pool=bad), dict(slots=bad), dict(new_slots=bad), dict(count=bad),
                   dict(workspace=bad)):
            expect(2, "must be a tensor", kda.kda_pool_compact,
                   **{**dict(pool=torch.zeros(5, 64), slots=ids), **kw})
        for kw in (dict(pool=bad), dict(src=bad), dict(dst=bad), dict(source=bad)):
            expect(2, "must be a tensor", kda.kda_pool_copy,
                   **{**dict(pool=torch.zeros(5, 64), src=ids, dst=ids), **kw})
        for name in ("x", "gate", "weight", "residual", "next_weight", "out", "next_out"):
            expect(2, "must be a tensor", kda.kda_gated_norm, **{"x": torch.zeros(2, 64), name: bad})
