"""The gated norm against its formula in FP64.

Tolerance: the result's own rounding (u = 2^-8 for BF16, 2^-24 for FP32, of |y|), and FP32
arithmetic: a thread adds at most 64 squares and 10 levels join the threads, so the mean
square is off by 74 2^-24 and its root by half of that; sigmoid (exp of e: |e| + 2, sum, reciprocal:
4) and the products add 16 + 2 |e|: 2^-24 (56 + 2 |e|) of the gated part, and one more for
the sum with the residual. z adds the same again for its own norm, plus what the relative
error of y moves in it.
"""

import numpy as np
import pytest

from oracle import gated_norm_fp64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    kda.load_library()


def host(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def check(x, gate=None, weight=None, residual=None, next_weight=None, act="sigmoid", scale=1.0,
          eps=1e-6, name="", **kw):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else E
    ref = lambda **z: gated_norm_fp64(host(x), host(gate), host(weight),
                                      z.pop("residual", host(residual)), eps=float(np.float32(eps)),
                                      act=act, scale=float(np.float32(scale)), **z)
    part, y_ref = ref(residual=None), ref()
    e = np.abs(host(gate)) if gate is not None else 0.0
    err = E * (56 + 2 * e) * np.abs(part) + E * np.abs(y_ref)
    both = next_weight is not None or kw.get("next_out") is not None
    z_ref = ref(next_weight=host(next_weight), next_norm=True)[1] if both else None
    got = kda.kda_gated_norm(x, gate, weight, residual, next_weight=next_weight, eps=eps,
                             gate_act=act, scale=scale, **kw)
    torch.cuda.synchronize()
    y, z = got if both else (got, None)
    slack = err + u * np.abs(y_ref)
    bad = np.abs(host(y) - y_ref) - slack
    print(f"[case] norm {name}: y {np.max(np.abs(host(y) - y_ref) / np.maximum(slack, 1e-300)):.3f}"
          " of its bound", flush=True)
    assert np.all(np.isfinite(host(y))) and np.max(bad) <= 0, name
    if both:
        w = 1.0 if next_weight is None else np.abs(host(next_weight))
        r = 1 / np.sqrt(np.mean(y_ref ** 2, -1, keepdims=True) + eps)
        moved = np.sqrt(np.mean(err ** 2, -1, keepdims=True)) * r  # of the row's norm
        slack = w * r * err + np.abs(z_ref) * (moved + E * 56 + u)
        assert np.max(np.abs(host(z) - z_ref) - slack) <= 0, name + " z"
    return y, z


def rand(*shape, dt, seed=0):
    import torch

    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(
        {"bf16": torch.bfloat16, "fp32": torch.float32}[dt])


# every launch shape and its borders: one row to many, D from 8 to 16384
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("M,D", [(1, 8), (33, 8), (5, 64), (65, 72), (17, 128), (100, 136),
                                 (9, 256), (9, 264), (3, 512), (3, 520), (7, 2048), (2, 2056),
                                 (3, 4096), (2, 4104), (2, 6144), (2, 6152), (2, 8192), (2, 8200),
                                 (2, 12288), (2, 12296), (3, 16384)])
def test_sizes(dt, M, D):
    x, gate, res = (rand(M, D, dt=dt, seed=s) for s in (1, 2, 3))
    w, nw = 1 + 0.1 * rand(D, dt="fp32", seed=4), 1 + 0.1 * rand(D, dt="fp32", seed=5)
    check(x, name=f"plain {M}x{D}")
    check(x, gate, w, res, nw, "silu", 0.5, name=f"full {M}x{D}")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [128, 1024])
def test_each_part(dt, D):
    import torch

    x, gate, res = (rand(2, 5, 3, D, dt=dt, seed=s) for s in (1, 2, 3))
    w = 1 + 0.1 * rand(D, dt="fp32", seed=4)
    for use in range(8):
        check(x, gate if use & 1 else None, w if use & 2 else None, res if use & 4 else None,
              name=f"parts {use}", scale=-1.25)
    check(x, gate, w, res, w, name="next")
    check(x, next_out=torch.empty_like(x), name="next without weight")


@pytest.mark.parametrize("D", [64, 128, 2048])
def test_slices_of_a_projection(D):
    x = rand(3, 4, 2, D, dt="bf16", seed=1)
    proj = rand(3, 4, 5, 2, D + 8, dt="bf16", seed=2)
    gate, res = proj[:, :, 3, :, :D], proj[:, :, 1, :, :D]
    check(x, gate, None, res, act="silu", name="slices")
    check(proj[:, :, 0, :, :D], gate, name="sliced x")
    check(x, x[:, :, :1].expand(3, 4, 2, D), name="one gate for all heads")


def test_in_place():
    import torch

    for D in (128, 1536):
        x, gate, res = (rand(7, D, dt="fp32", seed=s) for s in (1, 2, 3))
        want, _ = check(x, gate, None, res)
        for which in range(3):
            t = [x.clone(), gate.clone(), res.clone()]
            import chunkwise_delta_rule_kda_amd as kda

            kda.kda_gated_norm(t[0], t[1], None, t[2], out=t[which])
            assert torch.equal(t[which], want), which
            for i in range(3):
                assert i == which or torch.equal(t[i], (x, gate, res)[i])


def test_zero_rows_large_values_and_gates():
    import torch

    x = rand(6, 256, dt="fp32", seed=1)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    gate = rand(6, 256, dt="fp32", seed=2)
    gate[3] = 80.0
    gate[4] = -80.0
    check(x, gate, name="extremes")
    check(x, name="zero rows stay zero")
    import chunkwise_delta_rule_kda_amd as kda

    x[5, 7] = float("nan")
    y = kda.kda_gated_norm(x, gate)
    assert bool(y[5].isnan().all()) and bool(y[:5].isfinite().all())
    gate[0, 3], gate[0, 4] = float("inf"), -float("inf")
    y = kda.kda_gated_norm(rand(6, 256, dt="fp32", seed=3), gate)
    assert y[0, 4] == 0 and bool(y[0].isfinite().all())


def test_eps_zero_and_empty():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    check(rand(3, 64, dt="fp32"), eps=0.0, name="eps 0")
    assert kda.kda_gated_norm(torch.empty(0, 4, 64, device="cuda")).shape == (0, 4, 64)


def test_one_row_of_one_axis():
    check(rand(128, dt="bf16"), name="1-D")


def test_graph_and_stream():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    x, gate = rand(64, 24, 128, dt="bf16", seed=1), rand(64, 24, 128, dt="bf16", seed=2)
    want = kda.kda_gated_norm(x, gate)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_gated_norm(x, gate, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gated_norm(x, gate, out=out)
    for _ in range(3):
        out.zero_()
        torch.randn(1 << 18, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["sequence first", "heads and tokens exchanged"])
def test_single_tokens_in_other_axis_orders(dt, layout):
    """[B, 1, G, D] tensors that are contiguous although the strides of their token axis are
    not those of a dense tensor, as x, gate and residual, alone and together."""
    def make(seed):
        if layout == "sequence first":
            return rand(1, 5, 4, 128, dt=dt, seed=seed).transpose(0, 1)
        return rand(5, 4, 1, 128, dt=dt, seed=seed).transpose(1, 2)

    x, gate, res = make(1), make(2), make(3)
    assert x.shape == (5, 1, 4, 128) and x.is_contiguous()
    dense = [t.clone().as_strided(t.shape, (512, 512, 128, 1)) for t in (x, gate, res)]
    w = 1 + 0.1 * rand(128, dt="fp32", seed=4)
    for use in range(1, 8):
        t = [(a if use >> i & 1 else b) for i, (a, b) in enumerate(zip((x, gate, res), dense))]
        check(t[0], t[1], w, t[2], name=f"{layout} {use}")


def test_one_token_of_the_linear_attention():
    """o of kda_linear for single tokens in a sequence-first layout, normed and gated."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    q, k, v = (rand(1, 5, 4, 128, dt="bf16", seed=s).transpose(0, 1) for s in (1, 2, 3))
    o, _ = kda.kda_linear(q, k, v)
    assert o.shape == (5, 1, 4, 128)
    check(o, rand(5, 1, 4, 128, dt="bf16", seed=4), name="o of kda_linear")
