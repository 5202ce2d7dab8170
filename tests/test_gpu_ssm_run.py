"""The short convolution, the selective scan, kda_prefill and the pools in a run as a server
makes it. Two layers: q, k and v through the convolution into KDA, and an input through the
convolution, a projection to step sizes, B and C, and the scan. Two prompts packed into one
call, one of them forked into three continuations, single and draft tokens for each, an ended
continuation, all pools compacted, further tokens. Every step against the FP64 oracles on the
whole token sequences of each continuation, from the inputs that the layer before gave: the
convolution and the scan within their oracles' bounds, KDA within the library's 2e-2 of the
largest entry."""

import numpy as np
import pytest

from kda_testlib import rel_err
from oracle import kda_recurrence_fp64, selective_scan_fp64, short_conv_fp64

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24


def test_prompts_fork_tokens_compact():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    dev, H, D, S, W = "cuda", 2, 72, 16, 4
    gen = torch.Generator(device=dev)
    gen.manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev)
    host = lambda t: t.detach().float().cpu().numpy().astype(np.float64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    qkv_w = 0.5 * r(3 * H * 128, W)
    in_w, in_b = 0.5 * r(D, W), 0.1 * r(D)
    proj = r(D, 8 + 2 * S) * D ** -0.5
    dt_w, dt_b = 0.3 * r(8, D), torch.log(torch.expm1(0.01 + 0.3 * torch.rand(D, device=dev)))
    A, skip = -torch.arange(1, S + 1, device=dev).float().repeat(D, 1), 1 + 0.1 * r(D)

    slots_n = 12
    pools = dict(qkv=torch.zeros(slots_n, W - 1, 3 * H * 128, dtype=torch.bfloat16, device=dev),
                 kda=torch.zeros(slots_n, H, 128, 128, dtype=torch.bfloat16, device=dev),
                 inp=torch.zeros(slots_n, W - 1, D, device=dev),
                 ssm=torch.zeros(slots_n, D, S, device=dev))

    def layers(B, T, read, write=None, cu=None):
        """One call of both layers on fresh tokens; what went in and came out, by name."""
        to = dict(ssm_state_indices=read, state_out_indices=write)
        x = r(B, T, 3 * H * 128).bfloat16()
        qkv, _ = kda.kda_short_conv(x, qkv_w, None, pools["qkv"], cu, **to)
        q, k, v = (t.contiguous() for t in qkv.unflatten(2, (3, H, 128)).unbind(2))
        g = (-5 * torch.sigmoid(r(B, T, H, 128))).bfloat16()
        beta = torch.sigmoid(r(B, T, H)).bfloat16()
        if write is not None:  # kda_prefill reads and writes one slot: copied first
            kda.kda_pool_copy(pools["kda"], read, write)
        o, _ = kda.kda_prefill(q, k, v, g, beta, pools["kda"], cu, l2norm_qk=True,
                               ssm_state_indices=read if write is None else write)
        xz = r(B, T, 2 * D)
        u, _ = kda.kda_short_conv(xz[..., :D], in_w, in_b, pools["inp"], cu, **to)
        p = u @ proj
        delta = p[..., :8] @ dt_w
        Bm, Cm = p[..., 8:8 + S], p[..., 8 + S:]
        y, _ = kda.kda_selective_scan(u, delta, A, Bm, Cm, skip, xz[..., D:], pools["ssm"], cu,
                                      delta_bias=dt_b, **to)
        return dict(x=x, qkv=qkv, q=q, k=k, v=v, g=g, beta=beta, o=o, xz=xz, u=u, delta=delta,
                    B=Bm, C=Cm, y=y)

    cut = lambda step, b, a=None, e=None: {n: t[b:b + 1] if a is None else t[b:b + 1, a:e]
                                           for n, t in step.items()}
    first = layers(1, 170, i32([9, 2]), cu=torch.tensor([0, 100, 170], device=dev))
    seen = [[cut(first, 0, 0, 100)], [cut(first, 0, 100, 170)]]
    # slot 9's continuations read it and write their own slots; the other one goes on in place
    step = layers(4, 1, i32([9, 9, 9, 2]), i32([3, 7, 6, 10]))
    seen = [seen[i] + [cut(step, b)] for b, i in enumerate((0, 0, 0, 1))]
    slots = i32([3, 7, 6, 10])
    step = layers(4, 4, slots)  # draft tokens
    seen = [s + [cut(step, b)] for b, s in enumerate(seen)]
    # the second one ends, the others move to the pools' front
    seen, slots = [seen[i] for i in (0, 2, 3)], slots[[0, 2, 3]].contiguous()
    moved = [kda.kda_pool_compact(p, slots) for p in pools.values()]
    assert all(torch.equal(m[0], moved[0][0]) and m[1].item() == 3 for m in moved)
    slots = moved[0][0]
    assert sorted(slots.tolist()) == [0, 1, 2]
    step = layers(3, 1, slots)
    seen = [s + [cut(step, b)] for b, s in enumerate(seen)]
    torch.cuda.synchronize()

    for b, steps in enumerate(seen):
        cat = lambda n: np.concatenate([host(s[n]) for s in steps], 1)
        slot = slots[b].item()
        qkv, state, err = short_conv_fp64(cat("x"), host(qkv_w))
        assert np.all(np.abs(cat("qkv") - qkv) <= U * np.abs(qkv) + E * err)
        assert np.array_equal(host(pools["qkv"][slot]), state[0])
        l2 = lambda t: t / np.sqrt((t * t).sum(-1, keepdims=True) + 1e-6)
        o, state = kda_recurrence_fp64(l2(cat("q")), l2(cat("k")), cat("v"), cat("g"), cat("beta"))
        assert rel_err(cat("o"), o) <= 2e-2 and rel_err(host(pools["kda"][slot]), state[0]) <= 2e-2
        xz = cat("xz")
        u, state, err = short_conv_fp64(xz[..., :D], host(in_w), host(in_b))
        assert np.all(np.abs(cat("u") - u) <= E * (np.abs(u) + err))
        assert np.array_equal(host(pools["inp"][slot]), state[0])
        y, state, y_err, s_err = selective_scan_fp64(
            cat("u"), cat("delta"), host(A), cat("B")[:, :, None], cat("C")[:, :, None],
            host(skip), xz[..., D:], delta_bias=host(dt_b))
        assert np.all(np.abs(cat("y") - y) <= E * (np.abs(y) + y_err))
        assert np.all(np.abs(host(pools["ssm"][slot]) - state[0]) <= E * (np.abs(state[0]) + s_err[0]))
