"""The operators in a run as a server makes it: two layers (KDA and linear attention with one
decay per head) whose states live in pools; a prompt, a fork into three continuations that
share it, tokens for each, the gated norm on the outputs, an ended continuation, and the
pools compacted before further tokens. Every step against the FP64 oracles on the whole
token sequences of each continuation; the bound on the BF16 run is the library's 2e-2 of
the largest entry (KDA) and, for the linear layer in FP32, 1e-4."""

import numpy as np
import pytest

from oracle import gated_norm_fp64, kda_recurrence_fp64, linear_recurrence_fp64
from kda_testlib import rel_err

pytestmark = pytest.mark.gpu


def test_prompt_fork_tokens_compact():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    dev, H, D = "cuda", 2, 128
    gen = torch.Generator(device=dev)
    gen.manual_seed(3)
    host = lambda t: t.detach().float().cpu().numpy().astype(np.float64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)

    def tokens(B, T):
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        r = lambda *s: torch.randn(*s, generator=gen, device=dev)
        bf = torch.bfloat16
        kx = dict(q=unit(r(B, T, H, D)).to(bf), k=unit(r(B, T, H, D)).to(bf),
                  v=r(B, T, H, D).to(bf), g=(-5 * torch.sigmoid(r(B, T, H, D))).to(bf),
                  beta=torch.sigmoid(r(B, T, H)).to(bf))
        lx = dict(q=unit(r(B, T, 1, D)), k=unit(r(B, T, 1, D)), v=r(B, T, H, D),
                  g=-0.2 * torch.rand(B, T, H, generator=gen, device=dev))
        return kx, lx

    kpool = torch.zeros(10, H, D, D, dtype=torch.bfloat16, device=dev)
    lpool = torch.zeros(10, H, D, D, device=dev)
    slots = i32([9])
    kx, lx = tokens(1, 70)
    seen = [[(kx, lx, 0)]]  # the tokens of each sequence: (inputs, row)
    step_k = lambda x, i: kda.kda_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], kpool,
                                          ssm_state_indices=i)[0]
    step_l = lambda x, i, **kw: kda.kda_linear(x["q"], x["k"], x["v"], x["g"], lpool,
                                               ssm_state_indices=i, **kw)[0]
    outs = [(step_k(kx, slots), step_l(lx, slots))]
    # three continuations of the prompt: the KDA states are copied, the linear layer's
    # first tokens read the shared state and write their own slots
    slots = i32([3, 7, 6])
    kda.kda_pool_copy(kpool, i32([9, 9, 9]), slots)
    kx, lx = tokens(3, 1)
    seen = [seen[0] + [(kx, lx, b)] for b in range(3)]
    outs = [(step_k(kx, slots), step_l(lx, i32([9, 9, 9]), state_out_indices=slots))]
    kx, lx = tokens(3, 4)  # draft tokens
    seen = [s + [(kx, lx, b)] for b, s in enumerate(seen)]
    outs.append((step_k(kx, slots), step_l(lx, slots)))
    # the second one ends; the others move to the pools' front
    seen = [seen[0], seen[2]]
    last = [o[[0, 2]] for o in outs[-1]]
    slots = slots[[0, 2]].contiguous()
    new, count = kda.kda_pool_compact(kpool, slots)
    new2, _ = kda.kda_pool_compact(lpool, slots)
    assert count.item() == 2 and torch.equal(new, new2) and sorted(new.tolist()) == [0, 1]
    kx, lx = tokens(2, 1)
    seen = [s + [(kx, lx, b)] for b, s in enumerate(seen)]
    final = (step_k(kx, new), step_l(lx, new))
    gate, w = torch.randn(2, 1, H, D, device=dev), 1 + 0.1 * torch.randn(D, device=dev)
    normed = kda.kda_gated_norm(final[1], gate, w)
    torch.cuda.synchronize()

    for b, steps in enumerate(seen):
        cat = lambda which, n: np.concatenate([host(s[which][n][s[2]:s[2] + 1]) for s in steps], 1)
        ko, ks = kda_recurrence_fp64(*(cat(0, n) for n in ("q", "k", "v", "g", "beta")))
        lo, ls, _, _ = linear_recurrence_fp64(*(cat(1, n) for n in "qkvg"))
        slot = new[b].item()
        assert rel_err(host(final[0][b:b + 1]), ko[:, -1:]) <= 2e-2
        assert rel_err(host(last[0][b:b + 1]), ko[:, -5:-1]) <= 2e-2
        assert rel_err(host(kpool[slot]), ks[0]) <= 2e-2
        assert rel_err(host(final[1][b:b + 1]), lo[:, -1:]) <= 1e-4
        assert rel_err(host(last[1][b:b + 1]), lo[:, -5:-1]) <= 1e-4
        assert rel_err(host(lpool[slot]), ls[0]) <= 1e-4
        want = gated_norm_fp64(lo[:, -1:], host(gate[b:b + 1]), host(w))
        assert rel_err(host(normed[b:b + 1]), want) <= 1e-4
