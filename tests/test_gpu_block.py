"""The operators together, as a block uses them: pre-norm, router with its balance loss, the
experts, the post-norm with gate and residual, the next pre-norm, an output head; and back through the
norms and the router's loss.  Each stage is checked against the float64 oracle on the values that
the stage before it produced."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gsa_b200 as nv
from oracle import operators as P
from oracle import routing as R
from tests import test_gpu_balance as B
from tests import test_gpu_norm as N
from tests import test_gpu_w4a16 as W
from tests._gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 13])
def test_block_forward_and_back(T):
    H, I, E, k, V = 256, 128, 8, 2, 300
    w1, w2, f1, f2 = W.make_experts(E, H, I, seed=21)
    head, headf = W.make_weight(V, H, seed=22)
    a = N.make(T, H, torch.float32, "token", True, True, 23)
    router = torch.randn(E, H, generator=torch.Generator().manual_seed(24)).to(DEV) * H ** -0.5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    # a stream that is not the tensors' own, one workspace for both FFN calls, then a replayed graph
    ws = torch.empty(nv.moe_ffn_w4a16_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device=DEV)

    def block():
        _, x, _, rs0 = nv.residual_norm(a["r"], None, pre_gamma=a["pre_gamma"], eps=N.EPS)
        logits = x.float() @ router.t()
        route = nv.permute(logits, k, status=status)
        loss, counts, tokens, dlogits = nv.balance_loss(logits, route["ids"], 0.01, want_grad=True,
                                                        status=status)
        y = nv.moe_ffn_w4a16(x, None, k, w1, w2, ids=route["ids"], weights=route["weights"], ws=ws,
                             status=status)
        direct = nv.moe_ffn_w4a16(x, logits, k, w1, w2, ws=ws, status=status)
        r2, n, rs1, rs2 = nv.residual_norm(a["r"], y, a["post_gamma"], a["gate"], 0.5,
                                           a["pre_gamma"], N.EPS)
        out = nv.linear_w4a16(n, head, out_dtype=torch.float32, status=status)
        back = nv.residual_norm_backward(r2, n, a["r"], y, rs1, rs2, a["post_gamma"], a["gate"], 0.5,
                                         a["pre_gamma"], status=status)
        first = nv.residual_norm_backward(back["dr"], x, a["r"], None, None, rs0,
                                          pre_gamma=a["pre_gamma"], status=status)
        return x, logits, route["ids"], loss, counts, tokens, dlogits, y, direct, r2, n, rs1, rs2, out, \
            back, first

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            v = block()
    g.replay()
    torch.cuda.synchronize()
    x, logits, ids, loss, counts, tokens, dlogits, y, direct, r2, n, rs1, rs2, out, back, first = v
    assert nv.read_status(status) == (0, 0)
    z = logits.cpu().numpy()
    ids_o, wts = R.route_topk(z, k)
    assert np.array_equal(ids.cpu().numpy(), ids_o)
    B.check(z, ids_o, 0.01, [0, T], None, 1.0, loss, counts, tokens, dlogits)
    W.check_ffn(y, x, ids_o, wts, f1, f2)
    assert torch.equal(y, direct)
    b = dict(a, y=y)
    N.check_forward(b, (r2, n, rs1, rs2), 0.5, N.EPS)
    W.check(out, *P.linear(n.double().cpu().numpy(), headf))
    N.check_backward(b, back, r2, n, 0.5, N.EPS)
    N.check_backward(dict(a, y=None, gate=None, post_gamma=None), first, back["dr"], x, 1.0, N.EPS)


def test_calls_on_two_streams_at_once():
    """Two streams, each with its own inputs and workspaces, many calls in flight: the results of
    either are those of the calls alone."""
    T, H, I, E, k = 6, 256, 128, 8, 2
    w1, w2, _, _ = W.make_experts(E, H, I, seed=31)
    head, _ = W.make_weight(20000, H, seed=32)
    runs = []
    for seed in (33, 34):
        a = N.make(T, H, torch.bfloat16, "channel", True, True, seed)
        lg = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).to(DEV)

        def step(a=a, lg=lg):
            x = nv.residual_norm(a["r"], a["y"], a["post_gamma"], a["gate"], 1.0, a["pre_gamma"])
            y = nv.moe_ffn_w4a16(x[1], lg, k, w1, w2)
            d = nv.residual_norm_backward(x[0], y, a["r"], a["y"], x[2], x[3], a["post_gamma"],
                                          a["gate"], 1.0, a["pre_gamma"])
            ids = nv.permute(lg, k)["ids"]
            return [y, nv.linear_w4a16(y, head), d["dy"], d["dpost_gamma"],
                    *nv.balance_loss(lg, ids, 0.1, want_grad=True)]
        runs.append((step, step(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (step, _, s) in enumerate(runs):
            with torch.cuda.stream(s):
                got[i].append(step())
    torch.cuda.synchronize()
    for i, (_, want, _) in enumerate(runs):
        for g in got[i]:
            for u, v in zip(g, want):
                assert torch.equal(u, v)
