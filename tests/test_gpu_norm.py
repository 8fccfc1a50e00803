"""GPU parity of the norms around a block and their gradients against the float64 oracle.

Bounds.  A row's sum of squares adds at most 32 values per thread and 10 levels of a tree: relative error
below 2^-18, of which rstd sees half, and a handful of roundings follow: 2^-17 of the magnitudes
for float32 results.  The backward pass adds three such sums and combines them: 2^-15 of the
magnitudes of all terms.  Sums over rows add at most 2^-24 per row in a CTA's sequence, 2^-15 for
every count here.  bf16 results are off by half a step more."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gsa_b200 as nv
from oracle import operators as P
from tests._gpu_util import DEV

pytestmark = pytest.mark.gpu
FWD, BWD = 2.0 ** -17, 2.0 ** -15
HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: 2.0 ** -24}
EPS = 1e-5


def make(T, H, res, gate, post, pre, seed, y=True):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16, mean=0.0):
        return (torch.randn(*shape, generator=g) + mean).to(dtype).to(DEV)

    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return dict(r=rand(T, H, dtype=res) * 4, y=rand(T, H) if y else None,
                post_gamma=rand(H, mean=1.0) if post else None,
                gate=None if shape is None else rand(*shape),
                pre_gamma=rand(H, mean=1.0) if pre else None)


def to64(v):
    return None if v is None else v.double().cpu().numpy()


def oracle_args(a, scale, eps):
    gate = a["gate"]
    return dict(r=to64(a["r"]), y=to64(a["y"]), post_gamma=to64(a["post_gamma"]),
                gate=1.0 if gate is None else to64(gate), pre_gamma=to64(a["pre_gamma"]), scale=scale,
                eps=eps)


def close(got, ref, tol):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = tol + HALF[got.dtype] * np.abs(ref) * (1 + BWD) + 1e-38
    assert (err <= tol).all(), float((err / tol).max())


def check_forward(a, out, scale, eps):
    rn, n, rs_y, rs_r, add = P.residual_norm(**oracle_args(a, scale, eps))
    got_r, got_n, got_y, got_s = out
    dr = FWD * np.abs(add)
    close(got_r, rn, dr)
    if a["post_gamma"] is not None:
        close(got_y, rs_y[:, 0], FWD * rs_y[:, 0])
    if a["pre_gamma"] is None:
        assert got_n is None and got_s is None
        return
    # r' moves n directly and through its norm: |drstd| <= rstd^2 * rms(dr')
    w = np.abs(to64(a["pre_gamma"]))
    rms = np.sqrt((dr ** 2).mean(1, keepdims=True))
    close(got_s, rs_r[:, 0], (FWD * rs_r + rs_r ** 2 * rms)[:, 0])
    close(got_n, n, FWD * np.abs(n) + rs_r * w * (dr + np.abs(rn) * rs_r * rms))


SHAPES = [(1, 8), (1, 7168), (2, 64), (3, 72), (5, 264), (4, 1000), (7, 2048), (3, 8200), (2, 16384),
          (33, 520)]


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, res, gate):
    a = make(T, H, res, gate, True, True, T + H)
    check_forward(a, nv.residual_norm(**a, scale=0.7, eps=EPS), 0.7, EPS)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_forward_of_many_rows(res):
    a = make(1203, 264, res, "token", True, True, 3)
    check_forward(a, nv.residual_norm(**a, eps=EPS), 1.0, EPS)


@pytest.mark.parametrize("post,pre,gate", [(False, True, "channel"), (True, False, "none"),
                                           (False, False, "token")])
def test_forward_without_some_of_the_norms(post, pre, gate):
    a = make(6, 136, torch.bfloat16, gate, post, pre, 1)
    check_forward(a, nv.residual_norm(**a, scale=-1.5, eps=0.0), -1.5, 0.0)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_plain_pre_norm(res):
    a = make(5, 256, res, "none", False, True, 2, y=False)
    out = nv.residual_norm(a["r"], None, pre_gamma=a["pre_gamma"], eps=EPS)
    assert out[0] is a["r"] and out[2] is None
    check_forward(a, out, 1.0, EPS)


def test_in_place_strided_rows_and_given_outputs():
    a = make(9, 512, torch.float32, "full", True, True, 4)
    want = nv.residual_norm(**a, eps=EPS)
    wide_r = torch.zeros(9, 1024, device=DEV)
    wide_y = torch.zeros(18, 512, dtype=torch.bfloat16, device=DEV)
    wide_r[:, 512:] = a["r"]
    wide_y[::2] = a["y"]
    got = nv.residual_norm(wide_r[:, 512:], wide_y[::2], a["post_gamma"], a["gate"], 1.0,
                           a["pre_gamma"], EPS)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert (wide_r[:, :512] == 0).all() and (wide_y[1::2] == 0).all()
    buf = torch.full((10, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    r = a["r"].clone()
    got = nv.residual_norm(r, a["y"], a["post_gamma"], a["gate"], 1.0, a["pre_gamma"], EPS, out_r=r,
                           out_n=buf[:9])
    assert torch.equal(r, want[0]) and torch.equal(buf[:9], want[1]) and (buf[9] == 3).all()
    with pytest.raises(nv.Nvfp4Error):
        nv.residual_norm(wide_r[:, 2:514], a["y"])  # rows not 16-byte aligned


def test_zero_rows_empty_batch_and_non_finite_rows():
    a = make(4, 64, torch.bfloat16, "none", True, True, 5)
    a["y"][1] = 0
    a["r"][1] = 0
    a["y"][2, 3] = float("inf")
    a["r"][3, 5] = float("nan")
    rn, n, rs_y, rs_r = nv.residual_norm(**a, eps=EPS)
    assert (rn[1] == 0).all() and (n[1] == 0).all()
    assert rs_r[1].item() == pytest.approx(EPS ** -0.5, rel=1e-6)
    assert torch.isnan(n[3]).all() and not torch.isfinite(rn[2]).all()
    keep = [0, 1]
    sub = {k: v[keep] if k in ("r", "y") else v for k, v in a.items()}
    check_forward(sub, (rn[keep], n[keep], rs_y[keep], rs_r[keep]), 1.0, EPS)
    none = nv.residual_norm(a["r"][:0], a["y"][:0], a["post_gamma"], pre_gamma=a["pre_gamma"])
    assert none[0].shape == (0, 64) and none[1].shape == (0, 64)
    z = nv.residual_norm_backward(a["r"][:0], a["y"][:0], a["r"][:0], a["y"][:0], none[2], none[3],
                                  a["post_gamma"], pre_gamma=a["pre_gamma"])
    assert (z["dpost_gamma"] == 0).all() and (z["dpre_gamma"] == 0).all()


# ------------------------------------------------------------------------------- backward

def check_backward(a, got, dr_new, dn, scale, eps):
    o = P.residual_norm_grad(to64(dr_new), to64(dn), **oracle_args(a, scale, eps))
    close(got["dr"], o["dr"][0], BWD * o["dr"][1])
    if a["y"] is None:
        assert got["dy"] is None
    else:
        close(got["dy"], o["dy"][0], BWD * o["dy"][1])
    for name in ("dpost_gamma", "dpre_gamma"):
        if got[name] is not None and name in o:
            close(got[name], o[name][0], BWD * o[name][1])
    if a["gate"] is not None:
        val, mag = o["dgate"]
        shape = a["gate"].shape
        if got["dgate"].dtype == torch.float32:
            axis = 0 if len(shape) == 1 else 1
            val, mag = val.sum(axis), mag.sum(axis)
        assert got["dgate"].shape == shape
        close(got["dgate"].reshape(val.shape), val, BWD * mag)


def run_backward(a, scale, eps, seed, with_r=True, with_n=True):
    T, H = a["r"].shape
    g = torch.Generator().manual_seed(seed)
    dr_new = torch.randn(T, H, generator=g).to(a["r"].dtype).to(DEV) if with_r else None
    dn = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV) if with_n else None
    _, _, rs_y, rs_r = nv.residual_norm(**a, scale=scale, eps=eps)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = nv.residual_norm_backward(dr_new, dn, a["r"], a["y"], rs_y, rs_r, a["post_gamma"],
                                    a["gate"], scale, a["pre_gamma"], status=status)
    assert nv.read_status(status) == (0, 0)
    return got, dr_new, dn


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES + [(300, 136), (1300, 64), (450, 1032)])
def test_backward(T, H, res, gate):
    a = make(T, H, res, gate, True, True, T + H + 1)
    got, dr_new, dn = run_backward(a, 0.7, EPS, T)
    check_backward(a, got, dr_new, dn, 0.7, EPS)


@pytest.mark.parametrize("post,pre,gate,y,with_r,with_n", [
    (True, True, "channel", True, False, True), (True, True, "full", True, True, False),
    (False, True, "channel", True, True, True), (True, False, "token", True, True, False),
    (False, False, "none", True, True, False), (False, True, "none", False, True, True),
    (False, True, "none", False, False, True),
])
def test_backward_without_some_of_it(post, pre, gate, y, with_r, with_n):
    a = make(40, 200, torch.bfloat16, gate, post, pre, 9, y=y)
    got, dr_new, dn = run_backward(a, 1.3, EPS, 10, with_r, with_n)
    check_backward(a, got, dr_new, dn, 1.3, EPS)
    if pre and not with_n:
        assert (got["dpre_gamma"] == 0).all()


def test_backward_is_reproducible_on_a_stream_and_in_a_graph():
    a = make(700, 328, torch.float32, "channel", True, True, 11)
    want, dr_new, dn = run_backward(a, 1.0, EPS, 12)
    _, _, rs_y, rs_r = nv.residual_norm(**a, eps=EPS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fwd = nv.residual_norm(**a, eps=EPS)
            got = nv.residual_norm_backward(dr_new, dn, a["r"], a["y"], fwd[2], fwd[3],
                                            a["post_gamma"], a["gate"], 1.0, a["pre_gamma"])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    a["y"].copy_(a["y"].flip(0))
    g.replay()
    torch.cuda.synchronize()
    check_backward(a, got, dr_new, dn, 1.0, EPS)


def test_gradients_against_differences():
    """The kernel's gradients along a random direction against the difference quotient of the
    float64 forward."""
    T, H = 6, 96
    a = make(T, H, torch.float32, "channel", True, True, 13)
    got, dr_new, dn = run_backward(a, 0.9, EPS, 14)
    v = oracle_args(a, 0.9, EPS)
    weights = to64(dr_new), to64(dn)

    def value(v):
        rn, n = P.residual_norm(**v)[:2]
        return float((weights[0] * rn).sum() + (weights[1] * n).sum())

    rng = np.random.default_rng(15)
    o = P.residual_norm_grad(*weights, **v)
    for name, key in [("r", "dr"), ("y", "dy"), ("post_gamma", "dpost_gamma"),
                      ("pre_gamma", "dpre_gamma"), ("gate", "dgate")]:
        d = rng.normal(size=v[name].shape)
        up, dn_ = dict(v), dict(v)
        up[name], dn_[name] = v[name] + 1e-6 * d, v[name] - 1e-6 * d
        quotient = (value(up) - value(dn_)) / 2e-6
        val = got[key].double().cpu().numpy()
        mag = o[key][1].sum(0) if key == "dgate" else o[key][1]
        tol = (BWD + HALF[got[key].dtype]) * float((mag * np.abs(d)).sum()) + 1e-5
        assert abs(float((val * d).sum()) - quotient) <= tol, name


@pytest.mark.parametrize("T,H,res,gate", [
    (161, 8200, torch.float32, "full"),       # a row across two CTAs, several rows each, uneven halves
    (300, 8208, torch.bfloat16, "token"),
    (149, 16384, torch.float32, "full"),      # the widest
    (450, 16376, torch.bfloat16, "channel"),
    (460, 4104, torch.float32, "none"),       # one CTA per SM, the fetches shared among its warps
])
def test_backward_of_wide_rows(T, H, res, gate):
    a = make(T, H, res, gate, True, True, T + H)
    got, dr_new, dn = run_backward(a, 0.7, EPS, T)
    check_backward(a, got, dr_new, dn, 0.7, EPS)
    again, _, _ = run_backward(a, 0.7, EPS, T)
    for key, v in got.items():
        assert v is None or torch.equal(v, again[key])


@pytest.mark.parametrize("post,pre,gate,y,with_r,with_n", [
    (True, True, "channel", True, False, True), (True, False, "full", True, True, False),
    (False, True, "none", False, True, True),
])
def test_backward_of_wide_rows_without_some_of_it(post, pre, gate, y, with_r, with_n):
    a = make(155, 9000, torch.bfloat16, gate, post, pre, 19, y=y)
    got, dr_new, dn = run_backward(a, 1.3, EPS, 20, with_r, with_n)
    check_backward(a, got, dr_new, dn, 1.3, EPS)


@pytest.mark.parametrize("T,H,res,gate", [(601, 2056, torch.bfloat16, "channel"),
                                          (592, 7168, torch.float32, "full"),
                                          (593, 16384, torch.bfloat16, "none"),
                                          (700, 2048, torch.float32, "token")])
def test_forward_of_many_long_rows(T, H, res, gate):
    a = make(T, H, res, gate, True, True, T + H)
    check_forward(a, nv.residual_norm(**a, scale=0.3, eps=EPS), 0.3, EPS)


@pytest.mark.parametrize("T,H", [(1, 64), (5, 2056), (700, 520)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_outputs_in_the_place_of_the_same_rows(T, H, res):
    a = make(T, H, res, "full", True, True, T + H)
    want = nv.residual_norm(**a, eps=EPS)
    same = res == torch.bfloat16
    for place_r, place_n in [("r", "y"), ("r", "gate")] + ([("y", "r"), ("gate", "y")] if same else []):
        b = {k: v.clone() for k, v in a.items()}
        got = nv.residual_norm(**b, eps=EPS, out_r=b[place_r], out_n=b[place_n])
        assert got[0].data_ptr() == b[place_r].data_ptr()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_outputs_over_other_rows_are_refused():
    a = make(4, 64, torch.bfloat16, "none", True, True, 3)
    buf = torch.zeros(9, 64, dtype=torch.bfloat16, device=DEV)
    buf[:4] = a["r"]
    a["r"] = buf[:4]
    for kw in (dict(out_r=buf[1:5]), dict(out_n=buf[3:7]), dict(out_r=buf[4:8], out_n=buf[5:9])):
        with pytest.raises(nv.Nvfp4Error):
            nv.residual_norm(**a, **kw)
    wide = torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV)
    a["r"] = wide[:, :64]
    with pytest.raises(nv.Nvfp4Error):
        nv.residual_norm(**a, out_n=wide.view(8, 64)[:4])
    out = nv.residual_norm(**a, out_n=buf[:4], out_r=buf[4:8])  # apart
    assert out[1].data_ptr() == buf.data_ptr()


def test_backward_in_place_of_its_gradients():
    """The C call with dr over dr', dy over dn (bf16 residual) or y."""
    for res, over in ((torch.bfloat16, "dn"), (torch.float32, "y")):
        a = make(300, 520, res, "channel", True, True, 4)
        want, dr_new, dn = run_backward(a, 0.9, EPS, 5)
        _, _, rs_y, rs_r = nv.residual_norm(**a, scale=0.9, eps=EPS)
        T, H = a["r"].shape
        dr, dy = dr_new.clone(), {"dn": dn, "y": a["y"]}[over].clone()
        dn_, y_ = (dy, a["y"]) if over == "dn" else (dn, dy)
        grads = [torch.empty(H, device=DEV) for _ in range(3)]
        ws = torch.empty(int(nv.lib().nvfp4_residual_norm_backward_workspace_size(T, H)),
                         dtype=torch.uint8, device=DEV)
        p = torch.Tensor.data_ptr
        rc = nv.lib().nvfp4_residual_norm_backward(
            p(dr), p(dn_), p(a["r"]), 0 if res == torch.float32 else 1, H, p(y_), H, T, H,
            p(a["post_gamma"]), p(a["gate"]), 1, 0.9, p(a["pre_gamma"]), p(rs_y), p(rs_r), p(dr),
            p(dy), p(grads[0]), p(grads[1]), p(grads[2]), p(ws), ws.numel(), None,
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        for g, key in zip([dr, dy] + grads, ("dr", "dy", "dpost_gamma", "dpre_gamma", "dgate")):
            assert torch.equal(g, want[key]), key


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H,res", [
    (7001, 8, torch.bfloat16),       # one warp a row, more rows than CTAs: the stages go round
    (9001, 256, torch.float32),
    (5003, 520, torch.bfloat16),
    (4001, 1032, torch.float32),
    (2500, 2048, torch.bfloat16),
])
def test_backward_of_many_narrow_rows(T, H, res, gate):
    a = make(T, H, res, gate, True, True, T + H)
    got, dr_new, dn = run_backward(a, 0.7, EPS, T)
    check_backward(a, got, dr_new, dn, 0.7, EPS)
    again, _, _ = run_backward(a, 0.7, EPS, T)
    for key, v in got.items():
        assert v is None or torch.equal(v, again[key])


def test_outputs_between_the_rows_of_strided_inputs():
    a = make(3, 64, torch.bfloat16, "none", True, True, 6)
    want = nv.residual_norm(**a, eps=EPS)
    big = torch.zeros(3, 1024, dtype=torch.bfloat16, device=DEV)
    big[:, :64] = a["r"]
    a["r"] = big[:, :64]
    out_r, out_n = big[0, 128:320].view(3, 64), big[1, 512:704].view(3, 64)
    got = nv.residual_norm(**a, eps=EPS, out_r=out_r, out_n=out_n)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    with pytest.raises(nv.Nvfp4Error):
        nv.residual_norm(**a, eps=EPS, out_r=torch.empty_like(out_r),
                         out_n=big.view(-1)[1024 - 128:1024 + 64].view(3, 64))
