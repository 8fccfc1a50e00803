"""GPU parity of the products of NVFP4 weights with unquantized activations (linear_w4a16,
moe_ffn_w4a16) against the float64 oracle, element by element.

Bounds.  Decoded weights and (within 2^-29 of a row's maximum) activations are exact.  A float32
output is off by what the sums lose: at most 32 MMA accumulations in a row, each losing at most
2^-21 of the magnitudes (the tensor cores align addends to a little over 22 bits), one float32 add per
two steps of 256, the CTAs' sums and the division: (32 * 2^-21 + (K / 512 + 24) * 2^-24) * sum|x||w|,
below 2^-15 of it for every K here; a bf16 output by half a step more (2^-8)."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gsa_b200 as nv
from oracle import formats as F
from oracle import moe as M
from oracle import operators as P
from oracle import quant as Q
from oracle import routing as R
from tests._gpu_util import DEV, to_dev, upload_weights

pytestmark = pytest.mark.gpu
SUM = 2.0 ** -15
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def make_weight(N, K, seed, sd=0.02):
    """A quantized weight of any number of rows: (device weights, float64 values)."""
    rng = np.random.default_rng(seed)
    w = bf16(rng.normal(size=(N, K)) * sd).float().numpy()
    gs = Q.global_scale(w)
    codes, sf = Q.quantize(w, gs)
    return raw_weight(codes, sf, gs), Q.dequantize(codes, sf, gs)


def raw_weight(codes, sf, gs):
    N, K = codes.shape
    pad = np.full(((N + 127) // 128 * 128, K // 16), 0x7F, np.uint8)  # NaN scales behind the rows
    pad[:N] = sf
    return nv.NVFP4Weights(to_dev(F.pack_nibbles(codes)), to_dev(Q.tile_sf(pad)),
                           to_dev(np.array([gs], np.float32)), 1, N, K)


def check(got, ref, mag):
    half = BF16_HALF if got.dtype == torch.bfloat16 else 0.0
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    tol = SUM * mag + half * np.abs(ref) * (1 + SUM) + 1e-37
    assert np.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M_,N,K", [
    (1, 1, 64), (1, 129, 64), (2, 70, 192), (3, 300, 256), (4, 128, 7168), (5, 128, 7168),
    (7, 1000, 320), (8, 257, 704), (8, 96, 2048), (9, 200, 320), (16, 384, 4096), (17, 130, 1088),
    (32, 128, 2048), (33, 100, 512), (65, 640, 256), (1, 20000, 128), (6, 19000, 576),
])
def test_linear_matches_the_oracle(M_, N, K, out):
    w, wf = make_weight(N, K, seed=N + K)
    rng = np.random.default_rng(M_)
    x = bf16(rng.normal(size=(M_, K)) * np.exp(rng.normal(size=(M_, 1)) * 3))
    ref, mag = P.linear(x.double().numpy(), wf)
    check(nv.linear_w4a16(x.to(DEV), w, out_dtype=out), ref, mag)


def test_every_code_and_scale_is_decoded_exactly():
    # weight row n holds code n % 16 everywhere, its group c the scale byte 16 * (n // 16) + c: all
    # finite scales; one-hot activations read single elements, so a float32 output is the value
    N, K = 128, 256
    codes = np.repeat((np.arange(N) % 16).astype(np.uint8)[:, None], K, 1)
    sf = (16 * (np.arange(N) // 16)[:, None] + np.arange(K // 16)[None, :]).astype(np.uint8)
    sf[sf == 0x7F] = 0x7E
    w = raw_weight(codes, sf, np.float32(4.0))
    wf = Q.dequantize(codes, sf, np.float32(4.0))
    for k0 in range(0, K, 64):
        x = np.zeros((64, K))
        x[np.arange(64), k0 + np.arange(64)] = np.where(np.arange(64) % 2, -1.0, 0.5)
        got = nv.linear_w4a16(bf16(x).to(DEV), w, out_dtype=torch.float32).double().cpu().numpy()
        assert np.array_equal(got, P.linear(x, wf)[0])
        one = nv.linear_w4a16(bf16(x[:1]).to(DEV), w, out_dtype=torch.float32)  # the other path
        assert np.array_equal(one.double().cpu().numpy(), P.linear(x[:1], wf)[0])


@pytest.mark.parametrize("M_", [1, 6])
@pytest.mark.parametrize("top", [3.0e38, 1.0, 2.0 ** -100, 1e-38, 2.0 ** -133])
def test_activations_keep_their_bits_at_any_magnitude(top, M_):
    # an identity weight passes the activations through: those within 2^-29 of the row's maximum are
    # exact, smaller ones off by at most 2^-40 of it
    K = 2048
    codes = np.zeros((K, K), np.uint8)
    np.fill_diagonal(codes, 2)  # E2M1 1.0
    sf = np.full((K, K // 16), 0x38, np.uint8)  # E4M3 1.0
    w = raw_weight(codes, sf, np.float32(1.0))
    rng = np.random.default_rng(5)
    x = bf16(rng.uniform(1, 2, size=(M_, K)) * top * 2.0 ** -rng.integers(1, 60, size=(M_, K)))
    x[:, 7] = top
    got = nv.linear_w4a16(x.to(DEV), w, out_dtype=torch.float32).double().cpu()
    x = x.double()
    big = x.abs() >= x.abs().amax(1, keepdim=True) * 2.0 ** -28
    normal = x.abs() >= 2.0 ** -126  # float32 outputs below may be flushed
    assert torch.equal(got[big & normal], x[big & normal])
    lim = x.abs().amax(1, keepdim=True) * 2.0 ** -39 + 2.0 ** -126
    assert ((got - x).abs() <= lim).all()


@pytest.mark.parametrize("M_", [3, 12, 20])
def test_infinities_and_nans_stay_in_their_row(M_):
    w, wf = make_weight(200, 512, seed=1)
    x = bf16(np.random.default_rng(2).normal(size=(M_, 512)))
    x[0, 3], x[1, 500], x[2] = float("inf"), float("nan"), 0.0
    got = nv.linear_w4a16(x.to(DEV), w)
    assert not torch.isfinite(got[0]).any() or (wf[:, 3] == 0).any()
    assert torch.isnan(got[1]).all()
    assert (got[2] == 0).all()
    if M_ > 3:
        ref, mag = P.linear(x[3:].double().numpy(), wf)
        check(got[3:], ref, mag)


def test_strided_rows_an_output_and_no_rows():
    w, wf = make_weight(300, 256, seed=3)
    big = bf16(np.random.default_rng(4).normal(size=(40, 512))).to(DEV)
    for x in (big[::2, :256][:5], big[1:4, 256:], big[3:4, 256:], big[:, :256]):
        ref, mag = P.linear(x.double().cpu().numpy(), wf)
        buf = torch.full((x.shape[0] + 1, 300), 7.0, dtype=torch.bfloat16, device=DEV)
        out = nv.linear_w4a16(x, w, out=buf[:-1])
        check(out, ref, mag)
        assert out.data_ptr() == buf.data_ptr() and (buf[-1] == 7).all()
    assert nv.linear_w4a16(big[:0, :256], w).shape == (0, 300)
    with pytest.raises(nv.Nvfp4Error):
        nv.linear_w4a16(big[:2, 4:260], w)           # rows not 16-byte aligned
    with pytest.raises(nv.Nvfp4Error):
        nv.linear_w4a16(big[:1, :256].expand(4, 256), w)  # rows on top of one another


@pytest.mark.parametrize("M_", [2, 11])
def test_linear_on_another_stream_and_in_a_graph(M_):
    w, wf = make_weight(260, 1024, seed=6)
    xs = [bf16(np.random.default_rng(s).normal(size=(M_, 1024))).to(DEV) for s in range(3)]
    want = [nv.linear_w4a16(x, w) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = xs[0].clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(nv.linear_w4a16(x, w), want[0])
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = nv.linear_w4a16(x, w)
            again = nv.linear_w4a16(x, w)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(again, want[i])  # and reproducible


def test_prepacked_weights_of_any_row_count():
    wf = bf16(np.random.default_rng(8).normal(size=(200, 128)) * 0.05)
    w = nv.quantize_weights(lambda e: wf.to(DEV), 1, 200, 128)
    assert w.sf.numel() == nv.sf_bytes(200, 128)
    codes = F.unpack_nibbles(w.codes.cpu().numpy())
    sf = Q.untile_sf(w.sf.cpu().numpy(), 256, 8)[:200]
    deq = Q.dequantize(codes, sf, w.gs.cpu().numpy()[0])
    assert np.abs(deq - wf.double().numpy()).max() < 0.05
    x = bf16(np.random.default_rng(9).normal(size=(3, 128)))
    ref, mag = P.linear(x.double().numpy(), deq)
    check(nv.linear_w4a16(x.to(DEV), w), ref, mag)


# --------------------------------------------------------------------------------- expert FFN

def make_experts(E, H, I, seed):
    rng = np.random.default_rng(seed)
    w1 = M.QuantWeights.from_float(bf16(rng.normal(size=(E, 2 * I, H)) * 0.05).float().numpy())
    w2 = M.QuantWeights.from_float(bf16(rng.normal(size=(E, H, I)) * 0.05).float().numpy())
    return (upload_weights(w1, w1=True), upload_weights(w2),
            np.stack([w1.dequant(e) for e in range(E)]), np.stack([w2.dequant(e) for e in range(E)]))


def check_ffn(got, x, ids, wts, f1, f2):
    ref, bound = P.moe_ffn(x.double().cpu().numpy(), ids, wts, f1, f2)
    got = got.double().cpu().numpy()
    tol = bound * (1 + BF16_HALF) + (BF16_HALF + 2.0 ** -20) * np.abs(ref) + 1e-37
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 128, 64, 1, 1),        # the smallest; a shared expert
    (1, 1024, 512, 16, 4),
    (3, 256, 192, 5, 5),       # every expert for every token
    (7, 384, 320, 8, 2),
    (9, 128, 2048, 3, 1),      # long second product
    (16, 256, 128, 4, 2),      # 8 tokens an expert: two token tiles
    (40, 128, 128, 2, 2),      # 40 tokens an expert: blocks of 32
    (33, 256, 64, 40, 6),
    (60, 128, 1152, 3, 2),     # shares that end inside a block, several units of an expert
    (3, 4096, 64, 6, 2),       # a long first product in short shares
])
def test_ffn_from_logits_and_from_its_routing(T, H, I, E, k):
    w1, w2, f1, f2 = make_experts(E, H, I, seed=T + E)
    rng = np.random.default_rng(T)
    x = bf16(rng.normal(size=(T, H)))
    lg = rng.normal(size=(T, E)).astype(np.float32)
    ids, wts = R.route_topk(lg, k)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = nv.moe_ffn_w4a16(x.to(DEV), to_dev(lg), k, w1, w2, status=status)
    check_ffn(got, x, ids, wts, f1, f2)
    # the same routing given
    r = nv.permute(to_dev(lg), k)
    again = nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=r["ids"], weights=r["weights"],
                             status=status)
    assert torch.equal(got, again)  # also: reproducible
    assert nv.read_status(status) == (0, 0)


@pytest.mark.parametrize("E", [2, 4, 64])
def test_ffn_routing_corner_cases(E):
    """Dropped slots and tokens, one expert for everybody, an expert twice in a token."""
    T, H, I, k = 21, 128, 128, 2
    w1, w2, f1, f2 = make_experts(E, H, I, seed=E)
    rng = np.random.default_rng(E)
    x = bf16(rng.normal(size=(T, H)))
    wts = rng.uniform(0.1, 1, size=(T, k)).astype(np.float32)
    wts[2, 1] = np.nan  # of a dropped slot: not read
    base = rng.integers(0, E, size=(T, k)).astype(np.int32)
    one = np.full((T, k), E - 1, np.int32)  # every slot of every token on one expert
    dropped = base.copy()
    dropped[::3] = -1
    for ids in (base, one, dropped):
        ids[2, 1] = -1
        got = nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=to_dev(ids), weights=to_dev(wts))
        check_ffn(got, x, ids, wts, f1, f2)
        assert (got[(ids < 0).all(1)] == 0).all()
    nothing = nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=to_dev(np.full((T, k), -1, np.int32)),
                               weights=to_dev(wts))
    assert (nothing == 0).all()
    empty = nv.moe_ffn_w4a16(x.to(DEV)[:0], None, k, w1, w2, ids=to_dev(base[:0]),
                             weights=to_dev(wts[:0]))
    assert empty.shape == (0, H)


def test_ffn_reports_and_drops_ids_out_of_range():
    T, H, I, E, k = 5, 128, 64, 3, 2
    w1, w2, f1, f2 = make_experts(E, H, I, seed=11)
    x = bf16(np.random.default_rng(1).normal(size=(T, H)))
    ids = np.array([[0, 3], [1, 2], [7, 7], [2, -4], [1, 1 << 30]], np.int32)
    wts = np.full((T, k), 0.5, np.float32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=to_dev(ids), weights=to_dev(wts),
                           status=status)
    assert nv.read_status(status)[0] == 2
    check_ffn(got, x, ids, wts, f1, f2)


def test_ffn_masked_logits_and_non_finite_tokens():
    T, H, I, E, k = 6, 256, 64, 8, 3
    w1, w2, f1, f2 = make_experts(E, H, I, seed=12)
    rng = np.random.default_rng(12)
    x = bf16(rng.normal(size=(T, H)))
    lg = rng.normal(size=(T, E)).astype(np.float32)
    lg[0, 2:] = -np.inf            # two experts left: one slot dropped
    lg[1] = -np.inf                # none left
    lg[2, :4] = np.finfo(np.float32).min
    x[3, 5], x[4, 7] = float("nan"), float("inf")
    ids, wts = R.route_topk(lg, k)
    got = nv.moe_ffn_w4a16(x.to(DEV), to_dev(lg), k, w1, w2)
    assert (got[1] == 0).all()
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[4]).all()
    fine = [0, 1, 2, 5]
    check_ffn(got[fine], x[fine], ids[fine], wts[fine], f1, f2)


def test_ffn_on_another_stream_and_in_a_graph():
    T, H, I, E, k = 5, 512, 256, 16, 4
    w1, w2, f1, f2 = make_experts(E, H, I, seed=13)
    rng = np.random.default_rng(13)
    xs = [bf16(rng.normal(size=(T, H))).to(DEV) for _ in range(3)]
    lgs = [to_dev(rng.normal(size=(T, E)).astype(np.float32)) for _ in range(3)]
    want = [nv.moe_ffn_w4a16(a, b, k, w1, w2) for a, b in zip(xs, lgs)]
    for a, b, c in zip(xs, lgs, want):
        ids, wts = R.route_topk(b.cpu().numpy(), k)
        check_ffn(c, a, ids, wts, f1, f2)
    x, lg = xs[0].clone(), lgs[0].clone()
    ws = torch.full((nv.moe_ffn_w4a16_workspace_bytes(T, H, I, E, k),), 0xFF, dtype=torch.uint8,
                    device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = nv.moe_ffn_w4a16(x, lg, k, w1, w2, ws=ws)
            out2 = nv.moe_ffn_w4a16(out, lg, k, w1, w2, ws=ws)  # the same workspace, back to back
    for i in (2, 0, 1):
        x.copy_(xs[i])
        lg.copy_(lgs[i])
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(out2, nv.moe_ffn_w4a16(want[i], lgs[i], k, w1, w2))


@pytest.mark.parametrize("big", [1e4, 1e30])
def test_ffn_of_gates_far_below_zero(big):
    # g = -x0 and u = x0 for every feature: silu(-big) * big is 0 although big * big may not be finite
    H, I = 128, 64
    w1, w2 = np.zeros((1, 2 * I, H), np.float32), np.ones((1, H, I), np.float32)
    w1[:, :I, 0], w1[:, I:, 0] = -1.0, 1.0
    q1, q2 = M.QuantWeights.from_float(w1), M.QuantWeights.from_float(w2)
    f1, f2 = q1.dequant(0)[None], q2.dequant(0)[None]
    x = bf16(np.zeros((3, H)))
    x[:, 0] = torch.tensor([big, -1.0, 2.0])
    ids, wts = np.zeros((3, 1), np.int32), np.ones((3, 1), np.float32)
    got = nv.moe_ffn_w4a16(x.to(DEV), None, 1, upload_weights(q1, w1=True), upload_weights(q2),
                           ids=to_dev(ids), weights=to_dev(wts))
    assert (got[0] == 0).all()
    with np.errstate(over="ignore"):
        check_ffn(got, x, ids, wts, f1, f2)


def test_ffn_output_in_the_place_of_its_input():
    T, H, I, E, k = 9, 256, 128, 6, 2
    w1, w2, _, _ = make_experts(E, H, I, seed=14)
    x = bf16(np.random.default_rng(14).normal(size=(T, H))).to(DEV)
    lg = to_dev(np.random.default_rng(15).normal(size=(T, E)).astype(np.float32))
    want = nv.moe_ffn_w4a16(x, lg, k, w1, w2)
    assert torch.equal(nv.moe_ffn_w4a16(x, lg, k, w1, w2, out=x), want)


# ------------------------------------------------- products with many output blocks, larger batches

def random_weight(N, K, seed):
    """Random codes and scales: (device weights, codes, scales, global scale)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    sf = rng.integers(0x28, 0x41, (N, K // 16), dtype=np.uint8)  # 2^-2 to 2^1
    gs = np.float32(37.5)
    return raw_weight(codes, sf, gs), codes, sf, gs


# (rows, N, K): one and two token tiles, one to four blocks of tokens, shares of a CTA that begin and end
# inside blocks (but for K 64, a step per block), odd numbers of rows of the weight
STREAMED = [(6, 531000, 64), (5, 265201, 320), (3, 65521, 2304), (9, 177003, 576),
            (16, 110001, 1152), (33, 60001, 704), (64, 33333, 1280)]


@pytest.mark.parametrize("M_,N,K", STREAMED)
def test_linear_with_many_output_blocks(M_, N, K):
    rows = (N + 127) // 128
    # the form that streams the blocks in even shares: its workspace holds float32 planes of the output
    assert nv.linear_w4a16_workspace_bytes(M_, N, K) >= M_ * rows * 128 * 4
    w, codes, sf, gs = random_weight(N, K, seed=N)
    rng = np.random.default_rng(M_)
    wide = bf16(rng.normal(size=(2 * M_, K + 64)) * np.exp(rng.normal(size=(2 * M_, 1)) * 3)).to(DEV)
    x = wide[1::2, 64:]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = {t: nv.linear_w4a16(x, w, out_dtype=t, status=status) for t in (torch.float32, torch.bfloat16)}
    again = nv.linear_w4a16(x, w, out_dtype=torch.float32)
    assert nv.read_status(status) == (0, 0) and torch.equal(again, got[torch.float32])
    x64 = x.double().cpu().numpy()
    for n0 in range(0, N, 20000):
        n = slice(n0, n0 + 20000)
        ref, mag = P.linear(x64, Q.dequantize(codes[n], sf[n], gs))
        for v in got.values():
            check(v[:, n], ref, mag)


@pytest.mark.parametrize("M_,N,K", [(1, 200, 512), (3, 200, 512), (12, 200, 512), (4, 265201, 320),
                                    (34, 60001, 704)])
def test_infinities_keep_their_sign_and_reach_every_output_of_the_row(M_, N, K):
    w, codes, sf, gs = random_weight(N, K, seed=N + 1)
    x = bf16(np.random.default_rng(2).normal(size=(M_, K)))
    x[0, 3] = float("inf")
    if M_ > 1:
        x[1, K - 1], x[2] = float("nan"), 0.0
    got = nv.linear_w4a16(x.to(DEV), w, out_dtype=torch.float32).cpu()
    col = F.e2m1_decode(codes[:, 3])
    # infinity times a weight of 0 is no number
    want = torch.from_numpy(np.where(col == 0, np.nan, np.copysign(np.inf, col))).float()
    assert torch.equal(torch.isnan(got[0]), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[0][ok], want[ok])
    if M_ > 1:
        assert torch.isnan(got[1]).all() and (got[2] == 0).all()
    for n0 in range(0, N, 20000):
        n = slice(n0, n0 + 20000)
        ref, mag = P.linear(x[3:].double().numpy(), Q.dequantize(codes[n], sf[n], gs))
        check(got[3:, n], ref, mag)


@pytest.mark.parametrize("M_,N,K", [(2, 531000, 64), (20, 90112, 704)])
def test_streamed_linear_on_two_streams_and_in_a_graph(M_, N, K):
    w, _, _, _ = random_weight(N, K, seed=7)
    xs = [bf16(np.random.default_rng(s).normal(size=(M_, K))).to(DEV) for s in range(2)]
    want = [nv.linear_w4a16(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(nv.linear_w4a16(xs[i], w))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])
    ws = torch.full((nv.linear_w4a16_workspace_bytes(M_, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        out = nv.linear_w4a16(x, w, ws=ws)
        again = nv.linear_w4a16(x, w, ws=ws)  # the same workspace, back to back
    for i in (1, 0):
        x.copy_(xs[i])
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(again, want[i])


def share_of(T, I, E, k, ids, blocks, K):
    """(steps of a block, steps of a CTA's share) of one of the FFN's products, as the kernels cut it."""
    S, steps = T * k, (K + 255) // 256
    tok = 8 if 2 * S // E <= 8 else 16
    counts = np.bincount(ids[ids >= 0], minlength=E)
    total = int(((counts + tok - 1) // tok).sum()) * blocks * steps
    least = 4 if S <= 64 and steps > 4 else steps
    return steps, max(least, -(-total // 296))


@pytest.mark.parametrize("T,H,I,E,k", [
    (9, 1152, 1152, 5, 2),     # few slots: shares of 4 steps of blocks of 5
    (8, 1408, 640, 24, 8),     # 64 slots: shares of more steps than the ring has stages
    (40, 640, 704, 48, 2),     # more slots, one token tile: shares longer than a block
    (60, 640, 384, 64, 6),     # two token tiles
])
def test_ffn_shares_that_cross_blocks(T, H, I, E, k):
    w1, w2, f1, f2 = make_experts(E, H, I, seed=T + E)
    rng = np.random.default_rng(T)
    x = bf16(rng.normal(size=(T, H)))
    lg = rng.normal(size=(T, E)).astype(np.float32)
    ids, wts = R.route_topk(lg, k)
    steps, per = share_of(T, I, E, k, ids, 2 * I // 128, H)
    assert per % steps and steps % per
    got = nv.moe_ffn_w4a16(x.to(DEV), to_dev(lg), k, w1, w2)
    check_ffn(got, x, ids, wts, f1, f2)
    r = nv.permute(to_dev(lg), k)
    assert torch.equal(got, nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=r["ids"],
                                             weights=r["weights"]))


@pytest.mark.parametrize("T,E,k", [(512, 16, 8), (4096, 256, 1), (1500, 2, 2), (128, 32, 32)])
def test_ffn_of_many_slots(T, E, k):
    H, I = 128, 64
    w1, w2, f1, f2 = make_experts(E, H, I, seed=T + E)
    rng = np.random.default_rng(T)
    x = bf16(rng.normal(size=(T, H)))
    lg = rng.normal(size=(T, E)).astype(np.float32)
    ids, wts = R.route_topk(lg, k)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = nv.moe_ffn_w4a16(x.to(DEV), to_dev(lg), k, w1, w2, status=status)
    check_ffn(got, x, ids, wts, f1, f2)
    # a given routing, with dropped slots and experts named twice by a token
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    ids[T // 2:] = np.where(ids[T // 2:] >= 0, E - 1, -1)
    wts = rng.uniform(0.1, 1, size=(T, k)).astype(np.float32)
    got = nv.moe_ffn_w4a16(x.to(DEV), None, k, w1, w2, ids=to_dev(ids), weights=to_dev(wts),
                           status=status)
    check_ffn(got, x, ids, wts, f1, f2)
    assert (got[(ids < 0).all(1)] == 0).all() and nv.read_status(status) == (0, 0)
