"""GPU parity of the router's balance loss, counts and gradient against the float64 oracle.

Bounds.  A probability comes from an exponential with relative error (2 + 1.4 |x|) 2^-24, x the
distance to the row's maximum (below 50 here wherever the probability counts), a sum of at most 256
terms in a tree over 16 lanes (21 roundings), a reciprocal and a product: below 2^-17.  f has three
roundings.  v_t adds 21 more on positive terms.  So the loss is within 2^-16 of itself, and a gradient
a p (f - v) within 2^-16 of a p (f + v)."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gsa_b200 as nv
from oracle import operators as P
from tests._gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


def problem(T, E, k, seed, S=1, mask=False, edge=False):
    rng = np.random.default_rng(seed)
    z = (rng.normal(size=(T, E)) * 2).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    lo, hi = (T // 7, T - T // 9) if edge else (0, T)
    offs = np.concatenate([[lo], np.sort(rng.integers(lo, hi + 1, size=S - 1)), [hi]]).astype(np.int32)
    keep = rng.random(T) > 0.3 if mask else None
    return z, ids, offs, keep


def check(z, ids, alpha, offs, keep, dloss, loss, counts, tokens, dlogits, extra=0.0):
    L, c, n, g = P.balance(z, ids, alpha, offs, keep, dloss)
    if counts is not None:
        assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    if loss is not None:
        assert abs(float(loss) - L) <= REL * abs(L) + 1e-37
    if dlogits is not None:
        got = dlogits.double().cpu().numpy() - extra
        k, E = ids.shape[1], z.shape[1]
        # a p (f + v) <= a p * 2 E/k: bounded through p with the row's own largest f
        tol = np.zeros_like(got)
        busy = max(int((n > 0).sum()), 1)
        for s in range(len(offs) - 1):
            if n[s] == 0:
                continue
            f = E * c[s] / (k * n[s])
            rows = slice(int(offs[s]), int(offs[s + 1]))
            zz = z[rows].astype(np.float64)
            with np.errstate(invalid="ignore"):
                p = np.exp(zz - zz.max(1, keepdims=True))
            p = np.nan_to_num(p / np.maximum(p.sum(1, keepdims=True), 1e-300))
            tol[rows] = REL * abs(dloss) * alpha / (busy * n[s]) * p * (f + (p @ f)[:, None])
        assert (np.abs(got - g) <= tol + 1e-37 + 2.0 ** -23 * np.abs(extra)).all()


@pytest.mark.parametrize("T,E,k,S,mask,edge", [
    (1, 1, 1, 1, False, False), (1, 2, 1, 1, False, False), (5, 3, 3, 1, True, False),
    (64, 8, 2, 1, False, False), (100, 7, 2, 3, False, True), (33, 16, 4, 33, True, False),
    (257, 17, 3, 5, True, True), (300, 60, 6, 2, False, False), (129, 64, 8, 1, True, False),
    (500, 100, 5, 9, True, True), (64, 128, 8, 1, False, False), (200, 160, 6, 4, True, False),
    (70, 255, 32, 2, False, False), (1030, 256, 8, 1, False, False), (90, 256, 8, 70, True, True),
    (3000, 5, 1, 1500, False, False),   # more sequences than the offsets' cache
])
def test_loss_counts_and_gradient(T, E, k, S, mask, edge):
    z, ids, offs, keep = problem(T, E, k, T + E, S, mask, edge)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    at = dict(seq_offs=to_dev(offs), mask=None if keep is None else to_dev(keep))
    dloss = torch.full((1,), 1.75, device=DEV)
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 0.3, want_grad=True,
                                              dloss=dloss, status=status, **at)
    check(z, ids, 0.3, offs, keep, 1.75, loss, counts, tokens, d)
    again = nv.balance_loss_backward(to_dev(z), counts, tokens, k, 0.3, dloss=dloss, **at)
    assert torch.equal(again, d)
    only, c2, n2, none = nv.balance_loss(to_dev(z), to_dev(ids), 0.3, **at)
    assert none is None and torch.equal(only, loss) and torch.equal(c2, counts)  # reproducible
    assert torch.equal(n2, tokens) and nv.read_status(status) == (0, 0)


def test_default_is_one_sequence_and_a_unit_gradient():
    z, ids, offs, _ = problem(50, 12, 2, 0)
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 0.01, want_grad=True)
    check(z, ids, 0.01, offs, None, 1.0, loss, counts, tokens, d)


def test_gradient_is_added_to_what_is_there():
    z, ids, offs, keep = problem(41, 24, 3, 1, 2, True, True)
    was = np.random.default_rng(3).normal(size=z.shape).astype(np.float32) * 1e-3
    at = dict(seq_offs=to_dev(offs), mask=to_dev(keep.astype(np.uint8)))
    buf = to_dev(was)
    _, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 0.5, want_grad=True, dlogits=buf,
                                           **at)
    assert d.data_ptr() == buf.data_ptr()
    check(z, ids, 0.5, offs, keep, 1.0, None, counts, tokens, d, extra=was.astype(np.float64))
    outside = np.ones(41, bool)
    outside[offs[0]:offs[-1]] = ~keep[offs[0]:offs[-1]]
    assert torch.equal(d.cpu()[outside], torch.from_numpy(was)[outside])  # not touched
    d2 = nv.balance_loss_backward(to_dev(z), counts, tokens, 3, 0.5, dlogits=to_dev(was), **at)
    assert torch.equal(d2, d)


def test_rows_that_mask_everything_and_masked_rows_of_anything():
    z, ids, offs, _ = problem(20, 10, 2, 4)
    z[3, 2:] = -np.inf
    z[4] = -np.inf
    z[5, :9] = np.finfo(np.float32).min
    z[9] = np.nan
    z[10, 1] = np.inf
    ids[4] = -1
    keep = np.ones(20, bool)
    keep[[9, 10]] = False
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 1.0, mask=to_dev(keep),
                                              want_grad=True)
    zz = z.copy()
    zz[[9, 10]] = 0.0
    check(zz, ids, 1.0, offs, keep, 1.0, loss, counts, tokens, d)
    assert (d[[4, 9, 10]] == 0).all() and torch.isfinite(d).all()
    # not masked, they show: in the loss, and in their own rows only
    loss, _, _, d = nv.balance_loss(to_dev(z), to_dev(ids), 1.0, want_grad=True)
    assert torch.isnan(loss).all()
    assert torch.isfinite(d).all(1).tolist() == [i not in (9, 10) for i in range(20)]


def test_nothing_to_count():
    z, ids, _, _ = problem(6, 4, 1, 5)
    none = torch.zeros(6, dtype=torch.bool, device=DEV)
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 1.0, mask=none, want_grad=True)
    assert loss.item() == 0 and (counts == 0).all() and (tokens == 0).all() and (d == 0).all()
    empty = torch.zeros(0, 4, device=DEV)
    loss, counts, tokens, d = nv.balance_loss(empty, torch.zeros(0, 1, dtype=torch.int32, device=DEV),
                                              1.0, want_grad=True)
    assert loss.item() == 0 and (counts == 0).all() and d.shape == (0, 4)


def test_bad_ids_and_offsets_are_reported():
    z, ids, _, _ = problem(12, 6, 2, 6)
    ids[3, 1], ids[7, 0] = 6, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 1.0, want_grad=True,
                                              status=status)
    assert nv.read_status(status)[0] == 2
    check(z, ids, 1.0, [0, 12], None, 1.0, loss, counts, tokens, d)  # they count for no expert
    status.zero_()
    offs = torch.tensor([-3, 5, 2, 40], dtype=torch.int32, device=DEV)
    nv.balance_loss(to_dev(z), to_dev(ids.clip(0, 5)), 1.0, seq_offs=offs, want_grad=True,
                    status=status)
    assert nv.read_status(status)[0] & 4


@pytest.mark.parametrize("E", [16, 18])
def test_strided_logits_stream_and_graph(E):
    z, ids, offs, keep = problem(80, E, 2, 7, 3, True)
    wide = torch.zeros(80, E + 5, device=DEV)
    wide[:, 1:1 + E] = to_dev(z)
    at = dict(seq_offs=to_dev(offs), mask=to_dev(keep))
    idd = to_dev(ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = nv.balance_loss(wide[:, 1:1 + E], idd, 0.2, want_grad=True, **at)
            more = nv.balance_loss_backward(wide[:, 1:1 + E], got[1], got[2], 2, 0.2, **at)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    check(z, ids, 0.2, offs, keep, 1.0, *got)
    assert torch.equal(more, got[3])
    z2, ids2, _, _ = problem(80, E, 2, 8)
    wide[:, 1:1 + E] = to_dev(z2)
    idd.copy_(to_dev(ids2))
    g.replay()
    torch.cuda.synchronize()
    check(z2, ids2, 0.2, offs, keep, 1.0, *got)


def test_gradient_against_differences_of_the_loss():
    z, ids, offs, keep = problem(30, 20, 3, 9, 2, True)
    d = np.random.default_rng(1).normal(size=z.shape)
    grad = nv.balance_loss(to_dev(z), to_dev(ids), 1.0, seq_offs=to_dev(offs), mask=to_dev(keep),
                           want_grad=True)[3].double().cpu().numpy()
    e = 1e-5
    z = z.astype(np.float64)
    quotient = (P.balance(z + e * d, ids, 1.0, offs, keep)[0] -
                P.balance(z - e * d, ids, 1.0, offs, keep)[0]) / (2 * e)
    scale = float(np.abs(grad * d).sum())
    assert abs(float((grad * d).sum()) - quotient) <= 4 * REL * scale + 1e-9


def test_counts_of_the_routers_own_output():
    T, E, k = 600, 32, 4
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(DEV)
    r = nv.permute(lg, k)
    _, counts, tokens, _ = nv.balance_loss(lg, r["ids"], 0.01)
    assert torch.equal(counts[0].long(), torch.bincount(r["ids"].flatten().long(), minlength=E))
    # the row map's segments hold exactly these counts, padded to 128
    seg = (r["offs"][1:] - r["offs"][:-1]).long()
    assert torch.equal(seg, (counts[0].long() + 127) // 128 * 128) and tokens.item() == T


@pytest.mark.parametrize("T,E", [(5, 3), (49, 2), (100, 5), (333, 8), (41, 32), (640, 6)])
def test_a_load_that_is_even_by_itself_has_no_gradient(T, E):
    # every token names every expert: f is 1 and f - v exactly 0, whatever the probabilities
    rng = np.random.default_rng(T)
    z = (rng.normal(size=(T, E)) * 3).astype(np.float32)
    ids = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.int32)
    dloss = torch.full((1,), 3.0, device=DEV)
    for keep in (None, rng.random(T) > 0.2):
        at = dict(mask=None if keep is None else to_dev(keep))
        loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 0.25, want_grad=True,
                                                  dloss=dloss, **at)
        assert abs(loss.item() - 0.25) <= REL * 0.25
        assert (d == 0).all()
        assert (nv.balance_loss_backward(to_dev(z), counts, tokens, E, 0.25, dloss=dloss, **at) == 0).all()


def test_far_probabilities_keep_their_bits():
    # Expert 0 takes every slot and, up to e^-30, all of the probability: z = 1, v = E, and the
    # gradient elsewhere is -a E p.  The logits' differences, a and E are exact, so what is left of
    # the relative error is the exponential's 2 * 2^-24 and six roundings: 2^-21.
    T, E = 64, 32
    z = -np.random.default_rng(11).integers(30 * 8, 80 * 8, size=(T, E)).astype(np.float32) / 8
    z[:, 0] = 0.0
    ids = np.zeros((T, 1), np.int32)
    ref = P.balance(z, ids, 0.5)[3]
    for shift in (0.0, 17.25):  # of the whole row: the same differences
        d = nv.balance_loss(to_dev(z + np.float32(shift)), to_dev(ids), 0.5, want_grad=True)[3]
        err = np.abs(d.double().cpu().numpy() - ref)[:, 1:] / np.abs(ref[:, 1:])
        assert err.max() <= 2.0 ** -21, err.max()


@pytest.mark.parametrize("T,E,k,S,mask,edge", [
    (8193, 256, 8, 1, False, False), (8193, 256, 8, 700, True, True), (20001, 160, 6, 13, True, True),
    (9001, 255, 4, 5, True, False), (120001, 2, 1, 3, True, True), (70011, 6, 3, 2000, False, True),
])
def test_long_batches(T, E, k, S, mask, edge):
    """More token groups than warps: a warp takes several, and meets sequences that its CTA did not
    start in; more CTAs than one round of the last sum."""
    assert int(nv.lib().moe_balance_loss_workspace_size(T, E)) > 256 + 256 * 8
    z, ids, offs, keep = problem(T, E, k, T + E, S, mask, edge)
    at = dict(seq_offs=to_dev(offs), mask=None if keep is None else to_dev(keep))
    dloss = torch.full((1,), 1.75, device=DEV)
    loss, counts, tokens, d = nv.balance_loss(to_dev(z), to_dev(ids), 0.3, want_grad=True, dloss=dloss,
                                              **at)
    check(z, ids, 0.3, offs, keep, 1.75, loss, counts, tokens, d)
    assert torch.equal(nv.balance_loss_backward(to_dev(z), counts, tokens, k, 0.3, dloss=dloss, **at), d)
    assert torch.equal(nv.balance_loss(to_dev(z), to_dev(ids), 0.3, **at)[0], loss)
