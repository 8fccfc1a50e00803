"""Workloads of the operators around the expert FFN, for timing and comparing them.

  linear_w4a16    out = x W^T with bf16 x as it is and an NVFP4 weight matrix, for few rows of x
  moe_ffn_w4a16   the expert FFN of few tokens, neither x nor the intermediate quantized
  balance_loss    the router's load-balance loss, the expert counts and the logits' gradient
  residual_norm   post-norm of a block's output, its gate, the scaled residual sum and the next
                  block's pre-norm, and the gradients of all of it

``run`` computes an operator in plain torch (float32 inside, one rounding at the end) or, with
``own`` set, calls the package.  ``exact`` computes the same from the definitions in float64.

Data formats: NVFP4 weights are E2M1 codes two per byte (element 2j in the low nibble), an E4M3
scale per 16 elements stored in atoms of 128 rows x 4 scale columns, and a float32 global scale
per expert that the value is divided by.  The first FFN matrix stores its gate and up rows in
alternating blocks of 16.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # one token through the shared expert's gate/up projection: the smallest call of a decode
        # step, where the launch and the first load count
        dict(name="linear_1x4096x7168", op="linear", M=1, N=4096, K=7168, out="bf16"),
        # the same projection for the decode batch of 16
        dict(name="linear_16x4096x7168", op="linear", M=16, N=4096, K=7168, out="bf16"),
        # a vocabulary head with an odd number of entries, float32 logits, a few sequences
        dict(name="linear_5x65521x7168", op="linear", M=5, N=65521, K=7168, out="f32"),
        # the tiny configuration with given routing and dropped slots: launch-bound
        dict(name="moe_tiny_routed", op="moe", T=7, H=256, I=128, E=8, k=2, routed=True),
        # one token of a decode step: 8 of 256 experts
        dict(name="moe_1_token", op="moe", T=1, H=7168, I=2048, E=256, k=8, routed=False),
        # the decode batch: 16 tokens, about 100 experts, some of them shared by tokens
        dict(name="moe_16_tokens", op="moe", T=16, H=7168, I=2048, E=256, k=8, routed=False),
        # a short training batch of a small model, one sequence
        dict(name="balance_64x8", op="balance", way="both", T=64, E=8, k=2, seqs=1, padded=False),
        # a training batch of the large configuration, loss and gradient in one step
        dict(name="balance_8192x256", op="balance", way="both", T=8192, E=256, k=8, seqs=1,
             padded=False),
        # packed ragged sequences with padding tokens, gradient from the stored counts
        dict(name="balance_grad_40961x160", op="balance", way="backward", T=40961, E=160, k=6,
             seqs=13, padded=True),
        # one token of a decode step through both norms
        dict(name="norm_1x7168", op="norm", way="forward", T=1, H=7168, gate="channel", res="bf16"),
        # a prefill or training batch, float32 residual stream, a gate value per token
        dict(name="norm_8192x7168", op="norm", way="forward", T=8192, H=7168, gate="token",
             res="f32"),
        # its backward pass with layer-scale gates, bf16 residual stream
        dict(name="norm_grad_8191x7168", op="norm", way="backward", T=8191, H=7168, gate="channel",
             res="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "moe", "balance", "norm"])
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 64), N=_log_int(rng, 64, 16384),
                    K=64 * _log_int(rng, 1, 128), out=rng.choice(["bf16", "f32"]))
    if op == "moe":
        E = rng.choice([4, 8, 15, 60, 64, 128, 256])
        return dict(op=op, T=_log_int(rng, 1, 16), H=128 * _log_int(rng, 1, 56),
                    I=64 * _log_int(rng, 1, 32), E=E, k=rng.randint(1, min(8, E)),
                    routed=rng.random() < 0.5)
    if op == "balance":
        T, E = _log_int(rng, 1, 40000), rng.choice([2, 5, 8, 16, 60, 64, 100, 128, 160, 256])
        return dict(op=op, way=rng.choice(["both", "forward", "backward"]), T=T, E=E,
                    k=rng.randint(1, min(8, E)), seqs=min(T, _log_int(rng, 1, 64)),
                    padded=rng.random() < 0.5)
    return dict(op=op, way=rng.choice(["forward", "backward"]), T=_log_int(rng, 1, 8191),
                H=8 * _log_int(rng, 8, 896), gate=rng.choice(["none", "channel", "token", "full"]),
                res=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _activations(g, rows, cols):
    """Unit normal activations with a few large channels, as a hidden state has."""
    x = _randn(g, rows, cols)
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device=DEV)
    x[:, big] *= 12.0
    return x.to(BF16)


def _quantize(w):
    """bf16 (N, K) -> packed codes, tiled scale bytes, global scale: round to nearest."""
    N, K = w.shape
    x = w.float().view(N, K // 16, 16)
    gs = 2688.0 / x.abs().amax()
    sf = (x.abs().amax(2) / 6.0 * gs).to(torch.float8_e4m3fn)
    a = x * (gs / sf.float()).nan_to_num(0.0, 0.0, 0.0)[..., None]
    mag = a.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=w.device)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += mag > edge
    code += (a < 0).to(torch.uint8) * 8
    code = code.view(N, K // 2, 2)
    rows = (N + 127) // 128 * 128
    s = torch.zeros(rows, K // 16, dtype=torch.uint8, device=w.device)
    s[:N] = sf.view(torch.uint8)
    s = s.view(rows // 128, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return code[..., 0] | (code[..., 1] << 4), s, gs


def _weights(g, E, N, K):
    codes = torch.empty(E * N, K // 2, dtype=torch.uint8, device=DEV)
    rows = (N + 127) // 128 * 128
    sf = torch.empty(E * rows * K // 16, dtype=torch.uint8, device=DEV)
    gs = torch.empty(E, dtype=F32, device=DEV)
    for e in range(E):
        c, s, v = _quantize((_randn(g, N, K) * 0.02).to(BF16))
        codes[e * N:(e + 1) * N] = c
        sf[e * s.numel():(e + 1) * s.numel()] = s
        gs[e] = v
    return dict(codes=codes, sf=sf, gs=gs, E=E, N=N, K=K)


def _routing(g, case):
    """Router logits with an uneven load, and what a router gives for them."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn(g, T, E) + 0.5 * _randn(g, E)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    return logits, ids[:, :k].to(torch.int32).contiguous(), torch.softmax(top[:, :k], 1).contiguous()


def _sequences(g, case):
    """Ragged packed sequences; with padding, masked tokens and rows behind the last sequence."""
    T, S = case["T"], case["seqs"]
    used = T - T // 16 if case["padded"] else T
    cuts = torch.sort(torch.randint(0, used + 1, (S - 1,), generator=g, device=DEV))[0]
    ends = torch.tensor([0, used], device=DEV)
    offs = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    mask = torch.rand(T, generator=g, device=DEV) > 0.1 if case["padded"] else None
    return offs, mask


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "linear":
        st["x"] = _activations(g, case["M"], case["K"])
        st["w"] = _weights(g, 1, case["N"], case["K"])
    elif case["op"] == "moe":
        st["x"] = _activations(g, case["T"], case["H"])
        st["logits"], ids, weights = _routing(g, case)
        if case["routed"]:  # some slots dropped by the caller's router
            drop = torch.rand(ids.shape, generator=g, device=DEV) < 0.1
            st["ids"], st["weights"] = ids.masked_fill(drop, -1), weights.masked_fill(drop, 0.0)
        st["w1"] = _weights(g, case["E"], 2 * case["I"], case["H"])
        st["w2"] = _weights(g, case["E"], case["H"], case["I"])
    elif case["op"] == "balance":
        st["logits"], st["ids"], _ = _routing(g, case)
        st["offs"], st["mask"] = _sequences(g, case)
        st["alpha"] = 0.01
        st["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
        if case["way"] == "backward":
            st["counts"], st["tokens"] = _count(st, _seq_of(st, st["logits"].shape[0]))
    else:
        T, H = case["T"], case["H"]
        res = BF16 if case["res"] == "bf16" else F32
        st["r"] = (_activations(g, T, H).float() * 3.0 + _randn(g, T, H)).to(res)
        st["y"] = _activations(g, T, H)
        st["post_gamma"] = (1.0 + 0.1 * _randn(g, H)).to(BF16)
        st["pre_gamma"] = (1.0 + 0.1 * _randn(g, H)).to(BF16)
        shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[case["gate"]]
        st["gate"] = None if shape is None else torch.sigmoid(_randn(g, *shape)).to(BF16)
        st["scale"] = 0.5
        if case["way"] == "backward":
            st["dr_new"] = _randn(g, T, H).to(res)
            st["dn"] = _randn(g, T, H).to(BF16)
            st["rstd_post"], st["rstd_pre"] = _norm_forward(st)[2:]
    if own:
        import nvfp4_block_scaled_gsa_b200 as nv
        for name in ("w", "w1", "w2"):
            if name in st:
                st[name + "_nv"] = nv.NVFP4Weights(**st[name])
    return st


# ---------------------------------------------------------------------------- the plain forms
def _dequant(w, e=None):
    """float32 weights: the whole matrix, or those of the experts e (a device tensor)."""
    N, K = w["N"], w["K"]
    codes, sf = w["codes"].view(w["E"], N, K // 2), w["sf"].view(w["E"], -1)
    gs = w["gs"]
    if e is not None:
        codes, sf, gs = codes[e], sf[e], gs[e]
    n = codes.shape[0]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=F32, device=DEV)
    v = lut[torch.stack([codes & 15, codes >> 4], dim=-1).int()].view(n, N, K // 16, 16)
    rows = (N + 127) // 128
    s = sf.view(n, rows, K // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, rows * 128, K // 16)
    v = v * s[:, :N].contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return v.view(n, N, K) / gs.view(n, 1, 1)


def _linear(st):
    out = st["x"].float() @ _dequant(st["w"])[0].t()
    return out if st["case"]["out"] == "f32" else out.to(BF16)


def _moe(st):
    case, x = st["case"], st["x"].float()
    k, I = case["k"], case["I"]
    if case["routed"]:
        ids, wts = st["ids"].long().clamp_min(0), st["weights"] * (st["ids"] >= 0)
    else:
        top, ids = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        ids, wts = ids[:, :k], torch.softmax(top[:, :k], 1)
    out = torch.empty_like(x)
    for t in range(case["T"]):
        a = (_dequant(st["w1"], ids[t]) @ x[t]).view(k, I // 16, 2, 16)
        gate, up = a[:, :, 0].reshape(k, I), a[:, :, 1].reshape(k, I)
        h = gate * up / (1.0 + torch.exp(-gate))
        y = (_dequant(st["w2"], ids[t]) @ h[..., None])[..., 0]
        out[t] = (wts[t][:, None] * y).sum(0)
    return out.to(BF16)


def _seq_of(st, T):
    """Sequence of each token, S for a token that counts in none."""
    S = st["offs"].numel() - 1
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    s = (t[:, None] >= st["offs"][None, 1:]).sum(1)
    if st["mask"] is not None:
        s = torch.where(st["mask"], s, S)
    return torch.where(t >= st["offs"][0], s, S)


def _count(st, seq):
    """Slots per sequence and expert, tokens per sequence (tokens in no sequence fall away)."""
    S, E = st["offs"].numel() - 1, st["case"]["E"]
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=DEV)
    slot = seq[:, None] * E + st["ids"].long().clamp_min(0)
    counts.index_add_(0, slot.reshape(-1), (st["ids"] >= 0).int().reshape(-1))
    tokens = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    tokens.index_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    return counts.view(S + 1, E)[:S].contiguous(), tokens[:S].contiguous()


def _balance(st):
    case = st["case"]
    E, k, way = case["E"], case["k"], case["way"]
    seq = _seq_of(st, case["T"])
    counts, tokens = (st["counts"], st["tokens"]) if way == "backward" else _count(st, seq)
    n = tokens.float()
    f = torch.where(n[:, None] > 0, counts.float() * E / (k * n[:, None]), 0.0)
    coef = st["alpha"] / (n > 0).sum() * torch.where(n > 0, 1.0 / n, 0.0)
    f, coef = torch.cat([f, torch.zeros_like(f[:1])])[seq], torch.cat([coef, coef.new_zeros(1)])[seq]
    z = torch.exp(st["logits"] - st["logits"].amax(1, keepdim=True))
    p = z / z.sum(1, keepdim=True)
    v = (f * p).sum(1)
    dlogits = (st["dloss"] * coef)[:, None] * p * (f - v[:, None])
    if way == "backward":
        return dlogits
    loss = (coef.double() * v.double()).sum().float().reshape(1)
    return (loss, counts, tokens) if way == "forward" else (loss, counts, tokens, dlogits)


def _gate(st):
    """The gate as float32 (T, H), (1, H), (T, 1), or 1."""
    kind = st["case"]["gate"]
    if kind == "none":
        return 1.0
    v = st["gate"].float()
    return v[None, :] if kind == "channel" else v[:, None] if kind == "token" else v


def _norm_forward(st):
    r, y = st["r"].float(), st["y"].float()
    rstd_post = 1.0 / torch.sqrt((y * y).mean(1) + EPS)
    z = y * rstd_post[:, None] * st["post_gamma"].float()
    r_new = r + st["scale"] * _gate(st) * z
    rstd_pre = 1.0 / torch.sqrt((r_new * r_new).mean(1) + EPS)
    n = r_new * rstd_pre[:, None] * st["pre_gamma"].float()
    return r_new.to(st["r"].dtype), n.to(BF16), rstd_post, rstd_pre


def _norm_backward(st):
    kind = st["case"]["gate"]
    gate, scale, gpost, gpre = _gate(st), st["scale"], st["post_gamma"].float(), st["pre_gamma"].float()
    r, y, dn = st["r"].float(), st["y"].float(), st["dn"].float()
    rs_y, rs_r = st["rstd_post"][:, None], st["rstd_pre"][:, None]
    yhat = y * rs_y
    rhat = (r + scale * gate * gpost * yhat) * rs_r
    u = dn * gpre
    a = st["dr_new"].float() + rs_r * (u - rhat * (u * rhat).mean(1, keepdim=True))
    dz = scale * gate * a
    d = dz * gpost
    dy = rs_y * (d - yhat * (d * yhat).mean(1, keepdim=True))
    out = [a.to(st["r"].dtype), dy.to(BF16), (dz * yhat).sum(0), (dn * rhat).sum(0)]
    if kind != "none":
        dg = scale * a * yhat * gpost
        out.append(dg.sum(0) if kind == "channel" else dg.sum(1) if kind == "token" else dg.to(BF16))
    return tuple(out)


# --------------------------------------------------------------------------- the package's calls
def _own(st):
    import nvfp4_block_scaled_gsa_b200 as nv

    case, op = st["case"], st["case"]["op"]
    if op == "linear":
        return nv.linear_w4a16(st["x"], st["w_nv"], out_dtype=F32 if case["out"] == "f32" else BF16)
    if op == "moe":
        if case["routed"]:
            return nv.moe_ffn_w4a16(st["x"], None, case["k"], st["w1_nv"], st["w2_nv"],
                                    ids=st["ids"], weights=st["weights"])
        return nv.moe_ffn_w4a16(st["x"], st["logits"], case["k"], st["w1_nv"], st["w2_nv"])
    if op == "balance":
        at = dict(seq_offs=st["offs"], mask=st["mask"])
        if case["way"] == "backward":
            return nv.balance_loss_backward(st["logits"], st["counts"], st["tokens"], case["k"],
                                            st["alpha"], dloss=st["dloss"], **at)
        if case["way"] == "forward":
            return nv.balance_loss(st["logits"], st["ids"], st["alpha"], **at)[:3]
        return nv.balance_loss(st["logits"], st["ids"], st["alpha"], want_grad=True,
                               dloss=st["dloss"], **at)
    at = dict(post_gamma=st["post_gamma"], pre_gamma=st["pre_gamma"], gate=st["gate"],
              scale=st["scale"])
    if case["way"] == "forward":
        return nv.residual_norm(st["r"], st["y"], eps=EPS, **at)
    d = nv.residual_norm_backward(st["dr_new"], st["dn"], st["r"], st["y"], st["rstd_post"],
                                  st["rstd_pre"], **at)
    return tuple(v for v in (d["dr"], d["dy"], d["dpost_gamma"], d["dpre_gamma"], d["dgate"])
                 if v is not None)


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "linear":
        return _linear(state)
    if case["op"] == "moe":
        return _moe(state)
    if case["op"] == "balance":
        return _balance(state)
    return _norm_forward(state) if case["way"] == "forward" else _norm_backward(state)


# ----------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=N * K * 9 / 16 + 2 * M * K + M * N * (4 if case["out"] == "f32" else 2),
                    flops=2 * M * N * K)
    if op == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        busy = E * (1.0 - (1.0 - k / E) ** T)  # distinct experts of T draws of k out of E
        return dict(bytes=busy * 3 * H * I * 9 / 16 + 4 * T * H + 4 * T * E, flops=6 * T * k * H * I)
    if op == "balance":
        T, E, k, way = case["T"], case["E"], case["k"], case["way"]
        used = T - T // 16 if case["padded"] else T
        read = used * E * 4 + (0 if way == "backward" else used * k * 4)
        return dict(bytes=read + (0 if way == "forward" else T * E * 4), flops=8 * used * E)
    n, res = case["T"] * case["H"], 2 if case["res"] == "bf16" else 4
    gate = 2 * n if case["gate"] == "full" else 0
    if case["way"] == "forward":
        return dict(bytes=n * (2 * res + 4) + gate, flops=9 * n)
    return dict(bytes=n * (3 * res + 6) + 2 * gate, flops=25 * n)


# ---------------------------------------------------------------------------------------- exact
def _decode64(w, e=0):
    """float64 weights of expert e, from the bit fields of the codes and scales."""
    N, K = w["N"], w["K"]
    c = w["codes"][e * N:(e + 1) * N].to(torch.int16)
    c = torch.stack([c % 16, c // 16], 2).reshape(N, K)
    ex, m = ((c // 2) % 4).double(), (c % 2).double()
    v = torch.where(ex == 0, m / 2, (1 + m / 2) * 2.0 ** (ex - 1)) * (1.0 - 2.0 * (c // 8).double())
    r = torch.arange(N, device=DEV)[:, None]
    b = torch.arange(K // 16, device=DEV)[None, :]
    rows = (N + 127) // 128 * 128
    at = ((r // 128) * (K // 64) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    s = w["sf"][e * rows * K // 16 + at].to(torch.int16)
    se, sm = (s // 8).double(), (s % 8).double()
    d = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * 2.0 ** (se - 7))
    return (v.view(N, K // 16, 16) * d[..., None]).view(N, K) / w["gs"][e].double()


def _exact_moe(st):
    case = st["case"]
    x, k, I = st["x"].double(), case["k"], case["I"]
    if case["routed"]:
        ids, wts = st["ids"].tolist(), st["weights"].double().tolist()
    else:
        z = st["logits"].double()
        order = [sorted(range(case["E"]), key=lambda e: (-row[e], e))[:k] for row in z.tolist()]
        ids = order
        zs = torch.gather(z, 1, torch.tensor(order, device=DEV))
        zs = torch.exp(zs - zs.amax(1, keepdim=True))
        wts = (zs / zs.sum(1, keepdim=True)).tolist()
    out = torch.zeros(case["T"], case["H"], dtype=F64, device=DEV)
    j = torch.arange(I, device=DEV)
    gate_rows = j // 16 * 32 + j % 16
    for e in range(case["E"]):
        mine = [(t, i) for t in range(case["T"]) for i in range(k) if ids[t][i] == e]
        if not mine:
            continue
        w1, w2 = _decode64(st["w1"], e), _decode64(st["w2"], e)
        for t, i in mine:
            a = torch.mv(w1, x[t])
            gate, up = a[gate_rows], a[gate_rows + 16]
            out[t] += wts[t][i] * torch.mv(w2, gate * torch.sigmoid(gate) * up)
    return out


def _exact_balance(st):
    case, z = st["case"], st["logits"].double()
    T, E, k, way = case["T"], case["E"], case["k"], case["way"]
    offs = st["offs"].tolist()
    ok = st["mask"] if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    S = len(offs) - 1
    counts = torch.zeros(S, E, dtype=torch.int32, device=DEV)
    tokens = torch.zeros(S, dtype=torch.int32, device=DEV)
    loss = torch.zeros(1, dtype=F64, device=DEV)
    dz = torch.zeros(T, E, dtype=F64, device=DEV)
    alive = 0
    for s in range(S):
        sel = torch.nonzero(ok[offs[s]:offs[s + 1]])[:, 0] + offs[s]
        n = sel.numel()
        if n == 0:
            continue
        alive += 1
        tokens[s] = n
        picked = st["ids"][sel].reshape(-1).long()
        counts[s] = torch.bincount(picked[picked >= 0], minlength=E).int()
        f = counts[s].double() * E / (k * n)
        p = torch.softmax(z[sel], 1)
        loss += (f * p.mean(0)).sum()
        dz[sel] = p * (f - (p @ f)[:, None]) / n
    scale = st["alpha"] / max(alive, 1)
    dz *= scale * st["dloss"].double()
    if way == "backward":
        return dz
    return (scale * loss, counts, tokens) if way == "forward" else (scale * loss, counts, tokens, dz)


def _exact_norm(st):
    """Values and gradients in float64, the backward pass by torch's differentiation."""
    case = st["case"]
    leaf = {n: st[n].double().requires_grad_() for n in ("r", "y", "post_gamma", "pre_gamma")}
    kind = case["gate"]
    gate = None
    if kind != "none":
        gate = st["gate"].double().requires_grad_()
    shaped = 1.0 if gate is None else gate.unsqueeze(1) if kind == "token" else gate
    r, y = leaf["r"], leaf["y"]
    rstd_post = (y.square().mean(1) + EPS).rsqrt()
    r_new = r + st["scale"] * shaped * (y * rstd_post[:, None] * leaf["post_gamma"])
    rstd_pre = (r_new.square().mean(1) + EPS).rsqrt()
    n = r_new * rstd_pre[:, None] * leaf["pre_gamma"]
    if case["way"] == "forward":
        return r_new.detach(), n.detach(), rstd_post.detach(), rstd_pre.detach()
    wrt = [r, y, leaf["post_gamma"], leaf["pre_gamma"]] + ([] if gate is None else [gate])
    return torch.autograd.grad([r_new, n], wrt, [st["dr_new"].double(), st["dn"].double()])


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "linear":
        x = st["x"].double()
        whole, step = st["w"], 8192
        outs = []
        for n0 in range(0, case["N"], step):  # in row blocks that are whole scale atoms
            n1 = min(case["N"], n0 + step)
            K = case["K"]
            outs.append(x @ _decode64(dict(codes=whole["codes"][n0:n1], sf=whole["sf"][n0 * K // 16:],
                                           gs=whole["gs"], N=n1 - n0, K=K)).t())
        return torch.cat(outs, 1)
    if case["op"] == "moe":
        return _exact_moe(st)
    return _exact_balance(st) if case["op"] == "balance" else _exact_norm(st)
