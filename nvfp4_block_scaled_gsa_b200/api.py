"""Torch-facing wrappers over the C ABI: allocate outputs with torch, pass pointers and the
current CUDA stream, check the status.  No arithmetic of the method happens here.
"""

from dataclasses import dataclass

import torch

from ._native import call, lib

U8, I32, F32, BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def round_up(v, m):
    return (v + m - 1) // m * m


def sf_bytes(rows, cols):
    """Bytes of a tiled block-scale buffer for `rows` rows of `cols` elements."""
    return round_up(rows, 128) * cols // 16


@dataclass
class NVFP4Weights:
    """Expert weights (E, N, K) as one NVFP4 tensor of E*N rows: codes (E*N, K/2) uint8, tiled
    scales, global scale per expert (E,) float32."""
    codes: torch.Tensor
    sf: torch.Tensor
    gs: torch.Tensor
    E: int
    N: int
    K: int


def quantize(x, gs=None, dst_row=None, k=1, out_rows=None, status=None):
    """NVFP4-quantize bf16 x (rows, cols).  gs=None: the global scale is computed on the GPU from
    amax (returned as a device tensor); otherwise gs (device float[1]) is used as given.
    dst_row/k/out_rows: permuted write (see nvfp4_quantize in the header)."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out_rows is None:
        out_rows = rows
    dev = x.device
    codes = torch.empty(out_rows, cols // 2, dtype=U8, device=dev)
    sf = torch.empty(sf_bytes(out_rows, cols), dtype=U8, device=dev)
    compute = gs is None
    if compute:
        gs = torch.empty(1, dtype=F32, device=dev)
    ws = torch.empty(int(lib().nvfp4_quantize_workspace_size()), dtype=U8, device=dev)
    call("nvfp4_quantize", _p(x), rows, cols, x.stride(0), _p(dst_row), k, out_rows, _p(codes),
         _p(sf), _p(gs), int(compute), _p(ws), ws.numel(), _p(status), _stream())
    return codes, sf, gs


def mxfp4_quantize(x, status=None):
    """MXFP4-quantize bf16 x (rows, cols): returns (codes (rows, cols/2) uint8, tiled UE8M0
    scales, one per 32 elements).  cols % 128 == 0; no global scale."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    codes = torch.empty(rows, cols // 2, dtype=U8, device=x.device)
    sf = torch.empty(round_up(rows, 128) * cols // 32, dtype=U8, device=x.device)
    call("mxfp4_quantize", _p(x), rows, cols, x.stride(0), _p(codes), _p(sf), _p(status),
         _stream())
    return codes, sf


def rmsnorm_quantize(x, gamma, eps, gs=None, dst_row=None, k=1, out_rows=None, status=None):
    """RMSNorm of bf16 x (rows, cols) with bf16 gamma (cols,), fused into the NVFP4 quantizer.
    Same outputs and options as quantize(); the normalized tensor itself is never written."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    assert gamma.dtype == BF16 and gamma.is_contiguous() and gamma.numel() == x.shape[1]
    rows, cols = x.shape
    if out_rows is None:
        out_rows = rows
    dev = x.device
    codes = torch.empty(out_rows, cols // 2, dtype=U8, device=dev)
    sf = torch.empty(sf_bytes(out_rows, cols), dtype=U8, device=dev)
    compute = gs is None
    if compute:
        gs = torch.empty(1, dtype=F32, device=dev)
    ws = torch.empty(int(lib().nvfp4_rmsnorm_quantize_workspace_size(rows)), dtype=U8, device=dev)
    call("nvfp4_rmsnorm_quantize", _p(x), rows, cols, x.stride(0), _p(gamma), float(eps),
         _p(dst_row), k, out_rows, _p(codes), _p(sf), _p(gs), int(compute), _p(ws), ws.numel(),
         _p(status), _stream())
    return codes, sf, gs


def gemm_dense(a_codes, a_sf, gs_a, M, w: "NVFP4Weights", out=None, ws=None, status=None):
    """Dense GEMM on NVFP4 activations (round_up(M, 128) rows of codes and tiled scales):
    bf16 (M, N) = A W^T with W one NVFP4 matrix (w.E == 1)."""
    assert w.E == 1
    if out is None:
        out = torch.empty(M, w.N, dtype=BF16, device=a_codes.device)
    need = int(lib().nvfp4_gemm_dense_workspace_size(M, w.N, w.K))
    if ws is None and need > 0:
        ws = torch.empty(need, dtype=U8, device=a_codes.device)
    call("nvfp4_gemm_dense", _p(a_codes), _p(a_sf), _p(gs_a), M, _p(w.codes), _p(w.sf), _p(w.gs),
         w.N, w.K, _p(out), _p(ws), 0 if ws is None else ws.numel(), _p(status), _stream())
    return out


def linear_workspace_bytes(M, N, K):
    return int(lib().nvfp4_linear_workspace_size(M, N, K))


def linear(x, w: "NVFP4Weights", gamma=None, eps=1e-6, out=None, ws=None, status=None):
    """Dense NVFP4 linear: bf16 x (M, K) -> bf16 (M, N) = x W^T, with W one NVFP4 matrix
    (w.E == 1, shape N x K).  gamma (bf16 (K,)) fuses an RMSNorm into the activation quantizer."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1 and w.E == 1
    M, K = x.shape
    assert K == w.K
    if out is None:
        out = torch.empty(M, w.N, dtype=BF16, device=x.device)
    if ws is None:
        ws = torch.empty(max(linear_workspace_bytes(M, w.N, K), 256), dtype=U8, device=x.device)
    call("nvfp4_linear", _p(x), M, K, x.stride(0), _p(gamma), float(eps), _p(w.codes), _p(w.sf),
         _p(w.gs), w.N, _p(out), _p(ws), ws.numel(), _p(status), _stream())
    return out


def shared_expert_workspace_bytes(M, H, I):
    return int(lib().nvfp4_shared_expert_workspace_size(M, H, I))


def shared_expert(x, w1: "NVFP4Weights", w2: "NVFP4Weights", gs_h, gamma=None, eps=1e-6,
                  out=None, ws=None, status=None):
    """The shared expert's FFN on every row of bf16 x (M, H): w1 from quantize_w1 with E = 1
    (gate/up interleave), w2 from quantize_weights with E = 1 (H x I); gs_h device float[1].
    gamma (bf16 (H,)) fuses an RMSNorm into the first quantizer.  Returns bf16 (M, H)."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1 and w1.E == 1 and w2.E == 1
    M, H = x.shape
    I = w1.N // 2
    assert w1.K == H and w2.N == H and w2.K == I
    if out is None:
        out = torch.empty(M, H, dtype=BF16, device=x.device)
    if ws is None:
        ws = torch.empty(max(shared_expert_workspace_bytes(M, H, I), 256), dtype=U8,
                         device=x.device)
    call("nvfp4_shared_expert", _p(x), M, H, x.stride(0), _p(gamma), float(eps), _p(w1.codes),
         _p(w1.sf), _p(w1.gs), _p(w2.codes), _p(w2.sf), _p(w2.gs), I, _p(gs_h), _p(out), _p(ws),
         ws.numel(), _p(status), _stream())
    return out


def quantize_weights(get_expert, E, N, K, device="cuda", row_map=None):
    """Pre-pack expert weights: get_expert(e) -> bf16 (N, K) on the device; each expert gets its
    own global scale from its amax.  row_map (device int32 [N]): stored row of each row."""
    codes = torch.empty(E * N, K // 2, dtype=U8, device=device)
    per_sf = sf_bytes(N, K)  # whole 128-row atoms: N need not be a multiple of 128
    sf = torch.empty(E * per_sf, dtype=U8, device=device)
    gs = torch.empty(E, dtype=F32, device=device)
    ws = torch.empty(int(lib().nvfp4_quantize_workspace_size()), dtype=U8, device=device)
    for e in range(E):
        w = get_expert(e)
        assert w.dtype == BF16 and tuple(w.shape) == (N, K)
        w = w.contiguous()
        call("nvfp4_quantize", _p(w), N, K, K, _p(row_map), 1, N, _p(codes[e * N:(e + 1) * N]),
             sf.data_ptr() + e * per_sf, gs.data_ptr() + 4 * e, 1, _p(ws), ws.numel(), None,
             _stream())
    return NVFP4Weights(codes, sf, gs, E, N, K)


def w1_row_map(I):
    """Host int32 [2I]: stored row of each logical W1 row (gate rows, then up rows)."""
    m = torch.empty(2 * I, dtype=I32)
    call("moe_w1_row_map", I, m.data_ptr())
    return m


def quantize_w1(get_expert, E, I, H, device="cuda"):
    """Pre-pack W1 (E experts of [2I][H]: gate rows then up rows) into the kernels' gate/up
    interleave of 16-row blocks (stored row 32j + i = gate row 16j + i, 32j + 16 + i = up row
    16j + i; moe_w1_row_map)."""
    row_map = w1_row_map(I).to(device)
    return quantize_weights(get_expert, E, 2 * I, H, device=device, row_map=row_map)


def rows_max(T, E, k):
    return int(lib().moe_rows_max(T, E, k))


def permute(logits, k, renormalize=True, ids=None, weights=None, E=None, status=None):
    """Top-k routing + expert-bucketed row map.  With logits=None, ids/weights (T, k) are the
    routing (ids < 0 dropped) and E must be given."""
    if logits is not None:
        T, E = logits.shape
        dev = logits.device
        ids = torch.empty(T, k, dtype=I32, device=dev)
        weights = torch.empty(T, k, dtype=F32, device=dev)
    else:
        T = ids.shape[0]
        dev = ids.device
    R = rows_max(T, E, k)
    offs = torch.empty(E + 1, dtype=I32, device=dev)
    dst_row = torch.empty(T * k, dtype=I32, device=dev)
    row_slot = torch.empty(max(R, 1), dtype=I32, device=dev)
    row_w = torch.empty(max(R, 1), dtype=F32, device=dev)
    ws_bytes = lib().moe_permute_workspace_size(T, E, k)
    ws = torch.empty(max(ws_bytes, 1), dtype=U8, device=dev)
    call("moe_permute", _p(logits), T, E, k, int(renormalize), _p(ids), _p(weights), _p(offs),
         _p(dst_row), _p(row_slot), _p(row_w), _p(ws), ws_bytes, _p(status), _stream())
    return dict(ids=ids, weights=weights, offs=offs, dst_row=dst_row, row_slot=row_slot,
                row_w=row_w, R_max=R, E=E, T=T, k=k)


def grouped_gemm(a_codes, a_sf, gs_a, w: NVFP4Weights, offs, out_dtype=F32, status=None,
                 out=None):
    """Plain 2D x 3D grouped GEMM: out[r] = A[r] . W_e^T / (gs_a * gs_w[e]).  Rows past
    offs[E] are left as they are (``out`` may be given, (R, N) of ``out_dtype``)."""
    R = a_codes.shape[0]
    if out is None:
        out = torch.empty(R, w.N, dtype=out_dtype, device=a_codes.device)
    assert out.shape == (R, w.N) and out.dtype == out_dtype and out.is_contiguous()
    call("nvfp4_grouped_gemm", _p(a_codes), _p(a_sf), _p(gs_a), _p(w.codes), _p(w.sf), _p(w.gs),
         _p(offs), w.E, w.N, w.K, R, _p(out), 0 if out_dtype == F32 else 1, _p(status), _stream())
    return out


def mxfp4_grouped_gemm(a_codes, a_sf, b_codes, b_sf, E, N, offs, out_dtype=F32, status=None,
                       out=None):
    """2D x 3D grouped GEMM on MXFP4 operands (mxfp4_quantize's format, no global scales):
    out[r] = A[r] . B_e^T for the rows r of expert e; B is [E*N][K]."""
    R = a_codes.shape[0]
    K = 2 * a_codes.shape[1]
    if out is None:
        out = torch.empty(R, N, dtype=out_dtype, device=a_codes.device)
    assert out.shape == (R, N) and out.dtype == out_dtype and out.is_contiguous()
    call("mxfp4_grouped_gemm", _p(a_codes), _p(a_sf), _p(b_codes), _p(b_sf), _p(offs), E, N, K, R,
         _p(out), 0 if out_dtype == F32 else 1, _p(status), _stream())
    return out


def l1_swiglu_q(a_codes, a_sf, gs_a, w1: NVFP4Weights, offs, gs_h, row_slot=None, status=None):
    """L1 GEMM + SwiGLU + NVFP4 re-quantization -> (h codes (R, I/2), h tiled scales).
    With row_slot, all-padding groups of 32 rows are skipped (left unwritten)."""
    R = a_codes.shape[0]
    I = w1.N // 2
    h = torch.empty(R, I // 2, dtype=U8, device=a_codes.device)
    sfh = torch.empty(sf_bytes(R, I), dtype=U8, device=a_codes.device)
    call("moe_grouped_gemm_l1_swiglu_q", _p(a_codes), _p(a_sf), _p(gs_a), _p(w1.codes),
         _p(w1.sf), _p(w1.gs), _p(offs), _p(row_slot), w1.E, w1.K, I, R, _p(gs_h), _p(h),
         _p(sfh), _p(status), _stream())
    return h, sfh


def l1_swiglu_q_stats(a_codes, a_sf, gs_a, w1: NVFP4Weights, offs, gs_h, row_slot=None,
                      h_stats=None, want_h32=False, status=None):
    """l1_swiglu_q, plus the epilogue's view of h: returns (h codes, h tiled scales, h_stats,
    h32).  h_stats: device uint32 (3,) accumulated into (zeroed here when not given): amax bits
    of |h| over real rows, saturated block scales, underflowed block scales.  h32 (with
    want_h32): the FP32 h values before quantization, (R, I), real rows only."""
    R = a_codes.shape[0]
    I = w1.N // 2
    dev = a_codes.device
    h = torch.empty(R, I // 2, dtype=U8, device=dev)
    sfh = torch.empty(sf_bytes(R, I), dtype=U8, device=dev)
    if h_stats is None:
        h_stats = torch.zeros(3, dtype=I32, device=dev)
    h32 = torch.zeros(R, I, dtype=F32, device=dev) if want_h32 else None
    call("moe_grouped_gemm_l1_swiglu_q_stats", _p(a_codes), _p(a_sf), _p(gs_a), _p(w1.codes),
         _p(w1.sf), _p(w1.gs), _p(offs), _p(row_slot), w1.E, w1.K, I, R, _p(gs_h), _p(h),
         _p(sfh), _p(h32), _p(h_stats), _p(status), _stream())
    return h, sfh, h_stats, h32


def scale_from_amax(amax_bits, gs):
    """gs (device float[1]) = 2688 / amax for the float bits in amax_bits (device 4-byte word),
    1.0 when not finite and positive; on the device, no host sync."""
    call("nvfp4_scale_from_amax", _p(amax_bits), _p(gs), _stream())
    return gs


def l2_scatter(h, sfh, gs_h, w2: NVFP4Weights, offs, row_slot, row_w, dst_row, T, k, status=None):
    """L2 GEMM + routing weight + scatter to token order -> (out fp32 (T, H), out bf16 (T, H))."""
    R = h.shape[0]
    H = w2.N
    I = w2.K
    ys = torch.empty(max(T * k, 1), H, dtype=F32, device=h.device)
    out32 = torch.empty(T, H, dtype=F32, device=h.device)
    out16 = torch.empty(T, H, dtype=BF16, device=h.device)
    call("moe_grouped_gemm_l2_scatter", _p(h), _p(sfh), _p(gs_h), _p(w2.codes), _p(w2.sf),
         _p(w2.gs), _p(offs), _p(row_slot), _p(row_w), _p(dst_row), w2.E, H, I, T, k, R, _p(ys),
         _p(out32), _p(out16), _p(status), _stream())
    return out32, out16


def l2_scatter_add(h, sfh, gs_h, w2: NVFP4Weights, offs, row_slot, row_w, dst_row, T, k,
                   status=None):
    """L2 GEMM + routing weight + scatter-ADD into token rows (reductions at L2, order not fixed)
    -> (out fp32 (T, H), out bf16 (T, H))."""
    R = h.shape[0]
    H, I = w2.N, w2.K
    acc = torch.empty(T, H, dtype=F32, device=h.device)
    out16 = torch.empty(T, H, dtype=BF16, device=h.device)
    call("moe_grouped_gemm_l2_scatter_add", _p(h), _p(sfh), _p(gs_h), _p(w2.codes), _p(w2.sf),
         _p(w2.gs), _p(offs), _p(row_slot), _p(row_w), _p(dst_row), w2.E, H, I, T, k, R,
         _p(acc), _p(out16), _p(status), _stream())
    return acc, out16


def l2_form(T, k, E, deterministic=False):
    """1 when moe_ffn_forward adds L2 rows into token rows for this batch, 0 for slot rows."""
    return int(lib().moe_ffn_l2_form(T, k, E, 2 if deterministic else 0))


def ffn_workspace_bytes(T, H, I, E, k):
    return int(lib().moe_ffn_workspace_size(T, H, I, E, k))


def moe_ffn_forward(x, logits, k, w1: NVFP4Weights, w2: NVFP4Weights, gs_h, out=None, ws=None,
                    status=None):
    """The whole expert FFN: bf16 x (T, H), float logits (T, E) -> bf16 out (T, H)."""
    T, H = x.shape
    E = logits.shape[1]
    I = w1.N // 2
    if out is None:
        out = torch.empty(T, H, dtype=BF16, device=x.device)
    need = ffn_workspace_bytes(T, H, I, E, k)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=U8, device=x.device)
    call("moe_ffn_forward", _p(x), _p(logits), T, H, I, E, k, _p(w1.codes), _p(w1.sf), _p(w1.gs),
         _p(w2.codes), _p(w2.sf), _p(w2.gs), _p(gs_h), _p(out), _p(ws), ws.numel(), _p(status),
         _stream())
    return out


FFN_DELAYED_GS_H = 1
FFN_DETERMINISTIC = 2


def moe_ffn_forward_ex(x, logits, k, w1: NVFP4Weights, w2: NVFP4Weights, gs_h, delayed=False,
                       deterministic=False, h_stats=None, out=None, ws=None, status=None):
    """moe_ffn_forward with options: h_stats (device int32 (3,), filled: amax bits of |h|,
    saturated and underflowed block scales); delayed=True: gs_h (device float[1]) replaced after
    use by 2688 / amax(h) for the next call; deterministic=True: the slot-ordered output sum."""
    T, H = x.shape
    E = logits.shape[1]
    I = w1.N // 2
    if out is None:
        out = torch.empty(T, H, dtype=BF16, device=x.device)
    need = ffn_workspace_bytes(T, H, I, E, k)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=U8, device=x.device)
    call("moe_ffn_forward_ex", _p(x), _p(logits), T, H, I, E, k, _p(w1.codes), _p(w1.sf),
         _p(w1.gs), _p(w2.codes), _p(w2.sf), _p(w2.gs), _p(gs_h),
         (FFN_DELAYED_GS_H if delayed else 0) | (FFN_DETERMINISTIC if deterministic else 0),
         _p(h_stats), _p(out), _p(ws), ws.numel(), _p(status), _stream())
    return out


def _call_on(dev, name, *args):
    """call(name, *args, stream) with dev current, on its current stream."""
    index = dev.index
    if index == torch._C._cuda_getDevice():
        call(name, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            call(name, *args, torch._C._cuda_getCurrentRawStream(index))


def _ptrs(dev, *tensors):
    """Data pointers (None for None) of tensors that all have to be on the CUDA device dev."""
    assert dev.type == "cuda", "CUDA tensors only"
    index = dev.index
    for t in tensors:
        assert t is None or t.get_device() == index, f"all tensors must be on {dev}"
    return [None if t is None else t.data_ptr() for t in tensors]


def _weight_ptrs(w: "NVFP4Weights", dev):
    """Pointers to the codes, scales and global scales of w, checked as the kernels index them."""
    codes, sf, gs = w.codes, w.sf, w.gs
    assert codes.dtype == U8 and codes.is_contiguous() and codes.shape == (w.E * w.N, w.K // 2)
    assert sf.dtype == U8 and sf.is_contiguous() and sf.numel() >= w.E * sf_bytes(w.N, w.K)
    assert gs.dtype == F32 and gs.is_contiguous() and gs.numel() >= w.E
    return _ptrs(dev, codes, sf, gs)


def _bytes(ws):
    if ws is None:
        return 0
    assert ws.is_contiguous()
    return ws.numel() * ws.element_size()


def _row_stride(x):
    """Row stride of a 2-D tensor (a single row has none that matters)."""
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def linear_w4a16_workspace_bytes(M, N, K):
    return int(lib().nvfp4_linear_w4a16_workspace_size(M, N, K))


def linear_w4a16(x, w: "NVFP4Weights", out_dtype=BF16, out=None, ws=None, status=None):
    """out (M, N) = x W^T with bf16 x (M, K) used as it is (not quantized, unlike linear()) and W
    one NVFP4 matrix (w.E == 1): for few rows (up to 8 of a large matrix, up to a few dozen of a
    small one linear() is slower).  out_dtype bf16 or float32; any N,
    K % 64 == 0; a given out must not overlap x."""
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1 and w.E == 1
    assert out_dtype in (BF16, F32)
    M, K = x.shape
    dev = x.device
    assert K == w.K
    weight = _weight_ptrs(w, dev)
    if out is None:
        out = torch.empty(M, w.N, dtype=out_dtype, device=dev)
    else:
        assert out.dtype == out_dtype and out.shape == (M, w.N) and out.is_contiguous()
    if ws is None:
        need = linear_w4a16_workspace_bytes(M, w.N, K)
        if need > 0:
            ws = torch.empty(need, dtype=U8, device=dev)
    px, pout, pws, pstatus = _ptrs(dev, x, out, ws, status)
    _call_on(dev, "nvfp4_linear_w4a16", px, M, K, _row_stride(x), *weight, w.N, pout,
             0 if out_dtype == F32 else 1, pws, _bytes(ws), pstatus)
    return out


def moe_ffn_w4a16_workspace_bytes(T, H, I, E, k):
    return int(lib().moe_ffn_w4a16_workspace_size(T, H, I, E, k))


def moe_ffn_w4a16(x, logits, k, w1: NVFP4Weights, w2: NVFP4Weights, ids=None, weights=None,
                  out=None, ws=None, status=None):
    """The expert FFN of a small batch with unquantized activations: bf16 x (T, H) -> bf16
    (T, H).  Routing from float32 logits (T, E), or logits=None with ids (T, k) int32 (< 0:
    dropped slot) and weights (T, k) float32.  w1 from quantize_w1, w2 from quantize_weights; T * k
    at most 4096 (moe_ffn_forward takes larger batches)."""
    assert x.dtype == BF16 and x.dim() == 2 and x.is_contiguous()
    T, H = x.shape
    E, I = w1.E, w1.N // 2
    assert w2.E == E and w1.K == H and w2.N == H and w2.K == I
    dev = x.device
    weight1, weight2 = _weight_ptrs(w1, dev), _weight_ptrs(w2, dev)
    if logits is not None:
        assert ids is None and weights is None
        assert logits.dtype == F32 and logits.shape == (T, E) and logits.is_contiguous()
    else:
        assert ids.dtype == I32 and ids.shape == (T, k) and ids.is_contiguous()
        assert weights.dtype == F32 and weights.shape == (T, k) and weights.is_contiguous()
    if out is None:
        out = torch.empty(T, H, dtype=BF16, device=dev)
    assert out.dtype == BF16 and out.shape == (T, H) and out.is_contiguous()
    if ws is None:
        ws = torch.empty(max(moe_ffn_w4a16_workspace_bytes(T, H, I, E, k), 256), dtype=U8,
                         device=dev)
    px, plogits, pids, pweights, pout, pws, pstatus = _ptrs(dev, x, logits, ids, weights, out, ws,
                                                            status)
    _call_on(dev, "moe_ffn_w4a16", px, plogits, pids, pweights, T, H, I, E, k, *weight1, *weight2,
             pout, pws, _bytes(ws), pstatus)
    return out


def _balance_operands(logits, seq_offs, mask, dloss, dlogits):
    """Checks shared by the balance loss and its gradient; returns (T, E, sequences)."""
    assert logits.dtype == F32 and logits.dim() == 2 and logits.stride(1) == 1
    T, E = logits.shape
    S = 1
    if seq_offs is not None:
        assert seq_offs.dtype == I32 and seq_offs.dim() == 1 and seq_offs.is_contiguous()
        S = seq_offs.numel() - 1
    assert T < 1 << 31 and S < 1 << 31
    if mask is not None:
        assert mask.dtype in (torch.bool, U8) and mask.shape == (T,) and mask.is_contiguous()
    if dloss is not None:
        assert dloss.dtype == F32 and dloss.numel() == 1
    if dlogits is not None:
        assert dlogits.dtype == F32 and dlogits.shape == (T, E) and dlogits.is_contiguous()
    return T, E, S


def balance_loss(logits, ids, alpha, seq_offs=None, mask=None, want_grad=False, dloss=None,
                 dlogits=None, ws=None, status=None):
    """The router's load-balance loss: alpha / S' * sum over the S' sequences that hold tokens of
    E * sum_e (share of their slots on e) * (mean softmax(logits)[e]).

    logits float32 (T, E) (rows may be strided), ids int32 (T, k) from permute().  seq_offs int32
    (S+1,): packed sequences (default: one of all tokens); mask (T,) bool or uint8: False/0 for
    padding tokens.  Returns (loss (1,), counts int32 (S, E), tokens int32 (S,), dlogits or
    None).  want_grad: dlogits (T, E) float32, times dloss (device float[1], default 1), in the
    same pass; a given dlogits is added to."""
    assert dlogits is None or want_grad, "dlogits is for want_grad=True"
    accumulate = dlogits is not None
    T, E, S = _balance_operands(logits, seq_offs, mask, dloss, dlogits)
    dev = logits.device
    assert ids.dtype == I32 and ids.dim() == 2 and ids.shape[0] == T and ids.is_contiguous()
    k = ids.shape[1]
    counts = torch.empty(S, E, dtype=I32, device=dev)
    tokens = torch.empty(S, dtype=I32, device=dev)
    loss = torch.empty(1, dtype=F32, device=dev)
    if want_grad and dlogits is None:
        dlogits = torch.empty(T, E, dtype=F32, device=dev)
    if ws is None:
        ws = torch.empty(int(lib().moe_balance_loss_workspace_size(T, E)), dtype=U8, device=dev)
    p = _ptrs(dev, logits, ids, seq_offs, mask, counts, tokens, loss, dloss, dlogits, ws, status)
    _call_on(dev, "moe_balance_loss", p[0], _row_stride(logits), T, E, k, p[1], p[2], S, p[3],
             float(alpha), p[4], p[5], p[6], p[7], p[8], int(accumulate), p[9], _bytes(ws), p[10])
    return loss, counts, tokens, dlogits


def balance_loss_backward(logits, counts, tokens, k, alpha, dloss=None, seq_offs=None, mask=None,
                          dlogits=None):
    """The gradient of balance_loss with respect to the logits, from its counts and tokens: float32
    (T, E), times dloss (device float[1], default 1).  A given dlogits is added to."""
    accumulate = dlogits is not None
    T, E, S = _balance_operands(logits, seq_offs, mask, dloss, dlogits)
    dev = logits.device
    assert counts.dtype == I32 and counts.shape == (S, E) and counts.is_contiguous()
    assert tokens.dtype == I32 and tokens.shape == (S,) and tokens.is_contiguous()
    if dlogits is None:
        dlogits = torch.empty(T, E, dtype=F32, device=dev)
    p = _ptrs(dev, logits, counts, tokens, seq_offs, mask, dloss, dlogits)
    _call_on(dev, "moe_balance_loss_backward", p[0], _row_stride(logits), T, E, k, p[1], p[2], p[3],
             S, p[4], float(alpha), p[5], p[6], int(accumulate))
    return dlogits


def _norm_operands(r, y, post_gamma, gate, pre_gamma):
    """Checks shared by residual_norm and its gradient; returns (T, H, gate kind)."""
    assert r.dtype in (BF16, F32) and r.dim() == 2 and r.stride(1) == 1
    T, H = r.shape
    if y is not None:
        assert y.dtype == BF16 and y.shape == (T, H) and y.stride(1) == 1
    for g in (post_gamma, pre_gamma):
        assert g is None or (g.dtype == BF16 and g.shape == (H,) and g.is_contiguous())
    kind = 0
    if gate is not None:
        assert gate.dtype == BF16 and gate.is_contiguous()
        shape = tuple(gate.shape)
        kind = (1 if shape == (H,) else 2 if shape in ((T,), (T, 1)) else
                3 if shape == (T, H) else -1)
        assert kind > 0, "gate must be (H,), (T,), (T, 1) or (T, H)"
    return T, H, kind


def residual_norm(r, y, post_gamma=None, gate=None, scale=1.0, pre_gamma=None, eps=1e-6,
                  out_r=None, out_n=None):
    """The norms around a block in one pass: z = RMSNorm(y) * post_gamma (z = y without one),
    r' = r + scale * gate * z, n = RMSNorm(r') * pre_gamma.

    r (T, H) bf16 or float32, y bf16 (T, H) (rows of both may be strided) or None (r' = r: a plain
    pre-norm); gammas bf16 (H,); gate bf16, (H,) per channel, (T,) or (T, 1) per token, (T, H), or
    None (a 1-D gate is per channel where T == H).  Returns (r', n, rstd of y (T,), rstd of r'
    (T,)): r' in r's type, n bf16 or None without pre_gamma, the last two float32 (or None) for
    residual_norm_backward.  out_r and out_n may be (T, H) inputs of the same type and row stride
    (out_r may be r itself), and overlap nothing otherwise."""
    T, H, kind = _norm_operands(r, y, post_gamma, gate, pre_gamma)
    assert out_n is None or pre_gamma is not None, "out_n needs a pre_gamma"
    dev = r.device
    if y is None:
        assert out_r is None
        out_r = r
    elif out_r is None:
        out_r = torch.empty(T, H, dtype=r.dtype, device=dev)
    assert out_r.dtype == r.dtype and out_r.shape == (T, H) and (y is None or out_r.is_contiguous())
    rstd_post = rstd_pre = None
    if post_gamma is not None:
        rstd_post = torch.empty(T, dtype=F32, device=dev)
    if pre_gamma is not None:
        rstd_pre = torch.empty(T, dtype=F32, device=dev)
        if out_n is None:
            out_n = torch.empty(T, H, dtype=BF16, device=dev)
        assert out_n.dtype == BF16 and out_n.shape == (T, H) and out_n.is_contiguous()
    p = _ptrs(dev, r, y, post_gamma, gate, pre_gamma, out_r, out_n, rstd_post, rstd_pre)
    _call_on(dev, "nvfp4_residual_norm", p[0], 0 if r.dtype == F32 else 1, _row_stride(r), p[1],
             H if y is None else _row_stride(y), T, H, p[2], p[3], kind, float(scale), p[4],
             float(eps), p[5], p[6], p[7], p[8])
    return out_r, out_n, rstd_post, rstd_pre


def residual_norm_backward(dr_new, dn, r, y, rstd_post, rstd_pre, post_gamma=None, gate=None,
                           scale=1.0, pre_gamma=None, ws=None, status=None):
    """The gradients of residual_norm from those of r' (dr_new, r's type) and n (dn, bf16), either
    None for zero; the other arguments as given to (r before an update in place) and returned by
    residual_norm.  Returns a dict:
    dr (r's type), dy (bf16), dpost_gamma and dpre_gamma (float32 (H,)), dgate (in the gate's
    shape: float32 per channel or token, bf16 (T, H)); None where there is no such input."""
    T, H, kind = _norm_operands(r, y, post_gamma, gate, pre_gamma)
    dev = r.device
    if dr_new is not None:
        assert dr_new.dtype == r.dtype and dr_new.shape == (T, H) and dr_new.is_contiguous()
    if dn is not None:
        assert dn.dtype == BF16 and dn.shape == (T, H) and dn.is_contiguous()
    for v in (rstd_post, rstd_pre):
        assert v is None or (v.dtype == F32 and v.shape == (T,) and v.is_contiguous())
    dr = torch.empty(T, H, dtype=r.dtype, device=dev)
    dy = dpost = dpre = dgate = None
    if y is not None:
        dy = torch.empty(T, H, dtype=BF16, device=dev)
    if post_gamma is not None:
        dpost = torch.empty(H, dtype=F32, device=dev)
    if pre_gamma is not None:
        dpre = torch.empty(H, dtype=F32, device=dev)
    if kind:
        dgate = torch.empty(gate.shape, dtype=BF16 if kind == 3 else F32, device=dev)
    if ws is None:
        ws = torch.empty(int(lib().nvfp4_residual_norm_backward_workspace_size(T, H)), dtype=U8,
                         device=dev)
    p = _ptrs(dev, dr_new, dn, r, y, post_gamma, gate, pre_gamma, rstd_post, rstd_pre, dr, dy, dpost,
              dpre, dgate, ws, status)
    _call_on(dev, "nvfp4_residual_norm_backward", p[0], p[1], p[2], 0 if r.dtype == F32 else 1,
             _row_stride(r), p[3], H if y is None else _row_stride(y), T, H, p[4], p[5], kind,
             float(scale), p[6], p[7], p[8], p[9], p[10], p[11], p[12], p[13], p[14], _bytes(ws), p[15])
    return dict(dr=dr, dy=dy, dpost_gamma=dpost, dpre_gamma=dpre, dgate=dgate)


def read_status(status):
    """Host copy of a device status word (synchronizes the current stream)."""
    host = torch.zeros(1, dtype=torch.int32)
    rc = lib().nvfp4_read_status(_p(status), host.data_ptr(), _stream())
    return int(host.item()), rc
