"""Host-side checks of the operators around the expert FFN (CPU only): workspace sizes, and every
refusal before anything is launched."""

import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch

import nvfp4_block_scaled_gsa_b200 as nv
from nvfp4_block_scaled_gsa_b200 import build as B
from nvfp4_block_scaled_gsa_b200 import _native as N

F = ctypes.c_void_p(1 << 20)         # never dereferenced: every call below fails host validation
G = ctypes.c_void_p(1 << 21)         # another such
ODD = ctypes.c_void_p((1 << 20) + 8)  # 4- but not 16-byte aligned
BAD4 = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    B.build()
    return N.lib()


def test_linear_w4a16_workspace(L):
    ws = L.nvfp4_linear_w4a16_workspace_size
    assert ws(1, 4096, 7168) == 0                       # a few rows: none
    # 16 rows of 28 steps of 576 bytes and one word per row, in 256-byte units
    assert ws(16, 4096, 7168) == 16 * 28 * 576 + 256
    assert ws(100, 64, 64) == 112 * 576 + 512           # rows in blocks of 16, K in whole steps
    # many output blocks: also float32 planes, 4 for each row (2 pieces of 2 K warps)
    assert ws(5, 65521, 7168) == 8 * 28 * 576 + 256 + 5 * 4 * 512 * 128 * 4
    assert ws(0, 64, 64) == 0 and ws(-1, 64, 64) == 0 and ws(4, 0, 64) == 0


@pytest.mark.parametrize("change,code", [
    (dict(K=100, ld=128), 2),            # K % 64
    (dict(ld=64), 1),                    # ld < K
    (dict(ld=132), 2),                   # ld % 8
    (dict(M=-1), 1),
    (dict(M=16 * 65535 + 1), 2),
    (dict(N=0), 1),
    (dict(out_dtype=2), 1),
    (dict(x=None), 1),
    (dict(w=None), 1),
    (dict(sf=None), 1),
    (dict(gs=None), 1),
    (dict(out=None), 1),
    (dict(x=ODD), 3),
    (dict(w=ODD), 3),
    (dict(sf=ODD), 3),
    (dict(out=ODD), 3),
    (dict(ws=ODD), 3),
    (dict(gs=BAD4), 3),
    (dict(status=BAD4), 3),
    (dict(ws=None), 4),
    (dict(ws_bytes=16), 4),
    (dict(M=0, x=None, out=None, ws=None, ws_bytes=0), 0),
])
def test_linear_w4a16_refusals(L, change, code):
    a = dict(x=F, M=16, K=128, ld=128, w=F, sf=F, gs=F, N=256, out=F, out_dtype=1, ws=F,
             ws_bytes=BIG, status=None, stream=None)
    a.update(change)
    assert L.nvfp4_linear_w4a16(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(H=192), 2),                    # H % 128
    (dict(I=96), 2),                     # I % 64
    (dict(E=257), 2),
    (dict(E=0), 2),
    (dict(k=9), 2),                      # k > E
    (dict(k=0), 2),
    (dict(T=4096 // 2 + 1), 2),          # more slots than the form takes
    (dict(T=-1), 2),
    (dict(x=None), 1),
    (dict(logits=None), 1),              # neither logits nor a routing
    (dict(ids=F, w=F), 1),               # both
    (dict(logits=None, ids=F), 1),       # half a routing
    (dict(ws=None), 1),
    (dict(ws_bytes=100), 4),
    (dict(w1=ODD), 3),
    (dict(sf2=ODD), 3),
    (dict(out=ODD), 3),
    (dict(logits=BAD4), 3),
    (dict(ws=ctypes.c_void_p((1 << 20) + 64)), 3),
    (dict(T=0, x=None, ws=None, out=None), 0),
])
def test_moe_ffn_w4a16_refusals(L, change, code):
    a = dict(x=F, logits=F, ids=None, w=None, T=4, H=256, I=128, E=8, k=2, w1=F, sf1=F, gs1=F, w2=F,
             sf2=F, gs2=F, out=F, ws=F, ws_bytes=BIG, status=None, stream=None)
    a.update(change)
    assert L.moe_ffn_w4a16(*a.values()) == code


def test_moe_ffn_w4a16_workspace(L):
    ws = L.moe_ffn_w4a16_workspace_size
    S, H, I = 16 * 8, 7168, 2048
    assert ws(16, H, I, 256, 8) >= S * (H * 4 + I * 4 + I * 2) + 16 * H * 2
    assert ws(-1, H, I, 256, 8) == 0 and ws(0, H, I, 256, 8) > 0


@pytest.mark.parametrize("change,code", [
    (dict(E=257, ld=257), 2),
    (dict(k=33, E=64, ld=64), 2),
    (dict(k=9), 2),
    (dict(k=0), 1),
    (dict(T=-1), 1),
    (dict(ld=7), 1),
    (dict(S=0), 1),
    (dict(S=2, offs=None), 1),           # several sequences need their offsets
    (dict(T=1 << 30), 2),                # T * k
    (dict(logits=None), 1),
    (dict(ids=None), 1),
    (dict(counts=None), 1),
    (dict(tokens=None), 1),
    (dict(loss=None), 1),
    (dict(dlogits=F), 1),                # in place of the logits
    (dict(ws=None), 1),
    (dict(ws_bytes=8), 4),
    (dict(logits=BAD4), 3),
    (dict(offs=BAD4), 3),
    (dict(dlogits=BAD4), 3),
    (dict(ws=ODD), 3),
])
def test_balance_loss_refusals(L, change, code):
    a = dict(logits=F, ld=8, T=16, E=8, k=2, ids=F, offs=F, S=1, mask=None, alpha=0.01, counts=F,
             tokens=F, loss=F, dloss=None, dlogits=None, acc=0, ws=F, ws_bytes=BIG, status=None,
             stream=None)
    a.update(change)
    assert L.moe_balance_loss(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(E=300, ld=300), 2),
    (dict(ld=4), 1),
    (dict(S=3, offs=None), 1),
    (dict(counts=None), 1),
    (dict(tokens=None), 1),
    (dict(dlogits=None), 1),
    (dict(dlogits=F), 1),                # in place of the logits
    (dict(dloss=BAD4), 3),
    (dict(T=0, logits=None, dlogits=None), 0),
])
def test_balance_loss_backward_refusals(L, change, code):
    a = dict(logits=F, ld=8, T=16, E=8, k=2, counts=F, tokens=F, offs=None, S=1, mask=None,
             alpha=0.01, dloss=None, dlogits=G, acc=0, stream=None)
    a.update(change)
    assert L.moe_balance_loss_backward(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(H=60, ld_r=64, ld_y=64), 2),             # H % 8
    (dict(H=16392, ld_r=16392, ld_y=16392), 2),    # wider than the form takes
    (dict(ld_r=56), 1),
    (dict(ld_y=56), 1),
    (dict(ld_r=68), 2),
    (dict(ld_y=68), 2),
    (dict(dtype=2), 1),
    (dict(T=-1), 1),
    (dict(kind=4), 1),
    (dict(kind=1), 1),                             # a kind without a gate
    (dict(gate=F), 1),                             # a gate without a kind
    (dict(y=None), 1),                             # a post-norm of nothing
    (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1),
    (dict(r=None), 1),
    (dict(r_out=None), 1),
    (dict(n_out=None), 1),
    (dict(r=ODD), 3),
    (dict(y=ODD), 3),
    (dict(post=ODD), 3),
    (dict(n_out=ODD), 3),
    (dict(gate=ODD, kind=1), 3),
    (dict(gate=ctypes.c_void_p((1 << 20) + 1), kind=2), 3),
    (dict(rs1=BAD4), 3),
    (dict(T=0, r=None, r_out=None), 0),
])
def test_residual_norm_refusals(L, change, code):
    a = dict(r=F, dtype=1, ld_r=64, y=F, ld_y=64, T=4, H=64, post=F, gate=None, kind=0, scale=1.0,
             pre=F, eps=1e-6, r_out=F, n_out=F, rs1=F, rs2=F, stream=None)
    a.update(change)
    assert L.nvfp4_residual_norm(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(H=60, ld_r=64, ld_y=64), 2),
    (dict(dr_new=None, dn=None), 1),               # no gradient comes in
    (dict(pre=None, dpre=None), 1),                # dn without a pre-norm
    (dict(rs2=None), 1),
    (dict(rs1=None), 1),
    (dict(r=None), 1),
    (dict(dr=None), 1),
    (dict(dy=None), 1),
    (dict(post=None), 1),                          # dpost_gamma without a post-norm
    (dict(dgate=F), 1),                            # dgate without a gate
    (dict(ws=None), 4),
    (dict(ws_bytes=100), 4),
    (dict(dr_new=ODD), 3),
    (dict(dn=ODD), 3),
    (dict(dr=ODD), 3),
    (dict(ws=ODD), 3),
    (dict(gate=F, kind=3, dgate=ODD), 3),
    (dict(dpost=BAD4), 3),
])
def test_residual_norm_backward_refusals(L, change, code):
    a = dict(dr_new=F, dn=F, r=F, dtype=1, ld_r=64, y=F, ld_y=64, T=4, H=64, post=F, gate=None,
             kind=0, scale=1.0, pre=F, rs1=F, rs2=F, dr=F, dy=F, dpost=F, dpre=F, dgate=None, ws=F,
             ws_bytes=BIG, status=None, stream=None)
    a.update(change)
    assert L.nvfp4_residual_norm_backward(*a.values()) == code


def test_residual_norm_backward_workspace(L):
    ws = L.nvfp4_residual_norm_backward_workspace_size
    assert ws(8192, 7168) == 148 * 2 * 7168 * 4    # one CTA per SM, two column sums each
    assert ws(5, 64) == 5 * 2 * 64 * 4
    assert ws(0, 64) == 0 and ws(4, 60) == 0 and ws(4, 1 << 20) == 0


def test_wrappers_refuse_tensors_off_the_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = nv.NVFP4Weights(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                        torch.ones(1), 1, 8, 64)
    with pytest.raises(AssertionError):
        nv.linear_w4a16(x, w)
    with pytest.raises(AssertionError):
        nv.balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), 0.1)
    with pytest.raises(AssertionError):
        nv.residual_norm(x, x)
    with pytest.raises(AssertionError):
        nv.residual_norm(x.half(), x)              # a type it does not take


@pytest.mark.parametrize("x,out", [
    (1 << 20, 1 << 20),                                  # in place
    (1 << 20, (1 << 20) + (15 * 256 + 128) * 2 - 16),    # from x's last 16 bytes on
    ((1 << 20) + 16 * 256 * 4 - 16, 1 << 20),            # x from out's last 16 bytes on
])
def test_linear_w4a16_refuses_an_output_over_its_input(L, x, out):
    a = dict(x=ctypes.c_void_p(x), M=16, K=128, ld=256, w=F, sf=F, gs=F, N=256,
             out=ctypes.c_void_p(out), out_dtype=0, ws=F, ws_bytes=BIG, status=None, stream=None)
    assert L.nvfp4_linear_w4a16(*a.values()) == 1


def test_residual_norm_refuses_dense_rows_over_strided_ones(L):
    assert L.nvfp4_residual_norm(F, 1, 128, G, 64, 4, 64, F, None, 0, 1.0, F, 1e-6, F, F, None,
                                 None, None) == 1


def test_copying_warps_always_wait_for_their_last_copies():
    # Another warp's wait may run out when the copying warp has nothing left to wait for, and the
    # stages are then reused, or the CTA ends, under copies in flight.  No wait of a product can be
    # made to run out on a GPU without a fault, so the rule is checked in the source: each of the
    # two copying roles ends with an unconditional drain of what it issued.
    with open(os.path.join(B.CSRC, "w4a16.cu")) as f:
        src = f.read()
    ends = re.findall(r"\n( *)([^\n]*ring\.drain\(\w+\);)\n  \} else \{", src)
    assert [e[1] for e in ends] == ["ring.drain(issued);", "ring.drain(i);"]
    assert src.count("ring.drain(") == 2


def at(base, off):
    return ctypes.c_void_p(base + off)


ROW = 64 * 2  # bytes of a bf16 row of 64


# T = 4 rows of 64, r float32 or bf16 with rows of ld_r, y bf16 with rows of ld_y; the base addresses
# are far apart unless said otherwise
@pytest.mark.parametrize("change,code", [
    (dict(r_out=at(1 << 20, ROW)), 1),                      # one row behind r
    (dict(r_out=at(1 << 20, -ROW)), 1),                     # one row in front of it
    (dict(r_out=at(1 << 20, 4 * ROW - 16)), 1),             # over r's last 16 bytes
    (dict(n_out=at(1 << 20, ROW)), 1),
    (dict(n_out=at(1 << 21, 2 * ROW)), 1),                  # over y
    (dict(ld_r=128, n_out=at(1 << 20, 0)), 1),              # dense rows over strided ones
    (dict(ld_y=128, n_out=at(1 << 21, 0)), 1),
    (dict(ld_y=128, r_out=at(1 << 21, 0)), 1),
    (dict(dtype=0, n_out=at(1 << 20, 0)), 1),               # bf16 rows over float32 ones
    (dict(n_out=at(1 << 22, 3 * ROW)), 1),                  # over r_out
    (dict(post=at(1 << 22, 0)), 1),                         # r_out over a gamma
    (dict(pre=at(1 << 23, 2 * ROW)), 1),
    (dict(gate=at(1 << 22, 128), kind=3), 1),               # r_out over part of a full gate
    (dict(gate=at(1 << 23, 4 * ROW - 16), kind=1), 1),
    (dict(rs1=at(1 << 20, 0)), 1),                          # the rows' rstd over r
    (dict(rs2=at(1 << 22, 0)), 1),                          # ... over r_out
])
def test_residual_norm_refuses_outputs_over_other_rows(L, change, code):
    a = dict(r=at(1 << 20, 0), dtype=1, ld_r=64, y=at(1 << 21, 0), ld_y=64, T=4, H=64,
             post=at(1 << 24, 0), gate=None, kind=0, scale=1.0, pre=at(1 << 25, 0), eps=1e-6,
             r_out=at(1 << 22, 0), n_out=at(1 << 23, 0), rs1=at(1 << 26, 0), rs2=at(1 << 27, 0),
             stream=None)
    a.update(change)
    assert L.nvfp4_residual_norm(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(dr=at(1 << 20, ROW)), 1),                         # one row behind dr_new
    (dict(dr=at(1 << 22, -ROW)), 1),                        # one row in front of r
    (dict(dy=at(1 << 21, 2 * ROW)), 1),                     # over other rows of dn
    (dict(dy=at(1 << 23, ROW)), 1),                         # ... of y
    (dict(ld_y=128, dy=at(1 << 23, 0)), 1),                 # dense rows over strided ones
    (dict(ld_r=128, dr=at(1 << 22, 0)), 1),
    (dict(dtype=0, dr=at(1 << 21, 0)), 1),                  # float32 rows over bf16 ones
    (dict(dy=at(1 << 24, ROW)), 1),                         # over dr
    (dict(gate=at(1 << 27, 0), kind=3, dgate=at(1 << 27, ROW)), 1),
    (dict(gate=at(1 << 24, 0), kind=2), 1),                 # dr over a gate per token
    (dict(dpost=at(1 << 20, 0)), 1),
    (dict(dpre=at(1 << 28, 128)), 1),                       # over dpost
    (dict(ws=at(1 << 24, 0)), 1),                           # the workspace over dr
    (dict(rs2=at(1 << 25, 0)), 1),                          # dy over the rows' rstd
])
def test_residual_norm_backward_refuses_outputs_over_other_rows(L, change, code):
    a = dict(dr_new=at(1 << 20, 0), dn=at(1 << 21, 0), r=at(1 << 22, 0), dtype=1, ld_r=64,
             y=at(1 << 23, 0), ld_y=64, T=4, H=64, post=at(1 << 26, 0), gate=None, kind=0, scale=1.0,
             pre=at((1 << 26) + 4096, 0), rs1=at(1 << 29, 0), rs2=at((1 << 29) + 64, 0),
             dr=at(1 << 24, 0), dy=at(1 << 25, 0), dpost=at(1 << 28, 0), dpre=at((1 << 28) + 256, 0),
             dgate=None, ws=at(1 << 30, 0), ws_bytes=1 << 16, status=None, stream=None)
    a.update(change)
    assert L.nvfp4_residual_norm_backward(*a.values()) == code


# T = 16 rows of 8 logits, in rows of ld
@pytest.mark.parametrize("change", [
    dict(dlogits=at(1 << 20, 32)),                     # one row behind the logits
    dict(dlogits=at(1 << 20, -32)),
    dict(dlogits=at(1 << 20, 15 * 32 + 28)),           # over their last word
    dict(ld=16, dlogits=at(1 << 20, 15 * 64 + 28)),    # the same in strided rows
    dict(ld=16, dlogits=at(1 << 20, 32)),              # dense rows among strided ones
])
def test_balance_loss_refuses_a_gradient_over_the_logits(L, change):
    a = dict(logits=at(1 << 20, 0), ld=8, T=16, E=8, k=2, ids=F, offs=None, S=1, mask=None, alpha=0.01,
             counts=G, tokens=G, loss=G, dloss=None, dlogits=None, acc=0, ws=G, ws_bytes=BIG,
             status=None, stream=None)
    a.update(change)
    assert L.moe_balance_loss(*a.values()) == 1
    b = dict(logits=at(1 << 20, 0), ld=8, T=16, E=8, k=2, counts=G, tokens=G, offs=None, S=1,
             mask=None, alpha=0.01, dloss=None, dlogits=None, acc=1, stream=None)
    b.update(change)
    assert L.moe_balance_loss_backward(*b.values()) == 1


@pytest.mark.parametrize("out,w", [
    (1 << 20, (1 << 20) + 4 * 256 * 2 - 4),   # the routing weights in out's last bytes
    ((1 << 20) + 16, 1 << 20),                # out from inside the routing weights on
])
def test_moe_ffn_w4a16_refuses_an_output_over_its_routing_weights(L, out, w):
    a = dict(x=G, logits=None, ids=G, w=ctypes.c_void_p(w), T=4, H=256, I=128, E=8, k=2, w1=G, sf1=G,
             gs1=G, w2=G, sf2=G, gs2=G, out=ctypes.c_void_p(out), ws=G, ws_bytes=BIG, status=None,
             stream=None)
    assert L.moe_ffn_w4a16(*a.values()) == 1


def test_balance_loss_takes_a_gradient_buffer_only_when_it_is_wanted():
    with pytest.raises(AssertionError, match="want_grad"):
        nv.balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), 0.1,
                        dlogits=torch.zeros(2, 4))


def test_residual_norm_takes_no_output_that_it_would_not_fill():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="pre_gamma"):
        nv.residual_norm(x, x, out_n=torch.zeros_like(x))


def test_overlap_of_strided_rows_is_exact():
    # outputs between the rows of a strided input overlap nothing: compiled and run on the host
    src = '''
#include "launch.h"
#include <stdio.h>
int main() {
  long long rows, pitch, row, at, n, bad = 0;
  for (rows = 1; rows <= 4; ++rows) for (pitch = 4; pitch <= 9; ++pitch) for (row = 1; row <= pitch; ++row)
  for (at = -12; at <= 40; ++at) for (n = 1; n <= 7; ++n) {
    bool want = false;
    for (long long r = 0; r < rows; ++r)
      want = want || (r * pitch < at + n && at < r * pitch + row);
    const char* p = reinterpret_cast<const char*>(1 << 20);
    bad += nvfp4::rows_overlap(p, rows, pitch, row, p + at, n) != want;
    bad += nvfp4::rows_overlap(nullptr, rows, pitch, row, p, n) || nvfp4::rows_overlap(p, rows, pitch, row, nullptr, n);
  }
  printf("%lld\\n", bad);
}
'''
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "t.cpp"), "w") as f:
            f.write(src)
        cuda = os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")
        subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, "-I", cuda, "-o", os.path.join(d, "t"),
                        os.path.join(d, "t.cpp")], check=True)
        out = subprocess.run([os.path.join(d, "t")], check=True, capture_output=True, text=True).stdout
    assert out.strip() == "0"
