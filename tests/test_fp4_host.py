"""Refusals of the microscaled 4-bit entry points, on the host: every call below is rejected
(or has nothing to do) before any CUDA call."""
import pytest
import torch

from bit_nf4_quantized_unpack_b200 import build, qlora
from bit_nf4_quantized_unpack_b200.qlora import CFP4Matrix

P = 1 << 20          # 16-byte aligned fake pointer, never dereferenced
Q = (1 << 20) + 8    # misaligned fake pointer
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return qlora.lib()


def mat(rows=512, cols=1024, codes=P, scales=P, g=P, gn=1, fmt=1):
    return CFP4Matrix(codes, scales, g, gn, rows, cols, fmt)


def test_scales_bytes(L):
    f = L.qlora_fp4_scales_bytes
    assert f(128, 64, 1) == 512 and f(129, 64, 1) == 1024 and f(128, 96, 1) == 1024
    assert f(128, 128, 0) == 512 and f(1, 160, 0) == 1024 and f(0, 64, 0) == 0
    assert f(1, 48, 1) == 0 and f(1, 0, 1) == 0 and f(-1, 32, 1) == 0 and f(1, 32, 2) == 0
    assert f(1, 1 << 28, 0) == (1 << 28) // 128 * 512 and f(1, (1 << 28) + 32, 0) == 0
    assert f(1 << 31, 32, 1) == 0 and f(1 << 20, (1 << 20) + 32, 1) == 0


def test_quantize_refusals(L):
    def call(X=P, dt=1, rows=4, cols=64, fmt=1, codes=P, scales=P, g=P):
        return L.qlora_fp4_quantize(X, dt, rows, cols, fmt, codes, scales, g, None)
    assert call(rows=0) == 0 and call(rows=0, X=None) == 0
    assert call(fmt=2) == 1 and call(fmt=-1) == 1 and call(dt=2) == 1
    assert call(X=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1 and call(g=None) == 1
    assert call(cols=48) == 2 and call(cols=0) == 2 and call(rows=-1) == 2
    assert call(rows=(1 << 31) - 255) == 2 and call(rows=1 << 20, cols=(1 << 20) + 32) == 2
    assert call(X=Q) == 3 and call(codes=Q) == 3 and call(scales=Q) == 3 and call(g=Q) == 3


def test_quantize_weight_refusals(L):
    need = L.qlora_fp4_quantize_weight_workspace_size()
    def call(W=P, dt=1, n=64, k=64, fmt=1, c=P, s=P, g=P, tc=P, ts=P, ws=P, wsb=need):
        return L.qlora_fp4_quantize_weight(W, dt, n, k, fmt, c, s, g, tc, ts, ws, wsb, None)
    assert call(W=None) == 1 and call(c=None) == 1 and call(s=None) == 1 and call(g=None) == 1
    assert call(tc=None) == 1 and call(ts=None) == 1 and call(fmt=3) == 1 and call(dt=5) == 1
    assert call(n=48) == 2 and call(k=80) == 2 and call(n=0) == 2 and call(n=1 << 22) == 2
    assert call(W=Q) == 3 and call(tc=Q) == 3 and call(ts=Q) == 3 and call(ws=Q) == 3
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4


def test_dequant_refusals(L):
    f = L.qlora_fp4_dequant
    assert f(mat(rows=0, codes=None), 1, None, None) == 0
    assert f(mat(), 1, None, None) == 1 and f(mat(), 3, P, None) == 1
    assert f(mat(codes=None), 1, P, None) == 1 and f(mat(scales=None), 1, P, None) == 1
    assert f(mat(fmt=7), 1, P, None) == 1
    assert f(mat(cols=1000), 1, P, None) == 2 and f(mat(gn=3), 1, P, None) == 2
    assert f(mat(gn=0), 1, P, None) == 2
    assert f(mat(), 1, Q, None) == 3 and f(mat(g=Q), 1, P, None) == 3


def test_matmul_refusals(L):
    f = L.qlora_fp4_matmul
    assert f(mat(rows=0), mat(), 1, None, None) == 0
    assert f(mat(), mat(fmt=0), 1, P, None) == 1 and f(mat(), mat(), 1, None, None) == 1
    assert f(mat(), mat(), 4, P, None) == 1
    assert f(mat(), mat(cols=512), 1, P, None) == 2
    assert f(mat(), mat(rows=12), 1, P, None) == 2 and f(mat(), mat(rows=0), 1, P, None) == 2
    assert f(mat(), mat(), 1, Q, None) == 3


def test_linear_refusals(L):
    need = L.qlora_fp4_linear_fwd_workspace_size(64, 512, 1024, 8, 1)
    bneed = L.qlora_fp4_linear_bwd_workspace_size(64, 512, 1024, 8, 1)
    assert need > 0 and bneed > 0
    for bad in ((64, 500, 1024, 8, 1), (64, 512, 1000, 8, 1), (64, 512, 1024, 12, 1),
                (64, 512, 1024, 72, 1), (64, 512, 1024, 8, 2), (-1, 512, 1024, 8, 1)):
        assert L.qlora_fp4_linear_fwd_workspace_size(*bad) == 0
        assert L.qlora_fp4_linear_bwd_workspace_size(*bad) == 0

    def fwd(X=P, M=64, w=None, A=P, B=P, r=8, scale=2.0, Y=P, T=None, ws=P, wsb=need):
        return L.qlora_fp4_linear_fwd(X, M, w or mat(), A, B, r, scale, Y, T, ws, wsb, None)
    assert fwd(M=0, X=None, Y=None) == 0
    assert fwd(X=None) == 1 and fwd(A=None) == 1 and fwd(B=None) == 1 and fwd(Y=None) == 1
    assert fwd(r=4) == 1 and fwd(r=12) == 1 and fwd(r=72) == 1 and fwd(scale=NAN) == 1
    assert fwd(w=mat(rows=520)) == 2 and fwd(w=mat(gn=512)) == 2 and fwd(M=-1) == 2
    assert fwd(X=Q) == 3 and fwd(T=Q) == 3 and fwd(ws=Q) == 3 and fwd(w=mat(codes=Q)) == 3
    assert fwd(ws=None) == 4 and fwd(wsb=need - 1) == 4

    def bwd(dY=P, X=P, T=None, M=64, wt=None, A=P, B=P, r=8, scale=2.0, dX=P, dA=P, dB=P, ws=P,
            wsb=bneed):
        return L.qlora_fp4_linear_bwd(dY, X, T, M, wt or mat(1024, 512), A, B, r, scale, dX, dA,
                                      dB, ws, wsb, None)
    assert bwd(dY=None) == 1 and bwd(X=None) == 1 and bwd(dA=None) == 1 and bwd(dB=None) == 1
    assert bwd(scale=float("inf")) == 1 and bwd(wt=mat(1000, 512)) == 2
    assert bwd(dX=Q) == 3 and bwd(T=Q) == 3 and bwd(dA=Q) == 3 and bwd(wsb=bneed - 1) == 4


def test_binding_refuses_what_it_cannot_pass_on():
    """Host tensors, wrong types and shapes, and storage smaller than its sizes say."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_quantize(x)
    with pytest.raises(TypeError):
        qlora.qlora_fp4_quantize(x.half())
    with pytest.raises(qlora.QLoraError):
        qlora.FP4Matrix.empty(4, 48, device="cpu")
    q = qlora.FP4Matrix.empty(4, 64, device="cpu")
    assert q.codes.shape == (4, 32) and q.scales.numel() == 512 and q.gscale.numel() == 4
    with pytest.raises(ValueError):
        qlora.qlora_fp4_dequant(q)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_matmul(q, q)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_linear_bwd(x, x, None, qlora.FP4Weight(q), x, x, 1.0)


def test_mxfp4_output_with_a_gscale_is_refused():
    """Quantizing to MXFP4 writes no gscale, and a product would multiply by the one left there."""
    q = qlora.FP4Matrix.empty(64, 64, qlora.FP4_MXFP4, device="cpu")
    q.gscale = torch.full((64,), 3.0)
    with pytest.raises(ValueError, match="gscale"):
        qlora.qlora_fp4_quantize(torch.zeros(64, 64), qlora.FP4_MXFP4, out=q)
    q.gscale = q.gscale[:1]
    with pytest.raises(ValueError, match="gscale"):
        qlora.qlora_fp4_quantize_weight(torch.zeros(64, 64), qlora.FP4_MXFP4, transposed=False,
                                        out=qlora.FP4Weight(q))


@pytest.mark.parametrize("fmt", [qlora.FP4_MXFP4, qlora.FP4_NVFP4])
def test_weight_output_whose_transpose_would_go_stale_is_refused(fmt):
    """transposed=False into a weight that has a transposed copy would leave the copy's old codes, which
    the backward would multiply by under the new gscale."""
    out = qlora.FP4Weight(qlora.FP4Matrix.empty(64, 96, fmt, device="cpu", gscale_rows=1),
                          qlora.FP4Matrix.empty(96, 64, fmt, device="cpu", gscale_rows=1))
    with pytest.raises(ValueError, match="out.wt"):
        qlora.qlora_fp4_quantize_weight(torch.zeros(64, 96), fmt, transposed=False, out=out)


def test_backward_in_place_is_refused(L):
    """dX over X or dY, which dA and dB read beside or behind the product that writes it: the same
    address, and ranges that overlap at either end (64 x 1024 and 64 x 512 bf16)."""
    need = L.qlora_fp4_linear_bwd_workspace_size(64, 512, 1024, 8, 1)
    x, dy = 1 << 24, 1 << 26

    def bwd(dX):
        return L.qlora_fp4_linear_bwd(dy, x, None, 64, mat(1024, 512), P, P, 8, 1.0, dX, P, P, P, need, None)
    for dX in (x, dy, x + 131072 - 16, x - 131072 + 16, dy + 65536 - 16, dy - 131072 + 16):
        assert bwd(dX) == 1, dX
