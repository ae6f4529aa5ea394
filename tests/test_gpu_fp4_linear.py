"""GPU parity of the microscaled 4-bit product and of the linear layer on it against the fp64
oracle.

Tolerances, element by element. u = 2^-23 bounds the relative error of one fp32 addition,
rounded or truncated. A product of K values is a chain of K / 64 additions into the
accumulator, each of which may also drop bits below u of the running sum of magnitudes S, so
its error is at most (K / 64 + 8) u S; a rank-r product (K / 16 steps, then at most 64 partial
sums) at most (K / 16 + 80) u S. A bf16 hi + lo pair keeps 2^-16 of its value. bf16 outputs add
half a bf16 step, 2^-8 of the value, and the errors of what is rounded."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_unpack_b200 import qlora
from oracle import fp4_oracle as F
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

FMTS = [qlora.FP4_MXFP4, qlora.FP4_NVFP4]
U, PAIR, BF16 = 2.0 ** -23, 2.0 ** -16, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert qlora.qlora_device_error() == 0


def normal(seed, *shape, std=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.normal(0, std, shape)).to(torch.bfloat16)


def within(got, want, tol, what):
    got, tol = got.detach().double().cpu().numpy(), np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    bad = np.abs(got - want) > tol
    i = np.unravel_index(np.argmax(np.abs(got - want) - tol), want.shape) if want.size else None
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst at {i}: {got[i]} for {want[i]}, tol {tol[i]}"


def product_tol(a, b):
    return (a.shape[1] / 64 + 8) * U * (np.abs(a) @ np.abs(b).T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 32), (2, 136, 64), (31, 128, 96), (32, 256, 256), (33, 1000, 288), (64, 40, 1056),
    (65, 264, 4096), (128, 128, 512), (129, 520, 544), (256, 256, 1024), (300, 1000, 1056),
    (513, 384, 160), (1, 4096, 11008), (16, 4096, 4096), (700, 2056, 2048)])
def test_matmul(M, N, K, fmt):
    a, b = normal(M + K, M, K).cuda(), normal(N, N, K, std=0.02).cuda()
    a[M // 2] = 0.0
    qa, qb = qlora.qlora_fp4_quantize(a, fmt), qlora.qlora_fp4_quantize(b, fmt)
    va, vb = (F.dequant(F.quantize(t.double().cpu().numpy(), fmt)) for t in (a, b))
    want, tol = va @ vb.T, product_tol(va, vb)
    big = torch.full((M + 2, N), 7.0, device="cuda")
    got = qlora.qlora_fp4_matmul(qa, qb, out=big[1:M + 1])
    within(got, want, tol, "fp32")
    assert (big[0] == 7).all() and (big[M + 1] == 7).all()
    got16 = qlora.qlora_fp4_matmul(qa, qb)
    within(got16, want, tol + BF16 * (np.abs(want) + tol), "bf16")
    assert torch.equal(got, qlora.qlora_fp4_matmul(qa, qb, torch.float32))  # the same bits again


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (2600, 4128, 288),     # several rounds of the CTA pairs, accumulators in turn, K ends in a step
    (300, 12544, 160),     # several rounds of narrow tiles
    (300, 50176, 32),      # many rounds of one step, narrow and (below) wide
    (8000, 2048, 32),
    (130, 256, 32),        # one tile, one MMA
    (8, 20000, 2304),      # more weight tiles than SMs, two CTAs to an SM
    (128, 24576, 320),     # the same with one CTA to an SM
    (40, 128, 8192),       # one tile, its K shared by eight CTAs
])
def test_matmul_schedules(M, N, K, fmt):
    a, b = normal(M + K, M, K).cuda(), normal(N, N, K, std=0.02).cuda()
    qa, qb = qlora.qlora_fp4_quantize(a, fmt), qlora.qlora_fp4_quantize(b, fmt)
    va, vb = (qlora.qlora_fp4_dequant(q, torch.float32).double() for q in (qa, qb))
    want = (va @ vb.t()).cpu().numpy()
    tol = (K / 64 + 8) * U * (va.abs() @ vb.abs().t()).cpu().numpy()
    for _ in range(2):
        got = qlora.qlora_fp4_matmul(qa, qb, torch.float32)
        within(got, want, tol, "fp32")
    within(qlora.qlora_fp4_matmul(qa, qb), want, tol + BF16 * (np.abs(want) + tol), "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (20000, 288, 32),      # wide tiles, every second one with 32 rows of the weight
    (9000, 928, 32),       # the last of four with 160
    (20000, 1152, 64),     # the last of five in one CTA of the pair
    (5000, 4128, 32),
    (300, 12320, 32),      # narrow tiles
])
def test_matmul_tiles_past_the_last_weight_row(M, N, K, fmt):
    """Many tiles a CTA pair, some of whose warps have no weight row: the rows that such a warp
    finished before stay as they are. Both epilogues scale the same fp32 sums in the same order, so the
    bf16 output is the fp32 one rounded."""
    a, b = normal(M + K, M, K).cuda(), normal(N, N, K, std=0.02).cuda()
    qa, qb = qlora.qlora_fp4_quantize(a, fmt), qlora.qlora_fp4_quantize(b, fmt)
    got = qlora.qlora_fp4_matmul(qa, qb, torch.float32)
    for _ in range(10):
        assert torch.equal(qlora.qlora_fp4_matmul(qa, qb), got.to(torch.bfloat16))
    va, vb = (qlora.qlora_fp4_dequant(q, torch.float32).double() for q in (qa, qb))
    want, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    assert ((got.double() - want).abs() <= (K / 64 + 8) * U * mag).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_reads_every_scale_in_its_place(fmt):
    """One-hot codes under scales that all differ: each output is one product of a code and two
    scales, exact in fp32."""
    g = np.random.default_rng(1)
    b = F.BLOCK[fmt]
    for M, N, K in ((40, 136, 416), (300, 264, 288)):
        def one_hot(rows):
            codes = np.zeros((rows, K), np.uint8)
            codes[np.arange(rows), g.integers(0, K, rows)] = g.integers(1, 16, rows)
            lo, hi = (100, 150) if fmt == F.MX else (1, 127)
            return {"codes": codes, "bytes": g.integers(lo, hi, (rows, K // b)).astype(np.uint8),
                    "g": np.ones(1), "fmt": fmt}
        def full(rows):
            q = one_hot(rows)
            q["codes"] = np.full((rows, K), 2, np.uint8)
            return q
        for ra, rb in ((one_hot(M), full(N)), (full(M), one_hot(N))):
            qa, qb = (qlora.FP4Matrix(torch.from_numpy(F.pack(r["codes"])).cuda(),
                                      torch.from_numpy(F.store_scales(r["bytes"])).cuda(), None,
                                      *r["codes"].shape, fmt) for r in (ra, rb))
            want = F.dequant(ra) @ F.dequant(rb).T
            got = qlora.qlora_fp4_matmul(qa, qb, torch.float32)
            assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 300])
def test_matmul_nan_blocks_and_gscales(M, fmt):
    """A NaN block reaches the outputs of its row (column) alone; gscales per row and single."""
    K, N = 544, 136
    a, b = normal(3, M, K).cuda(), normal(4, N, K).cuda()
    a[2, 100], b[7, 540] = float("nan"), float("inf")
    qa, qb = qlora.qlora_fp4_quantize(a, fmt), qlora.qlora_fp4_quantize(b, fmt)
    out = qlora.qlora_fp4_matmul(qa, qb, torch.float32)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[2], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(out), nan)
    ga = torch.rand(M, device="cuda") + 0.5
    gb = torch.rand(1, device="cuda") + 0.5
    bare = [qlora.FP4Matrix(q.codes, q.scales, None, q.rows, q.cols, fmt) for q in (qa, qb)]
    base = qlora.qlora_fp4_matmul(*bare, torch.float32)
    got = qlora.qlora_fp4_matmul(qlora.FP4Matrix(qa.codes, qa.scales, ga, M, K, fmt),
                                 qlora.FP4Matrix(qb.codes, qb.scales, gb, N, K, fmt), torch.float32)
    want = (base * gb) * ga[:, None]
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def layer(seed, M, N, K, r, fmt):
    W, A, B = normal(seed, N, K, std=0.02), normal(seed + 1, K, r, std=0.02), normal(seed + 2, r, N, std=0.02)
    X, dY = normal(seed + 3, M, K), normal(seed + 4, M, N)
    if M > 4:
        X[M // 2] = 0.0
        dY[M - 1] = 0.0
    return W, A, B, X, dY


def check_layer(M, N, K, r, fmt, scale=0.5, saved_T=True):
    W, A, B, X, dY = layer(M + N + K, M, N, K, r, fmt)
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    Xc, Ac, Bc, dYc = X.cuda(), A.cuda(), B.cuda(), dY.cuda()
    Y, T = qlora.qlora_fp4_linear_fwd(Xc, q, Ac, Bc, scale)
    dX, dA, dB = qlora.qlora_fp4_linear_bwd(dYc, Xc, T if saved_T else None, q, Ac, Bc, scale)
    A64, B64, X64, dY64 = (t.double().numpy() for t in (A, B, X, dY))
    w, _ = F.quantize_weight(W.double().numpy(), fmt)
    Y64, T64 = F.linear_forward(X64, w, A64, B64, scale)
    dX64, dA64, dB64 = F.linear_backward(dY64, X64, w, A64, B64, scale)
    a = np.abs
    Wv, Xq, dYq = F.dequant(w), F.dequant(F.quantize(X64, fmt)), F.dequant(F.quantize(dY64, fmt))
    T_tol = (K / 16 + 80) * U * (a(X64) @ a(A64))
    within(T, T64, T_tol, "T")
    lora = lambda v, tol, m: abs(scale) * ((PAIR + 16 * U) * (a(v) @ a(m)) + tol @ a(m))
    y_tol = product_tol(Xq, Wv) + lora(T64, T_tol, B64)
    within(Y, Y64, y_tol + BF16 * (a(Y64) + y_tol), "Y")
    G64 = dY64 @ B64.T
    G_tol = (N / 16 + 80) * U * (a(dY64) @ a(B64).T)
    x_tol = product_tol(dYq, Wv.T) + lora(G64, G_tol, A64.T)
    within(dX, dX64, x_tol + BF16 * (a(dX64) + x_tol), "dX")
    steps = (M / 16 + 80) * U + PAIR
    within(dA, dA64, abs(scale) * (steps * (a(X64).T @ a(G64)) + a(X64).T @ G_tol), "dA")
    within(dB, dB64, abs(scale) * (steps * (a(T64).T @ a(dY64)) + T_tol.T @ a(dY64)), "dB")
    return q, (Xc, Ac, Bc, dYc), (Y, T, dX, dA, dB)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r", [
    (1, 32, 32, 8), (1, 1024, 4096, 16), (5, 160, 96, 8), (16, 512, 1024, 64), (33, 416, 288, 24),
    (64, 256, 544, 40), (128, 288, 256, 16), (129, 352, 1056, 8), (300, 384, 640, 64), (520, 1056, 512, 32)])
def test_linear(M, N, K, r, fmt):
    check_layer(M, N, K, r, fmt)


@pytest.mark.parametrize("M", [1, 70, 200])
def test_linear_recomputes_T(M):
    check_layer(M, 160, 320, 16, qlora.FP4_NVFP4, saved_T=False)


@pytest.mark.parametrize("M,N,K,r", [
    (2, 96, 8256, 8),         # T in three parts of K
    (100, 8256, 96, 64),      # G in three parts of N
    (2600, 4128, 288, 24),    # several rounds with the rank-r steps, forward
    (2600, 288, 4128, 64),    # and for dX
    (300, 12544, 160, 40),
    (17, 20000, 64, 16),
])
def test_linear_schedules(M, N, K, r):
    check_layer(M, N, K, r, qlora.FP4_NVFP4 if r != 24 else qlora.FP4_MXFP4)


def product(a, b):
    """a b of small fp64 matrices term by term: a library's product may add 0 times an infinity."""
    with np.errstate(invalid="ignore"):
        return np.stack([(a[:, :, None] * b[None, :, j:j + 8]).sum(1) for j in range(0, b.shape[1], 8)], 1).reshape(
            a.shape[0], b.shape[1])


def same_class(got, want, what):
    """Infinities with their signs and NaNs where the formula has them, finite values elsewhere."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want)), what


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 100, 300, 1100])
def test_layer_with_values_that_are_not_finite(M, fmt):
    """An infinity or a NaN in each operand in turn. G and T are exact in bf16 in half of the columns,
    so that their lower parts are 0 there."""
    N, K, r, scale, inf, nan = 96, 64, 8, 0.5, float("inf"), float("nan")
    W, A, B, X, dY = (t.clone() for t in layer(51, M, N, K, r, fmt))
    X[X == 0], dY[dY == 0] = 0.5, 0.25                     # no 0 times an infinity but where it is meant
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    T = torch.from_numpy(np.random.default_rng(5).normal(0, 1, (M, r))).float()
    T[:, ::2] = T[:, ::2].to(torch.bfloat16).float()

    def run(X, T, dY, A, B):
        Y, _ = qlora.qlora_fp4_linear_fwd(X.cuda(), q, A.cuda(), B.cuda(), scale)
        dX, dA, dB = qlora.qlora_fp4_linear_bwd(dY.cuda(), X.cuda(), T.cuda(), q, A.cuda(), B.cuda(), scale)
        X, T, dY, A, B = (t.double().numpy() for t in (X, T, dY, A, B))
        with np.errstate(invalid="ignore", over="ignore"):
            G = product(dY, B.T)
            return Y, dX, dA, dB, product(product(X, A), B), product(G, A.T), product(X.T, G), product(T.T, dY)

    def put(t, *at):
        t = t.clone()
        for i, j, v in at:
            t[i, j] = v
        return t
    base = run(X, T, dY, A, B)
    for got, what in zip(base[:4], ("Y", "dX", "dA", "dB")):
        assert torch.isfinite(got).all(), what
    m = M - 2
    # T: dB alone
    out = run(X, put(T, (m, 1, inf), (0, 2, -inf), (1, 3, nan)), dY, A, B)
    assert torch.equal(out[0], base[0]) and torch.equal(out[1], base[1]) and torch.equal(out[2], base[2])
    same_class(out[3], out[7], "dB of T")
    # X: its rows of Y, its rows of dA
    out = run(put(X, (m, 5, inf), (0, 9, -inf), (1, 40, nan)), T, dY, A, B)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[m, 0, 1]] = True
    assert torch.isnan(out[0][bad]).all() and torch.equal(out[0][~bad], base[0][~bad])
    assert torch.equal(out[1], base[1]) and torch.equal(out[3], base[3])
    same_class(out[2], out[6], "dA of X")
    # X against a G that is exact in bf16, so that its lower parts are 0
    one = put(torch.zeros_like(dY), (m, 7, 1.0))
    out = run(put(X, (m, 5, inf)), T, one, A, B)
    same_class(out[2][5], out[6][5], "dA of X, exact G")
    # dY: its rows of dX, columns of dB, and dA through G
    out = run(X, T, put(dY, (m, 11, -inf)), A, B)
    assert torch.isnan(out[1][m]).all()
    keep = torch.arange(M, device="cuda") != m
    assert torch.equal(out[1][keep], base[1][keep])
    same_class(out[2], out[6], "dA of dY")
    same_class(out[3], out[7], "dB of dY")
    # A: Y through T; B: dA and dX through G
    out = run(X, T, dY, put(A, (3, 2, inf)), B)
    same_class(out[0], out[4], "Y of A")
    out = run(X.abs(), T, dY.abs(), A, put(B, (4, 13, -inf)))
    same_class(out[1], out[5], "dX of B")
    same_class(out[2], out[6], "dA of B")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 100, 300, 1100])
def test_gradients_hold_T_and_G_to_the_last_bit(M, fmt):
    """dB with one 1 in each column of dY is that token's T, and dA with one 1 in each column of X that
    token's G, 24 bits of each: three bf16 parts hold 8 bits each, and adding them to one another and
    to zeros is exact in fp32. G is a sum of three products of 8 bits at 1, 2^-8 and 2^-16, whose partial
    sums are fp32 numbers."""
    N, K, r = 160, 96, 16
    g = np.random.default_rng(M)
    W, A, X = normal(61, N, K, std=0.02), normal(62, K, r, std=0.02), normal(63, M, K)
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    T = torch.from_numpy(g.uniform(1, 2, (M, r)) * g.choice([-1.0, 1.0], (M, r))).float()
    assert (T.view(torch.int32) & 0xFF).any()                # bits of the third part
    tok = g.integers(0, M, N)
    dY = torch.zeros(M, N)
    dY[tok, np.arange(N)] = 1.0
    B = normal(64, r, N, std=0.02)
    for need_dX in (True, False):
        _, _, dB = qlora.qlora_fp4_linear_bwd(dY.to(torch.bfloat16).cuda(), X.cuda(), T.cuda(), q, A.cuda(), B.cuda(),
                                              1.0, need_dX=need_dX)
        assert torch.equal(dB.cpu(), T[tok].t())
    # G[m, j] = B[j, n0] + B[j, n1] + B[j, n2], the columns in three different places of N
    bits = g.integers(128, 256, (3, r, N)).astype(np.float64)
    B = np.zeros((r, N))
    for i, cols in enumerate((slice(0, 40), slice(40, 100), slice(100, N))):
        B[:, cols] = bits[i][:, cols] * 2.0 ** (-7 - 8 * i)
    n = np.stack([g.integers(0, 40, M), g.integers(40, 100, M), g.integers(100, N, M)])
    dY = torch.zeros(M, N)
    for i in range(3):
        dY[np.arange(M), n[i]] = 1.0
    G = dY.double().numpy() @ B.T
    assert np.array_equal(G, G.astype(np.float32)) and (G.astype(np.float32).view(np.int32) & 0xFF).any()
    tok = g.integers(0, M, K)
    X = torch.zeros(M, K)
    X[tok, np.arange(K)] = 1.0
    for need_dX in (True, False):
        _, dA, _ = qlora.qlora_fp4_linear_bwd(dY.to(torch.bfloat16).cuda(), X.to(torch.bfloat16).cuda(), T.cuda(), q, A.cuda(),
                                              torch.from_numpy(B).to(torch.bfloat16).cuda(), 1.0, need_dX=need_dX)
        assert np.array_equal(dA.double().cpu().numpy(), G[tok])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gscale", [None, 0.37, 2.9e-4])
@pytest.mark.parametrize("M", [3, 90, 200, 1100])
def test_layer_on_any_gscale(M, gscale, fmt):
    """A weight whose gscale is no power of two, one in MXFP4 that has a gscale, one in NVFP4 without:
    the rank-r term is carried in its units."""
    N, K, r, scale = 160, 288, 16, 0.5
    W, A, B, X, dY = layer(71 + M, M, N, K, r, fmt)
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    g = None if gscale is None else torch.tensor([gscale], device="cuda")
    q.w.gscale = q.wt.gscale = g
    w, _ = F.quantize_weight(W.double().numpy(), fmt)
    w["g"] = np.ones(1) if g is None else g.double().cpu().numpy()
    Y, T = qlora.qlora_fp4_linear_fwd(X.cuda(), q, A.cuda(), B.cuda(), scale)
    dX, dA, dB = qlora.qlora_fp4_linear_bwd(dY.cuda(), X.cuda(), None, q, A.cuda(), B.cuda(), scale)
    A64, B64, X64, dY64 = (t.double().numpy() for t in (A, B, X, dY))
    Y64, T64 = F.linear_forward(X64, w, A64, B64, scale)
    dX64, dA64, dB64 = F.linear_backward(dY64, X64, w, A64, B64, scale)
    a = np.abs
    Wv, Xq, dYq = F.dequant(w), F.dequant(F.quantize(X64, fmt)), F.dequant(F.quantize(dY64, fmt))
    T_tol, G64 = (K / 16 + 80) * U * (a(X64) @ a(A64)), dY64 @ B64.T
    G_tol = (N / 16 + 80) * U * (a(dY64) @ a(B64).T)
    lora = lambda v, tol, m: abs(scale) * ((PAIR + 16 * U) * (a(v) @ a(m)) + tol @ a(m))
    within(T, T64, T_tol, "T")
    tol = product_tol(Xq, Wv) + lora(T64, T_tol, B64)
    within(Y, Y64, tol + BF16 * (a(Y64) + tol), "Y")
    tol = product_tol(dYq, Wv.T) + lora(G64, G_tol, A64.T)
    within(dX, dX64, tol + BF16 * (a(dX64) + tol), "dX")
    steps = (M / 16 + 80) * U
    within(dA, dA64, abs(scale) * (steps * (a(X64).T @ a(G64)) + a(X64).T @ G_tol), "dA")
    within(dB, dB64, abs(scale) * (steps * (a(T64).T @ a(dY64)) + T_tol.T @ a(dY64)), "dB")


@pytest.mark.parametrize("M,N,K,r", [(2, 96, 8256, 8), (100, 8256, 96, 64), (2600, 288, 4128, 64),
                                     (300, 12544, 160, 40), (17, 20000, 64, 16), (1300, 4128, 160, 16)])
def test_linear_schedules_in_mxfp4(M, N, K, r):
    check_layer(M, N, K, r, qlora.FP4_MXFP4)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r,scale", [
    (130, 32, 32, 8, 0.5), (1000, 64, 32, 64, 0.5), (200, 96, 416, 56, -2.0), (70, 96, 160, 48, -2.0),
    (3, 64, 64, 8, 0.0), (200, 64, 64, 8, 0.0)])
def test_linear_smallest_weights_ranks_and_scales(M, N, K, r, scale, fmt):
    check_layer(M, N, K, r, fmt, scale=scale)


@pytest.mark.parametrize("fmt", FMTS)
def test_codec_and_product_in_a_graph(fmt):
    """A weight laid out, activations quantized, their product and both read back, captured once and
    replayed on new inputs, and the same calls on a stream of their own."""
    M, N, K = 300, 160, 288
    def step(x, w):
        q, a = qlora.qlora_fp4_quantize_weight(w, fmt), qlora.qlora_fp4_quantize(x, fmt)
        return (qlora.qlora_fp4_matmul(a, q.w), qlora.qlora_fp4_matmul(a, q.w, torch.float32),
                qlora.qlora_fp4_dequant(a), qlora.qlora_fp4_dequant(q.w), qlora.qlora_fp4_dequant(q.wt, torch.float32))
    ins = [(normal(s, M, K).cuda(), normal(s + 1, N, K, std=0.02).cuda()) for s in (81, 83)]
    want = [step(*i) for i in ins]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = step(*ins[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    x, w = (t.clone() for t in ins[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, w)
    for i in (1, 0):
        x.copy_(ins[i][0]), w.copy_(ins[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("fmt", FMTS)
def test_weight_offsets_past_32_bits(fmt):
    """A weight of more than 2^32 values: its last rows and columns, in both orientations and as the
    operand of a product."""
    N, K = 65600, 65568
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    band, cols = normal(85, 64, K, std=0.02).cuda(), normal(86, N, 32, std=0.02).cuda()
    W[:32], W[-64:] = band[:32], band
    W[:, -32:] = cols
    W[0, 0] = 1.0                                            # the matrix's largest value, in every part below
    q = qlora.qlora_fp4_quantize_weight(W, fmt)
    part = W[-64:].clone()
    part[0, 0] = 1.0
    p = qlora.qlora_fp4_quantize_weight(part, fmt)
    assert torch.equal(q.w.codes[-32:], p.w.codes[-32:])
    right = W[:, -64:].clone()
    right[0, 0] = 1.0
    t = qlora.qlora_fp4_quantize_weight(right, fmt)
    assert torch.equal(q.wt.codes[-32:], t.wt.codes[-32:])
    if fmt == qlora.FP4_NVFP4:
        assert q.w.gscale.item() == p.w.gscale.item() == t.w.gscale.item()
    for M in (3, 200):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        x[:, -32:] = normal(87, M, 32).cuda()
        a = qlora.qlora_fp4_quantize(x, fmt)
        got = qlora.qlora_fp4_matmul(a, q.w, torch.float32)
        small = qlora.qlora_fp4_quantize(x[:, -64:].contiguous(), fmt)
        va, vb = (qlora.qlora_fp4_dequant(m, torch.float32).double() for m in (small, t.w))
        va[:, :32] = 0
        # all but 32 products are exact zeros: one group of 64 columns adds up, as in the small product
        want, mag = (va @ vb.t()), va.abs() @ vb.abs().t()
        assert ((got.double() - want).abs() <= 16 * U * mag).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_recomputes_T_of_a_large_batch(fmt):
    check_layer(1100, 160, 320, 16, fmt, saved_T=False)


@pytest.mark.parametrize("fmt", FMTS)
def test_gradients_against_differences(fmt):
    """The layer without its roundings is linear in A and in B and, on the 4-bit grid, in X: the
    difference of two outputs along a direction is the gradient's inner product with it. The
    outputs differenced here are the oracle's, the gradients the kernels'."""
    M, N, K, r, scale = 24, 64, 96, 8, 0.5
    q, (X, A, B, dY), (_, _, dX, dA, dB) = check_layer(M, N, K, r, fmt)
    Wv = qlora.qlora_fp4_dequant(q.w, torch.float32).double().cpu().numpy()
    dYq = qlora.qlora_fp4_dequant(qlora.qlora_fp4_quantize(dY, fmt), torch.float32).double().cpu().numpy()
    X, A, B, dY = (t.double().cpu().numpy() for t in (X, A, B, dY))
    f = lambda X_, A_, B_: np.sum((X_ @ Wv.T) * dYq) + scale * np.sum((X_ @ A_ @ B_) * dY)
    g = np.random.default_rng(3)
    for grad, i, rel in ((dX, 0, BF16), (dA, 1, 2.0 ** -14), (dB, 2, 2.0 ** -14)):
        grad = grad.double().cpu().numpy()
        V = g.normal(0, 1, grad.shape)
        hi, lo = [X, A, B], [X, A, B]
        hi[i], lo[i] = hi[i] + V, lo[i] - V
        assert abs((f(*hi) - f(*lo)) / 2 - np.sum(grad * V)) <= rel * np.sum(np.abs(grad * V)) + 1e-6


def test_empty_batch_and_partial_outputs():
    W, A, B, X, dY = (t.cuda() for t in layer(9, 20, 64, 96, 8, 1))
    q = qlora.qlora_fp4_quantize_weight(W)
    Y, T = qlora.qlora_fp4_linear_fwd(X[:0], q, A, B, 1.0)
    assert Y.shape == (0, 64) and T.shape == (0, 8)
    dX, dA, dB = qlora.qlora_fp4_linear_bwd(dY[:0], X[:0], None, q, A, B, 1.0)
    assert dX.shape == (0, 96) and not dA.any() and not dB.any()
    full = qlora.qlora_fp4_linear_bwd(dY, X, None, q, A, B, 1.0)
    none, dA, dB = qlora.qlora_fp4_linear_bwd(dY, X, None, q, A, B, 1.0, need_dX=False)
    assert none is None and torch.equal(dA, full[1]) and torch.equal(dB, full[2])
    Y1, none = qlora.qlora_fp4_linear_fwd(X, q, A, B, 1.0, save_T=False)
    assert none is None and torch.equal(Y1, qlora.qlora_fp4_linear_fwd(X, q, A, B, 1.0)[0])


def test_layer_after_its_weight_in_one_stream():
    """The forward fetches its weight ahead of its tokens, but never before the kernels that
    wrote it: laying a new weight out into the same storage and using it at once, repeatedly."""
    M, N, K, r = 4, 2048, 1024, 8
    W, A, B, X, dY = (t.cuda() for t in layer(31, M, N, K, r, 1))
    ws = [W, W.flip(0).contiguous(), W * 2]
    want = []
    for w in ws:
        q = qlora.qlora_fp4_quantize_weight(w)
        torch.cuda.synchronize()
        y, t = qlora.qlora_fp4_linear_fwd(X, q, A, B, 0.5)
        want.append((y, qlora.qlora_fp4_linear_bwd(dY, X, t, q, A, B, 0.5)[0]))
        torch.cuda.synchronize()
    q = qlora.qlora_fp4_quantize_weight(W)
    for i in range(12):
        qlora.qlora_fp4_quantize_weight(ws[i % 3], out=q)
        y, t = qlora.qlora_fp4_linear_fwd(X, q, A, B, 0.5)
        dx = qlora.qlora_fp4_linear_bwd(dY, X, t, q, A, B, 0.5)[0]
        assert torch.equal(y, want[i % 3][0]) and torch.equal(dx, want[i % 3][1])


def test_caller_buffers_and_refusals_on_the_device():
    M, N, K, r = 20, 64, 96, 8
    W, A, B, X, dY = (t.cuda() for t in layer(41, M, N, K, r, 1))
    q = qlora.qlora_fp4_quantize_weight(W)
    Y, T = qlora.qlora_fp4_linear_fwd(X, q, A, B, 1.0)
    ws = torch.empty(qlora.qlora_fp4_linear_fwd_workspace_size(M, N, K, r), dtype=torch.uint8, device="cuda")
    Y1, T1 = torch.empty_like(Y), torch.empty_like(T)
    got = qlora.qlora_fp4_linear_fwd(X, q, A, B, 1.0, Y=Y1, T=T1, workspace=ws)
    assert got[0] is Y1 or got[0].data_ptr() == Y1.data_ptr()
    assert torch.equal(Y1, Y) and torch.equal(T1, T)
    with pytest.raises(qlora.QLoraError):
        qlora.qlora_fp4_linear_fwd(X, q, A, B, 1.0, workspace=ws[:16])
    with pytest.raises(qlora.QLoraError):                      # r = 12
        qlora.qlora_fp4_linear_fwd(X, q, torch.zeros(K, 12, dtype=torch.bfloat16, device="cuda"),
                                   torch.zeros(12, N, dtype=torch.bfloat16, device="cuda"), 1.0)
    with pytest.raises(qlora.QLoraError):                      # a misaligned address
        qlora.qlora_fp4_quantize(torch.zeros(33, device="cuda")[1:].view(1, 32))
    with pytest.raises(ValueError):
        qlora.qlora_fp4_linear_fwd(X[:, :64].contiguous(), q, A, B, 1.0)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_linear_fwd(X, q, A.cpu(), B, 1.0)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_quantize(W.t())
    with pytest.raises(TypeError):
        qlora.qlora_fp4_quantize(W.half())
    with pytest.raises(TypeError):
        qlora.qlora_fp4_dequant(q.w, torch.float16)
    short = qlora.FP4Matrix(q.w.codes, q.w.scales[:512], q.w.gscale, 256, K, 1)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_dequant(short)
    with pytest.raises(ValueError):
        qlora.qlora_fp4_linear_bwd(dY, X, T, qlora.FP4Weight(q.w), A, B, 1.0)
    mx = qlora.qlora_fp4_quantize(X, qlora.FP4_MXFP4)
    with pytest.raises(qlora.QLoraError):
        qlora.qlora_fp4_matmul(mx, q.w)


@pytest.mark.parametrize("M", [20, 200])
def test_backward_into_its_inputs_is_refused_and_beside_them_is_not(M):
    W, A, B, X, dY = (t.cuda() for t in layer(43, M, 96, 96, 8, 1))
    q = qlora.qlora_fp4_quantize_weight(W)
    for dX in (X, dY):
        with pytest.raises(qlora.QLoraError) as e:
            qlora.qlora_fp4_linear_bwd(dY, X, None, q, A, B, 1.0, dX=dX)
        assert e.value.status == 1
    want = qlora.qlora_fp4_linear_bwd(dY, X, None, q, A, B, 1.0)
    both = torch.cat([X, torch.zeros_like(X), dY])           # dX between X and dY, all touching
    got = qlora.qlora_fp4_linear_bwd(both[2 * M:], both[:M], None, q, A, B, 1.0, dX=both[M:2 * M])
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(both[:M], X) and torch.equal(both[2 * M:], dY)


def test_streams_and_graphs():
    """The same bits on another stream, in a captured and replayed graph with new inputs, and
    from two streams at once."""
    for M in (3, 200):
        W, A, B, X, dY = (t.cuda() for t in layer(11, M, 256, 320, 16, 1))
        q = qlora.qlora_fp4_quantize_weight(W)

        def step(x, dy):
            y, t = qlora.qlora_fp4_linear_fwd(x, q, A, B, 0.5)
            return (y, t) + qlora.qlora_fp4_linear_bwd(dy, x, t, q, A, B, 0.5)
        want, X2, dY2 = step(X, dY), X.flip(0).contiguous(), dY.flip(0).contiguous()
        want2 = step(X2, dY2)
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = {}
        for _ in range(3):
            for name, s, args in (("a", s1, (X, dY)), ("b", s2, (X2, dY2))):
                with torch.cuda.stream(s):
                    got[name] = step(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got["a"], want))
        assert all(torch.equal(x, y) for x, y in zip(got["b"], want2))
        bx, bdy = X.clone(), dY.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(bx, bdy)
        for src, ref in (((X2, dY2), want2), ((X, dY), want)):
            bx.copy_(src[0]), bdy.copy_(src[1])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, ref))


@pytest.mark.parametrize("fmt", FMTS)
def test_large_batch_on_streams_and_in_graphs(fmt):
    """A batch whose quantizer runs beside the rank-r product: against the formulas, on two
    streams at once, in a replayed graph, and in a graph captured by a thread that has made no
    call before (which has no side stream and runs everything in order)."""
    import threading
    check_layer(1100, 96, 160, 16, fmt)
    W, A, B, X, dY = (t.cuda() for t in layer(13, 1100, 96, 160, 16, fmt))
    q = qlora.qlora_fp4_quantize_weight(W, fmt)

    def step(x, dy):
        y, t = qlora.qlora_fp4_linear_fwd(x, q, A, B, 0.5)
        return (y, t) + qlora.qlora_fp4_linear_bwd(dy, x, t, q, A, B, 0.5)
    X2, dY2 = X.flip(0).contiguous(), dY.flip(0).contiguous()
    want, want2 = step(X, dY), step(X2, dY2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = {}
    for _ in range(3):
        for name, s, args in (("a", s1, (X, dY)), ("b", s2, (X2, dY2))):
            with torch.cuda.stream(s):
                got[name] = step(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got["a"], want))
    assert all(torch.equal(x, y) for x, y in zip(got["b"], want2))
    bx, bdy = X.clone(), dY.clone()
    made = []

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(bx, bdy)
        made.append((graph, out))
    capture()
    t = threading.Thread(target=capture)
    t.start()
    t.join()
    assert len(made) == 2
    for graph, out in made:
        for src, ref in (((X2, dY2), want2), ((X, dY), want)):
            bx.copy_(src[0]), bdy.copy_(src[1])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, ref))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [600, 4200])
def test_quantizer_on_and_off_the_side_stream(M, fmt):
    """Beside the rank-r product (in a capture, and in an eager call of many tokens) or in order: the formulas,
    and the same bits in eager calls, on two streams at once and in a replayed graph."""
    check_layer(M, 96, 160, 16, fmt)
    W, A, B, X, dY = (t.cuda() for t in layer(19, M, 96, 160, 16, fmt))
    q = qlora.qlora_fp4_quantize_weight(W, fmt)

    def step(x, dy):
        y, t = qlora.qlora_fp4_linear_fwd(x, q, A, B, 0.5)
        return (y, t) + qlora.qlora_fp4_linear_bwd(dy, x, t, q, A, B, 0.5)
    ins = [(X, dY), (X.flip(0).contiguous(), dY.flip(0).contiguous())]
    want = [step(*i) for i in ins]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = step(*ins[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))
    bx, bdy = X.clone(), dY.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(bx, bdy)
    for i in (1, 0, 1):
        bx.copy_(ins[i][0]), bdy.copy_(ins[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[i]))


@pytest.mark.parametrize("M", [2, 150, 700, 1100])
def test_calls_back_to_back_on_one_buffer(M):
    """Kernels of a call start before their predecessors end: the input rewritten between calls
    without a synchronisation, the workspace and the outputs' memory reused by every call."""
    W, A, B, X, dY = (t.cuda() for t in layer(17, M, 512, 1024, 16, 1))
    q = qlora.qlora_fp4_quantize_weight(W)
    xs = [X, X.flip(0).contiguous(), (X * 3).contiguous()]
    ws = torch.empty(max(qlora.qlora_fp4_linear_fwd_workspace_size(M, 512, 1024, 16),
                         qlora.qlora_fp4_linear_bwd_workspace_size(M, 512, 1024, 16)),
                     dtype=torch.uint8, device="cuda")
    want = []
    for x in xs:
        y, t = qlora.qlora_fp4_linear_fwd(x, q, A, B, 0.5)
        want.append((y, t) + qlora.qlora_fp4_linear_bwd(dY, x, t, q, A, B, 0.5))
        torch.cuda.synchronize()
    buf, got = torch.empty_like(X), []
    for i in range(30):
        buf.copy_(xs[i % 3])
        y, t = qlora.qlora_fp4_linear_fwd(buf, q, A, B, 0.5, workspace=ws)
        got.append((y, t) + qlora.qlora_fp4_linear_bwd(dY, buf, t, q, A, B, 0.5, workspace=ws))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 3])), i


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [7, 128, 136, 600, 4200])
def test_one_tensor_in_two_places(M, fmt):
    """A matrix times its own transpose, one tensor as X and as dY, and a forward over its own input."""
    N = K = 160
    W, A, B, X, _ = (t.cuda() for t in layer(91, M, N, K, 16, fmt))
    q, a = qlora.qlora_fp4_quantize_weight(W, fmt), qlora.qlora_fp4_quantize(X, fmt)
    if M % 8 == 0:
        copy = qlora.FP4Matrix(a.codes.clone(), a.scales.clone(), a.gscale, M, K, fmt)
        p = qlora.qlora_fp4_matmul(a, a, torch.float32)
        assert torch.equal(p, qlora.qlora_fp4_matmul(a, copy, torch.float32))
    Y, T = qlora.qlora_fp4_linear_fwd(X, q, A, B, 0.5)
    want = qlora.qlora_fp4_linear_bwd(X.clone(), X, T, q, A, B, 0.5)
    got = qlora.qlora_fp4_linear_bwd(X, X, T, q, A, B, 0.5)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    over = X.clone()
    Y1, T1 = qlora.qlora_fp4_linear_fwd(over, q, A, B, 0.5, Y=over)
    assert torch.equal(over, Y) and torch.equal(T1, T)


@pytest.mark.parametrize("fmt", FMTS)
def test_two_host_threads(fmt):
    """Calls of two threads, each on its own stream, on one weight."""
    import threading
    W, A, B, X, dY = (t.cuda() for t in layer(93, 4200, 96, 160, 16, fmt))
    q = qlora.qlora_fp4_quantize_weight(W, fmt)
    sizes, bad, done = (5, 100, 300, 1100, 4200), [], []

    def step(M):
        y, t = qlora.qlora_fp4_linear_fwd(X[:M], q, A, B, 0.5)
        return (y, t) + qlora.qlora_fp4_linear_bwd(dY[:M], X[:M], t, q, A, B, 0.5)
    want = {M: step(M) for M in sizes}
    torch.cuda.synchronize()

    def work(order):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(20):
                for M in order:
                    got = step(M)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want[M])):
                        bad.append((i, M))
        done.append(order)
    threads = [threading.Thread(target=work, args=(o,)) for o in (sizes, sizes[::-1])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(done) == 2 and not bad


def test_training_step_on_a_microscaled_weight():
    """The operators together: lay the weight out, forward, backward, optimizer step, and the
    next forward on the updated adapter."""
    from oracle import adamw_oracle as AW
    W, A, B, X, dY = layer(21, 96, 128, 160, 8, 1)
    scale = 0.25
    q = qlora.qlora_fp4_quantize_weight(W.cuda())
    p0 = torch.cat([A.reshape(-1), B.reshape(-1)]).float()
    p, pb = p0.cuda(), torch.empty(p0.numel(), dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(qlora.qlora_adamw_state_bytes(p.numel(), 8), dtype=torch.uint8, device="cuda")
    Y, T = qlora.qlora_fp4_linear_fwd(X.cuda(), q, A.cuda(), B.cuda(), scale)
    _, dA, dB = qlora.qlora_fp4_linear_bwd(dY.cuda(), X.cuda(), T, q, A.cuda(), B.cuda(), scale)
    g = torch.cat([dA.reshape(-1), dB.reshape(-1)])
    qlora.qlora_adamw_step(p, g, state, 1, lr=1e-2, p_bf16=pb)
    A1, B1 = pb[:160 * 8].view(160, 8), pb[160 * 8:].view(8, 128)
    Y1, _ = qlora.qlora_fp4_linear_fwd(X.cuda(), q, A1, B1, scale)
    want, _, _ = AW.adamw_step_8bit(p0.numpy(), g.cpu().numpy(), AW.zero_state_8bit(p0.numel()), lr=1e-2,
                                    beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    assert np.array_equal(p.cpu().numpy(), want)
    w, _ = F.quantize_weight(W.double().numpy(), 1)
    Y64, T64 = F.linear_forward(X.double().numpy(), w, A1.double().cpu().numpy(),
                                B1.double().cpu().numpy(), scale)
    tol = 1e-4 * np.abs(T64) @ np.abs(B1.double().cpu().numpy()) + 1e-4 * np.abs(X.double().numpy()) @ np.abs(F.dequant(w)).T
    within(Y1, Y64, tol + BF16 * (np.abs(Y64) + tol), "Y after the step")
    assert not torch.equal(Y, Y1)
