"""GPU parity of the microscaled 4-bit codec: codes, scales and gscale bit for bit against the
oracle, values read back bit for bit."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_unpack_b200 import qlora
from oracle import fp4_oracle as F
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

FMTS = [qlora.FP4_MXFP4, qlora.FP4_NVFP4]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def draw(rows, cols, seed=0, spread=6):
    g = np.random.default_rng(seed)
    x = g.normal(0, 1, (rows, cols)) * 2.0 ** g.integers(-spread, spread + 1, (rows, cols // 16)).repeat(16, 1)
    return torch.from_numpy(x).float()


def same_matrix(q, ref, what=""):
    assert np.array_equal(q.codes.cpu().numpy(), F.pack(ref["codes"])), what
    R, B = ref["bytes"].shape
    assert np.array_equal(q.scales.cpu().numpy()[F.scale_index(R, B)], ref["bytes"]), what
    if q.fmt == qlora.FP4_NVFP4:
        assert np.array_equal(q.gscale.cpu().numpy().astype(np.float64), ref["g"]), what


def check_rows(x, fmt):
    q = qlora.qlora_fp4_quantize(x.cuda(), fmt)
    ref = F.quantize(x.double().numpy(), fmt)
    same_matrix(q, ref)
    # blocks past the last column inside the last scale tile hold 0
    B, s = ref["bytes"].shape[1], q.scales.cpu().numpy()
    pad = F.scale_index(x.shape[0], -(-B // 4) * 4)[:, B:]
    assert not s[pad].any()
    for dtype in DTYPES:
        got = qlora.qlora_fp4_dequant(q, dtype).cpu()
        want = torch.from_numpy(F.dequant(ref)).float().to(dtype)
        assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))
    return q


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 64), (257, 544), (16, 4160), (5, 11008),
                                       (2, 16384), (2, 16416), (1, 40000), (300, 4096)])
def test_rows(rows, cols, dtype, fmt):
    check_rows(draw(rows, cols, rows + cols).to(dtype), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_special_values(fmt):
    x = draw(40, 192, 3)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5], x[3, 100], x[4, 191] = float("nan"), float("inf"), -float("inf")
    x[5] = float("nan")
    x[6] *= 2.0 ** -120          # maxima near the smallest normal numbers
    x[7] = 2.0 ** -140
    x[8] *= 2.0 ** 110
    x[9] = 3.0e38
    x[10, 16:] = 0.0
    x[11] *= 1e-3
    x[11, 0] = 1e6               # blocks far below the row's top: scales down to 0
    for i, m in enumerate(F.E2M1[1:]):
        x[12 + i] = torch.from_numpy(np.resize([m, -m, 6.0], 192)).float()
    check_rows(x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_rounding_borders(fmt):
    """Every border of the E2M1 and E4M3 roundings, and the fp32 numbers beside it."""
    mid = torch.from_numpy((F.E2M1[1:] + F.E2M1[:-1]) / 2).float()
    mid = torch.cat([mid, torch.nextafter(mid, torch.tensor(9.0)), torch.nextafter(mid, torch.tensor(0.0))])
    b = F.BLOCK[fmt]
    rows = []
    t = torch.from_numpy(F.e4m3_table()).float()
    for c in t[1:]:
        # a block whose scale is exactly c: its largest value 6 c (7.9 c would do for powers of two)
        blk = torch.zeros(2, b)
        blk[:, 0] = 6 * c
        blk[0, 1:1 + min(b - 1, 21)] = (mid * c)[: min(b - 1, 21)]
        blk[1, 1:1 + min(b - 1, 21)] = -(mid * c)[-min(b - 1, 21):]
        rows.append(blk.reshape(-1))
    x = torch.stack(rows)
    x = torch.cat([x, torch.zeros(len(rows), -(2 * b + 16) % 32 + 16)], 1)
    x[:, -1] = 2688.0            # gscale 1
    check_rows(x, fmt)
    tm = (t[1:] + t[:-1]) / 2    # scales on the borders of E4M3
    y = torch.zeros(3 * 126, 32)
    y[:, 0] = torch.cat([6 * tm, torch.nextafter(6 * tm, torch.tensor(9e9)), torch.nextafter(6 * tm, torch.tensor(0.0))])
    y[:, 16] = 2688.0
    check_rows(y, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_do_not_depend_on_each_other(fmt):
    x = draw(70, 1024, 8).cuda()
    whole = qlora.qlora_fp4_dequant(qlora.qlora_fp4_quantize(x, fmt))
    part = qlora.qlora_fp4_dequant(qlora.qlora_fp4_quantize(x[33:34].contiguous(), fmt))
    assert torch.equal(whole[33:34], part)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(32, 32), (96, 160), (160, 96), (256, 416), (1056, 224), (4096, 64)])
def test_weight(n, k, dtype, fmt):
    W = (draw(n, k, n + k, spread=3) * 0.02).to(dtype)
    W[: min(n, 32), :32] = 0.0
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    w, wt = F.quantize_weight(W.double().numpy(), fmt)
    same_matrix(q.w, w, "w")
    same_matrix(q.wt, wt, "wt")
    for m, ref in ((q.w, w), (q.wt, wt)):
        B = ref["bytes"].shape[1]
        pad = F.scale_index(ref["bytes"].shape[0], -(-B // 4) * 4)[:, B:]
        assert not m.scales.cpu().numpy()[pad].any()
    only = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt, transposed=False)
    assert only.wt is None and torch.equal(only.w.codes, q.w.codes)
    assert torch.equal(qlora.qlora_fp4_dequant(q.w), qlora.qlora_fp4_dequant(q.wt).t())


@pytest.mark.parametrize("fmt", FMTS)
def test_weight_special_values(fmt):
    W = draw(128, 128, 5)
    W[40, 70] = float("nan")
    W[100, 3] = float("inf")
    W[64:96, 64:96] = 0.0
    q = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
    w, wt = F.quantize_weight(W.double().numpy(), fmt)
    same_matrix(q.w, w)
    same_matrix(q.wt, wt)
    zero = qlora.qlora_fp4_quantize_weight(torch.zeros(64, 64, device="cuda"), fmt)
    assert not qlora.qlora_fp4_dequant(zero.w).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dequant_of_any_storage(fmt, dtype):
    """Every scale byte and code, gscales that are no powers of two, one and one per row."""
    g = np.random.default_rng(6)
    R, C = 300, 32 * 37
    top = 256 if fmt == F.MX else 128
    ref = {"codes": g.integers(0, 16, (R, C)).astype(np.uint8),
           "bytes": g.integers(0, top, (R, C // F.BLOCK[fmt])).astype(np.uint8), "fmt": fmt}
    for gs in (None, g.uniform(0.1, 3, 1), g.uniform(0.1, 3, R)):
        gs = None if gs is None else gs.astype(np.float32)
        q = qlora.FP4Matrix(torch.from_numpy(F.pack(ref["codes"])).cuda(),
                            torch.from_numpy(F.store_scales(ref["bytes"])).cuda(),
                            None if gs is None else torch.from_numpy(gs).cuda(), R, C, fmt)
        got = qlora.qlora_fp4_dequant(q, dtype).cpu()
        v32 = torch.from_numpy(F.dequant({**ref, "g": np.ones(1)})).float()  # exact, or inf past fp32
        want = (v32 if gs is None else v32 * torch.from_numpy(gs).view(-1, 1)).to(dtype)
        assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


def test_outputs_stay_inside_their_buffers():
    """Quantizing and reading back write nothing outside their outputs."""
    for fmt in FMTS:
        x = draw(37, 96, 9).cuda()
        big = torch.full((37 * 48 + 64,), 0xAB, dtype=torch.uint8, device="cuda")
        q = qlora.FP4Matrix.empty(37, 96, fmt)
        q.codes = big[32:32 + 37 * 48].view(37, 48)
        qlora.qlora_fp4_quantize(x, fmt, out=q)
        assert (big[:32] == 0xAB).all() and (big[-32:] == 0xAB).all()
        out = torch.full((37 * 96 + 64,), 7.0, device="cuda")
        qlora.qlora_fp4_dequant(q, torch.float32, out=out[32:-32].view(37, 96))
        assert (out[:32] == 7).all() and (out[-32:] == 7).all()


def test_empty():
    x = torch.zeros(0, 64, device="cuda")
    for fmt in FMTS:
        q = qlora.qlora_fp4_quantize(x, fmt)
        assert qlora.qlora_fp4_dequant(q).shape == (0, 64)


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """A matrix of more than 2^32 bytes: its last rows, whose offsets need 64 bits."""
    rows, cols = 70001, 32768                      # 2.3e9 bf16 values
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    pick = [0, 32767, 32768, 65535, 65536, 69999, 70000]
    x.zero_()
    for i in pick:
        x[i] = torch.randn(cols, generator=g, device="cuda").to(torch.bfloat16) * 2.0 ** (i % 5)
    q = qlora.qlora_fp4_quantize(x, fmt)
    v = qlora.qlora_fp4_dequant(q)
    ref = F.quantize(x[pick].double().cpu().numpy(), fmt)
    want = torch.from_numpy(F.dequant(ref)).to(torch.bfloat16)
    assert torch.equal(v[pick].cpu(), want)
    for i, row in enumerate(pick):
        assert np.array_equal(q.codes[row].cpu().numpy(), F.pack(ref["codes"][i:i + 1])[0])
    # and as the operand of a product: the last rows' tokens
    w = qlora.qlora_fp4_quantize(torch.eye(32, cols, device="cuda"), fmt)
    one = F.dequant(F.quantize(np.eye(1, 32), fmt))[0, 0]  # what the format stores for 1
    out = qlora.qlora_fp4_matmul(q, w, torch.float32)
    assert torch.equal(out[pick].cpu(), want[:, :32].float() * float(one))  # exact products
    assert not out[1:32767].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_signs_of_zeros(fmt, dtype):
    """A negative zero, and a negative value that rounds to zero, keep the sign bit."""
    x = draw(64, 128, 12, spread=1)
    x[:, ::3] = -0.0
    x[:, 1::3] *= 2.0 ** -12
    x[:, 2::6] = 0.0
    x = x.to(dtype)
    q = check_rows(x, fmt)
    assert (q.codes.cpu() & 15 == 8).any()
    w = qlora.qlora_fp4_quantize_weight(x.cuda(), fmt)
    ref, ref_t = F.quantize_weight(x.double().numpy(), fmt)
    same_matrix(w.w, ref)
    same_matrix(w.wt, ref_t)


@pytest.mark.parametrize("fmt", FMTS)
def test_tiny_and_huge_rows(fmt):
    """gscales over their whole range, 2^-126 to 2^116, with blocks far below each row's top, and
    fp32 values beside the borders."""
    g = np.random.default_rng(31)
    e = np.arange(-126, 118, 2)
    x = torch.from_numpy(g.normal(0, 1, (e.size, 128))).float()
    x[:, 64:] *= 2.0 ** -6
    x[:, 0] = 2000.0
    x = (x.double() * torch.from_numpy(2.0 ** e.astype(np.float64))[:, None]).float()
    check_rows(x, fmt)
    for row in (0, 10, 17, 18, 19, 60, e.size - 1):
        W = x[row].repeat(32, 1)[:, :32].contiguous()
        w = qlora.qlora_fp4_quantize_weight(W.cuda(), fmt)
        same_matrix(w.w, F.quantize_weight(W.double().numpy(), fmt)[0], row)


def test_refusals_name_their_reason():
    """An unknown format is an invalid argument (1), columns or rows that are no multiple a shape (2)."""
    def status(fn, *args, **kw):
        with pytest.raises(qlora.QLoraError) as e:
            fn(*args, **kw)
        return e.value.status
    x, odd = torch.zeros(64, 64, device="cuda"), torch.zeros(64, 48, device="cuda")
    for fn in (qlora.qlora_fp4_quantize, qlora.qlora_fp4_quantize_weight):
        assert status(fn, x, 7) == 1 and status(fn, x, -1) == 1
        assert status(fn, odd) == 2 and status(fn, odd[:, :0].contiguous()) == 2
    assert status(qlora.qlora_fp4_quantize, x[:0], 7) == 1
    assert status(qlora.qlora_fp4_quantize_weight, x[:40]) == 2
    assert status(qlora.qlora_fp4_quantize_weight, x[:40], transposed=False) == 2
    assert status(qlora.qlora_fp4_quantize_weight, x[:0]) == 2
