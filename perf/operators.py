"""The microscaled 4-bit floating-point operators: cases, plain forms and 64-bit results.

Two storage formats of a matrix whose blocks run along its columns:
  MXFP4: blocks of 32 E2M1 values, one power of two (E8M0) per block;
  NVFP4: blocks of 16 E2M1 values, one E4M3 scale per block, and one fp32 power of two
         (gscale) per row (activations) or per matrix (weights).
Codes: uint8 [rows, cols / 2], the even column in the low nibble. Scales: uint8, tiles of
128 rows x 4 blocks of 512 bytes each, ordered by row tile, then block tile; inside a tile the
byte of (row, block) is (row % 32) * 16 + (row // 32) * 4 + block.
"""
import math

import torch

own = False

MX, NV = "mxfp4", "nvfp4"
BLOCK = {MX: 32, NV: 16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's activations of a small batch, before a 4096-wide linear
        {"name": "quantize_nv_16x4096", "op": "quantize", "fmt": NV, "M": 16, "K": 4096, "dtype": "bf16"},
        # a prefill's MLP activations
        {"name": "quantize_nv_8192x11008", "op": "quantize", "fmt": NV, "M": 8192, "K": 11008, "dtype": "bf16"},
        # laying out a 7B attention weight for training (both orientations), from fp32
        {"name": "weight_nv_4096x4096", "op": "weight", "fmt": NV, "N": 4096, "K": 4096, "dtype": "f32"},
        # laying out a 7B MLP weight, power-of-two scales
        {"name": "weight_mx_11008x4096", "op": "weight", "fmt": MX, "N": 11008, "K": 4096, "dtype": "bf16"},
        # reading a small shard of a weight back, odd row count
        {"name": "dequant_nv_777x1056", "op": "dequant", "fmt": NV, "M": 777, "K": 1056, "dtype": "f32"},
        # exporting a 65B MLP weight to bf16
        {"name": "dequant_mx_8192x22016", "op": "dequant", "fmt": MX, "M": 8192, "K": 22016, "dtype": "bf16"},
        # a ragged batch against a ragged weight: no size a multiple of the tiles
        {"name": "matmul_mx_333x1000x1056", "op": "matmul", "fmt": MX, "M": 333, "N": 1000, "K": 1056, "dtype": "f32"},
        # the 65B attention linear over a long prompt: the matrix-bound end
        {"name": "matmul_nv_8192x8192x8192", "op": "matmul", "fmt": NV, "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16"},
        # one token through the 7B gate linear: weight streaming and latency
        {"name": "fwd_nv_1x11008x4096", "op": "fwd", "fmt": NV, "M": 1, "N": 11008, "K": 4096, "r": 16},
        # the 7B gate linear of a training step
        {"name": "fwd_nv_4096x11008x4096", "op": "fwd", "fmt": NV, "M": 4096, "N": 11008, "K": 4096, "r": 64},
        # gradients of a short, ragged training batch
        {"name": "bwd_mx_257x4096x4096", "op": "bwd", "fmt": MX, "M": 257, "N": 4096, "K": 4096, "r": 16},
        # gradients of the 7B gate linear of a training step
        {"name": "bwd_nv_4096x11008x4096", "op": "bwd", "fmt": NV, "M": 4096, "N": 11008, "K": 4096, "r": 64},
    ]


def _size(rng, lo, hi, step):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["quantize", "weight", "dequant", "matmul", "fwd", "bwd"])
    case = {"op": op, "fmt": rng.choice([MX, NV])}
    K = _size(rng, 32, 12288, 32)
    if op in ("quantize", "dequant"):
        return {**case, "M": _size(rng, 1, 8192, 1), "K": K, "dtype": rng.choice(["bf16", "f32"])}
    if op == "weight":
        return {**case, "N": _size(rng, 32, 12288, 32), "K": K, "dtype": rng.choice(["bf16", "f32"])}
    if op == "matmul":
        return {**case, "M": _size(rng, 1, 8192, 1), "N": _size(rng, 8, 8192, 8), "K": min(K, 8192),
                "dtype": rng.choice(["bf16", "f32"])}
    M, N = _size(rng, 1, 8192, 1), _size(rng, 32, 12288, 32)
    while M * N * K > 4096 * 11008 * 4096:  # the largest listed training step
        M = (M + 1) // 2
    return {**case, "M": M, "N": N, "K": K, "r": 8 * rng.randint(1, 8)}


# ------------------------------------------------------------------ storage, laid out with torch
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tile(s):
    """Scale bytes [rows, blocks] in the stored order."""
    R, B = s.shape
    p = torch.zeros(-(-R // 128) * 128, -(-B // 4) * 4, dtype=torch.uint8, device=s.device)
    p[:R, :B] = s
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(t, R, B):
    rt, bt = -(-R // 128), -(-B // 4)
    return t.view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)[:R, :B]


# ------------------------------------------------------------------ plain forms
def _round_e2m1(y):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, 6 at most), signed."""
    a = y.abs()
    f = y.dtype
    v = 0.5 * ((a > 0.25).to(f) + (a >= 0.75).to(f) + (a > 1.25).to(f) + (a >= 1.75).to(f))
    v = v + (a > 2.5).to(f) + (a >= 3.5).to(f) + 2 * (a > 5.0).to(f)
    return torch.copysign(v, y)


def _pow2(e):
    return torch.exp2(e.to(torch.float64)).to(torch.float32)


def _plain_scales(amax, fmt, gmax):
    """(scale values, gscale) of block maxima `amax`; gmax: the maximum each gscale covers,
    shaped to broadcast against amax."""
    if fmt == MX:
        e = torch.frexp(amax)[1] - 3
        e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
        return _pow2(e), None
    m, e = torch.frexp(gmax.double() / 2688.0)
    e = torch.where(m > 0.5, e, e - 1).clamp(-126, 127)
    g = torch.where(gmax > 0, _pow2(e), torch.ones_like(gmax))
    c = (amax / g / 6.0).to(torch.float8_e4m3fn).float()
    return c, g


def _plain_values(x, s, g):
    """x on the 4-bit grid of its scales, as fp32 values."""
    y = x if g is None else x / g
    q = torch.where(s > 0, _round_e2m1(y / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(y)) * s
    return q if g is None else q * g


def _plain_quantize(X, fmt):
    R, C = X.shape
    x = X.float().view(R, C // BLOCK[fmt], BLOCK[fmt])
    amax = x.abs().amax(2, keepdim=True)
    s, g = _plain_scales(amax, fmt, amax.amax(1, keepdim=True))
    return _plain_values(x, s, g).view(R, C)


def _plain_weight(W, fmt):
    """(values [N, K], scale per square block [N/b, K/b], gscale)."""
    b = BLOCK[fmt]
    N, K = W.shape
    x = W.float().view(N // b, b, K // b, b)
    amax = x.abs().amax((1, 3), keepdim=True)
    s, g = _plain_scales(amax, fmt, amax.amax().view(1, 1, 1, 1))
    return _plain_values(x, s, g).view(N, K), s.view(N // b, K // b), g


def _decode(codes, scales, g, fmt):
    """Values of a stored matrix, fp32."""
    R, C = codes.shape[0], codes.shape[1] * 2
    lev = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6.], device=codes.device)
    lev = torch.cat([lev, -lev])
    v = torch.stack([lev[(codes & 15).int()], lev[(codes >> 4).int()]], 2).view(R, -1, BLOCK[fmt])
    s = _untile(scales, R, C // BLOCK[fmt])
    s = _pow2(s.int() - 127) if fmt == MX else s.view(torch.float8_e4m3fn).float()
    v = (v * s.unsqueeze(2)).view(R, C)
    return v if g is None else v * g.view(-1, 1)


# ------------------------------------------------------------------ inputs
def _activations(gen, M, K, dtype):
    """Unit activations with a few strong channels; in larger batches the last rows are padding."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x[:, :: max(1, K // 8)] *= 12.0
    if M >= 32:
        x[M - M // 16:] = 0.0
    return x.to(dtype)


def _store(values, scale_values, g, fmt):
    """Stored form of values that lie on the grid of scale_values [R, blocks]."""
    R, C = values.shape
    s = scale_values.repeat_interleave(BLOCK[fmt], 1)
    y = values / torch.where(s > 0, s, torch.ones_like(s))
    if g is not None:
        y = y / g.view(-1, 1)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    code = torch.bucketize(y.abs(), mid).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    if fmt == MX:
        s8 = (torch.frexp(scale_values)[1] + 126).to(torch.uint8)
    else:
        s8 = scale_values.to(torch.float8_e4m3fn).view(torch.uint8)
    return {"codes": codes, "scales": _tile(s8), "g": None if g is None else g.reshape(-1).contiguous()}


def _stored_rows(x, fmt):
    R, C = x.shape
    v = x.float().view(R, -1, BLOCK[fmt])
    amax = v.abs().amax(2, keepdim=True)
    s, g = _plain_scales(amax, fmt, amax.amax(1, keepdim=True))
    return _store(_plain_values(v, s, g).view(R, C), s.view(R, -1), g, fmt)


def _stored_weight(W, fmt):
    v, s, g = _plain_weight(W, fmt)
    b = BLOCK[fmt]
    return {"w": _store(v, s.repeat_interleave(b, 0), g, fmt),
            "wt": _store(v.t().contiguous(), s.t().repeat_interleave(b, 0), g, fmt)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, fmt = case["op"], case["fmt"]
    st = {"case": dict(case)}

    def randn(*shape, std, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    if op == "quantize":
        st["X"] = _activations(gen, case["M"], case["K"], _DT[case["dtype"]])
    elif op == "weight":
        st["W"] = randn(case["N"], case["K"], std=0.02, dtype=_DT[case["dtype"]])
    elif op == "dequant":
        st["q"] = _stored_rows(randn(case["M"], case["K"], std=0.02), fmt)
    elif op == "matmul":
        st["a"] = _stored_rows(_activations(gen, case["M"], case["K"], torch.bfloat16), fmt)
        st["b"] = _stored_rows(randn(case["N"], case["K"], std=0.02), fmt)
    else:
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        st["W"] = _stored_weight(randn(N, K, std=0.02), fmt)
        st["A"], st["B"] = randn(K, r, std=0.02), randn(r, N, std=0.02)
        st["X"] = _activations(gen, M, K, torch.bfloat16)
        if op == "bwd":
            st["dY"] = randn(M, N, std=1.0)
            st["T"] = st["X"].float() @ st["A"].float()  # what the forward saved
    return st


# ------------------------------------------------------------------ one pass
SCALE = 0.25  # alpha / r


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    case = st["case"]
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        return _plain_quantize(st["X"], fmt).to(torch.bfloat16)
    if op == "weight":
        v = _plain_weight(st["W"], fmt)[0].to(torch.bfloat16)
        return v, v.t().contiguous()
    if op == "dequant":
        return _decode(st["q"]["codes"], st["q"]["scales"], st["q"]["g"], fmt).to(_DT[case["dtype"]])
    if op == "matmul":
        a, b = (_decode(st[k]["codes"], st[k]["scales"], st[k]["g"], fmt) for k in ("a", "b"))
        return (a @ b.t()).to(_DT[case["dtype"]])
    A, B, X = st["A"].float(), st["B"].float(), st["X"].float()
    w = st["W"]["w"]
    W = _decode(w["codes"], w["scales"], w["g"], fmt)
    if op == "fwd":
        T = X @ A
        return (_plain_quantize(st["X"], fmt) @ W.t() + SCALE * (T @ B)).to(torch.bfloat16), T
    dY = st["dY"].float()
    G = dY @ B.t()
    dX = _plain_quantize(st["dY"], fmt) @ W + SCALE * (G @ A.t())
    return dX.to(torch.bfloat16), SCALE * (X.t() @ G), SCALE * (st["T"].t() @ dY)


def _run_own(st):
    from bit_nf4_quantized_unpack_b200 import qlora as q
    case = st["case"]
    op, fmt = case["op"], {MX: q.FP4_MXFP4, NV: q.FP4_NVFP4}[case["fmt"]]

    def matrix(s, rows, cols):
        return q.FP4Matrix(s["codes"], s["scales"], s["g"], rows, cols, fmt)

    if op == "quantize":
        return q.qlora_fp4_dequant(q.qlora_fp4_quantize(st["X"], fmt))
    if op == "weight":
        w = q.qlora_fp4_quantize_weight(st["W"], fmt)
        return q.qlora_fp4_dequant(w.w), q.qlora_fp4_dequant(w.wt)
    if op == "dequant":
        return q.qlora_fp4_dequant(matrix(st["q"], case["M"], case["K"]), _DT[case["dtype"]])
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return q.qlora_fp4_matmul(matrix(st["a"], M, K), matrix(st["b"], N, K), _DT[case["dtype"]])
    N, K = case["N"], case["K"]
    w = q.FP4Weight(matrix(st["W"]["w"], N, K), matrix(st["W"]["wt"], K, N))
    if op == "fwd":
        return q.qlora_fp4_linear_fwd(st["X"], w, st["A"], st["B"], SCALE)
    return q.qlora_fp4_linear_bwd(st["dY"], st["X"], st["T"], w, st["A"], st["B"], SCALE)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, bits = case["op"], 0.5 + 1.0 / BLOCK[case["fmt"]]
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 2)
    if op == "quantize":  # read, stored, read back as bf16
        n = case["M"] * case["K"]
        return {"bytes": n * (size + 2 * bits + 2), "flops": 4 * n}
    if op == "weight":  # the same, stored and read back in both orientations
        n = case["N"] * case["K"]
        return {"bytes": n * (size + 4 * bits + 4), "flops": 4 * n}
    if op == "dequant":
        n = case["M"] * case["K"]
        return {"bytes": n * (bits + size), "flops": 2 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "matmul":
        return {"bytes": (M + N) * K * bits + M * N * size, "flops": 2 * M * N * K}
    r = case["r"]
    if op == "fwd":
        return {"bytes": N * K * bits + 2 * M * (K + N) + 2 * r * (N + K) + 4 * M * r,
                "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    return {"bytes": N * K * bits + 2 * M * (2 * K + N) + 6 * r * (N + K) + 4 * M * r,
            "flops": 2 * M * N * K + 4 * M * r * (N + K)}


# ------------------------------------------------------------------ the definition in 64 bits
def _nearest(v, levels):
    """The nearest entry of ascending `levels` (ties to the even index, the last at most)."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo, hi = torch.bucketize(v, mid), torch.bucketize(v, mid, right=True)
    return levels[torch.where(lo % 2 == 0, lo, hi)]


def _exact_grid(x, fmt, dims, gdims):
    """x (fp64) on its grid: blocks are the axes `dims`, one gscale per the axes `gdims`."""
    dev = x.device
    e2m1 = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6.], dtype=torch.float64, device=dev)
    amax = x.abs().amax(dims, keepdim=True)
    if fmt == MX:
        e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -140)))
        e = e + (torch.exp2(e + 1) <= amax).double() - (torch.exp2(e) > amax).double()
        step = torch.exp2((e - 2).clamp(-127, 127))
    else:
        bytes_ = torch.arange(127, device=dev)
        ex, man = (bytes_ // 8).double(), (bytes_ % 8).double()
        e4m3 = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex - 7))
        top = amax.amax(gdims, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -160) / 2688))
        e = e + (2688 * torch.exp2(e) < top).double() - (2688 * torch.exp2(e - 1) >= top).double()
        g = torch.where(top > 0, torch.exp2(e.clamp(-126, 127)), torch.ones_like(top))
        step = _nearest(amax / g / 6, e4m3) * g
    some = torch.where(step > 0, step, torch.ones_like(step))
    return torch.where(step > 0, torch.copysign(_nearest(x.abs() / some, e2m1), x) * step, torch.zeros_like(x))


def _exact_rows(X, fmt):
    R, C = X.shape
    return _exact_grid(X.double().view(R, C // BLOCK[fmt], BLOCK[fmt]), fmt, (2,), (1, 2)).view(R, C)


def _exact_decode(s, R, C, fmt):
    c = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).view(R, C).long()
    low, ex = (c % 2).double(), (c // 2) % 4
    mag = torch.where(ex == 0, low / 2, (1 + low / 2) * torch.exp2(ex.double() - 1))
    row, blk = torch.arange(R, device=c.device)[:, None], torch.arange(C // BLOCK[fmt], device=c.device)[None]
    tiles = -(-(C // BLOCK[fmt]) // 4)
    b = s["scales"][((row // 128) * tiles + blk // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + blk % 4].long()
    if fmt == MX:
        sc = torch.exp2(b.double() - 127)
    else:
        sc = torch.where(b < 8, b.double() / 8 * 2.0 ** -6, (1 + (b % 8).double() / 8) * torch.exp2((b // 8).double() - 7))
        sc = sc * s["g"].double().view(-1, 1)
    return torch.where(c >= 8, -mag, mag) * sc.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        return _exact_rows(st["X"], fmt)
    if op == "weight":
        b, (N, K) = BLOCK[fmt], st["W"].shape
        v = _exact_grid(st["W"].double().view(N // b, b, K // b, b), fmt, (1, 3), (0, 1, 2, 3)).view(N, K)
        return v, v.t().contiguous()
    if op == "dequant":
        return _exact_decode(st["q"], case["M"], case["K"], fmt)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "matmul":
        return _exact_decode(st["a"], M, K, fmt) @ _exact_decode(st["b"], N, K, fmt).t()
    A, B, X = st["A"].double(), st["B"].double(), st["X"].double()
    W = _exact_decode(st["W"]["w"], N, K, fmt)
    if op == "fwd":
        T = X @ A
        return _exact_rows(st["X"], fmt) @ W.t() + SCALE * (T @ B), T
    dY = st["dY"].double()
    G = dY @ B.t()
    return (_exact_rows(st["dY"], fmt) @ W + SCALE * (G @ A.t()), SCALE * (X.t() @ G),
            SCALE * (st["T"].double().t() @ dY))
