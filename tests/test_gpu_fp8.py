"""Block-scaled 8-bit floats on the GPU against the float64 oracle.

Quantization is exact: scales, codes and (in float32) values must be equal; a
16-bit Wq is the float32 value rounded.  Products: the error before the rounding
to Y's type is at most oracle.fp8_error_bound, for a 16-bit Y
oracle.fp8_stored_bound; a 16-bit Y adds half a unit of its type (2^-8 relative
for bfloat16, 2^-11 for float16, at least 2^-25 absolute there)."""
import numpy as np
import pytest

import oracle
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g(gpu_lib):
    import post_weight_quantization_11_amd as g
    return g


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(list(seed))))


def _to(a, dtype, cols=None):
    """Device tensor of `dtype` (and its float64 values); `cols`: leading dimension."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(_dt(dtype))
    if cols is not None:
        buf = torch.full((t.shape[0], cols), float("nan"), dtype=t.dtype)
        buf[:, :t.shape[1]] = t
        d = buf.cuda()[:, :t.shape[1]]
    else:
        d = t.cuda()
    return d, t.double().numpy()


# ---------------------------------------------------------------------------
# Quantization.
# ---------------------------------------------------------------------------
def _check_quantized(q, W64, block_rows, dtype):
    import torch
    codes, scales = oracle.fp8_quantize(W64, block_rows)
    gs = q["scales"].cpu().numpy()
    assert np.array_equal(gs, scales, equal_nan=True)
    gc = q["codes"].view(torch.uint8).cpu().numpy()
    assert np.array_equal(gc, codes)
    if q["Wq"] is not None:
        with np.errstate(over="ignore"):
            v = oracle.fp8_dequantize(codes, scales, block_rows).astype(np.float32)
        want = torch.from_numpy(v).to(_dt(dtype))
        assert torch.equal(torch.nan_to_num(q["Wq"].cpu(), nan=-7.0), torch.nan_to_num(want, nan=-7.0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,ld", [(1, 1, None), (3, 127, None), (2, 128, None), (5, 129, None), (256, 256, None),
                                    (127, 1000, None), (130, 1031, 1037), (300, 64, 72), (1, 20001, None)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_matches_oracle(g, dtype, m, n, ld, block_rows):
    rng = _rng(m, n, 1)
    W, W64 = _to(rng.standard_normal((m, n)) * 0.02 * np.exp(rng.standard_normal((m, 1))), dtype, ld)
    for want_wq in (False, True):
        q = g.gptq_block_quantize(W, block_rows, want_wq=want_wq)
        assert q["codes"].shape == W.shape and q["codes"].stride(0) % 16 == 0
        _check_quantized(q, W64, block_rows, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_borders_of_every_code(g, dtype):
    """Blocks whose scale is a power of two, so that their quotients meet the
    midpoints between codes, with the type's neighbours of each; and float32
    blocks of arbitrary scales with the float32 numbers around mid * scale."""
    import torch
    v = oracle.FP8_VALUES[:127]
    mids = (v[1:] + v[:-1]) / 2
    step = float(torch.finfo(_dt(dtype)).eps)
    rows = []
    for e in (-8, -3, 0, 3, 6) if dtype == "f16" else (-126, -100, -40, -8, 0, 5, 60, 118):
        for pts in (v[1:127], mids, mids * (1 + step), mids * (1 - step / 2)):
            r = np.zeros(128)
            r[:len(pts)] = pts
            r[127] = -448.0
            rows.append(np.ldexp(r * np.where(np.arange(128) % 3 == 0, -1, 1), e))
    if dtype == "f32":
        rng = _rng(9)
        for top in np.exp(rng.uniform(-80, 80, size=60)).astype(np.float32):
            s = np.float32(np.float64(top) / 448.0)
            near = (mids * np.float64(s)).astype(np.float32)
            for k in (-2, -1, 0, 1, 2):
                r = np.zeros(128, dtype=np.float32)
                r[:126] = (near.view(np.int32) + k).view(np.float32)
                r[127] = top
                rows.append(r.astype(np.float64))
    W = torch.from_numpy(np.stack(rows)).to(_dt(dtype))
    q = g.gptq_block_quantize(W.cuda(), want_wq=True)
    _check_quantized(q, W.double().numpy(), 1, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_range_ends_and_special_blocks(g, dtype, block_rows):
    import torch
    t = _dt(dtype)
    info = torch.finfo(t)
    tiny = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dtype]
    W = torch.ones((block_rows, 14 * 128), dtype=torch.float64)
    for j, val in enumerate([0.0, -0.0, tiny, float(info.tiny), float(info.max), -float(info.max), float("nan"),
                             float("inf"), float("-inf"), 447 * tiny, 500 * tiny, 1.0, 448.0, 3.4]):
        W[:, 128 * j:128 * j + 128] = torch.linspace(0, 1, 128) * val if np.isfinite(val) else 1.0
        W[-1, 128 * j + 127] = val
    W = W.to(t)
    _check_quantized(g.gptq_block_quantize(W.cuda(), block_rows, want_wq=True), W.double().numpy(), block_rows, dtype)


def test_quantize_writes_only_its_elements(g):
    import torch
    rng = _rng(3)
    W, W64 = _to(rng.standard_normal((133, 145)), "bf16", 150)
    for block_rows in (1, 128):
        rb = 133 if block_rows == 1 else 2
        codes = torch.full((133, 151), 9, dtype=torch.uint8, device="cuda")
        scales = torch.full((rb, 5), 9.0, device="cuda")
        wq = torch.full((133, 147), 3.0, dtype=torch.bfloat16, device="cuda")
        out = dict(codes=codes[:, :145].view(torch.float8_e4m3fn), scales=scales[:, :2], Wq=wq[:, :145])
        _check_quantized(g.gptq_block_quantize(W, block_rows, out=out), W64, block_rows, "bf16")
        assert (codes[:, 145:] == 9).all() and (scales[:, 2:] == 9).all() and (wq[:, 145:] == 3.0).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_stack_of_experts(g, block_rows):
    # Blocks do not cross from one matrix into the next, whose rows may lie apart.
    import torch
    rng = _rng(4)
    E, m, n = 6, 150, 70
    W, W64 = _to(rng.standard_normal((2 * E * m, n)) * np.exp(rng.standard_normal((2 * E * m, 1))), "f16")
    q = g.gptq_block_quantize(W.view(2 * E, m, n)[::2], block_rows, want_wq=True)
    assert q["codes"].shape == (E, m, n) and q["scales"].shape == (E, m if block_rows == 1 else 2, 1)
    for e in range(E):
        _check_quantized({k: q[k][e] for k in q}, W64.reshape(2 * E, m, n)[2 * e], block_rows, "f16")
    for shape in ((0, 70), (5, 0), (0, 5, 70), (3, 0, 70)):
        q = g.gptq_block_quantize(torch.empty(shape, device="cuda"), block_rows)
        assert q["codes"].numel() == 0 and q["scales"].numel() == 0


def test_quantize_many_rows(g):
    # More rows than one grid dimension of 65535 workgroups would take.
    import torch
    W = torch.randn((700001, 33), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    at = torch.tensor([0, 1, 65535, 65536, 349999, 700000], device="cuda")
    q = g.gptq_block_quantize(W, want_wq=True)
    _check_quantized(dict(codes=q["codes"].view(torch.uint8)[at].view(torch.float8_e4m3fn), scales=q["scales"][at],
                          Wq=q["Wq"][at]), W[at].double().cpu().numpy(), 1, "bf16")
    q = g.gptq_block_quantize(W, 128, want_wq=True)
    lo = 128 * (700001 // 128)
    _check_quantized({k: q[k][lo // 128 if k == "scales" else lo:] for k in q}, W[lo:].double().cpu().numpy(), 128, "bf16")


# ---------------------------------------------------------------------------
# Products.
# ---------------------------------------------------------------------------
def _codes(rng, m, n, ld=None):
    """Codes drawn as normal data gives them, one in eight from all values: a
    device matrix (`ld`: leading dimension, the padding NaN codes) and a host one."""
    import torch
    c = oracle.fp8_nearest_code(rng.standard_normal((m, n)) * 120)
    c = np.where(rng.random((m, n)) < 0.125, rng.integers(0, 256, size=(m, n)), c).astype(np.uint8)
    c = np.where(c & 127 == 127, c - 1, c).astype(np.uint8)
    buf = np.full((m, ld or n), 127, dtype=np.uint8)
    buf[:, :n] = c
    return torch.from_numpy(buf).cuda()[:, :n].view(torch.float8_e4m3fn), c


def _scales(rng, rows, blocks, ld=None, lo=-12.0, hi=-4.0):
    import torch
    s = np.exp2(rng.uniform(lo, hi, size=(rows, blocks))).astype(np.float32)
    buf = np.full((rows, ld or blocks), np.nan, dtype=np.float32)
    buf[:, :blocks] = s
    return torch.from_numpy(buf).cuda()[:, :blocks], s


def _operands(rng, m, n, batch, pads=(None,) * 4):
    nb = oracle.fp8_blocks(n)
    W, wc = _codes(rng, m, n, pads[0])
    S, ws = _scales(rng, -(-m // 128), nb, pads[1])
    X, xc = _codes(rng, batch, n, pads[2])
    XS, xs = _scales(rng, batch, nb, pads[3])
    return (W, S, X, XS), (wc, ws, xc, xs)


def _tol(n, mags, cut, want, out):
    if out == "f32":
        return oracle.fp8_error_bound(n, mags)
    t = oracle.fp8_stored_bound(n, mags, cut)
    if out == "bf16":
        return t + 2.0 ** -8 * (np.abs(want) + t)
    return t + np.maximum(2.0 ** -11 * (np.abs(want) + t), 2.0 ** -25)


def _check(Y, res, n, out, what, keep=None):
    want, mags, cut = res
    got = Y.double().cpu().numpy()
    assert got.shape == want.shape
    tol = _tol(n, mags, cut, want, out)
    with np.errstate(invalid="ignore"):
        err = np.abs(got - want)
    if keep is not None:
        err = np.where(keep, err, 0.0)
    log(f"  {what}: max |err| / tol {float(np.max(err / np.maximum(tol, 1e-300), initial=0.0)):.3e}")
    assert np.all(err <= tol)


GEMM = [
    # m, n, batch: row kernels, then tiles (more than 16 rows, 1.5e9 products), each with rows that are 16-byte
    # aligned and with rows that are not
    (1, 1, 1), (16, 128, 1), (17, 33, 2), (40, 7, 3), (70, 1000, 5), (33, 31, 16), (64, 4096, 1), (100, 2049, 17),
    (256, 256, 64), (130, 640, 33), (515, 515, 130), (300, 1031, 259), (1040, 256, 7), (2060, 6200, 3),
    (2060, 6203, 3), (8200, 520, 12), (8200, 515, 12),
    (2100, 8208, 40), (2100, 8201, 40), (4200, 1040, 140), (4200, 1031, 140), (1100, 4112, 300), (1100, 4099, 300),
    (2700, 768, 700), (2700, 775, 700), (1300, 1920, 530), (1300, 1925, 530), (4100, 1056, 1100), (4100, 1030, 1100),
    (6200, 400, 2100), (6200, 393, 2100), (2100, 8208, 100), (2100, 8201, 100),
]


@pytest.mark.parametrize("m,n,batch", GEMM)
def test_gemm_matches_oracle(g, m, n, batch):
    import torch
    rng = _rng(m, n, batch)
    dev, host = _operands(rng, m, n, batch)
    res = oracle.fp8_matmul(*host)
    for out in ("f32", "bf16", "f16"):
        Y = g.gptq_block_gemm(*dev, y_dtype=_dt(out))
        assert Y.dtype == _dt(out)
        _check(Y, res, n, out, f"block gemm {batch}x{m}x{n} ->{out}")
        assert torch.equal(Y, g.gptq_block_gemm(*dev, y_dtype=_dt(out)))      # the same bits every time


@pytest.mark.parametrize("m,n,batch", [(37, 70, 3), (300, 515, 70), (1300, 1925, 530), (1300, 1920, 530)])
def test_gemm_strided_operands_and_padding(g, m, n, batch):
    # Leading dimensions of their own, padding that must not be read (NaN codes
    # and scales) or written.
    import torch
    rng = _rng(m, n, batch, 7)
    nb = oracle.fp8_blocks(n)
    for pads in ((n + 3, nb + 2, n + 1, nb + 1), (n - n % 16 + 32, nb + 1, n - n % 16 + 16, nb + 3)):
        dev, host = _operands(rng, m, n, batch, pads)
        for out in ("f32", "bf16"):
            buf = torch.full((batch, m + 5), 4.0, device="cuda", dtype=_dt(out))
            Y = g.gptq_block_gemm(*dev, Y=buf[:, :m])
            _check(Y, oracle.fp8_matmul(*host), n, out, f"strided block gemm {batch}x{m}x{n} ->{out}")
            assert (buf[:, m:] == 4.0).all()


SHAPES = [(150, 300, 3), (140, 260, 260), (1300, 1925, 530), (4100, 1056, 1100)]


@pytest.mark.parametrize("m,n,batch", SHAPES)
def test_gemm_nan_codes_and_scales(g, m, n, batch):
    rng = _rng(17, m, batch)
    (W, S, X, XS), (wc, ws, xc, xs) = _operands(rng, m, n, batch)
    import torch
    W.view(torch.uint8)[5, 17] = 127                          # row 5 of W
    X.view(torch.uint8)[1, 130] = 255                         # row 1 of X
    S[1, 1] = float("nan")                                    # rows 128 .. 255 of W
    XS[2, 0] = float("inf")
    bad = np.zeros((batch, m), dtype=bool)
    bad[:, 5] = bad[1] = bad[2] = True
    bad[:, 128:256] = True
    res = oracle.fp8_matmul(wc, ws, xc, xs)
    for out in ("f32", "bf16"):
        Y = g.gptq_block_gemm(W, S, X, XS, y_dtype=_dt(out))
        got = Y.double().cpu().numpy()
        assert not np.isfinite(got[bad]).any() and np.isfinite(got[~bad]).all()
        _check(Y, res, n, out, f"NaN codes {batch}x{m}x{n} ->{out}", ~bad)


@pytest.mark.parametrize("m,n,batch", SHAPES)
def test_gemm_wide_scales(g, m, n, batch):
    # Blocks that span two hundred binades, the products of scales inside
    # float32's normal range.
    rng = _rng(19, m, batch)
    nb = oracle.fp8_blocks(n)
    W, wc = _codes(rng, m, n)
    X, xc = _codes(rng, batch, n)
    S, ws = _scales(rng, -(-m // 128), nb, None, -60, 50)
    XS, xs = _scales(rng, batch, nb, None, -60, 50)
    res = oracle.fp8_matmul(wc, ws, xc, xs)
    for out in ("f32", "bf16"):
        _check(g.gptq_block_gemm(W, S, X, XS, y_dtype=_dt(out)), res, n, out, f"wide scales {batch}x{m}x{n} ->{out}")


@pytest.mark.parametrize("m,n,batch", SHAPES)
def test_gemm_sums_built_for_the_bounds(g, m, n, batch):
    """One large term and many that the running sum rounds away or the stored
    form cuts, all of one sign: the bounds hold where roundings line up."""
    import torch
    w = np.full((m, n), 0x08, dtype=np.uint8)                 # 2^-6
    x = np.full((batch, n), 0x38, dtype=np.uint8)             # 1
    w[:, ::8], x[:, ::8] = 0x7E, 0x40                         # 448 and 2: 2^-16 of it is the others'
    w[1::2, 1::8], x[:, 1::8] = 0x01, 0x7E                    # 2^-9 times 448
    ws = np.full((-(-m // 128), oracle.fp8_blocks(n)), 1.0 / 3, dtype=np.float32)
    xs = np.full((batch, oracle.fp8_blocks(n)), 1.0 / 7, dtype=np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (w, ws, x, xs)]
    dev[0], dev[2] = dev[0].view(torch.float8_e4m3fn), dev[2].view(torch.float8_e4m3fn)
    res = oracle.fp8_matmul(w, ws, x, xs)
    for out in ("f32", "bf16", "f16"):
        _check(g.gptq_block_gemm(*dev, y_dtype=_dt(out)), res, n, out, f"one-sided sums {batch}x{m}x{n} ->{out}")


def test_gemm_empty(g):
    import torch
    f8 = torch.float8_e4m3fn
    X, XS = torch.ones((3, 64), device="cuda").to(f8), torch.ones((3, 1), device="cuda")
    W0, S0 = torch.zeros((0, 64), device="cuda").to(f8), torch.zeros((0, 1), device="cuda")
    assert g.gptq_block_gemm(W0, S0, X, XS).shape == (3, 0)
    W, S = torch.zeros((5, 64), device="cuda").to(f8), torch.zeros((1, 1), device="cuda")
    assert g.gptq_block_gemm(W, S, X[:0], XS[:0]).shape == (0, 5)
    for out in ("f32", "bf16"):
        Y = g.gptq_block_gemm(W[:, :0], S[:, :0], X[:, :0], XS[:, :0], Y=torch.full((3, 5), 2.0, device="cuda").to(_dt(out)))
        assert (Y == 0).all()


@pytest.mark.parametrize("which", ["W", "X"])
def test_gemm_rows_far_apart(g, which):
    # Offsets past 32 bits: 300 rows 16 MiB apart.
    import torch
    rng = _rng(23)
    m, n, batch = (300, 260, 40) if which == "W" else (40, 260, 300)
    (W, S, X, XS), host = _operands(rng, m, n, batch)
    far = torch.empty((300, 1 << 24), dtype=torch.uint8, device="cuda")[:, :n].view(torch.float8_e4m3fn)
    far.copy_(W if which == "W" else X)
    dev = (far, S, X, XS) if which == "W" else (W, S, far, XS)
    for out in ("f32", "f16"):
        _check(g.gptq_block_gemm(*dev, y_dtype=_dt(out)), oracle.fp8_matmul(*host), n, out, f"far rows of {which} ->{out}")


# ---------------------------------------------------------------------------
# Grouped by expert.
# ---------------------------------------------------------------------------
def _stack(rng, E, m, n, align=False):
    """Codes (rows 16-byte aligned or dense) and scales of E matrices."""
    import torch
    ld = -(-n // 16) * 16 if align else n
    W, wc = _codes(rng, E * m, n, ld)
    S, ws = _scales(rng, E * -(-m // 128), oracle.fp8_blocks(n))
    dense = torch.as_strided(W, (E, m, n), (m * ld, ld, 1))
    return (dense, S.view(E, -1, S.shape[1])), (wc.reshape(E, m, n), ws.reshape(E, -1, S.shape[1]))


def _grouped_oracle(host, xc, xs, off, Y0):
    wc, ws = host
    res = [Y0.copy(), np.zeros_like(Y0), np.zeros_like(Y0)]
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a < b:
            for r, v in zip(res, oracle.fp8_matmul(wc[e], ws[e], xc[a:b], xs[a:b])):
                r[a:b] = v
    return res


GROUPED = [
    # experts, m, n, offsets, rows
    (1, 33, 70, [0, 5], 5),
    (3, 140, 100, [0, 0, 7, 7], 7),                      # the first and the last without rows
    (4, 150, 128, [0, 1, 2, 3, 4], 4),                   # one row each
    (5, 264, 260, [2, 4, 30, 30, 95, 99], 110),          # rows before and behind that belong to none
    (2, 130, 515, [0, 300, 301], 301),
    (70, 20, 64, list(range(0, 71 * 3, 3)), 213),        # more experts than lanes of a wave
    (130, 16, 40, [0] * 100 + [9] * 30 + [12], 12),
    (3, 260, 1024, [0, 17, 17, 600], 600),
    (8, 300, 999, [0, 16, 32, 33, 34, 200, 460, 461, 777], 777),
    (300, 264, 144, sorted(list(range(0, 1200, 4)) + [1200]), 1200),
    (2, 1300, 1040, [0, 500, 1100], 1100),
    (2, 1300, 1025, [0, 500, 1100], 1100),
    (2, 3300, 520, [0, 700, 1500], 1500),
    (2, 3300, 525, [0, 700, 1500], 1500),
    (6, 640, 256, [0, 60, 130, 190, 250, 320, 400], 400),
    (6, 640, 250, [0, 60, 130, 190, 250, 320, 400], 400),
    (20, 132, 300, [33 * i for i in range(21)], 660),
    (20, 833, 2003, [0, 0, 40, 56, 89, 90, 110, 141, 173, 190, 205, 269, 274, 304, 316, 336, 356, 364, 392, 396, 402],
     410),
]


@pytest.mark.parametrize("experts,m,n,off,rows", GROUPED)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_matches_oracle(g, experts, m, n, off, rows, out):
    import torch
    rng = _rng(experts, m, n, rows)
    for align in (False, True):
        dev, host = _stack(rng, experts, m, n, align)
        X, xc = _codes(rng, rows, n, -(-n // 16) * 16 if align else None)
        XS, xs = _scales(rng, rows, oracle.fp8_blocks(n))
        Y = torch.full((rows, m), 7.0, device="cuda", dtype=_dt(out))
        got = g.gptq_block_gemm_grouped(*dev, X, XS, torch.tensor(off, dtype=torch.int32, device="cuda"), Y=Y)
        assert got is Y
        _check(Y, _grouped_oracle(host, xc, xs, off, np.full((rows, m), 7.0)), n, out,
               f"grouped {experts} x {m}x{n}, {rows} rows ->{out}")


def test_grouped_strided_experts(g):
    import torch
    rng = _rng(23)
    E, m, n, rows = 3, 140, 270, 30
    (W, S), host = _stack(rng, E, m, n)
    P = torch.full((E, m + 2, 275), 127, dtype=torch.uint8, device="cuda")
    Q = torch.full((E, 4, 5), float("nan"), device="cuda")
    P[:, :m, :n] = W.view(torch.uint8)
    Q[:, :2, :3] = S
    off = [0, 11, 12, 30]
    X, xc = _codes(rng, rows, n, 280)
    XS, xs = _scales(rng, rows, 3, 4)
    Y = torch.zeros((rows, m + 1), device="cuda")
    g.gptq_block_gemm_grouped(P[:, :m, :n].view(torch.float8_e4m3fn), Q[:, :2, :3], X, XS,
                              torch.tensor(off, dtype=torch.int32, device="cuda"), Y=Y[:, :m])
    _check(Y[:, :m], _grouped_oracle(host, xc, xs, off, np.zeros((rows, m))), n, "f32", "strided experts")
    assert (Y[:, m] == 0).all()


@pytest.mark.parametrize("rows", [12, 900])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_offsets_beyond_the_rows_are_confined(g, rows, out):
    # Offsets below 0 and above the row count mean the rows there are; the rows
    # around Y's (one buffer) stay.  Offsets that go down leave it open which rows
    # are computed.
    import torch
    rng = _rng(29, rows)
    E, m, n = 3, 1024, 256
    dev, host = _stack(rng, E, m, n)
    X, xc = _codes(rng, rows, n)
    XS, xs = _scales(rng, rows, 2)
    buf = torch.full((rows + 20, m), 5.0, device="cuda", dtype=_dt(out))
    off = torch.tensor([-(1 << 31), 4, 9, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    g.gptq_block_gemm_grouped(*dev, X, XS, off, Y=buf[10:10 + rows])
    _check(buf[10:10 + rows], _grouped_oracle(host, xc, xs, [0, 4, 9, rows], np.zeros((rows, m))), n, out,
           f"confined offsets, {rows} rows ->{out}")
    off = torch.tensor([rows, 3, (1 << 31) - 1, -5], dtype=torch.int32, device="cuda")
    g.gptq_block_gemm_grouped(*dev, X, XS, off, Y=buf[10:10 + rows])
    assert (buf[:10] == 5.0).all() and (buf[10 + rows:] == 5.0).all()


def test_grouped_empty(g):
    import torch
    f8 = torch.float8_e4m3fn
    X, XS = torch.ones((4, 64), device="cuda").to(f8), torch.ones((4, 1), device="cuda")
    W, S = torch.zeros((2, 8, 64), device="cuda").to(f8), torch.zeros((2, 1, 1), device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y = torch.full((4, 8), 3.0, device="cuda")
    g.gptq_block_gemm_grouped(W, S, X, XS, off, Y=Y)                        # no rows in any expert
    assert (Y == 3.0).all()
    g.gptq_block_gemm_grouped(W[:0], S[:0], X, XS, off[:1], Y=Y)            # no experts
    assert (Y == 3.0).all()
    assert g.gptq_block_gemm_grouped(W, S, X[:0], XS[:0], off).shape == (0, 8)
    off[1:] = 4
    g.gptq_block_gemm_grouped(W[:, :, :0], S[:, :, :0], X[:, :0], XS[:, :0], off, Y=Y)      # no columns: empty sums
    assert (Y == 0).all()


# ---------------------------------------------------------------------------
# On streams, in graphs, refused.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("batch", [2, 77, 1300])
def test_side_stream(g, batch):
    import torch
    rng = _rng(47, batch)
    m, n = 600, 1000
    dev, host = _operands(rng, m, n, batch)
    A, A64 = _to(rng.standard_normal((batch, n)), "f16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    Y = g.gptq_block_gemm(*dev, stream=s)
    q = g.gptq_block_quantize(A, want_wq=True, stream=s)
    Z = g.gptq_block_gemm(dev[0], dev[1], q["codes"], q["scales"], stream=s)
    s.synchronize()
    _check(Y, oracle.fp8_matmul(*host), n, "f32", "side stream")
    _check_quantized(q, A64, 1, "f16")
    _check(Z, oracle.fp8_matmul(host[0], host[1], *oracle.fp8_quantize(A64, 1)), n, "f32", "side stream, quantized")


def test_graphs_replayed_in_turn(g):
    """Graphs over the operators, replayed several times in turn with new
    inputs and eager calls between, each replay against the eager result."""
    import torch
    rng = _rng(53)
    E, m, n = 4, 300, 8200
    layers = []
    for batch in (3, 290, 640):
        (W, S), _ = _stack(rng, E, m, n)
        X, _ = _to(rng.standard_normal((batch, n)), "bf16")
        off = torch.tensor([0, 1, 1, batch // 2, batch], dtype=torch.int32, device="cuda")
        layers.append(dict(W=W, S=S, X=X, off=off, Yg=torch.zeros((batch, m), device="cuda")))
    assert g.load().gptq_block_gemm_ws_bytes(m, n, 640, 1) > 0              # split columns: a workspace each

    def step(L):
        q = g.gptq_block_quantize(L["X"])
        x = q["codes"], q["scales"]
        return (g.gptq_block_gemm(L["W"][0], L["S"][0], *x),
                g.gptq_block_gemm(L["W"][1], L["S"][1], *x, y_dtype=torch.bfloat16),
                g.gptq_block_gemm_grouped(L["W"], L["S"], *x, L["off"], Y=L["Yg"]))

    graphs = []
    for L in layers:
        step(L)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(L)
        graphs.append((gr, out))
    for k in range(4):
        for L, (gr, out) in zip(layers, graphs):
            L["X"].copy_(torch.randn(L["X"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)))
            gr.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            for x, y in zip(got, step(L)):
                assert torch.equal(x, y)


def test_binding_refusals(g):
    import torch
    f8 = torch.float8_e4m3fn
    W, S = torch.zeros((140, 64), device="cuda").to(f8), torch.zeros((2, 1), device="cuda")
    X, XS = torch.zeros((3, 64), device="cuda").to(f8), torch.zeros((3, 1), device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    wide = torch.zeros((140, 64), device="cuda")
    bad = [
        lambda: g.gptq_block_quantize(wide, 64), lambda: g.gptq_block_quantize(wide.double()),
        lambda: g.gptq_block_quantize(wide.t()), lambda: g.gptq_block_quantize(wide[0]),
        lambda: g.gptq_block_quantize(wide, 1, out=dict(codes=W[:139])),
        lambda: g.gptq_block_quantize(wide, 128, out=dict(scales=S[:1])),
        lambda: g.gptq_block_quantize(wide, 1, out=dict(Wq=wide.half())),
        lambda: g.gptq_block_gemm(W.view(torch.uint8), S, X, XS), lambda: g.gptq_block_gemm(W, S, X.view(torch.uint8), XS),
        lambda: g.gptq_block_gemm(W, S[:1], X, XS), lambda: g.gptq_block_gemm(W, S.double(), X, XS),
        lambda: g.gptq_block_gemm(W, S, X[:, :63], XS), lambda: g.gptq_block_gemm(W, S, X, XS[:2]),
        lambda: g.gptq_block_gemm(W, S, X, XS.cpu()), lambda: g.gptq_block_gemm(W[None], S, X, XS),
        lambda: g.gptq_block_gemm(W, S, X, XS, Y=torch.zeros((3, 139), device="cuda")),
        lambda: g.gptq_block_gemm(W, S, X, XS, y_dtype=torch.float64),
        lambda: g.gptq_block_gemm(W, S, X, XS, ws=torch.zeros(4)),
        lambda: g.gptq_block_gemm_grouped(W, S, X, XS, off), lambda: g.gptq_block_gemm_grouped(W[None], S, X, XS, off),
        lambda: g.gptq_block_gemm_grouped(W[None], S[None], X, XS, off[:1]),
        lambda: g.gptq_block_gemm_grouped(W[None], S[None], X, XS, off.long()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    m, n, batch = 1100, 12000, 200
    need = g.load().gptq_block_gemm_ws_bytes(m, n, batch, 1)
    W, S = torch.zeros((m, n), device="cuda").to(f8), torch.zeros((9, 94), device="cuda")
    X, XS = torch.zeros((batch, n), device="cuda").to(f8), torch.zeros((batch, 94), device="cuda")
    with pytest.raises(g.GptqError):
        g.gptq_block_gemm(W, S, X, XS, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    g.gptq_block_gemm(W, S, X, XS, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_many_blocks(g, dtype):
    # Enough blocks that a workgroup takes four; three strips of rows of them, the
    # last one partial, and the last columns of all.
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    W = (torch.randn((20010, 1800), device="cuda", generator=gen) * 0.05).to(_dt(dtype))
    q = g.gptq_block_quantize(W, 128, want_wq=True)
    for strip in (0, 77, 156):
        rows = slice(128 * strip, 128 * strip + 128)
        part = {k: q[k][slice(strip, strip + 1) if k == "scales" else rows] for k in q}
        _check_quantized(part, W[rows].double().cpu().numpy(), 128, dtype)
