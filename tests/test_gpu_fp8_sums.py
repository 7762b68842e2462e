"""Products of 8-bit floats for a 16-bit Y: sums are float32's whatever the number
of rows of X, so a Y is off by at most oracle.fp8_error_bound and half a step of its
type (2^-8 of the value for bfloat16; 2^-11 for float16, at least 2^-25)."""
import numpy as np
import pytest

import oracle
from tests.gpu_util import log
from tests.test_gpu_fp8 import _codes, _dt, _grouped_oracle, _operands, _rng, _scales, _stack

pytestmark = pytest.mark.gpu

# m, n, batch: tiles of every size, rows that are 16-byte aligned and rows that are not; 16 and 17 rows.
SIZES = [(300, 520, 16), (300, 520, 17), (140, 260, 260), (2100, 8208, 40), (2100, 8201, 40), (4200, 1040, 140),
         (1100, 4112, 300), (1100, 4099, 300), (1300, 1920, 530), (2700, 775, 700), (4100, 1056, 1100), (6200, 400, 2100)]


@pytest.fixture(scope="module")
def g(gpu_lib):
    import post_weight_quantization_11_amd as g
    return g


def _check(Y, res, n, out, what):
    want, mags, _ = res
    t = oracle.fp8_error_bound(n, mags)
    tol = t + (2.0 ** -8 * (np.abs(want) + t) if out == "bf16" else
               np.maximum(2.0 ** -11 * (np.abs(want) + t), 2.0 ** -25))
    err = np.abs(Y.double().cpu().numpy() - want)
    log(f"  {what}: max |err| / tol {float(np.max(err / np.maximum(tol, 1e-300))):.3e}")
    assert np.all(err <= tol)


@pytest.mark.parametrize("m,n,batch", SIZES)
def test_sums_of_a_16_bit_result(g, m, n, batch):
    dev, host = _operands(_rng(m, n, batch, 61), m, n, batch)
    res = oracle.fp8_matmul(*host)
    for out in ("bf16", "f16"):
        _check(g.gptq_block_gemm(*dev, y_dtype=_dt(out)), res, n, out, f"block gemm {batch}x{m}x{n} ->{out}")


@pytest.mark.parametrize("m,n,batch", SIZES)
def test_large_terms_that_cancel(g, m, n, batch):
    """Of every eight columns two have products of 448 * 448 that cancel, the others
    add 3 each, less than 2^-13 of those: what is left is all of the result."""
    import torch
    w = np.full((m, n), 0x3C, dtype=np.uint8)                 # 1.5
    x = np.full((batch, n), 0x40, dtype=np.uint8)             # 2
    pairs = n // 8
    w[:, 0:8 * pairs:8], w[:, 1:8 * pairs:8] = 0x7E, 0xFE     # 448 and -448
    x[:, 0:8 * pairs:8], x[:, 1:8 * pairs:8] = 0x7E, 0x7E
    ws = np.full((-(-m // 128), oracle.fp8_blocks(n)), 2.0 ** -9, dtype=np.float32)
    xs = np.full((batch, oracle.fp8_blocks(n)), 2.0 ** -3, dtype=np.float32)
    W, S, X, XS = (torch.from_numpy(a).cuda() for a in (w, ws, x, xs))
    res = oracle.fp8_matmul(w, ws, x, xs)
    for out in ("bf16", "f16"):
        Y = g.gptq_block_gemm(W.view(torch.float8_e4m3fn), S, X.view(torch.float8_e4m3fn), XS, y_dtype=_dt(out))
        _check(Y, res, n, out, f"terms that cancel {batch}x{m}x{n} ->{out}")


@pytest.mark.parametrize("experts,m,n,off,rows", [
    (1, 300, 520, [0, 13], 13), (1, 300, 520, [0, 16], 16), (2, 300, 528, [0, 9, 16], 16),
    (3, 260, 1024, [0, 17, 17, 600], 600), (2, 3300, 520, [0, 700, 1500], 1500), (8, 1100, 640, list(range(0, 2700, 300)), 2400),
])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_sums_of_a_16_bit_result_by_expert(g, experts, m, n, off, rows, out):
    import torch
    rng = _rng(experts, m, n, rows, 67)
    dev, host = _stack(rng, experts, m, n, True)
    X, xc = _codes(rng, rows, n, -(-n // 16) * 16)
    XS, xs = _scales(rng, rows, oracle.fp8_blocks(n))
    Y = torch.full((rows, m), 7.0, device="cuda", dtype=_dt(out))
    g.gptq_block_gemm_grouped(*dev, X, XS, torch.tensor(off, dtype=torch.int32, device="cuda"), Y=Y)
    _check(Y, _grouped_oracle(host, xc, xs, off, np.full((rows, m), 7.0)), n, out,
           f"grouped {experts} x {m}x{n}, {rows} rows ->{out}")
