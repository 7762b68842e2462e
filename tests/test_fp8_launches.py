"""What the 8-bit products launch, from their sizes and addresses alone,
recorded without a GPU."""
import re

import pytest

from tests import launch_recorder

F32, F16, BF16 = 0, 1, 2
P = 0x1000                        # 16-byte aligned, never followed
NAME = re.compile(r"_ZN\w*?\d+(fp8_\w+?_kernel)(?:I((?:L[ib]\d+E)+)E)?E")


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return launch_recorder.build(str(tmp_path_factory.mktemp("recorder")))


def _kernel(mangled):
    m = NAME.match(mangled)
    return (m.group(1), tuple(int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2) or ""))) if m else (mangled, ())


def _record(recorder, calls):
    out, pending = [], []
    for w in launch_recorder._run(recorder, calls):
        if w[0] == "call":
            out.append((int(w[2]), pending))
            pending = []
        elif w[0] == "launch":
            pending.append((_kernel(w[1]), [int(v) for v in w[2:9]]))
    return out


def _up(a, b):
    return -(-a // b)


def _gemm(m, n, rows, out, ldx=None):
    nb = _up(n, 128)
    return ("gptq_block_gemm", [P, m, n, n, P, nb, P, rows, ldx or n, P, nb, P, out, m, P, 1 << 50, None])


def _grouped(experts, m, n, rows, out, ld=None):
    nb, ld = _up(n, 128), ld or n
    return ("gptq_block_gemm_grouped", [P, experts, m, n, ld, m * ld, P, nb, _up(m, 128) * nb, P, rows, ld, P, nb, P, P,
                                        out, m, None, 0, None])


def _kind(kernel):
    name, a = kernel
    return (32 * a[1] * a[3], 32 * a[2] * a[4]) if name == "fp8_tile_kernel" else ("rows", a[0])


# Rows of X, of W and columns of sizes measured on two kernels, and the faster one.
MEASURED = [
    (1, 4096, 4096, BF16, ("rows", 1)), (1, 4096, 11008, BF16, ("rows", 1)), (16, 4096, 4096, F32, ("rows", 1)),
    (24, 4096, 4096, BF16, ("rows", 2)), (1, 49152, 12288, F32, ("rows", 2)), (32, 4096, 4096, BF16, ("rows", 2)),
    (64, 4096, 4096, BF16, ("rows", 2)), (24, 12288, 12288, BF16, (128, 32)), (77, 4096, 11008, BF16, (128, 64)),
    (16, 12288, 12289, BF16, ("rows", 2)), (24, 4099, 4097, F32, (128, 32)), (77, 4099, 11007, F32, (128, 128)),
    (512, 4096, 4096, BF16, (128, 64)),
    (2048, 4096, 4096, BF16, (128, 128)), (4096, 4096, 4096, BF16, (256, 256)), (4096, 4096, 4096, F32, (128, 128)),
    (4096, 12288, 12288, BF16, (256, 256)),
]


@pytest.mark.parametrize("rows,m,n,out,want", MEASURED)
def test_the_plan_takes_the_kernel_that_measured_faster(recorder, rows, m, n, out, want):
    rc, launches = _record(recorder, [_gemm(m, n, rows, out)])[0]
    assert rc == 0 and _kind(launches[0][0]) == want


@pytest.mark.parametrize("experts,rows,m,n,ld,want", [
    (64, 256, 2048, 4096, 4096, ("rows", 2)), (4, 4, 512, 512, 512, ("rows", 1)), (64, 256, 2048, 1024, 1024, "tiles"),
    (8, 256, 11008, 4096, 4096, ("rows", 4)), (64, 1600, 1300, 2048, 2048, "tiles"),
    (64, 16, 2048, 1024, 1024, ("rows", 2)), (64, 1600, 1300, 2048, 2052, ("rows", 4)),
    (8, 512, 11008, 4096, 4096, "tiles"),
])
def test_the_plan_of_grouped_products(recorder, experts, rows, m, n, ld, want):
    rc, launches = _record(recorder, [_grouped(experts, m, n, rows, BF16, ld)])[0]
    kind = _kind(launches[0][0])
    assert rc == 0 and len(launches) == 1 and (kind == want or (want == "tiles" and kind[0] != "rows"))


def test_a_launch_has_fewer_than_2_to_the_32_threads(recorder):
    calls = [_grouped(2048, 131072, 8, 8191, F32), _grouped(65536, 4096, 32, 196608, BF16),
             _grouped(65536, 1 << 20, 1, 1 << 20, F16), _gemm(4096, 32, 1 << 20, F32, ldx=1 << 23),
             _gemm(1 << 20, 64, 1 << 20, BF16), _gemm(130, 8192, 65600, F32), _gemm(256, 1 << 20, 70000, BF16)]
    for call, (rc, launches) in zip(calls, _record(recorder, calls)):
        assert rc == 0 and launches, call
        for _, k in launches:
            assert k[0] * k[3] < 1 << 32 and k[1:3] == [1, 1], (call, k)


def test_gpu_tests_reach_every_kernel(recorder):
    from tests import test_gpu_fp8 as sizes

    held = {_kernel(w[1]) for w in launch_recorder._run(recorder, []) if w[0] == "kernel"}
    held = {k for k in held if k[0].startswith("fp8_") and "quantize" not in k[0]}
    assert len(held) == 17
    calls = [_gemm(*s, out) for s in sizes.GEMM for out in (F32, F16, BF16)]
    calls += [_grouped(e, m, n, rows, out, ld) for e, m, n, _, rows in sizes.GROUPED for out in (F32, BF16)
              for ld in (n, _up(n, 16) * 16)]
    reached = set()
    for rc, launches in _record(recorder, calls):
        assert rc == 0
        reached |= {k for k, _ in launches}
    assert reached == held
