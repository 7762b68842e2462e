"""What the microscaled products launch, from their sizes alone: grids within
the limits of a launch, recorded without a GPU."""
import pytest

from tests import launch_recorder

F16, BF16, MX = 1, 2, 3
P = 0x1000                        # 16-byte aligned, never followed
MAX_YZ = 65535                    # workgroups along y and z


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return launch_recorder.build(str(tmp_path_factory.mktemp("recorder")))


def _up(a, b):
    return -(-a // b)


def _gemm(m, n, rows, x, ldx=None, ldp=None, out=0):
    words, blocks = ldp or _up(n, 8), _up(n, 32)
    if x == MX:
        return ("gptq_mx_scaled_gemm", [P, m, n, words, P, blocks, P, rows, ldx or _up(n, 8), P, blocks, P, out, m, P,
                                        1 << 50, None])
    return ("gptq_mx_gemm", [P, m, n, words, P, blocks, P, x, rows, ldx or n, P, out, m, P, 1 << 50, None])


def _record(recorder, calls):
    return launch_recorder.record(recorder, calls)


def test_the_sum_over_splits_stays_within_a_grid(recorder):
    # Split columns with more rows of X than a grid has along y.
    sizes = [(m, n, rows, x) for m, n, rows in ((130, 8192, 65600), (200, 8192, 70000), (256, 32768, 70000),
                                                (1, 1 << 20, 100000))
             for x in (F16, BF16, MX)]
    split = 0
    for (m, n, rows, x), (rc, launches) in zip(sizes, _record(recorder, [_gemm(*s) for s in sizes])):
        assert rc == 0
        for k in launches:
            assert k["grid"][1] <= MAX_YZ and k["grid"][2] <= MAX_YZ, (m, n, rows, x, k)
            if k["kernel"] == "mx_join_kernel":
                split += 1
                threads = k["grid"][0] * k["grid"][1] * k["block"][0]
                assert threads >= rows * _up(m, 4)
    assert split >= 4
