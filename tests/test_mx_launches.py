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


def _grouped(experts, m, n, rows, x, out=2):
    words, blocks = _up(n, 8), _up(n, 32)
    return ("gptq_mx_gemm_grouped", [P, experts, m, n, words, m * words, P, blocks, m * blocks, P, x, rows, n, P, P, out,
                                     m, None, 0, None])


def test_a_launch_has_fewer_than_2_to_the_32_threads(recorder):
    # Many experts with many rows of W on the row kernel and on tiles, and rows
    # of X too far apart for the tiles on the row kernel: parts of W's rows.
    calls = [_grouped(2048, 131072, 8, 8191, F16), _grouped(8192, 131072, 8, 34768, BF16),
             _grouped(65536, 4096, 32, 196608, BF16), _grouped(65536, 65536, 8, 262144, BF16), _grouped(65536, 1 << 20, 1, 1 << 20, F16),
             _gemm(4096, 32, 1 << 20, F16, ldx=3000000), _gemm(1 << 20, 64, 1 << 17, MX, ldx=1 << 21)]
    for call, (rc, launches) in zip(calls, _record(recorder, calls)):
        assert rc == 0 and len(launches) > 1, call
        for k in launches:
            assert k["grid"][0] * k["block"][0] < 1 << 32 and k["grid"][1:] == (1, 1), (call, k)


def test_usual_sizes_take_one_launch(recorder):
    calls = [_gemm(49152, 12288, 2048, F16), _gemm(1 << 20, 9216, 20, BF16), _grouped(64, 1024, 2048, 1531, F16),
             _grouped(1024, 1024, 9216, 20, BF16), _gemm(49152, 640, 80, F16, ldx=3000000)]
    for call, (rc, launches) in zip(calls, _record(recorder, calls)):
        assert rc == 0 and len(launches) == 1, call


def _kind(launch):
    """Kernel of a product, tiles as (W rows, X rows)."""
    k, a = launch["kernel"], launch["args"]
    if k in ("mx_tile_kernel", "mx_big_tile_kernel"):
        return 32 * a[1] * a[3], 32 * a[2] * a[4]
    return {"mx_rows_kernel": "rows", "mx_stream_kernel": "stream"}[k]


# Rows of X, of W and columns of sizes measured on two kernels, and the faster one.
MEASURED = [
    (64, 4096, 4096, MX, "rows"), (128, 4096, 4096, MX, (128, 32)), (8, 11008, 4096, MX, "rows"),
    (32, 11008, 4096, MX, (128, 32)), (512, 4096, 4096, MX, (128, 64)), (2048, 4096, 4096, MX, (128, 128)),
    (4096, 12288, 12288, MX, (256, 256)),
    (32, 4096, 4096, F16, "rows"), (64, 4096, 4096, F16, (128, 32)), (1, 4096, 11008, F16, "rows"),
    (4, 11008, 4096, F16, (128, 32)), (2, 4099, 11007, F16, (128, 32)), (8, 130, 1001, F16, "rows"),
    (1, 49152, 12288, F16, "stream"), (1, 28672, 8192, F16, "stream"), (1, 12288, 12288, F16, (128, 32)),
    (256, 4096, 4096, BF16, (128, 32)), (256, 11008, 4096, BF16, (128, 64)), (2048, 11008, 4096, BF16, (256, 128)),
    (4096, 8192, 8192, BF16, (256, 256)),
]


@pytest.mark.parametrize("rows,m,n,x,want", MEASURED)
def test_the_plan_takes_the_kernel_that_measured_faster(recorder, rows, m, n, x, want):
    rc, launches = _record(recorder, [_gemm(m, n, rows, x)])[0]
    assert rc == 0 and _kind(launches[0]) == want


def test_gpu_tests_reach_every_kernel(recorder):
    """The sizes of the parity tests launch every kernel of the products in the
    library; those with scales that float16 does not hold, every one that
    multiplies float16 X."""
    from tests import test_gpu_mx as sizes

    def reached(calls):
        out = set()
        for rc, launches in _record(recorder, calls):
            assert rc == 0
            out |= {(k["kernel"], k["args"]) for k in launches}
        return out

    held = {k for k in launch_recorder.kernels(recorder) if k[0].startswith("mx_") and k[0] != "mx_quantize_kernel"}
    assert len(held) > 40
    shapes = sizes.GEMM + sizes.KINDS + sizes.ENDS
    large = [(4, m, n, 3000) for m, n in ((4096, 2048), (4099, 2056), (4090, 2061))]
    grouped = [(e, m, n, rows) for e, m, n, _, rows in sizes.GROUPED] + large
    assert reached([_gemm(*s, x) for s in shapes for x in (F16, BF16, MX)] +
                   [_grouped(*s, x) for s in grouped for x in (F16, BF16)]) == held
    far = [_gemm(*s, F16) for s in sizes.ENDS + sizes.FAR_MORE]
    far += [_grouped(e, m, n, rows, F16) for e, m, n, _, rows in sizes.GROUPED] + [_grouped(*s, F16) for s in large]
    assert {k for k in held if k[1][:1] == (F16,)} <= reached(far)
