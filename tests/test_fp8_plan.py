"""Plans of the 8-bit products at sizes that were measured on several kernels,
recorded without a GPU."""
import pytest

from tests import launch_recorder
from tests.test_fp8_launches import BF16, F16, F32, _gemm, _grouped, _kind, _record

ROWS = "rows"


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return launch_recorder.build(str(tmp_path_factory.mktemp("recorder")))


# Rows of X, of W and columns, and the kernel that measured faster: rows, or a tile and
# its splits of the columns.
MEASURED = [
    # us on rows and on the tiles: 17.8 / 18.3, then 21.8 / 20.5, 22.0 / 20.8, 22.4 / 21.4, 26.1 / 21.7, 26.8 / 22.1
    (28, 11008, 4096, (ROWS, 1)), (34, 11008, 4096, (128, 64, 2)), (40, 11008, 4096, (128, 64, 2)),
    (48, 11008, 4096, (128, 64, 2)), (56, 11008, 4096, (128, 64, 2)), (64, 11008, 4096, (128, 64, 2)),
    # 13.5 / 16.2, 14.1 / 16.9, 17.0 / 18.0, 23.4 / 19.8
    (77, 4096, 4096, (ROWS, 1)), (96, 4096, 4096, (ROWS, 1)), (17, 4096, 11008, (ROWS, 1)), (33, 4096, 11008, (128, 64, 8)),
    # 4.7 / 7.3, 9.6 / 11.5, 16.9 / 11.9, 4.4 / 5.5, 7.1 / 5.5
    (256, 1024, 1024, (ROWS, 1)), (256, 2048, 2048, (ROWS, 1)), (512, 2048, 2048, (128, 32, 1)), (24, 8192, 512, (ROWS, 1)),
    (64, 8192, 512, (128, 32, 1)),
    # 128 x 128 with four splits 101, 128 x 64 with two 122
    (256, 12288, 12288, (128, 128, 4)), (1024, 11008, 4096, (128, 128, 1)),
]


@pytest.mark.parametrize("rows,m,n,want", MEASURED)
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_the_plan_is_the_faster_one(recorder, rows, m, n, want, out):
    rc, launches = _record(recorder, [_gemm(m, n, rows, out)])[0]
    kind = _kind(launches[0][0])
    assert rc == 0
    if kind[0] == ROWS:
        got = (ROWS, len(launches))
    else:
        tiles = -(-m // kind[0]) * -(-rows // kind[1])
        got = (*kind, max(s for s in range(1, 17) if -(-tiles * s // 8) * 8 == launches[0][1][0]))
        assert len(launches) == (1 if got[2] == 1 else 2)
    assert got == want


# Experts, all rows of X (spread over the experts by popularities), of W, columns, bytes
# from row to row, and the kernel that measured faster.
GROUPED = [
    # us on rows and on the tiles: 33.8 / 39.0, 36.4 / 37.9, 43.2 / 49.6
    (64, 512, 1030, 1300, 1312, (ROWS, 2)), (64, 512, 1408, 1536, 1536, (ROWS, 2)), (64, 512, 1030, 1999, 2000, (ROWS, 2)),
    # rows at odd addresses, 64 rows of W a workgroup: 49.8 / 45.6, 53.7 / 60.0, 62.8 / 72.3
    (64, 1536, 1030, 1100, 1101, "tiles"), (64, 1536, 1030, 1540, 1541, (ROWS, 4)), (64, 1536, 1030, 1999, 1999, (ROWS, 4)),
    # aligned: 73.1 / 83.6, 72.3 / 54.6
    (64, 1536, 1030, 4096, 4096, (ROWS, 4)), (64, 1536, 1408, 2304, 2304, (128, 64)),
    # 128 x 64 24.2, 128 x 32 30.5; 128 x 64 144, 128 x 128 141, 256 x 256 238; 128 x 128 767, 256 x 256 843;
    # 128 x 128 15.0, 128 x 32 22.4; many rows an expert, but small: 6.3 / 27, 19.6 / 44, 18.5 / 20, 17.5 / 11.4
    (64, 896, 1030, 1024, 1024, (128, 64)), (8, 3000, 4096, 4096, 4096, 128),
    (8, 8192, 11008, 4096, 4096, (128, 128)), (100, 3200, 512, 512, 512, (128, 128)),
    (2, 120, 128, 5312, 5312, (ROWS, 1)), (20, 457, 172, 9051, 9056, (ROWS, 2)), (20, 683, 488, 3162, 3168, (ROWS, 2)),
    (3, 147, 3780, 1062, 1072, "tiles"),
    # at odd addresses: 7.9 / 53, 19.1 / 87, 24.5 / 51
    (2, 120, 128, 5312, 5313, (ROWS, 1)), (20, 457, 172, 9051, 9051, (ROWS, 2)), (8, 1306, 256, 5376, 5377, (ROWS, 2)),
]


@pytest.mark.parametrize("experts,rows,m,n,ld,want", GROUPED)
@pytest.mark.parametrize("out", [F32, BF16])
def test_the_plan_by_expert_is_the_faster_one(recorder, experts, rows, m, n, ld, want, out):
    rc, launches = _record(recorder, [_grouped(experts, m, n, rows, out, ld)])[0]
    kind = _kind(launches[0][0])
    assert rc == 0 and len(launches) == 1
    assert kind == want or kind[0] == want or (want == "tiles" and kind[0] != ROWS)
