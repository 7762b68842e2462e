"""The routes that the GPU tests compare with the oracle reach the router in one
workgroup with more than one token a wave; recorded without a GPU."""
import pytest

from tests import launch_recorder
from tests.test_gpu_moe_route import ROUTES
from tests.test_moe_launches import _record, _route


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return launch_recorder.build(str(tmp_path_factory.mktemp("recorder")))


def test_routes_of_17_to_64_tokens_take_one_workgroup(recorder):
    assert min(t for t, _, _ in ROUTES) == 17 and max(t for t, _, _ in ROUTES) == 64
    for rc, launches in _record(recorder, [_route(*r) for r in ROUTES]):
        assert rc == 0 and [k[0] for k, _ in launches] == ["moe_route_kernel"]
        assert launches[0][1][:3] == [1, 1, 1]
