"""What the router and the layers of experts launch, recorded without a GPU."""
import re

import pytest

from tests import launch_recorder

F32, F16, BF16 = 0, 1, 2
P = 0x1000                        # 16-byte aligned, never followed
LDS = 160 * 1024                  # of a CU
NAME = re.compile(r"_ZN\w*?\d+(moe_\w+?_kernel)(?:I((?:L[ib]\d+E)+)E)?E")


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


def _route(tokens, experts, k, dtype=F32):
    return ("gptq_moe_route", [P, dtype, tokens, experts, experts, k, 1, P, P, P, P, None])


def _layer(fmt, tokens, experts, k, d, f, dtype):
    if fmt == "mx":
        gu, dn = (_up(d, 8), 2 * f * _up(d, 8), _up(d, 32), 2 * f * _up(d, 32)), (_up(f, 8), d * _up(f, 8), _up(f, 32), d * _up(f, 32))
    else:
        gu = d, 2 * f * d, _up(d, 128), _up(2 * f, 128) * _up(d, 128)
        dn = f, d * f, _up(f, 128), _up(d, 128) * _up(f, 128)
    return (f"gptq_{fmt}_moe", [P, gu[0], gu[1], P, gu[2], gu[3], P, dn[0], dn[1], P, dn[2], dn[3], experts, d, f, P, dtype,
                                tokens, d, P, F32, experts, k, 1, P, F32, d, P, 1 << 50, None])


def test_gpu_tests_reach_every_kernel(recorder):
    from tests import test_gpu_moe as sizes

    held = {_kernel(w[1]) for w in launch_recorder._run(recorder, []) if w[0] == "kernel"}
    held = {k for k in held if k[0].startswith("moe_")}
    assert len(held) == 15
    calls = [_route(*r) for r in sizes.ROUTES]
    calls += [_layer(fmt, *s, dtype) for s in sizes.LAYERS for fmt in ("mx", "block") for dtype in (F16, BF16)]
    reached = set()
    for rc, launches in _record(recorder, calls):
        assert rc == 0 and 1 <= len(launches) <= 3
        reached |= {k for k, _ in launches}
    assert reached == held


def test_a_layer_is_two_launches_three_for_many_tokens_within_their_limits(recorder):
    sizes = [(64, 1024, 16, 1 << 20, 1 << 19), (64, 1024, 16, 64, 64), (1, 1, 1, 1 << 20, 1), (64, 1, 1, 1, 1 << 19),
             (1, 8, 2, 4096, 11008), (16, 64, 6, 2048, 1024)]
    calls = [_layer(fmt, *s, dtype) for s in sizes for fmt in ("mx", "block") for dtype in (F16, BF16)]
    for call, (rc, launches) in zip(calls, _record(recorder, calls)):
        assert rc == 0 and len(launches) == (3 if call[1][-13] > 16 else 2), call
        for _, k in launches:
            assert k[0] >= 1 and k[0] * k[3] < 1 << 32 and k[1:3] == [1, 1] and k[6] <= LDS - 64, (call, k)


def test_few_tokens_route_in_one_launch(recorder):
    for tokens, experts, want in ((1, 100, 1), (16, 1024, 1), (17, 120, 1), (64, 32, 1), (64, 33, 2), (17, 121, 2), (65, 4, 2),
                                  (1 << 20, 100, 2)):
        rc, launches = _record(recorder, [_route(tokens, experts, 4)])[0]
        assert rc == 0 and len(launches) == want, (tokens, experts)
        for _, k in launches:
            assert k[0] * k[3] < 1 << 32
