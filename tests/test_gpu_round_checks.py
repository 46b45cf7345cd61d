"""The debug build (-DSV_CHECKS) runs rotations, appends and log probabilities like
the release build, and none of its checks fires."""
import numpy as np
import pytest

import speculative_decoding_verification_63_gb300 as sv
from test_gpu_checks import checks_lib  # noqa: F401 (fixture)
from test_gpu_kvcache import as_type, flags, i32, new_ws
from test_gpu_logprobs import check
from test_gpu_rotate import check_append, near
import round_util as ru

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,dim,inter,dtype", [(1, 128, 128, False, "bf16"),
                                                 (70, 64, 32, True, "fp16"),
                                                 (9, 80, 80, False, "fp32")])
def test_rotate(checks_lib, T, D, dim, inter, dtype):  # noqa: F811
    rng = np.random.default_rng(31)
    rope = sv.rope(dim, interleaved=inter)
    x, x64 = as_type(rng.normal(size=(3, T, 5, D)), dtype)
    ws, start = new_ws(), [5, 0, 900]
    got = sv.rotate(x, start=i32(start), rope=rope, eps=1e-6, ws=ws)["q"]
    near(got, *ru.rotated(x64, ru.positions(start, None, 3, T), rope, None, 1e-6), dtype)
    assert flags(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("lens,new,T,H,P,D,dtype", [
    ([0, 5, 16, 31], [1, 1, 1, 1], 1, 2, 16, 64, "bf16"),
    ([0, 100, 127, 128, 129], [33, 33, 2, 32, 0], 33, 9, 128, 128, "bf16"),
    ([3, 64], [200, 131], 200, 2, 64, 128, "fp32"),
])
def test_append(checks_lib, lens, new, T, H, P, D, dtype):  # noqa: F811
    rng = np.random.default_rng(32)
    check_append(rng, lens, new, T, 4, H, P, D, dtype, sv.rope(64), 1e-6)


@pytest.mark.parametrize("B,N,V,dtype,top", [(1, 1, 128256, "bf16", 20), (3, 4, 32003, "fp32", 5),
                                             (2, 90, 4099, "bf16", 64), (1, 1, 1 << 20, "fp32", 1)])
def test_logprobs(checks_lib, B, N, V, dtype, top):  # noqa: F811
    rng = np.random.default_rng(33)
    x, x64 = as_type(rng.normal(size=(B, N, V)), dtype)
    tokens, ws = rng.integers(0, V, (B, N)), new_ws()
    got = sv.token_logprobs(x, i32(tokens), top=top, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    check(x64, got, tokens, top)


def test_logprobs_of_equal_logits(checks_lib):  # noqa: F811
    x, x64 = as_type(np.zeros((1, 2, 40000)), "bf16")
    ws = new_ws()
    got = sv.token_logprobs(x, top=20, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    check(x64, got, top=20)
