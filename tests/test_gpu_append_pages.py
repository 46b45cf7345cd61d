"""Appends whose pages take blocks of 512 threads, two chunks a thread (pages of 128
tokens, heads of 128 channels, more than 64 tokens a request): each type and kind of
pairs, in the release and the debug build."""
import numpy as np
import pytest

import speculative_decoding_verification_63_gb300 as sv
from speculative_decoding_verification_63_gb300 import _binding, _build
from test_gpu_rotate import check_append

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["release", "debug"])
def build(request):
    old = _binding.lib()
    if request.param == "debug":
        _binding._lib_handle = _binding.lib(_build.build_library(checks=True))
    try:
        yield request.param
    finally:
        _binding._lib_handle = old


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,H,dim,norm", [(65, 3, 1, 128, True), (130, 8, 5, 48, True),
                                             (257, 4, 2, 128, False)])
def test_blocks_of_512_threads(build, T, Hq, H, dim, norm, inter, dtype):
    """Pages begun and full ones, requests with a token, with none and with all."""
    rng = np.random.default_rng(T + dim)
    lens, new = [0, 1, 127, 128, 100, 63], [T, T, T, 1, 0, T - 1]
    check_append(rng, lens, new, T, Hq, H, 128, 128, dtype,
                 sv.rope(dim, 5e5, interleaved=inter), 1e-6 if norm else None)
