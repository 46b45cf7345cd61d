"""The debug build (-DSV_CHECKS) runs the cache's calls like the release build,
and none of its checks fires."""
import numpy as np
import pytest

import kv_util as ku
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_checks import checks_lib  # noqa: F401 (fixture)
from test_gpu_kvcache import as_type, check_attention, flags, i32, new_ws, same_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new,H,P,D,dtype,T", [
    ([0, 5, 16, 31], [1, 1, 1, 1], 2, 16, 64, "bf16", 1),
    ([0, 100, 127, 128, 129], [33, 33, 2, 32, 0], 1, 128, 128, "bf16", 33),
    ([3, 64], [200, 131], 2, 64, 128, "fp32", 200),
])
def test_write_and_read(checks_lib, lens, new, H, P, D, dtype, T):  # noqa: F811
    rng = np.random.default_rng(81)
    total = [a + n for a, n in zip(lens, new)]
    ref = ku.random_cache(rng, sum(-(-x // P) for x in total), H, P, D)
    table = ku.tables(rng, ref.k.shape[0], total, P)
    dev, ws = ku.to_device(ref), new_ws()
    k, k64 = as_type(rng.normal(size=(len(lens), T, H, D)), dtype)
    ref.write(table, lens, new, k64, k64)
    sv.kv_write(dev, i32(table), i32(lens), k, k, num_new=i32(new), ws=ws)
    same_cache(dev, ref)
    rows = np.tile(np.arange(T, dtype=np.int32), (len(lens), 1))
    for r in (None, i32(rows)):
        got = sv.kv_read(dev, i32(table), i32(lens), i32(new), T, rows=r, ws=ws)
        for b, n in enumerate(new):
            want = ref.values("v", table[b], lens[b] + np.arange(n))
            assert np.array_equal(got["v"][b, :n].double().cpu().numpy(), want)
    assert flags(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("lens,new,T,Hq,H,P,D,dtype", [
    ([0, 1, 14, 15, 16, 63, 64, 65], [1] * 8, 1, 8, 2, 16, 128, "bf16"),
    ([6001], [5], 5, 16, 1, 128, 128, "bf16"),
    ([2000], [3], 3, 12, 12, 16, 64, "fp16"),
    ([37, 0, 300], [200, 150, 77], 200, 4, 2, 64, 128, "bf16"),
    ([77, 0, 64, 129], [25, 24, 1, 0], 25, 4, 2, 16, 64, "bf16"),
])
def test_attention(checks_lib, lens, new, T, Hq, H, P, D, dtype):  # noqa: F811
    check_attention(np.random.default_rng(82), lens, new, T, Hq, H, P, D, dtype)


def test_attention_tree(checks_lib):  # noqa: F811
    rng = np.random.default_rng(83)
    check_attention(rng, [1000, 31], [33, 32], 33, 10, 2, 128, 128, "bf16",
                    mask=ku.random_tree_mask(rng, 2, 33))
