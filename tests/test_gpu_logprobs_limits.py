"""Log probabilities at the ends of their ranges, against the plain 64-bit
implementation (round_util)."""
import numpy as np
import pytest
import torch

import round_util as ru
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_kvcache import as_type, flags, i32, new_ws
from test_gpu_logprobs import f32

pytestmark = pytest.mark.gpu

# Largest logits of rows in which one token holds (nearly) everything: most of them times
# log2(e) / t are no fp32 numbers.
LARGEST = np.concatenate([[0.3, 20.1, 300.7, -5.9, 0.0, 1e-3, -1e4],
                          np.random.default_rng(5).uniform(-500, 500, 57)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,rest", [(1, None), (37, -np.inf), (37, -300.0), (5003, -np.inf),
                                    (40000, -60.0), (5003, -3.3e38)])
def test_no_log_probability_is_above_zero(dtype, V, rest):
    """... and no entropy below: one token left by a mask, or far ahead of the others."""
    n = len(LARGEST)
    x = np.empty((1, n, V))
    x[0] = -np.inf if rest in (None, -np.inf) else np.maximum(LARGEST[:, None] + rest, -3e38)
    x[0, np.arange(n), (np.arange(n) * 17) % V] = LARGEST
    x, x64 = as_type(x, dtype)
    best = i32([(np.arange(n) * 17) % V])
    for t in (None, 0.0, 0.7, 3.1):
        ws = new_ws()
        got = sv.token_logprobs(x, best, top=3, ws=ws, temperature=None if t is None else f32([t]))
        assert flags(ws) == (sv.SV_OK, 0)
        for name in ("logprobs", "top_logprobs"):
            assert (got[name] <= 0).all(), (name, float(got[name].max()))
        assert (got["entropy"] >= 0).all(), float(got["entropy"].min())
        for r in range(n):
            row = ru.Row(x64[0, r], 1.0 if t is None else t)
            lp_off, h_off = row.bounds()
            at = int(best[0, r])
            assert abs(float(got["logprobs"][0, r]) - row.lp[at]) <= lp_off[at]
            assert float(got["top_logprobs"][0, r, 0]) == float(got["logprobs"][0, r])
            assert abs(float(got["entropy"][0, r]) - row.entropy) <= h_off


def test_rows_without_values_keep_their_nan():
    """What is cut off at zero is no NaN."""
    x = torch.zeros(1, 3, 100, device="cuda")
    x[0, 1, 5] = float("nan")
    x[0, 2] = float("-inf")
    got = sv.token_logprobs(x, i32([[3, -1, 3]]), top=2, ws=new_ws())
    assert torch.isnan(got["entropy"][0, 1:]).all() and torch.isnan(got["logprobs"][0, 1:]).all()
    assert torch.isnan(got["top_logprobs"][0, 1:]).all()
    assert not torch.isnan(got["entropy"][0, 0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_temperatures_at_the_ends_of_fp32(dtype):
    """Subnormal ones count as the least normal one; the largest ones level the logits."""
    t = np.array([1e-45, 1e-40, 2.0 ** -127, 2.0 ** -126, 3e-38, 1e38, 3.4e38], np.float32)
    x = np.tile([0.0, -1e-3, 0.0, -1.0, -2.0 ** -120], (len(t), 1))[:, None]
    x, x64 = as_type(x, dtype)
    tokens = i32(np.tile(np.arange(5), (len(t), 1, 1)))
    ws = new_ws()
    got = sv.token_logprobs(x, tokens, temperature=f32(t), ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    for b in range(len(t)):
        row = ru.Row(x64[b, 0], max(float(t[b]), 2.0 ** -126))
        lp_off, h_off = row.bounds()
        lp = got["logprobs"][b, 0].double().cpu().numpy()
        assert (np.abs(lp - row.lp) <= lp_off).all(), (t[b], lp, row.lp)
        assert abs(float(got["entropy"][b, 0]) - row.entropy) <= h_off
