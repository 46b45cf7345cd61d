"""Log probabilities at the ends of their ranges, against the plain 64-bit
implementation (round_util)."""
import numpy as np
import pytest
import torch

import round_util as ru
import speculative_decoding_verification_63_gb300 as sv
from speculative_decoding_verification_63_gb300 import _binding, _build
from test_gpu_kvcache import as_type, flags, i32, new_ws
from test_gpu_logprobs import check, f32

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


# ------------------------------------------- the search for the likeliest groups

def spread_over_a_warp(rng, V, cluster):
    """Different logits, the largest all in the groups of one warp of one CTA of the row's
    (every 8 * cluster-th 32 groups): more groups than a CTA reads again reach the bound."""
    group = np.arange(V) // 16
    return rng.normal(size=V) + 10.0 * ((group // 32) % (8 * cluster) == 5 * cluster + cluster - 1)


SEARCHED = {
    "constant": lambda rng, V, cluster: np.full(V, -2.5),
    "two values": lambda rng, V, cluster: np.where(rng.random(V) < 0.02, 2.0, 1.0),
    "a few above": lambda rng, V, cluster: np.where(rng.random(V) < 30 / V, 2.0, 1.0) +
    (rng.random(V) < 10 / V),
    "integers": lambda rng, V, cluster: rng.integers(-3, 4, V).astype(float),
    "lowest": lambda rng, V, cluster: np.where(rng.random(V) < 1 - 40 / V, -3e38,
                                               rng.normal(size=V)),
    "a warp": spread_over_a_warp,
}


@pytest.fixture(params=["release", "debug"])
def build(request):
    old = _binding.lib()
    if request.param == "debug":
        _binding._lib_handle = _binding.lib(_build.build_library(checks=True))
    try:
        yield
    finally:
        _binding._lib_handle = old


@pytest.mark.parametrize("kind", list(SEARCHED))
@pytest.mark.parametrize("rows,cluster,dtype,V", [
    (5, 8, "bf16", 160016), (5, 8, "fp32", 300016), (40, 4, "fp32", 300016), (40, 4, "bf16", 20011),
    (200, 2, "bf16", 160016), (200, 2, "fp32", 80003), (700, 1, "bf16", 80000),
    (700, 1, "fp32", 40003)])
def test_many_logits_reach_the_bound(build, kind, rows, cluster, dtype, V):
    """A row by 1, 2, 4 and 8 CTAs; two rows by their definition, the others are the same."""
    rng = np.random.default_rng(V + rows)
    x, x64 = as_type(np.stack([SEARCHED[kind](rng, V, cluster) for _ in range(2)])[None], dtype)
    if kind == "lowest":
        x = torch.where(x < -1e38, torch.finfo(x.dtype).min, x)
        x64 = x.double().cpu().numpy()
    many = x.expand(rows // 2 + 1, 2, V).contiguous().view(1, -1, V)[:, :rows]
    for top in (1, 20, 64):
        ws = new_ws()
        got = sv.token_logprobs(many, top=top, ws=ws)
        assert flags(ws) == (sv.SV_OK, 0)
        check(x64, {n: t[:, :2] for n, t in got.items()}, top=top)
        for i in range(2):
            # (rows that begin at other places of 32 bytes have other groups and orders of
            # sums: the same tokens, and values that are each within the bounds)
            lp_off, h_off = ru.Row(x64[0, i]).bounds()
            ids = got["top_tokens"][0, i::2]
            assert (ids == ids[:1]).all()
            there = ids[0].cpu().numpy()
            off = 2 * torch.from_numpy(np.where(there < 0, 0.0, lp_off[there])).cuda()
            best, entropy = got["top_logprobs"][0, i::2], got["entropy"][0, i::2]
            same = best == best[:1]  # (-inf too)
            assert (same | ((best - best[:1]).abs() <= off)).all()
            assert ((entropy - entropy[0]).abs() <= 2 * h_off).all()


# ------------------------------------------------------------- long rows

def long_bounds(row, turns, groups):
    """Of a row's log probabilities and its entropy, for any data, where a thread takes
    `turns` turns of `groups` groups, in units of 2^-24 of Z.  A weight: ex2 is off by 4;
    its exponent's roundings (c, the product and sum: 3 of itself) and those of the rises
    behind it (3 of each, which together are the exponent that is left) are 6 times the
    mean distance to the maximum.  A rise, at most one a turn and three on the way from
    thread to row: ex2 (4) and a product (1).  Additions: 8 a group, one for the pair and
    one a turn, 5 in the warp, 2 and 5 over the warps.  The logarithm, the reference and
    the differences: 4 of what they are made of (round_util.Row.bounds)."""
    z = (4 + 5 * (turns + 3) + 8 * groups + 1 + turns + 12 + 6 * row.spread) * 2.0 ** -24
    with np.errstate(invalid="ignore"):
        d = np.abs(row.x - row.m) / row.t
    lp = z + 4 * 2.0 ** -24 * (d + abs(row.log_z))
    h = z * (1 + 2 * row.spread) + 8 * 2.0 ** -24 * (abs(row.log_z) + row.spread)
    return np.where(np.isfinite(lp), lp, 0.0), h


LONG = {
    "ascending": lambda rng, V: np.linspace(-20, 20, V),
    "barely ascending": lambda rng, V: np.linspace(0, 0.01, V),
    "slowly ascending": lambda rng, V: np.linspace(0, 1, V),
    "steps": lambda rng, V: np.arange(V) // 8192 * 0.05,
    "descending": lambda rng, V: np.linspace(20, -20, V),
    "random": lambda rng, V: rng.normal(size=V),
}


@pytest.mark.parametrize("kind", list(LONG))
@pytest.mark.parametrize("dtype,groups", [("bf16", 4), ("fp32", 2)])
@pytest.mark.parametrize("V", [1 << 20, 152064])
def test_long_rows_by_one_cta(kind, dtype, groups, V):
    """More rows than run at once, the same one: up to 128 turns a thread, whose reference
    rises at every one of them."""
    rng = np.random.default_rng(9)
    x, x64 = as_type(LONG[kind](rng, V), dtype)
    row = ru.Row(x64)
    lp_off, h_off = long_bounds(row, -(-(V // 16) // (256 * groups)), groups)
    tokens = np.array([0, V // 3, V - 1, int(np.argmax(x64))])
    ws = new_ws()
    got = sv.token_logprobs(x.expand(1, 700, V), i32(np.tile(tokens, (1, 700, 1))), ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    lp = got["logprobs"].double().cpu().numpy()
    assert (np.abs(lp - row.lp[tokens]) <= lp_off[tokens]).all()
    assert (np.abs(got["entropy"].double().cpu().numpy() - row.entropy) <= h_off).all()
