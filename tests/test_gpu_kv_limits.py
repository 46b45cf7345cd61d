"""The cache's attention where rounds, requests and codes are unusual: many
units to a CTA with NaN codes among them."""
import numpy as np
import pytest
import torch

import kv_util as ku
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_kvcache import as_type, flags, i32, new_ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,H,D", [(13, 4, 1, 128), (25, 4, 2, 64), (33, 4, 1, 128)])
def test_nan_codes_in_some_of_many_units(T, Hq, H, D):
    """Short requests, several units to a CTA, every third of them with a NaN
    value in the round: the rows that see it are NaN in its channel alone, the
    units before and after it are untouched, and every run gives the same."""
    rng = np.random.default_rng(21)
    B, P = 220, 16
    lens = rng.integers(0, 30, B)
    new = [T] * B
    total = [int(a) + T for a in lens]
    c = ku.random_cache(rng, sum(-(-x // P) for x in total), H, P, D)
    table = ku.tables(rng, c.k.shape[0], total, P)
    q, q64 = as_type(rng.normal(size=(B, T, Hq, D)), "bf16")
    out, lse, spr, xerr = ku.attention(q64, c, table, lens, new, None, 0.125)
    tol, _ = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
    bad = ku.Cache(c.k, c.v, c.ks, c.vs)
    want_nan = np.zeros(out.shape, bool)
    for b in range(0, B, 3):
        t, d, h = int(rng.integers(0, T)), int(rng.integers(0, D)), int(rng.integers(0, H))
        at = int(lens[b]) + t
        bad.v[table[b, at // P], h, at % P, d] = 0x7f
        G = Hq // H
        want_nan[b, t:, h * G:(h + 1) * G, d] = True
    dev = ku.to_device(bad)
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(B, T, Hq, H, D))
    run = lambda: sv.kv_attention(q, dev, i32(table), i32(lens), scale=0.125, ws=ws)["out"]
    got = run()
    assert flags(ws) == (sv.SV_OK, 0)
    o = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(o), want_nan)
    assert (np.abs(o - out) <= tol)[~want_nan].all()
    for _ in range(20):
        assert torch.equal(run().view(torch.int16), got.view(torch.int16))
    assert flags(ws) == (sv.SV_OK, 0)
