"""Log probabilities, entropies and likeliest tokens on the GPU against the
plain 64-bit implementation (round_util)."""
import numpy as np
import pytest
import torch

import round_util as ru
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_kvcache import as_type, flags, i32, new_ws

pytestmark = pytest.mark.gpu


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def check(x64, got, tokens=None, top=0, rows=None, num=None, temperature=None, R=None):
    """got against the definition, row by row."""
    B, N, V = x64.shape
    R = R or N
    ent = got["entropy"].cpu().numpy()
    lps = got["logprobs"].cpu().numpy().reshape(B, R, -1) if tokens is not None else None
    for b in range(B):
        n = R if num is None else num[b]
        assert np.isnan(ent[b, n:]).all()
        if top:
            assert (got["top_tokens"][b, n:].cpu() == -1).all()
            assert torch.isnan(got["top_logprobs"][b, n:]).all()
        for r in range(n):
            if (x64[b, r if rows is None else rows[b][r]] == -np.inf).all():  # no mass
                assert np.isnan(ent[b, r])
                assert not top or (got["top_tokens"][b, r].cpu() == -1).all()
                assert tokens is None or np.isnan(lps[b, r]).all()
                continue
            row = ru.Row(x64[b, r if rows is None else rows[b][r]],
                         1.0 if temperature is None else temperature[b])
            lp_off, h_off = row.bounds()
            assert abs(ent[b, r] - row.entropy) <= h_off, (b, r, ent[b, r], row.entropy, h_off)
            if tokens is not None:
                for i, t in enumerate(np.asarray(tokens[b][r]).reshape(-1)):
                    if t < 0:
                        assert np.isnan(lps[b, r, i])
                    elif row.lp[t] == -np.inf:
                        assert lps[b, r, i] == -np.inf
                    else:
                        assert abs(lps[b, r, i] - row.lp[t]) <= lp_off[t]
            if top:
                want = row.top(top)
                ids = got["top_tokens"][b, r].cpu().numpy()
                best = got["top_logprobs"][b, r].cpu().numpy()
                assert np.array_equal(ids[:len(want)], want), (b, r, ids[:8], want[:8])
                assert (ids[len(want):] == -1).all() and (best[len(want):] == -np.inf).all()
                assert (np.abs(best[:len(want)] - row.lp[want]) <= lp_off[want]).all()


CASES = [  # B, N, V, dtype, top, M
    (1, 1, 1, "bf16", 1, 1),
    (2, 3, 2, "fp32", 5, 2),
    (3, 2, 15, "bf16", 20, 1),
    (2, 2, 16, "bf16", 16, 3),
    (2, 5, 17, "fp32", 1, 0),
    (1, 4, 250, "bf16", 64, 7),
    (2, 3, 4097, "bf16", 5, 300),
    (1, 7, 32000, "bf16", 0, 1),
    (2, 3, 32003, "fp32", 20, 1),
    (1, 2, 128256, "bf16", 64, 1),
    (3, 7, 50001, "bf16", 5, 1),
    (40, 41, 4099, "bf16", 3, 1),
    (30, 50, 1000, "fp32", 1, 0),
    (1, 1, 1 << 20, "fp32", 20, 2),
    (1, 3, 1 << 20, "bf16", 64, 1),
]


@pytest.mark.parametrize("B,N,V,dtype,top,M", CASES)
def test_rows(B, N, V, dtype, top, M):
    rng = np.random.default_rng(V + N)
    x, x64 = as_type(rng.normal(size=(B, N, V)) * 3 - 1.1 * np.log(np.arange(1, V + 1)), dtype)
    t = rng.choice([0.0, 0.3, 0.8, 1.0, 2.5], B).astype(np.float32)
    num = rng.integers(0, N + 1, B)
    num[0] = N
    tokens = rng.integers(-1, V, (B, N, M)) if M else None
    if M == 1:
        tokens = tokens[:, :, 0]
    ws = new_ws()
    got = sv.token_logprobs(x, None if tokens is None else i32(tokens), num_rows=i32(num),
                            temperature=f32(t), top=top, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    check(x64, got, tokens, top, num=num, temperature=t)
    # without anything optional: the same entropies at temperature 1
    got = sv.token_logprobs(x, ws=ws)
    assert set(got) == {"entropy"}
    check(x64, got)


@pytest.mark.parametrize("dtype,V,pad,off", [("bf16", 32001, 3, 1), ("bf16", 5000, 8, 7),
                                             ("fp32", 9001, 1, 3), ("bf16", 7, 9, 5)])
def test_unaligned_and_strided_rows(dtype, V, pad, off):
    """Rows that begin anywhere, with logits around them that are not theirs."""
    rng = np.random.default_rng(V)
    B, N = 2, 6
    buf = torch.full((B * N * (V + pad) + off + 64,), 3e4, dtype=ru.TYPES[dtype], device="cuda")
    x, x64 = as_type(rng.normal(size=(B, N, V)), dtype)
    view = buf[off:off + B * N * (V + pad)].view(B, N, V + pad)[:, ::2, :V]
    view.copy_(x[:, ::2])
    tokens = rng.integers(0, V, (B, 3))
    got = sv.token_logprobs(view, i32(tokens), top=5)
    check(x64[:, ::2], got, tokens, 5)


ROWS = {
    "constant": lambda rng, V: np.full(V, -2.5),
    "integers": lambda rng, V: rng.integers(-3, 4, V).astype(float),
    "ascending": lambda rng, V: np.linspace(-20, 20, V),
    "descending": lambda rng, V: np.linspace(20, -20, V),
    "two values": lambda rng, V: np.where(np.arange(V) % 5 == 3, 2.0, 1.0),
    "lowest": lambda rng, V: np.where(rng.random(V) < 0.9995, LOWEST, rng.normal(size=V)),
    "one and lowest": lambda rng, V: np.where(np.arange(V) == V // 3, 0.5, LOWEST),
    "masked": lambda rng, V: np.where(rng.random(V) < 0.9995, -np.inf, rng.normal(size=V)),
    "one": lambda rng, V: np.where(np.arange(V) == V - 1, 0.5, -np.inf),
    "peaked": lambda rng, V: rng.normal(size=V) + 30.0 * (np.arange(V) == V // 2),
    # the largest all in the groups of a few threads
    "one thread": lambda rng, V: np.where(np.arange(V) // 16 % 256 == 7, 5.0, 0.0) +
    0.01 * rng.normal(size=V),
    "large": lambda rng, V: rng.normal(size=V) * 1e4,
    "zeros of both signs": lambda rng, V: np.where(rng.random(V) < 0.5, -0.0, 0.0),
    "block": lambda rng, V: np.where((np.arange(V) > 100) & (np.arange(V) < 1200), 4.0, 0.0),
}
LOWEST = -3e38


@pytest.mark.parametrize("kind", list(ROWS))
@pytest.mark.parametrize("dtype,V", [("bf16", 40000), ("fp32", 20011), ("bf16", 300)])
def test_unusual_rows(kind, dtype, V):
    rng = np.random.default_rng(17)
    x, x64 = as_type(np.stack([ROWS[kind](rng, V) for _ in range(3)])[None], dtype)
    if "lowest" in kind:
        x = torch.where(x < -1e38, torch.finfo(x.dtype).min, x)
        x64 = x.double().cpu().numpy()
    tokens = np.stack([np.array([0, V // 3, V // 2, V - 1])] * 3)[None]
    many = torch.cat([x] * 500) if V == 40000 else x  # a CTA a row
    # (of 300 masked logits none may be left)
    mass = (x64 > -np.inf).any(-1).all()
    state = (sv.SV_OK, 0) if mass else (sv.SV_EDATA, sv.SV_DERR_MASS)
    for top in (1, 20, 64):
        ws = new_ws()
        got = sv.token_logprobs(x, i32(tokens), top=top, ws=ws)
        assert flags(ws) == state
        check(x64, got, tokens, top)
        if many is not x:
            all_ = sv.token_logprobs(many, top=top, ws=ws)
            assert flags(ws) == (sv.SV_OK, 0)
            assert (all_["top_tokens"] == got["top_tokens"]).all()
            off = max(ru.Row(r).bounds()[1] for r in x64[0])
            assert ((all_["entropy"] - got["entropy"]).abs() <= 2 * off).all()


def test_bad_rows():
    """NaN, +inf, rows without mass, row indices, counts, temperatures and tokens:
    each reported, and only the rows concerned are without values."""
    V = 1000
    rng = np.random.default_rng(18)
    clean, x64 = as_type(rng.normal(size=(4, 3, V)), "fp32")
    tokens = np.array([[[1, 2]] * 3] * 4)

    def call(x=None, rows=None, num=None, t=None, tok=tokens, want=None):
        ws = new_ws()
        got = sv.token_logprobs(clean if x is None else x, i32(tok), R=3,
                                rows=None if rows is None else i32(rows),
                                num_rows=None if num is None else i32(num),
                                temperature=None if t is None else f32(t), top=4, ws=ws)
        assert flags(ws) == (sv.SV_EDATA, want)
        return got

    def gone(got, rows):
        bad = torch.isnan(got["entropy"]).cpu().numpy()
        assert np.array_equal(np.argwhere(bad), np.array(rows))
        bad = torch.from_numpy(bad).cuda()
        assert torch.isnan(got["logprobs"][bad]).all() and (got["top_tokens"][bad] == -1).all()
        assert torch.isnan(got["top_logprobs"][bad]).all()
        assert not torch.isnan(got["logprobs"][~bad]).any()
        assert (got["top_tokens"][~bad] >= 0).all()

    for value, at in ((np.nan, 0), (np.nan, 999), (np.inf, 500)):
        x = clean.clone()
        x[2, 1, at] = value
        gone(call(x, want=sv.SV_DERR_NONFINITE), [[2, 1]])
    x = clean.clone()
    x[0, 2] = -np.inf
    gone(call(x, want=sv.SV_DERR_MASS), [[0, 2]])
    rows = np.array([[0, 1, 2], [2, 2, 3], [0, -1, 0], [1, 0, 1]])
    got = call(rows=rows, want=sv.SV_DERR_ARG)
    gone(got, [[1, 2], [2, 1]])
    assert torch.equal(got["entropy"][3, 0], got["entropy"][3, 2])
    gone(call(num=[3, 4, 3, -1], want=sv.SV_DERR_ARG), [[1, 0], [1, 1], [1, 2], [3, 0], [3, 1],
                                                        [3, 2]])
    gone(call(t=[1, -1, np.nan, np.inf], want=sv.SV_DERR_ARG),
         [[b, r] for b in (1, 2, 3) for r in range(3)])
    tok = tokens.copy()
    tok[1, 1, 0], tok[2, 2, 1] = V, -2
    got = call(tok=tok, want=sv.SV_DERR_TOKEN)
    assert torch.isnan(got["logprobs"]).sum() == 2
    assert torch.isnan(got["logprobs"][1, 1, 0]) and torch.isnan(got["logprobs"][2, 2, 1])


def test_temperatures():
    """From 1e-30, where the largest logits share everything, to 1e30, where all
    are equal."""
    rng = np.random.default_rng(19)
    V = 3000
    x64 = np.repeat(rng.normal(size=(1, 1, V)), 5, 0)
    x64[:, :, 7] = x64[:, :, 1700] = 9.0
    x, x64 = as_type(x64, "fp32")
    t = np.array([1e-30, 1e-3, 0.0, 1e3, 1e30])
    got = sv.token_logprobs(x, i32([[1700]] * 5), temperature=f32(t), top=3)
    check(x64, got, [[1700]] * 5, 3, temperature=t)
    assert abs(float(got["logprobs"][0, 0]) + np.log(2)) < 1e-6


def test_path_rows():
    """Rows of a tree, by node; the same row twice."""
    rng = np.random.default_rng(20)
    B, N, V = 3, 9, 5003
    x, x64 = as_type(rng.normal(size=(B, N, V)) * 2, "bf16")
    rows = np.array([[0, 3, 8, -1], [0, 0, 0, 0], [0, -1, -1, -1]])
    num = np.array([3, 4, 1])
    tokens = rng.integers(0, V, (B, 4))
    ws = new_ws()
    got = sv.token_logprobs(x, i32(tokens), rows=i32(rows), num_rows=i32(num), top=2, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    check(x64, got, tokens, 2, rows=rows, num=num, R=4)


def test_rows_past_32_bits():
    """Rows more than 2^32 logits apart."""
    V, stride = 1003, (1 << 32) + 5
    buf = torch.zeros(2 * stride + 1000 + V, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(21)
    x, x64 = as_type(rng.normal(size=(1, 3, V)), "bf16")
    view = buf.as_strided((1, 3, V), (0, stride, 1))
    view.copy_(x)
    got = sv.token_logprobs(view, i32([[1, 2, 3]]), top=4)
    check(x64, got, [[1, 2, 3]], 4)


def test_in_a_graph_and_on_a_side_stream():
    rng = np.random.default_rng(22)
    x, _ = as_type(rng.normal(size=(2, 5, 32000)), "bf16")
    tokens, num = i32(rng.integers(0, 32000, (2, 5))), i32([5, 3])
    want = sv.token_logprobs(x, tokens, num_rows=num, top=5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), 7.0), torch.nan_to_num(b.float(), 7.0))
    with torch.cuda.stream(s):
        other = sv.token_logprobs(x, tokens, num_rows=num, top=5)
        with torch.cuda.graph(g, stream=s):
            got = sv.token_logprobs(x, tokens, num_rows=num, top=5)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert same(got[n], want[n]) and same(other[n], want[n]), n


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("B,N,V,dtype", [(5, 128, 40003, "bf16"), (5, 128, 20003, "fp32"),
                                         (1, 40, 300001, "bf16"), (1, 9, 300001, "fp32"),
                                         (2, 17, 41, "bf16"), (2, 17, 1003, "fp32")])
def test_one_bad_logit_anywhere(B, N, V, dtype, top):
    """A NaN or +inf at the row's ends and all over it, before and behind ordinary
    logits of the same thread, at the first, the next turn or in an edge's group:
    the row is without values and its neighbours keep theirs."""
    rng = np.random.default_rng(V + N)
    x, _ = as_type(rng.normal(size=(B, N, V)), dtype)
    at = np.linspace(0, V - 1, B * N).astype(int).reshape(B, N)
    for value in (np.nan, np.inf):
        bad = x.clone()
        for b in range(B):
            for r in range(0, N, 2):
                bad[b, r, at[b, r]] = value
        ws = new_ws()
        got = sv.token_logprobs(bad, i32(np.zeros((B, N))), top=top, ws=ws)
        assert flags(ws) == (sv.SV_EDATA, sv.SV_DERR_NONFINITE)
        for name in ("entropy", "logprobs") + (("top_logprobs",) if top else ()):
            gone = torch.isnan(got[name]).cpu().numpy().reshape(B, N, -1)
            assert gone[:, ::2].all(), (name, value, np.argwhere(~gone[:, ::2]).tolist()[:4])
            assert not gone[:, 1::2].any()
        if top:
            assert (got["top_tokens"][:, ::2] == -1).all()
