"""Norms and rotations of queries and keys on the GPU, alone and on the keys'
way into the 8-bit cache, against the plain 64-bit implementations (round_util,
kv_util)."""
import numpy as np
import pytest
import torch

import kv_util as ku
import round_util as ru
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_kvcache import as_type, flags, i32, new_ws

pytestmark = pytest.mark.gpu


def near(got, y, size, dtype):
    off = ru.rounding(dtype, y, ru.rotation_bound(size))
    d = np.abs(got.double().cpu().numpy() - y)
    assert (d <= off).all(), float((d / off).max())


def weights(rng, D, dtype):
    return as_type(np.exp(0.3 * rng.normal(size=D)), dtype)


ROTATES = [  # B, T, Hq, Hk, D, dim, interleaved, norm, dtype, start, scaling
    (1, 1, 1, 0, 16, 16, False, True, "fp32", 0, None),
    (3, 1, 32, 8, 128, 128, False, True, "bf16", 2047, None),
    (2, 7, 5, 3, 128, 128, True, True, "fp16", 131071, {"type": "linear", "factor": 4}),
    (4, 33, 12, 12, 64, 32, True, False, "fp16", 8192, None),
    (2, 200, 9, 2, 128, 128, False, True, "bf16", 1 << 30,
     {"type": "yarn", "factor": 8, "context": 8192}),
    (1, 65, 3, 1, 80, 48, False, True, "bf16", 100, {"type": "ntk", "factor": 2.0}),
    (2, 19, 2, 2, 96, 96, True, True, "fp32", 1000,
     {"type": "wavelength", "factor": 8, "context": 8192}),
    (1, 9, 4, 4, 256, 64, False, True, "fp32", 77, None),
    (2, 5, 2, 1, 112, 112, False, False, "bf16", 5, None),
    (1, 1500, 40, 8, 128, 64, True, True, "bf16", 3, None),
    (2, 3, 8, 2, 192, 0, False, True, "fp16", 3, None),
]


@pytest.mark.parametrize("B,T,Hq,Hk,D,dim,inter,norm,dtype,start,scaling", ROTATES)
def test_rotate(B, T, Hq, Hk, D, dim, inter, norm, dtype, start, scaling):
    rng = np.random.default_rng(D * 1000 + T)
    rope = sv.rope(dim, 5e5, interleaved=inter, scaling=scaling) if dim else None
    eps = 1e-5 if norm else None
    num = rng.integers(0, T + 1, B)
    num[-1] = T
    first = start + rng.integers(0, 3, B)
    ws, out = new_ws(), {}
    args, ref = {}, {}
    for name, H in (("q", Hq), ("k", Hk)):
        if H:
            args[name], ref[name] = as_type(
                rng.normal(size=(B, T, H, D)) * 2.0 ** rng.integers(-3, 4, (B, T, H, 1)), dtype)
    w = {n: weights(rng, D, dtype) for n in "qk"} if norm else {}
    out = sv.rotate(args["q"], args.get("k"), start=i32(first), num=i32(num), rope=rope, eps=eps,
                    q_weight=w["q"][0] if norm else None,
                    k_weight=w["k"][0] if norm and Hk else None, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    pos = ru.positions(first, None, B, T)
    for name in args:
        y, size = ru.rotated(ref[name], pos, rope, w[name][1] if norm else None, eps)
        for b in range(B):
            y[b, num[b]:] = size[b, num[b]:] = 0
        assert out[name].dtype == args[name].dtype
        near(out[name], y, size, dtype)
        for b in range(B):
            assert not out[name][b, num[b]:].any()
    # in place, the same bits
    again = {n: x.clone() for n, x in args.items()}
    sv.rotate(again["q"], again.get("k"), start=i32(first), num=i32(num), rope=rope, eps=eps,
              q_weight=w["q"][0] if norm else None,
              k_weight=w["k"][0] if norm and Hk else None, inplace=True, ws=ws)
    for name in args:
        assert torch.equal(again[name], out[name])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_rotate_slices(dtype, off):
    """Heads of a fused projection, whose rows need not be aligned; offsets of a
    tree; weights of another type; no weight."""
    rng = np.random.default_rng(5)
    B, T, Hq, Hk, D = 3, 21, 4, 2, 64
    buf = torch.zeros(B * T * (Hq + 2 * Hk) * D + off, dtype=ru.TYPES[dtype], device="cuda")
    x, x64 = as_type(rng.normal(size=(B, T, (Hq + 2 * Hk), D)), dtype)
    view = buf[off:].view(B, T, Hq + 2 * Hk, D)
    view.copy_(x)
    q, k = view[:, :, :Hq], view[:, :, Hq:Hq + Hk]
    rope = sv.rope(64, 1e4, interleaved=off == 8)
    depth = rng.integers(-3, 40, (B, T))
    start = np.array([7, 0, 4000])
    w, w64 = weights(rng, D, "fp32")
    pos = ru.positions(start, depth, B, T)
    got = sv.rotate(q, k, start=i32(start), offset=i32(depth), rope=rope, k_weight=w, eps=1e-6)
    near(got["q"], *ru.rotated(x64[:, :, :Hq], pos, rope, None, 1e-6), dtype)
    near(got["k"], *ru.rotated(x64[:, :, Hq:Hq + Hk], pos, rope, w64, 1e-6), dtype)
    # in place, within the projection; the rest of it stays
    sv.rotate(q, k, start=i32(start), offset=i32(depth), rope=rope, k_weight=w, eps=1e-6,
              inplace=True)
    assert torch.equal(q, got["q"]) and torch.equal(k, got["k"])
    assert torch.equal(view[:, :, Hq + Hk:], x[:, :, Hq + Hk:])


def test_rotate_far_positions():
    """Positions of any 32-bit sum, negative ones too, and frequencies above half
    a turn a position."""
    rng = np.random.default_rng(6)
    x, x64 = as_type(rng.normal(size=(4, 2, 1, 64)), "fp32")
    rope = sv.rope(64)
    rope["freq"] = sv.rope_turns(rng.uniform(-6, 6, 32).tolist())
    start = np.array([2 ** 31 - 1, -2 ** 31, -5, 0])
    offset = np.array([[2 ** 31 - 1, 0], [-2 ** 31, 0], [4, 5], [-1, 1]])
    pos = ru.positions(start, offset, 4, 2)
    got = sv.rotate(x, start=i32(start), offset=i32(offset), rope=rope)
    near(got["q"], *ru.rotated(x64, pos, rope), "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_extremes(dtype):
    """Values whose squares pass the range of fp32, tiny ones beside eps, rows of
    zeros, infinities and NaN."""
    rng = np.random.default_rng(7)
    x = rng.normal(size=(8, 1, 2, 128))
    x[0] *= 1e30
    x[1] *= 1e37
    x[2] *= 1e-30
    x[3] = 0
    x[4, 0, 0, 1:] = 1e-30
    x[4, 0, 0, 0] = 3e38
    x[5, 0, 0, 5] = np.inf
    x[6, 0, 1, 7] = np.nan
    t, x64 = as_type(x, dtype)
    rope = sv.rope(128)
    start = np.arange(8) * 11
    got = sv.rotate(t, start=i32(start), rope=rope, eps=1e-6)["q"]
    y, size = ru.rotated(x64, ru.positions(start, None, 8, 1), rope, None, 1e-6)
    fine = np.isfinite(x64).all(-1)
    off = ru.rounding(dtype, y, ru.rotation_bound(size))
    d = np.abs(got.double().cpu().numpy() - y)
    assert (d <= off)[fine].all()
    assert not got[3].any()
    # a row with an infinity: the others become 0, the infinity NaN, which turn together
    assert torch.isnan(got[5, 0, 0]).sum() == 2 and torch.isnan(got[6, 0, 1]).all()


def test_rows_past_32_bits():
    """Tokens more than 2^31 values apart, in place and on their way into the cache."""
    rng = np.random.default_rng(8)
    stride, T, H, D = (1 << 31) + 128, 3, 2, 64
    buf = torch.zeros((T - 1) * stride + H * D, dtype=torch.bfloat16, device="cuda")
    view = buf.as_strided((1, T, H, D), (0, stride, D, 1))
    x, x64 = as_type(rng.normal(size=(1, T, H, D)), "bf16")
    view.copy_(x)
    rope, pos = sv.rope(64), [[5, 6, 7]]
    ref = ku.random_cache(rng, 2, H, 16, D)
    dev = ku.to_device(ref)
    q = sv.kv_append(dev, i32([[1]]), i32([5]), view, view, view, rope=rope, eps=1e-6)["q"]
    y, size = ru.rotated(x64, pos, rope, None, 1e-6)
    near(q, y, size, "bf16")
    ref.write(np.array([[1]]), [5], [T], y, x64)
    _, v, ks, vs = ku.from_device(dev)
    assert np.array_equal(v, ref.v) and np.array_equal(ks, ref.ks) and np.array_equal(vs, ref.vs)
    sv.rotate(view, start=i32([5]), rope=rope, eps=1e-6, inplace=True)
    assert torch.equal(view, q)


def test_rotate_bad_num_and_empty():
    x = torch.ones(3, 4, 2, 64, device="cuda", dtype=torch.bfloat16)
    ws = new_ws()
    got = sv.rotate(x, x.clone(), num=i32([5, 2, -1]), rope=sv.rope(64), ws=ws)
    assert flags(ws) == (sv.SV_EDATA, sv.SV_DERR_ARG)
    for n in "qk":
        assert not got[n][0].any() and not got[n][2].any() and got[n][1, :2].all()
        assert not got[n][1, 2:].any()
    assert sv.rotate(x[:0], rope=sv.rope(64))["q"].shape == (0, 4, 2, 64)


# ------------------------------------------------------------------ append

def check_append(rng, lens, new, T, Hq, H, P, D, dtype, rope, eps, depth=None, split=None,
                 spread=1.0, q_dtype=None):
    B = len(lens)
    total = [a + n for a, n in zip(lens, new)]
    pages = sum(-(-x // P) for x in total) + 2
    ref = ku.random_cache(rng, pages, H, P, D)
    table = ku.tables(rng, pages, total, P)
    dev, ws = ku.to_device(ref, split), new_ws()
    x, x64 = as_type(rng.normal(size=(B, T, Hq + 2 * H, D)) * spread *
                     2.0 ** rng.integers(-4, 4, (B, T, 1, 1)), dtype)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]
    wq, wk = (weights(rng, D, dtype) for _ in "qk")
    pos = ru.positions(lens, depth, B, T)
    yq, sq = ru.rotated(x64[:, :, :Hq], pos, rope, wq[1], eps)
    yk, sk = ru.rotated(x64[:, :, Hq:Hq + H], pos, rope, wk[1], eps)
    for b in range(B):
        yq[b, new[b]:] = sq[b, new[b]:] = 0
    ref.write(table, lens, new, yk, x64[:, :, Hq + H:])
    got = sv.kv_append(dev, i32(table), i32(lens), q, k, v, num_new=i32(new),
                       offset=None if depth is None else i32(depth), rope=rope, eps=eps,
                       q_weight=wq[0] if eps else None, k_weight=wk[0] if eps else None,
                       q_dtype=q_dtype, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    name = dtype if q_dtype is None else {v: k for k, v in ru.TYPES.items()}[q_dtype]
    near(got["q"], yq, sq, name)
    gk, gv, ks, vs = ku.from_device(dev)
    assert np.array_equal(vs, ref.vs) and np.array_equal(gv, ref.v)
    # scales of keys: the definition's (the seeds put no largest key within the
    # rounding of a step between scales), codes: within half a step of the key, and
    # the other tokens' as they are
    assert np.array_equal(ks, ref.ks)
    touched = np.zeros(ref.k.shape, bool)
    for b in range(B):
        for t in range(new[b]):
            at = lens[b] + t
            page, row = table[b, at // P], at % P
            touched[page, :, row] = True
            s = ref.ks[page][:, None]
            y, off = yk[b, t], ru.rotation_bound(sk[b, t])
            value = ku.E4M3[gk[page, :, row]] * s
            half = np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10)
            assert (np.abs(value - y) <= half + 2 * off).all()
    assert np.array_equal(gk[~touched], ref.k[~touched])
    return dev, table, got


APPENDS = [  # lens, new, T, Hq, H, P, D, dtype, dim, interleaved, norm
    ([0, 5, 16, 31], [1, 1, 1, 1], 1, 8, 2, 16, 64, "bf16", 64, False, True),
    ([0, 1, 15, 16, 17, 40], [7, 0, 1, 3, 7, 6], 7, 3, 3, 16, 128, "fp16", 64, True, False),
    ([0, 100, 127, 128, 129], [33, 33, 2, 32, 0], 33, 16, 1, 128, 128, "bf16", 128, False, True),
    ([3, 64], [200, 131], 200, 4, 2, 64, 128, "fp32", 128, True, True),
    ([0, 30], [64, 65], 65, 10, 5, 32, 64, "fp32", 16, False, True),
    ([60], [512], 512, 32, 8, 64, 128, "bf16", 128, False, True),
    ([127, 1], [1, 300], 300, 1, 1, 128, 64, "fp16", 48, False, True),
    ([9], [3000], 3000, 16, 4, 64, 128, "bf16", 96, True, False),
]


@pytest.mark.parametrize("lens,new,T,Hq,H,P,D,dtype,dim,inter,norm", APPENDS)
def test_append(lens, new, T, Hq, H, P, D, dtype, dim, inter, norm):
    rng = np.random.default_rng(P + D + T)
    check_append(rng, lens, new, T, Hq, H, P, D, dtype, sv.rope(dim, 5e5, interleaved=inter),
                 1e-6 if norm else None)


@pytest.mark.parametrize("split", ["interleaved", "heads"])
def test_append_tree_and_cache_strides(split):
    rng = np.random.default_rng(11)
    depth = np.array([[0, 1, 2, 1, 2, 3, 1], [0, 1, 1, 2, 2, -1, -1]])
    check_append(rng, [30, 64], [7, 5], 7, 6, 2, 32, 128, "bf16", sv.rope(128), 1e-6, depth=depth,
                 split=split)


def test_append_grows_scales_and_converts_queries():
    rng = np.random.default_rng(12)
    for spread, dtype, q_dtype in ((300.0, "fp32", torch.bfloat16), (1e-4, "fp32", torch.float16),
                                   (50.0, "bf16", torch.float32)):
        check_append(rng, [5, 17, 40], [4, 2, 30], 30, 4, 2, 32, 64, dtype, sv.rope(32), None,
                     spread=spread, q_dtype=q_dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_without_rotation_is_a_write(dtype):
    rng = np.random.default_rng(13)
    lens, new, T, H, P, D = [3, 16, 9], [21, 20, 1], 21, 4, 16, 64
    total = [a + n for a, n in zip(lens, new)]
    ref = ku.random_cache(rng, 12, H, P, D)
    table = i32(ku.tables(rng, 12, total, P))
    k, _ = as_type(rng.normal(size=(3, T, H, D)), dtype)
    v, _ = as_type(rng.normal(size=(3, T, H, D)), dtype)
    a, b = ku.to_device(ref), ku.to_device(ref)
    sv.kv_write(a, table, i32(lens), k, v, num_new=i32(new))
    assert sv.kv_append(b, table, i32(lens), None, k, v, num_new=i32(new)) == {}
    for x in a:
        assert torch.equal(a[x].view(torch.uint8), b[x].view(torch.uint8)), x


def test_append_bad_requests():
    """Bad lengths and pages: reported, the cache's other parts and the queries'
    rows as the header says."""
    rng = np.random.default_rng(14)
    H, P, D, T = 2, 16, 64, 5
    ref = ku.random_cache(rng, 8, H, P, D)
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 99], [-1, 7], [2, 3]], np.int32)
    lens, new = np.array([-1, 30, 0, 14, 14, 3]), np.array([1, 3, 6, 5, 5, -1])
    dev, ws = ku.to_device(ref), new_ws()
    k, k64 = as_type(rng.normal(size=(6, T, H, D)), "bf16")
    got = sv.kv_append(dev, i32(table), i32(lens), k, k, k, num_new=i32(new), ws=ws)
    assert flags(ws) == (sv.SV_EDATA, sv.SV_DERR_ARG | sv.SV_DERR_PAGE)
    for b in range(6):
        assert bool(got["q"][b].any()) == (b in (3, 4))
    # of requests 3 and 4 only the page that exists is written
    want = ku.Cache(ref.k, ref.v, ref.ks, ref.vs)
    one = np.zeros((1, 5, H, D))
    one[:, :2] = k64[3:4, :2]
    want.write(np.array([[6]]), [14], [2], one, one)
    two = np.zeros((1, 3, H, D))
    two[:] = k64[4:5, 2:]
    want.write(np.array([[7]]), [0], [3], two, two)
    gk, gv, ks, vs = ku.from_device(dev)
    assert np.array_equal(gk, want.k) and np.array_equal(gv, want.v)
    assert np.array_equal(ks, want.ks) and np.array_equal(vs, want.vs)


def test_append_reports_what_is_not_finite():
    H, P, D = 1, 16, 64
    for bad, norm in ((np.inf, False), (np.nan, False), (np.inf, True)):
        rng = np.random.default_rng(15)
        ref = ku.random_cache(rng, 2, H, P, D)
        x = rng.normal(size=(1, 3, H, D))
        x[0, 1, 0, 5] = bad
        k, k64 = as_type(x, "fp32")
        dev, ws = ku.to_device(ref), new_ws()
        rope = sv.rope(16)
        sv.kv_append(dev, i32([[1]]), i32([0]), None, k, k, rope=rope, eps=1e-6 if norm else None,
                     ws=ws)
        assert flags(ws) == (sv.SV_EDATA, sv.SV_DERR_NONFINITE)
        with np.errstate(invalid="ignore"):
            y, _ = ru.rotated(k64, [[0, 1, 2]], rope, None, 1e-6 if norm else None)
        a = np.abs(y[np.isfinite(y)]).max()
        gk, _, ks, _ = ku.from_device(dev)
        assert ks[1, 0] == 2.0 ** ku.needed_exp(a)
        row = ku.E4M3[gk[1, 0, 1]] * ks[1, 0]
        assert np.array_equal(np.isnan(row), np.isnan(y[0, 1, 0]))
        assert np.isfinite(ku.E4M3[gk[1, 0, [0, 2]]]).all()


def test_calls_in_a_graph_and_on_a_side_stream():
    rng = np.random.default_rng(16)
    lens, T, H, P, D = [3, 16], 4, 2, 16, 64
    ref = ku.random_cache(rng, 6, H, P, D)
    table, length = i32(ku.tables(rng, 6, [7, 20], P)), i32(lens)
    x, _ = as_type(rng.normal(size=(2, T, 8, D)), "bf16")
    rope = sv.rope(64)
    eager, replayed = ku.to_device(ref), ku.to_device(ref)
    want = sv.kv_append(eager, table, length, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], rope=rope)
    turned = sv.rotate(x, start=length, rope=rope, eps=1e-6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(sv.rotate(x, start=length, rope=rope, eps=1e-6)["q"], turned["q"])
        with torch.cuda.graph(g, stream=s):
            got = sv.kv_append(replayed, table, length, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:],
                               rope=rope)
            again = sv.rotate(x, start=length, rope=rope, eps=1e-6)
    for _ in range(2):
        got["q"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["q"], want["q"]) and torch.equal(again["q"], turned["q"])
        for n in eager:
            assert torch.equal(eager[n].view(torch.uint8), replayed[n].view(torch.uint8))


def test_many_requests_and_none():
    """1024 requests with a token each or none; a round without tokens leaves the cache
    as it is."""
    rng = np.random.default_rng(17)
    B, H, P, D = 1024, 1, 16, 64
    lens, new = rng.integers(0, 16, B), rng.integers(0, 2, B)
    lens = np.minimum(lens, 15)
    ref = ku.random_cache(rng, B, H, P, D)
    table = np.arange(B, dtype=np.int32)[rng.permutation(B)].reshape(B, 1)
    dev, ws = ku.to_device(ref), new_ws()
    x, x64 = as_type(rng.normal(size=(B, 1, 3, D)), "bf16")
    rope = sv.rope(64)
    zero = i32(np.zeros(B))
    got = sv.kv_append(dev, i32(table), i32(lens), x[:, :, :1], x[:, :, 1:2], x[:, :, 2:],
                       num_new=zero, rope=rope, eps=1e-6, ws=ws)
    assert not got["q"].any()
    gk, gv, ks, vs = ku.from_device(dev)
    assert np.array_equal(gk, ref.k) and np.array_equal(gv, ref.v) and np.array_equal(ks, ref.ks)
    pos = ru.positions(lens, None, B, 1)
    y, size = ru.rotated(x64, pos, rope, None, 1e-6)
    got = sv.kv_append(dev, i32(table), i32(lens), x[:, :, :1], x[:, :, 1:2], x[:, :, 2:],
                       num_new=i32(new), rope=rope, eps=1e-6, ws=ws)
    ref.write(table, lens, new, y[:, :, 1:2], x64[:, :, 2:])
    gk, gv, ks, vs = ku.from_device(dev)
    assert np.array_equal(gv, ref.v) and np.array_equal(ks, ref.ks) and np.array_equal(vs, ref.vs)
    y[new == 0] = size[new == 0] = 0
    near(got["q"], y[:, :, :1], size[:, :, :1], "bf16")
    turned = sv.rotate(x, start=i32(lens), num=i32(new), rope=rope, eps=1e-6, ws=ws)["q"]
    assert torch.equal(turned[:, :, :1], got["q"])
    assert flags(ws) == (sv.SV_OK, 0)


def test_two_streams_at_once():
    """Calls of two streams share nothing but the error word."""
    rng = np.random.default_rng(18)
    x, _ = as_type(rng.normal(size=(4, 600, 12, 128)), "bf16")
    rope, start = sv.rope(128), i32([0, 5, 9, 1000])
    want = sv.rotate(x, start=start, rope=rope, eps=1e-6)["q"]
    logits, _ = as_type(rng.normal(size=(2, 100, 32000)), "bf16")
    said = sv.token_logprobs(logits, top=5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((sv.rotate(x, start=start, rope=rope, eps=1e-6)["q"],
                               sv.token_logprobs(logits, top=5)))
    torch.cuda.synchronize()
    for q, lp in got[0] + got[1]:
        assert torch.equal(q, want)
        assert all(torch.equal(lp[n], said[n]) for n in said)


@pytest.mark.parametrize("Hq,dtype,inter", [(20, "bf16", False), (33, "fp16", True)])
def test_more_tokens_than_run_at_once(Hq, dtype, inter):
    """Blocks of the same tokens one behind the other: requests of odd lengths, lanes
    without channels, parts of different sizes."""
    rng = np.random.default_rng(Hq)
    B, T, Hk, D = 3, 2003, 5, 80
    rope, num = sv.rope(64, 5e5, interleaved=inter), np.array([2003, 0, 1001])
    first = np.array([0, 7, 90001])
    x, x64 = as_type(rng.normal(size=(B, T, Hq + Hk, D)), dtype)
    got = sv.rotate(x[:, :, :Hq], x[:, :, Hq:], start=i32(first), num=i32(num), rope=rope, eps=1e-5)
    y, size = ru.rotated(x64, ru.positions(first, None, B, T), rope, None, 1e-5)
    for b in range(B):
        y[b, num[b]:] = size[b, num[b]:] = 0
    near(got["q"], y[:, :, :Hq], size[:, :, :Hq], dtype)
    near(got["k"], y[:, :, Hq:], size[:, :, Hq:], dtype)


MIXED = [  # rounds of very different lengths in one call: T, Hq, H, P, D, dtype
    (47, 10, 5, 64, 128, "bf16"),   # two chunks a thread, one group or several
    (200, 4, 3, 128, 128, "fp16"),  # blocks of 512 threads
    (18, 16, 2, 64, 128, "bf16"),   # groups of five warps
    (100, 24, 12, 16, 64, "fp32"),  # several groups, two sets of heads
    (27, 7, 7, 32, 128, "bf16"),    # groups of seven warps, heads no group's multiple
    (2, 1, 1, 16, 64, "fp16"),      # a block of two warps
]


@pytest.mark.parametrize("T,Hq,H,P,D,dtype", MIXED)
def test_append_rounds_of_mixed_lengths(T, Hq, H, P, D, dtype):
    rng = np.random.default_rng(T)
    new = np.array([T, 0, 1, T // 2, T, T // 3, max(T - 1, 1), 1])
    lens = np.array([P - 1, 5, P, 0, 2 * P - T % P, 3 * P + 1, 1, P - 1])
    check_append(rng, lens, new, T, Hq, H, P, D, dtype, sv.rope(D // 2, 1e4), 1e-6)
