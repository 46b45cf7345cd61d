"""The 8-bit key/value cache on the GPU against the plain 64-bit
implementation (kv_util): writes and reads code for code, attention within
bounds derived from its roundings."""
import numpy as np
import pytest
import torch

import kv_util as ku
import speculative_decoding_verification_63_gb300 as sv

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def flags(ws):
    st, f = sv.sv_get_error(ws)
    return st, f


def new_ws(nbytes=sv.SV_MIN_WORKSPACE_BYTES):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    sv.sv_workspace_init(ws)
    return ws


def as_type(x, dtype):
    """x rounded to dtype, as the device tensor and its float64 values."""
    t = torch.from_numpy(x).to(TYPES[dtype])
    return t.cuda(), t.double().numpy()


def same_cache(dev, ref):
    k, v, ks, vs = ku.from_device(dev)
    assert np.array_equal(ks, ref.ks) and np.array_equal(vs, ref.vs)
    # NaN codes may carry either sign
    for got, want in ((k, ref.k), (v, ref.v)):
        nan = want & 0x7f == 0x7f
        assert np.array_equal(got & 0x7f == 0x7f, nan)
        assert np.array_equal(got[~nan], want[~nan])


# ------------------------------------------------------------------- write

WRITES = [  # lens, new, H, P, D, dtype, T
    ([0, 5, 16, 31], [1, 1, 1, 1], 2, 16, 64, "bf16", 1),
    ([0, 1, 15, 16, 17, 40], [7, 0, 1, 3, 7, 6], 3, 16, 128, "fp16", 7),
    ([0, 100, 127, 128, 129], [33, 33, 2, 32, 0], 1, 128, 128, "bf16", 33),
    ([3, 64], [200, 131], 2, 64, 128, "fp32", 200),
    ([0, 30], [64, 65], 5, 32, 64, "fp32", 65),
    ([60], [512], 8, 64, 128, "bf16", 512),
    ([127, 1], [1, 300], 1, 128, 64, "fp16", 300),
]


@pytest.mark.parametrize("lens,new,H,P,D,dtype,T", WRITES)
def test_write(lens, new, H, P, D, dtype, T):
    rng = np.random.default_rng(len(lens) * 1000 + P + D)
    total = [a + n for a, n in zip(lens, new)]
    pages = sum(-(-x // P) for x in total) + 2
    ref = ku.random_cache(rng, pages, H, P, D)
    table = ku.tables(rng, pages, total, P)
    dev, ws = ku.to_device(ref), new_ws()
    size = 2.0 ** rng.integers(-6, 6, (len(lens), T, H, 1))
    k, k64 = as_type(rng.normal(size=(len(lens), T, H, D)) * size, dtype)
    v, v64 = as_type(rng.normal(size=(len(lens), T, H, D)) * size[::-1], dtype)
    ref.write(table, lens, new, k64, v64)
    sv.kv_write(dev, i32(table), i32(lens), k, v, num_new=i32(new), ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    same_cache(dev, ref)
    # again: the same codes and scales
    sv.kv_write(dev, i32(table), i32(lens), k, v, num_new=i32(new), ws=ws)
    same_cache(dev, ref)


def test_write_grows_and_renews_scales():
    """Tokens that stay are rounded again when a page's scale grows; a page
    with none starts anew, whatever rejected tokens left there."""
    rng = np.random.default_rng(3)
    H, P, D = 2, 32, 64
    ref = ku.random_cache(rng, 6, H, P, D)
    table = ku.tables(rng, 6, [64, 64], P)
    dev, ws = ku.to_device(ref), new_ws()
    for lens, size in [([20, 31], 2.0 ** 9), ([10, 40], 1e-3), ([32, 0], 2.0 ** -20),
                       ([5, 33], 3.0), ([6, 60], 0.0)]:
        k, k64 = as_type(rng.normal(size=(2, 4, H, D)) * size, "fp32")
        v, v64 = as_type(rng.normal(size=(2, 4, H, D)) * size, "fp32")
        ref.write(table, lens, [4, 4], k64, v64)
        sv.kv_write(dev, i32(table), i32(lens), k, v, ws=ws)
        same_cache(dev, ref)
    assert flags(ws) == (sv.SV_OK, 0)


def test_write_extremes():
    """Values past the scales' range saturate or vanish; ties go to even;
    inf saturates, NaN stays; both are reported."""
    H, P, D = 1, 16, 64
    rng = np.random.default_rng(4)
    ref = ku.random_cache(rng, 4, H, P, D)
    table = np.arange(4, dtype=np.int32).reshape(4, 1)
    x = np.zeros((4, 3, H, D))
    x[0] = rng.normal(size=(3, H, D)) * 1e30
    x[1] = rng.normal(size=(3, H, D)) * 1e-30
    x[2, 0, 0] = np.resize((ku._GRID[1:60] + ku._GRID[:59]) / 2, D)  # ties
    x[2, 1, 0, 0] = 448.0
    x[3] = rng.normal(size=(3, H, D))
    x[3, 0, 0, 5], x[3, 1, 0, 6], x[3, 2, 0, 7] = np.inf, -np.inf, np.nan
    for n, finite in ((3, True), (4, False)):
        dev, ws = ku.to_device(ref), new_ws()
        want = ku.Cache(ref.k, ref.v, ref.ks, ref.vs)
        k, k64 = as_type(x[:n], "fp32")
        want.write(table[:n], [0] * n, [3] * n, k64, k64)
        sv.kv_write(dev, i32(table[:n]), i32([0] * n), k, k, ws=ws)
        same_cache(dev, want)
        st, f = flags(ws)
        assert (st, f) == ((sv.SV_OK, 0) if finite else (sv.SV_EDATA, sv.SV_DERR_NONFINITE))


@pytest.mark.parametrize("split", ["interleaved", "heads"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_write_strides(split, dtype):
    """A fused projection's slices, unaligned buffers, and caches whose heads
    or sides are not packed."""
    rng = np.random.default_rng(5)
    B, T, H, P, D = 3, 21, 4, 16, 64
    ref = ku.random_cache(rng, 12, H, P, D)
    lens, new = [3, 16, 9], [21, 20, 1]
    table = ku.tables(rng, 12, [a + n for a, n in zip(lens, new)], P)
    qkv, q64 = as_type(rng.normal(size=(B, T, (2 * H + 8) * D)), dtype)
    k64 = q64[:, :, 8 * D:(8 + H) * D].reshape(B, T, H, D)
    v64 = q64[:, :, (8 + H) * D:].reshape(B, T, H, D)
    ref.write(table, lens, new, k64, v64)
    for off in (0, 1):  # off 1: every row off its 16-byte boundary
        buf = torch.empty(qkv.numel() + 1, dtype=qkv.dtype, device="cuda")
        view = buf[off:off + qkv.numel()].view(qkv.shape)
        view.copy_(qkv)
        k = view[:, :, 8 * D:(8 + H) * D].unflatten(2, (H, D))
        v = view[:, :, (8 + H) * D:].unflatten(2, (H, D))
        if off == 0:
            v = v.contiguous()  # strides of its own
        start = ku.random_cache(np.random.default_rng(5), 12, H, P, D)
        dev, ws = ku.to_device(start, split), new_ws()
        sv.kv_write(dev, i32(table), i32(lens), k, v, num_new=i32(new), ws=ws)
        assert flags(ws) == (sv.SV_OK, 0)
        same_cache(dev, ref)


def test_write_bad_requests():
    rng = np.random.default_rng(6)
    H, P, D, T = 2, 16, 64, 5
    ref = ku.random_cache(rng, 8, H, P, D)
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 99], [-1, 7], [2, 3]], np.int32)
    lens, new = np.array([-1, 30, 0, 14, 14, 3]), np.array([1, 3, 6, 5, 5, -1])
    dev, ws = ku.to_device(ref), new_ws()
    k, k64 = as_type(rng.normal(size=(6, T, H, D)), "bf16")
    sv.kv_write(dev, i32(table), i32(lens), k, k, num_new=i32(new), ws=ws)
    # of requests 3 and 4 only the page that exists is written
    full = table.copy()
    full[3, 1], full[4, 0] = 2, 3
    scratch = ku.Cache(ref.k, ref.v, ref.ks, ref.vs)
    scratch.write(full[3:5], lens[3:5], new[3:5], k64[3:5], k64[3:5])
    for page in (6, 7):
        ref.k[page], ref.v[page] = scratch.k[page], scratch.v[page]
        ref.ks[page], ref.vs[page] = scratch.ks[page], scratch.vs[page]
    same_cache(dev, ref)
    st, f = flags(ws)
    assert st == sv.SV_EDATA and f == sv.SV_DERR_ARG | sv.SV_DERR_PAGE


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("H,P,D", [(1, 128, 128), (3, 16, 64), (8, 64, 128)])
def test_read(H, P, D, dtype):
    rng = np.random.default_rng(7)
    lens = [1, 17, 200, 64]
    c = ku.random_cache(rng, 40, H, P, D)
    table = ku.tables(rng, 40, lens, P)
    dev, ws = ku.to_device(c), new_ws()
    T = 70
    start, num = [0, 3, 190, 0], [1, 14, 10, 64]
    rows = np.full((4, T), -7, np.int32)
    for b in range(4):
        rows[b, :num[b]] = rng.integers(-start[b], lens[b] - start[b], num[b])
    for r in (None, rows):
        out = sv.kv_read(dev, i32(table), i32(start), i32(num), T, rows=None if r is None else i32(r),
                         dtype=TYPES[dtype], ws=ws)
        for side in "kv":
            want = np.zeros((4, T, H, D))
            for b in range(4):
                at = np.arange(num[b]) if r is None else r[b, :num[b]]
                want[b, :num[b]] = c.values(side, table[b], start[b] + at)
            want = torch.from_numpy(want).to(TYPES[dtype])
            assert torch.equal(out[side].cpu(), want)
    assert flags(ws) == (sv.SV_OK, 0)


def test_read_bad_requests_and_strides():
    rng = np.random.default_rng(8)
    H, P, D = 2, 16, 64
    c = ku.random_cache(rng, 6, H, P, D)
    table = np.array([[0, 1], [2, 6], [3, -1], [4, 5], [4, 5]], np.int32)
    start, num = [0, 14, 14, 30, 0], [2, 4, 4, 4, 5]
    dev, ws = ku.to_device(c, "heads"), new_ws()
    T = 4
    k = torch.full((T, 5, H, D + 1), 9.0, dtype=torch.bfloat16, device="cuda")[..., :D]
    v = torch.full((T, 5, H, D + 1), 9.0, dtype=torch.bfloat16, device="cuda")[..., :D]
    sv.sv_kv_read(dev, i32(table), i32(start), i32(num), k.transpose(0, 1), v.transpose(0, 1), ws)
    want = np.zeros((5, T, H, D))
    want[0, :2] = c.values("v", table[0], [0, 1])
    want[1, :2] = c.values("v", table[1], [14, 15])
    want[2, :2] = c.values("v", table[2], [14, 15])
    want[3, :2] = c.values("v", table[3], [30, 31])
    assert np.array_equal(v.transpose(0, 1).double().cpu().numpy(), want)
    st, f = flags(ws)
    assert st == sv.SV_EDATA and f == sv.SV_DERR_ARG | sv.SV_DERR_PAGE


def test_commit_of_a_tree_path():
    """verify_tree's accepted nodes move up behind the root; a read gives
    back their values, rounded at the new place's scale."""
    rng = np.random.default_rng(9)
    B, N, H, P, D, depth = 4, 32, 2, 16, 64, 5
    lens = [0, 13, 15, 40]
    c = ku.random_cache(rng, 20, H, P, D)
    table = ku.tables(rng, 20, [a + N for a in lens], P)
    nodes = np.full((B, depth), -1, np.int32)
    accept = [0, 5, 3, 1]
    for b in range(B):
        nodes[b, :accept[b]] = np.sort(rng.choice(np.arange(1, N), accept[b], replace=False))
    dev = ku.to_device(c)
    moved = {s: np.zeros((B, depth, H, D)) for s in "kv"}
    for b in range(B):
        for s in "kv":
            moved[s][b, :accept[b]] = c.values(s, table[b], lens[b] + nodes[b, :accept[b]])
    c.write(table, [x + 1 for x in lens], accept, moved["k"], moved["v"])
    ws = new_ws()
    sv.kv_commit(dev, i32(table), i32(lens), i32(accept), i32(nodes), ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    same_cache(dev, c)


# --------------------------------------------------------------- attention

def check_attention(rng, lens, new, T, Hq, H, P, D, dtype, mask=None, split=None, cache=None,
                    scale=None, q_of=None, spread=1.0, words=None):
    total = [a + n for a, n in zip(lens, new)]
    pages = sum(-(-x // P) for x in total) + 1
    c = cache or ku.random_cache(rng, pages, H, P, D, spread)
    table = ku.tables(rng, pages, total, P)
    q, q64 = as_type(rng.normal(size=(len(lens), T, Hq, D)), dtype)
    if q_of is not None:
        q = q_of(q)
    scale = D ** -0.5 if scale is None else scale
    dev = ku.to_device(c, split)
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(len(lens), T, Hq, H, D))
    words = None if mask is None else torch.from_numpy(ku.mask_words(mask, words)).cuda()
    run = lambda: sv.kv_attention(q, dev, i32(table), i32(lens), num_new=i32(new), mask=words,
                                  scale=scale, with_lse=True, ws=ws)
    got = run()
    assert flags(ws) == (sv.SV_OK, 0)
    assert not ws.any()  # the workspace is left zeroed
    out, lse, spr, xerr = ku.attention(q64, c, table, lens, new, mask, scale)
    tol, dx = ku.out_bounds(out, spr, xerr, D, TYPES[dtype])
    o, l = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.isfinite(o).all()
    worst = (np.abs(o - out) / tol).max()
    assert worst <= 1, worst
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), none)
    assert (np.abs(l - lse)[~none] <= (dx + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20)[~none]).all()
    again = run()
    assert torch.equal(again["out"], got["out"]) and torch.equal(again["lse"], got["lse"])
    return got


ATTENTION = [  # lens, new, T, Hq, H, P, D, dtype
    ([0], [1], 1, 1, 1, 16, 64, "bf16"),
    ([0, 1, 14, 15, 16, 63, 64, 65], [1] * 8, 1, 8, 2, 16, 128, "bf16"),
    ([700, 3, 0, 129], [1, 1, 1, 0], 1, 32, 8, 64, 128, "fp16"),
    ([500, 33, 1, 0, 255], [7, 3, 7, 5, 0], 7, 8, 2, 32, 128, "bf16"),
    ([40, 1000, 5], [5, 2, 4], 5, 5, 1, 128, 64, "fp16"),
    ([333, 90], [33, 20], 33, 6, 3, 64, 64, "bf16"),
    ([2000], [3], 3, 12, 12, 16, 64, "fp16"),
    ([6001], [5], 5, 16, 1, 128, 128, "bf16"),
    ([37, 0, 300], [200, 150, 77], 200, 4, 2, 64, 128, "bf16"),
    ([77, 0, 64, 129], [25, 24, 1, 0], 25, 4, 2, 16, 64, "bf16"),
    ([150, 65], [20, 17], 20, 5, 5, 64, 64, "fp16"),
    ([3001, 4], [8, 5], 8, 8, 2, 128, 128, "bf16"),
    ([5000, 0, 700], [60, 60, 1], 60, 1, 1, 64, 128, "bf16"),
    ([9000], [12], 12, 16, 4, 32, 64, "fp16"),
]


@pytest.mark.parametrize("lens,new,T,Hq,H,P,D,dtype", ATTENTION)
def test_attention_causal(lens, new, T, Hq, H, P, D, dtype):
    check_attention(np.random.default_rng(sum(lens) + T), lens, new, T, Hq, H, P, D, dtype)


@pytest.mark.parametrize("lens,new,T,Hq,H,P,D,dtype", [
    ([0, 17, 100, 63], [32, 32, 9, 0], 32, 4, 1, 16, 128, "bf16"),
    ([200, 5], [64, 63], 64, 8, 4, 64, 64, "fp16"),
    ([1000, 31], [33, 32], 33, 10, 2, 128, 128, "bf16"),
    ([3], [1], 1, 2, 2, 32, 64, "bf16"),
    ([60, 0, 31], [16, 9, 1], 16, 4, 2, 16, 128, "fp16"),
    ([10, 500], [31, 30], 31, 1, 1, 32, 64, "bf16"),
])
def test_attention_tree(lens, new, T, Hq, H, P, D, dtype):
    rng = np.random.default_rng(T)
    mask = ku.random_tree_mask(rng, len(lens), T)
    for words in (None, (T + 31) // 32 + 1):
        check_attention(rng, lens, new, T, Hq, H, P, D, dtype, mask=mask, words=words)


@pytest.mark.parametrize("split", ["interleaved", "heads"])
def test_attention_layouts(split):
    """Queries from a fused projection, off their boundaries; caches whose
    sides or heads are not packed."""
    rng = np.random.default_rng(11)

    def fused(q):
        wide = torch.zeros(q.shape[:2] + (q.shape[2] + 3, q.shape[3]), dtype=q.dtype, device="cuda")
        wide[:, :, 2:2 + q.shape[2]] = q
        return wide[:, :, 2:2 + q.shape[2]]

    def odd(q):
        wide = torch.zeros(q.shape[:3] + (q.shape[3] + 1,), dtype=q.dtype, device="cuda")
        wide[..., 1:] = q
        return wide[..., 1:]

    for q_of in (fused, odd):
        for T, Hq in ((4, 6), (7, 8), (30, 8)):
            check_attention(rng, [100, 30], [T, T - 1], T, Hq, 2, 32, 128, "bf16", split=split,
                            q_of=q_of)


def test_attention_of_wide_scores():
    """Scores that climb along the context and cover hundreds: the running
    reference moves; pages of very different scales are weighed together."""
    rng = np.random.default_rng(12)
    H, P, D = 2, 16, 64
    lens, new = [900, 20], [4, 4]
    pages = 60
    for T in (4, 10, 40):
        new = [T, T]
        c = ku.random_cache(rng, 64, H, P, D)
        c.ks = 2.0 ** rng.integers(-12, -2, c.ks.shape)
        c.vs = 2.0 ** rng.integers(-12, 4, c.vs.shape)
        total = [a + n for a, n in zip(lens, new)]
        assert sum(-(-x // P) for x in total) + 1 <= 64
        table = ku.tables(rng, 64, total, P)
        q, q64 = as_type(rng.normal(size=(2, T, 4, D)), "bf16")
        dev = ku.to_device(c)
        got = sv.kv_attention(q, dev, i32(table), i32(lens), num_new=i32(new), scale=0.5,
                              with_lse=True)
        out, lse, spr, xerr = ku.attention(q64, c, table, lens, new, None, 0.5)
        tol, dx = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
        assert (np.abs(got["out"].double().cpu().numpy() - out) <= tol).all()
        assert (np.abs(got["lse"].double().cpu().numpy() - lse)
                <= dx + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20).all()


@pytest.mark.parametrize("T", [4, 10, 40])
@pytest.mark.parametrize("scale", [0.0, -0.25, 40.0])
def test_attention_scales(T, scale):
    check_attention(np.random.default_rng(13), [70, 3], [T, T], T, 4, 2, 16, 64, "fp16",
                    scale=scale, spread=0.02)


@pytest.mark.parametrize("T,Hq,H,D", [(6, 2, 1, 64), (40, 6, 2, 128), (7, 8, 2, 128), (10, 2, 1, 64),
                                       (12, 8, 2, 64)])
def test_what_a_row_does_not_see_does_not_reach_it(T, Hq, H, D):
    """NaN codes in places a row does not see, in stale tokens behind the
    round and in unused page slots leave its result as it is; rows that see
    one are NaN; a row that sees nothing is 0 with lse -inf."""
    rng = np.random.default_rng(14)
    P = 16
    lens, new = [37, 0], [T - 1, T]
    total = [a + n for a, n in zip(lens, new)]
    pages = 12
    c = ku.random_cache(rng, pages, H, P, D)
    table = ku.tables(rng, pages, total, P)
    mask = ku.random_tree_mask(rng, 2, T)
    mask[1, 2] = False          # request 1, row 2: nothing to see
    mask[:, :, 4] = False       # token 4 is seen by nobody ..
    mask[:, 5, 4] = True        # .. but row 5
    q, q64 = as_type(rng.normal(size=(2, T, Hq, D)), "bf16")
    words = torch.from_numpy(ku.mask_words(mask)).cuda()
    out, lse, spr, xerr = ku.attention(q64, c, table, lens, new, mask, 0.125)
    tol, _ = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
    bad = ku.Cache(c.k, c.v, c.ks, c.vs)
    for b in range(2):
        for pos in range(total[b], -(-total[b] // P) * P):   # stale codes
            bad.k[table[b, pos // P], :, pos % P] = 0x7f
            bad.v[table[b, pos // P], :, pos % P] = 0xff
        at = lens[b] + 4
        bad.v[table[b, at // P], :, at % P, 3] = 0x7f        # one channel of token 4
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(2, T, Hq, H, D))
    got = sv.kv_attention(q, ku.to_device(bad), i32(table), i32(lens), num_new=i32(new),
                          mask=words, scale=0.125, with_lse=True, ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    o, l = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    want_nan = np.zeros(o.shape, bool)
    for b in range(2):
        want_nan[b, 5, :, 3] = new[b] > 5  # a row past the round is zero
    assert np.array_equal(np.isnan(o), want_nan)
    assert (np.abs(o - out) <= tol)[~want_nan].all()
    assert not o[1, 2].any() and np.isneginf(l[1, 2]).all()
    # a NaN key: the rows that see it are NaN, the others are not
    bad = ku.Cache(c.k, c.v, c.ks, c.vs)
    for b in range(2):
        at = lens[b] + 4
        bad.k[table[b, at // P], :, at % P, 7] = 0x7f
    got = sv.kv_attention(q, ku.to_device(bad), i32(table), i32(lens), num_new=i32(new),
                          mask=words, scale=0.125, ws=ws)
    o = got["out"].double().cpu().numpy()
    want_nan[:] = False
    for b in range(2):
        want_nan[b, 5] = new[b] > 5
    assert np.array_equal(np.isnan(o), want_nan)
    assert (np.abs(o - out) <= tol)[~want_nan].all()


@pytest.mark.parametrize("T", [3, 12, 40])
def test_attention_bad_requests(T):
    """Requests out of range give zero rows, pages that do not exist are seen
    by no row; the others keep their results."""
    rng = np.random.default_rng(15)
    H, P, D, Hq = 2, 16, 64, 4
    c = ku.random_cache(rng, 24, H, P, D)
    lens, new = [20, -1, 90, 20, 17], [T, 1, T, T + 1, T]
    slots = 6
    table = rng.permutation(24).reshape(4, slots)
    table = np.concatenate([table, table[:1]]).astype(np.int32)
    table[4, 1] = 24           # positions 16 .. 31 of request 4 are nowhere
    q, q64 = as_type(rng.normal(size=(5, T, Hq, D)), "bf16")
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(5, T, Hq, H, D))
    lens[2] = slots * P - T + 1
    got = sv.kv_attention(q, ku.to_device(c), i32(table), i32(lens), num_new=i32(new),
                          scale=0.125, with_lse=True, ws=ws)
    st, f = flags(ws)
    assert st == sv.SV_EDATA and f == sv.SV_DERR_ARG | sv.SV_DERR_PAGE
    o = got["out"].double().cpu().numpy()
    assert not o[1:4].any() and torch.isneginf(got["lse"][1:4]).all()
    out, _, spr, xerr = ku.attention(q64[:1], c, table[:1], lens[:1], new[:1], None, 0.125)
    tol, _ = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
    assert (np.abs(o[:1] - out) <= tol).all()
    # request 4 without the positions of the missing page
    ok = ku.Cache(c.k, c.v, c.ks, c.vs)
    for t in range(T):
        pos = np.array([p for p in range(17 + t + 1) if not 16 <= p < 32])
        fixed = np.where(table[4:5] == 24, 0, table[4:5])
        for j in range(Hq):
            x = ok.values("k", fixed[0], pos)[:, j // 2] @ q64[4, t, j] * 0.125
            w = np.exp(x - x.max())
            w /= w.sum()
            want = w @ ok.values("v", fixed[0], pos)[:, j // 2]
            assert np.abs(o[4, t, j] - want).max() <= 2.0 ** -6 * np.abs(
                ok.values("v", fixed[0], pos)).max()


def test_attention_without_requests_or_tokens():
    dev = sv.kv_cache(2, 16, 1, 64)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = sv.kv_attention(torch.zeros((0, 3, 2, 64), dtype=torch.bfloat16, device="cuda"), dev,
                          torch.zeros((0, 1), dtype=torch.int32, device="cuda"), z)
    assert out["out"].shape == (0, 3, 2, 64)
    out = sv.kv_attention(torch.ones((2, 3, 2, 64), dtype=torch.bfloat16, device="cuda"), dev,
                          i32([[0], [1]]), i32([5, 0]), num_new=i32([0, 0]), with_lse=True)
    assert not out["out"].any() and torch.isneginf(out["lse"]).all()


def test_offsets_beyond_32_bits():
    """A cache of more than 4 GiB a side, used at its far end."""
    H, P, D, pages = 8, 128, 128, 33000
    assert pages * H * P * D > 2 ** 32
    k = torch.empty((pages, H, P, D), dtype=torch.uint8, device="cuda")
    v = torch.empty((pages, H, P, D), dtype=torch.uint8, device="cuda")
    k[-2:], v[-2:] = 0, 0
    dev = dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn),
               k_scale=torch.ones((pages, H), device="cuda"),
               v_scale=torch.ones((pages, H), device="cuda"))
    rng = np.random.default_rng(16)
    kn, k64 = as_type(rng.normal(size=(1, 140, H, D)), "bf16")
    vn, v64 = as_type(rng.normal(size=(1, 140, H, D)), "bf16")
    table = i32([[pages - 1, pages - 2]])
    sv.kv_write(dev, table, i32([0]), kn, vn)
    small = ku.Cache(np.zeros((2, H, P, D), np.uint8), np.zeros((2, H, P, D), np.uint8),
                     np.ones((2, H)), np.ones((2, H)))
    st = np.array([[1, 0]], np.int32)
    small.write(st, [0], [140], k64, v64)
    got = sv.kv_read(dev, table, i32([0]), i32([140]), 140, dtype=torch.float32)
    for s in "kv":
        assert np.array_equal(got[s][0].double().cpu().numpy(),
                              small.values(s, st[0], np.arange(140)))
    for T in (2, 4, 40):
        q, q64 = as_type(rng.normal(size=(1, T, 16, D)), "bf16")
        o = sv.kv_attention(q, dev, table, i32([140 - T]))["out"].double().cpu().numpy()
        out, _, spr, xerr = ku.attention(q64, small, st, [140 - T], [T], None, D ** -0.5)
        tol, _ = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
        assert (np.abs(o - out) <= tol).all()


@pytest.mark.parametrize("T", [1, 4, 7, 32])
def test_a_round_on_a_side_stream_and_in_a_graph(T):
    """write, attention and read on a stream of their own, then captured in a
    CUDA graph and replayed on new inputs: the eager results."""
    rng = np.random.default_rng(17)
    B, Hq, H, P, D = 3, 8, 2, 16, 64
    lens = [50, 0, 33]
    c = ku.random_cache(rng, 30, H, P, D)
    table = i32(ku.tables(rng, 30, [x + T for x in lens], P))
    length = i32(lens)
    k, _ = as_type(rng.normal(size=(B, T, H, D)), "bf16")
    q, _ = as_type(rng.normal(size=(B, T, Hq, D)), "bf16")
    k2, _ = as_type(rng.normal(size=(B, T, H, D)), "bf16")

    def round_(dev, k, ws):
        sv.kv_write(dev, table, length, k, k.flip(0), ws=ws)
        o = sv.kv_attention(q, dev, table, length, ws=ws)["out"]
        r = sv.kv_read(dev, table, length, None, T, ws=ws)
        return o, r["k"], r["v"]

    size = sv.sv_kv_attention_workspace_bytes(B, T, Hq, H, D)
    eager, ws = ku.to_device(c), new_ws(size)
    want1 = [x.clone() for x in round_(eager, k, ws)]
    want2 = [x.clone() for x in round_(eager, k2, ws)]
    dev, ws = ku.to_device(c), new_ws(size)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        first = round_(dev, k, ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, want1))
    inp = k.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = round_(dev, inp, ws)
    for x, want in ((k, want1), (k2, want2)):
        inp.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_one_workspace_with_the_verification():
    """The cache's calls and a chain verification share a workspace."""
    from gpu_util import dev as to_dev
    from speculative_decoding_verification_63_gb300 import workloads as wl
    inp = wl.make_chain(2, B=3, V=5000)
    need = max(sv.sv_chain_workspace_bytes(3, 4, 5000, sv.SV_BF16, 0),
               sv.sv_kv_attention_workspace_bytes(2, 5, 8, 2, 64))
    ws = new_ws(need)
    chain = lambda: sv.verify_chain(*(to_dev(inp[x]) for x in ("target", "draft", "tokens",
                                                                "temperature", "uniforms")), ws=ws)
    a = chain()["out_tokens"].clone()
    rng = np.random.default_rng(18)
    c = ku.random_cache(rng, 64, 2, 16, 64)
    table = i32(ku.tables(rng, 64, [900, 40], 16))
    q, _ = as_type(rng.normal(size=(2, 5, 8, 64)), "bf16")
    x = sv.kv_attention(q, ku.to_device(c), table, i32([895, 35]), ws=ws)["out"]
    assert torch.equal(chain()["out_tokens"], a)
    y = sv.kv_attention(q, ku.to_device(c), table, i32([895, 35]), ws=ws)["out"]
    assert torch.equal(x, y) and flags(ws) == (sv.SV_OK, 0)
