"""The cache's calls at their limits: NaN codes among many short units, default
workspaces in graphs and on several streams, rows without a token, the ends of
the number ranges, dominant keys, scales no write made, many requests, wide
groups, full requests."""
import numpy as np
import pytest
import torch

import kv_util as ku
import speculative_decoding_verification_63_gb300 as sv
from test_gpu_kvcache import TYPES, as_type, check_attention, flags, i32, new_ws, same_cache

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


# ------------------------------------------- workspaces the caller does not give

def attention_call(seed, lens, T, Hq, H, P, D):
    """A call without a workspace, and its result with one of its own."""
    rng = np.random.default_rng(seed)
    total = [a + T for a in lens]
    c = ku.random_cache(rng, sum(-(-x // P) for x in total), H, P, D)
    table, length, dev = i32(ku.tables(rng, c.k.shape[0], total, P)), i32(lens), ku.to_device(c)
    q, _ = as_type(rng.normal(size=(len(lens), T, Hq, D)), "bf16")
    run = lambda ws=None: sv.kv_attention(q, dev, table, length, ws=ws)["out"]
    want = run(new_ws(sv.sv_kv_attention_workspace_bytes(len(lens), T, Hq, H, D)))
    return run, want.clone()


DECODE = (31, [3000, 17, 900], 1, 16, 2, 32, 128)   # cut units, few rows
PROMPT = (32, [2000, 64], 120, 4, 2, 64, 128)       # cut units, tensor memory


def capture(run):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    return graph, out


@pytest.mark.parametrize("first", ["eager", "capture"])
def test_a_graph_keeps_its_workspace(first, monkeypatch):
    """A decode captured on the default workspace, larger calls and other
    tensors in between, replayed; also when the capture is the first use."""
    monkeypatch.setattr(sv, "_ws_cache", {})
    decode, want = attention_call(*DECODE)
    prompt, want_prompt = attention_call(*PROMPT)
    if first == "eager":
        assert torch.equal(decode(), want)
    graph, out = capture(lambda: (decode(), decode())[1])
    assert torch.equal(decode(), want)              # eager, before the first replay
    for _ in range(3):
        assert torch.equal(prompt(), want_prompt)
        junk = [torch.full((n << 20,), 0xff, dtype=torch.uint8, device="cuda")
                for n in (1, 2, 3, 5, 6, 8, 16, 21, 32)]
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
        assert all((x == 0xff).all() for x in junk)
        del junk
        assert torch.equal(decode(), want)
    prompt_graph, prompt_out = capture(prompt)
    for _ in range(3):
        out.zero_(), prompt_out.zero_()
        graph.replay()
        prompt_graph.replay()
        assert torch.equal(out, want) and torch.equal(prompt_out, want_prompt)


def test_other_calls_captured_first(monkeypatch):
    """Writes, reads and masks whose first use of their workspace is inside a
    capture: neither the graph nor later calls find garbage."""
    monkeypatch.setattr(sv, "_ws_cache", {})
    parent = i32([[-1, 0, 0, 1]])
    cache = sv.kv_cache(4, 16, 2, 64)
    table, length = i32([[0, 1, 2, 3]]), i32([5])
    x = torch.randn((1, 4, 2, 64), device="cuda", dtype=torch.bfloat16)

    def run():
        sv.kv_write(cache, table, length, x, x)
        return sv.kv_read(cache, table, length, None, 4)["k"], sv.tree_mask(parent)["mask"]

    graph, (k, mask) = capture(run)
    junk = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    del junk
    graph.replay()
    want_k, want_mask = run()
    assert torch.equal(k, want_k) and torch.equal(mask, want_mask)
    for key in ("kv", "mask"):
        sv.check_device_errors(sv.workspace(1, "cuda", key))


def test_streams_have_workspaces_of_their_own():
    """Prompts on one stream, decoding on two others, at the same time."""
    calls = [attention_call(*PROMPT), attention_call(*DECODE), attention_call(34, *DECODE[1:])]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(30):
        for (run, _), stream, outs in zip(calls, streams, got):
            with torch.cuda.stream(stream):
                outs.append(run())
    torch.cuda.synchronize()
    for (_, want), outs in zip(calls, got):
        assert all(torch.equal(o, want) for o in outs)


def test_errors_of_a_captured_call():
    """The graph's own workspace, asked for inside the capture."""
    rng = np.random.default_rng(35)
    dev = ku.to_device(ku.random_cache(rng, 4, 2, 16, 64))
    q, _ = as_type(rng.normal(size=(2, 1, 4, 64)), "bf16")
    table, length = i32([[0], [1]]), i32([5, 5])
    need, held = sv.sv_kv_attention_workspace_bytes(2, 1, 4, 2, 64), {}

    def run():
        held["ws"] = sv.workspace(need, "cuda", "kv_attention")
        return sv.kv_attention(q, dev, table, length)["out"]

    graph, _ = capture(run)
    graph.replay()
    assert flags(held["ws"]) == (sv.SV_OK, 0)
    length.copy_(i32([5, 99]))
    graph.replay()
    assert flags(held["ws"]) == (sv.SV_EDATA, sv.SV_DERR_ARG)


# ------------------------------------------------- rows without a token

@pytest.mark.parametrize("B,T,Hq,H,D", [(1, 5, 2, 1, 64), (33, 3, 8, 2, 128), (200, 2, 5, 5, 64),
                                        (70, 40, 4, 2, 64), (33, 64, 1, 1, 128), (2, 700, 2, 2, 64)])
def test_rows_without_a_token_are_cleared(B, T, Hq, H, D):
    """Every row t >= num_new of every request, whatever the outputs held."""
    rng = np.random.default_rng(41)
    new = rng.integers(0, T + 1, B)
    new[rng.random(B) < 0.3] = T
    if B > 2:
        new[B // 2] = T + 1  # out of range: no row holds a token
    lens, P = rng.integers(0, 20, B), 32
    slots = -(-(20 + T) // P)
    c = ku.random_cache(rng, 40, H, P, D)
    table = i32(rng.integers(0, 40, (B, slots)))
    q, _ = as_type(rng.normal(size=(B, T, Hq, D)), "bf16")
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, Hq), 7.0, device="cuda")
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(B, T, Hq, H, D))
    sv.sv_kv_attention(q, ku.to_device(c), table, i32(lens), out, ws, 0.1, num_new=i32(new), lse=lse)
    assert flags(ws) == ((sv.SV_EDATA, sv.SV_DERR_ARG) if B > 2 else (sv.SV_OK, 0))
    empty = torch.arange(T)[None] >= torch.from_numpy(np.where(new > T, 0, new))[:, None]
    out, lse = out.cpu().float(), lse.cpu()
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    assert torch.isfinite(lse[~empty]).all() and (out[~empty] != 7).any(-1).all()


def test_a_ragged_prompt_costs_what_it_writes():
    """One token in a call of 8192: 67 MB of zeros are the GPU's work, not one
    warp's (a fill of the same buffer is the measure)."""
    T, Hq, D = 8192, 32, 128
    dev = sv.kv_cache(70, 128, 8, D)
    table, length, new = i32([list(range(70))]), i32([100]), i32([1])
    q = torch.zeros((1, T, Hq, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(1, T, Hq, 8, D))

    def best(call):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
            a.record()
            for _ in range(10):
                call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 100)  # us a call
        return min(times)

    fill = best(out.zero_)
    call = best(lambda: sv.sv_kv_attention(q, dev, table, length, out, ws, 0.1, num_new=new))
    print(f"fill {fill:.1f} us, call {call:.1f} us")
    assert call <= 3 * fill + 30, (call, fill)


# --------------------------------------------------- far ends of the ranges

@pytest.mark.parametrize("T", [4, 12, 40])
@pytest.mark.parametrize("qexp,kexp,scale,coded", [
    (116, -48, 2.0 ** -60, True), (126, -48, 2.0 ** -70, True), (126, 0, 2.0 ** -120, True),
    (126, 48, 0.125, False), (20, 0, 2.0 ** 127, False), (-110, -48, 0.125, True)])
def test_attention_at_the_ends_of_the_ranges(T, qexp, kexp, scale, coded):
    """Queries up to bf16's largest, scales and pages at the ends of theirs:
    scores are moderate (channel 0 of every second key) or exactly zero, while
    a factor of theirs, or the factors' product, passes the range of fp32."""
    rng = np.random.default_rng(51)
    H, P, D, Hq, B = 2, 16, 64, 4, 2
    lens = [60, 150]
    total = [a + T for a in lens]
    c = ku.random_cache(rng, sum(-(-x // P) for x in total), H, P, D)
    c.ks[:] = 2.0 ** kexp
    c.k[:] = 0                       # zero codes ..
    c.k[..., 1:] = np.where(rng.random(c.k[..., 1:].shape) < 0.5, 0, 0x80)
    if coded:
        c.k[:, :, ::2, 0] = 0x01     # .. and one smallest code in every second key
    table = ku.tables(rng, c.k.shape[0], total, P)
    q, q64 = as_type(1.5 * 2.0 ** qexp * rng.choice([-1.0, 1.0], (B, T, Hq, D)), "bf16")
    assert np.isfinite(q64).all()
    ws = new_ws(sv.sv_kv_attention_workspace_bytes(B, T, Hq, H, D))
    got = sv.kv_attention(q, ku.to_device(c), i32(table), i32(lens), scale=scale, with_lse=True,
                          ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    out, lse, spr, xerr = ku.attention(q64, c, table, lens, [T] * B, None, scale)
    tol, dx = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
    o, l = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.isfinite(o).all() and np.isfinite(l).all()
    assert (np.abs(o - out) <= tol).all()
    assert (np.abs(l - lse) <= dx + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20).all()


# ------------------------------------- a dominant key and a long tail behind it

@pytest.mark.parametrize("where", [0, 100, 7000])
@pytest.mark.parametrize("nats", [12, 15, 18])
@pytest.mark.parametrize("T,G,D,dtype", [(1, 1, 64, "fp16"), (1, 4, 128, "bf16"), (5, 4, 64, "fp16"),
                                         (13, 4, 128, "fp16"), (40, 2, 64, "bf16"),
                                         (32, 4, 128, "fp16")])
def test_a_dominant_key_leaves_the_tail_its_bits(T, G, D, dtype, nats, where):
    """One key with a value of zero, `nats` above a nearly uniform context:
    the output is the context's, weighted 2^-17 to 2^-26 of the key's.  Bound:
    a weight is off by 2^-11 of itself, or by 2^-19 of the largest in its
    aligned 128 positions and at most 2^-28 of the row's largest; sums in 32
    bits as in kv_util.out_bounds.  (Every request holds the same pages: long
    contexts for each CTA.)"""
    rng = np.random.default_rng(61)
    B, P, L = 320, 128, 8000 - T
    slots = -(-(L + T) // P)
    c = ku.random_cache(rng, slots, 1, P, D)
    c.ks[:], c.vs[:] = 1.0, 2.0 ** -6
    c.k[:] = ku.encode(rng.normal(size=c.k.shape) * 0.002)  # few bits, far below channel 0
    c.k[..., 0] = ku.encode(rng.uniform(-0.3, 0.3, c.k.shape[:-1]))
    c.v[:] = ku.encode((1 + 0.3 * rng.normal(size=c.v.shape)) * 64)
    c.k[where // P, 0, where % P, 0] = ku.encode(np.array(float(nats)))
    c.v[where // P, 0, where % P] = 0
    order = rng.permutation(slots).astype(np.int32)
    dev = ku.to_device(ku.Cache(c.k[np.argsort(order)], c.v[np.argsort(order)], c.ks, c.vs))
    q = rng.normal(size=(B, T, G, D)) * 0.1
    q[..., 0] = rng.choice([3.75, 4.0], (B, T, G))
    q, q64 = as_type(q, dtype)
    half = torch.finfo(TYPES[dtype]).eps / 2
    got = sv.kv_attention(q, dev, i32(np.tile(order, (B, 1))), i32([L] * B), scale=0.25,
                          with_lse=True)
    o, l = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.isfinite(o).all()
    row = np.arange(slots, dtype=np.int64)
    k, v = (c.values(s, row, np.arange(L + T))[:, 0] for s in "kv")
    for b in (0, 7, 151, 152, 319):
        for t in {0, T // 2, T - 1}:
            n = L + t + 1
            for g in {0, G - 1}:
                x = k[:n] @ q64[b, t, g] * 0.25
                dx = D * 2.0 ** -24 * (np.abs(k[:n]) @ np.abs(q64[b, t, g])).max() * 0.25 + 2.0 ** -21
                w = np.exp(x - x.max())
                blocks = np.pad(w, (0, -n % 128)).reshape(-1, 128).max(1)
                dw = np.maximum(2.0 ** -11 * w, np.minimum(2.0 ** -19 * np.repeat(blocks, 128)[:n],
                                                           2.0 ** -28 * w.max()))
                z = w.sum()
                want, spread = w @ v[:n] / z, w @ np.abs(v[:n]) / z
                d = dw @ np.abs(v[:n]) / z + spread * (2.0 ** -12 + 2 * dx)
                tol = d + half * (np.abs(want) + d) + 2.0 ** -24
                assert (np.abs(o[b, t, g] - want) <= tol).all(), (np.abs(o[b, t, g] - want) / tol).max()
                lse = x.max() + np.log(z)
                assert abs(l[b, t, g] - lse) <= dx + 2.0 ** -22 * abs(lse) + 2.0 ** -20


@pytest.mark.parametrize("shape", ["falling", "rising", "alternating"])
@pytest.mark.parametrize("T,G,D", [(1, 4, 64), (13, 4, 128), (40, 2, 64)])
def test_scores_that_fall_or_alternate_far(T, G, D, shape):
    """Scores over hundreds of powers of two, block by block: the reference
    moves at every block, up to where the sums' range ends."""
    rng = np.random.default_rng(62)
    B, P, L = 320, 64, 2900 - T
    slots = -(-(L + T) // P)
    c = ku.random_cache(rng, slots, 1, P, D)
    c.ks[:], c.vs[:] = 1.0, 2.0 ** -6
    at = np.arange(slots * P).reshape(slots, P)
    size = {"falling": 400 - 800 * at / (L + T), "rising": 800 * at / (L + T) - 400,
            "alternating": np.where(at // 128 % 2, 200.0, 160.0)}[shape]
    c.k[:, 0] = ku.encode(rng.normal(size=c.k[:, 0].shape) * 0.01)
    c.k[:, 0, :, 0] = ku.encode(size)
    table = np.tile(np.arange(slots, dtype=np.int32), (B, 1))
    q = rng.normal(size=(B, T, G, D))
    q[..., 0] = 1.0
    q, q64 = as_type(q, "bf16")
    got = sv.kv_attention(q, ku.to_device(c), i32(table), i32([L] * B), scale=1.0, with_lse=True)
    o, l = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    pick = [0, 151, 319]
    out, lse, spr, xerr = ku.attention(q64[pick], c, table[pick], [L] * 3, [T] * 3, None, 1.0)
    tol, dx = ku.out_bounds(out, spr, xerr, D, torch.bfloat16)
    assert (np.abs(o[pick] - out) <= tol).all()
    assert (np.abs(l[pick] - lse) <= dx + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20).all()


# ------------------------------------------------- scales that no write made

@pytest.mark.parametrize("T,Hq", [(2, 4), (9, 8), (40, 6)])
@pytest.mark.parametrize("bad,counts", [(3.0, 2.0), (0.75, 0.5), (-2.0, 2.0), (0.0, 2.0 ** -48),
                                        (2.0 ** -60, 2.0 ** -48), (2.0 ** 90, 2.0 ** 48),
                                        (float("inf"), 2.0 ** 48), (float("nan"), 2.0 ** 48)])
def test_scales_that_are_no_powers_of_two(bad, counts, T, Hq):
    """Reads, attention and writes take such a scale as the same power of two
    and say so."""
    rng = np.random.default_rng(71)
    H, P, D, lens = 2, 16, 64, [50, 20]
    table = i32([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]])
    c = ku.random_cache(rng, 12, H, P, D)
    q, _ = as_type(rng.normal(size=(2, T, Hq, D)) * 0.1, "bf16")
    x, _ = as_type(rng.normal(size=(2, 2, H, D)), "bf16")
    side = rng.choice(["k", "v"])
    results = []
    for value in (bad, counts):
        dev = ku.to_device(c)
        dev[side + "_scale"][1, 0] = value
        ws = new_ws(sv.sv_kv_attention_workspace_bytes(2, T, Hq, H, D))
        want = (sv.SV_OK, 0) if value == counts else (sv.SV_EDATA, sv.SV_DERR_ARG)
        read = sv.kv_read(dev, table, i32([0, 0]), i32([40, 20]), 40, dtype=torch.float32, ws=ws)
        assert flags(ws) == want
        att = sv.kv_attention(q, dev, table, i32(lens), num_new=i32([T, 1]), with_lse=True, ws=ws)
        assert flags(ws) == want
        # a write behind tokens of that page that stay
        sv.kv_write(dev, table, i32([25, 3]), x, x, ws=ws)
        assert flags(ws) == want
        again = sv.kv_read(dev, table, i32([0, 0]), i32([27, 5]), 27, dtype=torch.float32, ws=ws)
        results.append([read["k"], read["v"], att["out"], att["lse"], again["k"], again["v"]])
    for a, b in zip(*results):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
        assert torch.equal(torch.isnan(a), torch.isnan(b))


# ------------------------------------------------------- many requests, wide groups

@pytest.mark.parametrize("B,T,Hq,H,D", [(500, 2, 2, 1, 64), (1024, 1, 3, 3, 64), (700, 50, 1, 1, 64),
                                        (1000, 13, 4, 1, 128)])
def test_attention_of_more_requests_than_a_pass_scans(B, T, Hq, H, D):
    rng = np.random.default_rng(91)
    lens, new = rng.integers(0, 50, B).tolist(), rng.integers(0, T + 1, B).tolist()
    check_attention(rng, lens, new, T, Hq, H, 16, D, "bf16")


@pytest.mark.parametrize("lens,new,T,Hq,H,P,D,dtype", [
    ([300, 5], [1, 1], 1, 17, 1, 64, 64, "bf16"),
    ([300, 70, 0], [1, 1, 1], 1, 64, 2, 16, 128, "fp16"),
    ([1000], [1], 1, 48, 1, 64, 128, "bf16"),
    ([130, 7], [1, 1], 1, 256, 1, 32, 64, "bf16"),
    ([200, 0], [5, 3], 5, 100, 4, 64, 128, "bf16"),
    ([90], [3], 3, 256, 256, 16, 64, "fp16"),
])
def test_attention_of_wide_groups(lens, new, T, Hq, H, P, D, dtype):
    check_attention(np.random.default_rng(92), lens, new, T, Hq, H, P, D, dtype)


def test_commit_beside_a_full_request():
    """A request that holds as many tokens as its pages do, and takes no part in
    the round, is no error of the batch's."""
    rng = np.random.default_rng(95)
    H, P, D = 2, 16, 64
    c = ku.random_cache(rng, 6, H, P, D)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    lens, accept = [2 * P, 10, 2 * P - 1], [0, 2, 0]
    nodes = np.array([[-1, -1], [2, 5], [-1, -1]], np.int32)
    dev, ws = ku.to_device(c), new_ws()
    x, x64 = as_type(rng.normal(size=(3, 6, H, D)), "bf16")
    new = [0, 6, 1]
    sv.kv_write(dev, i32(table), i32(lens), x, x, num_new=i32(new), ws=ws)
    c.write(table, lens, new, x64, x64)
    moved = {s: np.zeros((3, 2, H, D)) for s in "kv"}
    for s in "kv":
        moved[s][1] = c.values(s, table[1], 10 + nodes[1])
    c.write(table, [n + 1 for n in lens], accept, moved["k"], moved["v"])
    sv.kv_commit(dev, i32(table), i32(lens), i32(accept), i32(nodes), ws=ws)
    assert flags(ws) == (sv.SV_OK, 0)
    same_cache(dev, c)
    # tokens that do not fit stay one
    sv.kv_write(dev, i32(table), i32(lens), x, x, num_new=i32([1, 0, 0]), ws=ws)
    assert flags(ws) == (sv.SV_EDATA, sv.SV_DERR_ARG)
    same_cache(dev, c)
