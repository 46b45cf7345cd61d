"""Norms and rotations of queries and keys and log probabilities without a GPU:
struct layouts, refusals before any device work, the binding's checks, the
frequencies, and the plain implementations' own pins."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import round_util as ru
import speculative_decoding_verification_63_gb300 as sv
from speculative_decoding_verification_63_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, WS = 0x100000, ctypes.c_void_p(0x200000)
BIG = 1 << 30


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_verification_63_gb300 import _binding
    _build.build_library()
    _binding.lib()
    return _binding


def test_struct_layout_matches_binding(tmp_path, b):
    lines = ['#include "specverify.h"', "#include <stdio.h>", "#include <stddef.h>",
             "int main(void) {"]
    expect = []
    for cname, cls in [("sv_rope", b.SvRope), ("sv_head_norm", b.SvHeadNorm),
                       ("sv_heads", b.SvHeads), ("sv_rotate_args", b.SvRotateArgs),
                       ("sv_kv_append_args", b.SvKvAppendArgs),
                       ("sv_token_logprobs_args", b.SvTokenLogprobsArgs)]:
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        expect.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({cname}, {f}));')
            expect.append(getattr(cls, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", f"-I{os.path.join(ROOT, 'include')}", "-o", str(exe),
                    str(c)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in got.split()] == expect


# ---------------------------------------------------------------- refusals

def _heads(h, heads=4, D=64, **kw):
    h.x, h.out, h.heads = FAKE, FAKE + (1 << 16), heads
    h.batch_stride = h.out_batch_stride = 1 << 12
    h.token_stride = h.out_token_stride = heads * D
    h.head_stride = h.out_head_stride = D
    for k, v in kw.items():
        if k in ("weight", "weight_dtype", "eps"):
            setattr(h.norm, k, v)
        else:
            setattr(h, k, v)


def _rope(r, **kw):
    r.dim, r.interleaved, r.scale, r.freq = 64, 0, 1.0, FAKE
    for k, v in kw.items():
        setattr(r, k, v)


def _rotate(b, q=None, k=None, rope=None, **kw):
    a = b.SvRotateArgs()
    a.B, a.T, a.D, a.dtype = 2, 4, 64, b.SV_BF16
    _heads(a.q, **(q or {}))
    if k is not None:
        _heads(a.k, **k)
    _rope(a.rope, **(rope or {}))
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _append(b, cache=None, q=None, rope=None, norm=None, **kw):
    a = b.SvKvAppendArgs()
    c = a.cache
    c.num_pages, c.page_size, c.Hkv, c.D, c.slots = 8, 16, 2, 64, 4
    c.k = c.v = c.k_scale = c.v_scale = c.page_table = FAKE
    c.head_stride, c.page_stride = 16 * 64, 2 * 16 * 64
    for name, v in (cache or {}).items():
        setattr(c, name, v)
    a.B, a.T, a.dtype = 2, 4, b.SV_BF16
    a.k_new = a.v_new = a.kv_len = FAKE
    _heads(a.q, **(q or {}))
    _rope(a.rope, **(rope or {}))
    for name, v in (norm or {}).items():
        setattr(a.k_norm, name, v)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _logprobs(b, **kw):
    a = b.SvTokenLogprobsArgs()
    a.B, a.N, a.R, a.M, a.V, a.dtype, a.top = 2, 4, 4, 1, 1000, b.SV_BF16, 3
    a.batch_stride, a.row_stride = 4000, 1000
    for f in ("logits", "tokens", "logprob", "entropy", "top_token", "top_logprob"):
        setattr(a, f, FAKE)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _call(b, name, a, ws=WS, n=BIG):
    return getattr(b.lib(), name)(bytes(a), ws, n, None)


CALLS = [("sv_rotate", _rotate), ("sv_kv_append", _append), ("sv_token_logprobs", _logprobs)]


@pytest.mark.parametrize("name,make", CALLS)
def test_refusals_of_all(b, name, make):
    assert getattr(b.lib(), name)(None, WS, BIG, None) == b.SV_EINVAL
    assert _call(b, name, make(b, B=0)) == b.SV_OK
    for kw in [dict(B=-1), dict(B=b.SV_MAX_B + 1), dict(dtype=3), dict(dtype=-1)]:
        assert _call(b, name, make(b, **kw)) == b.SV_EINVAL, kw
    ok = make(b)
    assert _call(b, name, ok, ws=ctypes.c_void_p(0)) == b.SV_EWORKSPACE
    assert _call(b, name, ok, ws=ctypes.c_void_p(0x200010)) == b.SV_EWORKSPACE
    assert _call(b, name, ok, n=b.SV_MIN_WORKSPACE_BYTES - 1) == b.SV_EWORKSPACE


BAD_ROPES = [dict(dim=-16), dict(dim=8), dict(dim=40), dict(dim=80), dict(freq=None),
             dict(freq=FAKE + 8), dict(scale=math.nan), dict(scale=math.inf)]
BAD_HEADS = [dict(heads=-1), dict(heads=257), dict(x=None), dict(out=None), dict(x=FAKE + 1),
             dict(out=FAKE + 1), dict(out_dtype=3), dict(out=FAKE, out_dtype=1),
             dict(out=FAKE, out_token_stride=64), dict(out_batch_stride=0),
             dict(out_token_stride=0), dict(out_head_stride=0), dict(eps=-1e-6), dict(eps=1e-31),
             dict(eps=math.inf), dict(eps=math.nan), dict(weight=FAKE),
             dict(weight=FAKE, eps=1e-6, weight_dtype=3), dict(weight=FAKE + 1, eps=1e-6)]


@pytest.mark.parametrize("name,make", CALLS[:2])
def test_refusals_of_rotations(b, name, make):
    for kw in [dict(T=0), dict(T=b.SV_MAX_KV_T + 1)] + [dict(rope=r) for r in BAD_ROPES] + [
            dict(q=h) for h in BAD_HEADS]:
        assert _call(b, name, make(b, **kw)) == b.SV_EINVAL, kw
    if name == "sv_rotate":
        for kw in [dict(D=8), dict(D=72), dict(D=272), dict(D=0)] + [dict(k=h) for h in BAD_HEADS]:
            assert _call(b, name, make(b, **kw)) == b.SV_EINVAL, kw
        assert _call(b, name, make(b, q=dict(heads=0))) == b.SV_OK
    else:
        for kw in [dict(cache=dict(D=80)), dict(cache=dict(page_size=48)), dict(cache=dict(k=None)),
                   dict(k_new=None), dict(v_new=None), dict(kv_len=None), dict(k_new=FAKE + 1),
                   dict(v_new=FAKE + 1), dict(norm=dict(weight=FAKE)), dict(norm=dict(eps=-1.0))]:
            assert _call(b, name, make(b, **kw)) == b.SV_EINVAL, kw


def test_refusals_of_log_probabilities(b):
    for kw in [dict(N=0), dict(N=65537), dict(R=0), dict(R=65537), dict(R=5), dict(M=-1),
               dict(M=b.SV_MAX_GIVEN + 1), dict(V=0), dict(V=b.SV_MAX_V + 1), dict(top=-1),
               dict(top=b.SV_MAX_TOPK + 1), dict(dtype=b.SV_FP16), dict(logits=None),
               dict(logits=FAKE + 1), dict(tokens=None), dict(logprob=None), dict(top_token=None),
               dict(top_logprob=None), dict(batch_stride=-1), dict(row_stride=-1)]:
        assert _call(b, "sv_token_logprobs", _logprobs(b, **kw)) == b.SV_EINVAL, kw


# ----------------------------------------------------------------- binding

@pytest.fixture(scope="module")
def native(b):
    _build.build_native()
    return b._native()


def tensors(op):
    """Arguments of the compiled binding, in its order, on the CPU; entry 0 gives the
    packed structure back."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = lambda h: torch.zeros((2, 3, h, 64), dtype=torch.bfloat16)  # noqa: E731
    codes = lambda: torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(  # noqa: E731
        torch.float8_e4m3fn)
    a = dict(entry=0, workspace=torch.zeros(8192, dtype=torch.uint8), stream=None)
    if op == "token_logprobs":
        return a | dict(logits=torch.zeros(2, 3, 50), R=None, tokens=i32(2, 3), num_rows=i32(2),
                        rows=i32(2, 3), temperature=torch.ones(2), top=4, allocate=False,
                        logprobs=torch.zeros(2, 3), entropy=torch.zeros(2, 3),
                        top_tokens=i32(2, 3, 4), top_logprobs=torch.zeros(2, 3, 4))
    w = torch.ones(64, dtype=torch.bfloat16)
    tail = dict(offset=i32(2, 3), rope=sv.rope(64, device="cpu"), q_weight=w, k_weight=w.clone(),
                eps=1e-6)
    if op == "rotate":
        return a | dict(q=x(4), q_out=x(4), k=x(2), k_out=x(2), start=i32(2), num=i32(2)) | tail
    cache = dict(k=codes(), v=codes(), k_scale=torch.ones(4, 2), v_scale=torch.ones(4, 2))
    return a | dict(cache=cache, page_table=i32(2, 2), kv_len=i32(2), q=x(4), q_out=x(4),
                    q_dtype=None, k_new=x(2), v_new=x(2), num_new=i32(2)) | tail


OPS = ["rotate", "kv_append", "token_logprobs"]


def packed(b, native, op, a):
    cls = {"rotate": b.SvRotateArgs, "kv_append": b.SvKvAppendArgs,
           "token_logprobs": b.SvTokenLogprobsArgs}[op]
    raw = getattr(native, op)(*a.values())
    assert len(raw) == ctypes.sizeof(cls)
    return cls.from_buffer_copy(raw)


@pytest.mark.parametrize("op", OPS)
def test_packed_arguments(b, native, op):
    """What the binding packs is the structure's fields."""
    a = tensors(op)
    s = packed(b, native, op, a)
    if op == "token_logprobs":
        assert (s.B, s.N, s.R, s.M, s.V, s.top, s.dtype) == (2, 3, 3, 1, 50, 4, b.SV_FP32)
        assert (s.batch_stride, s.row_stride) == (150, 50)
        for f, t in [("logits", "logits"), ("tokens", "tokens"), ("rows", "rows"),
                     ("num_rows", "num_rows"), ("temperature", "temperature"),
                     ("logprob", "logprobs"), ("entropy", "entropy"), ("top_token", "top_tokens"),
                     ("top_logprob", "top_logprobs")]:
            assert getattr(s, f) == a[t].data_ptr(), f
        return
    assert (s.B, s.T, s.dtype, s.q.heads, s.q.out_dtype) == (2, 3, b.SV_BF16, 4, b.SV_BF16)
    assert (s.q.x, s.q.out) == (a["q"].data_ptr(), a["q_out"].data_ptr())
    assert (s.q.batch_stride, s.q.token_stride, s.q.out_head_stride) == (768, 256, 64)
    assert s.q.norm.weight == a["q_weight"].data_ptr() and abs(s.q.norm.eps - 1e-6) < 1e-12
    assert (s.rope.dim, s.rope.interleaved, s.rope.scale) == (64, 0, 1.0)
    assert s.rope.freq == a["rope"]["freq"].data_ptr() and s.offset == a["offset"].data_ptr()
    k = s.k.norm if op == "rotate" else s.k_norm
    assert k.weight == a["k_weight"].data_ptr() and k.weight_dtype == b.SV_BF16
    if op == "rotate":
        assert (s.D, s.k.heads, s.start, s.num) == (64, 2, a["start"].data_ptr(),
                                                    a["num"].data_ptr())
    else:
        c = s.cache
        assert (c.num_pages, c.page_size, c.Hkv, c.D, c.slots) == (4, 16, 2, 64, 2)
        assert (c.page_stride, c.head_stride, c.k) == (2048, 1024, a["cache"]["k"].data_ptr())
        assert (c.v_scale, c.page_table) == (a["cache"]["v_scale"].data_ptr(),
                                             a["page_table"].data_ptr())
        assert (s.k_new, s.v_token_stride) == (a["k_new"].data_ptr(), 128)
        assert (s.kv_len, s.num_new) == (a["kv_len"].data_ptr(), a["num_new"].data_ptr())


def test_packed_strides_and_options(b, native):
    """Slices of a projection, dimensions of size one, in place, no norm, no rope, no
    keys; tokens [B][R][M]; what is not asked for."""
    x = torch.zeros(2, 3, 8, 64, dtype=torch.float16)
    a = tensors("rotate") | dict(q=x[:, :, 2:6], q_out=..., k=None, k_out=None, rope=None,
                                 q_weight=None, k_weight=None, eps=None, start=None)
    s = packed(b, native, "rotate", a)
    assert (s.q.x, s.q.out, s.q.heads) == (x.data_ptr() + 2 * 64 * 2, x.data_ptr() + 2 * 64 * 2, 4)
    assert (s.q.token_stride, s.q.out_token_stride) == (512, 512)
    assert (s.k.heads, s.q.norm.eps, s.rope.dim, s.rope.scale, s.start) == (0, 0.0, 0, 1.0, None)
    one = torch.zeros(1, 1, 1, 64).as_strided((1, 1, 1, 64), (7, 9, 11, 1))
    a = tensors("rotate") | dict(q=one, q_out=None, k=None, k_out=None, num=None, offset=None,
                                 start=None, q_weight=None, k_weight=None)
    s = packed(b, native, "rotate", a)
    assert (s.q.batch_stride, s.q.token_stride, s.q.head_stride) == (0, 0, 0)
    assert s.q.out not in (None, s.q.x)
    a = tensors("kv_append") | dict(q_out=None, q_dtype=torch.float16)
    assert packed(b, native, "kv_append", a).q.out_dtype == b.SV_FP16
    a = tensors("kv_append") | dict(q=None, q_out=None, q_weight=None)
    assert packed(b, native, "kv_append", a).q.heads == 0
    a = tensors("token_logprobs") | dict(tokens=torch.zeros(2, 2, 5, dtype=torch.int32),
                                         logprobs=None, entropy=None, rows=None, top=0,
                                         top_tokens=None, top_logprobs=None)
    s = packed(b, native, "token_logprobs", a)
    assert (s.R, s.M, s.logprob, s.top_token) == (2, 5, None, None)
    s = packed(b, native, "token_logprobs", a | dict(allocate=True, top=3))
    assert s.logprob and s.entropy and s.top_token and s.top_logprob


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_another_device_are_refused(native, op):
    ok = tensors(op)
    for name, t in ok.items():
        if isinstance(t, torch.Tensor):
            wrong = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="meta")
        elif name == "rope":
            wrong = dict(t, freq=t["freq"].to("meta"))
        elif name == "cache":
            wrong = dict(t, v_scale=t["v_scale"].to("meta"))
        else:
            continue
        with pytest.raises(ValueError):
            getattr(native, op)(*(ok | {name: wrong}).values())


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_the_cpu_are_refused(b, native, op):
    """... by a call that is not asked for its structure."""
    a = tensors(op) | dict(entry=b._entry({"rotate": "sv_rotate", "kv_append": "sv_kv_append",
                                           "token_logprobs": "sv_token_logprobs"}[op]))
    with pytest.raises(ValueError, match="device tensors"):
        getattr(native, op)(*a.values())


WRONG = {
    "rotate": [dict(k=torch.zeros(2, 3, 2, 64)), dict(k=torch.zeros(2, 4, 2, 64).bfloat16()),
               dict(q_out=torch.zeros(2, 3, 5, 64).bfloat16()), dict(eps=None), dict(eps=0.0),
               dict(eps=math.nan), dict(k=None, k_out=None), dict(q=torch.zeros(2, 3, 64)),
               dict(q=torch.zeros(2, 3, 64, 4).bfloat16().transpose(2, 3)),
               dict(q=torch.zeros(2, 3, 4, 64, dtype=torch.int32)), dict(q=None), dict(q=3),
               dict(q_weight=torch.ones(32)), dict(q_weight=torch.ones(64, dtype=torch.int32)),
               dict(start=torch.zeros(2)), dict(num=torch.zeros(3, dtype=torch.int32)),
               dict(offset=torch.zeros(3, 2, dtype=torch.int32)), dict(rope=5), dict(rope={})],
    "kv_append": [dict(q=torch.zeros(2, 3, 4, 64)), dict(q=torch.zeros(2, 3, 4, 128).bfloat16()),
                  dict(v_new=torch.zeros(2, 3, 2, 64)), dict(eps=None), dict(eps=-1.0),
                  dict(kv_len=torch.zeros(2, dtype=torch.int64)), dict(q_dtype=3),
                  dict(k_new=torch.zeros(2, 3, 3, 64).bfloat16()), dict(cache={}), dict(cache=1),
                  dict(page_table=torch.zeros(4, dtype=torch.int32)), dict(q=None, q_out=None),
                  dict(k_weight=torch.ones(128)), dict(offset=torch.zeros(2, dtype=torch.int32))],
    "token_logprobs": [dict(logits=torch.zeros(2, 3, 50).half()), dict(logits=torch.zeros(2, 150)),
                       dict(logits=torch.zeros(2, 50, 3).transpose(1, 2)), dict(R=4),
                       dict(tokens=torch.zeros(2, 4, dtype=torch.int32)),
                       dict(tokens=torch.zeros(2, dtype=torch.int32)), dict(top=65), dict(top=-1),
                       dict(logprobs=torch.zeros(2, 3, 1)), dict(top_tokens=torch.zeros(2, 3, 4)),
                       dict(temperature=torch.ones(3)), dict(R=-1, allocate=True),
                       dict(rows=torch.zeros(2, 2, dtype=torch.int32))],
}


@pytest.mark.parametrize("op", OPS)
def test_wrong_types_and_shapes_are_refused(native, op):
    ok = tensors(op)
    for kw in WRONG[op]:
        with pytest.raises(ValueError):
            getattr(native, op)(*(ok | kw).values())
    if op != "token_logprobs":
        rope = ok["rope"]
        for bad in (dict(rope, dim=32), dict(rope, freq=torch.zeros(32))):
            with pytest.raises(ValueError):
                getattr(native, op)(*(ok | dict(rope=bad)).values())
    if op == "kv_append":
        for bad in (dict(v=torch.zeros(4, 2, 16, 64)), dict(k_scale=torch.ones(4, 3)),
                    dict(k=torch.zeros(4, 2, 16, 64)), dict(v_scale=torch.ones(4, 2).double())):
            with pytest.raises(ValueError):
                native.kv_append(*(ok | dict(cache=ok["cache"] | bad)).values())
    # new tensors belong to the current stream
    own = {"rotate": dict(k_out=None), "kv_append": dict(q_out=None),
           "token_logprobs": dict(allocate=True)}[op]
    getattr(native, op)(*(ok | own).values())
    with pytest.raises(ValueError, match="stream"):
        getattr(native, op)(*(ok | own | dict(stream=7)).values())
    for n in (0, 3, 40):
        with pytest.raises(TypeError):
            getattr(native, op)(*[None] * n)


def test_a_missing_build_is_reported(b, monkeypatch):
    monkeypatch.setattr(b, "_native_module", None)
    monkeypatch.setitem(__import__("sys").modules, b.__package__ + "._native", None)
    monkeypatch.delattr(sv, "_native", raising=False)
    with pytest.raises(RuntimeError, match="build"):
        b._native()


# -------------------------------------------------------------------- rope

def test_frequencies():
    """Each kind of scaling at the pairs where its value is known."""
    radians = lambda r: [x % (1 << 64) / 2.0 ** 64 * 2 * math.pi  # noqa: E731
                         for x in r["freq"].tolist()]
    rope = lambda **kw: sv.rope(128, 5e5, device="cpu", **kw)  # noqa: E731
    plain = radians(rope())
    assert plain == pytest.approx([5e5 ** (-c / 64) for c in range(64)], rel=1e-14)
    assert radians(rope(scaling=dict(type="linear", factor=4))) == pytest.approx(
        [x / 4 for x in plain], rel=1e-14)
    ntk = radians(rope(scaling=dict(type="ntk", factor=4)))
    assert ntk[0] == 1 and ntk[63] == pytest.approx(plain[63] / 4, rel=1e-12)
    yarn = rope(scaling=dict(type="yarn", factor=8, context=8192))
    assert yarn["scale"] == pytest.approx(0.1 * math.log(8) + 1)
    y = [a / b for a, b in zip(radians(yarn), plain)]
    turns = [8192 * x / (2 * math.pi) for x in plain]
    for ratio, n in zip(y, turns):
        assert 1 / 8 - 1e-9 <= ratio <= 1 + 1e-9
        if n > 40:
            assert ratio == pytest.approx(1)
        if n < 0.8:
            assert ratio == pytest.approx(1 / 8)
    assert all(a >= c - 1e-9 for a, c in zip(y, y[1:]))
    wave = [a / b for a, b in zip(radians(rope(scaling=dict(
        type="wavelength", factor=8, context=8192, low=1, high=4))), plain)]
    for ratio, n in zip(wave, turns):
        want = 1 if n >= 4 else 1 / 8 if n <= 1 else (n - 1) / 3 + (1 - (n - 1) / 3) / 8
        assert ratio == pytest.approx(want, rel=1e-9)
    f = radians(rope(scaling=dict(type="factors", factors=[2.0] * 32 + [5.0] * 32)))
    assert f[0] == pytest.approx(0.5) and f[63] == pytest.approx(plain[63] / 5)
    # above half a turn, and backwards: the same angles
    r = dict(freq=sv.rope_turns([5.0, -1.0], "cpu"))
    assert radians(r) == pytest.approx([5.0, 2 * math.pi - 1])
    for bad in (dict(dim=24), dict(dim=0), dict(dim=272), dict(base=0.0), dict(base=math.inf),
                dict(scaling=dict(type="other")), dict(scaling=dict(type="factors", factors=[1])),
                dict(scaling=dict(type="factors", factors=[0.0] * 32)), dict(scaling={}, dim=8),
                dict(scaling=dict(factor=2)), dict(scaling=dict(type="linear")),
                dict(scaling=dict(type="linear", factor=0)), dict(scaling=dict(type="yarn", factor=2)),
                dict(scaling=dict(type="yarn", factor=2, context=8192), base=1.0),
                dict(scaling=dict(type="linear", factor=2, context=8192)),
                dict(scaling=dict(type="wavelength", factor=2, context=8192, low=4, high=4))):
        with pytest.raises(ValueError):
            sv.rope(**(dict(dim=64, device="cpu") | bad))


# --------------------------------------------- the plain implementations' pins

def test_plain_rotation():
    """A quarter turn, norms that survive turning, and positions that only matter
    by their differences."""
    rope = dict(freq=torch.tensor([1 << 62] * 8), dim=16, interleaved=False, scale=1.0)
    x = np.arange(16.0).reshape(1, 1, 1, 16)
    y, _ = ru.rotated(x, [[1]], rope)
    assert np.allclose(y[0, 0, 0], np.concatenate([-np.arange(8, 16), np.arange(8)]))
    y, _ = ru.rotated(x, [[1]], dict(rope, interleaved=True))
    assert np.allclose(y[0, 0, 0, :4], [-1, 0, -3, 2])
    rng = np.random.default_rng(1)
    rope = sv.rope(64, device="cpu", interleaved=True)
    q, k = rng.normal(size=(2, 1, 1, 1, 64))
    dots = [np.vdot(ru.rotated(q, [[a]], rope)[0], ru.rotated(k, [[c]], rope)[0])
            for a, c in ((5, 2), (1000003, 1000000), (0, -3))]
    assert np.allclose(dots, dots[0], atol=1e-9)
    y, _ = ru.rotated(q, [[9]], None, None, 1e-9)
    assert np.isclose((y ** 2).mean(), 1)


def test_plain_log_probabilities():
    row = ru.Row(np.log(np.array([0.5, 0.25, 0.125, 0.125])) + 3.0)
    assert np.allclose(np.exp(row.lp), [0.5, 0.25, 0.125, 0.125])
    assert np.isclose(row.entropy, 1.75 * math.log(2))
    assert row.top(3).tolist() == [0, 1, 2]
    row = ru.Row(np.array([1.0, -np.inf, 1.0, 1.0]), 0.5)
    assert np.isclose(row.entropy, math.log(3)) and row.top(9).tolist() == [0, 2, 3]
    assert (np.isfinite(row.bounds()[0])).all()


# ------------------------------------------------------------------ builds

def preprocessed(name, **kw):
    flags = [f for f in _build.compile_flags(**kw) if f.startswith(("-I", "-D", "-std"))]
    return subprocess.run([_build.nvcc(), "-E", "-x", "cu", *flags,
                           os.path.join(_build.CSRC, name)], capture_output=True, text=True,
                          check=True).stdout


def test_nvtx_build_opens_a_range_per_call():
    for unit, names in (("rotate.cu", ("sv_rotate", "sv_kv_append")),
                        ("logprobs.cu", ("sv_token_logprobs",))):
        out = preprocessed(unit, nvtx=True)
        for name in names:
            assert re.search(r"sv_status\s+" + name + r"\s*\([^{]*\{\s*const\s+SvKvRange\s+sv_range_"
                             r"\s*\(\s*\"" + name + r"\"\s*\)", out), name
        assert "SvKvRange" not in preprocessed(unit)


# ------------------------------------------------------- the likeliest tokens

def search(keys, n, bound, top):
    """The steps in which the kernel looks for the n-th largest of `keys` (at least
    n of them, or not, reach `bound`): (it, the next key up, how many reach that)."""
    lo, hi, above, enough, step = bound, top, 0, True, 0
    while step < 20 and enough and (step == 0 or hi - lo > 1):
        part = (hi - lo) // 4
        at = ([lo, lo + 1, lo + 2 * part] if step == 0 else
              [lo + max(part, 1), lo + max(2 * part, 1), lo + max(3 * part, 1)])
        count = [int((keys >= x).sum()) for x in at]
        for q in (2, 1, 0):
            if count[q] < n:
                hi, above = at[q], count[q]
        enough = hi != lo
        for x in at:
            if lo < x < hi:
                lo = x
        step += 1
    return (lo, hi, above) if enough else None


def test_the_search_finds_the_last_group():
    rng = np.random.default_rng(2)
    for trial in range(2000):
        top = 0x10000 if trial % 2 else 0xffffffff
        span = int(rng.choice([1, 2, 5, 100, 5000, top - 300]))
        base = int(rng.integers(129, top - 100 - span)) if span < top - 300 else 129
        keys = np.minimum(base + rng.integers(0, span + 1, rng.integers(1, 200)), top - 1)
        n = int(rng.integers(1, 65))
        bound = int(rng.choice([keys.min(), 128]))
        got = search(keys, n, bound, top)
        if len(keys) < n:
            assert got is None
        else:
            last = int(np.sort(keys)[-n])
            assert got == (last, last + 1, int((keys > last).sum()))


def test_the_best_groups_hold_the_likeliest_tokens():
    """The n largest logits (lower ids first among equal ones) lie in the n groups of
    largest maxima (lower groups first), and reach the last of these maxima; a bound
    from maxima of disjoint sets of groups leaves none of them out."""
    rng = np.random.default_rng(3)
    for trial in range(300):
        V, n = int(rng.integers(1, 900)), int(rng.integers(1, 65))
        kind = trial % 4
        x = (rng.normal(size=V) if kind == 0 else rng.integers(0, 3, V).astype(float) if kind == 1
             else np.zeros(V) if kind == 2 else np.sort(rng.normal(size=V)))
        want = ru.Row(x).top(n)
        padded = np.append(x, np.full(-V % 16, -np.inf)).reshape(-1, 16)
        groups = padded.max(1)
        best = np.lexsort((np.arange(len(groups)), -groups))[:n]
        assert set(want // 16) <= set(best)
        if len(groups) >= n:
            assert (x[want] >= groups[best[-1]]).all()
        sets = [groups[i::7].max() for i in range(7) if i < len(groups)]
        if len(sets) >= n:
            bound = np.sort(sets)[-n]
            assert (groups >= bound).sum() >= n and (x[want] >= bound).all()


def test_results_without_tokens_and_head_counts_past_32_bits_are_refused(native):
    a = tensors("token_logprobs")
    with pytest.raises(ValueError, match="no tokens"):
        native.token_logprobs(*(a | dict(tokens=None)).values())
    native.token_logprobs(*(a | dict(tokens=None, logprobs=None)).values())
    many = torch.zeros(64, dtype=torch.bfloat16).as_strided((2, 3, (1 << 32) + 4, 64), (0, 0, 0, 1))
    with pytest.raises(ValueError, match="out of range"):
        native.rotate(*(tensors("rotate") | dict(q=many, q_out=...)).values())
