"""The 8-bit key/value cache without a GPU: struct layouts, refusals before
any device work, the plain implementation's own pins, and the attention's
division of work."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import kv_util

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, WS = 0x100000, ctypes.c_void_p(0x200000)
BIG = 1 << 30


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_verification_63_gb300 import _binding, _build
    _build.build_library()
    _binding.lib()
    return _binding


def test_struct_layout_matches_binding(tmp_path, b):
    header = os.path.join(ROOT, "include")
    lines = ['#include "specverify.h"', "#include <stdio.h>", "#include <stddef.h>",
             "int main(void) {"]
    expect = []
    for cname, cls in [("sv_kv_cache", b.SvKvCache), ("sv_kv_write_args", b.SvKvWriteArgs),
                       ("sv_kv_read_args", b.SvKvReadArgs),
                       ("sv_kv_attention_args", b.SvKvAttentionArgs)]:
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        expect.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({cname}, {f}));')
            expect.append(getattr(cls, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", f"-I{header}", "-o", str(exe), str(c)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in got.split()] == expect


def _cache(c, **kw):
    c.num_pages, c.page_size, c.Hkv, c.D, c.slots = 8, 16, 2, 64, 4
    c.k = c.v = c.k_scale = c.v_scale = c.page_table = FAKE
    c.head_stride, c.page_stride = 16 * 64, 2 * 16 * 64
    for k, v in kw.items():
        setattr(c, k, v)


def _args(b, op, cache=None, **kw):
    a = {"write": b.SvKvWriteArgs, "read": b.SvKvReadArgs,
         "attention": b.SvKvAttentionArgs}[op]()
    _cache(a.cache, **(cache or {}))
    a.B, a.T, a.dtype = 2, 4, b.SV_BF16
    for f, t in a._fields_:
        if t is ctypes.c_void_p and f not in ("lse", "mask", "num_new", "num", "rows"):
            setattr(a, f, FAKE)
    if op == "attention":
        a.Hq, a.scale = 4, 0.125
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _call(b, op, a, ws=WS, n=BIG):
    return getattr(b.lib(), "sv_kv_" + op)(bytes(a), ws, n, None)


BAD_CACHES = [dict(num_pages=0), dict(slots=0), dict(Hkv=0), dict(Hkv=257), dict(page_size=8),
              dict(page_size=48), dict(page_size=256), dict(D=32), dict(D=96), dict(k=None),
              dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 1), dict(k_scale=None),
              dict(v_scale=None), dict(page_table=None), dict(head_stride=16 * 64 - 16),
              dict(head_stride=16 * 64 + 8), dict(page_stride=2 * 16 * 64 + 4),
              dict(page_stride=-16), dict(slots=1 << 28)]


@pytest.mark.parametrize("op", ["write", "read", "attention"])
def test_refusals(b, op):
    assert getattr(b.lib(), "sv_kv_" + op)(None, WS, BIG, None) == b.SV_EINVAL
    assert _call(b, op, _args(b, op, B=0)) == b.SV_OK
    for kw in [dict(B=-1), dict(B=b.SV_MAX_B + 1), dict(T=0), dict(T=-3), dict(dtype=3),
               dict(dtype=-1)]:
        assert _call(b, op, _args(b, op, **kw)) == b.SV_EINVAL, kw
    for c in BAD_CACHES:
        if op == "attention" and c.get("Hkv") == 257:
            continue
        assert _call(b, op, _args(b, op, cache=c)) == b.SV_EINVAL, c
    need = {"write": ["k_new", "v_new", "kv_len"], "read": ["k_out", "v_out"],
            "attention": ["q", "out", "kv_len"]}[op]
    for f in need:
        assert _call(b, op, _args(b, op, **{f: None})) == b.SV_EINVAL, f
    ok = _args(b, op)
    assert _call(b, op, ok, ws=ctypes.c_void_p(0)) == b.SV_EWORKSPACE
    assert _call(b, op, ok, ws=ctypes.c_void_p(0x200010)) == b.SV_EWORKSPACE
    assert _call(b, op, ok, n=b.SV_MIN_WORKSPACE_BYTES - 1) == b.SV_EWORKSPACE


def test_refusals_of_one_call(b):
    att = lambda **kw: _call(b, "attention", _args(b, "attention", **kw))
    assert att(dtype=b.SV_FP32) == b.SV_EINVAL
    for kw in [dict(Hq=3), dict(Hq=1), dict(Hq=258), dict(scale=math.nan), dict(scale=math.inf),
               dict(out=FAKE + 8), dict(q=FAKE + 1), dict(T=b.SV_MAX_KV_T + 1),
               dict(mask=FAKE, words=0), dict(mask=FAKE, T=33, words=1),
               dict(mask=FAKE, T=65, words=3)]:
        assert att(**kw) == b.SV_EINVAL, kw
    assert b.sv_kv_attention_workspace_bytes(1, 1, 8, 2, 128) > b.SV_MIN_WORKSPACE_BYTES
    for bad in [(-1, 1, 8, 2, 128), (1025, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 8, 3, 128),
                (1, 1, 8, 2, 80), (1, 1, 0, 0, 128), (1, 1, 512, 2, 64)]:
        assert b.sv_kv_attention_workspace_bytes(*bad) == 0, bad
    assert _call(b, "attention", _args(b, "attention"), n=1 << 14) == b.SV_EWORKSPACE
    assert _call(b, "write", _args(b, "write", T=b.SV_MAX_KV_T + 1)) == b.SV_EINVAL
    assert _call(b, "write", _args(b, "write", k_new=FAKE + 1)) == b.SV_EINVAL


def _tensors(pages=4, H=2, P=16, D=64, B=2, slots=2):
    z = torch.zeros((pages, H, P, D), dtype=torch.uint8).view(torch.float8_e4m3fn)
    one = torch.ones((pages, H))
    return (dict(k=z, v=z.clone(), k_scale=one, v_scale=one.clone()),
            torch.zeros((B, slots), dtype=torch.int32), torch.zeros(B, dtype=torch.int32))


def test_binding_refuses_wrong_tensors(b):
    import speculative_decoding_verification_63_gb300 as sv
    ws = torch.zeros(8192, dtype=torch.uint8)
    x = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)

    def refused(change, what):
        cache, table, length = _tensors()
        args = dict(cache=cache, page_table=table, kv_len=length, k=x, v=x, q=q, num=None, mask=None)
        change(args)
        with pytest.raises(ValueError):
            if what == "write":
                sv.kv_write(args["cache"], args["page_table"], args["kv_len"], args["k"],
                            args["v"], num_new=args["num"], ws=ws)
            else:
                sv.kv_attention(args["q"], args["cache"], args["page_table"], args["kv_len"],
                                num_new=args["num"], mask=args["mask"], ws=ws)

    for what in ("write", "attention"):
        refused(lambda a: a["cache"].update(k=a["cache"]["k"].view(torch.uint8)), what)
        refused(lambda a: a["cache"].update(v=a["cache"]["v"][:2]), what)
        refused(lambda a: a["cache"].update(v=a["cache"]["v"].transpose(0, 1)), what)
        refused(lambda a: a["cache"].update(k_scale=torch.ones(4, 2, dtype=torch.float64)), what)
        refused(lambda a: a["cache"].update(v_scale=torch.ones(4, 3)), what)
        refused(lambda a: a.update(page_table=a["page_table"].long()), what)
        refused(lambda a: a.update(page_table=a["page_table"][:1]), what)
        refused(lambda a: a.update(kv_len=torch.zeros(3, dtype=torch.int32)), what)
        refused(lambda a: a.update(num=torch.zeros(2)), what)
        refused(lambda a: None, what)  # not on a device
    refused(lambda a: a.update(k=x[..., :32]), "write")
    refused(lambda a: a.update(v=x.float()), "write")
    refused(lambda a: a.update(k=x.transpose(2, 3).contiguous().transpose(2, 3)), "write")
    refused(lambda a: a.update(q=q.float()), "attention")
    refused(lambda a: a.update(q=q[..., :32]), "attention")
    refused(lambda a: a.update(mask=torch.zeros(2, 3, dtype=torch.int32)), "attention")


def test_packed_arguments_are_the_structs(b):
    """The binding's packed arguments have the layout of the C structs."""
    import struct
    for cls in (b.SvKvWriteArgs, b.SvKvReadArgs, b.SvKvAttentionArgs):
        packer = b._packer(cls)
        flat = []
        for name, t in cls._fields_:
            flat += [(name, f, u) for f, u in t._fields_] if issubclass(t, ctypes.Structure) \
                else [(None, name, t)]
        values = [0.25 * i if t is ctypes.c_float else 1000 + i for i, (_, _, t) in enumerate(flat)]
        a = cls.from_buffer_copy(packer.pack(*values))
        for (outer, name, _), want in zip(flat, values):
            assert getattr(getattr(a, outer) if outer else a, name) == want, name
        assert isinstance(packer, struct.Struct)


# ------------------------------------------------ the plain implementation

def test_e4m3_grid():
    v = kv_util.E4M3
    assert v[0x7e] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9
    assert math.isnan(v[0x7f]) and math.isnan(v[0xff]) and v[0xfe] == -448.0
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, v, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=20000) * 2.0 ** rng.integers(-10, 9, 20000),
                        (kv_util._GRID[1:] + kv_util._GRID[:-1]) / 2, kv_util._GRID])
    x = np.clip(np.concatenate([x, -x]), -448, 448)
    want = torch.from_numpy(x).float()
    keep = want.double().numpy() == x  # exact in fp32: no double rounding
    got = kv_util.encode(x)
    ref = want.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got[keep], ref[keep]) and keep.sum() > 500
    assert kv_util.encode(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7e, 0xfe, 0x7f]


def test_needed_exponent():
    assert kv_util.needed_exp(448.0) == 0 and kv_util.needed_exp(448.1) == 1
    assert kv_util.needed_exp(224.0) == -1 and kv_util.needed_exp(0.0) == kv_util.EXP_LO
    assert kv_util.needed_exp(1e-30) == kv_util.EXP_LO and kv_util.needed_exp(1e30) == kv_util.EXP_HI


# ------------------------------------------------- the attention's division

@pytest.mark.parametrize("seed", range(40))
def test_division_of_work(seed):
    """The attention cuts the list of all blocks into equal parts, one a CTA.
    A unit that is cut is joined by the CTA that arrives last: its parts lie
    with CTAs first .. last, each in a slot of its own, and its ticket is its
    first CTA's alone.  The integer expressions are the kernel's."""
    rng = np.random.default_rng(seed)
    units = rng.integers(1, rng.choice([2, 5, 80, 700]), rng.integers(1, 300))
    total, grid, least = int(units.sum()), int(rng.integers(1, 305)), int(rng.choice([2, 4]))
    parts = max(1, min(grid, total // least))
    per = total // parts
    more = total - per * parts
    bound = [c * per + min(c, more) for c in range(parts + 1)]

    def part_of(x):
        cut = more * (per + 1)
        return x // (per + 1) if x < cut else more + (x - cut) // per

    held, tickets, slots = np.zeros(total, int), {}, set()
    starts = np.concatenate([[0], np.cumsum(units)])
    for u, n in enumerate(units):
        u0 = int(starts[u])
        first, last = part_of(u0), part_of(u0 + int(n) - 1)
        assert bound[first] <= u0 < bound[first + 1]
        assert bound[last] <= u0 + n - 1 < bound[last + 1]
        if first == last:
            continue
        assert first not in tickets
        tickets[first] = u
        for c in range(first, last + 1):
            begins_here = bound[c] <= u0
            slot = (c, 1 if begins_here else 0)
            assert begins_here == (c == first) and slot not in slots
            slots.add(slot)
    for c in range(parts):
        assert bound[c] < bound[c + 1]
        held[bound[c]:bound[c + 1]] += 1
    assert bound[-1] == total and (held == 1).all()


def test_rows_divide_by_the_group():
    """A row's round token is the high word of row * (floor(2^32 / G) + 1),
    for every group and every row a call can have."""
    for G in range(2, 257):
        magic = 2 ** 32 // G + 1
        rows = np.unique(np.concatenate([np.arange(0, 3000), 65536 * G - 1 - np.arange(0, 3000),
                                         G * np.random.default_rng(G).integers(0, 65536, 3000)
                                         - 1 + np.array([[0], [1]])], axis=None))
        rows = rows[(rows >= 0) & (rows < 65536 * G)].astype(np.uint64)
        assert (rows < 2 ** 24).all() and ((rows * np.uint64(magic)) >> np.uint64(32)
                                           == rows // np.uint64(G)).all(), G


def test_chunks_divide_by_a_tokens_chunks():
    """The read kernel's division of a block's chunk index (below 1024 + one
    token's chunks) by the chunks of a token."""
    for heads in range(1, 257):
        for d in (4, 8):
            per = heads * d
            at = np.arange(0, max(1, 1024 // per) * per + 1024, dtype=np.uint64)
            magic = 2 ** 32 // per + 1
            assert ((at * np.uint64(magic)) >> np.uint64(32) == at // np.uint64(per)).all()
