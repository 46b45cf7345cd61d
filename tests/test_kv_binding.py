"""The cache's Python calls without a GPU: which workspace serves whom."""
import gc
import weakref

import pytest
import torch

import speculative_decoding_verification_63_gb300 as sv


class FakeBuffer:
    def __init__(self, n):
        self.n = n

    def numel(self):
        return self.n

    def data_ptr(self):
        return 256


class FakeGpu:
    """What workspace() asks of torch and the library."""
    stream, capture = 7, 0

    def __init__(self, mp):
        mp.setattr(sv, "_ws_cache", {})
        mp.setattr(torch, "empty", lambda n, **kw: FakeBuffer(n))
        mp.setattr(sv, "sv_workspace_init", lambda buf, stream=None: None)
        mp.setattr(sv, "sv_stream_capture_id", lambda stream: self.capture, raising=False)
        mp.setattr(sv, "current_raw_stream", lambda device: self.stream)
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capture != 0)
        mp.setattr(torch.cuda, "current_stream", lambda device=None: self)

    def synchronize(self):
        pass


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch)


DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("key", ["kv_attention", "kv", "chain"])
def test_a_replaced_workspace_stays_allocated(gpu, key):
    small = sv.workspace(5_000_000, DEV, key)
    assert sv.workspace(4_000_000, DEV, key) is small
    alive = weakref.ref(small)
    del small
    big = sv.workspace(21_000_000, DEV, key)
    gc.collect()
    assert alive() is not None and alive() is not big
    assert sv.workspace(1, DEV, key) is big


def test_attention_has_one_workspace_a_stream(gpu):
    first, other = sv.workspace(100, DEV, "kv_attention"), sv.workspace(100, DEV, "kv")
    gpu.stream = 8
    second = sv.workspace(100, DEV, "kv_attention")
    assert second is not first and sv.workspace(100, DEV, "kv") is other
    gpu.stream = 7
    assert sv.workspace(100, DEV, "kv_attention") is first


def test_a_capture_has_workspaces_of_its_own(gpu):
    eager, kv = sv.workspace(100, DEV, "kv_attention"), sv.workspace(100, DEV, "kv")
    gpu.capture = 1
    one = sv.workspace(100, DEV, "kv_attention")
    assert one is not eager and sv.workspace(90, DEV, "kv_attention") is one
    assert sv.workspace(100, DEV, "kv") is kv        # only its error word is used
    new = sv.workspace(100, DEV, "tree")
    gpu.capture = 2
    two = sv.workspace(100, DEV, "kv_attention")
    assert two is not one and two is not eager
    gpu.capture = 0
    assert sv.workspace(100, DEV, "kv_attention") is eager
    assert sv.workspace(100, DEV, "tree") is not new  # the graph's stays the graph's


# ------------------------------------------------------------------ devices

class OnDevice:
    """A CPU tensor that says it lives on a GPU."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)

    @property
    def is_cuda(self):
        return True


class Launches(list):
    def __getattr__(self, name):
        return lambda *args: (self.append(name), 0)[1]


OPERANDS = {"write": ["page_table", "kv_len", "k_new", "v_new", "num_new", "workspace"],
            "read": ["page_table", "start", "num", "k_out", "v_out", "rows", "workspace"],
            "attention": ["page_table", "kv_len", "q", "out", "num_new", "mask", "lse",
                          "workspace"]}


def kv_arguments(op):
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    z = lambda: torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = lambda h: torch.zeros((2, 3, h, 64), dtype=torch.bfloat16)
    a = dict(k=z(), v=z(), k_scale=torch.ones(4, 2), v_scale=torch.ones(4, 2), page_table=i32(2, 2),
             workspace=torch.zeros(8192, dtype=torch.uint8))
    a.update({"write": dict(kv_len=i32(2), k_new=x(2), v_new=x(2), num_new=i32(2)),
              "read": dict(start=i32(2), num=i32(2), k_out=x(2), v_out=x(2), rows=i32(2, 3)),
              "attention": dict(kv_len=i32(2), q=x(4), out=x(4), num_new=i32(2), mask=i32(2, 3, 1),
                                lse=torch.zeros(2, 3, 4))}[op])
    return a


def kv_call(op, a):
    a = dict(a)
    cache = {n: a.pop(n) for n in ("k", "v", "k_scale", "v_scale")}
    if op == "attention":
        a["scale"] = 0.125
    getattr(sv, "sv_kv_" + op)(cache, **a) if op != "attention" else \
        sv.sv_kv_attention(a.pop("q"), cache, **a)


@pytest.mark.parametrize("op", ["write", "read", "attention"])
def test_tensors_of_another_device_are_refused(op, monkeypatch):
    """Every tensor has to be on the workspace's device and that one be current;
    nothing is launched otherwise."""
    b = sv._binding
    launches = Launches()
    monkeypatch.setattr(b, "_lib_handle", launches)
    current = [0]
    monkeypatch.setattr(b, "_current_device", lambda: current[0])
    monkeypatch.setattr(b, "current_raw_stream", lambda d: 0)
    args = kv_arguments(op)
    names = ["k", "v", "k_scale", "v_scale"] + OPERANDS[op]
    assert sorted(names) == sorted(args)
    everywhere = lambda index: {n: OnDevice(t, index) for n, t in args.items()}
    kv_call(op, everywhere(0))
    assert launches == ["sv_kv_" + op]
    for n in names:
        with pytest.raises(ValueError, match="device"):
            kv_call(op, dict(everywhere(0), **{n: OnDevice(args[n], 1)}))
        with pytest.raises(ValueError, match="device"):
            kv_call(op, dict(everywhere(0), **{n: args[n]}))
    with pytest.raises(ValueError, match="current device"):
        kv_call(op, everywhere(1))
    with pytest.raises(ValueError, match="device tensors"):
        kv_call(op, args)
    assert len(launches) == 1
    current[0] = 1
    kv_call(op, everywhere(1))
    assert len(launches) == 2


# ------------------------------------------------------------------ strides

def packed_arguments(op, args, monkeypatch):
    """The C arguments of a call, without launching it."""
    b, out = sv._binding, []
    cls = {"write": b.SvKvWriteArgs, "read": b.SvKvReadArgs, "attention": b.SvKvAttentionArgs}[op]
    monkeypatch.setattr(b, "_kv_call", lambda name, packed, *rest: out.append(packed))
    kv_call(op, args)
    return cls.from_buffer_copy(out[0])


def test_strides_of_dimensions_of_one(monkeypatch):
    """They say nothing, and differ between tensors that are laid out alike."""
    odd = lambda t, dim, stride: t.as_strided(
        t.shape, [stride if i == dim else s for i, s in enumerate(t.stride())])
    raw = torch.zeros((1, 1, 16, 64), dtype=torch.uint8)
    code = lambda t: t.view(torch.float8_e4m3fn)
    cache = dict(k=code(raw), v=code(odd(odd(raw, 0, 8), 1, 8)), k_scale=torch.ones(1, 1),
                 v_scale=torch.ones(1, 1))
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    ws = torch.zeros(8192, dtype=torch.uint8)
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    y = odd(odd(odd(x, 0, 3), 1, 5), 2, 7)
    a = packed_arguments("read", dict(cache, page_table=i32(1, 1), start=i32(1), num=i32(1), k_out=x,
                                      v_out=y, workspace=ws), monkeypatch)
    assert (a.cache.page_stride, a.cache.head_stride) == (0, 16 * 64)
    assert (a.out_batch_stride, a.out_token_stride, a.out_head_stride) == (0, 0, 0)
    a = packed_arguments("write", dict(cache, page_table=i32(1, 1), kv_len=i32(1), k_new=y, v_new=x,
                                       workspace=ws), monkeypatch)
    assert (a.k_batch_stride, a.k_token_stride, a.k_head_stride) == (0, 0, 0)
    a = packed_arguments("attention", dict(cache, page_table=i32(1, 1), kv_len=i32(1), q=y,
                                           out=torch.zeros_like(x), workspace=ws), monkeypatch)
    assert (a.q_batch_stride, a.q_token_stride, a.q_head_stride) == (0, 0, 0)
    # strides of other dimensions count as before
    args = kv_arguments("read")
    a = packed_arguments("read", args, monkeypatch)
    assert (a.out_batch_stride, a.out_token_stride, a.out_head_stride) == (384, 128, 64)
    wide = torch.zeros((2, 3, 2, 80), dtype=torch.bfloat16)[..., :64]
    with pytest.raises(ValueError):
        packed_arguments("read", dict(args, v_out=wide), monkeypatch)
    with pytest.raises(ValueError):
        packed_arguments("read", dict(args, v=torch.zeros((4, 2, 17, 64), dtype=torch.uint8).view(
            torch.float8_e4m3fn)[:, :, :16]), monkeypatch)


@pytest.mark.parametrize("op,name", [("write", "k_new"), ("write", "v_new"), ("read", "v_out"),
                                     ("attention", "q"), ("write", "k"), ("read", "page_table")])
def test_other_numbers_of_dimensions_are_refused(op, name):
    args = kv_arguments(op)
    for t in (args[name][0], args[name][None], args[name].flatten()):
        with pytest.raises(ValueError):
            kv_call(op, dict(args, **{name: t}))
