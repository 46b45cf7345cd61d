"""Calls around the target's pass that are refused, without a GPU."""
import numpy as np
import pytest

import speculative_decoding_verification_63_gb300 as sv
from test_round_host import FAKE, _append, _call, _rotate, b, native, tensors  # noqa: F401


class Unclear:
    """Has no truth value."""

    def __bool__(self):
        raise KeyError("unclear")


def test_flags_without_a_truth_value_are_refused(b, native):  # noqa: F811
    """... with their own error, before the call gets as far as the device."""
    entry = lambda op: b._entry("sv_" + op)  # noqa: E731
    for op in ("rotate", "kv_append"):
        a = tensors(op) | dict(entry=entry(op))
        for what, error in ((np.zeros(2), "truth value"), (Unclear(), "unclear")):
            a["rope"] = dict(a["rope"], interleaved=what)
            with pytest.raises((ValueError, KeyError), match=error):
                getattr(native, op)(*a.values())
        a["rope"] = dict(a["rope"], interleaved=np.ones(1, bool))  # (this one has one)
        with pytest.raises(ValueError, match="device tensors"):
            getattr(native, op)(*a.values())
    for what, error in ((np.zeros(2), "truth value"), (Unclear(), "unclear")):
        a = tensors("token_logprobs") | dict(entry=entry("token_logprobs"), allocate=what)
        with pytest.raises((ValueError, KeyError), match=error):
            native.token_logprobs(*a.values())


# ------------------------------------------------- results that share places

def places(at, heads, step, D, es):
    """Bytes of the heads of one token."""
    return {x for h in range(heads) for x in range(at + h * step * es, at + (h * step + D) * es)}


LAYOUTS = [  # q: x, out, heads, step; k: x, out, heads, step (elements of two bytes from one place)
    ((0, 0, 4, 64), (256, 256, 2, 64)),          # in place, slices of one projection
    ((0, 0, 4, 64), (0, 0, 4, 64)),              # the same heads twice
    ((0, 0, 4, 64), (128, 128, 4, 64)),          # heads of both
    ((0, 0, 4, 192), (64, 64, 4, 192)),          # side by side, kind by kind
    ((0, 0, 4, 192), (32, 32, 4, 192)),
    ((0, 0, 3, 128), (64, 64, 2, 256)),          # other steps, apart
    ((0, 0, 3, 128), (64, 64, 2, 192)),          # other steps, one head of both
    ((0, 1024, 4, 64), (1024, 4096, 2, 64)),     # q's results are k's input
    ((0, 1024, 4, 64), (4096, 192, 2, 64)),      # k's results are q's input
    ((0, 1024, 4, 64), (4096, 1216, 2, 64)),     # results of both
    ((0, 1024, 4, 64), (0, 2048, 4, 64)),        # the same input, results apart
    ((0, 64, 4, 64), (4096, 8192, 2, 64)),       # a head further on in its own input
    ((0, 32, 1, 0), (4096, 8192, 1, 0)),
    ((0, 64, 2, 128), (4096, 8192, 2, 64)),      # between its own input's heads
    ((512, 512, 4, -64), (576, 576, 4, 64)),     # backwards, apart
    ((512, 512, 4, -64), (320, 320, 4, 64)),     # backwards, two heads of both
]


@pytest.mark.parametrize("q,k", LAYOUTS)
def test_results_that_share_places_are_refused(b, q, k):  # noqa: F811
    """Against the sets of bytes of the first token: EINVAL, or on to the workspace's check."""
    D, es = 64, 2
    heads = []
    for x, out, n, step in (q, k):
        heads.append(dict(x=FAKE + x * es, out=FAKE + out * es, heads=n, head_stride=step,
                          out_head_stride=step, D=D))
    sets = [[places(f * es, n, step, D, es) for f in (x, out)] for x, out, n, step in (q, k)]
    own = any(x != out and sets[i][0] & sets[i][1] for i, (x, out, _, _) in enumerate((q, k)))
    both = bool(sets[0][1] & sets[1][1] or sets[0][1] & sets[1][0] or sets[1][1] & sets[0][0])
    for kw in heads:
        kw.update(batch_stride=1 << 14, out_batch_stride=1 << 14, token_stride=1 << 12,
                  out_token_stride=1 << 12)
    args = [{n: v for n, v in kw.items() if n != "D"} for kw in heads]
    want = b.SV_EINVAL if own or both else b.SV_EWORKSPACE
    assert _call(b, "sv_rotate", _rotate(b, q=args[0], k=args[1]), n=0) == want
    assert _call(b, "sv_rotate", _rotate(b, q=args[1], k=args[0]), n=0) == want
    # in an append, k's input stands for the keys or the values
    alone = bool(q[0] != q[1] and sets[0][0] & sets[0][1])
    want = b.SV_EINVAL if alone or sets[0][1] & sets[1][0] else b.SV_EWORKSPACE
    far = dict(k_new=FAKE + (1 << 20), v_new=FAKE + (1 << 20), cache=dict(Hkv=k[2]))
    for side in "kv":
        a = _append(b, q=args[0], **far | {side + "_new": args[1]["x"], side + "_head_stride": k[3]})
        assert _call(b, "sv_kv_append", a, n=0) == want, side


# -------------------------------------------------------------------- rope

@pytest.mark.parametrize("fast,slow", [(1, 32), (0.5, 1)])
def test_yarn_bounds_that_contradict_are_refused(fast, slow):
    """No frequency can be kept as a fast one and stretched as a slow one."""
    with pytest.raises(ValueError, match="slow <= fast"):
        sv.rope(64, device="cpu", scaling=dict(type="yarn", factor=4, context=8192, fast=fast,
                                               slow=slow))


def test_yarn_bounds_that_are_equal_part_the_frequencies():
    radians = lambda **kw: [x % (1 << 64) / 2.0 ** 64 * 2 * np.pi for x in  # noqa: E731
                            sv.rope(64, device="cpu", **kw)["freq"].tolist()]
    plain = radians()
    got = radians(scaling=dict(type="yarn", factor=4, context=8192, fast=4, slow=4))
    for x, y in zip(plain, got):
        turns = 8192 * x / (2 * np.pi)
        assert y == pytest.approx(x if turns > 4 else x / 4, rel=1e-9) or 3 < turns < 5.5
