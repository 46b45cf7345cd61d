"""Calls around the target's pass that are refused, without a GPU."""
import numpy as np
import pytest

from test_round_host import b, native, tensors  # noqa: F401


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
