"""The tree-decoding example: mask, write, attention, verification and commit
of several rounds together, the attention of each against a plain one on the
cache's values."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "tree_decoding", os.path.join(ROOT, "examples", "tree_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rounds_attend_to_what_was_accepted():
    """The cache holds, round after round, the keys of the accepted tokens (up
    to their rounding: half a step of e4m3 for values whose page's scale did
    not grow, and half a step of each scale before), and the attention is the
    formula's on those values."""
    import speculative_decoding_verification_63_gb300 as sv
    ex = example()
    model = ex.Target()
    prompts = [[5, 17, 301, 44, 9], [700], list(range(100, 140))]
    seen = []

    def check(q, cache, table, length, mask, out):
        B, N = q.shape[:2]
        total = int(length.max()) + N
        got = sv.kv_read(cache, table, torch.zeros_like(length), length + N, total,
                         dtype=torch.float32)
        k, v = (got[s].double().repeat_interleave(ex.HEADS // ex.KV_HEADS, 2) for s in "kv")
        pos = torch.arange(total, device="cuda") - length[:, None]  # [B][total]
        bits = mask[:, :, 0][:, :, None] >> pos.clamp(0, 31)[:, None] & 1
        sees = (pos < 0)[:, None] | ((pos >= 0) & (pos < N))[:, None] & (bits == 1)
        x = torch.einsum("bthd,bshd->bhts", q.double(), k) * ex.DIM ** -0.5
        p = x.masked_fill(~sees[:, None], -torch.inf).softmax(-1)
        want = torch.einsum("bhts,bshd->bthd", p, v)
        size = torch.einsum("bhts,bshd->bthd", p, v.abs())
        # bf16 results (2^-8), weights of 11 bits and scores in 32 bits
        assert ((out.double() - want).abs() <= want.abs() * 2 ** -8 + size * 2 ** -9).all()
        seen.append((cache, table, length.clone()))

    emitted = ex.decode(prompts, 6, model, check)
    assert len(seen) == 6
    _, table, _ = seen[-1]
    cache = seen[-1][0]
    assert any(len(e) > 6 for e in emitted)  # some draft was accepted
    for b, (prompt, tokens) in enumerate(zip(prompts, emitted)):
        held = (prompt + tokens)[:-1]  # the last token is the next root
        n = torch.tensor([len(held)], dtype=torch.int32, device="cuda")
        got = sv.kv_read(cache, table[b:b + 1], torch.zeros_like(n), n, len(held),
                         dtype=torch.float32)
        _, _, k, v = model.qkv(torch.tensor([held], device="cuda"))
        for s, x in (("k", k), ("v", v)):
            # |x| <= 448 * scale on its page and head; e4m3 steps of a value are
            # at most 2^-3 of it, its last place 2^-9 * scale.  A page's scale
            # grows a few times at most, each time by half a step more.
            scale = cache[s + "_scale"][table[b].long()].repeat_interleave(ex.PAGE, 0)[:len(held)]
            err = (got[s][0] - x[0].float()).abs()
            bound = x[0].float().abs() * 2 ** -3 + scale[:, :, None] * 2 ** -8
            assert (err <= bound).all()
