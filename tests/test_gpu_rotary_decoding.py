"""The rotary decoding example: append, attention, verification, commit and log
probabilities of several rounds together, each against its plain form."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import round_util as ru  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "rotary_decoding", os.path.join(ROOT, "examples", "rotary_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rounds():
    import speculative_decoding_verification_63_gb300 as sv
    ex = example()
    model = ex.RotaryTarget()
    prompts = [[5, 17, 301, 44, 9], [700], list(range(100, 140))]
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    wq, wk = f64(model.q_norm), f64(model.k_norm)
    rounds = []

    def check(cache, table, length, tokens, q, logits, got, said):
        B, N = tokens.shape
        depth = [0, 1, 2, 2, 1, 2, 2]
        _, plain_q, _, _ = model.qkv(tokens)
        pos = [[int(length[b]) + d for d in depth] for b in range(B)]
        y, size = ru.rotated(f64(plain_q), pos, model.rope, wq, ex.EPS)
        off = ru.rounding("bf16", y, ru.rotation_bound(size))
        assert (np.abs(f64(q) - y) <= off).all()
        # what the round emitted, under the logits of its rows
        out_len = got["out_len"].tolist()
        for b, n in enumerate(out_len):
            rows = [0] + got["accepted_nodes"][b].tolist()
            for r in range(n):
                row = ru.Row(f64(logits[b, rows[r]]))
                lp_off, h_off = row.bounds()
                t = int(got["out_tokens"][b, r])
                assert abs(float(said["logprobs"][b, r]) - row.lp[t]) <= lp_off[t]
                assert abs(float(said["entropy"][b, r]) - row.entropy) <= h_off
                best = row.top(3)
                assert said["top_tokens"][b, r].tolist() == best.tolist() and best[0] == t
            assert torch.isnan(said["entropy"][b, n:]).all()
        rounds.append(out_len)

    emitted = ex.decode(prompts, 6, model, check=check)
    assert len(rounds) == 6 and any(n > 1 for r in rounds for n in r)
    assert [len(e) for e in emitted] == np.array(rounds).sum(0).tolist()


def test_the_cache_holds_keys_at_their_places():
    """After prompts and rounds, the cached keys are those of the tokens in order,
    turned to their places (up to their rounding: half a step of e4m3, more for pages
    whose scale grew)."""
    import speculative_decoding_verification_63_gb300 as sv
    ex = example()
    model = ex.RotaryTarget()
    prompts = [[5, 17, 301, 44, 9], [700], list(range(100, 140))]
    last = {}
    emitted = ex.decode(prompts, 6, model, check=lambda **kw: last.update(kw))
    cache, table = last["cache"], last["table"]
    for b, (prompt, said) in enumerate(zip(prompts, emitted)):
        held = (prompt + [t for t, *_ in said])[:-1]  # the last token is the next root
        n = torch.tensor([len(held)], dtype=torch.int32, device="cuda")
        got = sv.kv_read(cache, table[b:b + 1], torch.zeros_like(n), n, len(held),
                         dtype=torch.float32)
        _, _, k, _ = model.qkv(torch.tensor([held], device="cuda"))
        y, _ = ru.rotated(k.double().cpu().numpy(), [list(range(len(held)))], model.rope,
                          model.k_norm.double().cpu().numpy(), ex.EPS)
        y = torch.from_numpy(y[0]).cuda()
        scale = cache["k_scale"][table[b].long()].repeat_interleave(ex.PAGE, 0)[:len(held)]
        err = (got["k"][0].double() - y).abs()
        assert (err <= y.abs() * 2 ** -3 + scale[:, :, None] * 2 ** -8).all()
