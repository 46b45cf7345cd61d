"""Around the target model's pass over a round: what is measured.

Three operators beside the verification and the 8-bit key/value cache:

- rotate:   queries and keys as the projections leave them get their heads'
            norms and the rotation of their positions, in one pass;
- append:   the same for a round's queries, keys and values on their way to the
            attention: keys are rotated and, with the values, quantised into the
            paged 8-bit cache, queries come back rotated;
- logprobs: log probabilities of given tokens (those a round emitted, or a
            prompt's), each row's entropy and its most likely tokens.

Rotation.  Channel pairs of the first `rot` channels of a head, (i, i + rot/2)
or, interleaved, (2i, 2i + 1), turn by position * freq[i].  freq is held as a
64-bit fraction of a turn, so positions may be as far as they like.  Token t of
request b sits at start[b] + offset[b][t] (a tree's depths), or start[b] + t.

The cache is a dict of tensors: k, v [pages][heads][page][D] e4m3 codes and
k_scale, v_scale [pages][heads] fp32, powers of two.  page_table [B][slots]
names the page of tokens slot*page .. of each request (-1: none).

Plain forms of the operators, in 32 bits (angles in 64), stand beside the calls
of the library; `own` chooses.  `exact` computes them again in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0          # largest e4m3 value
EXP_LO, EXP_HI = -48, 48  # exponents of a page's scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
LARGEST_BYTES = 7.5e8     # no drawn case reads and writes more than this


# ------------------------------------------------------------------- cases

def _rotate(name, **kw):
    return dict(dict(op="rotate", B=64, T=1, q_heads=32, heads=8, D=128, rot=128, base=1e4,
                     interleaved=False, scaling="none", norm=True, dtype="bf16", tree=False,
                     ragged=False, len=2048), name=name, **kw)


def _append(name, **kw):
    return _rotate(name, **dict(dict(op="append", page=64), **kw))


def _logprobs(name, **kw):
    return dict(dict(op="logprobs", B=64, N=7, R=7, M=1, V=128256, dtype="bf16", top=0,
                     tempered=False, ragged=False, nodes=False, masked=False), name=name, **kw)


def listed():
    return [
        # one token a request: only the call's latency counts
        _rotate("rotate token B=64"),
        # the nodes of a tree, by depth; a quarter of each head turns, pairs side by side
        _rotate("rotate tree B=16 N=32", B=16, T=32, D=64, q_heads=12, heads=12, rot=32,
                interleaved=True, norm=False, dtype="fp16", tree=True, ragged=True, len=8192),
        # a long context far out, frequencies stretched for it
        _rotate("rotate prompt B=2 T=8190", B=2, T=8190, base=5e5, scaling="yarn", len=115000),
        # plain decoding into the cache
        _append("append token B=64"),
        # a chain round of the headline batch (K = 6 drafts), drafts of unequal length
        _append("append chain B=64 T=7", T=7, rot=64, interleaved=True, norm=False, dtype="fp16",
                ragged=True, page=16),
        # the tree round: 32 nodes a request
        _append("append tree B=16 N=32", B=16, T=32, base=5e5, scaling="wavelength", tree=True,
                len=8192),
        # prompts entering the cache, with a last page that is not full
        _append("append prompt B=4 T=8190", B=4, T=8190, len=33),
        # one greedy step of one request
        _logprobs("logprobs token B=1", B=1, N=1, R=1, V=32000),
        # what the headline chain round emitted, with the five likeliest tokens a row
        _logprobs("logprobs chain B=64 R=7", top=5, ragged=True),
        # the accepted paths of tree rounds under a grammar's mask, an odd vocabulary
        _logprobs("logprobs path B=16 R=6", B=16, N=32, R=6, V=32003, dtype="fp32", top=20,
                  tempered=True, ragged=True, nodes=True, masked=True),
        # one step of a large batch, twenty alternatives, with temperatures
        _logprobs("logprobs batch B=256", B=256, N=1, R=1, V=152064, top=20, tempered=True),
        # a prompt scored token by token
        _logprobs("logprobs prompt R=2047", B=1, N=2047, R=2047),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotation(rng, append):
    kind = rng.choice(["token", "chain", "chain", "tree", "tree", "prompt"])
    T = {"token": 1, "chain": rng.randint(2, 33), "tree": rng.randint(2, 64),
         "prompt": _log(rng, 65, 8190)}[kind]
    D = rng.choice([64, 128, 128] if append else [64, 80, 96, 128, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8, 8, 12])
    case = dict(B=_log(rng, 1, 8 if kind == "prompt" else 256), T=T, D=D, heads=heads,
                q_heads=heads * rng.choice([1, 2, 4, 4, 5, 8]),
                rot=min(D, 16 * rng.choice([1, 2, 4, D // 16, D // 16, D // 16])),
                base=rng.choice([1e4, 5e5, 1e6]), interleaved=rng.random() < 0.4,
                scaling=rng.choice(["none", "none", "linear", "yarn", "wavelength"]),
                norm=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                tree=kind == "tree", ragged=rng.random() < 0.5,
                len=_log(rng, 1, 4096) if append else _log(rng, 1, 131071))
    if append:
        case["page"] = rng.choice([16, 32, 64, 64, 128])
    return case


def _draw_logprobs(rng):
    nodes = rng.random() < 0.3
    R = rng.randint(1, 9) if nodes or rng.random() < 0.6 else _log(rng, 1, 2047)
    V = rng.choice([32000, 128256, 152064, _log(rng, 1, 152064), _log(rng, 4096, 200000)])
    return dict(B=_log(rng, 1, 256 if R < 10 else 8), N=rng.randint(R, 32) if nodes else R, R=R,
                M=rng.choice([0, 1, 1, 1, rng.randint(2, 16)]), V=V,
                dtype=rng.choice(["bf16", "bf16", "fp32"]),
                top=rng.choice([0, 0, 1, 5, 20, rng.randint(1, 64)]),
                tempered=rng.random() < 0.5, ragged=rng.random() < 0.5, nodes=nodes,
                masked=rng.random() < 0.25)


def draw(rng):
    while True:
        op = rng.choice(["rotate", "append", "logprobs"])
        case = dict(op=op)
        case.update(_draw_logprobs(rng) if op == "logprobs" else
                    _draw_rotation(rng, op == "append"))
        size = work(case)["bytes"]
        if op == "logprobs":  # the rows that no token is asked of are there too
            size = max(size, case["B"] * case["N"] * case["V"] * BYTES[case["dtype"]])
        if size <= LARGEST_BYTES:
            return case


def _counts(case):
    """Tokens before the round and tokens of it, of every request: fixed by the case, ragged."""
    r = random.Random(1000003 * case["B"] + 31 * case.get("len", case.get("V")) + case.get("T", 0))
    B = case["B"]
    T = case["R"] if case["op"] == "logprobs" else case["T"]
    L = case.get("len", 1)
    length = [L if B == 1 else r.randint((L + 1) // 2, L) for _ in range(B)]
    new = [r.randint(0, T) if case["ragged"] else T for _ in range(B)]
    if T not in new:
        new[r.randrange(B)] = T
    return length, new


def work(case):
    length, new = _counts(case)
    e = BYTES[case["dtype"]]
    if case["op"] == "logprobs":
        rows, all_rows = sum(new), case["B"] * case["R"]
        return {"bytes": rows * case["V"] * e + all_rows * (8 * case["M"] + 4 + 8 * case["top"]),
                "flops": 4 * rows * case["V"]}
    D, H, Hq, T = case["D"], case["heads"], case["q_heads"], case["T"]
    n, rest = sum(new), case["B"] * case["T"] - sum(new)
    flops = (4 * case["norm"] * D + 3 * case["rot"]) * n * (H + Hq)
    if case["op"] == "rotate":
        return {"bytes": (2 * n + rest) * (H + Hq) * D * e, "flops": flops}
    pages = sum((l + m - 1) // case["page"] - l // case["page"] + 1
                for l, m in zip(length, new) if m > 0)
    return {"bytes": (2 * n + rest) * Hq * D * e + n * 2 * H * D * (e + 1) + 8 * pages * H,
            "flops": flops + 4 * n * H * D}


# ------------------------------------------------------------------ inputs

def _inverse_frequencies(case):
    """Radians a position of each channel pair, as a model's configuration gives them, and the
    factor of the rotated channels: plain, every frequency divided by 8 ("linear"), the low ones
    by 8 and the others kept with a ramp over the pair's index between ("yarn") or over the
    wavelength ("wavelength")."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = case["base"] ** (-2.0 * i / case["rot"])
    factor, context, scale = 8.0, 8192.0, 1.0
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "yarn":
        # the pair that turns n times over the trained context
        at = lambda n: (case["rot"] * math.log(context / (n * 2 * math.pi)) /  # noqa: E731
                        (2 * math.log(case["base"])))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), case["rot"] - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif case["scaling"] == "wavelength":
        keep = ((context * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, scale


def _rope(case):
    """The plan that a program keeps: frequencies in 2^-64 turns."""
    f, scale = _inverse_frequencies(case)
    turns = [round(x / (2 * math.pi) * 2.0 ** 64) for x in f.tolist()]
    return dict(freq=torch.tensor(turns, dtype=torch.int64).cuda(), dim=case["rot"],
                interleaved=case["interleaved"], scale=scale)


def _codes_of(x):
    """Codes of x [pages][heads][page][D] with a power-of-two scale a page and head."""
    e = _exponent(x.abs().amax((2, 3)))
    s = torch.exp2(e)
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _cache_side(gen, pages, H, P, D):
    codes = torch.empty((pages, H, P, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, H), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (H * P * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn((n, H, P, D), generator=gen, device="cuda")
        codes[at:at + n], scale[at:at + n] = _codes_of(x)
    return codes, scale


def _depths(rng, B, T, new):
    """Depths of random trees in depth-first order (depth <= 5); -1 where no node is."""
    depth = np.full((B, T), -1, np.int32)
    for b in range(B):
        d = 0
        for i in range(new[b]):
            d = 0 if i == 0 else rng.randint(1, min(d + 1, 5))
            depth[b, i] = d
    return torch.from_numpy(depth).cuda()


def _prepare_rotation(case, gen, rng):
    length, new = _counts(case)
    B, T, H, Hq, D = (case[x] for x in ("B", "T", "heads", "q_heads", "D"))
    dtype = DTYPES[case["dtype"]]
    s = dict(op=case["op"], T=T, rope=_rope(case), eps=1e-6 if case["norm"] else None,
             start=torch.tensor(length, dtype=torch.int32).cuda(),
             num=torch.tensor(new, dtype=torch.int32).cuda(),
             offset=_depths(rng, B, T, new) if case["tree"] else None)
    # a round's projections lie side by side in one buffer: [tokens][Q heads, K heads, V heads];
    # each channel has its own size, and each token
    x = torch.randn((B, T, Hq + 2 * H, D), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, 1, Hq + 2 * H, D), generator=gen, device="cuda"))
    x *= torch.exp(0.3 * torch.randn((B, T, 1, 1), generator=gen, device="cuda"))
    x = x.to(dtype)
    s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]
    for w in ("q_weight", "k_weight"):
        one = torch.exp(0.3 * torch.randn(D, generator=gen, device="cuda")).to(dtype)
        s[w] = one if case["norm"] else None
    if case["op"] == "append":
        P = case["page"]
        slots = [(l + T + P - 1) // P for l in length]
        pages = sum(slots) + 1
        order = list(range(pages))
        rng.shuffle(order)
        table, at = np.full((B, max(slots)), -1, np.int32), 0
        for b in range(B):
            table[b, :slots[b]] = order[at:at + slots[b]]
            at += slots[b]
        k, ks = _cache_side(gen, pages, H, P, D)
        v, vs = _cache_side(gen, pages, H, P, D)
        s.update(cache=dict(k=k, v=v, k_scale=ks, v_scale=vs),
                 page_table=torch.from_numpy(table).cuda())
    return s


def _prepare_logprobs(case, gen, rng):
    _, new = _counts(case)
    B, N, R, M, V = (case[x] for x in ("B", "N", "R", "M", "V"))
    dtype = DTYPES[case["dtype"]]
    logits = torch.empty((B, N, V), dtype=dtype, device="cuda")
    flat = logits.view(B * N, V)
    zipf = 1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
    step = max(1, (1 << 28) // V)
    for at in range(0, B * N, step):  # normal, likelier tokens first, a few peaks a row
        n = min(step, B * N - at)
        x = 3.0 * torch.randn((n, V), generator=gen, device="cuda") - zipf
        peaks = torch.randint(0, V, (n, 3), generator=gen, device="cuda")
        x.scatter_add_(1, peaks, torch.full((n, 3), 8.0, device="cuda"))
        if case["masked"]:  # what a grammar rules out: nine tokens of ten
            x.masked_fill_(torch.rand((n, V), generator=gen, device="cuda") < 0.9, -math.inf)
            x[:, V // 2] = 0.0  # (something is always allowed)
        flat[at:at + n] = x.to(dtype)
    num = torch.tensor(new, dtype=torch.int32)
    live = torch.arange(R) < num[:, None]
    tokens = None
    if M:  # likelier tokens more often; -1 behind the last row
        u = torch.rand((B, R, M), generator=gen, device="cuda")
        tokens = (torch.exp(u * math.log(V)) - 1).to(torch.int32).clamp(0, V - 1)
        tokens = torch.where(live.cuda()[:, :, None], tokens, -1)
        tokens = tokens[:, :, 0].contiguous() if M == 1 else tokens
    rows = None
    if case["nodes"]:
        rows = np.full((B, R), -1, np.int32)
        for b in range(B):
            if new[b]:
                rows[b, :new[b]] = [0] + sorted(rng.sample(range(1, N), new[b] - 1))
        rows = torch.from_numpy(rows).cuda()
    t = None
    if case["tempered"]:
        t = 0.3 + torch.rand(B, generator=gen, device="cuda")
        t[::4] = 0.0  # greedy requests
    return dict(op="logprobs", logits=logits, tokens=tokens, rows=rows, num_rows=num.cuda(), R=R,
                temperature=t, top=case["top"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    make = _prepare_logprobs if case["op"] == "logprobs" else _prepare_rotation
    return make(case, gen, rng)


# --------------------------------------------------------------- the calls

def run(state):
    if own:
        return _run_library(state)
    return {"rotate": _plain_rotate, "append": _plain_append, "logprobs": _plain_logprobs}[
        state["op"]](state)


def _run_library(s):
    import speculative_decoding_verification_63_gb300 as sv
    if s["op"] == "logprobs":
        return sv.token_logprobs(s["logits"], s["tokens"], num_rows=s["num_rows"], rows=s["rows"],
                                 R=s["R"], temperature=s["temperature"], top=s["top"])
    how = dict(rope=s["rope"], offset=s["offset"], q_weight=s["q_weight"],
               k_weight=s["k_weight"], eps=s["eps"])
    if s["op"] == "rotate":
        return sv.rotate(s["q"], s["k"], start=s["start"], num=s["num"], **how)
    out = sv.kv_append(s["cache"], s["page_table"], s["start"], s["q"], s["k"], s["v"],
                       num_new=s["num"], **how)
    return dict(out, **s["cache"])


# ------------------------------------------------------------- plain forms

def _live(s):
    return torch.arange(s["T"], device="cuda") < s["num"][:, None]


def _rotated(s, x, weight):
    """x [B][T][heads][D] with its heads' norms and the rotation of its positions, in 32 bits."""
    x = x.float()
    if s["eps"] is not None:
        x = x * torch.rsqrt((x * x).mean(3, keepdim=True) + s["eps"]) * weight.float()
    t = torch.arange(s["T"], device="cuda") if s["offset"] is None else s["offset"].double()
    turns = (s["start"].double()[:, None] + t)[:, :, None] * (s["rope"]["freq"].double() * 2.0 ** -64)
    angle = 2 * math.pi * (turns - torch.floor(turns))
    cos = (torch.cos(angle) * s["rope"]["scale"]).float()[:, :, None]
    sin = (torch.sin(angle) * s["rope"]["scale"]).float()[:, :, None]
    dim = s["rope"]["dim"]
    if s["rope"]["interleaved"]:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 4).flatten(3)
    else:
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 3)
    return torch.cat([turned, x[..., dim:]], 3)


def _plain_rotate(s):
    live = _live(s)[:, :, None, None]
    return {x: torch.where(live, _rotated(s, s[x], s[x + "_weight"]), 0.0).to(s[x].dtype)
            for x in "qk"}


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the scale's range."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)  # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, EXP_LO).clamp(EXP_LO, EXP_HI).float()


def _codes(x, s):
    return (x / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append(s):
    q = torch.where(_live(s)[:, :, None, None], _rotated(s, s["q"], s["q_weight"]), 0.0)
    _append_side(s, "k", _rotated(s, s["k"], s["k_weight"]))
    _append_side(s, "v", s["v"].float())
    return dict(s["cache"], q=q.to(s["q"].dtype))


def _append_side(s, side, new):
    """new [B][T][heads][D] into the codes and scales of one side of the cache."""
    codes, scale = s["cache"][side], s["cache"][side + "_scale"]
    start, num, table = s["start"].long(), s["num"].long(), s["page_table"].long()
    H, P = codes.shape[1:3]
    B, T = new.shape[:2]
    raw = codes.view(torch.uint8)
    live = _live(s)
    pos = start[:, None] + torch.arange(T, device="cuda")              # [B][T]
    first = start // P
    slot = pos // P - first[:, None]                                   # page of the round
    S = (T + P - 2) // P + 1
    size = torch.where(live[:, :, None], new.abs().amax(3), 0.0)       # [B][T][H]
    amax = torch.zeros((B, S, H), device="cuda").scatter_reduce(
        1, slot[:, :, None].expand(B, T, H), size, "amax")
    which = first[:, None] + torch.arange(S, device="cuda")            # [B][S]
    used = (which <= ((start + num - 1) // P)[:, None]) & (num > 0)[:, None]
    page = table.gather(1, which.clamp(max=table.shape[1] - 1)).clamp(min=0)
    held = start - first * P                                           # tokens that stay
    kept = (held > 0) & (num > 0)
    before = scale[page[:, 0]]
    e = _exponent(amax)
    e[:, 0] = torch.where(kept[:, None], torch.maximum(e[:, 0], torch.frexp(before)[1] - 1.0),
                          e[:, 0])
    now = torch.exp2(e)                                                # [B][S][H]
    # tokens that stay in a page whose scale grows are rounded again
    grows = kept[:, None] & (now[:, 0] > before)
    again = _codes(raw[page[:, 0]].view(codes.dtype).float() * before[:, :, None, None],
                   now[:, 0][:, :, None, None])
    b, h, p = (grows[:, :, None] & (torch.arange(P, device="cuda") < held[:, None, None])
               ).nonzero(as_tuple=True)
    raw[page[b, 0], h, p] = again.view(torch.uint8)[b, h, p]
    b, i = used.nonzero(as_tuple=True)
    scale[page[b, i]] = now[b, i]
    b, i = live.nonzero(as_tuple=True)
    j = slot[b, i]
    raw[page[b, j], :, pos[b, i] % P] = _codes(new[b, i], now[b, j][:, :, None]).view(torch.uint8)


def _plain_logprobs(s):
    logits, R = s["logits"], s["R"]
    B, N, V = logits.shape
    live = torch.arange(R, device="cuda") < s["num_rows"][:, None]
    raw = logits[:, :R] if s["rows"] is None else logits.gather(
        1, s["rows"].long().clamp(min=0)[:, :, None].expand(B, R, V))
    raw = raw.float()
    x = raw
    if s["temperature"] is not None:
        t = torch.where(s["temperature"] > 0, s["temperature"], 1.0)
        x = raw / t[:, None, None]
    m = x.amax(2, keepdim=True)
    d = x - m
    w = torch.exp(d)
    z = w.sum(2, keepdim=True)
    log_z = torch.log(z)
    out = dict(entropy=_rows(live, (log_z - (w * torch.where(w > 0, d, 0.0)).sum(
        2, keepdim=True) / z)[:, :, 0]))
    if s["tokens"] is not None:
        tokens = s["tokens"].view(B, R, -1).long()
        given = d.gather(2, tokens.clamp(min=0)) - log_z
        given = torch.where(tokens >= 0, given, math.nan)
        out["logprobs"] = _rows(live, given).view(s["tokens"].shape)
    if s["top"]:
        # the largest logits, the lower token first among equals: one whole number for both
        bits = (raw + 0.0).view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        key = (order << 20) + (V - 1 - torch.arange(V, device="cuda"))
        n = min(s["top"], V)
        at = (V - 1) - (key.topk(n, 2).values & ((1 << 20) - 1))
        best = d.gather(2, at) - log_z
        there = live[:, :, None] & (best > -math.inf)
        ids = torch.full((B, R, s["top"]), -1, dtype=torch.int32, device="cuda")
        ids[:, :, :n] = torch.where(there, at, -1).to(torch.int32)
        top = torch.full((B, R, s["top"]), -math.inf, device="cuda")
        top[:, :, :n] = best
        out.update(top_tokens=ids, top_logprobs=_rows(live, top))
    return out


def _rows(live, x):
    """x, NaN in rows behind a request's last."""
    return torch.where(live if x.dim() == 2 else live[:, :, None], x, math.nan)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    length, new = _counts(case)
    if case["op"] == "logprobs":
        return _exact_logprobs(s, new)
    out = {x: _exact_rotated(case, s, x, length, new) for x in "qk"}
    if case["op"] == "rotate":
        return out
    keys = out.pop("k")
    for side, x in (("k", keys), ("v", s["v"].double())):
        out[side], out[side + "_scale"] = _exact_side(s, side, x, length, new)
    return out


def _exact_frequencies(case):
    """Radians a position, pair by pair, from the definitions."""
    out, context, factor = [], 8192.0, 8.0
    rot, base = case["rot"], case["base"]
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "yarn":
            lo = max(0, math.floor(rot * math.log(context / (64 * math.pi)) / (2 * math.log(base))))
            hi = min(rot - 1, math.ceil(rot * math.log(context / (2 * math.pi)) /
                                        (2 * math.log(base))))
            part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f * (1 - part) + f / factor * part
        elif case["scaling"] == "wavelength":
            wave = 2 * math.pi / f
            if wave > context:
                f /= factor
            elif wave > context / 4:
                part = (context / wave - 1) / 3
                f = part * f + (1 - part) * f / factor
        out.append(f)
    return out


def _exact_rotated(case, s, name, length, new):
    x = s[name].double()
    B, T, H, D = x.shape
    if case["norm"]:
        x = x / torch.sqrt((x ** 2).sum(3, keepdim=True) / D + 1e-6) * s[name + "_weight"].double()
    f = torch.tensor(_exact_frequencies(case), dtype=torch.float64, device="cuda")
    offset = s["offset"].tolist() if case["tree"] else [list(range(T))] * B
    pos = torch.tensor([[length[b] + o for o in offset[b]] for b in range(B)],
                       dtype=torch.float64, device="cuda")
    angle = pos[:, :, None, None] * f
    size = 0.1 * math.log(8.0) + 1 if case["scaling"] == "yarn" else 1.0
    turn = torch.polar(torch.full_like(angle, size), angle)            # [B][T][1][rot/2]
    rot = case["rot"]
    part = x[..., :rot].unflatten(3, (rot // 2, 2)) if case["interleaved"] else \
        x[..., :rot].unflatten(3, (2, rot // 2)).transpose(3, 4)
    part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
    part = part if case["interleaved"] else part.transpose(3, 4)
    y = torch.cat([part.flatten(3), x[..., rot:]], 3)
    for b in range(B):
        y[b, new[b]:] = 0.0
    return y


def _round_e4m3(x):
    """x (float64, |x| <= 448) to the nearest e4m3 value, ties to even: the grid has steps of
    2^(e - 3) for values in [2^e, 2^(e + 1)), e >= -6."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1
    step = _pow2(e - 3)
    return torch.round(x / step) * step


def _pow2(e):
    """2^e in float64, by its bits: exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(amax):
    """The least power of two that amax / 448 does not exceed."""
    m, e = torch.frexp(amax / E4M3_MAX)          # m in [1/2, 1): a power of two has m = 1/2
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, EXP_LO).clamp(EXP_LO, EXP_HI)
    return _pow2(e)


def _exact_side(s, side, x, length, new):
    table = s["page_table"].cpu().numpy()
    codes, scale = s["cache"][side].float(), s["cache"][side + "_scale"].double()
    P = codes.shape[2]
    for b, (l, n) in enumerate(zip(length, new)):
        for i in range(l // P, (l + n - 1) // P + 1 if n else 0):
            page, kept = int(table[b, i]), max(0, l - i * P)
            at = slice(max(0, i * P - l), min(n, (i + 1) * P - l))
            to = at.start + l - i * P
            size = _exact_scale(x[b, at].abs().amax((0, 2)))
            if kept:
                size = torch.maximum(size, scale[page])
                was = codes[page, :, :kept].double() * scale[page][:, None, None]
                codes[page, :, :kept] = _round_e4m3(was / size[:, None, None]).float()
            scale[page] = size
            y = (x[b, at] / size[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            codes[page, :, to:to + at.stop - at.start] = _round_e4m3(y).permute(1, 0, 2).float()
    return codes, scale


def _exact_logprobs(s, new):
    logits, R, top = s["logits"], s["R"], s["top"]
    B, N, V = logits.shape
    wanted = None if s["tokens"] is None else s["tokens"].view(B, R, -1).tolist()
    nan = lambda *shape: torch.full(shape, math.nan, dtype=torch.float64,  # noqa: E731
                                    device="cuda")
    entropy = nan(B, R)
    given = None if wanted is None else nan(B, R, len(wanted[0][0]))
    ids = torch.full((B, R, top), -1, dtype=torch.int32, device="cuda")
    best = nan(B, R, top)
    t = [1.0] * B if s["temperature"] is None else [x or 1.0 for x in s["temperature"].tolist()]
    step = max(1, (1 << 25) // V)
    for b in range(B):
        for r0 in range(0, new[b], step):
            r1 = min(new[b], r0 + step)
            which = list(range(r0, r1)) if s["rows"] is None else s["rows"][b, r0:r1].tolist()
            raw = logits[b, which].double()
            lp = torch.log_softmax(raw / t[b], 1)
            entropy[b, r0:r1] = -torch.where(lp > -math.inf, torch.exp(lp) * lp, 0.0).sum(1)
            if wanted is not None:
                tokens = torch.tensor(wanted[b][r0:r1], device="cuda")
                given[b, r0:r1] = lp.gather(1, tokens)
            if top:
                n = min(top, V)
                order = raw.sort(dim=1, descending=True, stable=True)
                at = order.indices[:, :n]
                there = order.values[:, :n] > -math.inf
                ids[b, r0:r1, :n] = torch.where(there, at, -1).to(torch.int32)
                best[b, r0:r1] = -math.inf
                best[b, r0:r1, :n] = lp.gather(1, at)
    out = dict(entropy=entropy)
    if wanted is not None:
        out["logprobs"] = given.view(s["tokens"].shape)
    if top:
        out.update(top_tokens=ids, top_logprobs=best)
    return out
