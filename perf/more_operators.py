"""Operators of linear attention with a decay for each head, as cases to measure.

What a recurrent decoder without the delta rule needs from its prompts to its single tokens, and to train:

  attn      linear attention over whole sequences (prompts): outputs for every token and the state after
            the last one, which the step continues from
  attn_bwd  its backward pass
  step      its single-token form over a pool of states, with rotary positions of q and k or without
  rotary    rotary positions of q and k over a batch of tokens, and (inverse) the gradients through them

`run` computes them in plain form from elementary torch operations, or, with `own` set, through the
package's entry points. `exact` gives the 64-bit result of the definition.
"""
import math

import torch

own = False


def _gdn():
    import ssm_recurrent_decode_gb300 as gdn
    return gdn


# ------------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one short prompt before a chat turn's first token: a latency-bound call
        {"name": "attn_prompt", "op": "attn", "dtype": "bf16", "lengths": "1x100", "H": 16, "HV": 32, "K": 128, "V": 128,
         "fixed": False, "resume": False},
        # a serving step's ragged prompts packed end to end (lengths from 0 and 1 token to a long document),
        # continuing from states in a slot pool, each token with its own decay
        {"name": "attn_ragged", "op": "attn", "dtype": "bf16", "lengths": "ragged24x8000", "H": 16, "HV": 32, "K": 128,
         "V": 128, "fixed": False, "resume": True},
        # one long document, one fixed decay a head: few rows, a long axis
        {"name": "attn_long", "op": "attn", "dtype": "bf16", "lengths": "1x32768", "H": 32, "HV": 32, "K": 128, "V": 128,
         "fixed": True, "resume": False},
        # an evaluation in full precision, odd value size
        {"name": "attn_fp32", "op": "attn", "dtype": "f32", "lengths": "3x777", "H": 12, "HV": 12, "K": 64, "V": 50,
         "fixed": False, "resume": True},
        # gradients of one short fp32 sequence: fine-tuning at batch one
        {"name": "attn_bwd_small", "op": "attn_bwd", "dtype": "f32", "lengths": "1x500", "H": 12, "HV": 12, "K": 64, "V": 64,
         "fixed": True, "resume": False},
        # gradients of a training batch
        {"name": "attn_bwd_batch", "op": "attn_bwd", "dtype": "bf16", "lengths": "8x2048", "H": 32, "HV": 32, "K": 128,
         "V": 128, "fixed": False, "resume": False},
        # gradients through packed documents with carried states, value heads that share q and k
        {"name": "attn_bwd_ragged", "op": "attn_bwd", "dtype": "bf16", "lengths": "ragged10x5000", "H": 8, "HV": 16,
         "K": 64, "V": 128, "fixed": False, "resume": True},
        # one request's token: latency-bound; half of each head turned by its position
        {"name": "step_one", "op": "step", "dtype": "bf16", "state": "f32", "B": 1, "H": 16, "HV": 32, "K": 128, "V": 128,
         "fixed": True, "turned": 64},
        # a serving batch over a pool of fp32 states
        {"name": "step_batch", "op": "step", "dtype": "bf16", "state": "f32", "B": 256, "H": 16, "HV": 32, "K": 128,
         "V": 128, "fixed": False, "turned": 128},
        # states stored in bf16, odd value size, no positions
        {"name": "step_bf16_state", "op": "step", "dtype": "bf16", "state": "bf16", "B": 40, "H": 24, "HV": 24, "K": 64,
         "V": 100, "fixed": False, "turned": 0},
        # a prompt batch's q and k at positions of a long context (frequencies scaled for it), in halves
        {"name": "rotary_prompts", "op": "rotary", "dtype": "bf16", "T": 16384, "H": 32, "HK": 16, "D": 128, "turned": 128,
         "interleaved": False, "inverse": False, "far": 1000000, "factor": 16.0},
        # the gradients of fp32 q and k through it, neighbouring pairs, a quarter of each head turned
        {"name": "rotary_gradients", "op": "rotary", "dtype": "f32", "T": 4999, "H": 12, "HK": 12, "D": 96, "turned": 24,
         "interleaved": True, "inverse": True, "far": 8192, "factor": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn_bwd", "attn_bwd", "attn_bwd", "step", "step", "rotary"])
    if op in ("attn", "attn_bwd"):
        K = rng.choice([16, 32, 64, 128, 128])
        V = rng.choice([64, 128, 128, rng.randint(1, 128)])
        H = rng.randint(1, 24)
        HV = H * rng.choice([1, 1, 2, 3])
        most = (32768 * 32 if op == "attn" else 8 * 2048 * 32) // HV
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        T = _log_int(rng, 32, max(64, min(32768, most if dtype == "bf16" else most // 4)))
        if rng.random() < 0.5:
            S = min(T, _log_int(rng, 1, 16))
            lengths = f"{S}x{T // S}"
        else:
            lengths = f"ragged{_log_int(rng, 2, 40)}x{T}"
        return {"op": op, "dtype": dtype, "lengths": lengths, "H": H, "HV": HV, "K": K, "V": V,
                "fixed": rng.random() < 0.4, "resume": rng.random() < 0.5}
    if op == "step":
        K = rng.choice([16, 32, 64, 128, 128])
        V = rng.choice([64, 128, 128, rng.randint(1, 300)])
        H = rng.randint(1, 32)
        HV = H * rng.choice([1, 2, 4])
        B = _log_int(rng, 1, max(2, min(512, 256 * 32 * 128 * 128 // (HV * K * V))))
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "state": rng.choice(["f32", "f32", "bf16"]), "B": B,
                "H": H, "HV": HV, "K": K, "V": V, "fixed": rng.random() < 0.4,
                "turned": rng.choice([0, K, K // 2, 2 * rng.randint(1, K // 2)])}
    D = 2 * rng.randint(8, 128)
    H, HK = rng.randint(1, 40), rng.randint(1, 16)
    T = _log_int(rng, 1, max(2, min(65536, 16384 * 48 * 128 // (D * (H + HK)))))
    dtype = rng.choice(["bf16", "f32"])
    return {"op": op, "dtype": dtype, "T": T if dtype == "bf16" else -(-T // 2), "H": H, "HK": HK, "D": D,
            "turned": rng.choice([D, 2 * rng.randint(1, D // 2)]), "interleaved": rng.random() < 0.5,
            "inverse": rng.random() < 0.4, "far": _log_int(rng, 100, 2000000), "factor": rng.choice([1.0, 4.0, 40.0])}


def _lengths(spec, seed):
    """Sequence lengths of "SxL" (S sequences of L tokens) or "raggedSxT" (S sequences, T tokens in all)."""
    if not spec.startswith("ragged"):
        s, l = spec.split("x")
        return [int(l)] * int(s)
    s, t = (int(v) for v in spec[6:].split("x"))
    g = torch.Generator().manual_seed(seed * 7 + 3)
    w = torch.exp(torch.rand(s, generator=g) * 5.0)      # lengths over a factor of 150
    n = (w / w.sum() * t).long()
    n[0], n[s // 2] = 0, 1                               # an empty and a one-token sequence
    n[s - 1] += t - int(n.sum())
    return [int(v) for v in n]


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64                                              # tokens the plain form takes together


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"attn": _prepare_attn, "attn_bwd": _prepare_attn, "step": _prepare_step, "rotary": _prepare_rotary}
    return {"case": dict(case), **make[case["op"]](case, seed, g)}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _decays(g, T, HV, fixed):
    """Log decays: from heads that remember a thousand tokens to heads that remember one; a token's own is
    its head's times what a gate makes of it."""
    base = -torch.exp(torch.rand(HV, generator=g, device="cuda") * math.log(1000.0) - math.log(1000.0))
    if fixed:
        return base
    return base * torch.exp(0.5 * _normal(g, T, HV))


def _prepare_attn(case, seed, g):
    H, HV, K, V, t = case["H"], case["HV"], case["K"], case["V"], _TYPES[case["dtype"]]
    lengths = _lengths(case["lengths"], seed)
    T, S = sum(lengths), len(lengths)
    # q, k and v are parts of one projection's rows (row views)
    qkv = _normal(g, T, 2 * H * K + HV * V).to(t)
    dev = lambda v, d=torch.int64: torch.tensor(v, dtype=d, device="cuda")
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    # the plain form's chunks: rows of tokens (T where there is none), whether a sequence begins or ends there
    rows, first, last, seq = [], [], [], []
    for s, n in enumerate(lengths):
        for at in range(0, n, _CHUNK):
            m = min(_CHUNK, n - at)
            rows.append((cu[s] + at, m))
            first.append(at == 0), last.append(at + m == n), seq.append(s)
    start, count = dev([r[0] for r in rows]), dev([r[1] for r in rows])
    col = torch.arange(_CHUNK, device="cuda")
    rows = torch.where(col < count[:, None], start[:, None] + col, T)
    slots = torch.randperm(S + 3, generator=torch.Generator().manual_seed(seed))[:S].to(torch.int32).cuda()
    st = {"q": qkv[:, :H * K].unflatten(1, (H, K)), "k": qkv[:, H * K:2 * H * K].unflatten(1, (H, K)),
          "v": qkv[:, 2 * H * K:].unflatten(1, (HV, V)), "g": _decays(g, T, HV, case["fixed"]), "S": S,
          "uniform": not case["lengths"].startswith("ragged"), "lengths": lengths, "cu": dev(cu, torch.int32),
          "rows": rows, "first": dev(first, torch.bool), "last": dev(last, torch.bool), "seq": dev(seq), "slots": slots,
          "initial": _normal(g, S + 3, HV, V, K) if case["resume"] else None}
    if case["op"] == "attn":
        st["o"] = torch.empty(T, HV, V, dtype=t, device="cuda")
        st["final"] = torch.zeros(S + 3, HV, V, K, device="cuda")
        return st
    st["do"] = _normal(g, T, HV, V).to(t)
    st["d_final"] = 0.1 * _normal(g, S + 3, HV, V, K) if case["resume"] else None
    st["grads"] = {"dq": torch.empty(T, H, K, dtype=t, device="cuda"), "dk": torch.empty(T, H, K, dtype=t, device="cuda"),
                   "dv": torch.empty(T, HV, V, dtype=t, device="cuda"), "dg": torch.empty_like(st["g"]),
                   "d_initial_state": torch.zeros(S + 3, HV, V, K, device="cuda") if case["resume"] else None}
    return st


def _frequencies(turned, factor):
    """Radians a position of each pair; scaled for a context `factor` times the trained one of 4096 positions: what
    turns more than 32 times there keeps its frequency, what turns less than once is divided, linearly between."""
    f = 10000.0 ** (-torch.arange(0, turned, 2, dtype=torch.float64) / turned)
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * (keep + (1.0 - keep) / factor)).cuda()


def _prepare_step(case, seed, g):
    B, H, HV, K, V, t = case["B"], case["H"], case["HV"], case["K"], case["V"], _TYPES[case["dtype"]]
    qkv = _normal(g, B, 2 * H * K + HV * V).to(t)
    slots = torch.randperm(B + 5, generator=torch.Generator().manual_seed(seed))[:B].to(torch.int32).cuda()
    st = {"q": qkv[:, :H * K].unflatten(1, (H, K)), "k": qkv[:, H * K:2 * H * K].unflatten(1, (H, K)),
          "v": qkv[:, 2 * H * K:].unflatten(1, (HV, V)), "g": _decays(g, B, HV, case["fixed"]), "slots": slots,
          "state": _normal(g, B + 5, HV, V, K).to(_TYPES[case["state"]]),
          "out": torch.empty(B, HV, V, dtype=t, device="cuda"), "positions": None, "frequencies": None}
    if case["turned"]:
        st["positions"] = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda", dtype=torch.int32)
        st["frequencies"] = _frequencies(case["turned"], 1.0)
    return st


def _prepare_rotary(case, seed, g):
    T, H, HK, D, t = case["T"], case["H"], case["HK"], case["D"], _TYPES[case["dtype"]]
    qk = _normal(g, T, (H + HK) * D).to(t)
    # packed prompts: runs of positions, the last far into a long context
    at = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda", dtype=torch.int32)
    positions = torch.arange(T, device="cuda", dtype=torch.int32) % (T // 3 + 1)
    positions[T // 2:] += at
    return {"q": qk[:, :H * D].unflatten(1, (H, D)), "k": qk[:, H * D:].unflatten(1, (HK, D)), "positions": positions,
            "frequencies": _frequencies(case["turned"], case["factor"]),
            "magnitude": 0.1 * math.log(case["factor"]) + 1.0,
            "q_out": torch.empty(T, H, D, dtype=t, device="cuda"), "k_out": torch.empty(T, HK, D, dtype=t, device="cuda")}


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _workspace(s, backward):
    _, H, K = s["q"].shape
    T, HV, V = s["v"].shape
    return _gdn().linear_attention_workspace(T, H, HV, K, V, sequences=s["S"], uniform=s["uniform"], backward=backward,
                                             dtype=s["q"].dtype)


def _sequences(s):
    return {"sequences": s["S"] if s["uniform"] else None, "cu_seqlens": None if s["uniform"] else s["cu"],
            "state_indices": s["slots"], "initial_state": s["initial"], "workspace": s["workspace"], "prepare": True}


def _own_attn(s):
    if "call" not in s:                                    # a user's program keeps its workspace and prepared call
        s["workspace"] = _workspace(s, False)
        s["call"] = _gdn().gdn_linear_attention(s["q"], s["k"], s["v"], s["g"], s["o"], final_state=s["final"],
                                                **_sequences(s))
    s["call"]()
    return {"o": s["o"], "final": s["final"]}


def _own_attn_bwd(s):
    if "call" not in s:
        s["workspace"] = _workspace(s, True)
        s["call"] = _gdn().gdn_linear_attention_backward(s["q"], s["k"], s["v"], s["g"], s["do"],
                                                         d_final_state=s["d_final"], **s["grads"], **_sequences(s))
    s["call"]()
    return {k: v for k, v in s["grads"].items() if v is not None}


def _own_step(s):
    if "call" not in s:
        s["call"] = _gdn().gdn_linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["out"], s["slots"],
                                                     positions=s["positions"], frequencies=s["frequencies"], prepare=True)
    s["call"]()
    return {"out": s["out"], "state": s["state"]}


def _own_rotary(s):
    if "call" not in s:
        c = s["case"]
        s["call"] = _gdn().gdn_rotary(s["q"], s["k"], s["positions"], s["frequencies"], q_out=s["q_out"], k_out=s["k_out"],
                                      interleaved=c["interleaved"], inverse=c["inverse"], magnitude=s["magnitude"],
                                      prepare=True)
    s["call"]()
    return {"q": s["q_out"], "k": s["k_out"]}


# ---- plain forms -------------------------------------------------------------------------------
def _carried(a, b):
    """h_c = a_c h_{c-1} + b_c along the first axis (h_{-1} = 0), by doubling the span that each entry covers."""
    a, span, n = a[..., None, None], 1, b.shape[0]
    while span < n:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _chunked(s, *names):
    """Tensors [T, heads, dim] as fp32 chunks [chunks, HV, tokens, dim], zeros behind a sequence's end."""
    HV, out = s["v"].shape[1], []
    for n in names:
        x = torch.nn.functional.pad(s[n].float(), (0, 0, 0, 0, 0, 1))[s["rows"]].transpose(1, 2)
        out.append(x.repeat_interleave(HV // x.shape[1], 1))
    return out


def _flat(s, x):
    """Chunks [chunks, heads, tokens, ...] back to token rows."""
    x = x.transpose(1, 2).flatten(0, 1)
    return x[(s["rows"] < s["v"].shape[0]).flatten()]


def _chunk_states(s):
    T, HV = s["v"].shape[:2]
    q, k, v = _chunked(s, "q", "k", "v")
    g = s["g"].expand(T, HV)
    # sums of many log decays, whose differences are taken: in 64 bits
    G = torch.nn.functional.pad(g.double(), (0, 0, 0, 1))[s["rows"]].transpose(1, 2).cumsum(2)
    low = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device="cuda").tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    toend = torch.exp(G[..., -1:] - G).float()[..., None]
    fromstart = torch.exp(G).float()[..., None]
    decay = fromstart[..., -1, 0]
    local = v.transpose(2, 3) @ (k * toend)
    start = torch.zeros_like(local[:1]) if s["initial"] is None else s["initial"][s["slots"][s["seq"]].long()]
    begin = s["first"][:, None, None, None]
    local = local + torch.where(begin, decay[..., None, None] * start, 0.0)
    after = _carried(torch.where(s["first"][:, None], 0.0, decay), local)
    before = torch.where(begin, start, torch.cat([torch.zeros_like(after[:1]), after[:-1]]))
    return q, k, v, D, toend, fromstart, decay, before, after


def _scale(s):
    return s["q"].shape[2] ** -0.5


def _plain_attn(s):
    T, HV, V = s["v"].shape
    final = torch.zeros_like(s["final"])
    slots = s["slots"].long()
    if s["initial"] is not None:
        final[slots] = s["initial"][slots]                 # an empty sequence keeps its state
    q, k, v, D, _, fromstart, _, before, after = _chunk_states(s)
    o = ((q @ k.transpose(2, 3)) * D) @ v + fromstart * (q @ before.transpose(2, 3))
    final[slots[s["seq"][s["last"]]]] = after[s["last"]]
    return {"o": _flat(s, o * _scale(s)).to(s["q"].dtype), "final": final}


def _plain_attn_bwd(s):
    T, HV, V = s["v"].shape
    t, H, slots, scale = s["q"].dtype, s["q"].shape[1], s["slots"].long(), _scale(s)
    q, k, v, D, toend, fromstart, decay, before, after = _chunk_states(s)
    do, = _chunked(s, "do")
    do = do * scale
    # e: the gradient of the state behind each chunk, carried backwards over the chunks
    end = s["last"][:, None, None, None]
    given = torch.zeros_like(after[:1]) if s["d_final"] is None else s["d_final"][slots[s["seq"]]]
    local = do.transpose(2, 3) @ (q * fromstart)
    own_end = torch.where(end, given, 0.0)
    nxt = torch.cat([decay[1:], torch.zeros_like(decay[:1])])
    nxt = torch.where(s["last"][:, None], 0.0, nxt)
    pushed = torch.where(end, 0.0, torch.cat([local[1:], torch.zeros_like(local[:1])]))
    e = _carried(nxt.flip(0), (pushed + own_end).flip(0)).flip(0)
    P, dP = (q @ k.transpose(2, 3)) * D, (do @ v.transpose(2, 3)) * D
    dq = dP @ k + fromstart * (do @ before)
    dk = dP.transpose(2, 3) @ q + toend * (v @ e)
    dv = P.transpose(2, 3) @ do + toend * (k @ e.transpose(2, 3))
    # differences of long sums: in 64 bits, and no longer than a chunk
    dG = (q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)
    dg = dG.flip(2).cumsum(2).flip(2) + (e.double() * after).sum((-2, -1))[..., None]
    dg = _flat(s, dg)
    heads = lambda x: _flat(s, x).unflatten(1, (H, HV // H)).sum(2).to(t)
    out = {"dq": heads(dq), "dk": heads(dk), "dv": _flat(s, dv).to(t),
           "dg": (dg.sum(0) if s["g"].dim() == 1 else dg).float()}
    if s["initial"] is not None:
        d0 = torch.zeros_like(s["initial"])
        if s["d_final"] is not None:
            d0[slots] = s["d_final"][slots]
        d0[slots[s["seq"][s["first"]]]] = (local + decay[..., None, None] * e)[s["first"]]
        out["d_initial_state"] = d0
    return out


def _turn(x, positions, frequencies, magnitude, interleaved, inverse):
    """x [T, heads, D] in fp32 with its first channels turned, pair by pair, by their position's angles."""
    angle = positions.double()[:, None, None] * frequencies          # far positions: the angle in 64 bits
    c, s = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * magnitude).float()
    if inverse:
        s = -s
    n = frequencies.numel()
    x, turned, rest = x.float(), x[..., :2 * n].float(), x[..., 2 * n:].float()
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :n], turned[..., n:])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _plain_rotary(s):
    c = s["case"]
    turn = lambda x: _turn(x, s["positions"], s["frequencies"], s["magnitude"], c["interleaved"], c["inverse"]).to(x.dtype)
    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_step(s):
    B, HV, V = s["v"].shape
    q, k, v, slots = s["q"].float(), s["k"].float(), s["v"].float(), s["slots"].long()
    if s["frequencies"] is not None:
        q, k = (_turn(x, s["positions"], s["frequencies"], 1.0, False, False) for x in (q, k))
    q, k = (x.repeat_interleave(HV // x.shape[1], 1) for x in (q, k))
    decay = torch.exp(s["g"].expand(B, HV))[..., None, None]
    S = s["state"][slots].float() * decay + v[..., :, None] * k[..., None, :]
    out = (S * q[..., None, :]).sum(-1) * _scale(s)
    s["state"][slots] = S.to(s["state"].dtype)
    return {"out": out.to(s["q"].dtype), "state": s["state"]}


_OWN = {"attn": _own_attn, "attn_bwd": _own_attn_bwd, "step": _own_step, "rotary": _own_rotary}
_PLAIN = {"attn": _plain_attn, "attn_bwd": _plain_attn_bwd, "step": _plain_step, "rotary": _plain_rotary}


# ------------------------------------------------------------------------------------------------
# what one pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "rotary":
        T, heads, D = case["T"], case["H"] + case["HK"], case["D"]
        return {"bytes": 2 * T * heads * D * e + 4 * T + 4 * case["turned"], "flops": 3 * T * heads * case["turned"]}
    H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
    if op == "step":
        B, se = case["B"], 2 if case["state"] == "bf16" else 4
        # per state entry: decay, multiply-add into the state, multiply-add into the output
        return {"bytes": 2 * B * HV * K * V * se + B * (2 * H * K + 2 * HV * V) * e + 4 * HV * (1 if case["fixed"] else B) + 4 * B,
                "flops": 5 * B * HV * K * V}
    spec = case["lengths"]
    if spec.startswith("ragged"):
        S, T = (int(v) for v in spec[6:].split("x"))
    else:
        S, L = (int(v) for v in spec.split("x"))
        T = S * L
    g, states, resume = 4 * HV * (1 if case["fixed"] else T), 4 * S * HV * K * V, int(case["resume"])
    if op == "attn":
        # q, k, v in, o out; the states. Per state entry: multiply-add into the state and into the output
        return {"bytes": 2 * T * (H * K + HV * V) * e + g + states * (1 + resume), "flops": 4 * T * HV * K * V}
    # q, k, v, do in, dq, dk, dv out. Per state entry: the states, their gradients, dq, dk, dv
    return {"bytes": T * (4 * H * K + 3 * HV * V) * e + 2 * g + 3 * states * resume, "flops": 10 * T * HV * K * V}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "attn_bwd": _exact_attn, "step": _exact_step, "rotary": _exact_rotary}[case["op"]](s)


def _exact_attn(s):
    """Token by token, all sequences side by side (position p of each that is long enough)."""
    T, HV, V = s["v"].shape
    H, K = s["q"].shape[1:]
    G, scale = HV // H, K ** -0.5
    lengths, slots = s["lengths"], s["slots"].long()
    q, k, v = s["q"].double() * scale, s["k"].double(), s["v"].double()
    a = torch.exp(s["g"].double().expand(T, HV))
    order = sorted(range(s["S"]), key=lambda i: -lengths[i])           # long ones first: the live ones are a prefix
    starts = torch.tensor([sum(lengths[:i]) for i in order], device="cuda")
    where = slots[torch.tensor(order, device="cuda")]
    longest = max(lengths)
    counts = [sum(1 for i in order if lengths[i] > p) for p in range(longest)]
    S = torch.zeros(s["S"], HV, V, K, dtype=torch.float64, device="cuda")
    if s["initial"] is not None:
        S = s["initial"].double()[where]
    wide = lambda x: x.repeat_interleave(G, 1)
    backward = "do" in s
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    o, dq = new(T, HV, V), new(T, HV, K)
    do = s["do"].double() if backward else None
    for p, n in enumerate(counts):
        at = starts[:n] + p
        now = a[at][..., None, None] * S[:n]
        now += v[at][..., :, None] * wide(k[at])[..., None, :]
        S[:n] = now
        if backward:
            dq[at] = (do[at][..., None, :] @ now)[..., 0, :] * scale
        else:
            o[at] = (now @ wide(q[at])[..., :, None])[..., 0]
    if not backward:
        final = new(*s["final"].shape)
        final[where] = S
        return {"o": o, "final": final}
    D = new(*S.shape) if s["d_final"] is None else s["d_final"].double()[where]
    dk, dv, dg = new(T, HV, K), new(T, HV, V), new(T, HV)
    # d/dg_t: how the terms of q (o_t's) and of k at t and behind it change with the decay they are reached through
    behind = (D * S).sum((-2, -1))
    for p in range(longest - 1, -1, -1):
        n = counts[p]
        at = starts[:n] + p
        kk, qq = wide(k[at]), wide(q[at])
        now = D[:n] + do[at][..., :, None] * qq[..., None, :]
        dk[at] = (v[at][..., None, :] @ now)[..., 0, :]
        dv[at] = (now @ kk[..., :, None])[..., 0]
        behind[:n] += (wide(s["q"][at].double()) * dq[at]).sum(-1) - (kk * dk[at]).sum(-1)
        dg[at] = behind[:n]
        D[:n] = a[at][..., None, None] * now
    group = lambda x: x.unflatten(1, (H, G)).sum(2)
    out = {"dq": group(dq), "dk": group(dk), "dv": dv, "dg": dg.sum(0) if s["g"].dim() == 1 else dg}
    if s["initial"] is not None:
        out["d_initial_state"] = new(*s["initial"].shape)
        out["d_initial_state"][where] = D
    return out


def _turned64(x, positions, frequencies, magnitude, interleaved, inverse):
    """Each pair as a complex number times magnitude e^(i angle)."""
    n, out = frequencies.numel(), x.double().clone()
    pair = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = torch.complex(out[..., pair[0]], out[..., pair[1]])
    angle = positions.double()[:, None] * frequencies * (-1.0 if inverse else 1.0)
    z = z * torch.polar(torch.full_like(angle, magnitude), angle)[:, None, :]
    out[..., pair[0]], out[..., pair[1]] = z.real, z.imag
    return out


def _exact_rotary(s):
    c = s["case"]
    return {n: _turned64(s[n], s["positions"], s["frequencies"], s["magnitude"], c["interleaved"], c["inverse"])
            for n in ("q", "k")}


def _exact_step(s):
    B, HV, V = s["v"].shape
    H, K = s["q"].shape[1:]
    q, k = s["q"].double(), s["k"].double()
    if s["frequencies"] is not None:
        q, k = (_turned64(x, s["positions"], s["frequencies"], 1.0, False, False) for x in (q, k))
    state, out = s["state"].double(), torch.empty(B, HV, V, dtype=torch.float64, device="cuda")
    slots, g = s["slots"].tolist(), s["g"].double().expand(B, HV)
    for b in range(B):
        S = torch.exp(g[b])[:, None, None] * state[slots[b]]
        S += torch.einsum("hv,hk->hvk", s["v"][b].double(), k[b].repeat_interleave(HV // H, 0))
        out[b] = torch.einsum("hvk,hk->hv", S, q[b].repeat_interleave(HV // H, 0)) * K ** -0.5
        state[slots[b]] = S
    return {"out": out, "state": state}
