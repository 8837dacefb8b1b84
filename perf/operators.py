"""Operators of prompt processing, training and beam search over recurrent states, as cases to measure.

Four operators that a recurrent decoder needs around its decode step:

  scan      the Mamba-1 selective scan over whole sequences (prompts): outputs for every token and the
            state after the last one, which the decode step continues from
  scan_bwd  its backward pass
  select    one beam-search selection: the best K of beams x vocabulary by cumulative log-probability
  reorder   the recurrent states of the surviving beams moved to their children, inside the slot pool

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
        {"name": "scan_prompt", "op": "scan", "dtype": "bf16", "lengths": "1x128", "D": 1536, "N": 16,
         "gate": True, "resume": False},
        # a serving step's ragged prompts packed end to end (lengths from 0 and 1 token to a long
        # document), continuing from states in a slot pool
        {"name": "scan_ragged", "op": "scan", "dtype": "bf16", "lengths": "ragged24x8000", "D": 1536, "N": 16,
         "gate": True, "resume": True},
        # one long document: few rows, a long axis
        {"name": "scan_long", "op": "scan", "dtype": "bf16", "lengths": "1x32768", "D": 1536, "N": 16,
         "gate": True, "resume": False},
        # a batch with wide states in fp32, as an evaluation in full precision runs it
        {"name": "scan_wide_fp32", "op": "scan", "dtype": "f32", "lengths": "4x1024", "D": 1536, "N": 128,
         "gate": True, "resume": True},
        # gradients of one short fp32 sequence: fine-tuning at batch one
        {"name": "scan_bwd_small", "op": "scan_bwd", "dtype": "f32", "lengths": "1x500", "D": 1536, "N": 16,
         "gate": True, "resume": False},
        # gradients of a training batch
        {"name": "scan_bwd_batch", "op": "scan_bwd", "dtype": "bf16", "lengths": "8x2048", "D": 1536, "N": 16,
         "gate": True, "resume": False},
        # gradients through packed documents with carried states, odd channel count, wide state
        {"name": "scan_bwd_ragged", "op": "scan_bwd", "dtype": "bf16", "lengths": "ragged10x5000", "D": 1000, "N": 64,
         "gate": False, "resume": True},
        # one request's decode step: four beams, latency-bound
        {"name": "select_one", "op": "select", "dtype": "bf16", "batch": 1, "beams": 4, "vocab": 32000, "K": 4,
         "finished": False, "masked": 0.0},
        # a serving batch over a large vocabulary, some beams already at their end
        {"name": "select_batch", "op": "select", "dtype": "bf16", "batch": 32, "beams": 8, "vocab": 131072, "K": 8,
         "finished": True, "masked": 0.0},
        # fp32 logits of an odd vocabulary with most tokens forbidden, twice as many candidates as beams
        {"name": "select_masked_fp32", "op": "select", "dtype": "f32", "batch": 12, "beams": 5, "vocab": 50021, "K": 10,
         "finished": False, "masked": 0.9},
        # a few beams over small per-layer diagonal states
        {"name": "reorder_small", "op": "reorder", "batch": 2, "beams": 4, "pools": 4, "slot_floats": 1536 * 16,
         "conv_values": 0},
        # a serving batch over matrix states of 32 heads x 128 x 128 and their convolution taps
        {"name": "reorder_large", "op": "reorder", "batch": 16, "beams": 4, "pools": 4,
         "slot_floats": 32 * 128 * 128, "conv_values": 3 * 4096 * 3},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "select", "reorder"])
    if op in ("scan", "scan_bwd"):
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64, 128])
        D = _log_int(rng, 64, 2048)
        most = (32768 * 1536 * 16 if op == "scan" else 8 * 2048 * 1536 * 16) // (D * N)
        T = _log_int(rng, 64, max(65, min(32768, most)))
        if rng.random() < 0.5:
            S = min(T, _log_int(rng, 1, 16))
            lengths = f"{S}x{T // S}"
        else:
            lengths = f"ragged{_log_int(rng, 2, 40)}x{T}"
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "lengths": lengths, "D": D, "N": N,
                "gate": rng.random() < 0.7, "resume": rng.random() < 0.5}
    if op == "select":
        beams = rng.randint(2, 16)
        vocab = _log_int(rng, 1000, 131072)
        batch = _log_int(rng, 1, max(2, min(64, 32 * 8 * 131072 // (beams * vocab))))
        return {"op": op, "dtype": rng.choice(["bf16", "f32"]) if batch * beams * vocab < 16 << 20 else "bf16",
                "batch": batch, "beams": beams, "vocab": vocab, "K": rng.choice([beams, beams, 2 * beams]),
                "finished": rng.random() < 0.5, "masked": rng.choice([0.0, 0.0, 0.9, 0.999])}
    beams = rng.randint(2, 16)
    slot_floats = 4 * _log_int(rng, 64, 32 * 128 * 128 // 4)
    pools = rng.randint(1, 6)
    batch = _log_int(rng, 1, max(2, min(64, (1 << 27) // (slot_floats * pools * beams))))
    return {"op": op, "batch": batch, "beams": beams, "pools": pools, "slot_floats": slot_floats,
            "conv_values": rng.choice([0, 3 * 4 * _log_int(rng, 16, 4096)])}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"scan": _prepare_scan, "scan_bwd": _prepare_scan, "select": _prepare_select, "reorder": _prepare_reorder}
    return {"case": dict(case), **make[case["op"]](case, seed, g)}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_scan(case, seed, g):
    D, N, t = case["D"], case["N"], _TYPES[case["dtype"]]
    lengths = _lengths(case["lengths"], seed)
    T, S = sum(lengths), len(lengths)
    # x and z are the two halves of one projection's rows, and dt, B and C the parts of another's (row views)
    r = -(-N // 8) * 8
    xz = _normal(g, T, 2 * D)
    xz[:, :D] = xz[:, :D] * torch.sigmoid(xz[:, :D])     # x leaves a convolution and a SiLU
    xz = xz.to(t)
    bc = _normal(g, T, 2 * r).to(t)
    # step sizes as a softplus gives them after the usual initialisation: 0.001 to 0.1 around their
    # channel's value
    base = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    dt = (base * torch.exp(0.5 * _normal(g, T, D))).to(t)
    A = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * _normal(g, D, N)))
    first, last, live, at = [], [], [], 0
    for s, n in enumerate(lengths):
        if n:
            live.append(s), first.append(at), last.append(at + n - 1)
        at += n
    dev = lambda v, d=torch.int64: torch.tensor(v, dtype=d, device="cuda")
    uniform = not case["lengths"].startswith("ragged")
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    slots = torch.randperm(S + 3, generator=torch.Generator().manual_seed(seed))[:S]
    st = {"x": xz[:, :D], "z": xz[:, D:] if case["gate"] else None, "dt": dt, "Bm": bc[:, :N], "Cm": bc[:, r:r + N],
          "A": A, "Dskip": torch.ones(D, device="cuda") + 0.1 * _normal(g, D),
          "S": S, "longest": max(lengths), "uniform": uniform, "lengths": lengths,
          "cu": dev(cu, torch.int32), "first": dev(first), "last": dev(last), "live": dev(live),
          "slots": slots.to(torch.int32).cuda(), "h0": None,
          "y": torch.empty(T, D, dtype=t, device="cuda"),
          "h_last": torch.zeros(S + 3, D, N, device="cuda")}
    if case["resume"]:
        st["h0"] = _normal(g, S + 3, D, N)
    if case["op"] == "scan_bwd":
        st["dy"] = _normal(g, T, D).to(t)
        st["dh_last"] = 0.1 * _normal(g, S + 3, D, N) if case["resume"] else None
        like = lambda n: torch.empty(T, n, dtype=t, device="cuda")
        st["grads"] = {"dx": like(D), "ddt": like(D), "dBm": like(N), "dCm": like(N),
                       "dA": torch.empty(D, N, device="cuda"), "dDskip": torch.empty(D, device="cuda"),
                       "dz": like(D) if case["gate"] else None,
                       "dh0": torch.zeros(S + 3, D, N, device="cuda") if case["resume"] else None}
    return st


def _prepare_select(case, seed, g):
    batch, beams, V, K, t = case["batch"], case["beams"], case["vocab"], case["K"], _TYPES[case["dtype"]]
    R = batch * beams
    logits = 2.5 * _normal(g, R, V)
    if case["masked"]:
        logits[torch.rand(R, V, generator=g, device="cuda") < case["masked"]] = -math.inf
    scores = -30.0 * torch.rand(batch, beams, generator=g, device="cuda")
    scores = scores.sort(dim=1, descending=True).values
    finished = None
    if case["finished"]:
        finished = (torch.rand(batch, beams, generator=g, device="cuda") < 0.2).to(torch.uint8)
    rows = torch.randperm(R, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    return {"logits": logits.to(t), "scores": scores, "finished": finished, "eos": 2, "rows": rows,
            "out_scores": torch.empty(batch, K, device="cuda"),
            "out_parents": torch.empty(batch, K, dtype=torch.int32, device="cuda"),
            "out_tokens": torch.empty(batch, K, dtype=torch.int32, device="cuda")}


def _prepare_reorder(case, seed, g):
    batch, beams = case["batch"], case["beams"]
    num_slots = batch * beams + 1                          # slot 0 is the pool's null slot
    pools = [_normal(g, num_slots, case["slot_floats"]) for _ in range(case["pools"])]
    if case["conv_values"]:
        pools += [_normal(g, num_slots, case["conv_values"]).to(torch.bfloat16) for _ in range(case["pools"])]
    h = torch.Generator().manual_seed(seed)
    slots = 1 + torch.randperm(batch * beams, generator=h).to(torch.int32).view(batch, beams)
    # children by score: the better beams have more of them
    p = torch.floor(torch.rand(batch, beams, generator=h) ** 1.5 * beams).to(torch.int32).clamp_(0, beams - 1)
    return {"pools": pools, "slots": slots.cuda(), "parents": p.cuda(), "new_slots": torch.empty_like(slots, device="cuda")}


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_scan(s):
    if "call" not in s:                                    # a user's program keeps its workspace and prepared call
        gdn = _gdn()
        T, D = s["x"].shape
        s["workspace"] = gdn.mamba_scan_workspace(T, D, s["A"].shape[1], sequences=s["S"],
                                                  uniform=s["uniform"])
        s["call"] = gdn.mamba_selective_scan(
            s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["y"], Dskip=s["Dskip"], z=s["z"],
            sequences=s["S"] if s["uniform"] else None, cu_seqlens=None if s["uniform"] else s["cu"],
            h0=s["h0"], h_last=s["h_last"], state_indices=s["slots"], workspace=s["workspace"], prepare=True)
    s["call"]()
    return {"y": s["y"], "h_last": s["h_last"]}


def _own_scan_bwd(s):
    if "call" not in s:
        gdn = _gdn()
        T, D = s["x"].shape
        s["workspace"] = gdn.mamba_scan_workspace(T, D, s["A"].shape[1], sequences=s["S"],
                                                  uniform=s["uniform"], backward=True)
        s["call"] = gdn.mamba_selective_scan_backward(
            s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], Dskip=s["Dskip"], z=s["z"],
            sequences=s["S"] if s["uniform"] else None, cu_seqlens=None if s["uniform"] else s["cu"],
            h0=s["h0"], dh_last=s["dh_last"], state_indices=s["slots"], workspace=s["workspace"], prepare=True,
            **s["grads"])
    s["call"]()
    return {k: v for k, v in s["grads"].items() if v is not None}


def _own_select(s):
    if "call" not in s:
        gdn = _gdn()
        batch, beams = s["scores"].shape
        s["workspace"] = gdn.beam_select_workspace(batch, beams, s["logits"].shape[1], s["out_scores"].shape[1])
        s["call"] = gdn.gdn_beam_select(
            s["logits"], s["scores"], s["out_scores"], s["out_parents"], s["out_tokens"], rows=s["rows"],
            finished=s["finished"], eos_token=s["eos"], workspace=s["workspace"], prepare=True)
    s["call"]()
    return {"scores": s["out_scores"], "parents": s["out_parents"], "tokens": s["out_tokens"]}


def _own_reorder(s):
    if "call" not in s:
        s["call"] = _gdn().gdn_beam_reorder(s["pools"], s["slots"], s["parents"], s["new_slots"], prepare=True)
    s["call"]()
    return {"slots": s["new_slots"], "pools": s["pools"]}


# ---- plain forms -------------------------------------------------------------------------------
def _linear_scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis (h_{-1} = 0), by doubling the span that each entry covers."""
    span = 1
    while span < longest:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _states(s):
    """The decays a [T, D, N] and states h [T, D, N] of every token, and the states each sequence starts from."""
    dt = s["dt"].float()
    # decays just below one, multiplied thousands of times: exp in 64 bits, rounded once
    a = torch.exp(dt.double()[:, :, None] * s["A"].double()).float()
    b = (dt * s["x"].float())[:, :, None] * s["Bm"].float()[:, None, :]
    start = None
    reset = a
    if s["longest"]:
        if s["h0"] is not None:
            start = s["h0"][s["slots"][s["live"]].long()]
            b[s["first"]] += a[s["first"]] * start
        reset = a.clone()
        reset[s["first"]] = 0.0                            # nothing passes from one sequence to the next
    return a, _linear_scan(reset, b, s["longest"]), start


def _silu(z):
    return z * (1.0 / (1.0 + torch.exp(-z)))


def _plain_scan(s):
    _, h, _ = _states(s)
    y = (h * s["Cm"].float()[:, None, :]).sum(-1) + s["Dskip"] * s["x"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    h_last = torch.zeros_like(s["h_last"])
    slots = s["slots"].long()
    if s["h0"] is not None:
        h_last[slots] = s["h0"][slots]                     # an empty sequence keeps its state
    h_last[slots[s["live"]]] = h[s["last"]]
    return {"y": y.to(s["x"].dtype), "h_last": h_last}


def _plain_scan_bwd(s):
    t, slots = s["x"].dtype, s["slots"].long()
    x, dt, Bm, Cm, dy = (s[k].float() for k in ("x", "dt", "Bm", "Cm", "dy"))
    a, h, start = _states(s)
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        pre = (h * Cm[:, None, :]).sum(-1) + s["Dskip"] * x
        out["dz"] = (dy * pre * sig * (1.0 + z * (1.0 - sig))).to(t)
        dy = dy * z * sig
    # dh_t = C_t dy_t + a_{t+1} dh_{t+1}: the same scan, backwards
    b = dy[:, :, None] * Cm[:, None, :]
    if s["dh_last"] is not None:
        b[s["last"]] += s["dh_last"][slots[s["live"]]]
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
    nxt[s["last"]] = 0.0
    dh = _linear_scan(nxt.flip(0), b.flip(0), s["longest"]).flip(0)
    out["dCm"] = (dy[:, :, None] * h).sum(1).to(t)
    out["dBm"] = (dh * (dt * x)[:, :, None]).sum(1).to(t)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[s["first"]] = 0.0 if start is None else start
    da = dh * a * prev
    du = (dh * Bm[:, None, :]).sum(-1)
    out["dx"] = (du * dt + s["Dskip"] * dy).to(t)
    out["ddt"] = (du * x + (da * s["A"]).sum(-1)).to(t)
    out["dA"] = (da * dt[:, :, None]).sum(0)
    out["dDskip"] = (dy * x).sum(0)
    if s["h0"] is not None:
        dh0 = torch.zeros_like(s["h0"])
        if s["dh_last"] is not None:
            dh0[slots] = s["dh_last"][slots]
        dh0[slots[s["live"]]] = dh[s["first"]] * a[s["first"]]
        out["dh0"] = dh0
    return out


def _plain_select(s):
    batch, beams = s["scores"].shape
    V, K = s["logits"].shape[1], s["out_scores"].shape[1]
    x = s["logits"][s["rows"].long()].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.max(dim=1, keepdim=True).values
    total = torch.where(x == top, 1.0, torch.exp(x - top)).sum(1, keepdim=True, dtype=torch.float64)
    # the k best of each row, equal ones by index
    k = min(K, V)
    kth = torch.topk(x, k, dim=1).values[:, -1:]
    above, equal = x > kth, x == kth
    take = above | (equal & (equal.cumsum(1, dtype=torch.int32) <= k - above.sum(1, keepdim=True)))
    place = torch.where(take, take.cumsum(1, dtype=torch.int32) - 1, k).long()
    ids = torch.arange(V, device="cuda").expand(batch * beams, V)
    token = torch.zeros(batch * beams, k + 1, dtype=torch.int64, device="cuda").scatter_(1, place, ids)[:, :k]
    picked = x.gather(1, token)
    # values next to one another in different rows: compared in 64 bits
    logp = torch.where(picked == top, 0.0, (picked - top).double()) - torch.log(total)
    cum = s["scores"].double().view(-1, 1)
    cum = torch.where(torch.isnan(cum), -math.inf, cum)
    score = torch.where(picked == -math.inf, -math.inf, cum + logp)
    if s["finished"] is not None:                          # a finished beam has one candidate: itself
        done = s["finished"].view(-1, 1).bool()
        column = torch.arange(k, device="cuda")
        token = torch.where(done, s["eos"], token)
        score = torch.where(done, torch.where(column == 0, cum, -math.inf), score)
    order = torch.sort(score.reshape(batch, -1), dim=1, descending=True, stable=True)
    best, at = order.values[:, :K], order.indices[:, :K]
    none = best == -math.inf
    parents = torch.where(none, -1, at // k).to(torch.int32)
    tokens = torch.where(none, -1, token.reshape(batch, -1).gather(1, at)).to(torch.int32)
    fill = K - best.shape[1]
    pad = lambda v, w: torch.nn.functional.pad(v, (0, fill), value=w)
    return {"scores": pad(best.float(), -math.inf), "parents": pad(parents, -1), "tokens": pad(tokens, -1)}


def _plain_reorder(s):
    slots, parents = s["slots"].long(), s["parents"].long()
    batch, beams = slots.shape
    beam = torch.arange(beams, device="cuda")
    same = parents[:, :, None] == parents[:, None, :]
    first = ~(same & (beam[None, :] < beam[:, None])).any(2)                 # no earlier child of the same beam
    lost = ~(parents[:, :, None] == beam).any(1)                             # beams without children
    # the n-th child that needs a slot gets the n-th slot that became free
    rank_free = torch.where(lost, lost.cumsum(1) - 1, beams)
    free = torch.zeros(batch, beams + 1, dtype=torch.int64, device="cuda").scatter_(1, rank_free, slots)[:, :beams]
    rank_need = ((~first).cumsum(1) - 1).clamp_min(0)
    new = torch.where(first, slots.gather(1, parents), free.gather(1, rank_need))
    src, dst = slots.gather(1, parents).view(-1), new.view(-1)
    for p in s["pools"]:
        p[dst] = p[src]
    return {"slots": new.to(torch.int32), "pools": s["pools"]}


_OWN = {"scan": _own_scan, "scan_bwd": _own_scan_bwd, "select": _own_select, "reorder": _own_reorder}
_PLAIN = {"scan": _plain_scan, "scan_bwd": _plain_scan_bwd, "select": _plain_select, "reorder": _plain_reorder}


# ------------------------------------------------------------------------------------------------
# what one pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("scan", "scan_bwd"):
        spec = case["lengths"]
        if spec.startswith("ragged"):
            S, T = (int(v) for v in spec[6:].split("x"))
        else:
            S, L = (int(v) for v in spec.split("x"))
            T = S * L
        D, N, e = case["D"], case["N"], 2 if case["dtype"] == "bf16" else 4
        gate, resume = int(case["gate"]), int(case["resume"])
        if op == "scan":
            # x, dt, z in, y out; B, C; A, D; the states
            return {"bytes": T * D * e * (3 + gate) + 2 * T * N * e + 4 * D * (N + 1) + 4 * S * D * N * (1 + resume),
                    # per state entry: dt A, exp, u B, multiply-add into h, multiply-add into y
                    "flops": 7 * T * D * N}
        return {"bytes": T * D * e * (5 + 2 * gate) + 4 * T * N * e + 8 * D * (N + 1) + 4 * S * D * N * 3 * resume,
                # the states again (5), dh (2), dB, dC, du (6), dh a, its product with h (2), ddt, dA (4)
                "flops": (19 + 2 * gate) * T * D * N}
    if op == "select":
        R, e = case["batch"] * case["beams"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": R * case["vocab"] * e + 8 * R + 12 * case["batch"] * case["K"], "flops": 4 * R * case["vocab"]}
    # every child but a beam's first takes a copy: about 0.35 of the beams at these parents
    slot = 4 * case["slot_floats"] + 2 * case["conv_values"]
    moved = max(1, round(0.35 * case["batch"] * case["beams"]))
    return {"bytes": 2 * moved * slot * case["pools"] + 12 * case["batch"] * case["beams"], "flops": 0}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "scan_bwd": _exact_scan, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](s)


def _exact_scan(s):
    """Token by token, all sequences side by side (position p of each that is long enough)."""
    d = {k: s[k].double() for k in ("x", "dt", "Bm", "Cm", "A", "Dskip")}
    z = None if s["z"] is None else s["z"].double()
    lengths, slots = s["lengths"], s["slots"].long()
    T, D = d["x"].shape
    N = d["A"].shape[1]
    order = sorted(range(s["S"]), key=lambda i: -lengths[i])           # long ones first: the live ones are a prefix
    starts = torch.tensor([sum(lengths[:i]) for i in order], device="cuda")
    where = slots[torch.tensor(order, device="cuda")]
    counts = [sum(1 for i in order if lengths[i] > p) for p in range(s["longest"])]
    h = torch.zeros(s["S"], D, N, dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h = s["h0"].double()[where]
    backward = "dy" in s
    if backward and T * D * N > 1 << 32:
        return None
    before = torch.empty(T, D, N, dtype=torch.float64, device="cuda") if backward else None
    pre = torch.empty(T, D, dtype=torch.float64, device="cuda")
    for p, n in enumerate(counts):
        at = starts[:n] + p
        if backward:
            before[at] = h[:n]
        dt = d["dt"][at]
        h[:n] = torch.exp(dt[:, :, None] * d["A"]) * h[:n] + (dt * d["x"][at])[:, :, None] * d["Bm"][at][:, None, :]
        pre[at] = torch.einsum("bdn,bn->bd", h[:n], d["Cm"][at]) + d["Dskip"] * d["x"][at]
    if not backward:
        y = pre if z is None else pre * z * torch.sigmoid(z)
        h_last = torch.zeros(s["h_last"].shape, dtype=torch.float64, device="cuda")
        h_last[where] = h
        return {"y": y, "h_last": h_last}
    dy = s["dy"].double()
    out = {}
    if z is not None:
        sig = torch.sigmoid(z)
        out["dz"] = dy * pre * (sig + z * sig * (1 - sig))
        dy = dy * z * sig
    g = torch.zeros_like(h) if s["dh_last"] is None else s["dh_last"].double()[where]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    out |= {"dx": new(T, D), "ddt": new(T, D), "dBm": new(T, N), "dCm": new(T, N), "dA": new(D, N)}
    out["dDskip"] = (dy * d["x"]).sum(0)
    for p in range(s["longest"] - 1, -1, -1):
        n = counts[p]
        at = starts[:n] + p
        dt, x, B, C = d["dt"][at], d["x"][at], d["Bm"][at], d["Cm"][at]
        a = torch.exp(dt[:, :, None] * d["A"])
        now = a * before[at] + (dt * x)[:, :, None] * B[:, None, :]
        out["dCm"][at] = torch.einsum("bd,bdn->bn", dy[at], now)
        gn = g[:n] + dy[at][:, :, None] * C[:, None, :]
        out["dBm"][at] = torch.einsum("bdn,bd->bn", gn, dt * x)
        du = torch.einsum("bdn,bn->bd", gn, B)
        w = gn * a * before[at]
        out["dx"][at] = du * dt + d["Dskip"] * dy[at]
        out["ddt"][at] = du * x + (w * d["A"]).sum(-1)
        out["dA"] += torch.einsum("bdn,bd->dn", w, dt)
        g[:n] = gn * a
    if s["h0"] is not None:
        out["dh0"] = new(*s["h0"].shape)
        out["dh0"][where] = g
    return out


def _exact_select(s):
    batch, beams = s["scores"].shape
    V, K = s["logits"].shape[1], s["out_scores"].shape[1]
    scores = torch.full((batch, K), -math.inf, dtype=torch.float64, device="cuda")
    parents = torch.full((batch, K), -1, dtype=torch.int32, device="cuda")
    tokens = torch.full((batch, K), -1, dtype=torch.int32, device="cuda")
    for b in range(batch):
        x = s["logits"][s["rows"][b * beams:(b + 1) * beams].long()].double()
        top = x.amax(1, keepdim=True)
        total = s["scores"][b].double()[:, None] + ((x - top) - torch.log(torch.exp(x - top).sum(1, keepdim=True)))
        total = torch.where(torch.isnan(total), -math.inf, total)      # a row without any finite logit
        if s["finished"] is not None:
            done = s["finished"][b].bool()
            total[done] = -math.inf
            total[done, s["eos"]] = s["scores"][b].double()[done]
        v, i = torch.sort(total.reshape(-1), descending=True, stable=True)
        n = min(K, int((v[:K] > -math.inf).sum()))
        scores[b, :n], parents[b, :n], tokens[b, :n] = v[:n], (i[:n] // V).int(), (i[:n] % V).int()
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _exact_reorder(s):
    slots, parents = s["slots"].tolist(), s["parents"].tolist()
    before = [p.clone() for p in s["pools"]]
    new = []
    for row, par in zip(slots, parents):
        free = [row[b] for b in range(len(row)) if b not in par]
        seen, out = set(), []
        for p in par:
            out.append(free.pop(0) if p in seen else row[p])
            seen.add(p)
        for to, p in zip(out, par):
            for q, old in zip(s["pools"], before):
                q[to] = old[row[p]]
        new.append(out)
    return {"slots": torch.tensor(new, dtype=torch.int32, device="cuda"), "pools": s["pools"]}
