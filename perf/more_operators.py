"""The workloads of the linear-attention layers: their recurrence for prompts and for single tokens, and the norms around it.

Four operators that a hybrid engine's linear-attention layer runs, one decay for each head:

  prompt    packed sequences: S_t = e^(g_t) S_(t-1) + k_t v_t^T, o_t = scale S_t^T q_t for all their tokens, with the states at
            chosen boundaries written to pages
  step      one token (or a few drafted ones) of every sequence of a batch, on states kept in a pool
  gated     the heads' outputs normalised and multiplied by an activated gate
  residual  a block's output normalised, gated, scaled and added to the residual stream, and the sum normalised for the next block

`listed()` names the fixed workloads, `draw()` makes others over the same ranges; `run()` is one call, in elementary torch
operations or, with `own` set, through the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

ES = {"bf16": 2, "f32": 4}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64                                # tokens per chunk of the plain form
EPS = 1e-6


def listed():
    return [
        # A long prompt of a full-size layer, continued from a state, checkpoints as a prefix cache keeps them.
        _prompt("prompt-long", lo=8192, hi=8192, stride=512, resume=True),
        # The largest: a prefill batch of prompts of mixed lengths, new sequences without a state.
        _prompt("prompt-batch", N=24, lo=512, hi=16384, stride=1024),
        # One very long document, few heads with fixed decays: the work has to be split along the tokens.
        _prompt("prompt-few", H=4, H_k=4, lo=65536, hi=65536, fixed=True),
        # Short turns of running conversations, odd lengths, one of them empty; heads that share keys and queries.
        _prompt("prompt-turns", N=19, H=48, H_k=8, dv=64, lo=0, hi=300, resume=True, resets=3),
        # A small model kept in fp32.
        _prompt("prompt-f32", N=3, H=8, H_k=8, dk=64, dv=32, lo=61, hi=1999, resume=True, dtype="f32"),
        # One conversation, one token. Latency is all that counts.
        _step("step-one", B=1),
        # A full decode batch over a pool of states, a few rows of the batch empty: the states' bandwidth.
        _step("step-batch", B=256, slots=True, padded=3),
        # Drafts of five tokens, of which each sequence accepted some: outputs, and the states after the accepted tokens to
        # other slots.
        _step("step-draft", B=32, steps=5, H=64, H_k=8, dv=64, slots=True, kind="accept", padded=1),
        # The head outputs of a decode batch.
        _gated("gated-batch", T=256),
        # The head outputs of a prefill batch; the gate is part of a wider projection.
        _gated("gated-prompt", T=32768),
        # Between two blocks, for a decode batch.
        _residual("residual-batch", T=256, D=4096),
        # The same for a prefill batch of a wider model, every part of it, the residual stream kept in fp32.
        _residual("residual-prompt", T=16384, D=6144, h="f32", post=True, gate=True, channel=True),
    ]


def _case(defaults, kw):
    assert set(kw) <= set(defaults)
    return {**defaults, **kw}


def _prompt(name, **kw):
    return _case({"name": name, "op": "prompt", "N": 1, "H": 32, "H_k": 32, "dk": 128, "dv": 128, "lo": 1, "hi": 1, "stride": 0,
                  "resume": False, "fixed": False, "resets": 0, "dtype": "bf16"}, kw)


def _step(name, **kw):
    return _case({"name": name, "op": "step", "B": 1, "steps": 1, "H": 32, "H_k": 32, "dk": 128, "dv": 128, "slots": False,
                  "kind": "advance", "fixed": False, "padded": 0, "dtype": "bf16"}, kw)


def _gated(name, **kw):
    return _case({"name": name, "op": "gated", "T": 1, "H": 32, "d": 128, "act": "sigmoid", "first": False, "per_head": False,
                  "dtype": "bf16"}, kw)


def _residual(name, **kw):
    return _case({"name": name, "op": "residual", "T": 1, "D": 4096, "h": "bf16", "post": False, "gate": False, "channel": False,
                  "act": "sigmoid", "dtype": "bf16"}, kw)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    kind = rng.choice(["prompt", "prompt", "step", "step", "gated", "residual"])
    H_k = rng.choice([1, 2, 4, 8, 8, 16, 32])
    H = H_k * rng.choice([1, 1, 1, 2, 3, 8])
    dk, dv = (128, 128) if rng.random() < 0.4 else (rng.choice([32, 64, 128]), rng.choice([32, 64, 128]))
    if kind == "prompt":
        while True:
            N = 1 if rng.random() < 0.4 else _log(rng, 2, 200)
            hi = _log(rng, 1, 65536)
            case = _prompt("", N=N, H=H, H_k=H_k, dk=dk, dv=dv, lo=rng.choice([0, 1, _log(rng, 1, hi), hi]), hi=hi,
                           stride=rng.choice([0, 0, 128, 384, 512, 1024]), resume=rng.random() < 0.5, fixed=rng.random() < 0.3,
                           resets=rng.choice([0, 0, 1, 5]), dtype=dtype)
            states = (sum(_checkpoints(case)) + N) * H * dk * dv
            if (work(case)["flops"] <= (4e10 if dtype == "f32" else 2e11) and states <= 1.5e9 and sum(_lengths(case)) <= 140000
                    and sum(_lengths(case)) > 0 and H * (N + sum(_lengths(case)) // CHUNK) ** 2 <= 2e8):
                break
    elif kind == "step":
        while True:
            B, steps = _log(rng, 1, 512), 1 if rng.random() < 0.6 else rng.randint(2, 16)
            case = _step("", B=B, steps=steps, H=H, H_k=H_k, dk=dk, dv=dv, slots=rng.random() < 0.6, fixed=rng.random() < 0.3,
                         kind="advance" if steps == 1 else rng.choice(["advance", "verify", "accept"]),
                         padded=0, dtype=dtype)
            case["padded"] = rng.randrange(0, 1 + B // 8) if case["slots"] else 0
            if B * H * dk * dv <= 300e6:
                break
    elif kind == "gated":
        T = _log(rng, 1, 32768)
        case = _gated("", T=T, H=max(1, min(H, 2 ** 27 // T // 128)), d=rng.choice([32, 64, 80, 96, 128, 128, 192, 256, 512]),
                      act=rng.choice(["sigmoid", "silu"]), first=rng.random() < 0.4, per_head=rng.random() < 0.4, dtype=dtype)
    else:
        D = 8 * _log(rng, 8, 1024)
        case = _residual("", T=_log(rng, 1, min(32768, 2 ** 27 // D)), D=D, h="f32" if dtype == "f32" or rng.random() < 0.4 else "bf16",
                         post=rng.random() < 0.5, gate=rng.random() < 0.5, channel=rng.random() < 0.3,
                         act=rng.choice(["sigmoid", "silu"]), dtype=dtype)
    del case["name"]
    return case


def _lengths(case):
    """Lengths of a batch of prompts: log-uniform quantiles between lo and hi."""
    n, lo, hi = case["N"], min(case["lo"], case["hi"]) + 1, case["hi"] + 1
    if n == 1:
        return [case["hi"]]
    return [int(round(lo * (hi / lo) ** (j / (n - 1)))) - 1 for j in range(n)]


def _checkpoints(case):
    return [n // case["stride"] if case["stride"] else 0 for n in _lengths(case)]


def work(case):
    es = ES[case["dtype"]]
    if case["op"] == "gated":
        n = case["T"] * case["H"] * case["d"]
        return {"bytes": 3 * n * es, "flops": 10 * n}
    if case["op"] == "residual":
        n = case["T"] * case["D"]
        return {"bytes": n * (2 * es + 2 * ES[case["h"]] + (es if case["gate"] else 0)), "flops": 12 * n}
    H, state = case["H"], case["dk"] * case["dv"]
    row = (2 * case["H_k"] * case["dk"] + 2 * H * case["dv"]) * es + (0 if case["fixed"] else 4 * H)
    if case["op"] == "prompt":
        T, N = sum(_lengths(case)), case["N"]
        moved = (1 + case["resume"]) * N + sum(_checkpoints(case))
        return {"bytes": T * row + moved * H * state * 4, "flops": 4 * T * H * state}
    live = case["B"] - case["padded"]
    moved = 1 if case["kind"] == "verify" else 2
    return {"bytes": live * (case["steps"] * row + moved * H * state * 4), "flops": 4 * live * case["steps"] * H * state}


# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    if case["op"] == "gated":
        T, H, d = case["T"], case["H"], case["d"]
        fused = normal(T, H * d + 64)                     # the gate's projection beside another small one
        weight = 1 + 0.1 * torch.randn((H, d) if case["per_head"] else (d,), generator=gen, device="cuda")
        return {"case": case, "x": normal(T, H, d), "gate": fused[:, :H * d].view(T, H, d), "weight": weight.to(dt)}
    if case["op"] == "residual":
        T, D = case["T"], case["D"]

        def about_one():
            return (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)

        return {"case": case, "y": normal(T, D), "h": (4 * torch.randn(T, D, generator=gen, device="cuda")).to(DT[case["h"]]),
                "pre": about_one(), "post": about_one() if case["post"] else None, "gate": normal(T, D) if case["gate"] else None,
                "channel": about_one() if case["channel"] else None, "scale": 0.5}

    H, H_k, dk, dv = case["H"], case["H_k"], case["dk"], case["dv"]

    def projections(rows):
        """q, k, v as views of one projection's output, and the log decays: heads that remember 4 to 4096 tokens."""
        fused = normal(rows, 2 * H_k * dk + H * dv)
        q, k, v = fused.split([H_k * dk, H_k * dk, H * dv], 1)
        rate = 4.0 ** -(1 + 5 * torch.rand(H, generator=gen, device="cuda"))
        g = -rate if case["fixed"] else -rate * 1.5 * torch.nn.functional.softplus(torch.randn(rows, H, generator=gen, device="cuda"))
        return {"q": q.view(rows, H_k, dk), "k": k.view(rows, H_k, dk), "v": v.view(rows, H, dv), "g": g}

    scale = dk ** -0.5
    if case["op"] == "step":
        B, steps = case["B"], case["steps"]
        slots = 2 * B + 1 if case["slots"] else B
        s = {"case": case, "scale": scale, "S": 0.5 * torch.randn(slots, H, dk, dv, generator=gen, device="cuda"), **projections(steps * B)}
        for n in ("q", "k", "v") + (() if case["fixed"] else ("g",)):
            s[n] = s[n].unflatten(0, (steps, B))
        ids = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        if case["slots"]:
            s["slot_in"] = ids[:B].clone()
            s["slot_in"][torch.randperm(B, generator=gen, device="cuda")[:case["padded"]]] = -1
        if case["kind"] == "accept":
            s["n_accepted"] = torch.randint(0, steps + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            if case["slots"]:
                s["slot_out"] = ids[B:2 * B].clone()
            else:
                s["S_new"] = torch.zeros_like(s["S"])
        return s
    lens = _lengths(case)
    order = torch.randperm(case["N"], generator=gen, device="cuda").tolist()
    cu = [0]
    for j in order:
        cu.append(cu[-1] + lens[j])
    T, n_ck = cu[-1], sum(_checkpoints(case))
    s = {"case": case, "scale": scale, "cu": cu, **projections(T)}
    if case["resets"] and not case["fixed"]:
        s["g"][torch.randint(0, T, (case["resets"],), generator=gen, device="cuda")] = -math.inf
    s["S0"] = 0.5 * torch.randn(case["N"], H, dk, dv, generator=gen, device="cuda") if case["resume"] else None
    if n_ck:
        # pages a little larger than a state, as a pool shared with other layers has them
        s["pages"] = torch.randn(n_ck + 2, H * dk * dv + 32, generator=gen, device="cuda")
        s["page_ids"] = torch.randperm(n_ck + 2, generator=gen, device="cuda")[:n_ck].to(torch.int32)
    return s


# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "step": _own_step, "gated": _own_gated, "residual": _own_residual}[op](state)
    return {"prompt": _plain_prompt, "step": _plain_step, "gated": _plain_gated, "residual": _plain_residual}[op](state)


def _own_prompt(s):
    from kda_delta_rule_gb300 import kda as K
    pages = {"page_pool": s["pages"].view(torch.uint8), "ckpt_page_ids": s["page_ids"]} if "pages" in s else {}
    o, S = K.kda_linattn_prefill(s["S0"], s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"], scale=s["scale"],
                                 ckpt_stride=s["case"]["stride"] if pages else 0, **pages)
    return {"o": o, "S": S, "pages": s.get("pages")}


def _own_step(s):
    from kda_delta_rule_gb300 import kda as K
    o = K.kda_linattn_step(s["S"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"], slot_in=s.get("slot_in"), slot_out=s.get("slot_out"),
                           n_accepted=s.get("n_accepted"), S_new=s.get("S_new"), write_state=s["case"]["kind"] != "verify")
    return {"o": o, "S": s.get("S_new", s["S"])}


def _own_gated(s):
    from kda_delta_rule_gb300 import kda as K
    return K.kda_gated_norm(s["x"], s["weight"], gate=s["gate"], eps=EPS, act=K.ACT_SILU if s["case"]["act"] == "silu" else K.ACT_SIGMOID,
                            gate_first=s["case"]["first"])


def _own_residual(s):
    from kda_delta_rule_gb300 import kda as K
    h, x = K.kda_residual_norm(s["h"], s["y"], s["pre"], post_weight=s["post"], gate=s["gate"], channel_scale=s["channel"],
                               res_scale=s["scale"], eps=EPS, act=K.ACT_SILU if s["case"]["act"] == "silu" else K.ACT_SIGMOID)
    return {"h": h, "x": x}


def _per_head(x, H):
    """(.., H_k, d) in fp32 for each of the H heads: consecutive heads share one."""
    return x.float().repeat_interleave(H // x.shape[-2], -2)


def _plain_prompt(s):
    """Chunks of 64 tokens: within them the masked products q k^T with their decays; between them the states, each a sum over the
    earlier chunks of its sequence with the decays from their ends."""
    case = s["case"]
    H, dk, dv, N, T = case["H"], case["dk"], case["dv"], case["N"], s["v"].shape[0]
    dev = s["v"].device
    cu = torch.tensor(s["cu"])
    lens = cu[1:] - cu[:-1]
    chunks = (lens + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(N), chunks)
    nth = torch.arange(len(seq)) - (chunks.cumsum(0) - chunks)[seq]
    pos = CHUNK * nth[:, None] + torch.arange(CHUNK)
    live = (pos < lens[seq][:, None]).to(dev)
    at = (cu[seq][:, None] + pos).to(dev).masked_fill(~live, 0)
    last, nth, seq = (chunks.cumsum(0) - 1).to(dev), nth.to(dev), seq.to(dev)

    def chunked(x):                                       # (T, H, d) -> (chunks, H, 64, d), zeros past the sequence's end
        return x[at].masked_fill(~live[..., None, None], 0).transpose(1, 2)

    q, k, v = chunked(_per_head(s["q"], H)), chunked(_per_head(s["k"], H)), chunked(s["v"].float())
    g = s["g"].double().clamp(min=-1e4).expand(T, H)      # e^-1e4 is 0; sums of logs in fp64, since their differences count
    b = chunked(g[..., None])[..., 0].cumsum(-1)           # (chunks, H, 64)
    near = torch.exp((b[..., :, None] - b[..., None, :]).tril()).float().tril()
    o = ((q @ k.transpose(-1, -2)) * near) @ v
    add = (k * torch.exp(b[..., -1:] - b).float()[..., None]).transpose(-1, -2) @ v
    total = b[..., -1].T                                   # (H, chunks)
    end = total.cumsum(-1)
    before = end - total
    same = (seq[:, None] == seq[None, :]).tril(-1)
    far = torch.exp((before[..., :, None] - end[..., None, :]).masked_fill(~same, -math.inf)).float()
    start = (far @ add.transpose(0, 1).flatten(2)).view(H, len(seq), dk, dv)
    if s["S0"] is not None:
        since = before - before[:, (last[seq] + 1 - chunks.to(dev)[seq])]
        start = start + torch.exp(since).float()[..., None, None] * s["S0"].transpose(0, 1)[:, seq]
    start = start.transpose(0, 1)
    o = (o + torch.exp(b).float()[..., None] * (q @ start)) * s["scale"]
    ends = torch.exp(total.T).float()[..., None, None] * start + add
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(N, H, dk, dv, device=dev)
    some = (chunks > 0).to(dev)
    S[some] = ends[last[some]]
    out = torch.empty(T, H, dv, device=dev, dtype=s["v"].dtype)
    out[at[live]] = o.transpose(1, 2)[live].to(out.dtype)
    if "pages" in s:
        reached = CHUNK * (nth + 1)
        states = ends[(reached % case["stride"] == 0) & (reached <= lens.to(dev)[seq])].flatten(1)
        s["pages"][s["page_ids"].long()] = torch.nn.functional.pad(states, (0, s["pages"].shape[1] - states.shape[1]))
    return {"o": out, "S": S, "pages": s.get("pages")}


def _plain_step(s):
    """A few tokens at once: token t reads the state before them, decayed, and the tokens up to itself, with their decays."""
    case = s["case"]
    H, steps, B, n_slots = case["H"], case["steps"], case["B"], s["S"].shape[0]
    ids = s.get("slot_in", torch.arange(B, device=s["S"].device)).long()
    live = (ids >= 0) & (ids < n_slots)
    S = s["S"][ids.clamp(min=0)]
    q, k, v = (x.permute(1, 2, 0, 3) for x in (_per_head(s["q"], H), _per_head(s["k"], H), s["v"].float()))      # (B, H, steps, d)
    g = s["g"].double().clamp(min=-1e4).expand(steps, B, H).permute(1, 2, 0)
    n = s.get("n_accepted", torch.full((B,), steps, device=S.device)).long()
    b = (g * (torch.arange(steps, device=S.device) < n[:, None, None])).cumsum(-1)
    near = torch.exp((b[..., :, None] - b[..., None, :]).tril()).float().tril()
    o = ((q @ k.transpose(-1, -2)) * near) @ v + torch.exp(b).float()[..., None] * (q @ S)
    taken = (torch.arange(steps, device=S.device) < n[:, None]) & live[:, None]
    o = (o * s["scale"]).masked_fill(~taken[:, None, :, None], 0).permute(2, 0, 1, 3).to(s["v"].dtype)
    if case["kind"] == "verify":
        return {"o": o, "S": s["S"]}
    add = (k * (torch.exp(b[..., -1:] - b).float() * taken[:, None])[..., None]).transpose(-1, -2) @ v
    S = torch.exp(b[..., -1]).float()[..., None, None] * S + add
    to, out = s.get("S_new", s["S"]), s.get("slot_out", ids).long()
    to[out[live]] = S[live]
    return {"o": o, "S": to}


def _activated(x, act):
    return x / (1 + torch.exp(-x)) if act == "silu" else 1 / (1 + torch.exp(-x))


def _normed(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_gated(s):
    x, gate = s["x"].float(), _activated(s["gate"].float(), s["case"]["act"])
    y = _normed(x * gate, s["weight"]) if s["case"]["first"] else _normed(x, s["weight"]) * gate
    return y.to(s["x"].dtype)


def _plain_residual(s):
    u = s["y"].float()
    if s["post"] is not None:
        u = _normed(u, s["post"])
    if s["gate"] is not None:
        u = u * _activated(s["gate"].float(), s["case"]["act"])
    if s["channel"] is not None:
        u = u * s["channel"].float()
    h = s["h"].float() + s["scale"] * u
    s["h"].copy_(h)
    return {"h": s["h"], "x": _normed(h, s["pre"]).to(s["y"].dtype)}


# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "prompt":
        longest = _lengths(case)
        # a pass over the states for each token position, about 100 us and their bytes
        states = sum(min(n, 1) for n in longest) * case["H"] * case["dk"] * case["dv"]
        if max(longest) * (1.5e-4 + 40 * states / 3e12) > 18:
            return None
        return _exact_prompt(prepare(case, seed))
    s = prepare(case, seed)
    return {"step": _exact_step, "gated": _exact_gated, "residual": _exact_residual}[case["op"]](s)


def _token(S, q, k, v, g):
    """The recurrence for one token: states (.., dk, dv), rows (.., d), log decays (..); the new states and the outputs."""
    S.mul_(torch.exp(g)[..., None, None])
    S.addcmul_(k[..., :, None], v[..., None, :])
    return torch.einsum("...i,...ij->...j", q, S)


def _exact_prompt(s):
    case = s["case"]
    H, share, N = case["H"], case["H"] // case["H_k"], case["N"]
    T, dev = s["v"].shape[0], s["v"].device
    lens = [b - a for a, b in zip(s["cu"], s["cu"][1:])]
    order = sorted(range(N), key=lambda j: -lens[j])      # the sequences that still run come first
    S = torch.zeros(N, H, case["dk"], case["dv"], dtype=torch.float64, device=dev)
    if s["S0"] is not None:
        S.copy_(s["S0"][order])
    o = torch.zeros(T, H, case["dv"], dtype=torch.float64, device=dev)
    g = s["g"].double().expand(T, H)
    first = torch.tensor([s["cu"][j] for j in order], device=dev)
    pages, stride = s["pages"].double() if "pages" in s else None, case["stride"]
    ck0 = [sum(n // stride for n in lens[:j]) for j in range(N)] if pages is not None else None
    ids = s["page_ids"].tolist() if pages is not None else None
    running = N
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        at = first[:running] + t
        head = (lambda x: x[at].double().repeat_interleave(share, 1))  # noqa: E731
        o[at] = _token(S[:running], head(s["q"]) * s["scale"], head(s["k"]), s["v"][at].double(), g[at])
        if pages is not None and (t + 1) % stride == 0:
            for j in range(running):
                page = pages[ids[ck0[order[j]] + (t + 1) // stride - 1]]
                page.zero_()
                page[:S[j].numel()] = S[j].flatten()
    S_final = torch.empty_like(S)
    S_final[order] = S
    return {"o": o, "S": S_final, "pages": pages}


def _exact_step(s):
    case = s["case"]
    H, share, B, steps = case["H"], case["H"] // case["H_k"], case["B"], case["steps"]
    S_all = s["S"].double()
    ids = s["slot_in"].tolist() if "slot_in" in s else list(range(B))
    rows = [b for b in range(B) if 0 <= ids[b] < len(S_all)]
    S = S_all[[ids[b] for b in rows]]
    n = s["n_accepted"].tolist() if "n_accepted" in s else [steps] * B
    o = torch.zeros(steps, B, H, case["dv"], dtype=torch.float64, device=S.device)
    g = s["g"].double().expand(steps, B, H)
    for t in range(steps):
        j = [i for i, b in enumerate(rows) if t < n[b]]
        if j:
            b = [rows[i] for i in j]
            part = S[j]
            o[t, b] = _token(part, s["q"][t, b].double().repeat_interleave(share, 1) * s["scale"],
                             s["k"][t, b].double().repeat_interleave(share, 1), s["v"][t, b].double(), g[t, b])
            S[j] = part
    if case["kind"] == "verify":
        return {"o": o, "S": s["S"].double()}
    out = s["slot_out"].tolist() if "slot_out" in s else ids
    to = s["S_new"].double() if "S_new" in s else S_all
    to[[out[b] for b in rows]] = S
    return {"o": o, "S": to}


def _exact_act(x, act):
    return torch.sigmoid(x) * (x if act == "silu" else 1)


def _exact_rms(x):
    return (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS).sqrt()


def _exact_gated(s):
    x, gate = s["x"].double(), _exact_act(s["gate"].double(), s["case"]["act"])
    if s["case"]["first"]:
        x = x * gate
        return x / _exact_rms(x) * s["weight"].double()
    return x / _exact_rms(x) * s["weight"].double() * gate


def _exact_residual(s):
    u = s["y"].double()
    if s["post"] is not None:
        u = u / _exact_rms(u) * s["post"].double()
    for name in ("gate", "channel"):
        if s[name] is not None:
            u = u * (_exact_act(s[name].double(), s["case"]["act"]) if name == "gate" else s[name].double())
    h = s["h"].double() + s["scale"] * u
    return {"h": h, "x": h / _exact_rms(h) * s["pre"].double()}
