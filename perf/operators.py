"""The workloads of the latent page cache: appending tokens to it, and attending to it.

Two operators of a hybrid engine's attention layers, which keep one latent row per token ([c | k_pe], d_c + d_r
values shared by all heads) in the MLA_KV pages of the unified page pool:

  append  new tokens' rows are normalised, rotated to their positions and written into their pages; the queries' position
          parts are rotated on the way
  attend  every query of a batch attends to the rows of a prefix that the whole batch shares and of its sequence's own pages

`listed()` names the fixed workloads, `draw()` makes others over the same ranges; `run()` is one call, in elementary torch
operations or, with `own` set, through the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

ES = {"bf16": 2, "f32": 4}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One conversation, one token: a single sequence early in its answer. Latency is all that counts.
        _attend("attend-one", B=1, n_q=1, H=32, page=512, prefix=0, lo=700, hi=700),
        # A full decode batch without anything shared, lengths as in a mixed service: the cache's bandwidth.
        _attend("attend-batch", B=256, n_q=1, H=32, page=512, prefix=0, lo=512, hi=8192),
        # A batch behind one long system prompt, each with a short turn of its own.
        _attend("attend-shared", B=128, n_q=1, H=32, page=512, prefix=16384, lo=16, hi=1024),
        # The same kind of batch verifying drafts of eight tokens, pages of 64 tokens.
        _attend("attend-draft", B=32, n_q=8, H=32, page=64, prefix=8000, lo=9, hi=600),
        # A few very long documents: the work has to be split along the tokens. Half the heads.
        _attend("attend-long", B=4, n_q=1, H=16, page=512, prefix=0, lo=100000, hi=131072),
        # The largest: many heads, a prefix of a whole code base, own turns of some thousand tokens.
        _attend("attend-heads", B=64, n_q=1, H=128, page=512, prefix=32768, lo=64, hi=4096),
        # Odd sizes throughout: heads and drafts that fill no tile, pages that end inside one, empty and padded rows.
        _attend("attend-odd", B=37, n_q=3, H=20, d_c=384, d_r=48, page=48, prefix=1003, lo=0, hi=1900, padded=2),
        # A small model kept in fp32.
        _attend("attend-f32", B=16, n_q=1, H=16, d_c=256, d_r=32, page=16, prefix=1024, lo=1, hi=500, dtype="f32"),
        # One decoded token of one sequence.
        _append("append-one", T=1, H=32, page=512),
        # One decoded token of every sequence of a full batch, some rows of the batch empty.
        _append("append-batch", T=256, H=32, page=512, padded=5),
        # A long prompt's tokens.
        _append("append-prompt", T=32768, H=32, page=512),
        # The small fp32 model's prompt, pairs interleaved, rows that come normalised.
        _append("append-f32", T=1999, H=16, d_c=256, d_r=32, page=16, norm=False, interleaved=True, dtype="f32"),
    ]


def _attend(name, **kw):
    case = {"name": name, "op": "attend", "B": 1, "n_q": 1, "H": 32, "d_c": 512, "d_r": 64, "page": 512, "prefix": 0, "lo": 1,
            "hi": 1, "padded": 0, "dtype": "bf16"}
    assert set(kw) <= set(case)
    return {**case, **kw}


def _append(name, **kw):
    case = {"name": name, "op": "append", "T": 1, "H": 32, "d_c": 512, "d_r": 64, "page": 512, "padded": 0, "norm": True,
            "interleaved": False, "dtype": "bf16"}
    assert set(kw) <= set(case)
    return {**case, **kw}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    f32 = rng.random() < 0.2
    d_c, d_r = (512, 64) if rng.random() < 0.5 else (rng.choice([128, 256, 384, 512]), rng.choice([16, 32, 48, 64]))
    page = rng.choice([16, 32, 48, 64, 80, 128, 256, 512, 512])
    if rng.random() < 0.35:
        T = _log(rng, 1, 8192 if f32 else 32768)
        case = _append("", T=T, H=_log(rng, 1, 48), d_c=d_c, d_r=d_r, page=page, padded=rng.randrange(0, 1 + T // 8),
                       norm=rng.random() < 0.7, interleaved=rng.random() < 0.4, dtype="f32" if f32 else "bf16")
    else:
        while True:
            B, n_q = _log(rng, 1, 256), 1 if rng.random() < 0.6 else rng.randint(2, 16)
            H = rng.choice([8, 12, 16, 20, 32, 32, 48, 64, 128])
            prefix = 0 if rng.random() < 0.4 else _log(rng, 64, 32768)
            hi = _log(rng, 8, 65536)
            lo = rng.choice([0, 1, _log(rng, 1, hi)])
            case = _attend("", B=B, n_q=n_q, H=H, d_c=d_c, d_r=d_r, page=page, prefix=prefix, lo=min(lo, hi), hi=hi,
                           padded=rng.randrange(0, 1 + B // 8), dtype="f32" if f32 else "bf16")
            rows = B * n_q * H
            if (work(case)["flops"] <= (1e11 if f32 else 5e11) and B * hi * (d_c + d_r) <= 1e9 and rows * prefix <= 3e8
                    and rows * hi <= 3e8):
                break
    del case["name"]
    return case


def _lengths(case):
    """Own lengths of a batch: log-uniform quantiles between lo and hi, then `padded` rows without a sequence."""
    n, lo, hi = case["B"] - case["padded"], case["lo"] + 1, case["hi"] + 1
    return [int(round(lo * (hi / lo) ** ((j + 0.5) / n))) - 1 for j in range(n)] + [-1] * case["padded"]


def _visible(case):
    """Sum over the queries of one head of the tokens that each sees."""
    seen = 0
    for n in _lengths(case):
        if n >= 0:
            seen += sum(case["prefix"] + max(0, n - (case["n_q"] - 1 - i)) for i in range(case["n_q"]))
    return seen


def work(case):
    es, d = ES[case["dtype"]], case["d_c"] + case["d_r"]
    if case["op"] == "append":
        T, live = case["T"], case["T"] - case["padded"]
        rows = 2 * live * d * es + 2 * T * case["H"] * case["d_r"] * es + T * (case["d_r"] * 4 + 8)
        return {"bytes": rows, "flops": 4 * live * case["d_c"] + 3 * T * (case["H"] + 1) * case["d_r"]}
    rows = case["B"] * case["n_q"] * case["H"]
    tokens = case["prefix"] + sum(max(0, n) for n in _lengths(case))
    return {"bytes": tokens * d * es + rows * (d + case["d_c"]) * es + rows * 4,
            "flops": 2 * case["H"] * _visible(case) * (2 * case["d_c"] + case["d_r"])}


# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, d = DT[case["dtype"]], case["d_c"] + case["d_r"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    def pages_of(n_pages):
        # A page holds `page` rows; the pool's pages are a little larger, their ends unused.
        page_elems = case["page"] * d + 64
        pages = torch.empty(n_pages, page_elems, device="cuda", dtype=dt)
        for i in range(0, n_pages, 4096):
            pages[i:i + 4096] = torch.randn(pages[i:i + 4096].shape, generator=gen, device="cuda")
        return pages

    if case["op"] == "append":
        return _prepare_append(case, gen, normal, pages_of)
    B, n_q, H, page = case["B"], case["n_q"], case["H"], case["page"]
    order = torch.randperm(B, generator=gen, device="cuda").tolist()
    lens = [_lengths(case)[j] for j in order]
    most = max(1, max(lens))
    n_prefix, n_own = -(-case["prefix"] // page), [-(-max(0, n) // page) for n in lens]
    n_pages = n_prefix + sum(n_own) + 3
    ids = torch.randperm(n_pages, generator=gen, device="cuda").tolist()
    table, at = torch.full((B, -(-most // page)), -1, dtype=torch.int32), n_prefix
    for b, n in enumerate(n_own):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return {"case": case, "q": normal(B, n_q, H, case["d_c"]), "q_pe": normal(B, n_q, H, case["d_r"]), "pages": pages_of(n_pages),
            "table": table.cuda(), "lens": torch.tensor(lens, dtype=torch.int32).cuda(), "most": most,
            "prefix_pages": torch.tensor(ids[:n_prefix], dtype=torch.int32).cuda(), "scale": (128 + case["d_r"]) ** -0.5}


def _prepare_append(case, gen, normal, pages_of):
    T, d_c, d_r, page = case["T"], case["d_c"], case["d_r"], case["page"]
    n_pages = 2 * (-(-T // page)) + 1
    # Decode batches land on rows of pages all over the pool; a prompt fills pages one after another.
    if T <= 512:
        slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:T]
    else:
        ids = torch.randperm(n_pages, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = ids[t // page] * page + t % page
    slots[torch.randperm(T, generator=gen, device="cuda")[:case["padded"]]] = -1
    n_pos = 65536
    positions = torch.randint(0, n_pos, (T,), generator=gen, device="cuda") if T <= 512 else torch.arange(T, device="cuda")
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(d_r // 2, dtype=torch.float64, device="cuda") / (d_r // 2))
    fused = normal(T, d_c + d_r)              # one projection's output: c and k_pe are views of its rows
    queries = normal(T, case["H"], 128 + d_r)  # the queries' plain and rotated parts side by side
    return {"case": case, "pages": pages_of(n_pages), "slots": slots.to(torch.int32), "positions": positions.to(torch.int32),
            "rope": torch.cat([angle.cos(), angle.sin()], 1).float(), "c": fused[:, :d_c], "k_pe": fused[:, d_c:],
            "q_pe": queries[:, :, 128:], "norm_weight": (1 + 0.1 * normal(d_c)) if case["norm"] else None}


# ---------------------------------------------------------------------------
def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attend(state) if own else _plain_attend(state)


def _own_append(s):
    from kda_delta_rule_gb300 import kda as K
    q_pe = K.kda_mla_append(s["pages"].view(torch.uint8), s["case"]["page"], s["slots"], s["positions"], s["rope"], s["c"], s["k_pe"],
                            q_pe=s["q_pe"], norm_weight=s["norm_weight"],
                            style=K.ROPE_INTERLEAVED if s["case"]["interleaved"] else K.ROPE_HALF)
    return {"pages": s["pages"], "q_pe": q_pe}


def _own_attend(s):
    from kda_delta_rule_gb300 import kda as K
    o, lse = K.kda_mla_decode(s["q"], s["q_pe"], s["pages"].view(torch.uint8), s["case"]["page"], s["table"], s["lens"], s["scale"],
                              prefix_pages=s["prefix_pages"], prefix_len=s["case"]["prefix"])
    return {"o": o, "lse": lse}


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    case = s["case"]
    c, k_pe, q_pe = s["c"].float(), s["k_pe"].float(), s["q_pe"].float()
    if s["norm_weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + 1e-6) * s["norm_weight"].float()
    cos, sin = s["rope"][s["positions"].long()].chunk(2, -1)
    row = torch.cat([c, _rotate(k_pe, cos, sin, case["interleaved"])], -1).to(s["pages"].dtype)
    q_out = _rotate(q_pe, cos[:, None], sin[:, None], case["interleaved"]).to(s["pages"].dtype)
    rows = _rows(s["pages"], case)
    slots = s["slots"].long()
    live = slots >= 0
    rows[slots[live] // case["page"], slots[live] % case["page"]] = row[live]
    return {"pages": s["pages"], "q_pe": q_out}


def _rows(pages, case):
    """The rows of the pages, (n_pages, page, d_c + d_r), without the pages' ends."""
    d = case["d_c"] + case["d_r"]
    return pages.as_strided((pages.shape[0], case["page"], d), (pages.stride(0), d, 1))


def _plain_attend(s):
    case, B, n_q, H = s["case"], s["case"]["B"], s["case"]["n_q"], s["case"]["H"]
    d_c, P, most = case["d_c"], case["prefix"], s["most"]
    rows = _rows(s["pages"], case)
    q = torch.cat([s["q"], s["q_pe"]], -1).float() * s["scale"]
    keys = rows[s["table"].clamp(min=0).long()].flatten(1, 2)[:, :most].float()        # (B, most, d)
    scores = torch.bmm(q.flatten(1, 2), keys.transpose(1, 2)).view(B, n_q, H, most)
    end = s["lens"][:, None] - torch.arange(n_q - 1, -1, -1, device=q.device)             # (B, n_q) own tokens seen
    seen = torch.arange(most, device=q.device) < end[:, :, None, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if P:
        shared = rows[s["prefix_pages"].long()].flatten(0, 1)[:P].float()
        first = (q.flatten(0, 2) @ shared.T).view(B, n_q, H, P)
        first = first.masked_fill(s["lens"].view(B, 1, 1, 1) < 0, -math.inf)
        top = torch.maximum(top, first.amax(-1, keepdim=True))
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - base)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.flatten(1, 2), keys[..., :d_c]).view(B, n_q, H, d_c)
    if P:
        p = torch.exp(first - base)
        total = total + p.sum(-1, keepdim=True)
        o = o + (p.flatten(0, 2) @ shared[:, :d_c]).view(B, n_q, H, d_c)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"o": o.to(s["q"].dtype), "lse": (base + torch.log(total)).squeeze(-1)}


# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    case, d_c = s["case"], s["case"]["d_c"]
    T, half = case["T"], case["d_r"] // 2
    pages = s["pages"].double()
    turn = torch.complex(s["rope"][:, :half].double(), s["rope"][:, half:].double())[s["positions"].long()]   # (T, d_r / 2)

    def turned(x):                      # the pairs of the last axis as complex numbers, times the turn
        pairs = x.double().reshape(*x.shape[:-1], half, 2) if case["interleaved"] else x.double().reshape(
            *x.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.complex(pairs[..., 0], pairs[..., 1]) * turn.view(T, *[1] * (x.dim() - 2), half)
        z = torch.stack([z.real, z.imag], -1)
        return z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)

    row = s["c"].double()
    if s["norm_weight"] is not None:
        row = row / ((row * row).sum(-1, keepdim=True) / d_c + 1e-6).sqrt() * s["norm_weight"].double()
    row = torch.cat([row, turned(s["k_pe"])], -1)
    d = row.shape[-1]
    slots = s["slots"].long()
    at = torch.nonzero(slots >= 0)[:, 0]
    flat = (slots[at] // case["page"]) * pages.shape[1] + (slots[at] % case["page"]) * d
    pages.view(-1)[flat[:, None] + torch.arange(d, device=flat.device)] = row[at]
    return {"pages": pages, "q_pe": turned(s["q_pe"])}


def _exact_attend(s):
    case = s["case"]
    if work(case)["flops"] > 3e12:
        return None
    d_c, d, page, n_q, H = case["d_c"], case["d_c"] + case["d_r"], case["page"], case["n_q"], case["H"]
    q = torch.cat([s["q"].double(), s["q_pe"].double()], -1) * s["scale"]
    o = torch.zeros(*q.shape[:3], d_c, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)

    def tokens(ids, n):
        return s["pages"][ids.long(), :page * d].reshape(-1, d)[:n].double()

    shared = tokens(s["prefix_pages"], case["prefix"])
    for b, n in enumerate(s["lens"].tolist()):
        if n < 0:
            continue
        keys = torch.cat([shared, tokens(s["table"][b, :-(-n // page)], n)])
        for i in range(n_q):
            k = keys[:case["prefix"] + max(0, n - (n_q - 1 - i))]
            if len(k):
                x = q[b, i] @ k.T
                lse[b, i] = torch.logsumexp(x, -1)
                o[b, i] = torch.softmax(x, -1) @ k[:, :d_c]
    return {"o": o, "lse": lse}
