"""Linear attention with one decay for each head on the GPU, against the fp64 oracle.

Bounds.  u = 2^-24 is fp32's rounding, 2^-8 bf16's.  A is what an output's terms come to by their size, from the oracle's run on
absolute values; n the number of terms.
fp32, and the states of every path but the tensor cores': each of n = T + dk additions rounds once, n u A; the factors of a decay
are powers within 2 ulp of batches of 16 tokens, one more u A each: together 2 n u A.
bf16 outputs of steps: the same, and one rounding, 2^-8 |o|.
bf16 prompts on the tensor cores, in chunks of 128 tokens: P = (q k^T) decay is rounded to bf16 for the product with v, 2^-8 of
sum |P| |v|, and the chunk's start state S for the product with q, 2^-8 of e^b sum |q| |S|; the decays are differences of
sums of up to 32 tokens that are at most 2^13 in size (a decay counts at most 2^8), off by 2^-11 each at worst: 2^-10 of
sum |P| |v|.  Their states take keys times decays as three bf16 numbers, which leave 2^-24, and are within 3 2^-16 A besides n u A
(what two numbers would have left) with room; the long memory's test holds them closer.
"""
import math

import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from oracle import kda_oracle as O

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import kda
    kda.kda_device_errors()
    return kda


def _rows(T, H, H_k, dk, dv, dtype, gen, fixed=False, rate=0.05, extra=24):
    """q, k, v as views of one wider projection whose other values, and rows behind the last, are NaN; log decays likewise."""
    w = 2 * H_k * dk + H * dv
    fused = torch.full((T + 150, w + extra), math.nan, dtype=dtype)
    fused[:T, 8:8 + w] = torch.randn(T, w, generator=gen).to(dtype)
    fused = fused.cuda()
    q, k, v = fused[:T, 8:8 + w].split([H_k * dk, H_k * dk, H * dv], 1)
    if fixed:
        g = (-rate * (0.1 + torch.rand(H, generator=gen))).cuda()
    else:
        wide = torch.full((T + 150, H + 3), math.nan)
        wide[:T, 1:1 + H] = -rate * torch.empty(T, H).exponential_(generator=gen)
        g = wide.cuda()[:T, 1:1 + H]
    return q.view(T, H_k, dk), k.view(T, H_k, dk), v.view(T, H, dv), g


def _chunk_sizes(q, k, v, g, states, scale, chunk=128):
    """Per output sum |P| |v| + e^b sum |q| |S| and the first part of it, with S the states at the chunks' starts."""
    T, H = v.shape[:2]
    share = H // q.shape[1]
    g = np.broadcast_to(g, (T, H))
    all_, p_only = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(0, T, chunk):
        n = min(chunk, T - t)
        b = np.cumsum(np.maximum(g[t:t + n], -200.0), 0)
        for h in range(H):
            qq, kk = q[t:t + n, h // share], k[t:t + n, h // share]
            w = np.tril(np.exp(np.tril(b[:, None, h] - b[None, :, h])))
            p = np.abs(scale) * np.abs((qq @ kk.T) * w) @ np.abs(v[t:t + n, h])
            p_only[t:t + n, h] = p
            all_[t:t + n, h] = p + np.abs(scale) * np.exp(b[:, h])[:, None] * (np.abs(qq) @ np.abs(states[t][h]))
    return all_, p_only


def _check_prompt(o, S, S0, q, k, v, g, scale, dtype):
    """One sequence's outputs and final state; returns the oracle's states and their bounds."""
    T, dk = len(v), q.shape[2]
    ro, states = O.linattn_recurrent(S0, q, k, v, g, scale)
    bo, bs = O.linattn_recurrent(S0, q, k, v, g, scale, bound=True)
    n = 2 * (T + dk)
    s_tol = n * U + (3 * 2.0 ** -16 if dtype == BF16 else 0)
    assert np.all(np.abs(f64(S) - states[-1]) <= s_tol * bs[-1] + 1e-30)
    if T:
        tol = n * U * bo
        if dtype == BF16:
            sizes, p_only = _chunk_sizes(q, k, v, g, states, scale)
            tol += 2.0 ** -8 * (np.abs(ro) + sizes) + 2.0 ** -10 * p_only
        assert np.all(np.abs(f64(o) - ro) <= tol + 1e-30)
    return states, bs, s_tol


PROMPTS = [
    # lens, H, H_k, dk, dv, stride, resume, fixed, rate
    ([1], 1, 1, 128, 128, 0, True, False, 0.05),
    ([127, 128, 129], 2, 2, 128, 128, 128, True, False, 0.05),
    ([0, 5, 0, 130, 1], 3, 1, 64, 64, 128, True, False, 0.05),
    ([300, 257], 4, 2, 128, 64, 256, False, False, 0.01),
    ([515], 2, 1, 64, 128, 0, False, True, 0.002),
    ([33, 390], 3, 3, 32, 32, 128, True, False, 0.2),
    ([200], 5, 5, 32, 128, 0, True, True, 0.05),
    ([260, 17], 2, 2, 128, 32, 0, False, False, 3.0),           # decays of whole magnitudes per token
    ([140], 6, 2, 64, 32, 128, True, False, 1e-5),               # states that hardly decay
    ([129], 1, 1, 32, 64, 0, True, False, 60.0),                 # nothing but the last tokens
    ([2100, 40], 1, 1, 128, 128, 384, True, False, 0.003),       # few heads: split into segments
    ([1030, 1601], 2, 1, 64, 64, 512, False, False, 0.01),
    ([1500], 1, 1, 32, 32, 0, True, True, 0.004),
    ([1800], 1, 1, 128, 64, 128, True, False, 0.3),
    # bf16: the longer ones on the tensor cores, the others beside them on the CUDA cores, with lengths on both sides of the choice
    ([24, 300, 25, 0, 23, 1, 130], 3, 1, 128, 128, 128, True, False, 0.05),
    ([97, 98, 400, 96, 1], 2, 2, 64, 64, 128, True, False, 0.05),
    ([128, 127, 129, 256, 3], 2, 1, 32, 32, 128, False, False, 0.05),
    ([1300, 48, 49, 9], 1, 1, 64, 128, 128, True, True, 0.01),
    # fewer rows than a tile has
    ([25], 1, 1, 128, 128, 0, True, False, 0.05),
    ([100], 3, 1, 128, 64, 0, False, True, 0.02),
    ([127], 2, 2, 64, 128, 0, True, False, 0.1),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,H,H_k,dk,dv,stride,resume,fixed,rate", PROMPTS)
def test_prefill_matches_oracle(K, lens, H, H_k, dk, dv, stride, resume, fixed, rate, dtype):
    gen = torch.Generator().manual_seed(sum(lens) + H)
    T, N = sum(lens), len(lens)
    q, k, v, g = _rows(T, H, H_k, dk, dv, dtype, gen, fixed, rate)
    cu = np.cumsum([0] + lens).tolist()
    S0 = torch.randn(N, H, dk, dv, generator=gen) if resume else None
    n_ck = sum(n // stride for n in lens) if stride else 0
    pages = torch.full((n_ck + 2, H * dk * dv + 12), 7.0, device="cuda")
    ids = torch.randperm(n_ck + 2, generator=gen)[:n_ck].to(torch.int32)
    pos = torch.full((n_ck,), -1, dtype=torch.int32, device="cuda")
    kw = dict(ckpt_stride=stride, page_pool=pages.view(torch.uint8), ckpt_page_ids=ids.cuda(), ckpt_pos=pos) if n_ck else {}
    scale = dk ** -0.5
    o, S = K.kda_linattn_prefill(None if S0 is None else S0.cuda(), q, k, v, g, cu_seqlens=cu, scale=scale, **kw)
    assert K.kda_device_errors() == 0
    c, at = 0, []
    for j in range(N):
        a, b = cu[j], cu[j + 1]
        start = f64(S0[j]) if resume else np.zeros((H, dk, dv))
        gg = f64(g) if fixed else f64(g[a:b])
        states, bs, tol = _check_prompt(o[a:b], S[j], start, f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), gg, scale, dtype)
        for t in range(stride, lens[j] + 1, stride) if stride else ():
            page = f64(pages[int(ids[c])])
            assert np.all(np.abs(page[:-12].reshape(H, dk, dv) - states[t]) <= tol * bs[t]) and np.all(page[-12:] == 0)
            at.append(t)
            c += 1
    assert pos.tolist() == at
    free = sorted(set(range(n_ck + 2)) - set(ids.tolist()))
    assert torch.all(pages[free] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_without_workspace_does_not_split(K, dtype):
    gen = torch.Generator().manual_seed(3)
    q, k, v, g = _rows(1400, 1, 1, 64, 64, dtype, gen, rate=0.01)
    assert K.kda_linattn_prefill_workspace_bytes(None, 1400, 1, 64, 64, dtype) > 0
    o, S = K.kda_linattn_prefill(None, q, k, v, g, workspace=None)
    _check_prompt(o, S[0], np.zeros((1, 64, 64)), f64(q), f64(k), f64(v), f64(g), 1.0, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,H", [([150, 200, 90], 2), ([1300, 70, 1300], 1)])
def test_a_sequence_of_nans_stays_by_itself(K, lens, H, dtype):
    """Tiles at a sequence's end hold the next one's rows."""
    gen = torch.Generator().manual_seed(4)
    T = sum(lens)
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, g = (x.clone() for x in _rows(T, H, H, 128, 128, dtype, gen))
    bad = slice(cu[1], cu[2])
    good_o, good_S = K.kda_linattn_prefill(None, q, k, v, g, cu_seqlens=cu)
    q[bad], k[bad], v[bad] = math.nan, math.inf, math.nan
    o, S = K.kda_linattn_prefill(None, q, k, v, g, cu_seqlens=cu)
    for j, rows in ((0, slice(0, cu[1])), (2, slice(cu[2], T))):
        assert torch.equal(o[rows], good_o[rows]) and torch.equal(S[j], good_S[j])
    assert torch.isnan(o[bad]).all() and torch.isnan(S[1]).all()


@pytest.mark.parametrize("T,H", [(500, 3), (1700, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_are_not_finite_leave_earlier_tokens(K, dtype, T, H):
    """bf16: those before the chunk of 128 that they lie in; fp32: all before them. Other heads and columns of v as well."""
    gen = torch.Generator().manual_seed(15)
    q, k, v, g = (x.clone() for x in _rows(T, H, H, 64, 64, dtype, gen))
    good_o, good_S = K.kda_linattn_prefill(None, q, k, v, g)
    v[300, 0, 7] = math.nan
    v[301, 0, 9] = math.inf
    o, S = K.kda_linattn_prefill(None, q, k, v, g)
    before = 256 if dtype == BF16 else 300
    assert torch.equal(o[:before], good_o[:before]) and torch.equal(o[:, 1:], good_o[:, 1:]) and torch.equal(S[:, 1:], good_S[:, 1:])
    rest = [c for c in range(64) if c not in (7, 9)]
    assert torch.equal(o[:, 0, rest], good_o[:, 0, rest]) and torch.equal(S[0, 0][:, rest], good_S[0, 0][:, rest])
    assert torch.isnan(o[300:, 0, 7]).all() and torch.isnan(S[0, 0, :, 7]).all() and not torch.isfinite(S[0, 0, :, 9]).any()


@pytest.mark.parametrize("B,steps", [(3, 1), (40, 4)])
def test_a_slot_read_by_several_rows(K, B, steps):
    """Drafts of one state, outputs alone or with their states going elsewhere."""
    gen = torch.Generator().manual_seed(16)
    q, k, v, g = (x.unflatten(0, (steps, B)) for x in _rows(steps * B, 2, 1, 64, 64, BF16, gen))
    S = torch.randn(B + 2, 2, 64, 64, generator=gen).cuda()
    old, ids = S.clone(), torch.full((B,), B, dtype=torch.int32, device="cuda")
    o = K.kda_linattn_step(S, q, k, v, g, slot_in=ids, write_state=False)
    many = old[B].expand(B, -1, -1, -1).contiguous()
    assert torch.equal(o, K.kda_linattn_step(many, q, k, v, g)) and torch.equal(S, old)
    o2 = K.kda_linattn_step(S, q, k, v, g, slot_in=ids, slot_out=torch.arange(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(o2, o) and torch.equal(S[:B], many) and torch.equal(S[B:], old[B:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(400, 3), (1700, 1)])
def test_decays_to_zero_forget_everything(K, T, H, dtype):
    """-infinity at a token: what lies before it is gone, and the decays of its neighbours keep their precision."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, g = (x.clone() for x in _rows(T, H, H, 64, 64, dtype, gen))
    cuts = [0, 1, 2, 131, 132, 250, 255, 256, 390]
    g[cuts] = -math.inf
    S0 = torch.randn(1, H, 64, 64, generator=gen)
    o, S = K.kda_linattn_prefill(S0.cuda(), q, k, v, g)
    _check_prompt(o, S[0], f64(S0[0]), f64(q), f64(k), f64(v), f64(g), 1.0, dtype)
    assert K.kda_device_errors() == 0
    # the same as sequences of their own from the cuts on
    o2, S2 = K.kda_linattn_prefill(None, q[390:], k[390:], v[390:], g[390:])
    _check_prompt(o[390:], S[0], np.zeros((H, 64, 64)), f64(q[390:]), f64(k[390:]), f64(v[390:]), f64(g[390:]), 1.0, dtype)
    _check_prompt(o2, S2[0], np.zeros((H, 64, 64)), f64(q[390:]), f64(k[390:]), f64(v[390:]), f64(g[390:]), 1.0, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_memory_keeps_its_precision(K, dtype):
    """A fixed decay that forgets over 8000 tokens: the factor's rounding, always the same, must not add up. 12000 tokens, against a
    cumulative form in fp64 on the GPU; bounds as above with the 12000 / 16 factors of the batches."""
    T, H, d = 12000, 2, 64
    gen = torch.Generator().manual_seed(6)
    q, k, v, _ = _rows(T, H, H, d, d, dtype, gen)
    g = torch.tensor([-1 / 8000, -1 / 3000], device="cuda")
    o, S = K.kda_linattn_prefill(None, q, k, v, g)
    w = torch.exp(g.double()[:, None] * torch.arange(T - 1, -1, -1, device="cuda"))           # (H, T)
    kd, vd = k.double().transpose(0, 1) * w[..., None], v.double().transpose(0, 1)
    ref, size = kd.transpose(1, 2) @ vd, kd.abs().transpose(1, 2) @ vd.abs()
    assert torch.all((S[0].double() - ref).abs() <= (3 * 2.0 ** -16 * (dtype == BF16) + 2 * T / 16 * U) * size)
    # random errors, not a drift: the whole state is within fp32's range of the exact one
    assert float((S[0].double() - ref).norm() / ref.norm()) < (1e-5 if dtype == BF16 else 2e-6)


@pytest.mark.parametrize("g", [0.5, math.nan])
def test_decays_out_of_range_are_flagged(K, g):
    x = torch.randn(200, 2, 64, device="cuda").bfloat16()
    decays = torch.full((200, 2), -0.1, device="cuda")
    K.kda_device_errors()
    K.kda_linattn_prefill(None, x, x, x, decays)
    assert K.kda_device_errors() == 0
    decays[77, 1] = g
    K.kda_linattn_prefill(None, x, x, x, decays)
    assert K.kda_device_errors() == K.DEVERR_GATE
    K.kda_linattn_prefill(None, x.float(), x.float(), x.float(), decays)
    assert K.kda_device_errors() == K.DEVERR_GATE
    K.kda_linattn_step(torch.zeros(200, 2, 64, 64, device="cuda"), x, x, x, decays)
    assert K.kda_device_errors() == K.DEVERR_GATE


def test_no_tokens_leave_the_states(K):
    S0 = torch.randn(3, 2, 64, 32, device="cuda")
    empty = torch.empty(0, 2, 64, device="cuda", dtype=BF16)
    for dtype in (BF16, F32):
        e, ev = empty.to(dtype), torch.empty(0, 2, 32, device="cuda", dtype=dtype)
        o, S = K.kda_linattn_prefill(S0, e, e, ev, torch.empty(0, 2, device="cuda"), cu_seqlens=[0, 0, 0, 0])
        assert o.shape == (0, 2, 32) and torch.equal(S, S0)
        _, S = K.kda_linattn_prefill(None, e, e, ev, torch.empty(0, 2, device="cuda"), cu_seqlens=[0, 0])
        assert torch.all(S == 0)


def test_more_sequences_than_one_launch_takes(K):
    gen = torch.Generator().manual_seed(7)
    lens = [j % 4 for j in range(1500)] + [200]
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, g = _rows(cu[-1], 1, 1, 32, 32, BF16, gen)
    pages = torch.zeros(1, 32 * 32, device="cuda")
    o, S = K.kda_linattn_prefill(None, q, k, v, g, cu_seqlens=cu, ckpt_stride=128, page_pool=pages.view(torch.uint8),
                                 ckpt_page_ids=torch.zeros(1, dtype=torch.int32, device="cuda"))
    zero = np.zeros((1, 32, 32))
    for j in (0, 1, 3, 1022, 1023, 1025, 1027, 1499, 1500):
        a, b = cu[j], cu[j + 1]
        states, bs, tol = _check_prompt(o[a:b], S[j], zero, f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), f64(g[a:b]), 1.0, BF16)
    assert np.all(np.abs(f64(pages[0]).reshape(1, 32, 32) - states[128]) <= tol * bs[128])


# ---------------------------------------------------------------------------
STEPS = [
    # B, steps, H, H_k, dk, dv, slots, fixed, rate
    (1, 1, 1, 1, 32, 32, False, False, 0.05),
    (1, 1, 32, 32, 128, 128, False, False, 0.05),
    (3, 1, 4, 2, 64, 128, True, True, 0.5),
    (5, 4, 6, 3, 128, 32, True, False, 0.05),
    (2, 16, 3, 1, 128, 128, False, False, 2.0),
    (9, 7, 8, 8, 32, 64, True, False, 0.01),
    (70, 2, 32, 4, 64, 64, True, False, 0.05),                  # wide slices
    (40, 1, 16, 16, 128, 128, True, False, 0.05),
    (40, 3, 16, 8, 32, 128, False, False, 40.0),
    (300, 1, 8, 8, 32, 32, True, True, 0.05),
]


def _check_step(o, S_new, S_old, rows, ids, out_ids, n, scale, dtype):
    """Live rows against the oracle; returns the slots that were written."""
    q, k, v, g = (f64(x) for x in rows)
    steps, B, H, dv = v.shape
    written = []
    for b in range(B):
        if ids[b] < 0 or ids[b] >= len(S_old):
            assert np.all(f64(o[:, b]) == 0)
            continue
        m = n[b]
        gb = g if g.ndim == 1 else g[:m, b]
        S0 = f64(S_old[ids[b]])
        ro, states = O.linattn_recurrent(S0, q[:m, b], k[:m, b], v[:m, b], gb, scale)
        bo, bs = O.linattn_recurrent(S0, q[:m, b], k[:m, b], v[:m, b], gb, scale, bound=True)
        tol = 2 * (m + q.shape[-1]) * U
        assert np.all(np.abs(f64(o[:m, b]) - ro) <= tol * bo + (2.0 ** -8 * np.abs(ro) if dtype == BF16 else 0) + 1e-30)
        assert np.all(f64(o[m:, b]) == 0)
        if S_new is not None:
            assert np.all(np.abs(f64(S_new[out_ids[b]]) - states[-1]) <= tol * bs[-1] + 1e-30)
            written.append(out_ids[b])
    return written


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,steps,H,H_k,dk,dv,slots,fixed,rate", STEPS)
def test_step_matches_oracle(K, B, steps, H, H_k, dk, dv, slots, fixed, rate, dtype):
    gen = torch.Generator().manual_seed(B + steps)
    q, k, v, g = _rows(steps * B, H, H_k, dk, dv, dtype, gen, fixed, rate)
    q, k, v = (x.unflatten(0, (steps, B)) for x in (q, k, v))
    g = g if fixed else g.unflatten(0, (steps, B))
    n_slots = 2 * B + 3 if slots else B
    S = torch.randn(n_slots, H, dk, dv, generator=gen).cuda()
    perm = torch.randperm(n_slots, generator=gen).tolist()
    ids = perm[:B] if slots else list(range(B))
    if slots:
        ids[B // 2] = -1
        if B > 2:
            ids[0] = n_slots                                      # as good as none
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, scale, full = (q, k, v, g), dk ** -0.5, [steps] * B
    old = S.clone()
    kw = dict(scale=scale, slot_in=i32(ids) if slots else None)
    # outputs alone: the states stay as they are
    o = K.kda_linattn_step(S, q, k, v, g, write_state=False, **kw)
    assert torch.equal(S, old)
    _check_step(o, None, old, rows, ids, None, full, scale, dtype)
    # some of the tokens, to other slots or another array
    n = [(3 * b + 1) % (steps + 1) for b in range(B)]
    if slots:
        out = perm[B:2 * B]
        o2 = K.kda_linattn_step(S, q, k, v, g, slot_out=i32(out), n_accepted=i32(n), **kw)
        written = _check_step(o2, S, old, rows, ids, out, n, scale, dtype)
        rest = sorted(set(range(n_slots)) - set(written))
        assert torch.equal(S[rest], old[rest])
        S.copy_(old)
    else:
        S_new = torch.full_like(S, 5.0)
        o2 = K.kda_linattn_step(S, q, k, v, g, S_new=S_new, n_accepted=i32(n), **kw)
        _check_step(o2, S_new, old, rows, ids, ids, n, scale, dtype)
        assert torch.equal(S, old)
    # in place
    o3 = K.kda_linattn_step(S, q, k, v, g, **kw)
    assert torch.equal(o3, o)
    written = _check_step(o3, S, old, rows, ids, ids, full, scale, dtype)
    rest = sorted(set(range(n_slots)) - set(written))
    assert torch.equal(S[rest], old[rest])
    assert K.kda_device_errors() == 0


def test_step_takes_one_token_without_a_steps_axis(K):
    gen = torch.Generator().manual_seed(1)
    q, k, v, g = _rows(4, 3, 1, 64, 64, BF16, gen)
    S = torch.randn(4, 3, 64, 64, generator=gen).cuda()
    S2 = S.clone()
    o = K.kda_linattn_step(S, q, k, v, g)
    o2 = K.kda_linattn_step(S2, q[None], k[None], v[None], g[None])
    assert o.shape == (4, 3, 64) and torch.equal(o, o2[0]) and torch.equal(S, S2)


def test_accepted_counts_are_clamped(K):
    gen = torch.Generator().manual_seed(2)
    q, k, v, g = (x.unflatten(0, (3, 2)) for x in _rows(6, 2, 2, 32, 32, F32, gen))
    S = torch.randn(2, 2, 32, 32, generator=gen).cuda()
    a, b = torch.empty_like(S), torch.empty_like(S)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o1 = K.kda_linattn_step(S, q, k, v, g, S_new=a, n_accepted=i32([-4, 99]))
    o2 = K.kda_linattn_step(S, q, k, v, g, S_new=b, n_accepted=i32([0, 3]))
    assert torch.equal(o1, o2) and torch.equal(a, b) and torch.equal(a[0], S[0])


def test_binding_refuses_rows_it_cannot_pass(K):
    x = torch.randn(4, 6, 64, device="cuda")
    g, S = -torch.rand(4, 3, device="cuda"), torch.zeros(4, 3, 64, 64, device="cuda")
    with pytest.raises(ValueError, match="heads must be dense"):
        K.kda_linattn_step(S, x[:, ::2], x[:, ::2], x[:, ::2], g)
    v = torch.randn(2, 4, 3, 64, device="cuda")[:, :3]          # three rows, a gap, three rows
    with pytest.raises(ValueError, match="evenly spaced"):
        K.kda_linattn_step(S[:3], v, v, v, torch.zeros(3, device="cuda"))
    y = x[:, :3].contiguous()
    with pytest.raises(ValueError, match="overlap"):
        K.kda_linattn_step(S, y, y, y, g[:1].expand(4, 3))
    with pytest.raises(K.KdaError):
        K.kda_linattn_step(torch.zeros(4, 3, 48, 64, device="cuda"), y[..., :48].contiguous(), y[..., :48].contiguous(), y, g)


# ---------------------------------------------------------------------------
def test_prompt_then_tokens_is_one_recurrence(K):
    """A prompt in two calls, a step of drafted tokens of which some are accepted, single steps: states handed on throughout."""
    gen = torch.Generator().manual_seed(8)
    T, H, H_k, dk, dv, scale = 600, 4, 2, 64, 128, 0.125
    q, k, v, g = _rows(T, H, H_k, dk, dv, BF16, gen, rate=0.02)
    f = [f64(x) for x in (q, k, v, g)]
    ro, states = O.linattn_recurrent(np.zeros((H, dk, dv)), *f, scale)
    _, bs = O.linattn_recurrent(np.zeros((H, dk, dv)), *f, scale, bound=True)
    tol = 3 * 2.0 ** -16 + 2 * (T + dk) * U
    _, S = K.kda_linattn_prefill(None, q[:333], k[:333], v[:333], g[:333], scale=scale)
    _, S = K.kda_linattn_prefill(S, q[333:580], k[333:580], v[333:580], g[333:580], scale=scale)
    assert np.all(np.abs(f64(S[0]) - states[580]) <= tol * bs[580])
    draft = [x[580:588, None] for x in (q, k, v, g)]
    checked = K.kda_linattn_step(S, *draft, scale=scale, write_state=False)
    kept = K.kda_linattn_step(S, *draft, scale=scale, n_accepted=torch.tensor([5], dtype=torch.int32, device="cuda"))
    assert torch.equal(kept[:5], checked[:5]) and torch.all(kept[5:] == 0)
    for t in range(585, T):
        o = K.kda_linattn_step(S, q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], scale=scale)
        size = scale * np.einsum("hi,hij->hj", np.repeat(np.abs(f[0][t]), 2, 0), bs[t + 1])
        assert np.all(np.abs(f64(o[0]) - ro[t]) <= 2.0 ** -8 * np.abs(ro[t]) + tol * size)
    assert np.all(np.abs(f64(S[0]) - states[T]) <= tol * bs[T])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_calls_and_other_streams(K, dtype):
    """Two graphs that share a workspace, replayed in turn on new inputs, and calls on a stream of their own, all bit-equal to eager calls."""
    gen = torch.Generator().manual_seed(9)
    sets = []
    for T in (1500, 1700):
        q, k, v, g = (x.clone() for x in _rows(T, 1, 1, 64, 64, dtype, gen))
        sets.append((q, k, v, g, torch.randn(1, 1, 64, 64, generator=gen).cuda()))
    need = max(K.kda_linattn_prefill_workspace_bytes(None, len(s[0]), 1, 64, 64, dtype) for s in sets)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(s, stream=None):
        q, k, v, g, S0 = s
        o, S = K.kda_linattn_prefill(S0, q, k, v, g, workspace=ws, stream=stream)
        o2 = K.kda_linattn_step(S, q[:1], k[:1], v[:1], g[:1], stream=stream)
        return o, S, o2

    graphs = []
    for s in sets:
        call(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(s)
        graphs.append((graph, out))
    for turn in range(3):
        for s, (graph, out) in zip(sets, graphs):
            s[2].copy_(torch.randn(s[2].shape, generator=gen).to(dtype))
            graph.replay()
        torch.cuda.synchronize()
        for s, (graph, out) in zip(sets, graphs):
            for a, b in zip(out, call(s)):
                assert torch.equal(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in sets:
        ref = call(s)
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream):
            out = call(s, stream)
            side.synchronize()
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_captured_calls_of_short_and_long_sequences(K):
    """Two prompt kernels side by side, and a step that reads their states, replayed on new inputs."""
    gen = torch.Generator().manual_seed(11)
    lens = [1200, 20, 24, 25, 5, 300]
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, g = (x.clone() for x in _rows(cu[-1], 2, 1, 128, 128, BF16, gen))
    S0 = torch.randn(len(lens), 2, 128, 128, generator=gen).cuda()
    S = torch.empty_like(S0)
    ws = torch.empty(max(K.kda_linattn_prefill_workspace_bytes(cu, cu[-1], 2, 128, 128, BF16), 1), dtype=torch.uint8, device="cuda")

    def call():
        o, _ = K.kda_linattn_prefill(S0, q, k, v, g, cu_seqlens=cu, S_final=S, workspace=ws)
        return o, K.kda_linattn_step(S, q[:6], k[:6], v[:6], g[:6])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for turn in range(3):
        v.copy_(torch.randn(v.shape, generator=gen).to(BF16))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*out, S)]
        for a, b in zip(got, (*call(), S)):
            assert torch.equal(a, b)
        for j, n in enumerate(lens):
            a = cu[j]
            f = [np.concatenate([f64(x[a:a + n]), f64(x[j:j + 1])]) for x in (q, k, v, g)]
            ro, states = O.linattn_recurrent(f64(S0[j]), *f, 1.0)
            bo, bs = O.linattn_recurrent(f64(S0[j]), *f, 1.0, bound=True)
            tol = 2 * (n + 1 + 128) * U + 3 * 2.0 ** -16
            assert np.all(np.abs(f64(S[j]) - states[-1]) <= tol * bs[-1])
            assert np.all(np.abs(f64(got[1][j]) - ro[-1]) <= 2.0 ** -8 * np.abs(ro[-1]) + tol * bo[-1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_calls_at_once(K, dtype):
    """On two streams, each with a workspace of its own: prompts in segments, many heads, steps."""
    gen = torch.Generator().manual_seed(12)
    a = [x.clone() for x in _rows(2500, 2, 1, 128, 64, dtype, gen)]
    b = [x.clone() for x in _rows(700, 40, 40, 64, 64, dtype, gen)]
    torch.cuda.synchronize()

    def work(x, stream):
        with torch.cuda.stream(stream):
            o, S = K.kda_linattn_prefill(None, *x)
            S2 = S.clone()
            return o, S, K.kda_linattn_step(S2, *(t[:1] for t in x)), S2

    main = torch.cuda.current_stream()
    ref = [[t.clone() for t in work(x, main)] for x in (a, b)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    out = [(i % 2, work((a, b)[i % 2], streams[i % 2])) for i in range(12)]
    torch.cuda.synchronize()
    for i, ts in out:
        for x, y in zip(ts, ref[i]):
            assert torch.equal(x, y)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_two_bindings_agree(K, dtype, monkeypatch):
    if K._native is None:
        pytest.skip("the native module is not built")
    gen = torch.Generator().manual_seed(13)
    q, k, v, g = _rows(1500, 2, 1, 64, 32, dtype, gen)
    steps = [x[:12].unflatten(0, (3, 4)) for x in (q, k, v, g)]
    S = torch.randn(9, 2, 64, 32, generator=gen).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, out, n = i32([3, -1, 5, 0]), i32([1, 2, 7, 8]), i32([3, 1, 0, 2])
    pages = torch.zeros(13, 2 * 64 * 32 * 4, dtype=torch.uint8, device="cuda")

    def calls():
        S1, S2, pos = S.clone(), torch.zeros_like(S), i32([-1] * 11)
        pages.zero_()
        r = [K.kda_linattn_step(S1, *steps, scale=0.5, slot_in=ids, slot_out=out, n_accepted=n), S1,
             K.kda_linattn_step(S, *steps, S_new=S2, slot_in=ids, slot_out=out), S2, K.kda_linattn_step(S, *steps, write_state=False, slot_in=ids),
             *K.kda_linattn_prefill(S[:3], q, k, v, g, cu_seqlens=[0, 700, 700, 1500], scale=0.5, ckpt_stride=128, page_pool=pages,
                                    ckpt_page_ids=i32(list(range(12, 1, -1))), ckpt_pos=pos), pos, pages.clone()]
        for bad in (lambda: K.kda_linattn_step(S, q[:4], k[:4], v[:4], g[0, 0]), lambda: K.kda_linattn_step(S, q[:4], k[:3], v[:4], g[:4]),
                    lambda: K.kda_linattn_prefill(S[:2], q, k, v, g), lambda: K.kda_linattn_prefill(None, q, k, v.float() if dtype == BF16 else v.bfloat16(), g)):
            with pytest.raises((TypeError, ValueError, K.KdaError)):
                bad()
        return r

    a = calls()
    monkeypatch.setattr(K, "_native", None)
    for x, y in zip(a, calls()):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(K):
    """Slots and rows that lie more than 2^32 elements behind the first, against the same values side by side."""
    gen = torch.Generator().manual_seed(14)
    H, d = 32, 128
    n_slots = (1 << 32) // (H * d * d) + 8
    S = torch.empty(n_slots, H, d, d, device="cuda")
    ids = [n_slots - 1, 0, n_slots - 3]
    q, k, v, g = _rows(3, H, H, d, d, BF16, gen)
    small = torch.randn(3, H, d, d, generator=gen).cuda()
    S[ids] = small
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o = K.kda_linattn_step(S, q, k, v, g, slot_in=i32(ids), slot_out=i32([n_slots - 2, 1, n_slots - 4]))
    assert torch.equal(S[ids], small)
    assert torch.equal(o, K.kda_linattn_step(small, q, k, v, g)) and torch.equal(S[[n_slots - 2, 1, n_slots - 4]], small)
    del S
    stride = 1 << 24
    for dtype, dk in ((BF16, 128), (BF16, 32), (F32, 64)):
        for T in (300, 270):
            dense = [x.contiguous() for x in _rows(T, 2, 2, dk, dk, dtype, gen)]
            wide = torch.empty(T, stride, dtype=dtype, device="cuda")
            rows = []
            for i, x in enumerate(dense[:3]):
                at = i * (1 << 20)
                wide[:, at:at + 2 * dk] = x.reshape(T, -1)
                rows.append(wide[:, at:at + 2 * dk].unflatten(1, (2, dk)))
            cu = None if T == 300 else [0, 150, 160, 270]
            for x, y in zip(K.kda_linattn_prefill(None, *rows, dense[3], cu_seqlens=cu), K.kda_linattn_prefill(None, *dense, cu_seqlens=cu)):
                assert torch.equal(x, y)
            del wide, rows


def test_same_call_twice_gives_the_same_bits(K):
    gen = torch.Generator().manual_seed(10)
    q, k, v, g = _rows(3000, 2, 2, 128, 128, BF16, gen)
    a, b = (K.kda_linattn_prefill(None, q, k, v, g) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
