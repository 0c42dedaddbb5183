"""The latent page cache's kernels one by one: shapes that select each of them, on data that reaches their rarer paths."""
import numpy as np
import pytest
import torch

from parity import TOL_F32
from test_gpu_mla import BF16, F32, LSE_TOL, _append_case, _case, _reference, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import kda
    kda.kda_device_errors()
    return kda


@pytest.mark.parametrize("through_ctypes", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 1), (1, 1)])
def test_append_rotates_in_place(K, T, H, dtype, through_ctypes):
    """The decode step of one sequence, and single heads: the stride of an axis of one entry has no say."""
    pages, slots, pos, table, fused, qs, w = _append_case(T, H, 128, 64, dtype, T + H, 2, 16)
    page = np.int64(16) if through_ctypes else 16
    args = (page, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :128], fused.cuda()[:, 128:])
    q = qs[:, :, 128:].contiguous().cuda()
    a, b = pages.cuda(), pages.cuda()
    out = K.kda_mla_append(a.view(torch.uint8), *args, q_pe=q)
    assert K.kda_mla_append(b.view(torch.uint8), *args, q_pe=q, q_pe_out=q) is q
    assert torch.equal(out, q) and torch.equal(a, b)
    assert K.kda_device_errors() == 0


# B, n_q, H, d_c, d_r, page, prefix, lens (range): what mla_parts makes of them
VARIANTS = {
    "16 rows": (24, 1, 16, 512, 64, 64, 0, (3000, 6000)),
    "32 rows": (60, 1, 20, 256, 32, 48, 0, (2000, 4000)),
    "64 rows": (40, 1, 64, 384, 48, 512, 0, (1000, 3000)),
    "64 rows, prefix and own tokens": (20, 1, 32, 512, 64, 64, 3000, (0, 2500)),
    "pair": (40, 3, 40, 512, 64, 64, 0, (1000, 3000)),
    "pair, d_c 128": (60, 8, 16, 128, 16, 16, 0, (1000, 4000)),
    "pair, d_c 384": (24, 2, 64, 384, 0, 80, 0, (500, 5000)),
    "pair, joint items": (24, 8, 32, 512, 64, 48, 2100, (0, 1500)),
    "pair, joint items, d_c 256": (16, 1, 128, 256, 32, 512, 4000, (0, 900)),
    "pair, joint items, d_c 384": (20, 6, 20, 384, 48, 16, 1500, (0, 2000)),
    "pair, prefix and own items": (30, 2, 40, 512, 0, 64, 3000, (10, 1500)),
    "pair, prefix and own items, d_c 128": (40, 1, 66, 128, 64, 32, 5000, (0, 2000)),
    "prefix by pairs, 32 rows": (64, 1, 32, 512, 64, 512, 9000, (1, 700)),
    "prefix by pairs, 64 rows, d_c 384": (50, 3, 20, 384, 48, 48, 7001, (0, 900)),
}
EVERY = [(BF16, n) for n in VARIANTS] + [(F32, n) for n in ("16 rows", "pair, joint items, d_c 384")]


def _lens(B, span):
    return torch.randint(span[0], span[1] + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()


@pytest.mark.parametrize("dtype,name", EVERY)
def test_decode_scores_far_below_zero(K, dtype, name):
    """Finite scores of -8e34, alone or before ordinary ones, are scores like others.

    In even heads channel 0 of q is 2^60 and its other channels are 0; tokens that carry -2^60 in channel 0 of c score
    -2^120 2^-4, exactly, and all the same.
    """
    B, n_q, H, d_c, d_r, page, prefix, span = VARIANTS[name]
    case = _case(B, n_q, H, d_c, d_r, page, prefix, _lens(B, span), dtype, seed=B + H)
    q, qp, pages, table, lens, pre = case
    q[:, :, 0::2], qp[:, :, 0::2] = 0, 0
    q[:, :, 0::2, 0] = 2.0 ** 60
    q[:, :, 1::2, 0] = 0
    d = d_c + d_r
    rows = pages[:, :page * d].view(-1, page, d)
    for b, (ids, n) in enumerate([(pre, prefix)] + [(table[b], n) for b, n in enumerate(lens.tolist())]):
        t = torch.arange(n)
        low = t < n if b % 3 else t < n // 2                     # every token, or the first half
        rows[ids[t // page].long(), t % page, 0] = torch.where(low, -2.0 ** 60, 0.0).to(dtype)
    o, lse = _run(K, case, page, prefix, 2.0 ** -4)
    ro, rl, ra = _reference(case, page, prefix, 2.0 ** -4)
    live = torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse), ~live)
    assert torch.all((lse.double() - rl)[live].abs() < LSE_TOL + 2.0 ** -20 * rl[live].abs())
    u, w = (2.0 ** -8, 2.0 ** -10) if dtype == BF16 else (2.0 ** -22, TOL_F32)
    assert torch.all((o.double() - ro).abs() <= u * (ro.abs() + ra) + w * ra)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("dtype,name", EVERY)
def test_decode_moving_references(K, dtype, name):
    """Scores that rise, fall or stay along the tokens, row by row, and by up to 2^11 from tile to tile: rows' running
    references move after sums exist, some rows' alone, at different tiles.

    Head h's scores have the slope SLOPE[h % 6] / 16 nats a token over a ramp that falls back in its last third, and random
    parts of a few nats.  A score of size X is off by at most 8 roundings of 2^-23 X (the ramp enters the sum with one
    product, after or before which at most 16 partial sums are rounded in 2^-24 X), a weight by that relative to itself, and
    a mean of c under such weights by twice that of sum p |c| / l.  fp32 sums of `top` terms: 2^-24 top of the same.
    """
    B, n_q, H, d_c, d_r, page, prefix, span = VARIANTS[name]
    case = _case(B, n_q, H, d_c, d_r, page, prefix, _lens(B, span), dtype, seed=B + H, gain=0.5)
    q, qp, pages, table, lens, pre = case
    d, top = d_c + d_r, prefix + max(lens.tolist())
    q *= 0.25
    slope = torch.tensor([1.0, -1.0, 0.25, 0.0, 0.5, -0.125])[torch.arange(H) % 6]
    at = 0 if d_r == 0 else d_c                                  # the ramp's channel: of c, or of the position part
    if d_r:
        qp.zero_()
        qp[..., 0] = slope.to(dtype)
    else:
        q[..., 0] = slope.to(dtype)
    rows = pages[:, :page * d].view(-1, page, d)
    for ids, n, first in [(pre, prefix, 0)] + [(table[b], n, prefix) for b, n in enumerate(lens.tolist())]:
        t = torch.arange(n)
        x = first + t
        ramp = torch.where(x < 2 * top // 3, x, 2 * (2 * top // 3) - x) / 16.0
        rows[ids[t // page].long(), t % page, at] = ramp.to(dtype)
    o, lse = _run(K, case, page, prefix, 1.0)
    ro, rl, ra = _reference(case, page, prefix, 1.0)
    live = torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse), ~live)
    X = top / 16.0 + 40
    assert (lse.double() - rl)[live].abs().max() < LSE_TOL + 8 * 2.0 ** -23 * X
    u, w = (2.0 ** -8, 2.0 ** -10) if dtype == BF16 else (2.0 ** -22, 2.0 ** -24 * top)
    assert torch.all((o.double() - ro).abs() <= u * (ro.abs() + ra) + (w + 16 * 2.0 ** -23 * X) * ra)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("dtype,name", EVERY)
def test_decode_bad_page_ids_read_zeros(K, dtype, name):
    """Ids that name no page, below and above the arena, of prefixes and of own tokens: their tokens are zeros."""
    B, n_q, H, d_c, d_r, page, prefix, span = VARIANTS[name]
    case = _case(B, n_q, H, d_c, d_r, page, prefix, _lens(B, span), dtype, seed=B + H)
    q, qp, pages, table, lens, pre = case
    n = pages.shape[0]
    bad = torch.zeros_like(table, dtype=torch.bool)
    width = torch.tensor([-(-max(0, m) // page) for m in lens.tolist()])
    used = torch.arange(table.shape[1])[None] < width[:, None]
    bad[used] = torch.rand(int(used.sum()), generator=torch.Generator().manual_seed(1)) < 0.3
    bad_pre = torch.arange(pre.numel()) % 3 == 1
    wrong = torch.tensor([-1, n, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32)
    for ids, mask in ((table, bad), (pre, bad_pre)):
        ids[mask] = wrong[torch.arange(int(mask.sum())) % 4]
    assert bad.any() and (prefix == 0 or bad_pre.any())
    o, lse = _run(K, case, page, prefix, 192 ** -0.5)
    assert K.kda_device_errors() == K.DEVERR_INDEX
    zero = torch.cat([pages, torch.zeros_like(pages[:1])])       # the zeros' page, where the oracle reads it
    ro, rl, ra = _reference((q, qp, zero, table.masked_fill(bad, n), lens, pre.masked_fill(bad_pre, n)), page, prefix, 192 ** -0.5)
    live = torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse), ~live)
    assert (lse.double() - rl)[live].abs().max() < LSE_TOL
    if dtype == F32:
        assert float((o.double() - ro).abs().max() / ro.abs().max()) < TOL_F32
    else:
        assert torch.all((o.double() - ro).abs() <= 2 ** -8 * (ro.abs() + ra) + 2 ** -10 * ra)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("through_ctypes", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_takes_queries_head_by_head(K, dtype, through_ctypes):
    """Queries as a matrix product per head leaves them, (H, T, ..): the same results as from a dense copy."""
    T, H, d_r = 37, 12, 48
    pages, slots, pos, table, fused, qs, w = _append_case(T, H, 128, d_r, dtype, 3, 4, 16)
    page = np.int64(16) if through_ctypes else 16
    args = (page, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :128], fused.cuda()[:, 128:])
    q = qs.cuda().transpose(0, 1).contiguous().transpose(0, 1)[:, :, 128:]
    assert q.stride(1) > q.stride(0)
    a, b = pages.cuda(), pages.cuda()
    out = K.kda_mla_append(a.view(torch.uint8), *args, q_pe=q)
    assert torch.equal(out, K.kda_mla_append(b.view(torch.uint8), *args, q_pe=q.contiguous())) and torch.equal(a, b)
    assert K.kda_device_errors() == 0
