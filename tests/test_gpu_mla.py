"""The latent page cache on the GPU against the fp64 oracle.

Bounds.  append computes in fp32 and rounds once: bf16 values are within one rounding, 2^-8 |x|, of the
exact ones, plus the fp32 error of the normalisation or rotation (a few 2^-24 of the pair's size).
decode, bf16: the softmax weights are rounded to bf16 for the product with c (2^-8 of sum p|c|/l, the
oracle's third result) and o once more (2^-8 |o|); the fp32 scores' error moves the weights by much less,
allowed 2^-10 of the same sum.  fp32: TOL_F32 of the largest value.  lse: scores are sums of 576 products of
total size ~30, rounded in fp32 (4 sqrt(576) 2^-24 30 < 2e-4).
"""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from oracle import kda_oracle as O
from parity import TOL_F32, rel

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LSE_TOL = 2e-4


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import kda
    kda.kda_device_errors()
    return kda


def _case(B, n_q, H, d_c, d_r, page, prefix, lens, dtype, seed=0, extra=40, gain=1.0):
    """Inputs with random page order; every value that no query may read is NaN, every page id past a length -1."""
    gen = torch.Generator().manual_seed(seed)
    d = d_c + d_r
    norm = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    n_pre = -(-prefix // page)
    need = [-(-max(0, n) // page) for n in lens]
    n_pages = n_pre + sum(need) + 2
    perm = torch.randperm(n_pages, generator=gen).tolist()
    pages = torch.full((n_pages, page * d + extra), float("nan"), dtype=dtype)
    pre, own, at = perm[:n_pre], [], n_pre
    for n in need:
        own.append(perm[at:at + n])
        at += n
    for ids, n in [(pre, prefix)] + [(own[b], max(0, n)) for b, n in enumerate(lens)]:
        for j, p in enumerate(ids):
            live = min(page, n - j * page)
            pages[p, :live * d] = (gain * torch.randn(live * d, generator=gen)).to(dtype)
    width = max(1, max(need))
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :need[b]] = torch.tensor(own[b], dtype=torch.int32)
    q, qp = norm(B, n_q, H, d_c), norm(B, n_q, H, d_r)
    return q, qp, pages, table, torch.tensor(lens, dtype=torch.int32), torch.tensor(pre, dtype=torch.int32)


def _run(K, case, page, prefix, scale, **kw):
    q, qp, pages, table, lens, pre = (t.cuda() for t in case)
    return K.kda_mla_decode(q, qp if qp.shape[-1] else None, pages.view(torch.uint8), page, table, lens, scale,
                            prefix_pages=pre if prefix else None, prefix_len=prefix, **kw)


def _check(case, page, prefix, scale, o, lse):
    q, qp, pages, table, lens, pre = case
    ro, rl, ra = O.mla_decode(f64(q), f64(qp), f64(pages), page, table.numpy(), lens.tolist(), scale, pre.tolist(), prefix)
    o, lse = f64(o), f64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    live = np.isfinite(rl)
    assert np.all(o[~live] == 0)
    if live.any():
        assert np.abs(lse[live] - rl[live]).max() < LSE_TOL
        if q.dtype == F32:
            assert rel(o, ro) < TOL_F32
        else:
            assert np.all(np.abs(o - ro) <= 2 ** -8 * (np.abs(ro) + ra) + 2 ** -10 * ra)


DECODE = [
    # B, n_q, H, d_c, d_r, page, prefix, lens
    (1, 1, 32, 512, 64, 512, 0, [1]),
    (1, 1, 32, 512, 64, 512, 0, [700]),
    (3, 1, 16, 512, 64, 64, 0, [63, 64, 65]),
    (2, 1, 4, 256, 64, 16, 0, [15, 129]),
    (4, 1, 20, 384, 48, 48, 0, [0, 1, -1, 100]),                # empty, padded
    (2, 1, 128, 512, 64, 128, 0, [500, 33]),                    # several row tiles per sequence
    (2, 16, 8, 512, 64, 64, 0, [40, 5]),                        # a draft longer than the sequence: empty rows
    (3, 3, 20, 128, 16, 80, 0, [200, 2, 127]),                  # rows that fill no tile
    (5, 1, 32, 512, 64, 512, 1000, [1, 20, 0, -1, 300]),        # prefix; rows that see it alone
    (3, 5, 12, 512, 32, 32, 77, [4, 64, 190]),
    (40, 1, 8, 128, 64, 16, 65, [j % 23 for j in range(40)]),
    (2, 1, 16, 512, 0, 64, 128, [70, 0]),                       # no position part
    (1, 2, 5, 256, 16, 16, 16, [0]),                            # the prefix alone
    (1, 1, 1, 512, 64, 96, 0, [9000]),                          # one row, many CTAs
    (6, 8, 16, 256, 32, 48, 900, [9, 100, 0, 257, -1, 640]),    # many rows on prefix and own tokens
    (70, 1, 16, 512, 0, 16, 257, [j % 31 for j in range(70)]),
    (2, 4, 64, 512, 64, 512, 3000, [1500, 10]),
    (30, 5, 20, 256, 16, 32, 128, [(j * 37) % 300 for j in range(30)]),
    (1, 16, 128, 512, 64, 64, 0, [2000]),
    (4, 5, 32, 384, 48, 48, 700, [0, 333, -1, 90]),             # channels that are no whole 256s
    (3, 1, 128, 128, 32, 64, 0, [1000, 65, 1]),
    (2, 2, 64, 384, 0, 16, 300, [500, 129]),
    (20, 4, 32, 128, 16, 32, 5, [j * 3 for j in range(20)]),    # many short items
    (9, 1, 32, 384, 64, 512, 900, [600, 5, 64, 65, 1, 0, 128, 127, 129]),
    (300, 1, 2, 128, 16, 16, 0, [(j * 7) % 40 - 1 for j in range(300)]),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", DECODE)
def test_decode_matches_oracle(K, shape, dtype):
    B, n_q, H, d_c, d_r, page, prefix, lens = shape
    case = _case(B, n_q, H, d_c, d_r, page, prefix, lens, dtype, seed=sum(lens) + H)
    o, lse = _run(K, case, page, prefix, 192 ** -0.5)
    _check(case, page, prefix, 192 ** -0.5, o, lse)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_growing_scores(K, dtype):
    """Scores that rise steeply along the tokens move the running reference again and again."""
    B, H, n = 2, 32, 900
    case = list(_case(B, 1, H, 512, 64, 64, 300, [n, 451], dtype, seed=5))
    q, qp, pages, table, lens, pre = case
    qp.zero_()
    qp[..., 0] = 8.0
    rows = pages[:, :64 * 576].view(-1, 64, 576)
    for ids, m, first in ((pre.tolist(), 300, 0), (table[0].tolist(), n, 300), (table[1].tolist(), 451, 300)):
        for t in range(m):
            rows[ids[t // 64], t % 64, 512] = (first + t) / 16.0
    scale = 0.5                                                   # up to 300 / e-folds over the line
    o, lse = _run(K, case, 64, 300, scale)
    ro, rl, ra = O.mla_decode(f64(q), f64(qp), f64(pages), 64, table.numpy(), lens.tolist(), scale, pre.tolist(), 300)
    assert np.abs(f64(lse) - rl).max() < 4e-6 * np.abs(rl).max() + LSE_TOL
    # fp32 scores of size ~300 are off by up to 300 2^-23 4: the weights by as much
    slack = 2e-4 if dtype == F32 else 2 ** -8 * 1.1
    assert np.all(np.abs(f64(o) - ro) <= slack * (np.abs(ro) + ra))


def _reference(case, page, prefix, scale):
    """The oracle's definition on the GPU in fp64, for sizes its loops are too slow for."""
    q, qp, pages, table, lens, pre = (t.cuda() for t in case)
    B, n_q, H, d_c = q.shape
    d = d_c + qp.shape[-1]
    full = torch.cat([q, qp], -1).double() * scale
    token = lambda ids, n: pages[ids.long(), :page * d].reshape(-1, d)[:n].double()  # noqa: E731
    o, ab = torch.zeros(2, B, n_q, H, d_c, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n_q, H), -float("inf"), dtype=torch.float64, device="cuda")
    shared = token(pre, prefix)
    for b, n in enumerate(lens.tolist()):
        if n < 0:
            continue
        keys = torch.cat([shared, token(table[b, :-(-n // page)], n)])
        for i in range(n_q):
            k = keys[:prefix + max(0, n - (n_q - 1 - i))]
            if len(k):
                x = full[b, i] @ k.T
                p = torch.softmax(x, -1)
                lse[b, i], o[b, i], ab[b, i] = torch.logsumexp(x, -1), p @ k[:, :d_c], p @ k[:, :d_c].abs()
    return o, lse, ab


@pytest.mark.parametrize("dtype,shape", [
    (BF16, (40, 1, 64, 512, 64, 512, 9000, (1, 700))),        # prefix by pairs of CTAs, own tokens by single ones
    (BF16, (24, 8, 32, 256, 32, 48, 3001, (0, 900))),         # joint items, pages that end inside tiles
    (BF16, (12, 3, 40, 384, 64, 16, 2000, (5, 600))),         # prefix and own items apart
    (BF16, (70, 3, 20, 128, 16, 80, 1003, (0, 300))),         # prefix by pairs; owners of 60 rows
    (BF16, (90, 1, 5, 384, 0, 32, 9999, (0, 200))),           # and of 5
    (BF16, (64, 1, 32, 512, 64, 512, 2048, (0, 700))),        # prefix and owners in one launch of single CTAs
    (BF16, (33, 3, 20, 384, 48, 48, 1003, (0, 900))),
    (BF16, (150, 1, 32, 512, 64, 64, 0, (2000, 5000))),       # many tiles and several items per CTA
    (BF16, (3, 1, 8, 128, 16, 512, 0, (30000, 60000))),       # few rows, many CTAs per row
    (BF16, (9, 2, 64, 512, 0, 64, 0, (1000, 4000))),          # pairs without a prefix
    (F32, (20, 2, 24, 512, 64, 32, 700, (3, 900))),
])
def test_decode_many_tiles(K, dtype, shape):
    B, n_q, H, d_c, d_r, page, prefix, (lo, hi) = shape
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(lo, hi + 1, (B,), generator=gen).tolist()
    case = _case(B, n_q, H, d_c, d_r, page, prefix, lens, dtype, seed=B + H)
    o, lse = _run(K, case, page, prefix, 192 ** -0.5)
    ro, rl, ra = _reference(case, page, prefix, 192 ** -0.5)
    live = torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse), ~live)
    assert (lse.double() - rl)[live].abs().max() < LSE_TOL
    if dtype == F32:
        assert float((o.double() - ro).abs().max() / ro.abs().max()) < TOL_F32
    else:
        assert torch.all((o.double() - ro).abs() <= 2 ** -8 * (ro.abs() + ra) + 2 ** -10 * ra)
    assert K.kda_device_errors() == 0


def test_decode_does_not_read_past_lengths(K):
    """Same live rows, other garbage (NaN, infinities, finite): the same bits."""
    case = _case(3, 2, 16, 512, 64, 48, 70, [50, 1, 97], BF16, seed=7)
    o, lse = _run(K, case, 48, 70, 0.08)
    for fill in (float("inf"), -float("inf"), 3.0):
        pages = torch.where(torch.isnan(case[2]), torch.tensor(fill, dtype=BF16), case[2])
        o2, lse2 = _run(K, (*case[:2], pages, *case[3:]), 48, 70, 0.08)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_same_bits_twice_and_on_another_stream(K):
    case = _case(9, 1, 32, 512, 64, 64, 500, [100 * j for j in range(9)], BF16, seed=8)
    o, lse = _run(K, case, 64, 500, 0.07)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    need = K.kda_mla_decode_workspace_bytes(9, 1, 32, 512, 500, BF16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # a workspace needs no clearing
    torch.cuda.synchronize()
    o2, lse2 = _run(K, case, 64, 500, 0.07, stream=st, workspace=ws)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("through_ctypes", [False, True])
def test_allocations_belong_to_the_calls_stream(K, through_ctypes):
    """Memory that the current stream has given back but not finished with is not taken for a call on another."""
    case = [t.cuda() for t in _case(3, 1, 16, 512, 64, 64, 0, [100, 5, 64], BF16, seed=11)]
    q, qp, pages, table, lens, _ = case
    args = (q, qp, pages.view(torch.uint8), np.int64(64) if through_ctypes else 64, table, lens, 0.07)
    want, want_lse = K.kda_mla_decode(*args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    sizes = [q.numel() * 2, 3 * 16 * 4, K.kda_mla_decode_workspace_bytes(3, 1, 16, 512, 0, BF16)]
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    given_back = {t.data_ptr() for t in held}
    del held
    for stream in (st, st.cuda_stream):
        o, lse = K.kda_mla_decode(*args, stream=stream)
        assert o.data_ptr() not in given_back and lse.data_ptr() not in given_back
        st.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    table2, pos = torch.zeros(8, 64, device="cuda"), torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    c, k = torch.zeros(2, 512, dtype=BF16, device="cuda"), torch.zeros(2, 64, dtype=BF16, device="cuda")
    qq = torch.ones(2, 16, 64, dtype=BF16, device="cuda")
    held = [torch.empty_like(qq) for _ in range(4)]
    given_back = {t.data_ptr() for t in held}
    del held
    torch.cuda.synchronize()
    out = K.kda_mla_append(pages.clone().view(torch.uint8), args[3], pos, pos, table2, c, k, q_pe=qq, stream=st)
    st.synchronize()
    assert out.data_ptr() not in given_back and torch.all(out == 0)


def test_decode_in_a_graph(K):
    """Lengths are device memory: a captured call follows them."""
    case = _case(4, 1, 32, 512, 64, 64, 100, [300, 10, 64, 129], BF16, seed=9)
    q, qp, pages, table, lens, pre = (t.cuda() for t in case)
    o, lse = torch.empty_like(q), torch.empty(4, 1, 32, device="cuda")
    ws = torch.empty(K.kda_mla_decode_workspace_bytes(4, 1, 32, 512, 100, BF16), dtype=torch.uint8, device="cuda")
    call = lambda: K.kda_mla_decode(q, qp, pages.view(torch.uint8), 64, table, lens, 0.07, prefix_pages=pre,  # noqa: E731
                                    prefix_len=100, o=o, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    short = torch.tensor([3, 10, -1, 65], dtype=torch.int32)
    lens.copy_(short)
    g.replay()
    torch.cuda.synchronize()
    _check((*case[:4], short, case[5]), 64, 100, 0.07, o, lse)


def test_decode_bad_page_id_raises_the_error_word(K):
    case = list(_case(2, 1, 8, 128, 16, 16, 0, [20, 30], F32, seed=10))
    case[3][1, 1] = 1000
    for dt in (F32, BF16):
        o, _ = _run(K, (case[0].to(dt), case[1].to(dt), case[2].to(dt), *case[3:]), 16, 0, 0.1)
        assert K.kda_device_errors() & K.DEVERR_INDEX
        assert torch.isfinite(o).all()
    assert K.kda_device_errors() == 0


def test_decode_offsets_past_32_bits(K):
    """A page arena of more than 4 GiB with the live pages at its end."""
    page, d, n_pages = 512, 576, 7600                            # 7600 * 512 * 576 * 2 B = 4.5 GB
    arena = torch.zeros(n_pages, page * d, dtype=BF16, device="cuda")
    rows = torch.randn(700, d, generator=torch.Generator().manual_seed(3)).to(BF16)
    arena[n_pages - 1] = rows[:512].reshape(-1).cuda()
    arena[n_pages - 2, :188 * d] = rows[512:].reshape(-1).cuda()
    q, qp, *_ = _case(1, 1, 16, 512, 64, 16, 0, [1], BF16, seed=4)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32)
    o, lse = K.kda_mla_decode(q.cuda(), qp.cuda(), arena.view(torch.uint8), page, table.cuda(),
                              torch.tensor([700], dtype=torch.int32, device="cuda"), 0.07)
    small = torch.zeros(2, page * d, dtype=BF16)
    small[0], small[1, :188 * d] = rows[:512].reshape(-1), rows[512:].reshape(-1)
    _check((q, qp, small, torch.tensor([[0, 1]], dtype=torch.int32), torch.tensor([700]), torch.tensor([])), page, 0, 0.07, o, lse)


# ---------------------------------------------------------------------------
def _append_case(T, H, d_c, d_r, dtype, seed, n_pages, page, n_pos=5000):
    gen = torch.Generator().manual_seed(seed)
    norm = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    slots = torch.randperm(n_pages * page, generator=gen)[:T].to(torch.int32)
    pos = torch.randint(0, n_pos, (T,), generator=gen).to(torch.int32)
    return (norm(n_pages, page * (d_c + d_r) + 24), slots, pos, torch.from_numpy(O.rope_table(n_pos, max(d_r, 2))).float(),
            norm(T, d_c + d_r), norm(T, H, 128 + d_r), 1 + 0.1 * norm(d_c))


APPEND = [(1, 32, 512, 64, 512), (7, 5, 384, 48, 48), (64, 1, 128, 16, 16), (33, 20, 256, 32, 80), (300, 128, 512, 64, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", APPEND)
def test_append_matches_oracle(K, shape, inter, dtype):
    T, H, d_c, d_r, page = shape
    n_pages = -(-T // page) + 2
    pages, slots, pos, table, fused, qs, w = _append_case(T, H, d_c, d_r, dtype, T + H, n_pages, page)
    if T > 3:
        slots[1], slots[2] = -1, n_pages * page                   # rows that are not written
    for weight in (w, None):
        dev = pages.cuda()
        q_out = K.kda_mla_append(dev.view(torch.uint8), page, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :d_c],
                                 fused.cuda()[:, d_c:], q_pe=qs.cuda()[:, :, 128:], norm_weight=None if weight is None else w.cuda(),
                                 style=K.ROPE_INTERLEAVED if inter else K.ROPE_HALF)
        ref, rq = O.mla_append(f64(pages), page, slots.tolist(), pos.tolist(), f64(table), f64(fused[:, :d_c]),
                               f64(fused[:, d_c:]), f64(qs[:, :, 128:]), None if weight is None else f64(w), 1e-6, inter)
        for x, y, z in ((dev, ref, f64(pages)), (q_out, rq, None)):
            x = f64(x)
            u = 2 ** -8 if dtype == BF16 else 2 ** -21
            assert np.all(np.abs(x - y) <= u * np.abs(y) + 2 ** -20 * 4)
            if z is not None:
                same = y == z                                     # everything else keeps its bits
                assert np.array_equal(x[same], z[same])
    assert K.kda_device_errors() == 0


def test_append_in_place_and_without_position_part(K):
    pages, slots, pos, table, fused, qs, w = _append_case(9, 6, 256, 32, BF16, 1, 2, 16)
    q = qs[:, :, 128:].contiguous()
    args = (16, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :256], fused.cuda()[:, 256:])
    a, b = pages.cuda(), pages.cuda()
    out = K.kda_mla_append(a.view(torch.uint8), *args, q_pe=q.cuda())
    inplace = q.cuda()
    assert K.kda_mla_append(b.view(torch.uint8), *args, q_pe=inplace, q_pe_out=inplace) is inplace
    assert torch.equal(out, inplace) and torch.equal(a, b)
    pages, slots, _, _, fused, _, w = _append_case(9, 6, 256, 0, F32, 2, 2, 16)
    dev = pages.cuda()
    assert K.kda_mla_append(dev.view(torch.uint8), 16, slots.cuda(), None, None, fused.cuda(), None, norm_weight=w.cuda()) is None
    ref, _ = O.mla_append(f64(pages), 16, slots.tolist(), [0] * 9, np.zeros((1, 0)), f64(fused), np.zeros((9, 0)), None, f64(w))
    assert np.abs(f64(dev) - ref).max() < 2 ** -20 * 4


def test_append_bad_position_raises_the_error_word(K):
    pages, slots, pos, table, fused, qs, _ = _append_case(4, 3, 128, 16, F32, 3, 1, 16)
    pos[1], pos[3] = -1, 5000
    qs[1] = float("nan")
    dev = pages.cuda()
    q = K.kda_mla_append(dev.view(torch.uint8), 16, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :128],
                         fused.cuda()[:, 128:], q_pe=qs.cuda()[:, :, 128:])
    assert K.kda_device_errors() == K.DEVERR_INDEX
    assert torch.all(q[1] == 0) and torch.all(q[3] == 0) and torch.all(q[0] != 0)
    assert torch.equal(dev[0, int(slots[1]) * 144:int(slots[1]) * 144 + 144].cpu(), pages[0, int(slots[1]) * 144:int(slots[1]) * 144 + 144])
    assert K.kda_device_errors() == 0


def test_append_then_decode_through_the_page_pool(K):
    """Pages of the unified pool: a prompt is appended, then token by token, and read back by attention."""
    page, H, B = 64, 16, 3
    pool = K.PagePool(page * 576 * 2 + 256, 12)
    state = pool.alloc(2, K.PAGE_KDA_STATE)
    pre = pool.alloc(2, K.PAGE_MLA_KV)
    own = [pool.alloc(2, K.PAGE_MLA_KV) for _ in range(B)]
    assert not set(state) & set(pre + sum(own, []))
    gen = torch.Generator().manual_seed(11)
    table = torch.from_numpy(O.rope_table(400, 64)).float()
    mirror = np.full((12, page * 576 + 128), 0.0)
    w = (1 + 0.1 * torch.randn(512, generator=gen)).to(BF16)

    def append(slots, positions, q_pe=None):
        nonlocal mirror
        rows = torch.randn(len(slots), 576, generator=gen).to(BF16)
        s, p = torch.tensor(slots, dtype=torch.int32), torch.tensor(positions, dtype=torch.int32)
        out = K.kda_mla_append(pool.pages, page, s.cuda(), p.cuda(), table.cuda(), rows.cuda()[:, :512], rows.cuda()[:, 512:],
                               q_pe=None if q_pe is None else q_pe.cuda(), norm_weight=w.cuda())
        mirror, _ = O.mla_append(mirror, page, slots, positions, f64(table), f64(rows[:, :512]), f64(rows[:, 512:]), None, f64(w))
        return out

    append([pre[t // page] * page + t % page for t in range(100)], list(range(100)))
    for t in range(66):                                            # crosses a page boundary
        q_pe = torch.randn(B, H, 64, generator=gen).to(BF16)
        rot = append([own[b][t // page] * page + t % page for b in range(B)], [100 + t] * B, q_pe)
    q = torch.randn(B, 1, H, 512, generator=gen).to(BF16)
    lens = [66, 66, 66]
    o, lse = K.kda_mla_decode(q.cuda(), rot.view(B, 1, H, 64), pool.pages, page, torch.tensor(own, dtype=torch.int32).cuda(),
                              torch.tensor(lens, dtype=torch.int32).cuda(), 0.07,
                              prefix_pages=torch.tensor(pre, dtype=torch.int32).cuda(), prefix_len=100)
    stored = pool.pages.view(BF16).float().double().cpu().numpy()
    live = mirror != 0
    assert np.all(np.abs(stored[live] - mirror[live]) <= 2 ** -8 * np.abs(mirror[live]) + 2 ** -20 * 4)
    full = torch.from_numpy(np.where(live, stored, 0.0)).to(BF16)
    _check((q, rot.view(B, 1, H, 64).cpu(), full, torch.tensor(own), torch.tensor(lens), torch.tensor(pre)), page, 100, 0.07, o, lse)


# ---------------------------------------------------------------------------
def _call(K, case, page, prefix, **kw):
    q, qp, pages, table, lens, pre = (t.cuda() for t in case)
    args = dict(q=q, q_pe=qp, pages=pages.view(torch.uint8), page_tokens=page, page_table=table, lens=lens, scale=0.1,
                prefix_pages=pre, prefix_len=prefix)
    return K.kda_mla_decode(**{**args, **{k: v(args) if callable(v) else v for k, v in kw.items()}})


def test_binding_refuses_and_says_why(K):
    case = _case(3, 2, 8, 128, 16, 16, 40, [9, 0, 33], BF16, seed=20)
    good, lse = _call(K, case, 16, 40)
    for kw, exc, word in [
        (dict(q=lambda a: a["q"].half()), TypeError, "float32 or bfloat16"), (dict(q=lambda a: a["q"].cpu()), TypeError, "CUDA"),
        (dict(q=lambda a: a["q"].transpose(1, 2)), (ValueError, TypeError), None), (dict(q_pe=lambda a: a["q_pe"][:2]), ValueError, "q_pe"),
        (dict(q_pe=lambda a: a["q_pe"].float()), TypeError, "q_pe"), (dict(pages=lambda a: a["pages"].view(-1)), ValueError, "pages"),
        (dict(pages=lambda a: a["pages"].view(BF16)), TypeError, "pages"), (dict(page_table=lambda a: a["page_table"].long()), TypeError, "page_table"),
        (dict(page_table=lambda a: a["page_table"][:2]), ValueError, "page_table"), (dict(lens=lambda a: a["lens"][:2]), ValueError, "lens"),
        (dict(lens=lambda a: a["lens"].cpu()), TypeError, "lens"), (dict(prefix_pages=None), (TypeError, AttributeError), None),
        (dict(prefix_len=1000), ValueError, "prefix_pages"), (dict(scale=-1.0), K.KdaError, "scale"), (dict(page_tokens=24), K.KdaError, "page_tokens"),
        (dict(page_tokens=512), K.KdaError, "page_bytes"), (dict(workspace=lambda a: torch.empty(1024, dtype=torch.uint8, device="cuda")), K.KdaError, "workspace"),
        (dict(o=lambda a: torch.empty(3, 2, 8, 64, dtype=BF16, device="cuda")), ValueError, "o "), (dict(lse=lambda a: torch.empty(3, 2, 8, device="cuda").half()), TypeError, "lse"),
        (dict(o=lambda a: a["q"]), K.KdaError, "overlap"),
    ]:
        with pytest.raises(exc, match=word):
            _call(K, case, 16, 40, **kw)
    again, lse2 = _call(K, case, 16, 40, prefix_len=np.int64(40))          # the way through ctypes
    assert torch.equal(good, again) and torch.equal(lse, lse2)
    o, l = torch.empty_like(good), torch.empty_like(lse)
    r = _call(K, case, 16, 40, o=o, lse=l, stream=torch.cuda.current_stream())
    assert r[0] is o and r[1] is l and torch.equal(o, good) and torch.equal(l, lse)
    assert K.kda_device_errors() == 0


def test_append_binding_refuses_and_says_why(K):
    pages, slots, pos, table, fused, qs, w = _append_case(5, 3, 128, 16, BF16, 30, 2, 16)
    base = dict(pages=pages.cuda().view(torch.uint8), page_tokens=16, slots=slots.cuda(), positions=pos.cuda(), rope=table.cuda(),
                c=fused.cuda()[:, :128], k_pe=fused.cuda()[:, 128:], q_pe=qs.cuda()[:, :, 128:], norm_weight=w.cuda())
    out = K.kda_mla_append(**base)
    for kw, exc, word in [
        (dict(c=base["c"].double()), TypeError, "float32 or bfloat16"), (dict(c=base["c"].t()), (ValueError, TypeError), None),
        (dict(k_pe=base["k_pe"][:3]), ValueError, "k_pe"), (dict(slots=base["slots"].long()), TypeError, "slots"),
        (dict(positions=base["positions"][:2]), ValueError, "positions"), (dict(rope=base["rope"].half()), TypeError, "rope"),
        (dict(rope=base["rope"][:, :8]), ValueError, "rope"), (dict(norm_weight=base["norm_weight"].float()), TypeError, "norm_weight"),
        (dict(q_pe=base["q_pe"].float()), TypeError, "q_pe"), (dict(style=7), K.KdaError, "style"), (dict(eps=-1.0), K.KdaError, "eps"),
        (dict(pages=base["pages"][0]), ValueError, "pages"), (dict(page_tokens=32), K.KdaError, "page_bytes"),
        (dict(q_pe_out=torch.empty(5, 3, 8, dtype=BF16, device="cuda")), ValueError, "q_pe_out"),
        (dict(c=fused.cuda()[:, 4:132]), K.KdaError, "aligned"),
    ]:
        with pytest.raises(exc, match=word):
            K.kda_mla_append(**{**base, **kw})
    mine = torch.empty_like(out)
    assert K.kda_mla_append(**base, q_pe_out=mine) is mine and torch.equal(mine, out)
    assert K.kda_mla_append(**{**base, "q_pe": None}) is None
    assert K.kda_device_errors() == 0
