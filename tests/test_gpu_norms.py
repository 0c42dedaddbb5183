"""The norms around a block on the GPU, against the fp64 oracle.

Bounds.  Everything is fp32 with one rounding at the end: 2^-8 of the value for bf16.  In fp32 the sum of d squares is off by at most
d 2^-24 of itself, the root halves that; the exponential of the gate's activation is within 2^-21, and a little more for each of
up to 16 in its argument (16 log2(e) 2^-24): (d / 2 + 40) 2^-24 of the value, of which the sum's part is far from reached.  h' adds two
numbers: the error of its second one, and 2^-24 of the sum.
"""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from oracle import kda_oracle as O

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
ROUND = {BF16: 2.0 ** -8, F32: U}


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import kda
    return kda


def _act(K, act):
    return {"none": K.ACT_NONE, "silu": K.ACT_SILU, "sigmoid": K.ACT_SIGMOID}[act]


def _wide(t, extra=16):
    """The same values as a view of wider rows, the rest NaN."""
    w = torch.full((t.shape[0] + 2, t[0].numel() + extra), float("nan"), dtype=t.dtype, device="cuda")
    w[1:1 + t.shape[0], 8:8 + t[0].numel()] = t.flatten(1).cuda()
    return w[1:1 + t.shape[0], 8:8 + t[0].numel()].view(t.shape)


GATED = [(1, 1, 8), (1, 32, 128), (5, 3, 32), (7, 2, 40), (3, 5, 64), (33, 4, 80), (9, 3, 96), (2, 6, 192), (4, 3, 256), (5, 2, 264), (3, 1, 512),
         (2, 3, 1000), (6, 1, 1024), (1000, 2, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("T,H,d", GATED)
def test_gated_norm(K, T, H, d, first, dtype):
    gen = torch.Generator().manual_seed(T + d)
    x, z = torch.randn(T, H, d, generator=gen).to(dtype), (3 * torch.randn(T, H, d, generator=gen)).to(dtype)
    x[0, 0] = 0
    act = ["sigmoid", "silu", "none"][(T + d) % 3]
    w = torch.randn((H, d) if T % 2 else (d,), generator=gen).to(dtype)
    y = K.kda_gated_norm(_wide(x), w.cuda(), gate=_wide(z), act=_act(K, act), gate_first=first)
    ref = O.gated_norm(f64(x), f64(w), f64(z), 1e-6, act, first)
    assert y.shape == (T, H, d) and y.is_contiguous()
    assert np.all(np.abs(f64(y) - ref) <= ((d / 2 + 40) * U + ROUND[dtype]) * np.abs(ref))
    y = K.kda_gated_norm(x.cuda(), w.cuda(), eps=0.5)             # no gate
    ref = O.gated_norm(f64(x), f64(w), None, 0.5)
    assert np.all(np.abs(f64(y) - ref) <= ((d / 2 + 40) * U + ROUND[dtype]) * np.abs(ref))


RESIDUAL = [(1, 8), (3, 64), (5, 256), (9, 264), (2, 2000), (4, 4096), (3, 4104), (2, 6144), (2, 8192), (3, 8200), (1, 16384), (130, 512)]


@pytest.mark.parametrize("dtype,h_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("parts", ["", "p", "g", "c", "pgc"])
@pytest.mark.parametrize("T,D", RESIDUAL)
def test_residual_norm(K, T, D, parts, dtype, h_dtype):
    gen = torch.Generator().manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    h, y, z = (2 * n(T, D)).to(h_dtype), n(T, D).to(dtype), (3 * n(T, D)).to(dtype)
    pre, post, cs = n(D).to(dtype), n(D).to(dtype), n(D).to(dtype)
    act = ["sigmoid", "silu", "none"][D % 3]
    kw = {"post_weight": post if "p" in parts else None, "gate": z if "g" in parts else None, "channel_scale": cs if "c" in parts else None}
    rh, rx = O.residual_norm(f64(h), f64(y), f64(pre), **{a: None if t is None else f64(t) for a, t in kw.items()}, res_scale=-0.7, act=act)
    on = {a: None if t is None else t.cuda() for a, t in kw.items()}
    if on["gate"] is not None:
        on["gate"] = _wide(z)
    hd = _wide(h)
    h2, x = K.kda_residual_norm(hd, _wide(y), pre.cuda(), res_scale=-0.7, act=_act(K, act), **on)
    assert h2 is hd and x.is_contiguous()
    u = np.abs(rh - f64(h))
    few = (D / 2 + 40) * U
    h_err = few * u + U * np.abs(rh)
    assert np.all(np.abs(f64(h2) - rh) <= h_err + ROUND[h_dtype] * np.abs(rh) + 1e-30)
    # an error of h moves its own x, and all by the norm: at most by the largest relative to the root of the mean square
    r = np.sqrt(np.mean(rh ** 2, -1, keepdims=True) + 1e-6)
    shift = np.sqrt(np.mean(h_err ** 2, -1, keepdims=True)) / r
    assert np.all(np.abs(f64(x) - rx) <= h_err / r * np.abs(f64(pre)) + (shift + few + ROUND[dtype]) * np.abs(rx) + 1e-30)
    # out of place: h stays
    before = h.cuda()
    to = torch.empty_like(before)
    h3, x3 = K.kda_residual_norm(before, y.cuda(), pre.cuda(), res_scale=-0.7, act=_act(K, act), h_out=to, **on)
    assert h3 is to and torch.equal(to, h2) and torch.equal(x3, x) and torch.equal(before, h.cuda())


def test_in_place(K):
    gen = torch.Generator().manual_seed(0)
    x, z, w = (torch.randn(*s, generator=gen).cuda().bfloat16() for s in ((50, 4, 128), (50, 4, 128), (128,)))
    ref = K.kda_gated_norm(x, w, gate=z)
    a, b = x.clone(), z.clone()
    assert torch.equal(K.kda_gated_norm(a, w, gate=z, y=a), ref)
    assert torch.equal(K.kda_gated_norm(x, w, gate=b, y=b), ref)
    with pytest.raises(K.KdaError):
        K.kda_gated_norm(a[:25], w, gate=z[:25], y=a[1:26])


def test_extremes(K):
    """Gates far out, rows of zeros with eps, infinite and NaN values in a row of their own."""
    x = torch.ones(5, 1, 32, device="cuda")
    z = torch.tensor([1e4, -1e4, 0.0, 0.0, 0.0], device="cuda")[:, None, None].expand(5, 1, 32).contiguous()
    x[2] = 0
    x[3, 0, 0] = float("nan")
    for act, at_top in ((K.ACT_SIGMOID, 1.0), (K.ACT_SILU, 1e4)):
        y = K.kda_gated_norm(x, torch.ones(32, device="cuda"), gate=z, act=act)
        assert torch.allclose(y[0], torch.full_like(y[0], at_top)) and torch.all(y[1] == 0) and torch.all(y[2] == 0)
        assert torch.isnan(y[3]).all() and torch.isfinite(y[4]).all()
    h = torch.zeros(3, 64, device="cuda")
    y = torch.zeros(3, 64, device="cuda")
    y[1, 5] = float("inf")
    h2, out = K.kda_residual_norm(h, y, torch.ones(64, device="cuda"))
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and torch.isinf(h2[1, 5]) and torch.isnan(out[1, 5])


def test_streams_and_graphs(K):
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda().bfloat16()  # noqa: E731
    x, z, w, h, pre = n(40, 4, 64), n(40, 4, 64), n(64), n(40, 256), n(256)

    def call(stream=None):
        y = K.kda_gated_norm(x, w, gate=z, stream=stream)
        return y, *K.kda_residual_norm(h, y.view(40, 256), pre, h_out=torch.empty_like(h), stream=stream)

    ref = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    x.copy_(n(40, 4, 64))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_the_two_bindings_agree(K, dtype, monkeypatch):
    if K._native is None:
        pytest.skip("the native module is not built")
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen).cuda().to(dtype)  # noqa: E731
    fused = n(30, 3 * 4 * 64)
    x, z = (t.view(30, 4, 64) for t in fused.split(256, 1)[:2])
    w, wh, pre, post, cs, h = n(64), n(4, 64), n(256), n(256), n(256), n(30, 256).float()

    def calls():
        h1, h2, y = h.clone(), torch.empty_like(h), torch.empty(30, 4, 64, device="cuda", dtype=dtype)
        r = [K.kda_gated_norm(x, w), K.kda_gated_norm(x, wh, gate=z, act=K.ACT_SILU, gate_first=True, y=y), y,
             *K.kda_residual_norm(h1, fused[:, :256], pre, gate=fused[:, 512:], act=K.ACT_NONE), h1,
             *K.kda_residual_norm(h, fused[:, :256], pre, post_weight=post, channel_scale=cs, res_scale=0.5, eps=1e-3, h_out=h2), h2]
        for bad in (lambda: K.kda_gated_norm(x, n(65)), lambda: K.kda_gated_norm(x, w, gate=z[:29]), lambda: K.kda_gated_norm(x, w, act=9),
                    lambda: K.kda_residual_norm(h, x, pre), lambda: K.kda_residual_norm(h, fused[:, :256], pre[:128]),
                    lambda: K.kda_residual_norm(h, fused[:, :256], pre, h_out=torch.empty(30, 512, device="cuda")[:, :256])):
            with pytest.raises((TypeError, ValueError, K.KdaError)):
                bad()
        return r

    a = calls()
    monkeypatch.setattr(K, "_native", None)
    for u, v in zip(a, calls()):
        assert torch.equal(u, v)


def test_offsets_past_32_bits(K):
    """The last rows of more than 2^32 values, and rows 2^24 values apart."""
    gen = torch.Generator().manual_seed(4)
    near = lambda got, ref, d: np.all(np.abs(f64(got) - ref) <= (2.0 ** -8 + (d / 2 + 40) * U) * np.abs(ref))  # noqa: E731
    T, H, d = (1 << 25) // 1024 + 3, 1024, 128
    last = torch.randn(2, H, d, generator=gen).cuda().bfloat16()
    x = torch.zeros(T, H, d, dtype=BF16, device="cuda")
    x[-2:] = last
    w = torch.ones(d, dtype=BF16, device="cuda")
    y = K.kda_gated_norm(x, w)
    assert near(y[-2:], O.rms(f64(last), 1e-6), d) and torch.all(y[:-2:997] == 0)
    del y
    D = 8192
    rows = x.view(-1, D)
    out = K.kda_residual_norm(rows, torch.zeros_like(rows), torch.ones(D, dtype=BF16, device="cuda"))[1]
    assert near(out[-32:], O.rms(f64(last).reshape(-1, D), 1e-6), D) and torch.equal(x[-2:], last)
    del out, rows, x
    wide = torch.empty(300, 1 << 24, dtype=BF16, device="cuda")
    wide[:, :1024] = torch.randn(300, 1024, generator=gen).cuda().bfloat16()
    a, b = wide[:, :512], wide[:, 512:1024]
    assert torch.equal(K.kda_gated_norm(a.unflatten(1, (4, d)), w, gate=b.unflatten(1, (4, d))),
                       K.kda_gated_norm(a.contiguous().view(300, 4, d), w, gate=b.contiguous().view(300, 4, d)))
    pre = torch.ones(512, dtype=BF16, device="cuda")
    h = torch.empty_like(wide)[:, :512]
    h.copy_(b)
    dense = K.kda_residual_norm(b.contiguous(), a.contiguous(), pre)
    for u, v in zip(K.kda_residual_norm(h, a, pre), dense):
        assert torch.equal(u, v)


def test_a_layer_of_a_hybrid_stack(K):
    """Norm, projections, linear attention, gated norm, projection, norm: prompt and decode steps as they would be used, against
    fp64. Every operator's inputs are the rounded ones that it got, so that each has its own bound; the last is the layer's whole
    way, 2^-8 for each of the seven roundings to bf16 on it (h, x, q k v, P and S, o, y, its projection), against the largest value."""
    gen = torch.Generator().manual_seed(2)
    D, H, d, T, steps = 256, 4, 64, 200, 5
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    w_in, w_out = (n(D, 3 * H * d + H * d) / D ** 0.5).bfloat16(), (n(H * d, D) / (H * d) ** 0.5).bfloat16()
    pre, head, nxt = ((1 + 0.1 * n(s)).bfloat16() for s in (D, d, D))
    decay = -torch.tensor([0.5, 0.1, 0.02, 0.004], device="cuda")

    def mix(x, S, one):
        p = x @ w_in
        q, k, v, z = (t.view(-1, H, d) for t in p.split(H * d, 1))
        o = (K.kda_linattn_step(S, q, k, v, decay, scale=d ** -0.5) if one else
             K.kda_linattn_prefill(None, q, k, v, decay, scale=d ** -0.5))
        o, S = (o, S) if one else o
        return K.kda_gated_norm(o, head, gate=z).view(-1, H * d) @ w_out, S

    h = n(T + steps, D)                                   # the residual stream, fp32
    first = h.clone()
    zero = torch.zeros(T + steps, D, device="cuda", dtype=BF16)
    outs, S = [], None
    for a, b in [(0, T)] + [(t, t + 1) for t in range(T, T + steps)]:
        _, x = K.kda_residual_norm(h[a:b], zero[a:b], pre)
        y, S = mix(x, S, a > 0)
        _, x2 = K.kda_residual_norm(h[a:b], y, nxt, res_scale=0.5)
        outs.append(x2)
    assert K.kda_device_errors() == 0
    x = O.rms(f64(first), 1e-6) * f64(pre)
    p = x @ f64(w_in)
    q, k, v, z = (t.reshape(-1, H, d) for t in np.split(p, 4, 1))
    o, states = O.linattn_recurrent(np.zeros((H, d, d)), q, k, v, f64(decay), d ** -0.5)
    y = O.gated_norm(o, f64(head), z).reshape(-1, H * d) @ f64(w_out)
    rh, rx = O.residual_norm(f64(first), y, f64(nxt), res_scale=0.5)
    for got, ref in ((h, rh), (torch.cat(outs), rx), (S[0], states[-1])):
        assert np.abs(f64(got) - ref).max() <= 7 * 2.0 ** -8 * np.abs(ref).max()
