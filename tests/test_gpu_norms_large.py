"""The norms around a block on the GPU at the sizes of prompts, where a lane has two rows and a CTA walks over rows, and with gates far out;
against the fp64 oracle, with the bounds of test_gpu_norms."""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from oracle import kda_oracle as O
from test_gpu_norms import BF16, F32, K, ROUND, U, _act, _wide  # noqa: F401

pytestmark = pytest.mark.gpu


def _randn(*shape, gen, dtype):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


# rows of heads: just above 152 * 64 warps' rows, none a multiple of a CTA's rows, and just below
GATED = [(25943, 3, 32), (12973, 3, 64), (6487, 3, 128), (19457, 1, 80), (3243, 3, 256), (9729, 1, 264), (6485, 3, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("T,H,d", GATED)
def test_gated_norm_of_many_rows(K, T, H, d, per_head, first, dtype):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x, z = _randn(T, H, d, gen=gen, dtype=dtype), _randn(T, H, d, gen=gen, dtype=dtype)
    w = _randn(*((H, d) if per_head else (d,)), gen=gen, dtype=dtype)
    act = ["sigmoid", "silu", "none"][(T + per_head) % 3]
    y = K.kda_gated_norm(_wide(x), w, gate=_wide(z), act=_act(K, act), gate_first=first)
    ref = O.gated_norm(f64(x), f64(w), f64(z), 1e-6, act, first)
    assert np.all(np.abs(f64(y) - ref) <= ((d / 2 + 40) * U + ROUND[dtype]) * np.abs(ref))
    y = K.kda_gated_norm(x, w)                              # no gate
    ref = O.gated_norm(f64(x), f64(w))
    assert np.all(np.abs(f64(y) - ref) <= ((d / 2 + 40) * U + ROUND[dtype]) * np.abs(ref))


# rows of one warp, of several, two and four vectors a thread: more rows than the CTAs of all SMs take at once
RESIDUAL = [(40003, 64), (20001, 256), (10007, 264), (8009, 512), (5003, 2000), (1501, 4096), (1003, 4104), (1003, 6144), (701, 8192), (407, 16384)]


@pytest.mark.parametrize("dtype,h_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("parts", ["", "pgc"])
@pytest.mark.parametrize("T,D", RESIDUAL)
def test_residual_norm_of_many_rows(K, T, D, parts, dtype, h_dtype):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    h, y, z = _randn(T, D, gen=gen, dtype=h_dtype), _randn(T, D, gen=gen, dtype=dtype), _randn(T, D, gen=gen, dtype=dtype)
    pre, post, cs = (_randn(D, gen=gen, dtype=dtype) for _ in range(3))
    kw = {"post_weight": post, "gate": z, "channel_scale": cs} if parts else {}
    act = ["sigmoid", "silu", "none"][(T + D) % 3]
    rh, rx = O.residual_norm(f64(h), f64(y), f64(pre), **{a: f64(t) for a, t in kw.items()}, res_scale=0.6, act=act)
    if parts:
        kw["gate"] = _wide(z)
    to = torch.empty_like(h)
    before = h.clone()
    h2, x2 = K.kda_residual_norm(h, _wide(y), pre, res_scale=0.6, act=_act(K, act), h_out=to, **kw)
    assert h2 is to and torch.equal(h, before)
    few = (D / 2 + 40) * U
    h_err = few * np.abs(rh - f64(h)) + U * np.abs(rh)
    assert np.all(np.abs(f64(h2) - rh) <= h_err + ROUND[h_dtype] * np.abs(rh) + 1e-30)
    r = np.sqrt(np.mean(rh ** 2, -1, keepdims=True) + 1e-6)
    shift = np.sqrt(np.mean(h_err ** 2, -1, keepdims=True)) / r
    assert np.all(np.abs(f64(x2) - rx) <= h_err / r * np.abs(f64(pre)) + (shift + few + ROUND[dtype]) * np.abs(rx) + 1e-30)
    h3, x3 = K.kda_residual_norm(h, _wide(y), pre, res_scale=0.6, act=_act(K, act), **kw)       # in place
    assert h3 is h and torch.equal(h, to) and torch.equal(x3, x2)
