"""Gates far out in the norms around a block, against the fp64 oracle.

Bounds, with u = 2^-24: the hardware's exponential of half the gate is within 2^-22, 4 u, and rounded once more; its square, 10 u; 1 + t,
u; the reciprocal within 2^-23, 2 u; four products and a sum, u each: together 18 u however far out the gate is, besides what test_gpu_norms
has for the norm.  bf16 outputs are good to their own rounding, with 2^-15 for an exponent rounded to 24 bits.  What is left of
a sigmoid below -87.3 is no subnormal number before the last product, so that one alone rounds to those, 2^-149."""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from oracle import kda_oracle as O
from test_gpu_norms import BF16, F32, K, ROUND, U, _act  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = {BF16: 2.0 ** -15, F32: 0.0}
Z = [0.0, -0.0, 1e-30, -3e-3, 1.0, 15.0, 16.64, 17.4, 60.0, 88.0, 90.0, 3e4, -1.0, -15.0, -16.64, -40.0, -79.9, -80.0, -86.5, -87.2, -87.35,
     -87.9, -88.5, -89.5, -92.0, -96.0, -100.0, -103.0, -110.0, -3e4, 3e38, -3e38]


def _gates(dtype, gen):
    z = torch.cat([torch.tensor(Z), 103 * torch.rand(480, generator=gen) * torch.randn(480, generator=gen).sign()]).to(dtype)
    return z, f64(z)


def _act64(z, act):
    with np.errstate(over="ignore"):
        return O.gate_of(z, act)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_norm(K, dtype, act):  # noqa: F811
    gen = torch.Generator().manual_seed(30)
    z, z64 = _gates(dtype, gen)
    d = len(z)
    x = torch.randn(3, 1, d, generator=gen).to(dtype)
    w = (1e12 * (1 + torch.rand(d, generator=gen))).to(dtype)   # so that products with subnormal factors are none
    y = K.kda_gated_norm(x.cuda(), w.cuda(), gate=z.expand(3, 1, d).contiguous().cuda(), act=_act(K, act))
    f = _act64(z64, act)
    plain = O.rms(f64(x), 1e-6) * f64(w)
    ref = plain * f
    big = np.abs(ref) > 3.3e38                              # these overflow
    err = np.abs(f64(y) - ref)
    assert np.all(((err <= ((d / 2 + 18) * U + ROUND[dtype] + FAR[dtype]) * np.abs(ref) + 1e-40) | big))


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_residual_norm(K, dtype, act):  # noqa: F811
    """The block's output alone: h starts at zero and is kept in fp32."""
    gen = torch.Generator().manual_seed(31)
    z, z64 = _gates(dtype, gen)
    z, z64 = z[np.abs(z64) < 4e4], z64[np.abs(z64) < 4e4]
    z, z64 = z[:len(z) // 8 * 8], z64[:len(z) // 8 * 8]
    D = len(z)
    y = (1e12 * torch.randn(2, D, generator=gen)).to(dtype)
    h = torch.zeros(2, D, device="cuda")
    K.kda_residual_norm(h, y.cuda(), torch.ones(D, dtype=dtype, device="cuda"), gate=z.expand(2, D).contiguous().cuda(), act=_act(K, act))
    ref = f64(y) * _act64(z64, act)
    assert np.all(np.abs(f64(h) - ref) <= 18 * U * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fp32_gates_keep_their_bits(K, dtype):  # noqa: F811
    """A gate's exponential is as good at -80 as at -1: the factor alone, by a row of ones."""
    z = torch.linspace(-86, 88, 1024).to(dtype)
    x, w = torch.ones(1, 1, 1024, dtype=dtype, device="cuda"), torch.ones(1024, dtype=dtype, device="cuda")
    for act in ("sigmoid", "silu"):
        y = K.kda_gated_norm(x, w, gate=z.view(1, 1, -1).cuda(), eps=0.0, act=_act(K, act))
        ref = _act64(f64(z), act)
        assert np.all(np.abs(f64(y)[0, 0] - ref) <= (18 * U + ROUND[dtype] + FAR[dtype]) * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_gates(K, dtype):  # noqa: F811
    """A gate of -infinity closes, one of infinity opens; one that is NaN is seen."""
    inf = float("inf")
    z = torch.tensor([inf, -inf, 0.0, 4e2, -4e2, 1.0, -1.0, 2.0], dtype=dtype, device="cuda").repeat(4)
    x = torch.full((2, 1, 32), 3.0, dtype=dtype, device="cuda")
    one = torch.ones(32, dtype=dtype, device="cuda")
    gate = z.expand(2, 1, 32).contiguous()
    gate[1, 0, 5] = float("nan")
    ref = 1 / (1 + np.exp(-f64(z)))
    with np.errstate(over="ignore"):
        y = f64(K.kda_gated_norm(x, one, gate=gate, eps=0.0))[:, 0]
    h = torch.zeros(2, 32, device="cuda")
    K.kda_residual_norm(h, one.expand(2, 32).contiguous(), one, gate=gate[:, 0])
    # e^-400 = 1.9e-174 is below fp32's smallest number, 2^-149
    for got, tol in ((y, 18 * U + ROUND[dtype]), (f64(h), 18 * U)):
        assert np.all(np.abs(got[0] - ref) <= tol * ref + 2.0 ** -149) and np.isnan(got[1, 5]) and np.isfinite(np.delete(got[1], 5)).all()
    y = f64(K.kda_gated_norm(x, one, gate=gate, eps=0.0, act=K.ACT_SILU))[0, 0]
    assert np.all(np.isposinf(y[0::8])) and np.all(np.isfinite(y[2::8]))
