"""Linear attention on the GPU where its numbers get large or small: factors of the outputs, values.  Bounds as in test_gpu_linattn."""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from test_gpu_linattn import BF16, F32, K, _check_prompt, _rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e9, -2.0 ** 100, 1e37, 1e-25, 2.0 ** -110])
@pytest.mark.parametrize("lens,dk,dtype", [([300], 64, BF16), ([20, 24], 128, BF16), ([300], 64, F32), ([1700], 32, BF16)])
def test_any_finite_factor_of_the_outputs(K, lens, dk, dtype, scale):  # noqa: F811
    """Blocks of 32 tokens that decay by 2^-99, and batches of 16 tokens that decay by 2^-23."""
    gen = torch.Generator().manual_seed(20)
    T, H = sum(lens), 2
    q, k, v, _ = _rows(T, H, H, dk, dk, dtype, gen)
    q, v = q.clone(), (0.03 * v).contiguous()              # outputs of a few units at most, the largest within bf16's range
    g = torch.tensor([-99 / 32 * np.log(2), -1.0], device="cuda", dtype=torch.float32)
    cu = np.cumsum([0] + lens).tolist()
    S0 = 0.03 * torch.randn(len(lens), H, dk, dk, generator=gen)
    # outputs as they are, and in the units of their factor: a power of two next to it, exact
    unit = 2.0 ** np.floor(np.log2(abs(scale)))
    o, S = K.kda_linattn_prefill(S0.cuda(), q, k, v, g, cu_seqlens=cu, scale=scale)
    for j, (a, b) in enumerate(zip(cu, cu[1:])):
        _check_prompt(o[a:b].double() / unit, S[j], f64(S0[j]), f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), f64(g), scale / unit, dtype)
    assert K.kda_device_errors() == 0


@pytest.mark.parametrize("rate", [0.05, 0.7, 1.0, 1.5, 1.7, 5.0])
@pytest.mark.parametrize("lens,dk,dv,dtype", [([200], 32, 64, F32), ([1500], 32, 32, F32), ([24, 17], 128, 128, BF16), ([90, 96], 32, 32, BF16),
                                              ([300], 64, 64, BF16)])
def test_states_of_any_size(K, lens, dk, dv, dtype, rate):  # noqa: F811
    """States, values and terms k v^T up to 2^85, and small ones, whatever they decay by."""
    gen = torch.Generator().manual_seed(21)
    T, H = sum(lens), 2
    q, k, v, _ = _rows(T, H, H, dk, dv, dtype, gen)
    cu = np.cumsum([0] + lens).tolist()
    g = torch.tensor([-rate, -1.01 * rate], device="cuda")
    S0 = torch.randn(len(lens), H, dk, dv, generator=gen)
    for up in (80, -40):                                    # |k v|, |S| within 2^5 of 2^up
        kk, vv, qq, s0 = k * 2.0 ** (up // 2), v * 2.0 ** (up - up // 2), q * 2.0 ** -up, S0 * 2.0 ** up
        o, S = K.kda_linattn_prefill(s0.cuda(), qq, kk, vv, g, cu_seqlens=cu)
        for j, (a, b) in enumerate(zip(cu, cu[1:])):
            _check_prompt(o[a:b], S[j].double() * 2.0 ** -up, f64(S0[j]), f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), f64(g), 1.0, dtype)
    assert K.kda_device_errors() == 0
