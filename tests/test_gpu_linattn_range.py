"""Linear attention on the GPU where its numbers get large, small or many: factors of the outputs, values near the ends of fp32's
range, decays that hardly decay over hundreds of chunks.

Bounds of single outputs and states: as in test_gpu_linattn.  Of a whole state, by its norm, for bf16 prompts on the tensor
cores: u = 2^-24; a chunk's 24 steps of 16 tokens (8 of tokens, each three parts) drop on average half a unit of the accumulator's 24 bits,
24 u; the state is rounded once a chunk, at random, sqrt(512) u / sqrt(3) = 13 u over the longest; a key's decay is the
product of two powers within 2 ulp each, rounded, 5 u; three parts of a decayed key leave u.  Together 43 u = 2.6e-6, within which a
factor between chunks that is off by one rounding, the same one every time, does not fit (6e-6 over 512 chunks), nor do keys of two
parts (test_linattn_parts: 9e-6).
"""
import numpy as np
import pytest
import torch

from kda_delta_rule_gb300.inputs import to_f64_numpy as f64
from test_gpu_linattn import BF16, F32, K, _check_prompt, _rows  # noqa: F401

pytestmark = pytest.mark.gpu
STATE_TOL = 43 * 2.0 ** -24


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


@pytest.mark.parametrize("lens", [[j % 5 for j in range(1300)] + [150], [1700], [9, 20]])
def test_a_power_of_two_multiplies_the_outputs_exactly(K, lens):  # noqa: F811
    """bf16, in more sequences than one launch takes, in segments, on CUDA cores alone; eagerly and captured."""
    gen = torch.Generator().manual_seed(25)
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, g = _rows(cu[-1], 1, 1, 64, 64, BF16, gen)

    def call(scale):
        return K.kda_linattn_prefill(None, q, k, v, g, cu_seqlens=cu, scale=scale)

    ref, S = call(1.0)
    for scale in (2.0 ** 40, -2.0 ** -40):
        o, S2 = call(scale)
        assert torch.equal(o.double(), ref.double() * scale) and torch.equal(S, S2)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o2, _ = call(scale)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, o)


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


def _state_error(q, k, v, g, S):
    """|S - exact| / |exact| for each head, against the sum over all tokens in fp64 on the GPU."""
    T = k.shape[0]
    w = torch.exp(g.double()[:, None] * torch.arange(T - 1, -1, -1, device="cuda"))           # (H, T)
    ref = (k.double().transpose(0, 1) * w[..., None]).transpose(1, 2) @ v.double().transpose(0, 1)
    return ((S.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)).tolist()


SLOW = [-1 / 3000, -1 / 8000, -1e-6, 0.0]


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 32), (128, 32), (64, 128)])
def test_states_are_as_good_as_three_parts_of_a_key(K, dk, dv, split):  # noqa: F811
    """bf16 prompts whose segments run at the same time, and which one CTA a head walks through."""
    gen = torch.Generator().manual_seed(22)
    T, H = 12000, len(SLOW)
    q, k, v, _ = _rows(T, H, H, dk, dv, BF16, gen)
    g = torch.tensor(SLOW, device="cuda")
    assert K.kda_linattn_prefill_workspace_bytes(None, T, H, dk, dv, BF16) > 0
    _, S = K.kda_linattn_prefill(None, q, k, v, g, workspace="auto" if split else None)
    assert max(_state_error(q, k, v, g, S[0])) <= STATE_TOL


def test_a_sequence_of_many_chunks_does_not_drift(K):  # noqa: F811
    """512 chunks one after another."""
    gen = torch.Generator().manual_seed(23)
    T, H, d = 65536, len(SLOW), 64
    q, k, v, _ = _rows(T, H, H, d, d, BF16, gen)
    g = torch.tensor(SLOW, device="cuda")
    _, S = K.kda_linattn_prefill(None, q, k, v, g, workspace=None)
    assert max(_state_error(q, k, v, g, S[0])) <= STATE_TOL


@pytest.mark.parametrize("split", [True, False])
def test_the_slowest_decays_count(K, split):  # noqa: F811
    """Fixed decays of 1e-10 a token are 1e-5 over 131072 of them: rounded to multiples of 2^-32, say, they would be off by half of that.
    1024 chunks' roundings of the state, sqrt(1024) u / sqrt(3) = 19 u in place of 13 u."""
    gen = torch.Generator().manual_seed(24)
    T, H, d = 131072, 4, 32
    q, k, v, _ = _rows(T, H, H, d, d, BF16, gen)
    g = torch.tensor([-0.49, -1.49, -0.3, -2.5], device="cuda") * 2.0 ** -32 * float(np.log(2))
    _, S = K.kda_linattn_prefill(None, q, k, v, g, workspace="auto" if split else None)
    assert max(_state_error(q, k, v, g, S[0])) <= STATE_TOL + 6 * 2.0 ** -24


@pytest.mark.parametrize("split", [True, False])
def test_states_of_fixed_decays_of_any_size(K, split):  # noqa: F811
    """On both sides of 2^(-1/4) a chunk, where its factor becomes one number."""
    gen = torch.Generator().manual_seed(26)
    rates = [1 / 60, 1 / 250, 1 / 500, 1 / 730, 1 / 745, 1 / 1000, 1 / 2000, 1 / 20000]
    T, H, d = 12000, len(rates), 64
    q, k, v, _ = _rows(T, H, H, d, d, BF16, gen)
    g = -torch.tensor(rates, device="cuda")
    _, S = K.kda_linattn_prefill(None, q, k, v, g, workspace="auto" if split else None)
    assert max(_state_error(q, k, v, g, S[0])) <= STATE_TOL


@pytest.mark.parametrize("dk,dv,B", [(32, 32, 1), (128, 128, 40)])
def test_many_steps_do_not_drift(K, dk, dv, B):  # noqa: F811
    """16384 tokens one after another, 16 a call, with fixed decays.  Each rounds the state twice, by up to u.  Roundings of neighbours are
    alike: what a decay of 1e-6 takes is some 17 2^-24 of the state, and a token changes the state by about a hundredth, so that what it takes moves by an eighth of
    the last place, and it is some 60 tokens until the rounding is another one: sqrt(64 T) u = 2^-14.  A factor rounded the same way for every
    token is off by up to 2^-25 T = 2^-11 (7e-4 was measured)."""
    gen = torch.Generator().manual_seed(27)
    T, H = 16384, len(SLOW)
    q, k, v, _ = _rows(T, H, H, dk, dv, BF16, gen)
    g = torch.tensor(SLOW, device="cuda")
    S = torch.zeros(B, H, dk, dv, device="cuda")
    per = [x.view(T // 16, 16, 1, H, -1) for x in (k, v)]
    for c in range(T // 16):
        kk, vv = (x[c].expand(16, B, H, x.shape[-1]).contiguous() for x in per)
        K.kda_linattn_step(S, kk, kk, vv, g)
    assert torch.equal(S, S[:1].expand_as(S))
    assert max(_state_error(q, k, v, g, S[0])) <= (64 * T) ** 0.5 * 2.0 ** -24
