"""What a decayed key loses as a sum of two or three bf16 numbers, on the CPU: the bound that the states of bf16 prompts are held to on
the GPU (test_gpu_linattn_range) lies between the two."""
import numpy as np
import pytest

BOUND = 43 * 2.0 ** -24                     # test_gpu_linattn_range's, of a whole state by its norm


def _bf16(x):
    u = x.astype(np.float32).view(np.uint32)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)


def _lead(x):
    return (x.view(np.uint32) & 0xffff0000).view(np.float32)


def _as_parts(x, n):
    """The leading bits, the leading bits of what they leave, and what those leave rounded; the first n of them."""
    hi = _lead(x)
    lo = _lead(x - hi)
    return sum(p.astype(np.float64) for p in (hi, lo, _bf16(x - hi - lo))[:n])


@pytest.mark.parametrize("g", [-1 / 3000, -1 / 8000, -1e-6])
def test_the_bound_lies_between_two_and_three_parts(g):
    r = np.random.default_rng(0)
    T, d = 4096, 64
    k, v = _bf16(r.standard_normal((T, d))), _bf16(r.standard_normal((T, d))).astype(np.float64)
    t = np.arange(T)
    here = np.exp(g * (127 - t % 128))       # from a token to its chunk's end, and on to the sequence's
    on = np.exp(g * (T - 1 - t)) / here
    x = k * here.astype(np.float32)[:, None]
    exact = (k * (here * on)[:, None]).T @ v
    two, three = (np.linalg.norm((_as_parts(x, n) * on[:, None]).T @ v - exact) / np.linalg.norm(exact) for n in (2, 3))
    assert two > 2 * BOUND and three < BOUND / 20


def test_one_rounded_factor_a_chunk_is_outside_the_bound():
    """The same fp32 factor after each of 512 chunks: the error grows with every one of them."""
    g, n = -1e-6, np.arange(511, -1, -1)
    exact = np.exp(128 * g * n)
    drift = float(np.float32(np.exp(128 * g))) ** n - exact
    assert np.linalg.norm(drift) / np.linalg.norm(exact) > 2 * BOUND
