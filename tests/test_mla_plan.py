"""Which attention kernels the tests' and the smoke check's shapes select, read off the workspace that a call asks for.

A call is one or two parts.  A part of n items of nr rows has n + 192 slots of nr rows (d_c sums and two statistics in fp32) and
two numbers an item, each array rounded to 256 bytes; nr is 16, 32 or 64 for the one-CTA kernel, 128 for the pair kernel.
"""
import pytest
import torch

import __graft_entry__ as entry
from test_gpu_mla_variants import VARIANTS


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import build
    build.build()
    from kda_delta_rule_gb300 import kda
    return kda


def _part(items, nr, d_c):
    return sum(-(-n // 256) * 256 for n in ((items + 192) * nr * d_c * 4, (items + 192) * nr * 8, items * 8))


def _plan(K, B, seq_rows, d_c, prefix):
    """(rows of the items with own tokens, where the prefix is) of a bf16 call."""
    def ask(prefix):
        return K.kda_mla_decode_workspace_bytes(B, 1, seq_rows, d_c, prefix, torch.bfloat16)

    need = ask(prefix)
    rows, found = B * seq_rows, []
    for nr in (16, 32, 64, 128):
        own = B * -(-seq_rows // nr)
        if prefix == 0 or nr == 128:
            found += [(nr, "joint" if prefix else "none")] * (need == _part(own, nr, d_c))
        if prefix:
            found += [(nr, "beside")] * (need == _part(own + -(-rows // nr), nr, d_c))
            found += [(nr, "pairs")] * (nr < 128 and need == _part(own, nr, d_c) + _part(-(-rows // 128), 128, d_c))
    # two plans may need the same; own tokens are the pair kernel's with a prefix where they are without one
    pairs = ask(0) == _part(B * -(-seq_rows // 128), 128, d_c)
    found = [f for f in found if (f[0] == 128) == pairs]
    assert len(found) == 1, found
    return found[0]


@pytest.mark.parametrize("name", VARIANTS)
def test_variants_are_what_they_say(K, name):
    B, n_q, H, d_c, _, _, prefix, _ = VARIANTS[name]
    nr, where = _plan(K, B, n_q * H, d_c, prefix)
    words = name.split(", ")
    if words[0] == "prefix by pairs":
        assert where == "pairs" and f"{nr} rows" == words[1]
    else:
        assert (nr == 128) if words[0] == "pair" else (f"{nr} rows" == words[0])
        assert where == ("joint" if "joint items" in name else "beside" if "prefix and own" in name else "none")


def test_smoke_reaches_every_attention_kernel(K):
    got = {(_plan(K, B, H, d_c, entry.MLA_PREFIX)[0], d_c % 256 > 0) for name, B, H, d_c in entry.MLA_SHAPES if name == "bf16"}
    assert {nr for nr, _ in got} == {16, 32, 64, 128} and {(128, False), (128, True)} <= got
    assert any(name == "f32" for name, *_ in entry.MLA_SHAPES)
