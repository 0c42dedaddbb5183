"""Linear attention's checkpoint positions are an output like the others: where they would be written over something that the call reads
or writes, it is refused before any launch (fake device pointers are never read)."""
import pytest

from test_linattn_abi import ALIAS, ALIGN, G, K, _prefill, _step  # noqa: F401


@pytest.mark.parametrize("at", [10 * G, 10 * G + 24, 10 * G - 24, G, 3 * G, 6 * G, 7 * G + 4096, 8 * G, 12 * G])
def test_positions_over_another_array_are_refused(K, at):  # noqa: F811
    """Over the page ids above all: a page number read after a position had taken its place would be one outside the arena."""
    assert _prefill(K, pos=at, ws=12 * G, ws_bytes=1 << 30) == ALIAS


@pytest.mark.parametrize("call,kw", [(_prefill, dict(pos=11 * G + 2)), (_prefill, dict(ids=10 * G + 1)), (_step, dict(si=2 * G + 2)),
                                     (_step, dict(so=8 * G + 1)), (_step, dict(n=9 * G + 3))])
def test_integers_that_are_not_aligned_are_refused(K, call, kw):  # noqa: F811
    assert call(K, **kw) == ALIGN
