"""Refusals of the latent page cache's entry points: every call here fails in the host's checks,
before any launch, so fake device pointers are never read."""
import ctypes
import math

import pytest

ARG, SHAPE, DTYPE, ALIGN, ALIAS = -1, -2, -3, -4, -7
G = 1 << 30


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import build
    build.build()
    from kda_delta_rule_gb300 import kda
    return kda


def _v(x):
    return None if x is None else ctypes.c_void_p(x)


def _append(K, **kw):
    a = dict(pages=G, page_bytes=512 * 1152, n_pages=4, page_tokens=512, slots=2 * G, positions=3 * G, rope=4 * G, n_pos=100,
             c=5 * G, c_stride=576, k_pe=5 * G + 1024, k_pe_stride=576, norm=6 * G, eps=1e-6, q=7 * G, qst=32 * 192, qsh=192,
             q_out=8 * G, T=3, H=32, d_c=512, d_r=64, dtype=K.KDA_BF16, style=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return K._lib.kda_mla_append(_v(a["pages"]), a["page_bytes"], a["n_pages"], a["page_tokens"], _v(a["slots"]),
                                 _v(a["positions"]), _v(a["rope"]), a["n_pos"], _v(a["c"]), a["c_stride"], _v(a["k_pe"]),
                                 a["k_pe_stride"], _v(a["norm"]), a["eps"], _v(a["q"]), a["qst"], a["qsh"], _v(a["q_out"]),
                                 a["T"], a["H"], a["d_c"], a["d_r"], a["dtype"], a["style"], None)


def _decode(K, **kw):
    a = dict(q=G, q_pe=2 * G, pages=3 * G, page_bytes=512 * 1152, n_pages=4, page_tokens=512, pp=4 * G, prefix=100, table=5 * G,
             max_pages=3, lens=6 * G, scale=0.1, o=7 * G, lse=8 * G, B=2, n_q=1, H=32, d_c=512, d_r=64, dtype=K.KDA_BF16,
             ws=16 * G, ws_bytes=G)
    assert set(kw) <= set(a)
    a.update(kw)
    return K._lib.kda_mla_decode(_v(a["q"]), _v(a["q_pe"]), _v(a["pages"]), a["page_bytes"], a["n_pages"], a["page_tokens"],
                                 _v(a["pp"]), a["prefix"], _v(a["table"]), a["max_pages"], _v(a["lens"]), a["scale"],
                                 _v(a["o"]), _v(a["lse"]), a["B"], a["n_q"], a["H"], a["d_c"], a["d_r"], a["dtype"],
                                 _v(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), DTYPE), (dict(d_c=500), SHAPE), (dict(d_c=640), SHAPE), (dict(d_r=8), SHAPE), (dict(d_r=80), SHAPE),
    (dict(T=-1), SHAPE), (dict(H=-1), SHAPE), (dict(style=2), ARG), (dict(pages=None), ARG), (dict(pages=G + 8), ALIGN),
    (dict(page_tokens=24), SHAPE), (dict(page_tokens=0), SHAPE), (dict(page_bytes=512 * 1152 - 16), SHAPE),
    (dict(page_bytes=512 * 1152 + 8), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 30), SHAPE), (dict(slots=None), ARG),
    (dict(c=None), ARG), (dict(k_pe=None), ARG), (dict(positions=None), ARG), (dict(rope=None), ARG), (dict(n_pos=0), SHAPE),
    (dict(c_stride=504), SHAPE), (dict(c_stride=580), SHAPE), (dict(k_pe_stride=60), SHAPE), (dict(eps=-1.0), ARG),
    (dict(eps=math.nan), ARG), (dict(q_out=None), ARG), (dict(qsh=32), SHAPE), (dict(qst=191), SHAPE), (dict(qst=192), SHAPE),
    (dict(c=5 * G + 4), ALIGN), (dict(q=7 * G + 2), ALIGN), (dict(norm=6 * G + 2), ALIGN), (dict(d_r=0), ARG),
    (dict(c=G + 1152), ALIAS), (dict(q_out=5 * G), ALIAS), (dict(q_out=G), ALIAS), (dict(q_out=7 * G), ALIAS),
])
def test_append_refusals(K, kw, status):
    assert _append(K, **kw) == status
    assert K._lib.kda_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(d_c=64), SHAPE), (dict(d_r=24), SHAPE), (dict(B=-1), SHAPE), (dict(H=-3), SHAPE),
    (dict(n_q=0), SHAPE), (dict(n_q=17), SHAPE), (dict(B=1 << 20, H=1 << 12), SHAPE), (dict(prefix=-1), SHAPE),
    (dict(prefix=1 << 31), SHAPE), (dict(page_tokens=8), SHAPE), (dict(page_bytes=1152), SHAPE), (dict(n_pages=0), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=math.inf), ARG),
    (dict(scale=math.nan), ARG), (dict(q=None), ARG), (dict(q_pe=None), ARG), (dict(pages=None), ARG), (dict(pp=None), ARG),
    (dict(table=None), ARG), (dict(lens=None), ARG), (dict(o=None), ARG), (dict(ws=None), ARG), (dict(ws_bytes=1000), SHAPE),
    (dict(ws=16 * G + 16), ALIGN), (dict(q=G + 4), ALIGN), (dict(o=7 * G + 8), ALIGN), (dict(q_pe=2 * G + 2), ALIGN),
    (dict(o=G), ALIAS), (dict(o=3 * G), ALIAS), (dict(lse=7 * G), ALIAS), (dict(ws=G), ALIAS), (dict(lse=6 * G), ALIAS),
])
def test_decode_refusals(K, kw, status):
    assert _decode(K, **kw) == status
    assert K._lib.kda_last_error()


def test_nothing_to_do(K):
    assert _append(K, T=0) == 0
    assert _decode(K, B=0) == 0 and _decode(K, H=0) == 0


def test_workspace_bytes(K):
    import torch
    f = K.kda_mla_decode_workspace_bytes
    one = f(1, 1, 32, 512, 0, torch.bfloat16)
    assert one > 0 and one % 256 == 0
    assert f(64, 1, 32, 512, 0, torch.bfloat16) > one
    assert f(64, 1, 32, 512, 100, torch.bfloat16) > f(64, 1, 32, 512, 0, torch.bfloat16)
    assert f(0, 1, 32, 512, 0, torch.bfloat16) == 0
    with pytest.raises(K.KdaError):
        f(1, 99, 32, 512, 0, torch.bfloat16)
    with pytest.raises(K.KdaError):
        f(1, 1, 32, 100, 0, torch.float32)


def test_binding_refuses_host_tensors(K):
    import torch
    with pytest.raises(TypeError):
        K.kda_mla_append(torch.zeros(1, 64, dtype=torch.uint8), 16, None, None, None, torch.zeros(1, 128), None)
    with pytest.raises(TypeError):
        K.kda_mla_decode(torch.zeros(1, 1, 1, 128), None, None, 16, None, None, 1.0)


@pytest.mark.parametrize("T,H,qst,qsh", [(3, 32, 32 * 64, 64), (1, 32, 0, 64), (1, 32, 192 * 32, 64), (3, 1, 64, 0), (3, 1, 64, 192),
                                         (1, 1, 0, 0), (1, 1, 64, 64)])
def test_append_in_place_strides_of_one_entry_say_nothing(K, T, H, qst, qsh):
    """Dense queries rotated in place are no overlap, whatever the stride of an axis of one entry. The queries lie in the
    pages here, so that a call that takes them as in place is refused for that, and none is launched."""
    assert _append(K, T=T, H=H, q=G, q_out=G, qst=qst, qsh=qsh) == ALIAS
    assert b"q_pe_out overlaps the pages" in K._lib.kda_last_error()


@pytest.mark.parametrize("T,H,qst,qsh", [(3, 32, 32 * 64 + 8, 64), (1, 32, 0, 72), (3, 1, 72, 64)])
def test_append_in_place_of_queries_that_are_not_dense_is_an_overlap(K, T, H, qst, qsh):
    assert _append(K, T=T, H=H, q=7 * G, q_out=7 * G, qst=qst, qsh=qsh) == ALIAS
    assert b"an output overlaps an input" in K._lib.kda_last_error()


@pytest.mark.parametrize("through_ctypes", [False, True])
def test_binding_refuses_tensors_of_another_device(K, through_ctypes):
    """With fake tensors: they have a device, no memory, and need no GPU."""
    import numpy as np
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    if torch.cuda.is_available() and torch.cuda.device_count() < 2:
        pytest.skip("with a GPU, fake tensors are made on devices that are there alone")
    i32, bf16 = torch.int32, torch.bfloat16
    page = np.int64(16) if through_ctypes else 16

    def fake(shapes, elsewhere):
        with FakeTensorMode():
            return {n: torch.empty(s, dtype=t, device="cuda:1" if n == elsewhere else "cuda:0") for n, (s, t) in shapes.items()}

    append = dict(pages=((4, 16 * 144 * 2), torch.uint8), slots=((3,), i32), positions=((3,), i32), rope=((9, 16), torch.float32),
                  c=((3, 128), bf16), k_pe=((3, 16), bf16), q_pe=((3, 4, 16), bf16), q_pe_out=((3, 4, 16), bf16), norm_weight=((128,), bf16))
    for name in append:
        with pytest.raises(ValueError, match="is on cuda:" + ("0" if name == "c" else "1")):
            K.kda_mla_append(page_tokens=page, stream=0, **fake(append, name))
    decode = dict(q=((2, 1, 4, 128), bf16), q_pe=((2, 1, 4, 16), bf16), pages=((4, 16 * 144 * 2), torch.uint8), page_table=((2, 3), i32),
                  lens=((2,), i32), prefix_pages=((1,), i32), o=((2, 1, 4, 128), bf16), lse=((2, 1, 4), torch.float32), workspace=((1 << 20,), torch.uint8))
    for name in decode:
        with pytest.raises(ValueError, match="is on cuda:" + ("0" if name == "q" else "1")):
            K.kda_mla_decode(page_tokens=page, scale=0.1, prefix_len=10, stream=0, **fake(decode, name))


@pytest.mark.parametrize("T,H,qst,qsh,taken", [(3, 32, 64, 192, True), (3, 32, 72, 208, True), (3, 32, 64, 184, False), (3, 32, 56, 192, False),
                                               (2, 2, 64, 64, False)])
def test_append_takes_queries_head_by_head(K, T, H, qst, qsh, taken):
    """(H, T, d_r) in memory, as a matrix product per head leaves them; tokens that overlap are refused. q_pe_out overlaps the
    pages, so that none is launched."""
    assert _append(K, T=T, H=H, qst=qst, qsh=qsh, q_out=G) == (ALIAS if taken else SHAPE)


@pytest.mark.parametrize("scale,status", [(3e38, ARG), (2.4e38, ARG), (2.3e38, ALIAS)])
def test_decode_scale_in_log2_units_is_finite(K, scale, status):
    """Scores are taken times log2(e), which has to fit fp32, too. o overlaps q, so that none is launched."""
    assert _decode(K, scale=scale, o=G) == status
