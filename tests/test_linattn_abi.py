"""Refusals of linear attention's entry points and of the norms': every call here fails in the host's checks, before any
launch, so fake device pointers are never read."""
import ctypes
import math

import pytest

ARG, SHAPE, DTYPE, ALIGN, ALIAS = -1, -2, -3, -4, -7
G = 1 << 32


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import build
    build.build()
    from kda_delta_rule_gb300 import kda
    return kda


def _v(x):
    return None if x is None else ctypes.c_void_p(x)


def _merge(a, kw):
    assert set(kw) <= set(a)
    return {**a, **kw}


def _step(K, **kw):
    a = _merge(dict(S=G, to=G, n_slots=9, si=2 * G, so=None, q=3 * G, qs=4096, k=4 * G, ks=4096, v=5 * G, vs=4096, g=6 * G, gs=32, n=None,
                    scale=0.1, o=7 * G, steps=2, B=4, H=32, H_k=32, dk=128, dv=128, dtype=K.KDA_BF16), kw)
    return K._lib.kda_linattn_step(_v(a["S"]), _v(a["to"]), a["n_slots"], _v(a["si"]), _v(a["so"]), _v(a["q"]), a["qs"], _v(a["k"]), a["ks"],
                                   _v(a["v"]), a["vs"], _v(a["g"]), a["gs"], _v(a["n"]), a["scale"], _v(a["o"]), a["steps"], a["B"], a["H"],
                                   a["H_k"], a["dk"], a["dv"], a["dtype"], None)


def _prefill(K, **kw):
    a = _merge(dict(S0=G, q=3 * G, qs=4096, k=4 * G, ks=4096, v=5 * G, vs=4096, g=6 * G, gs=32, cu=[0, 300, 1000], T=1000, H=32, H_k=32,
                    dk=128, dv=128, dtype=K.KDA_BF16, scale=0.1, stride=128, o=7 * G, Sf=8 * G, pool=9 * G, page_bytes=32 << 16,
                    ids=10 * G, pos=None, n_ck=7, ws=None, ws_bytes=0), kw)
    cu = a["cu"]
    arr = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
    return K._lib.kda_linattn_prefill(_v(a["S0"]), _v(a["q"]), a["qs"], _v(a["k"]), a["ks"], _v(a["v"]), a["vs"], _v(a["g"]), a["gs"], arr,
                                      1 if cu is None else len(cu) - 1, a["T"], a["H"], a["H_k"], a["dk"], a["dv"], a["dtype"], a["scale"],
                                      a["stride"], _v(a["o"]), _v(a["Sf"]), _v(a["pool"]), a["page_bytes"], _v(a["ids"]), _v(a["pos"]),
                                      a["n_ck"], _v(a["ws"]), a["ws_bytes"], None)


def _gated(K, **kw):
    a = _merge(dict(x=G, xs=4096, z=2 * G, zs=8192, w=3 * G, ws=0, eps=1e-6, act=2, first=0, y=4 * G, T=5, H=32, d=128, dtype=K.KDA_BF16), kw)
    return K._lib.kda_gated_norm(_v(a["x"]), a["xs"], _v(a["z"]), a["zs"], _v(a["w"]), a["ws"], a["eps"], a["act"], a["first"], _v(a["y"]),
                                 a["T"], a["H"], a["d"], a["dtype"], None)


def _residual(K, **kw):
    a = _merge(dict(y=G, ys=4096, z=2 * G, zs=8192, post=3 * G, cs=4 * G, rs=0.5, hi=5 * G, ho=5 * G, hs=4096, hd=K.KDA_F32, pre=6 * G,
                    eps=1e-6, act=2, x=7 * G, T=5, D=4096, dtype=K.KDA_BF16), kw)
    return K._lib.kda_residual_norm(_v(a["y"]), a["ys"], _v(a["z"]), a["zs"], _v(a["post"]), _v(a["cs"]), a["rs"], _v(a["hi"]), _v(a["ho"]),
                                    a["hs"], a["hd"], _v(a["pre"]), a["eps"], a["act"], _v(a["x"]), a["T"], a["D"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), DTYPE), (dict(dk=48), SHAPE), (dict(dv=256), SHAPE), (dict(H=-1), SHAPE), (dict(H=1 << 14), SHAPE), (dict(H_k=5), SHAPE),
    (dict(H_k=0), SHAPE), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(B=-1), SHAPE), (dict(steps=0), SHAPE),
    (dict(steps=17), SHAPE), (dict(B=1 << 26), SHAPE), (dict(n_slots=0), SHAPE), (dict(n_slots=1 << 40), SHAPE), (dict(si=None, n_slots=3), SHAPE),
    (dict(S=None), ARG), (dict(o=None), ARG), (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(g=None), ARG),
    (dict(qs=4088), SHAPE), (dict(ks=4100), SHAPE), (dict(vs=0), SHAPE), (dict(vs=1 << 33), SHAPE), (dict(gs=31), SHAPE), (dict(gs=-32), SHAPE),
    (dict(q=3 * G + 2), ALIGN), (dict(v=5 * G + 8), ALIGN), (dict(g=6 * G + 2), ALIGN), (dict(S=G + 4, to=G + 4), ALIGN), (dict(o=7 * G + 8), ALIGN),
    (dict(o=G), ALIAS), (dict(o=3 * G), ALIAS), (dict(to=G + 128), ALIAS), (dict(to=3 * G), ALIAS), (dict(o=2 * G), ALIAS), (dict(o=6 * G), ALIAS),
    (dict(to=None, o=G + 4096), ALIAS), (dict(n=7 * G), ALIAS),
])
def test_step_refusals(K, kw, status):
    assert _step(K, **kw) == status
    assert K._lib.kda_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), DTYPE), (dict(dk=16), SHAPE), (dict(H_k=7), SHAPE), (dict(scale=math.inf), ARG), (dict(T=-1), SHAPE), (dict(T=1001), SHAPE),
    (dict(T=1 << 31, cu=None), SHAPE), (dict(T=0x7fff0001, cu=None), SHAPE), (dict(T=0x7fffffff, cu=[0, 0x7fffffff]), SHAPE), (dict(cu=[0, 600, 300, 1000]), SHAPE), (dict(cu=[1, 1000]), SHAPE), (dict(cu=[0]), SHAPE), (dict(stride=64), SHAPE),
    (dict(stride=-128), SHAPE), (dict(Sf=None), ARG), (dict(S0=G + 8), ALIGN), (dict(q=None), ARG), (dict(g=None), ARG), (dict(o=None), ARG),
    (dict(o=7 * G + 4), ALIGN), (dict(qs=4095), SHAPE), (dict(gs=16), SHAPE), (dict(n_ck=6), SHAPE), (dict(pool=None), ARG), (dict(ids=None), ARG),
    (dict(pool=9 * G + 8), ALIGN), (dict(page_bytes=(32 << 16) - 16), SHAPE), (dict(page_bytes=(32 << 16) + 8), SHAPE),
    (dict(Sf=G), ALIAS), (dict(Sf=G + (1 << 21)), ALIAS), (dict(o=5 * G), ALIAS), (dict(Sf=7 * G), ALIAS), (dict(o=10 * G), ALIAS),
    (dict(ws=11 * G + 64, ws_bytes=1 << 30), ALIGN), (dict(ws=G, ws_bytes=1 << 30), ALIAS), (dict(ws=7 * G, ws_bytes=1 << 30), ALIAS),
    (dict(H=1, H_k=1, cu=None, T=65536, qs=128, ks=128, vs=128, gs=1, n_ck=512, ws=12 * G, ws_bytes=1 << 16), SHAPE),
])
def test_prefill_refusals(K, kw, status):
    assert _prefill(K, **kw) == status
    assert K._lib.kda_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(d=0), SHAPE), (dict(d=132), SHAPE), (dict(d=1032), SHAPE), (dict(H=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(act=3), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(x=None), ARG), (dict(w=None), ARG),
    (dict(y=None), ARG), (dict(first=2), ARG), (dict(ws=64), SHAPE), (dict(xs=4088), SHAPE), (dict(zs=4100), SHAPE), (dict(x=G + 8), ALIGN),
    (dict(z=2 * G + 2), ALIGN), (dict(w=3 * G + 4), ALIGN), (dict(y=G + 16), ALIAS), (dict(y=2 * G), ALIAS), (dict(y=3 * G), ALIAS),
    (dict(y=G, xs=8192), ALIAS),
])
def test_gated_norm_refusals(K, kw, status):
    assert _gated(K, **kw) == status
    assert K._lib.kda_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(hd=2), DTYPE), (dict(dtype=0, hd=1), DTYPE), (dict(D=0), SHAPE), (dict(D=4100), SHAPE), (dict(D=16392), SHAPE),
    (dict(T=-1), SHAPE), (dict(act=-1), ARG), (dict(eps=math.inf), ARG), (dict(rs=math.nan), ARG), (dict(y=None), ARG), (dict(hi=None), ARG),
    (dict(ho=None), ARG), (dict(pre=None), ARG), (dict(x=None), ARG), (dict(ys=4095), SHAPE), (dict(zs=4000), SHAPE), (dict(hs=4098), SHAPE),
    (dict(post=3 * G + 2), ALIGN), (dict(ho=5 * G + 4), ALIGN), (dict(x=G), ALIAS), (dict(ho=G), ALIAS), (dict(ho=5 * G + 16), ALIAS),
    (dict(x=5 * G), ALIAS), (dict(ho=7 * G), ALIAS), (dict(x=6 * G), ALIAS), (dict(x=2 * G), ALIAS),
])
def test_residual_norm_refusals(K, kw, status):
    assert _residual(K, **kw) == status
    assert K._lib.kda_last_error()


def test_nothing_to_do(K):
    assert _step(K, B=0) == 0 and _step(K, H=0) == 0
    assert _prefill(K, H=0) == 0
    assert _gated(K, T=0) == 0 and _gated(K, H=0) == 0
    assert _residual(K, T=0) == 0


def test_strides_of_a_single_row_say_nothing(K):
    """Their outputs overlap an input, so that none is launched."""
    assert _step(K, steps=1, B=1, qs=0, ks=3, vs=-1, gs=7, o=G) == ALIAS
    assert _gated(K, T=1, xs=0, zs=1, y=3 * G) == ALIAS
    assert _residual(K, T=1, ys=0, zs=1, hs=2, x=G) == ALIAS


def test_prefill_workspace_bytes(K):
    import torch
    f = K.kda_linattn_prefill_workspace_bytes
    bf16 = torch.bfloat16
    assert f(None, 100, 1, 128, 128, bf16) == 0                           # one chunk: nothing to split
    assert f([64 * i for i in range(257)], 256 * 64, 32, 128, 128, bf16) == 0  # many sequences fill the GPU as they are
    few = f(None, 65536, 4, 128, 128, bf16)
    assert few > 0 and few % 256 == 0
    # a segment's state for each of the SMs, not more than a few for each
    assert few <= 4 * 152 * 128 * 128 * 4
    assert f(None, 0, 4, 128, 128, bf16) == 0 and f(None, 4096, 0, 128, 128, bf16) == 0
    with pytest.raises(K.KdaError):
        f([0, 5, 3], 3, 4, 128, 128, bf16)
    with pytest.raises(K.KdaError):
        f(None, 100, 4, 100, 128, bf16)


def test_binding_refuses_host_tensors(K):
    import torch
    x = torch.zeros(2, 3, 32)
    with pytest.raises(TypeError):
        K.kda_linattn_step(torch.zeros(2, 3, 32, 32), x, x, x, torch.zeros(2, 3))
    with pytest.raises(TypeError):
        K.kda_linattn_prefill(None, x, x, x, torch.zeros(2, 3))
    with pytest.raises(TypeError):
        K.kda_gated_norm(x, torch.zeros(32))
    with pytest.raises(TypeError):
        K.kda_residual_norm(torch.zeros(2, 64), torch.zeros(2, 64), torch.zeros(64))


def test_binding_refuses_tensors_of_another_device(K):
    """With fake tensors: they have a device, no memory, and need no GPU."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    if torch.cuda.is_available() and torch.cuda.device_count() < 2:
        pytest.skip("with a GPU, fake tensors are made on devices that are there alone")
    i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32

    def refused(call, first, shapes, **kw):
        for name in shapes:
            with FakeTensorMode():
                t = {n: torch.empty(s, dtype=d, device="cuda:1" if n == name else "cuda:0") for n, (s, d) in shapes.items()}
            with pytest.raises(ValueError, match="is on cuda:" + ("0" if name == first else "1")):
                call(stream=0, **t, **kw)

    head = ((2, 4, 32), bf16)
    refused(K.kda_linattn_step, "v", dict(S=((5, 4, 32, 32), f32), q=head, k=head, v=head, g=((2, 4), f32), o=head, S_new=((5, 4, 32, 32), f32),
                                          slot_in=((2,), i32), slot_out=((2,), i32), n_accepted=((2,), i32)))
    refused(K.kda_linattn_prefill, "v", dict(S0=((1, 4, 32, 32), f32), q=head, k=head, v=head, g=((2, 4), f32), o=head, S_final=((1, 4, 32, 32), f32),
                                             page_pool=((2, 1 << 14), torch.uint8), ckpt_page_ids=((1,), i32), ckpt_pos=((1,), i32),
                                             workspace=((256,), torch.uint8)))
    refused(K.kda_gated_norm, "x", dict(x=head, weight=((32,), bf16), gate=head, y=head))
    row, w = ((2, 64), bf16), ((64,), bf16)
    refused(K.kda_residual_norm, "y", dict(h=row, y=row, pre_weight=w, post_weight=w, gate=row, channel_scale=w, h_out=row, x=row))
