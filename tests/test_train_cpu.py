"""The training form's calls on a machine without a GPU: sizes, and the
refusals, which come from the host before anything is launched."""
import ctypes

import pytest
import torch

import mxfp4_mixture_experts_02_gb300 as moe
from mxfp4_mixture_experts_02_gb300 import train

NULL, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4


def norm(**kw):
    return ctypes.byref(train._NormShape(**{**dict(rows=4, cols=64, dtype=0, w_dtype=2, eps=1e-5), **kw}))


def tokens(**kw):
    base = dict(T=4, E_global=8, E_local=8, expert_offset=0, top_k=2, num_shared=0, hidden=64, dtype=0)
    return ctypes.byref(train._TokenShape(**{**base, **kw}))


BAD_NORM = [dict(dtype=3), dict(dtype=-1), dict(w_dtype=1), dict(dtype=2, w_dtype=0), dict(rows=-1), dict(cols=0),
            dict(rows=(1 << 30) + 1), dict(cols=(1 << 20) + 1), dict(eps=-1.0), dict(eps=float("nan")),
            dict(eps=float("inf"))]
BAD_TOKENS = [dict(dtype=3), dict(hidden=0), dict(hidden=(1 << 20) + 1), dict(top_k=0), dict(top_k=9), dict(T=-1),
              dict(top_k=33, E_global=64), dict(E_global=1025), dict(num_shared=2),
              dict(num_shared=-1), dict(E_local=0), dict(E_global=1024, E_local=1024, num_shared=1),
              dict(expert_offset=-1), dict(expert_offset=1), dict(T=1 << 23), dict(expert_offset=2 ** 31 - 1)]


@pytest.mark.parametrize("kw", BAD_NORM)
def test_norm_shapes_refused(kw):
    L = moe.lib()
    assert L.moe_layer_norm(norm(**kw), 256, None, 256, 256, None, 512, 256, 256, None) == SHAPE
    assert L.moe_layer_norm_backward(norm(**kw), 256, 256, 256, 256, 256, None, 256, 256, 256, 256, 1 << 30,
                                     None) == SHAPE


def test_norm_arguments_refused():
    L = moe.lib()
    assert L.moe_layer_norm(None, 256, None, None, None, None, 256, 256, 256, None) == NULL
    good = [256, None, 256, 256, None, 512, 256, 256, None]
    for i in (0, 5, 6, 7):
        a = list(good)
        a[i] = None
        assert L.moe_layer_norm(norm(), *a) == NULL
    assert L.moe_layer_norm(norm(), 256, 256, 256, 256, None, 512, 256, 256, None) == NULL  # a residual without h
    for i, v in ((0, 257), (2, 258), (3, 257), (5, 513), (6, 258), (7, 258)):
        a = list(good)
        a[i] = v
        assert L.moe_layer_norm(norm(), *a) == ALIGN
    assert L.moe_layer_norm(norm(dtype=2), 258, None, None, None, None, 512, 256, 256, None) == ALIGN
    assert L.moe_layer_norm(norm(rows=0), None, None, None, None, None, None, None, None, None) == 0
    back = [256, 256, 256, 256, 256, None, 512, 256, 256, 256, 1 << 30, None]
    for i in (0, 1, 2, 3, 6, 9):
        a = list(back)
        a[i] = None
        assert L.moe_layer_norm_backward(norm(), *a) == NULL
    for i, v in ((0, 257), (1, 257), (2, 258), (4, 258), (5, 257), (6, 257), (7, 258), (9, 128)):
        a = list(back)
        a[i] = v
        assert L.moe_layer_norm_backward(norm(), *a) == ALIGN
    a = list(back)
    a[10] = moe.moe_layer_norm_workspace_bytes(4, 64) - 1
    assert L.moe_layer_norm_backward(norm(), *a) == WORKSPACE


def test_norm_workspace_bytes():
    assert moe.moe_layer_norm_workspace_bytes(0, 8) > 0
    a, b = moe.moe_layer_norm_workspace_bytes(10, 100), moe.moe_layer_norm_workspace_bytes(1 << 20, 100)
    assert a >= 10 * 2 * 100 * 4 and a < b == moe.moe_layer_norm_workspace_bytes(1 << 21, 100)
    for bad in ((-1, 8), (1, 0), (1, (1 << 20) + 1)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_layer_norm_workspace_bytes(*bad)
        assert e.value.rc == SHAPE
    assert moe.lib().moe_layer_norm_workspace_bytes(1, 1, None) == NULL


@pytest.mark.parametrize("kw", BAD_TOKENS)
def test_token_shapes_refused(kw):
    L, s = moe.lib(), tokens(**kw)
    n = ctypes.c_size_t()
    assert L.moe_token_map_workspace_bytes(s, ctypes.byref(n)) == SHAPE
    assert L.moe_token_map(s, 256, 256, 256, 256, 256, 1 << 30, None) == SHAPE
    assert L.moe_permute(s, 256, 256, 512, None) == SHAPE
    assert L.moe_permute_backward(s, 256, 256, 512, None) == SHAPE
    assert L.moe_unpermute(s, 256, 256, 256, 512, None) == SHAPE
    assert L.moe_unpermute_backward(s, 256, 256, 256, 256, 512, 256, None) == SHAPE
    if not {"dtype", "hidden", "E_local", "expert_offset"} & set(kw):
        assert L.moe_route_backward(s, 256, 1.0, 256, 256, 256, 512, 256, None) == SHAPE


def test_token_arguments_refused():
    L = moe.lib()
    calls = {
        "moe_token_map": ([256, 256, 256, 256, 256, 1 << 30, None], (0, 1, 2, 3, 4), {0: 258, 1: 258, 3: 257, 4: 128}),
        "moe_permute": ([256, 256, 512, None], (0, 1, 2), {0: 257, 1: 258, 2: 513}),
        "moe_permute_backward": ([256, 256, 512, None], (0, 1, 2), {0: 257, 1: 258, 2: 513}),
        "moe_unpermute": ([256, 256, 256, 512, None], (0, 1, 2, 3), {0: 257, 1: 258, 2: 258, 3: 513}),
        "moe_unpermute_backward": ([256, 256, 256, 256, 512, 256, None], (0, 1, 2, 3, 4, 5),
                                   {0: 257, 1: 257, 2: 258, 3: 258, 4: 513, 5: 258}),
    }
    for name, (args, needed, crooked) in calls.items():
        f = getattr(L, name)
        assert f(None, *args) == NULL, name
        for i in needed:
            a = list(args)
            a[i] = None
            assert f(tokens(), *a) == NULL, (name, i)
        for i, v in crooked.items():
            a = list(args)
            a[i] = v
            assert f(tokens(), *a) == ALIGN, (name, i)
        if name != "moe_token_map":
            assert f(tokens(T=0), *[None] * len(args)) == 0
    assert L.moe_token_map(tokens(), 256, 256, 256, 256, 256, 100, None) == WORKSPACE
    for i in (0, 1, 2, 3):
        ptrs = [256, 256, 256, 512]
        ptrs[i] = None
        assert L.moe_route_backward(tokens(), None, 1.0, *ptrs, None, None) == NULL
    assert L.moe_route_backward(tokens(num_shared=1), None, 1.0, 256, 256, 256, 512, 256, None) == NULL
    assert L.moe_route_backward(tokens(num_shared=1), 256, 1.0, 256, 256, 256, 512, None, None) == NULL
    assert L.moe_route_backward(tokens(), None, 1.0, 256, 256, 256, 514, None, None) == ALIGN
    assert L.moe_route_backward(tokens(T=0), None, 1.0, None, None, None, None, None, None) == 0


def adamw_config(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, seed=0, g_dtype=2, state=0)
    return ctypes.byref(train._AdamwConfig(**{**base, **kw}))


def test_adamw_arguments_refused():
    L = moe.lib()
    T = train._AdamwTensor
    ok = (T * 1)(T(256, 256, 256, 256, None, None, 8))
    assert L.moe_adamw(ok, 1, None, None, None) == NULL
    assert L.moe_adamw(None, 1, adamw_config(), None, None) == NULL
    assert L.moe_adamw(None, 0, adamw_config(), None, None) == 0
    for kw in (dict(step=0), dict(g_dtype=3), dict(g_dtype=-1), dict(state=2), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
               dict(beta2=float("nan")), dict(lr=float("inf")), dict(eps=-1.0), dict(eps=float("nan")),
               dict(weight_decay=float("nan"))):
        assert L.moe_adamw(ok, 1, adamw_config(**kw), None, None) == SHAPE, kw
    assert L.moe_adamw(ok, -1, adamw_config(), None, None) == SHAPE
    assert L.moe_adamw((T * 1)(T(256, 256, 256, 256, None, None, -1)), 1, adamw_config(), None, None) == SHAPE
    for i in range(4):
        f = [256] * 4
        f[i] = None
        assert L.moe_adamw((T * 1)(T(*f, None, None, 8)), 1, adamw_config(), None, None) == NULL
        f[i] = 258
        assert L.moe_adamw((T * 1)(T(*f, None, None, 8)), 1, adamw_config(), None, None) == ALIGN
    assert L.moe_adamw(ok, 1, adamw_config(state=1), None, None) == NULL  # MXFP8 without scales
    assert L.moe_adamw(ok, 1, adamw_config(), 258, None) == ALIGN
    # a refused tensor behind a good one: refused before the good one is launched
    two = (T * 2)(T(256, 256, 256, 256, None, None, 8), T(256, None, 256, 256, None, None, 8))
    assert L.moe_adamw(two, 2, adamw_config(), None, None) == NULL
    assert L.moe_adamw((T * 1)(T(None, None, None, None, None, None, 0)), 1, adamw_config(), None, None) == 0


def test_python_checks():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        moe.moe_layer_norm(x)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        moe.moe_token_map(moe.MoeTokenShape(4, 8, 8, 0, 2, 0, 64), torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="one length"):
        moe.MoeAdamwTensors([x], [], [x], [x])
    with pytest.raises(ValueError, match="both or none"):
        moe.MoeAdamwTensors([x], [x], [x], [x], [x])
    with pytest.raises(ValueError, match="contiguous CUDA"):
        moe.MoeAdamwTensors([x], [x], [x], [x])
    assert all(hasattr(moe, n) for n in moe.train.__all__)
