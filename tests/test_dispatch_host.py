"""Argument checks of the token dispatch and MXFP4 entry points on a machine without a GPU: each refusal's code
comes back before anything is looked up on a device, and the Python binding names the tensor it refuses."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_16_b200 import api, build

A = 0x10000                      # an aligned address that nothing dereferences
INV, UNS, WS = api.MOE_ERR_INVALID_ARG, api.MOE_ERR_UNSUPPORTED, api.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def f4(codes=A, scales=A):
    return ctypes.byref(api.MoeFp4Tensor(codes, scales))


def base(name):
    """Arguments, in order, that pass every check of moe_<name>."""
    ws = dict(workspace=A, workspace_bytes=256, stream=0)
    return {
        "sort_tokens": dict(T=4, k=2, E=8, topk_idx=A, offsets=A, slot_row=A, **ws),
        "dispatch": dict(T=4, k=2, d=64, dtype=0, x=A, slot_row=A, x_sorted=A, stream=0),
        "dispatch_backward": dict(T=4, k=2, d=64, dtype=0, dx_sorted=A, slot_row=A, dx=A, stream=0),
        "undispatch": dict(T=4, k=2, d=64, dtype=0, y=A, slot_row=A, topk_w=A, out=A, stream=0),
        "undispatch_backward": dict(T=4, k=2, d=64, dtype=0, dout=A, y=A, slot_row=A, topk_w=A, dy=A, dw=A, stream=0),
        "quantize_fp4": dict(G=1, rows=3, K=64, dtype=0, x=A, q=f4(), stream=0),
        "dequantize_fp4": dict(G=1, rows=3, K=64, dtype=0, q=f4(), x=A, stream=0),
        "dispatch_fp4": dict(T=4, k=2, d=64, dtype=0, x=A, slot_row=A, x_sorted=f4(), stream=0),
        "matmul_fp4": dict(rows=8, E=2, N=64, K=64, a=f4(), offsets=A, W=f4(), dtype=0, out=A, **ws),
        "swiglu_fp4": dict(rows=8, E=2, f=64, K=64, a=f4(), offsets=A, W_gate=f4(), W_up=f4(), h=f4(), **ws),
    }[name]


NAMES = ["sort_tokens", "dispatch", "dispatch_backward", "undispatch", "undispatch_backward", "quantize_fp4",
         "dequantize_fp4", "dispatch_fp4", "matmul_fp4", "swiglu_fp4"]


def call(lib, name, **change):
    args = base(name)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(lib, "moe_" + name)(*args.values())


@pytest.mark.parametrize("name", NAMES)
def test_null_and_misaligned_pointers(lib, name):
    for key, v in base(name).items():
        if key in ("workspace", "stream"):
            continue
        if v == A:
            assert call(lib, name, **{key: None}) == INV, key
            assert call(lib, name, **{key: A + 8}) == UNS, key
        elif not isinstance(v, int):
            assert call(lib, name, **{key: None}) == INV, key
            for bad, code in (((None, A), INV), ((A, None), INV), ((A + 4, A), UNS), ((A, A + 4), UNS)):
                assert call(lib, name, **{key: f4(*bad)}) == code, key


@pytest.mark.parametrize("name", ["sort_tokens", "matmul_fp4", "swiglu_fp4"])
def test_workspace(lib, name):
    assert call(lib, name, workspace=None) == WS
    assert call(lib, name, workspace=A + 128) == WS
    assert call(lib, name, workspace_bytes=255) == WS


SIZES = {"T": [(0, INV), (-1, INV), ((1 << 22) + 1, UNS)], "k": [(0, INV), (33, UNS)], "E": [(0, INV), (2049, UNS)],
         "d": [(0, INV), (-64, INV), (96, UNS), (65600, UNS)], "dtype": [(-1, INV), (3, INV)],
         "G": [(0, INV), (1 << 27, UNS)], "rows": [(0, INV), (-3, INV), ((1 << 27) + 1, UNS)],
         "K": [(0, INV), (32, UNS), (65600, UNS)], "N": [(0, INV), (65, UNS), (65600, UNS)],
         "f": [(0, INV), (96, UNS), (65600, UNS)]}


@pytest.mark.parametrize("name", NAMES)
def test_sizes(lib, name):
    for key in base(name):
        for bad, code in SIZES.get(key, []):
            assert call(lib, name, **{key: bad}) == code, (key, bad)


def test_binding_refusals(lib):
    i32, bf = torch.int32, torch.bfloat16
    host = torch.zeros(4, 2, dtype=i32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="topk_idx"):
        api.moe_sort_tokens(host, torch.zeros(9, dtype=i32), host, ws)                  # host tensors
    with pytest.raises(TypeError, match="x"):
        api.moe_dispatch(None, host, None)
    with pytest.raises(TypeError, match="x"):
        api.moe_dispatch(torch.zeros(4, 64, dtype=torch.float64), host, None)
    with pytest.raises(ValueError, match="x"):
        api.moe_dispatch(torch.zeros(4, 64, 1, dtype=bf), host, None)
    with pytest.raises(TypeError, match="pair"):
        api.moe_matmul_fp4(torch.zeros(1, 4, 32, dtype=torch.uint8), host, None, None, ws)
    with pytest.raises(TypeError, match="x_sorted"):
        api.moe_dispatch_fp4(torch.zeros(4, 64, dtype=bf), host, (1, 2, 3))


def test_fp4_empty_shapes():
    codes, scales = api.fp4_empty(3, 5, 192, device="cpu")
    assert codes.shape == (3, 5, 96) and scales.shape == (3, 2, 5, 4)
    ws = api.alloc_dispatch_workspace("cpu")
    assert ws.numel() == api.DISPATCH_WORKSPACE_BYTES and not ws.any()


def test_row_by_row_scales_become_the_layout():
    """The rearrangement that the binding's notes give, against the oracle's."""
    import numpy as np

    import fp4_ref as ref
    rng = np.random.default_rng(0)
    byte = rng.integers(0, 255, (2, 5, 8), dtype=np.uint8)               # K = 256
    want = ref.pack(np.zeros((2, 5, 256), dtype=int), byte)[1]
    got = torch.from_numpy(byte).view(2, 5, 2, 4).transpose(1, 2).contiguous()
    assert np.array_equal(got.numpy(), want)
