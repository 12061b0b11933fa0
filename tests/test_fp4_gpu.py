"""The MXFP4 operators on a B200 against numpy doubles: conversion both ways,
quantisation fused with dispatch, the experts' products and the gate/up product
with SwiGLU, alone and as a chain from the routing to the tokens."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
from mixture_experts_ffn_16_b200 import api

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_fp4(rng, G, rows, K, spread=3):
    """An MXFP4 tensor of random codes and scales around 1, and its values."""
    code = rng.integers(0, 16, (G, rows, K))
    byte = rng.integers(127 - spread, 128 + spread, (G, rows, K // 32))
    pair = ref.pack(code, byte)
    return tuple(map(dev, pair)), ref.dequantize(*pair)


# ---------------------------------------------------------------- conversion

def hard_rows(rng, rows, K, dtype):
    """Rows of many magnitudes, with zero blocks, exact ties and borders, and one value far above the rest."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-8, 8, (rows, 1)))
    x[0, :32] = 0.0
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.75, 0.125, 0.5, 4.0, -0.25, -5.0, -0.0])
    x[rows // 2, :32] = np.concatenate([ties, -ties]) * 4.0
    x[-1, 32:64] = 0.01
    x[-1, 40] = 500.0
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,rows,K", [(1, 1, 64), (1, 3, 128), (2, 7, 192), (3, 33, 320), (1, 5, 4096), (2, 2, 4160),
                                      (1, 300, 64), (1, 2, 65536)])
def test_quantize_matches_the_definition(G, rows, K, dtype):
    rng = np.random.default_rng(rows * K)
    x = torch.stack([hard_rows(rng, rows, K, dtype) for _ in range(G)])
    q = api.fp4_empty(G, rows, K)
    api.moe_quantize_fp4(x.cuda(), *q)
    back = torch.empty_like(x, device="cuda")
    api.moe_dequantize_fp4(*q, back)
    code, byte = ref.quantize(x.double().numpy())
    want = ref.pack(code, byte)
    assert np.array_equal(q[1].cpu().numpy(), want[1])
    assert np.array_equal(ref.unpack(q[0].cpu().numpy()) & 7, code & 7)
    got = ref.dequantize(q[0].cpu().numpy(), q[1].cpu().numpy())
    assert np.array_equal(got, ref.dequantize(*want))
    # the way back is exact, up to one rounding where the type cannot hold the value
    assert torch.equal(back.cpu(), torch.from_numpy(got).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(dtype):
    """Smallest and largest numbers of each type, infinities and NaN."""
    f = torch.finfo(dtype)
    x = torch.zeros(1, 8, 64, dtype=dtype)
    x[0, 0, 0], x[0, 0, 33] = f.max, -f.max
    x[0, 1, 5], x[0, 1, 40] = f.tiny, f.smallest_normal * f.eps      # smallest normal, smallest subnormal
    x[0, 2, :] = 1.0
    x[0, 2, 3] = float("inf")
    x[0, 3, :] = 1.0
    x[0, 3, 50] = float("nan")
    x[0, 4, :] = -float("inf")
    x[0, 5, 31], x[0, 5, 32] = 3.0, -3.0
    q = api.fp4_empty(1, 8, 64)
    api.moe_quantize_fp4(x.cuda(), *q)
    back = torch.empty_like(x, device="cuda")
    api.moe_dequantize_fp4(*q, back)
    code, byte = ref.quantize(x.double().numpy())
    want = ref.pack(code, byte)
    assert np.array_equal(q[1].cpu().numpy(), want[1])
    assert np.array_equal(ref.unpack(q[0].cpu().numpy()) & 7, code & 7)
    b = back.cpu()
    assert torch.isnan(b[0, 2, :32]).all() and torch.equal(b[0, 2, 32:], x[0, 2, 32:])
    assert torch.isnan(b[0, 3, 32:]).all() and torch.equal(b[0, 3, :32], x[0, 3, :32])
    assert torch.isnan(b[0, 4]).all()
    assert not torch.isnan(b[0, [0, 1, 5, 6, 7]]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,k,E", [(1, 64, 1, 1), (5, 192, 3, 4), (37, 4096, 8, 20), (3, 8256, 32, 40)])
def test_dispatch_fp4_is_quantize_then_dispatch(T, d, k, E, dtype):
    rng = np.random.default_rng(T + d)
    idx = ref.routing(rng, T, k, E, drop=0.2)
    offsets, slot_row = ref.sort_tokens(idx, E)
    x = hard_rows(rng, T, d, dtype) if T > 2 else torch.from_numpy(rng.standard_normal((T, d))).to(dtype)
    q = tuple(t.fill_(0xEE) for t in api.fp4_empty(1, T * k, d))
    api.moe_dispatch_fp4(x.cuda(), dev(slot_row), q)
    codes, scales = q[0].cpu().numpy(), q[1].cpu().numpy()
    code, byte = ref.quantize(x.double().numpy())
    n = offsets[-1]
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if r >= 0:
                assert np.array_equal(ref.unpack(codes[0, r]) & 7, code[t] & 7)
                assert np.array_equal(ref.rows_of_scales(scales, d)[0, r], byte[t])
    assert (codes[0, n:] == 0xEE).all() and (scales[0, :, n:] == 0xEE).all()      # rows behind the last expert


# ---------------------------------------------------------------- products

def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# (counts of rows per expert, rows behind the last expert)
COUNTS = [([1], 0), ([0, 5, 0], 2), ([16, 1, 33, 0, 7], 0), ([130, 0, 97, 300], 11), ([2] * 40 + [0] * 9, 1),
          ([0, 0, 0], 4), ([700], 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(64, 64), (192, 192), (256, 256), (320, 704), (128, 2048)])
@pytest.mark.parametrize("counts,behind", COUNTS)
def test_matmul(counts, behind, N, K, dtype):
    rng = np.random.default_rng(len(counts) * N + K)
    off = offsets_of(counts)
    E, rows = len(counts), int(off[-1]) + behind
    a, av = random_fp4(rng, 1, rows, K)
    w, wv = random_fp4(rng, E, N, K)
    out = torch.full((rows, N), 77.0, dtype=dtype, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_matmul_fp4(a, dev(off), w, out, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    got = out.double().cpu().numpy()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want = av[0, r] @ wv[e].T
        size = np.abs(av[0, r]) @ np.abs(wv[e]).T
        # products and block sums are exact in the MMA up to its alignment; every 64 elements of K the fp32
        # accumulator takes at most two units of 2^-23 of what it can hold; then one rounding to the type
        add = (K / 64) * 2.0 ** -22 * size
        assert ref.within(got[r], want, add + ref.half_step(dtype, np.abs(want) + add))
    assert bool((got[off[-1]:] == 77.0).all())


def check_swiglu(got_codes, got_scales, g, u, size_g, size_u, K):
    """Kernel h (codes, scale bytes [rows, f/32]) against doubles g, u."""
    # accumulator errors of both products, and a few fp32 ulps for the sigmoid
    dg, du = (K / 64) * 2.0 ** -22 * size_g, (K / 64) * 2.0 ** -22 * size_u
    s = 1.0 / (1.0 + np.exp(-g))
    h = g * s * u
    slope = np.abs(s * (1.0 + g * (1.0 - s)))
    delta = (slope + 1e-3) * dg * (np.abs(u) + du) + np.abs(g * s) * du + 2.0 ** -19 * (1 + np.abs(g)) * np.abs(h)
    rows, f = h.shape
    hb, db = np.abs(h).reshape(rows, -1, 32), delta.reshape(rows, -1, 32)
    # the block's largest magnitude lies between these, and the scale follows it
    low, high = (np.maximum(hb - db, 0)).max(-1), (hb + db).max(-1)
    byte = lambda m: np.where(m > 0, np.maximum(np.frexp(m)[1] - 3 + 127, 0), 0)
    assert bool((got_scales >= byte(low)).all() and (got_scales <= byte(high)).all())
    scale = np.ldexp(1.0, got_scales - 127).repeat(32, -1)
    val = ref.VALUES[got_codes]
    v = h / scale
    spacing = np.where(np.abs(v) < 2, 0.5, np.where(np.abs(v) < 4, 1.0, 2.0))     # of the numbers around v
    near = np.where((np.abs(val) >= 6) & (np.abs(v) > 6) & (np.sign(val) == np.sign(v)), 0.0, np.abs(val - v))
    assert bool((near <= spacing / 2 + delta / scale).all())


@pytest.mark.parametrize("f,K", [(64, 64), (128, 256), (192, 320), (256, 2048)])
@pytest.mark.parametrize("counts,behind", COUNTS)
def test_swiglu(counts, behind, f, K):
    rng = np.random.default_rng(len(counts) + f + K)
    off = offsets_of(counts)
    E, rows = len(counts), int(off[-1]) + behind
    a, av = random_fp4(rng, 1, rows, K, spread=1)
    # weights that keep g around 1
    wg, wgv = random_fp4(rng, E, f, K, spread=1)
    wu, wuv = random_fp4(rng, E, f, K, spread=1)
    down = 4 + int(np.log2(K) / 2)
    for w in (wg, wu):
        w[1].sub_(down)
    wgv, wuv = wgv * 2.0 ** -down, wuv * 2.0 ** -down
    h = tuple(t.fill_(0xEE) for t in api.fp4_empty(1, rows, f))
    ws = api.alloc_dispatch_workspace()
    api.moe_swiglu_fp4(a, dev(off), wg, wu, h, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    codes, scales = ref.unpack(h[0].cpu().numpy())[0], ref.rows_of_scales(h[1].cpu().numpy(), f)[0]
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if r.start < r.stop:
            x = av[0, r]
            check_swiglu(codes[r], scales[r], x @ wgv[e].T, x @ wuv[e].T, np.abs(x) @ np.abs(wgv[e]).T,
                         np.abs(x) @ np.abs(wuv[e]).T, K)
    assert (h[0][0, off[-1]:] == 0xEE).all() and (h[1][0, :, off[-1]:] == 0xEE).all()
