"""The MXFP4 operators on a B200 against numpy doubles: conversion both ways,
quantisation fused with dispatch, the experts' products and the gate/up product
with SwiGLU, alone and as a chain from the routing to the tokens."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
from mixture_experts_ffn_16_b200 import api
from mixture_experts_ffn_16_b200.inputs import MoEConfig, make_inputs

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
                                      (1, 300, 64), (1, 2, 65536), (3, 5, 1024)])
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
@pytest.mark.parametrize("K", [192, 2048])
def test_tensors_that_start_at_16_bytes(K, dtype):
    """x, codes and scales at addresses that are multiples of 16 bytes only give what aligned ones give."""
    def off16(t):
        room = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")
        view = room[16:].view(t.dtype).view(t.shape)
        assert view.data_ptr() % 32 == 16
        return view.copy_(t)

    rng = np.random.default_rng(K)
    x = hard_rows(rng, 9, K, dtype)[None].cuda()
    q, back = api.fp4_empty(1, 9, K), torch.empty_like(x)
    api.moe_quantize_fp4(x, *q)
    api.moe_dequantize_fp4(*q, back)
    x2, q2, back2 = off16(x), tuple(map(off16, api.fp4_empty(1, 9, K))), off16(back.clone().zero_())
    api.moe_quantize_fp4(x2, *q2)
    api.moe_dequantize_fp4(*q2, back2)
    assert torch.equal(q[0], q2[0]) and torch.equal(q[1], q2[1]) and torch.equal(back, back2)
    rows = torch.arange(9, dtype=torch.int32, device="cuda").view(9, 1)
    api.moe_dispatch_fp4(x2[0], off16(rows), tuple(t.fill_(1) for t in q2))
    assert torch.equal(q[0], q2[0]) and torch.equal(q[1], q2[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,k,E", [(1, 64, 1, 1), (5, 192, 3, 4), (37, 4096, 8, 20), (3, 8256, 32, 40),
                                     (6, 1024, 32, 7)])
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
    s = np.exp(-np.logaddexp(0.0, -g))
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
    a[0][0, 0], av[0, 0] = 0, 0.0                        # a row of zeros
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
    if f % 128:                                          # the spare bytes of the last word
        assert not h[1][0, -1, :off[-1], 2:].any()


# ---------------------------------------------------------------- special values, bounds, streams, graphs

def test_nan_scales_stay_in_their_rows_and_columns():
    """A NaN block of an activation row makes that row NaN, one of a weight row that output column; nothing else."""
    rng = np.random.default_rng(3)
    for counts in ([5, 9], [150, 120]):                  # single CTAs, CTA pairs
        off = offsets_of(counts)
        rows, N, K = int(off[-1]), 192, 256
        a, av = random_fp4(rng, 1, rows, K)
        w, wv = random_fp4(rng, 2, N, K)
        a[1][0, 1, 3, 2] = 255                           # row 3, elements 192..223
        w[1][1, 0, 70, 1] = 255                          # expert 1, output 70
        out = torch.empty(rows, N, device="cuda")
        ws = api.alloc_dispatch_workspace()
        api.moe_matmul_fp4(a, dev(off), w, out, ws)
        got = out.cpu().numpy()
        want = np.zeros((rows, N), dtype=bool)
        want[3], want[off[1]:, 70] = True, True
        assert np.array_equal(np.isnan(got), want)
        # through the gate/up product: the whole row, and the block of 32 the column lies in
        wu, _ = random_fp4(rng, 2, N, K)
        h = api.fp4_empty(1, rows, N)
        api.moe_swiglu_fp4(a, dev(off), w, wu, h, ws)
        nan = ref.rows_of_scales(h[1].cpu().numpy(), N)[0] == 255
        expect = np.zeros((rows, N // 32), dtype=bool)
        expect[3], expect[off[1]:, 70 // 32] = True, True
        assert np.array_equal(nan, expect)
        codes = ref.unpack(h[0].cpu().numpy())[0]
        assert not codes[nan.repeat(32, -1)].any()


@pytest.mark.parametrize("off", [[0, 90, 40, 200], [-7, 3, 10 ** 9, 5], [200, 100, 50, 0], [300, 300, 300, 300]])
def test_invalid_offsets_stay_in_bounds(off):
    """Offsets that decrease or leave [0, rows]: clamped, and no row outside the tensor is touched."""
    rng = np.random.default_rng(4)
    rows, N, K = 130, 128, 192
    a, _ = random_fp4(rng, 1, rows, K)
    w, _ = random_fp4(rng, 3, N, K)
    guarded = torch.full((rows + 64, N), 5.0, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_matmul_fp4(a, dev(np.array(off, dtype=np.int32)), w, guarded[32:32 + rows], ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    assert bool((guarded[:32] == 5).all()) and bool((guarded[32 + rows:] == 5).all())


def test_products_past_32_bit_offsets():
    """Outputs of more than 2^31 elements, in the last rows; K a multiple of 64 only."""
    rng = np.random.default_rng(6)
    rows, N, K = 33003, 65536, 192
    off = offsets_of([3, 32990])
    a, av = random_fp4(rng, 1, rows, K)
    w, wv = random_fp4(rng, 2, N, K)
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_matmul_fp4(a, dev(off), w, out, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    for r in (0, 3, 20000, 32980, 32992):
        want = wv[0 if r < 3 else 1] @ av[0, r]
        size = np.abs(wv[0 if r < 3 else 1]) @ np.abs(av[0, r])
        add = (K / 64) * 2.0 ** -22 * size
        assert ref.within(out[r].double().cpu().numpy(), want, add + ref.half_step(out.dtype, np.abs(want) + add))
    assert not bool(out[32993:].any())
    del out
    h = api.fp4_empty(1, rows, N)                        # 2^31 codes, and the scales behind them
    h[1].zero_()
    api.moe_swiglu_fp4(a, dev(off), w, w, h, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    r = 32992
    codes = ref.unpack(h[0][:, r:r + 1].cpu().numpy())[0]
    scales = ref.rows_of_scales(h[1][:, :, r:r + 1].cpu().numpy(), N)[0]
    x, big = av[0, r:r + 1], np.abs(av[0, r:r + 1]) @ np.abs(wv[1]).T
    check_swiglu(codes, scales, x @ wv[1].T, x @ wv[1].T, big, big, K)


class Chain:
    """One layer's experts from the routing to the tokens: route, sort, dispatch_fp4, swiglu, matmul, undispatch."""

    def __init__(self, T, d, f, E, k, seed):
        self.cfg = MoEConfig("fp4_chain", T=T, d=d, E=E, k=k, f=f, S=0, fs=0, score_fn="softmax", seed=seed)
        self.inp = make_inputs(self.cfg, device="cuda")
        self.shape = api.shape_of(self.cfg)
        self.route_ws = api.alloc_workspace(self.shape)
        self.ws = api.alloc_dispatch_workspace()
        q = {}
        for name in ("W_gate", "W_up", "W_down"):
            q[name] = api.fp4_empty(E, *self.inp[name].shape[1:])
            api.moe_quantize_fp4(self.inp[name], *q[name])
        self.q = q
        self.x = self.inp["x"].clone()
        self.idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.w = torch.empty(T, k, device="cuda")
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.slot_row = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.a, self.h = api.fp4_empty(1, T * k, d), api.fp4_empty(1, T * k, f)
        self.y = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")

    def __call__(self, stream=None):
        c = self.cfg
        api.moe_route(self.shape, self.x, self.inp["W_router"], None, c.score_fn, True, 1.0, self.idx, self.w,
                      self.route_ws, stream)
        api.moe_sort_tokens(self.idx, self.offsets, self.slot_row, self.ws, stream)
        api.moe_dispatch_fp4(self.x, self.slot_row, self.a, stream)
        api.moe_swiglu_fp4(self.a, self.offsets, self.q["W_gate"], self.q["W_up"], self.h, self.ws, stream)
        api.moe_matmul_fp4(self.h, self.offsets, self.q["W_down"], self.y, self.ws, stream)
        api.moe_undispatch(self.y, self.slot_row, self.w, self.out, stream)
        return self.out

    def state(self):
        return [t.clone() for t in (self.idx, self.w, self.offsets, self.slot_row, *self.a, *self.h, self.y, self.out)]


@pytest.mark.parametrize("T,d,f,E,k", [(1, 128, 64, 8, 2), (70, 256, 192, 12, 3), (500, 512, 256, 6, 2)])
def test_chain_of_an_expert_layer(T, d, f, E, k):
    """Each step checked in doubles from what the step before it left."""
    c = Chain(T, d, f, E, k, seed=T)
    c()
    assert api.moe_device_status(c.ws) == api.MOE_OK
    idx, slot_row = c.idx.cpu().numpy(), c.slot_row.cpu().numpy()
    off, rows = ref.sort_tokens(idx, E)
    assert np.array_equal(c.offsets.cpu().numpy(), off) and np.array_equal(slot_row, rows)
    a = ref.dequantize(*(t.cpu().numpy() for t in c.a))[0]
    xq = ref.dequantize(*ref.pack(*(t[None] for t in ref.quantize(c.x.double().cpu().numpy()))))[0]
    tok = np.empty(T * k, dtype=int)
    tok[rows.reshape(-1)] = np.arange(T * k) // k
    assert np.array_equal(a, xq[tok])
    W = {n: ref.dequantize(*(t.cpu().numpy() for t in c.q[n])) for n in c.q}
    hc, hs = ref.unpack(c.h[0].cpu().numpy())[0], ref.rows_of_scales(c.h[1].cpu().numpy(), f)[0]
    h = ref.dequantize(*(t.cpu().numpy() for t in c.h))[0]
    y = c.y.double().cpu().numpy()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if r.start == r.stop:
            continue
        check_swiglu(hc[r], hs[r], a[r] @ W["W_gate"][e].T, a[r] @ W["W_up"][e].T,
                     np.abs(a[r]) @ np.abs(W["W_gate"][e]).T, np.abs(a[r]) @ np.abs(W["W_up"][e]).T, d)
        want, size = h[r] @ W["W_down"][e].T, np.abs(h[r]) @ np.abs(W["W_down"][e]).T
        add = (f / 64 + 1) * 2.0 ** -22 * size
        assert ref.within(y[r], want, add + ref.half_step(c.y.dtype, np.abs(want) + add))
    w = c.w.double().cpu().numpy()
    terms = w[..., None] * y[rows]
    want, add = terms.sum(1), k * 2.0 ** -24 * np.abs(terms).sum(1)
    assert ref.within(c.out.double().cpu().numpy(), want, add + ref.half_step(c.out.dtype, np.abs(want) + add))


def test_chain_repeats_bitwise_on_another_stream_and_from_a_graph():
    """The same bits from the current stream, a side stream, and a captured graph replayed on other inputs."""
    c = Chain(300, 256, 192, 5, 2, seed=9)
    c()
    first = c.state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (c.idx, c.offsets, c.slot_row, *c.a, *c.h, c.y, c.out):
        t.fill_(1)
    side.wait_stream(torch.cuda.current_stream())
    c(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, c.state()))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c()
    other = torch.randn_like(c.x)
    c.x.copy_(other)
    c()
    want = c.state()
    assert not torch.equal(want[-1], first[-1])
    c.x.copy_(c.inp["x"])
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(first, c.state()))
    c.x.copy_(other)
    graph.replay()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(want, c.state()))
    assert api.moe_device_status(c.ws) == api.MOE_OK


def test_two_layers_on_two_streams_at_once():
    """Two chains, each with its own workspace, interleaved on two streams."""
    chains = [Chain(400, 512, 256, 4, 2, seed=21), Chain(37, 256, 128, 16, 4, seed=22)]
    want = []
    for c in chains:
        c()
        want.append(c.state())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(chains, streams):
            c(s)
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert all(torch.equal(p, q) for p, q in zip(w, c.state()))
        assert api.moe_device_status(c.ws) == api.MOE_OK


def test_refusals_on_the_device():
    rng = np.random.default_rng(8)
    a, _ = random_fp4(rng, 1, 8, 128)
    w, _ = random_fp4(rng, 2, 64, 128)
    off, ws = dev(offsets_of([3, 5])), api.alloc_dispatch_workspace()
    out = torch.full((8, 64), 3.0, device="cuda")
    with pytest.raises(ValueError, match="out"):
        api.moe_matmul_fp4(a, off, w, torch.empty(9, 64, device="cuda"), ws)
    with pytest.raises(ValueError, match="offsets"):
        api.moe_matmul_fp4(a, off[:2], w, out, ws)
    with pytest.raises(ValueError, match="a.scales"):
        api.moe_matmul_fp4((a[0], a[1][:, :, :7]), off, w, out, ws)
    with pytest.raises(ValueError, match="contiguous"):
        api.moe_matmul_fp4(a, off, w, torch.empty(64, 8, device="cuda").t(), ws)
    with pytest.raises(TypeError, match="out"):
        api.moe_matmul_fp4(a, off, w, torch.empty(8, 64, dtype=torch.float64, device="cuda"), ws)
    with pytest.raises(ValueError, match="offsets"):
        api.moe_matmul_fp4(a, off.cpu(), w, out, ws)
    with pytest.raises(api.MoEError) as e:
        api.moe_matmul_fp4(a, off, w, out, ws[:128])
    assert e.value.status == api.MOE_ERR_WORKSPACE
    with pytest.raises(api.MoEError) as e:                      # K = 32
        api.moe_quantize_fp4(torch.zeros(1, 2, 32, device="cuda"), *api.fp4_empty(1, 2, 32))
    assert e.value.status == api.MOE_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


def test_error_word_is_kept_by_products_and_cleared_by_the_sort():
    """A timeout recorded in the workspace (by the bounded-wait self-test, 1 ms) survives products, not the next sort."""
    rng = np.random.default_rng(10)
    a, av = random_fp4(rng, 1, 8, 128)
    w, wv = random_fp4(rng, 2, 64, 128)
    ws = api.alloc_dispatch_workspace()
    out = torch.empty(8, 64, device="cuda")
    api.moe_debug_wait_timeout(ws, 1000000)
    api.moe_matmul_fp4(a, dev(offsets_of([3, 5])), w, out, ws)
    assert api.moe_device_status(ws) == api.MOE_ERR_DEVICE_TIMEOUT
    assert np.allclose(out.cpu().numpy()[:3], av[0, :3] @ wv[0].T, rtol=1e-5)
    idx = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    api.moe_sort_tokens(idx, torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(idx), ws)
    assert api.moe_device_status(ws) == api.MOE_OK


@pytest.mark.parametrize("most", [3, 260])               # single CTAs, CTA pairs
def test_as_many_experts_as_there_may_be(most):
    """E = 2048: the products' tables at their largest, many experts empty."""
    rng = np.random.default_rng(most)
    counts = rng.integers(0, most, 2048)
    counts[rng.random(2048) < 0.2] = 0
    off = offsets_of(counts)
    rows, N, K = int(off[-1]), 64, 64
    a, av = random_fp4(rng, 1, rows, K)
    w, wv = random_fp4(rng, 2048, N, K)
    out, ws = torch.empty(rows, N, device="cuda"), api.alloc_dispatch_workspace()
    api.moe_matmul_fp4(a, dev(off), w, out, ws)
    h = api.fp4_empty(1, rows, N)
    api.moe_swiglu_fp4(a, dev(off), w, w, h, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    got = out.double().cpu().numpy()
    codes, scales = ref.unpack(h[0].cpu().numpy())[0], ref.rows_of_scales(h[1].cpu().numpy(), N)[0]
    g, size = np.empty((rows, N)), np.empty((rows, N))
    for e in range(2048):
        r = slice(off[e], off[e + 1])
        g[r], size[r] = av[0, r] @ wv[e].T, np.abs(av[0, r]) @ np.abs(wv[e]).T
    add = 2.0 ** -22 * size
    assert ref.within(got, g, add + ref.half_step(out.dtype, np.abs(g) + add))
    check_swiglu(codes, scales, g, g, size, size, K)


@pytest.mark.parametrize("K", [64, 320])
def test_accumulators_that_do_not_fit_side_by_side(K):
    """Runs of 193 to 256 tokens next to one another and to short ones, several units for every pair of CTAs."""
    rng = np.random.default_rng(K)
    off = offsets_of([256, 250, 40, 230, 193, 256, 500, 17, 256])
    E, rows, N = len(off) - 1, int(off[-1]), 4096
    a, av = random_fp4(rng, 1, rows, K)
    w, wv = random_fp4(rng, E, N, K)
    ws = api.alloc_dispatch_workspace()
    outs = [torch.empty(rows, N, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)]
    for out in outs:
        api.moe_matmul_fp4(a, dev(off), w, out, ws)
    h = api.fp4_empty(1, rows, N)
    api.moe_swiglu_fp4(a, dev(off), w, w, h, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    codes, scales = ref.unpack(h[0].cpu().numpy())[0], ref.rows_of_scales(h[1].cpu().numpy(), N)[0]
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want, size = av[0, r] @ wv[e].T, np.abs(av[0, r]) @ np.abs(wv[e]).T
        add = (K / 64) * 2.0 ** -22 * size
        for out in outs:
            assert ref.within(out[r].double().cpu().numpy(), want, add + ref.half_step(out.dtype, np.abs(want) + add))
        check_swiglu(codes[r], scales[r], want, want, size, size, K)


@pytest.mark.parametrize("K", [64, 512])
def test_products_repeat_bitwise(K):
    """Thirty runs of each product over runs of all lengths, on CTA pairs and on single CTAs, into cleared outputs."""
    rng = np.random.default_rng(K + 1)
    for counts in (rng.integers(0, 400, 60), rng.integers(0, 150, 120)):
        off = dev(offsets_of(counts))
        E, rows, N = len(counts), int(counts.sum()), 2048
        a, _ = random_fp4(rng, 1, rows, K)
        w, _ = random_fp4(rng, E, N, K)
        ws = api.alloc_dispatch_workspace()
        out, h = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"), api.fp4_empty(1, rows, N)
        first = None
        for _ in range(30):
            for t in (out, *h):
                t.zero_()
            api.moe_matmul_fp4(a, off, w, out, ws)
            api.moe_swiglu_fp4(a, off, w, w, h, ws)
            got = [t.clone() for t in (out, *h)]
            first = first or got
            assert all(torch.equal(p, q) for p, q in zip(first, got))
        assert api.moe_device_status(ws) == api.MOE_OK


def test_the_widest_rows():
    """K = 65,536, the longest accumulation: 256 stages for a unit."""
    rng = np.random.default_rng(2)
    for counts in ([2, 1], [120, 100]):
        off, N, K = offsets_of(counts), 64, 65536
        rows = int(off[-1])
        a, av = random_fp4(rng, 1, rows, K)
        w, wv = random_fp4(rng, 2, N, K)
        out, ws = torch.empty(rows, N, device="cuda"), api.alloc_dispatch_workspace()
        api.moe_matmul_fp4(a, dev(off), w, out, ws)
        assert api.moe_device_status(ws) == api.MOE_OK
        for e in range(2):
            r = slice(off[e], off[e + 1])
            want, size = av[0, r] @ wv[e].T, np.abs(av[0, r]) @ np.abs(wv[e]).T
            add = (K / 64) * 2.0 ** -22 * size
            assert ref.within(out[r].double().cpu().numpy(), want, add + ref.half_step(out.dtype, np.abs(want) + add))


def test_the_most_rows():
    """134,217,728 rows (the most a call takes) on 3 experts, sampled."""
    rows, N, K = 1 << 27, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    a = (torch.randint(0, 256, (1, rows, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
         torch.full((1, 1, rows, 4), 127, dtype=torch.uint8, device="cuda"))
    rng = np.random.default_rng(1)
    w, wv = random_fp4(rng, 3, N, K)
    off = np.array([0, 5, 70_000_003, rows - 2], dtype=np.int32)
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_matmul_fp4(a, dev(off), w, out, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    for r in (0, 4, 5, 70_000_002, 70_000_003, 100_000_000, rows - 3):
        x = ref.VALUES[ref.unpack(a[0][0, r].cpu().numpy())]
        want = wv[np.searchsorted(off, r, side="right") - 1] @ x
        assert ref.within(out[r].double().cpu().numpy(), want, ref.half_step(out.dtype, want) + 2.0 ** -22 * 64 * 36)
    assert not bool(out[rows - 2:].any())


def weight_row(value, blocks):
    """Codes and scale bytes [blocks] whose first elements add up to `value`, 2 bits or more a block (greedy)."""
    code, byte = np.zeros(blocks, dtype=int), np.full(blocks, 127)
    left = float(value)
    for i in range(blocks):
        if left == 0.0:
            break
        m, e = np.frexp(abs(left))                       # 0.5 <= m < 1: the nearest of 0.5, 0.75 and 1
        near = (0.5, 0.75, 1.0)[int(np.argmin([abs(m - 0.5), abs(m - 0.75), abs(m - 1.0)]))]
        four = int(near * 8)                             # 4 or 6 (code 6, 7) times 2^(e - 3); 8 is 4 times 2^(e - 2)
        up = int(four == 8)
        byte[i] = 127 + e - 3 + up
        code[i] = (7 if four == 6 else 6) + (8 if left < 0 else 0)
        left -= np.sign(left) * np.ldexp(near, int(e))
    return code, byte


def swiglu_of(g, u, counts):
    """h codes and scale bytes [rows, f] of gate sums g and up sums u [f], the same in every row, and the sums there were."""
    f, blocks = len(g), 16
    K = 32 * blocks
    off = offsets_of(counts)
    E, rows = len(counts), int(off[-1])
    one = np.zeros((1, rows, K), dtype=int)
    one[..., ::32] = 2                                   # 1.0 in the first element of every block
    a = tuple(map(dev, ref.pack(one, np.full((1, rows, blocks), 127))))
    weights, sums = [], []
    for target in (g, u):
        code, byte = np.zeros((E, f, K), dtype=int), np.empty((E, f, blocks), dtype=int)
        for j in range(f):
            c, b = weight_row(target[j], blocks)
            code[:, j, ::32], byte[:, j] = c, b
        pair = ref.pack(code, byte)
        weights.append(tuple(map(dev, pair)))
        sums.append(ref.dequantize(*pair)[0].sum(-1))
    h, ws = api.fp4_empty(1, rows, f), api.alloc_dispatch_workspace()
    api.moe_swiglu_fp4(a, dev(off), *weights, h, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    return ref.unpack(h[0].cpu().numpy())[0], ref.rows_of_scales(h[1].cpu().numpy(), f)[0], *sums


FORMS = [[3], [200, 120]]                                # single CTAs, CTA pairs


@pytest.mark.parametrize("counts", FORMS)
@pytest.mark.parametrize("gate", [-88.6, -87.5, -86.0, -80.0, -60.0, -40.0, -20.0, -8.0, -1.0, 0.5, 3.0, 20.0])
def test_swiglu_beside_the_borders(gate, counts):
    """Values of h a few ulps to either side of the borders between codes, at gates far from zero: the right code.

    In units of 2^-24 of the value: expf 4 (2 ulps), the sum 1, the quotient 1, the product 1, so 7 in all.  Values
    lie 8 or more from a border.  Feature 0 of each block of 32 is 4, so the block's scale is 1."""
    rng = np.random.default_rng(int(-gate * 10) % 1000)
    f = 64
    g = np.float32(gate) * (1 + rng.random(f) / 200)
    g = np.round(np.maximum(g, -88.7) * 2.0 ** 14) / 2.0 ** 14       # 21 bits
    silu = lambda x: x * np.exp(-np.logaddexp(0.0, -x))
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], f)
    side = rng.choice([-1.0, 1.0], f)
    u = border * (1 + side * 12 * 2.0 ** -24) / silu(g)
    m, e = np.frexp(u)
    u = np.ldexp(np.round(m * 2.0 ** 22), e - 22)        # 22 bits: every partial sum of the product is exact
    g[::32], u[::32] = 64.0, 2.0 ** -4
    codes, scales, g, u = swiglu_of(g, u, counts)
    h = silu(g) * u
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    gap = np.abs(np.abs(h)[:, None] / edges - 1).min(1) * 2.0 ** 24
    sure = gap >= 8                                      # rounding u to 22 bits brought some of them nearer
    assert sure.sum() >= f // 2 and (gap[sure] <= 40).sum() >= f // 3
    want = (np.abs(h)[:, None] > edges).sum(1)
    assert (scales == 127).all()
    assert np.array_equal((codes & 7)[:, sure], np.tile(want[sure], (len(codes), 1)))
    assert np.array_equal((codes >> 3)[:, sure], np.tile((h < 0)[sure], (len(codes), 1)))


@pytest.mark.parametrize("counts", FORMS)
def test_swiglu_at_the_ends_of_fp32(counts):
    """A product g u past fp32 makes its block NaN and no other; gates past the exponential's range give 0 or g u."""
    big = 2.0 ** 100
    g, u = np.full(192, 1.0), np.full(192, 1.0)
    g[3], u[3] = big, big                                # block 0: +inf
    g[40], u[40] = big, -big                             # block 1: -inf
    g[64:96], u[64:96] = -89.0 - np.arange(32), 2.0      # block 2: all of it 0 (|SiLU| below 2.6e-37 and flushed)
    g[96:128], u[96:128] = -1.5 * 2.0 ** 126, big        # block 3: 0
    g[128:160], u[128:160] = 1.5 * 2.0 ** 124, 2.0 ** -124        # block 4: SiLU(g) = g, h = 1.5
    g[160:], u[160:] = 0.0, big                          # block 5: 0
    codes, scales, _, _ = swiglu_of(g, u, counts)
    silu1 = 1.0 / (1.0 + np.exp(-1.0))                   # 0.731: scale 2^(-1 - 2), 5.85 rounds to 6
    assert (scales[:, :2] == 255).all() and not codes[:, :64].any()
    assert (scales[:, 2:4] == 0).all() and not (codes[:, 64:128] & 7).any()
    assert (scales[:, 4] == 125).all() and (codes[:, 128:160] == 7).all()
    assert (scales[:, 5] == 0).all() and not (codes[:, 160:] & 7).any()
    g[3] = u[3] = g[40] = u[40] = 1.0
    codes, scales, _, _ = swiglu_of(g, u, counts)
    assert silu1 * 8 > 5 and (scales[:, :2] == 124).all() and (codes[:, :64] == 7).all()


@pytest.mark.parametrize("N,K", [(512, 256), (2048, 1024), (1024, 2112)])
def test_scales_of_the_run_are_the_ones_used(N, K):
    """Two sets of inputs of one shape, whose scales differ by 2^16 and more, in turn: a scale left in shared or tensor
    memory by the call or the stage before would show.  On CTA pairs, each of whose CTAs copies its own scales."""
    rng = np.random.default_rng(N)
    off_host = offsets_of([130, 97, 256, 0, 301])
    off, E, rows = dev(off_host), len(off_host) - 1, int(off_host[-1])
    sets, ws = [], api.alloc_dispatch_workspace()
    for shift in (0, 24):
        a, av = random_fp4(rng, 1, rows, K, spread=2)
        w, wv = random_fp4(rng, E, N, K, spread=2)
        a[1].add_(shift)
        w[1].sub_(shift // 3)
        out, h = torch.zeros(rows, N, device="cuda"), api.fp4_empty(1, rows, N)
        up = (w[0], w[1] - (8 + shift))                  # keeps h finite
        api.moe_matmul_fp4(a, off, w, out, ws)
        api.moe_swiglu_fp4(a, off, w, up, h, ws)
        for e in range(E):
            r = slice(off_host[e], off_host[e + 1])
            scale = 2.0 ** (shift - shift // 3)
            want, size = av[0, r] @ wv[e].T * scale, np.abs(av[0, r]) @ np.abs(wv[e]).T * scale
            add = (K / 64) * 2.0 ** -22 * size
            assert ref.within(out[r].double().cpu().numpy(), want, add + ref.half_step(out.dtype, np.abs(want) + add))
        sets.append((a, w, up, out, h, [t.clone() for t in (out, *h)]))
    for _ in range(60):
        for a, w, up, out, h, first in sets:
            for t in (out, *h):
                t.zero_()
            api.moe_matmul_fp4(a, off, w, out, ws)
            api.moe_swiglu_fp4(a, off, w, up, h, ws)
            assert all(torch.equal(p, q) for p, q in zip(first, (out, *h)))
    assert api.moe_device_status(ws) == api.MOE_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [130, 700])             # single CTAs, CTA pairs
@pytest.mark.parametrize("off", [[0, 90, 40, 200], [-7, 3, 10 ** 9, 5], [200, 100, 50, 0], [300, 300, 300, 300],
                                 [0, 699, 1, 2 ** 31 - 1], [-2 ** 31, 650, -1, 700]])
def test_invalid_offsets_stay_in_bounds_in_every_form(off, rows, dtype):
    """Of both products: what lies around their outputs stays as it was."""
    rng = np.random.default_rng(5)
    N, K, pad = 192, 320, 64
    a, _ = random_fp4(rng, 1, rows, K)
    w, _ = random_fp4(rng, 3, N, K)
    offsets, ws = dev(np.array(off, dtype=np.int32)), api.alloc_dispatch_workspace()

    def guarded(shape, dtype):
        """A tensor of this shape with `pad` rows' worth of other bytes on either side, and those bytes."""
        n, around = int(np.prod(shape)), pad * N
        room = torch.full((n + 2 * around,), 93, dtype=dtype, device="cuda")
        return room[around:around + n].view(shape), lambda: bool((room[:around] == 93).all() and
                                                                 (room[around + n:] == 93).all())

    out, out_kept = guarded((rows, N), dtype)
    codes, codes_kept = guarded((1, rows, N // 2), torch.uint8)
    scales, scales_kept = guarded((1, 2, rows, 4), torch.uint8)
    api.moe_matmul_fp4(a, offsets, w, out, ws)
    api.moe_swiglu_fp4(a, offsets, w, w, (codes, scales), ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    assert out_kept() and codes_kept() and scales_kept()
    low, high = np.clip([min(off), max(off)], 0, rows)
    for t in (out, codes[0], scales[0].transpose(0, 1).reshape(rows, -1)):       # rows that no offsets enclose
        assert bool((t[:low] == 93).all() and (t[high:] == 93).all())


def test_two_graphs_of_one_workspace_and_two_threads_at_once():
    """Chains captured with the same dispatch workspace, replayed in turn; then two threads calling on streams of their
    own, each with its workspace: the bits of the calls made alone."""
    import threading
    chains = [Chain(300, 256, 192, 5, 2, seed=31), Chain(64, 512, 128, 24, 6, seed=32)]
    chains[1].ws = chains[0].ws
    want = []
    for c in chains:
        c()
        want.append(c.state())
    torch.cuda.synchronize()
    graphs = []
    for c in chains:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for _ in range(5):
        for c, g, w in zip(chains, graphs, want):
            for t in (c.idx, c.offsets, c.slot_row, *c.a, *c.h, c.y, c.out):
                t.fill_(1)
            g.replay()
            assert all(torch.equal(p, q) for p, q in zip(w, c.state()))
    chains[1].ws = api.alloc_dispatch_workspace()
    torch.cuda.synchronize()
    failed = []

    def work(c, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    c()
                    if not all(torch.equal(p, q) for p, q in zip(w, c.state())):
                        failed.append("differs")
        except Exception as e:               # a thread's exception would be lost
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=p) for p in zip(chains, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and all(api.moe_device_status(c.ws) == api.MOE_OK for c in chains)
