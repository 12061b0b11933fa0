"""Token dispatch on a B200 against numpy doubles: the sort, both directions and both gradients."""
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


def run_sort(idx, E):
    offsets = torch.full((E + 1,), -5, dtype=torch.int32, device="cuda")
    slot_row = torch.full(idx.shape, -5, dtype=torch.int32, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_sort_tokens(dev(idx), offsets, slot_row, ws)
    return offsets, slot_row, ws


@pytest.mark.parametrize("T,k,E,drop,skew", [
    (1, 1, 1, 0.0, 0.0), (1, 5, 7, 0.0, 0.0), (33, 3, 8, 0.3, 0.0), (64, 10, 512, 0.0, 0.0), (1000, 8, 256, 0.1, 1.0),
    (700, 32, 2048, 0.05, 0.5), (2100, 22, 896, 0.0, 0.7), (257, 1, 3, 0.5, 2.0), (40, 6, 4, 0.1, 0.0)])
def test_sort(T, k, E, drop, skew):
    rng = np.random.default_rng(T)
    idx = ref.routing(rng, T, k, E, drop, skew)
    offsets, slot_row, ws = run_sort(idx, E)
    assert api.moe_device_status(ws) == api.MOE_OK
    want_off, want_row = ref.sort_tokens(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(slot_row.cpu().numpy(), want_row)


@pytest.mark.parametrize("idx,E", [(np.full((9, 4), -1), 3), (np.full((50, 7), 2), 5), (np.full((4000, 5), 0), 1)])
def test_sort_one_sided(idx, E):
    """No expert at all; one expert for everything (a token naming it several times)."""
    idx = idx.astype(np.int32)
    offsets, slot_row, ws = run_sort(idx, E)
    want_off, want_row = ref.sort_tokens(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(slot_row.cpu().numpy(), want_row)
    assert api.moe_device_status(ws) == api.MOE_OK


def test_sort_reports_invalid_experts_and_clears_the_error_word():
    idx = np.array([[0, 1], [7, -2], [2, 0]], dtype=np.int32)      # 7 and -2 are no experts of 3
    offsets, slot_row, ws = run_sort(idx, 3)
    assert api.moe_device_status(ws) == api.MOE_ERR_INVALID_ARG
    assert slot_row.cpu().tolist() == [[0, 2], [-1, -1], [3, 1]]
    assert offsets.cpu().tolist() == [0, 2, 3, 4]
    api.moe_sort_tokens(dev(np.array([[0, 1]], dtype=np.int32)), offsets, torch.empty(1, 2, dtype=torch.int32).cuda(),
                        ws)
    assert api.moe_device_status(ws) == api.MOE_OK


def test_sort_of_a_large_batch():
    T, k, E = 60000, 9, 300
    rng = np.random.default_rng(5)
    idx = rng.integers(-1, E, (T, k)).astype(np.int32)
    offsets, slot_row, _ = run_sort(idx, E)
    flat = idx.reshape(-1)
    key = np.where(flat >= 0, flat, E)
    order = np.argsort(key, kind="stable")
    rows = np.empty(T * k, dtype=np.int64)
    rows[order] = np.arange(T * k)
    assert np.array_equal(slot_row.cpu().numpy().reshape(-1), np.where(flat >= 0, rows, -1))
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E)[:E])]))


SIZES = [(1, 64, 1, 1), (3, 64, 2, 5), (37, 192, 5, 8), (5, 2048, 8, 16), (64, 4096, 10, 512), (9, 7168, 22, 30),
         (2, 65536, 32, 40), (301, 128, 3, 6)]


def plan(T, k, E, seed):
    rng = np.random.default_rng(seed)
    offsets, slot_row = ref.sort_tokens(ref.routing(rng, T, k, E, drop=0.2), E)
    return rng, offsets, slot_row


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,k,E", SIZES)
def test_dispatch_and_its_gradient(T, d, k, E, dtype):
    rng, offsets, slot_row = plan(T, k, E, T + d)
    n = offsets[-1]
    x = torch.from_numpy(rng.standard_normal((T, d))).to(dtype)
    xs = torch.full((T * k, d), 9.0, dtype=dtype, device="cuda")
    api.moe_dispatch(x.cuda(), dev(slot_row), xs)
    got = xs.cpu()
    for t in range(T):
        for j in range(k):
            if slot_row[t, j] >= 0:
                assert torch.equal(got[slot_row[t, j]], x[t])
    assert (got[n:] == 9.0).all()

    dxs = torch.from_numpy(rng.standard_normal((T * k, d))).to(dtype)
    dxs[n:] = float("nan")                          # rows that no slot has are not read
    dx = torch.full((T, d), 9.0, dtype=dtype, device="cuda")
    api.moe_dispatch_backward(dxs.cuda(), dev(slot_row), dx)
    rows = dxs.double().numpy()
    want, size = np.zeros((T, d)), np.zeros((T, d))
    for j in range(k):
        has = slot_row[:, j] >= 0
        want[has] += rows[slot_row[has, j]]
        size[has] += np.abs(rows[slot_row[has, j]])
    # k fp32 additions, one rounding
    add = k * 2.0 ** -24 * size
    assert ref.within(dx.double().cpu().numpy(), want, add + ref.half_step(dtype, np.abs(want) + add))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,k,E", SIZES)
def test_undispatch_and_its_gradient(T, d, k, E, dtype):
    rng, offsets, slot_row = plan(T, k, E, 2 * T + d)
    n = offsets[-1]
    y = torch.from_numpy(rng.standard_normal((T * k, d))).to(dtype)
    y[n:] = float("nan")
    w = torch.from_numpy(rng.random((T, k))).float()
    w[torch.from_numpy(slot_row < 0)] = float("inf")          # weights of dropped slots are not used
    out = torch.full((T, d), 9.0, dtype=dtype, device="cuda")
    api.moe_undispatch(y.cuda(), dev(slot_row), w.cuda(), out)
    yv, wv = y.double().numpy(), w.double().numpy()
    want, size = np.zeros((T, d)), np.zeros((T, d))
    for j in range(k):
        has = slot_row[:, j] >= 0
        term = wv[has, j, None] * yv[slot_row[has, j]]
        want[has] += term
        size[has] += np.abs(term)
    add = k * 2.0 ** -24 * size                     # k fused multiply-adds, then one rounding
    assert ref.within(out.double().cpu().numpy(), want, add + ref.half_step(dtype, np.abs(want) + add))

    dout = torch.from_numpy(rng.standard_normal((T, d))).to(dtype)
    dy = torch.full((T * k, d), 9.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), 9.0, dtype=torch.float32, device="cuda")
    api.moe_undispatch_backward(dout.cuda(), y.cuda(), dev(slot_row), w.cuda(), dy, dw)
    gv, dyv, dwv = dout.double().numpy(), dy.double().cpu().numpy(), dw.double().cpu().numpy()
    assert (dyv[n:] == 9.0).all()
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if r < 0:
                assert dwv[t, j] == 0.0
                continue
            want = wv[t, j] * gv[t]
            # an fp32 product, then a rounding to the type
            first = 2.0 ** -24 * np.abs(want)
            assert ref.within(dyv[r], want, first + ref.half_step(dtype, np.abs(want) + first))
            # a sum of d fp32 products: a thread's share in a row, then a tree
            tol = (d / 256 + 8 + 16) * 2.0 ** -24 * np.abs(gv[t] * yv[r]).sum()
            assert abs(dwv[t, j] - gv[t] @ yv[r]) <= tol


def test_rows_out_of_range_count_as_none():
    """slot_row values outside [0, T k) are dropped slots: nothing is read or written for them."""
    T, k, d = 4, 2, 128
    slot_row = dev(np.array([[0, 8], [-3, 1], [2 ** 31 - 1, -2 ** 31], [3, 7]], dtype=np.int32))
    x = torch.randn(T, d, device="cuda")
    xs = torch.zeros(T * k, d, device="cuda")
    api.moe_dispatch(x, slot_row, xs)
    assert torch.equal(xs[[0, 1, 3, 7]], x[[0, 1, 3, 3]]) and not xs[[2, 4, 5, 6]].any()
    w = torch.ones(T, k, device="cuda")
    out = torch.empty(T, d, device="cuda")
    api.moe_undispatch(xs, slot_row, w, out)
    assert torch.equal(out[:2], x[:2]) and not out[2].any() and torch.equal(out[3], 2 * x[3])
    dy, dw = torch.zeros_like(xs), torch.empty(T, k, device="cuda")
    api.moe_undispatch_backward(x, xs, slot_row, w, dy, dw)
    assert torch.equal(dy, xs) and (dw[2] == 0).all() and dw[0, 1] == 0 and dw[1, 0] == 0


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements of sorted rows."""
    T, k, d = 4100, 8, 65536
    offsets, slot_row = ref.sort_tokens(np.random.default_rng(1).permuted(np.tile(np.arange(8, dtype=np.int32), (T, 1)),
                                                                          axis=1), 8)
    x = torch.randn(T, d, device="cuda").bfloat16()
    xs = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    rows = dev(slot_row)
    api.moe_dispatch(x, rows, xs)
    for j in range(k):
        for t0 in range(0, T, 1025):
            assert torch.equal(xs[rows[t0:t0 + 1025, j].long()], x[t0:t0 + 1025])
    w = torch.full((T, k), 0.125, device="cuda")
    out = torch.empty_like(x)
    api.moe_undispatch(xs, rows, w, out)                 # eight equal rows, weights that add up to 1: exact
    assert torch.equal(out, x)
    dy, dw = torch.zeros_like(xs), torch.empty(T, k, device="cuda")
    api.moe_undispatch_backward(x, xs, rows, w, dy, dw)
    assert torch.equal(dy[rows[4099, 7].long()], (x[4099].float() * 0.125).bfloat16())
    assert torch.equal(dy[T * k - 1], (xs[T * k - 1].float() * 0.125).bfloat16())
    want = x[4099].double().square().sum().item()
    assert abs(dw[4099, 3].item() - want) <= (d / 256 + 24) * 2.0 ** -24 * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_against_differences(dtype):
    """The loss sum(out * g) of dispatch -> undispatch, differentiated by dispatch_backward and undispatch_backward,
    against central differences of the loss in doubles (the loss is linear in x and in the weights: exact up to
    the kernels' own rounding)."""
    T, k, d, E = 7, 3, 64, 4
    rng = np.random.default_rng(12)
    offsets, slot_row = ref.sort_tokens(ref.routing(rng, T, k, E, drop=0.2), E)
    rows = dev(slot_row)
    x = torch.from_numpy(rng.standard_normal((T, d))).to(dtype).cuda()
    w = torch.from_numpy(rng.random((T, k))).float().cuda()
    g = torch.from_numpy(rng.standard_normal((T, d))).to(dtype).cuda()
    xs, dxs = torch.zeros(T * k, d, dtype=dtype, device="cuda"), torch.zeros(T * k, d, dtype=dtype, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    api.moe_dispatch(x, rows, xs)
    api.moe_undispatch_backward(g, xs, rows, w, dxs, dw)
    api.moe_dispatch_backward(dxs, rows, dx)

    xv, wv, gv = (t.double().cpu().numpy() for t in (x, w, g))
    has = slot_row >= 0

    def loss(xv, wv):
        return float(((has * wv).sum(1)[:, None] * xv * gv).sum())

    half = torch.finfo(dtype).eps / 2
    for t in range(T):
        for j in range(k):
            e = np.zeros_like(wv)
            e[t, j] = 0.5
            want = loss(xv, wv + e) - loss(xv, wv - e)
            size = np.abs(xv[t] * gv[t]).sum()
            # 64 products and sums in fp32; the differences lose 2^-52 of the whole loss
            assert abs(dw[t, j].item() - want) <= 24 * 2.0 ** -24 * size + 1e-12
        for i in range(0, d, 7):
            e = np.zeros_like(xv)
            e[t, i] = 0.5
            want = loss(xv + e, wv) - loss(xv - e, wv)
            size = np.abs(has[t] * wv[t] * gv[t, i]).sum()
            # each of k terms rounded to the type, k additions, one more rounding
            assert abs(dx[t, i].item() - want) <= (2 * half + (k + 1) * 2.0 ** -24) * 1.01 * size + 1e-12


def test_the_largest_sort_and_dispatch():
    """T = 4,194,304 tokens, k = 32: 134,217,728 rows, against a stable sort; the last tokens are dropped."""
    T, k, E, d = 1 << 22, 32, 2048, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32, device="cuda")
    idx[-5:] = -1
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    slot_row = torch.empty(T, k, dtype=torch.int32, device="cuda")
    ws = api.alloc_dispatch_workspace()
    api.moe_sort_tokens(idx, offsets, slot_row, ws)
    assert api.moe_device_status(ws) == api.MOE_OK
    key = idx.view(-1).clone()
    key[key < 0] = E
    order = torch.sort(key, stable=True).indices
    n = (T - 5) * k
    assert torch.equal(slot_row.view(-1)[order[:n]].long(), torch.arange(n, device="cuda"))
    assert bool((slot_row[-5:] == -1).all())
    counts = torch.bincount(key[:n], minlength=E)
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)) and offsets[0].item() == 0
    del order, key
    x = torch.randn(T, d, device="cuda").bfloat16()
    xs = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
    api.moe_dispatch(x, slot_row, xs)
    for j in (0, 13, 31):
        assert torch.equal(xs[slot_row[:-5, j].long()], x[:-5])
    assert not bool(xs[n:].any())
    dx = torch.empty_like(x)
    api.moe_dispatch_backward(xs, slot_row, dx)         # 32 equal rows: 32 x, exact
    assert torch.equal(dx[:-5], 32 * x[:-5]) and not bool(dx[-5:].any())
