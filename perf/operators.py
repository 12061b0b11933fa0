"""Cases of the token-dispatch and MXFP4 expert operators, with their plain forms.

Operators (all of ``mixture_experts_ffn_16_b200.api``):
  dispatch     moe_sort_tokens + moe_dispatch (training: + moe_dispatch_backward)
  undispatch   moe_undispatch (training: + moe_undispatch_backward)
  quantize     moe_quantize_fp4, and back with moe_dequantize_fp4
  matmul       moe_matmul_fp4: the experts' products of sorted rows
  ffn          moe_sort_tokens, moe_dispatch_fp4, moe_swiglu_fp4, moe_matmul_fp4: the expert FFN up to the
               sorted rows that moe_undispatch takes

MXFP4: blocks of 32 consecutive values share a power-of-two scale 2^(floor(log2 max|x|) - 2), stored as its
biased exponent byte; a value is the nearest E2M1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code) of
x / scale, at most 6.  Codes lie two to a byte (the even element in the low half) as [G, rows, K/2]; scale bytes
as [G, ceil(K/128), rows, 4].

With ``own`` false, ``run`` computes the operators from elementary torch operations in fp32.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a 512-expert layer: 64 sequences, one token each
        dict(name="dispatch_decode", op="dispatch", T=64, d=4096, k=10, E=512, dtype="bf16", drop=0.0, train=False),
        # a training micro-batch of a 256-expert layer whose last tokens are padding (expert -1)
        dict(name="dispatch_train", op="dispatch", T=8191, d=2048, k=8, E=256, dtype="bf16", drop=0.06, train=True),
        # back to token order, decode
        dict(name="undispatch_decode", op="undispatch", T=64, d=4096, k=10, E=512, dtype="bf16", drop=0.0,
             train=False),
        # back to token order with the gradients of rows and weights, fp32 rows as kept for a master-precision run
        dict(name="undispatch_train", op="undispatch", T=4095, d=2048, k=8, E=256, dtype="fp32", drop=0.06,
             train=True),
        # a layer's expert weights, quantised as they would be when a checkpoint is loaded, and read back
        dict(name="quantize_weights", op="quantize", G=64, rows=1024, K=2048, dtype="bf16"),
        # activation rows of an odd batch, quantised and read back (quantisation-aware training)
        dict(name="quantize_rows", op="quantize", G=1, rows=4097, K=7168, dtype="fp32"),
        # down product of one decode step: few rows an expert, the weights' bytes count
        dict(name="matmul_decode", op="matmul", T=64, k=10, E=512, N=4096, K=1024, dtype="bf16", skew=0.0, drop=0.0),
        # ragged: sizes that are no multiple of a tile, a skewed load, empty experts, rows behind the last expert
        dict(name="matmul_ragged", op="matmul", T=1001, k=3, E=40, N=1088, K=704, dtype="fp16", skew=1.0, drop=0.1),
        # large experts: 512 rows each
        dict(name="matmul_large", op="matmul", T=8192, k=4, E=64, N=4096, K=4096, dtype="bf16", skew=0.0, drop=0.0),
        # one decode step's whole expert FFN on a 512-expert layer
        dict(name="ffn_decode", op="ffn", T=64, d=4096, f=1024, k=10, E=512, skew=0.0, drop=0.0),
        # a prefill of 4,096 tokens on a 256-expert layer
        dict(name="ffn_prefill", op="ffn", T=4096, d=2048, f=512, k=8, E=256, skew=0.0, drop=0.0),
        # a prefill of 8,192 tokens on a 384-expert layer, load skewed, the batch padded at its end
        dict(name="ffn_large", op="ffn", T=8192, d=4096, f=1024, k=8, E=384, skew=0.25, drop=0.03),
    ]


def _log_int(rng, lo, hi, step=1):
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["dispatch", "undispatch", "quantize", "matmul", "ffn"])
    if op in ("dispatch", "undispatch"):
        T, d = _log_int(rng, 1, 8191), _log_int(rng, 64, 7168, 64)
        E = _log_int(rng, 8, 896)
        k = rng.randint(1, min(E, 22))
        while T * k * d > 8191 * 8 * 2048 // (1 if op == "dispatch" else 2):
            T = T // 2
        return dict(op=op, T=T, d=d, k=k, E=E, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    drop=rng.choice([0.0, 0.1]), train=rng.random() < 0.5)
    if op == "quantize":
        K = _log_int(rng, 64, 7168, 64)
        G, rows = rng.choice([1, 1, 3, 16]), _log_int(rng, 1, 4097)
        while G * rows * K > 64 * 1024 * 2048:
            rows //= 2
        return dict(op=op, G=G, rows=rows, K=K, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "matmul":
        E = _log_int(rng, 1, 256)
        k = rng.randint(1, min(E, 10))
        T, N, K = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096, 64), _log_int(rng, 64, 4096, 64)
        while E * N * K > 64 * 4096 * 4096:
            E //= 2
        k = min(k, E)
        while T * k * N * K > 8192 * 4 * 4096 * 4096 or T * k > 32768:
            T //= 2
        return dict(op=op, T=T, k=k, E=E, N=N, K=K, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    skew=rng.choice([0.0, 0.3]), drop=rng.choice([0.0, 0.1]))
    d, f, E = _log_int(rng, 64, 4096, 64), _log_int(rng, 64, 1024, 64), _log_int(rng, 2, 384)
    k = rng.randint(1, min(E, 10))
    T = _log_int(rng, 1, 8192)
    while T * k > 65536:
        T //= 2
    return dict(op="ffn", T=T, d=d, f=f, k=k, E=E, skew=rng.choice([0.0, 0.3]), drop=rng.choice([0.0, 0.1]))


def _touched(c):
    """Experts that some token picks, expected for an even load."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** _live(c))


def _live(c):
    return c["T"] - int(c["T"] * c.get("drop", 0.0))


def work(c):
    op = c["op"]
    if op == "quantize":
        n = c["G"] * c["rows"] * c["K"]
        es = DT[c["dtype"]].itemsize
        return {"bytes": 2.0 * n * (es + 0.5 + 1.0 / 32), "flops": 4.0 * n}
    T, k, L = c["T"], c["k"], _live(c)
    R = L * k
    if op == "dispatch":
        es = DT[c["dtype"]].itemsize
        one = es * c["d"] * (L + R)                        # every live row in once, every copy out once
        return {"bytes": 8.0 * T * k + 4 * c["E"] + one * (2 if c["train"] else 1),
                "flops": float(R * c["d"] if c["train"] else 0)}
    if op == "undispatch":
        es = DT[c["dtype"]].itemsize
        one = es * c["d"] * (R + T) + 8.0 * T * k
        return {"bytes": one + (es * c["d"] * (T + 2 * R) + 12.0 * T * k if c["train"] else 0.0),
                "flops": float(2 * R * c["d"] * (2.5 if c["train"] else 1))}
    four = 0.5 + 1.0 / 32
    if op == "matmul":
        N, K = c["N"], c["K"]
        return {"bytes": _touched(c) * N * K * four + R * K * four + R * N * DT[c["dtype"]].itemsize,
                "flops": 2.0 * R * N * K}
    d, f = c["d"], c["f"]
    return {"bytes": _touched(c) * 3 * f * d * four + 2.0 * L * d + 2.0 * R * d + 4.0 * T * k,
            "flops": 6.0 * R * f * d}


# ---------------------------------------------------------------- inputs

def _route(c, g):
    """topk_idx int32 [T, k]: k distinct experts a token, the load even or Zipf-like; the last tokens are padding (-1)."""
    T, E, k = c["T"], c["E"], c["k"]
    score = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)))
    if c.get("skew"):
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        score -= c["skew"] * torch.log(rank)
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    idx[_live(c):] = -1
    return idx.contiguous()


def _randn(shape, std, g, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _fp4_weights(G, rows, K, g):
    """(codes, scales) of G matrices drawn from N(0, 0.02), made in slabs."""
    codes = torch.empty(G, rows, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(G, (K + 127) // 128, rows, 4, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (rows * K))
    for i in range(0, G, step):
        n = min(step, G - i)
        w = torch.randn((n, rows, K), generator=g, device=DEV) * 0.02
        codes[i:i + n], scales[i:i + n] = quantize(w)
    return codes, scales


def _sorted_plan(idx, E):
    """What moe_sort_tokens writes, for cases that start behind it."""
    offsets, slot_row, _ = sort_tokens(idx, E)
    return offsets, slot_row


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(c)
    op = c["op"]
    if op == "quantize":
        dt = DT[c["dtype"]]
        G, rows, K = c["G"], c["rows"], c["K"]
        # rows of different magnitude, a few large values as activations have
        mag = torch.exp(torch.randn(G, rows, 1, generator=g, device=DEV) * 0.7)
        x = torch.randn(G, rows, K, generator=g, device=DEV) * mag
        x[..., :: max(1, K // 7)] *= 20.0
        s["x"] = x.to(dt)
        s["codes"] = torch.zeros(G, rows, K // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(G, (K + 127) // 128, rows, 4, dtype=torch.uint8, device=DEV)
        s["back"] = torch.zeros_like(s["x"])
        return s
    T, k, E = c["T"], c["k"], c["E"]
    R = T * k
    s["topk_idx"] = idx = _route(c, g)
    s["ws"] = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    if op == "dispatch":
        dt = DT[c["dtype"]]
        s["x"] = _randn((T, c["d"]), 1.0, g, dt)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        s["slot_row"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
        s["x_sorted"] = torch.zeros(R, c["d"], dtype=dt, device=DEV)
        if c["train"]:
            s["dx_sorted"] = _randn((R, c["d"]), 1.0, g, dt)
            s["dx"] = torch.zeros(T, c["d"], dtype=dt, device=DEV)
        return s
    s["offsets"], s["slot_row"] = _sorted_plan(idx, E)
    counts = s["offsets"][1:] - s["offsets"][:-1]
    s["most"] = max(1, int(counts.max()))                  # the plain form's padding
    if op == "undispatch":
        dt = DT[c["dtype"]]
        s["y"] = _randn((R, c["d"]), 1.0, g, dt)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["topk_w"] = w / w.sum(1, keepdim=True)
        s["out"] = torch.zeros(T, c["d"], dtype=dt, device=DEV)
        if c["train"]:
            s["dout"] = _randn((T, c["d"]), 1.0, g, dt)
            s["dy"] = torch.zeros(R, c["d"], dtype=dt, device=DEV)
            s["dw"] = torch.zeros(T, k, dtype=torch.float32, device=DEV)
        return s
    if op == "matmul":
        N, K = c["N"], c["K"]
        s["a"] = quantize(torch.randn(1, R, K, generator=g, device=DEV))
        s["w"] = _fp4_weights(E, N, K, g)
        s["out"] = torch.zeros(R, N, dtype=DT[c["dtype"]], device=DEV)
        return s
    d, f = c["d"], c["f"]
    s["x"] = _randn((T, d), 1.0, g, torch.bfloat16)
    s["w_gate"], s["w_up"] = _fp4_weights(E, f, d, g), _fp4_weights(E, f, d, g)
    s["w_down"] = _fp4_weights(E, d, f, g)
    u8 = dict(dtype=torch.uint8, device=DEV)
    s["a"] = torch.zeros(1, R, d // 2, **u8), torch.zeros(1, (d + 127) // 128, R, 4, **u8)
    s["h"] = torch.zeros(1, R, f // 2, **u8), torch.zeros(1, (f + 127) // 128, R, 4, **u8)
    s["out"] = torch.zeros(R, d, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def sort_tokens(idx, E):
    """(offsets int32 [E+1], slot_row int32 [T, k] (-1: no expert), live slots first in expert order)."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = counts[:E].cumsum(0)
    rows = torch.empty_like(key)
    rows[order] = torch.arange(key.numel(), device=idx.device)
    slot_row = torch.where(key < E, rows, -1)
    return offsets.int(), slot_row.int().reshape(idx.shape), order


def _two_to(e):
    """2^e in fp32 for whole e from -127 to 127, put together from its bits (a power function may be an ulp off)."""
    bits = torch.where(e > -127, (e.int() + 127) << 23, 1 << 22)
    return bits.int().view(torch.float32)


def quantize(x):
    """(codes, scales) of x [G, rows, K]."""
    G, rows, K = x.shape
    v = x.float().reshape(G, rows, K // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    exp = (torch.frexp(amax).exponent - 3).clamp(min=-127)           # floor(log2 amax) - 2
    exp = torch.where(amax > 0, exp, -127)
    q = v * _two_to(-exp)
    m = q.abs()
    step = 0.5 + 0.5 * (m >= 2) + (m >= 4)                           # spacing of the numbers around m
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = (2 * m).clamp(max=4) + (m - 2).clamp(0, 2) + (m - 4).clamp(0, 2) / 2
    code = code.to(torch.uint8) + (q < 0).to(torch.uint8) * 8
    code = code.reshape(G, rows, K // 2, 2)
    codes = code[..., 0] + code[..., 1] * 16
    byte = torch.zeros(G, rows, (K + 127) // 128 * 4, dtype=torch.uint8, device=x.device)
    byte[..., :K // 32] = (exp + 127).to(torch.uint8)[..., 0]
    return codes, byte.reshape(G, rows, -1, 4).transpose(1, 2).contiguous()


def dequantize(codes, scales):
    """fp32 [G, rows, K] of what quantize gives."""
    G, rows, half = codes.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    both = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)      # byte -> its two values
    v = both[codes.int()].reshape(G, rows, 2 * half // 32, 32)
    byte = scales.transpose(1, 2).reshape(G, rows, -1)[..., :2 * half // 32]
    return (v * _two_to(byte.int().unsqueeze(-1) - 127)).reshape(G, rows, 2 * half)


def _expert_rows(offsets, R, E):
    """(expert of each sorted row, E behind the last one; place inside the expert)."""
    at = torch.arange(R, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), at, right=True)
    return e, at - offsets.long()[e]


def _grouped(a, w, offsets, most):
    """fp32 [R, N]: row r of a times the matrix of r's expert, 0 behind the last expert."""
    E, R = w.shape[0], a.shape[0]
    e, at = _expert_rows(offsets, R, E)
    at = torch.where(e < E, at, 0)
    padded = torch.zeros(E + 1, most, a.shape[1], device=a.device)
    padded[e, at] = a
    y = torch.bmm(padded[:E], w.transpose(1, 2))
    return torch.where((e < E)[:, None], y[e.clamp(max=E - 1), at], 0.0)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        codes, scales = quantize(s["x"])
        return {"scales": scales, "back": dequantize(codes, scales).to(s["x"].dtype)}
    E = s["E"]
    if op == "dispatch":
        x, k = s["x"], s["k"]
        offsets, slot_row, order = sort_tokens(s["topk_idx"], E)
        live = torch.arange(order.numel(), device=x.device) < offsets[E]
        out = {"offsets": offsets, "slot_row": slot_row,
               "x_sorted": torch.where(live[:, None], x[order // k], torch.zeros((), dtype=x.dtype, device=x.device))}
        if s["train"]:
            rows = s["dx_sorted"][slot_row.long().clamp(min=0)].float()
            out["dx"] = torch.where((slot_row >= 0)[..., None], rows, 0.0).sum(1).to(x.dtype)
        return out
    if op == "undispatch":
        y, w, row = s["y"], s["topk_w"], s["slot_row"].long()
        has = (row >= 0)[..., None]
        rows = torch.where(has, y[row.clamp(min=0)].float(), 0.0)
        out = {"out": (rows * w[..., None]).sum(1).to(y.dtype)}
        if s["train"]:
            dout = s["dout"].float()[:, None, :]
            out["dw"] = (dout * rows).sum(-1)
            dy = torch.zeros(y.shape[0] + 1, y.shape[1], dtype=y.dtype, device=y.device)
            dy[torch.where(row >= 0, row, y.shape[0])] = (dout * w[..., None]).to(y.dtype)
            out["dy"] = dy[:-1]
        return out
    if op == "matmul":
        a = dequantize(*s["a"])[0]
        return _grouped(a, dequantize(*s["w"]), s["offsets"], s["most"]).to(DT[s["dtype"]])
    offsets, slot_row, order = sort_tokens(s["topk_idx"], E)
    a = dequantize(*quantize(s["x"][None]))[0][order // s["k"]]
    gate = _grouped(a, dequantize(*s["w_gate"]), offsets, s["most"])
    up = _grouped(a, dequantize(*s["w_up"]), offsets, s["most"])
    h = gate / (1.0 + torch.exp(-gate)) * up
    h = dequantize(*quantize(h[None]))[0]
    return _grouped(h, dequantize(*s["w_down"]), offsets, s["most"]).to(torch.bfloat16)


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from mixture_experts_ffn_16_b200 import api
    op = s["op"]
    if op == "quantize":
        api.moe_quantize_fp4(s["x"], s["codes"], s["scales"])
        api.moe_dequantize_fp4(s["codes"], s["scales"], s["back"])
        return {"scales": s["scales"], "back": s["back"]}
    if op == "dispatch":
        api.moe_sort_tokens(s["topk_idx"], s["offsets"], s["slot_row"], s["ws"])
        api.moe_dispatch(s["x"], s["slot_row"], s["x_sorted"])
        out = {"offsets": s["offsets"], "slot_row": s["slot_row"], "x_sorted": s["x_sorted"]}
        if s["train"]:
            api.moe_dispatch_backward(s["dx_sorted"], s["slot_row"], s["dx"])
            out["dx"] = s["dx"]
        return out
    if op == "undispatch":
        api.moe_undispatch(s["y"], s["slot_row"], s["topk_w"], s["out"])
        out = {"out": s["out"]}
        if s["train"]:
            api.moe_undispatch_backward(s["dout"], s["y"], s["slot_row"], s["topk_w"], s["dy"], s["dw"])
            out.update(dw=s["dw"], dy=s["dy"])
        return out
    if op == "matmul":
        api.moe_matmul_fp4(s["a"], s["offsets"], s["w"], s["out"], s["ws"])
        return s["out"]
    api.moe_sort_tokens(s["topk_idx"], s["offsets"], s["slot_row"], s["ws"])
    api.moe_dispatch_fp4(s["x"], s["slot_row"], s["a"])
    api.moe_swiglu_fp4(s["a"], s["offsets"], s["w_gate"], s["w_up"], s["h"], s["ws"])
    api.moe_matmul_fp4(s["h"], s["offsets"], s["w_down"], s["out"], s["ws"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    return _plain(s)


# ---------------------------------------------------------------- 64 bits, from the definitions

def _pow2(e):
    """2^e in doubles for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e2m1(x):
    """What a [..., K] tensor of doubles becomes in MXFP4, in doubles: the nearest of the 15 numbers, found by
    comparing with the midpoints (a tie goes to the number whose code is even)."""
    shape = x.shape
    x = x.reshape(-1, 32)
    top = x.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = torch.where(_pow2(e) > top, e - 1, e)
    e = torch.where(_pow2(e + 1) <= top, e + 1, e)
    scale = _pow2((e - 2).clamp(min=-127))
    m = x.abs() / scale
    r = torch.zeros_like(m)
    r = torch.where(m > 0.25, 0.5, r)
    r = torch.where(m >= 0.75, 1.0, r)
    r = torch.where(m > 1.25, 1.5, r)
    r = torch.where(m >= 1.75, 2.0, r)
    r = torch.where(m > 2.5, 3.0, r)
    r = torch.where(m >= 3.5, 4.0, r)
    r = torch.where(m > 5.0, 6.0, r)
    return (torch.sign(x) * r * scale).reshape(shape), scale.reshape(shape[:-1] + (-1,))


def _wide(pair, g):
    """Matrix g of a (codes, scales) pair in doubles."""
    codes, scales = pair[0][g].to(torch.int64), pair[1][g]
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    val = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                       device=codes.device)[nib]
    byte = torch.cat(list(scales), 1)[:, :nib.shape[1] // 32]
    return val * _pow2(byte.long() - 127).repeat_interleave(32, 1)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "quantize":
        back, scale = _e2m1(s["x"].double())
        return {"scales": None, "back": back}
    T, k, E = c["T"], c["k"], c["E"]
    R = T * k
    idx = s["topk_idx"].cpu().tolist()
    lists = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= idx[t][j] < E:
                lists[idx[t][j]].append((t, j))
    slots = [p for one in lists for p in one]
    dev = s["topk_idx"].device
    tok = torch.tensor([p[0] for p in slots], dtype=torch.int64, device=dev)
    col = torch.tensor([p[1] for p in slots], dtype=torch.int64, device=dev)
    n = len(slots)
    if op == "dispatch":
        out = {"offsets": None, "slot_row": None, "x_sorted": torch.zeros(R, c["d"], dtype=torch.float64, device=dev)}
        out["x_sorted"][:n] = s["x"].double()[tok]
        if c["train"]:
            out["dx"] = torch.zeros(T, c["d"], dtype=torch.float64, device=dev)
            for j in range(k):
                out["dx"][tok[col == j]] += s["dx_sorted"][:n].double()[col == j]
        return out
    if op == "undispatch":
        w = s["topk_w"].double()
        out = {"out": torch.zeros(T, c["d"], dtype=torch.float64, device=dev)}
        for j in range(k):
            out["out"][tok[col == j]] += w[tok[col == j], j, None] * s["y"][:n].double()[col == j]
        if c["train"]:
            out["dy"] = torch.zeros(R, c["d"], dtype=torch.float64, device=dev)
            out["dy"][:n] = w[tok, col][:, None] * s["dout"].double()[tok]
            out["dw"] = torch.zeros(T, k, dtype=torch.float64, device=dev)
            out["dw"][tok, col] = torch.einsum("rd,rd->r", s["y"][:n].double(), s["dout"].double()[tok])
        return out
    if op == "matmul":
        out = torch.zeros(R, c["N"], dtype=torch.float64, device=dev)
        a, at = _wide(s["a"], 0), 0
        for e in range(E):
            m = len(lists[e])
            if m:
                out[at:at + m] = a[at:at + m] @ _wide(s["w"], e).T
            at += m
        return out
    out = torch.zeros(R, c["d"], dtype=torch.float64, device=dev)
    x, at = _e2m1(s["x"].double())[0], 0
    for e in range(E):
        m = len(lists[e])
        if m:
            rows = x[tok[at:at + m]]
            z = rows @ _wide(s["w_gate"], e).T
            h = z * torch.sigmoid(z) * (rows @ _wide(s["w_up"], e).T)
            out[at:at + m] = _e2m1(h)[0] @ _wide(s["w_down"], e).T
        at += m
    return out
