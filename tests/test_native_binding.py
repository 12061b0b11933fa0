"""The native part of the binding: plain calls are its own and do what the Python part does; all else it leaves."""
import os
import subprocess
import sys
import sysconfig

import numpy as np
import pytest
import torch

import fp4_ref as ref
from mixture_experts_ffn_16_b200 import api
from mixture_experts_ffn_16_b200 import build

T, K, E, D, F = 37, 3, 5, 192, 128
NAMES = ["sort_tokens", "dispatch", "dispatch_backward", "undispatch", "undispatch_backward", "quantize_fp4",
         "dequantize_fp4", "dispatch_fp4", "matmul_fp4", "swiglu_fp4"]


def arguments(name, device):
    """(arguments, the outputs among them) of a call of `name`; the inputs are the same every time."""
    rng = np.random.default_rng(3)
    idx = ref.routing(rng, T, K, E, 0.1, 0.0)
    offsets, slot_row = (torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)
                         for a in ref.sort_tokens(idx, E))

    def rows(*shape, dtype=torch.bfloat16):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(device, dtype)

    def f4(G, n, k):
        codes = torch.from_numpy(rng.integers(0, 256, (G, n, k // 2), dtype=np.uint8)).to(device)
        scales = torch.from_numpy(rng.integers(124, 130, (G, -(-k // 128), n, 4), dtype=np.uint8)).to(device)
        return codes, scales

    def out(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    def f4_out(G, n, k):
        return out(G, n, k // 2, dtype=torch.uint8), out(G, -(-k // 128), n, 4, dtype=torch.uint8)

    ws = torch.zeros(api.DISPATCH_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
    R, i32, f32 = T * K, torch.int32, torch.float32
    if name == "sort_tokens":
        o = [out(E + 1, dtype=i32), out(T, K, dtype=i32)]
        return [torch.from_numpy(idx.astype(np.int32)).to(device), *o, ws], o
    if name == "dispatch":
        o = [out(R, D)]
        return [rows(T, D), slot_row, *o], o
    if name == "dispatch_backward":
        o = [out(T, D)]
        return [rows(R, D), slot_row, *o], o
    if name == "undispatch":
        o = [out(T, D)]
        return [rows(R, D), slot_row, rows(T, K, dtype=f32), *o], o
    if name == "undispatch_backward":
        o = [out(R, D), out(T, K, dtype=f32)]
        return [rows(T, D), rows(R, D), slot_row, rows(T, K, dtype=f32), *o], o
    if name == "quantize_fp4":
        o = f4_out(2, R, D)
        return [rows(2, R, D), *o], o
    if name == "dequantize_fp4":
        o = [out(2, R, D)]
        return [*f4(2, R, D), *o], o
    if name == "dispatch_fp4":
        o = f4_out(1, R, D)
        return [rows(T, D), slot_row, o], o
    if name == "matmul_fp4":
        o = [out(R, F)]
        return [f4(1, R, D), offsets, f4(E, F, D), *o, ws], o
    o = f4_out(1, R, F)
    return [f4(1, R, D), offsets, f4(E, F, D), f4(E, F, D), o, ws], o


class Sub(torch.Tensor):
    pass


def native(name, args):
    return getattr(api._fast(), name)(*args)


@pytest.mark.parametrize("name", NAMES)
def test_leaves_what_is_not_a_plain_call(name):
    """None, and nothing launched: CPU tensors, other objects, too few and too many arguments."""
    args, outs = arguments(name, "cpu")
    assert native(name, args) is None
    assert native(name, args[:-1]) is None
    assert native(name, args + [None]) is None
    for i in range(len(args)):
        assert native(name, args[:i] + [object()] + args[i + 1:]) is None
        assert native(name, args[:i] + [(1, 2)] + args[i + 1:]) is None
    assert all(not o.any() for o in outs)


def test_bind_takes_a_tuple_of_addresses():
    for wrong in (None, [1] * 10, (1,) * 9, (None,) * 10):
        with pytest.raises(TypeError):
            api._fast().bind(wrong)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_makes_plain_calls_as_the_python_part_does(name):
    """On the current stream, whichever that is; the Python part runs where a stream is given."""
    want, want_outs = arguments(name, "cuda")
    getattr(api, "moe_" + name)(*want, stream=torch.cuda.current_stream())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args, outs = arguments(name, "cuda")
    assert native(name, args) == api.MOE_OK
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side, side_outs = arguments(name, "cuda")
        assert native(name, on_side) == api.MOE_OK
    torch.cuda.synchronize()
    assert any(o.any() for o in want_outs)
    for a, b, c in zip(want_outs, outs, side_outs):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_leaves_wrong_tensors_to_the_python_part(name):
    """Each tensor in turn of another type, shape, layout or device, and as a subclass: the first four raise in the
    Python part, which takes the last."""
    args, outs = arguments(name, "cuda")
    flat = [(i, None) for i, a in enumerate(args) if isinstance(a, torch.Tensor)]
    flat += [(i, j) for i, a in enumerate(args) if isinstance(a, tuple) for j in range(2)]
    for i, j in flat:
        t = args[i] if j is None else args[i][j]

        def put(new):
            changed = list(args)
            changed[i] = new if j is None else tuple(new if q == j else args[i][q] for q in range(2))
            return changed

        if t.dim() > 1:
            # one more column is another width, or another tensor's rows or experts
            wider = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype, device="cuda")
            wrong = [t.double(), t.unsqueeze(0), wider[..., :-1], t.cpu()]
        else:
            wrong = [t.double(), t.unsqueeze(0), t.repeat(2)[::2], t.cpu()]
        if t.numel() == api.DISPATCH_WORKSPACE_BYTES:
            del wrong[1]                 # a workspace may have any shape
        for w in wrong:
            assert native(name, put(w)) is None
            with pytest.raises((TypeError, ValueError)):
                getattr(api, "moe_" + name)(*put(w))
        sub = put(t.as_subclass(Sub))
        assert native(name, sub) is None
    torch.cuda.synchronize()
    assert all(not o.any() for o in outs)
    getattr(api, "moe_" + name)(*sub)
    torch.cuda.synchronize()
    assert any(o.any() for o in outs)


def test_file_of_the_native_part_says_what_it_was_compiled_for(monkeypatch, tmp_path):
    """Another torch or Python has another file: what was built for one is neither kept nor loaded for the other."""
    here = build.build_fastcall()
    assert here == build.fastcall_path() and os.path.exists(here)
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert api._fast().__file__ == here
    made = []

    def compiler(cmd):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "w").close()

    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(subprocess, "check_call", compiler)
    first = build.build_fastcall()
    assert len(made) == 1 and build.build_fastcall() == first and len(made) == 1
    monkeypatch.setattr(torch, "__version__", "2.99.0+cu999")
    second = build.build_fastcall()
    assert second != first and len(made) == 2
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-none.so")
    assert build.build_fastcall() not in (first, second) and len(made) == 3


def test_library_is_built_without_torch_or_the_native_part(monkeypatch):
    """The C library first, whatever becomes of the binding's part."""
    code = ("import sys; sys.modules['torch'] = None\nfrom mixture_experts_ffn_16_b200 import build\n"
            "build._newer = lambda out, deps: out == build.LIB\nprint(build.build())")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(build.HERE))
    assert out.returncode == 0 and out.stdout.strip() == build.LIB, out.stderr
    order = []

    def failing(*args):
        order.append("native part")
        raise subprocess.CalledProcessError(1, "g++")

    monkeypatch.setattr(build, "build_library", lambda *args: order.append("library") or build.LIB)
    monkeypatch.setattr(build, "build_fastcall", failing)
    with pytest.warns(UserWarning, match="native part"):
        assert build.build() == build.LIB
    assert order == ["library", "native part"]


@pytest.fixture
def no_native_part(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "fastcall_path", lambda: str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(api, "_fastcall", None)
    with pytest.warns(UserWarning, match="ctypes"):
        api._fast()


@pytest.mark.parametrize("name", NAMES)
def test_without_the_native_part_the_python_part_checks(name, no_native_part):
    args, outs = arguments(name, "cpu")
    assert native(name, args) is None
    with pytest.raises(ValueError):                      # tensors of the host
        getattr(api, "moe_" + name)(*args)
    assert all(not o.any() for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_without_the_native_part_the_python_part_makes_the_calls(name, no_native_part):
    want, want_outs = arguments(name, "cuda")
    getattr(api, "moe_" + name)(*want, stream=torch.cuda.current_stream())
    args, outs = arguments(name, "cuda")
    getattr(api, "moe_" + name)(*args)
    torch.cuda.synchronize()
    assert any(o.any() for o in outs)
    assert all(torch.equal(a, b) for a, b in zip(want_outs, outs))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_refuses_views_that_negate(name):
    """A lazily negated view is contiguous and has the right type, but its memory holds the other sign."""
    args, outs = arguments(name, "cuda")
    for i, a in enumerate(args):
        for j in range(len(a) if isinstance(a, tuple) else 1):
            bad = list(args)
            if isinstance(a, tuple):
                bad[i] = tuple(torch._neg_view(t) if q == j else t for q, t in enumerate(a))
            else:
                bad[i] = torch._neg_view(a)
            assert native(name, bad) is None
            with pytest.raises(ValueError, match="negates"):
                getattr(api, "moe_" + name)(*bad)
    torch.cuda.synchronize()
    assert all(not o.any() for o in outs)


def test_refuses_a_host_view_that_negates():
    with pytest.raises(ValueError, match="x: .*negates"):
        api._p(torch._neg_view(torch.ones(4, 8)), torch.float32, (4, 8), "x", host=True)
