"""What the binding of the norm, the routing and the 8-bit form does around a library call, on the CPU:
the library is a stub that looks at its arguments, and tensors pass for tensors on a GPU."""
import contextlib
import copy
import math
import pickle

import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from error_bounded_lossy_amd import _binding  # noqa: E402
from test_mx_binding import OnGPU, Stub, gpu, holder, stub  # noqa: E402, F401


def form(*shape):
    *lead, cols = shape
    return ec.I8Tensor(gpu(torch.zeros(*lead, -(-cols // 128) * 128, dtype=torch.int8)), gpu(torch.zeros(lead)), cols)


def made(rows, cols):
    """A form as the library makes it."""
    return ec.i8_quantize(gpu(torch.zeros(rows, cols)))


def routing(tokens=6, choices=2, experts=4):
    i32 = lambda *s: gpu(torch.zeros(*s, dtype=torch.int32))  # noqa: E731
    return ec.Routing(i32(tokens * choices), i32(tokens, choices), i32(experts + 1), tokens, choices, experts)


# ---------------------------------------------------------------- workspaces and forms


def test_workspaces_live_through_the_call(stub):  # noqa: F811
    seen = []

    def look(at):
        def f(*args):
            workspace, size = args[at], args[at + 1]
            seen.append((size, len(holder(workspace, size)) if size else workspace))
            return ec.EC_OK
        return f

    stub(ec_i8_linear=look(11), ec_rms_norm_backward=look(11))
    ec.i8_linear(gpu(torch.zeros(100, 256)), form(40, 256))
    ec.i8_experts_linear(gpu(torch.zeros(100, 256)), form(2, 40, 256), gpu(torch.tensor([0, 50, 100], dtype=torch.int32)))
    ec.i8_linear(gpu(torch.zeros(1, 256)), form(40, 256))
    x, w = gpu(torch.zeros(300, 64)), gpu(torch.zeros(64))
    ec.rms_norm_backward(x, ec.rms_norm_forward(x, w)[1])
    ec.rms_norm_backward(x[:0], ec.rms_norm_forward(x[:0], w)[1])
    (size, alive), (size2, alive2), (none, address), (size3, alive3), (none2, address2) = seen
    assert size == size2 == 100 * 260 and alive and alive2
    assert size3 == ec.lib().ec_rms_norm_backward_workspace_bytes(300, 64) and alive3
    assert none == none2 == 0 and address is None and address2 is None


def test_forms_and_their_copies(stub):  # noqa: F811
    stub()
    for q in (form(3, 5, 200), made(7, 200)):
        assert q.codes.dtype == torch.int8 and q.codes.shape == (*q.lead, 256)
        assert q.scales.dtype == torch.float32 and q.scales.shape == q.lead and q.shape == (*q.lead, 200)
        assert q.pointers() == (q.codes.data_ptr(), q.scales.data_ptr())
        assert q.numel_bytes() == math.prod(q.lead) * 260
        q.codes.fill_(3)
        q.scales.fill_(0.5)
        for other in (copy.copy(q), copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
            assert torch.equal(other.codes, q.codes) and torch.equal(other.scales, q.scales) and other.shape == q.shape
        assert copy.deepcopy(q).pointers() != q.pointers()
    q = form(3, 200)
    q.home.data = torch.zeros(3, 256, dtype=torch.int8)  # replaced by memory of the same form
    assert q.pointers()[0] == q.home.data_ptr()
    q.home.data = torch.zeros(2, 256, dtype=torch.int8)
    with pytest.raises(ec.ECError):
        q.pointers()


@pytest.mark.parametrize("codes,scales,cols", [
    (torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(3), 100), (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(3, dtype=torch.float64), 100),
    (torch.zeros(3, 100, dtype=torch.int8), torch.zeros(3), 100), (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(4), 100),
    (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(3, 1), 100), (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(3), -1),
    (torch.zeros(128, 3, dtype=torch.int8).t(), torch.zeros(3), 100), (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(6)[::2], 100),
    (torch.zeros(3, 128, dtype=torch.int8), torch.zeros(3), 129)])
def test_forms_that_are_none(codes, scales, cols):
    with pytest.raises(ec.ECError) as e:
        ec.I8Tensor(codes, scales, cols)
    assert e.value.status == ec.EC_ERR_INVALID


def test_files_of_another_form_are_refused():
    from error_bounded_lossy_amd.i8 import _restored
    for home, lead, cols in ((torch.zeros(3 * 132), (3,), 100), (torch.zeros(3 * 132 - 1, dtype=torch.int8), (3,), 100),
                             (torch.zeros(6 * 132, dtype=torch.int8)[::2], (3,), 100)):
        with pytest.raises(ec.ECError):
            _restored(home, None, lead, cols)


# ---------------------------------------------------------------- what the gradients need


@pytest.mark.parametrize("residual", [False, True])
def test_saved_tensors_that_were_written_to_are_refused(stub, residual):  # noqa: F811
    s = stub()
    for which in ("h", "weight"):
        x, w, dy = gpu(torch.zeros(6, 64)), gpu(torch.zeros(64)), gpu(torch.zeros(6, 64))
        _, saved = ec.rms_norm_forward(x, w, residual=gpu(torch.zeros(6, 64)) if residual else None)
        assert (saved.h is x) == (not residual) and saved.weight is w
        ec.rms_norm_backward(dy, saved)
        for other in (copy.copy(saved), copy.deepcopy(saved), pickle.loads(pickle.dumps(saved))):
            ec.rms_norm_backward(dy, other)
        calls = len(s.calls)
        kept = copy.deepcopy(saved)
        getattr(saved, which).add_(1)
        for call in (lambda: ec.rms_norm_backward(dy, saved), lambda: copy.copy(saved), lambda: pickle.dumps(saved)):
            with pytest.raises(ec.ECError) as e:
                call()
            assert e.value.status == ec.EC_ERR_INVALID
        assert len(s.calls) == calls
        ec.rms_norm_backward(dy, kept)


def test_saved_inference_tensors_and_graphs(stub, monkeypatch):  # noqa: F811
    stub()
    with torch.inference_mode():
        x, w = gpu(torch.zeros(6, 64)), gpu(torch.zeros(64))
        _, saved = ec.rms_norm_forward(x, w)
    ec.rms_norm_backward(gpu(torch.zeros(6, 64)), saved)
    monkeypatch.setattr(_binding, "capturing", lambda t: True)
    x, w = gpu(torch.zeros(6, 64)), gpu(torch.zeros(64))
    _, saved = ec.rms_norm_forward(x, w)
    x.add_(1)  # what a replay reads is what the graph's input holds then
    ec.rms_norm_backward(gpu(torch.zeros(6, 64)), saved)


# ---------------------------------------------------------------- refusals


def refusals():
    z = lambda *s, t=torch.float32: gpu(torch.zeros(s, dtype=t))  # noqa: E731
    x, w, r = z(6, 64), z(64), routing()
    off = z(3, t=torch.int32)
    ids = z(6, 2, t=torch.int32)
    saved = ("saved", x, w)
    host = torch.zeros(6, 64)
    return [
        ("i8_quantize", (z(6, 0),)), ("i8_quantize", (z(6, 4, t=torch.float64),)), ("i8_quantize", (host,)), ("i8_quantize", (z(),)),
        ("i8_dequantize", (form(6, 64), torch.float64)), ("i8_dequantize", (form(6, 0), torch.float32)),
        ("i8_product", (form(6, 64), form(3, 65))), ("i8_product", (form(6, 64), form(2, 3, 64))), ("i8_product", (form(6, 64), form(0, 64))),
        ("i8_product", (form(6, 64), form(3, 64), torch.int8)), ("i8_product", (form(6, 0), form(3, 0))),
        ("i8_linear", (x, form(2, 3, 64))), ("i8_linear", (x, form(3, 63))), ("i8_linear", (x, form(0, 64))), ("i8_linear", (host, form(3, 64))),
        ("i8_linear", (z(), form(3, 64))),
        ("i8_experts_linear", (x, form(3, 64), off)), ("i8_experts_linear", (x, form(3, 8, 64), off)), ("i8_experts_linear", (z(1, 6, 64), form(2, 8, 64), off)),
        ("i8_experts_linear", (x, form(2, 8, 64), z(3, t=torch.int64))),
        ("i8_experts_product", (form(6, 64), form(2, 8, 64), z(4, t=torch.int32))), ("i8_experts_product", (form(6, 64), form(8, 64), off)),
        ("i8_experts_product", (form(6, 64), form(2, 0, 64), off)), ("i8_experts_product", (form(6, 64), form(2, 8, 64), off, torch.float64)),
        ("rms_norm", (x, z(63))), ("rms_norm", (x, z(1, 64))), ("rms_norm", (x, z(64, t=torch.float64))), ("rms_norm", (host, w)), ("rms_norm", (x, w, 1e-5, z(6, 63))),
        ("rms_norm", (x, w, 1e-5, z(6, 64, t=torch.float16))), ("rms_norm", (z(6, 0), z(0))), ("rms_norm", (z(), w)), ("rms_norm_i8", (x, z(63))),
        ("rms_norm_i8", (x, w, 1e-5, z(5, 64))), ("rms_norm_forward", (x, z(65))),
        ("rms_norm_backward", (z(6, 63), saved)), ("rms_norm_backward", (z(6, 64, t=torch.float16), saved)), ("rms_norm_backward", (x, saved, z(5, 64))),
        ("rms_norm_backward", (x, saved, z(6, 64, t=torch.bfloat16))),
        ("expert_route", (x, 0)), ("expert_route", (x, 65)), ("expert_route", (x, 2, "tanh")), ("expert_route", (x, 2, "softmax", z(63))),
        ("expert_route", (x, 2, "softmax", z(64, t=torch.float16))), ("expert_route", (x, 2, "softmax", None, 3)), ("expert_route", (x, 2, "softmax", None, 0)),
        ("expert_route", (x, 2, "softmax", None, 4, 0)), ("expert_route", (x, 2, "softmax", None, 4, 5)), ("expert_route", (x, 33, "softmax", None, 4, 2)),
        ("expert_route", (x, 2, "softmax", None, 1, 1, True, math.nan)), ("expert_route", (z(6, 0), 1)), ("expert_route", (z(2, 3, 4), 1)), ("expert_route", (host, 2)),
        ("expert_route_backward", (z(6, 2), x, z(6, 2, t=torch.int64))), ("expert_route_backward", (z(6, 3), x, ids)), ("expert_route_backward", (z(6, 2, t=torch.float16), x, ids)),
        ("expert_route_backward", (z(5, 2), x, ids[:5])), ("expert_route_backward", (z(6, 0), x, ids[:, :0])), ("expert_route_backward", (z(6, 2), x, ids, "none")),
        ("expert_route_backward", (z(6, 2), x, ids, "softmax", True, math.inf)), ("expert_route_backward", (z(12), x, z(12, t=torch.int32))),
        ("expert_dispatch_i8", (form(5, 64), r)), ("expert_dispatch_i8", (form(2, 3, 64), r)), ("expert_dispatch_i8", (form(6, 0), r)),
    ]


@pytest.mark.parametrize("at", range(len(refusals())))
def test_refusals(stub, at):  # noqa: F811
    s = stub()
    name, args = refusals()[at]
    args = [ec.RMSNormSaved(a[1], gpu(torch.zeros(6)), a[2]) if isinstance(a, tuple) else a for a in args]
    with pytest.raises(ec.ECError) as e:
        getattr(ec, name)(*args)
    assert e.value.status == ec.EC_ERR_INVALID and not s.calls, name


# ---------------------------------------------------------------- every call, on a stream of its own


def every_call():
    x, w = gpu(torch.zeros(6, 64)), gpu(torch.zeros(64))
    offsets = gpu(torch.tensor([0, 3, 6], dtype=torch.int32))
    dw, i = gpu(torch.zeros(6, 2)), gpu(torch.zeros(6, 2, dtype=torch.int32))
    _, saved = ec.rms_norm_forward(x, w, residual=gpu(torch.zeros(6, 64)))
    return {
        "i8_quantize": (x,), "i8_dequantize": (made(6, 64), torch.float16), "i8_product": (form(6, 64), made(32, 64), torch.float16),
        "i8_linear": (x, form(32, 64)), "i8_experts_linear": (x, form(2, 32, 64), offsets),
        "i8_experts_product": (form(6, 64), form(2, 32, 64), offsets, torch.float16),
        "rms_norm": (x, w, 1e-5, gpu(torch.zeros(6, 64))), "rms_norm_i8": (x, w, 1e-5, gpu(torch.zeros(6, 64))), "rms_norm_forward": (x, w),
        "rms_norm_backward": (x, saved, gpu(torch.zeros(6, 64))),
        "expert_route": (x, 2, "sigmoid", w, 4, 2, True, 2.5), "expert_route_backward": (dw, x, i, "sigmoid", False, 2.5),
        "expert_dispatch_i8": (made(6, 64), routing()),
    }


@pytest.mark.parametrize("elsewhere", [False, True])
def test_calls_elsewhere_make_the_same_library_calls(monkeypatch, stub, elsewhere):  # noqa: F811
    class Stream:
        device, stream_id = torch.device("cpu"), 1

    seen = []
    monkeypatch.setattr(Stub, "__getattr__", lambda self, name: (
        getattr(self.real, name) if name.endswith("_bytes") or "padded" in name else
        lambda *args: (seen.append((name, args)), ec.EC_OK)[1]))
    stub()
    for name in ("device", "stream"):
        monkeypatch.setattr(torch.cuda, name, lambda *a: contextlib.nullcontext())
    recorded = []
    monkeypatch.setattr(OnGPU, "record_stream", lambda self, s: recorded.append(self.data_ptr()), raising=False)
    public = {n for names in ec._LAYER_OPERATORS.values() for n in names if n[0].islower()}
    calls = every_call()
    assert set(calls) == public
    inputs = lambda args: [v for v in args if not isinstance(v, int) or 0 <= v < 1 << 32]  # noqa: E731 (no addresses)
    for name, args in calls.items():
        seen.clear()
        getattr(ec, name)(*args)
        plain = [(n, inputs(a)) for n, a in seen]
        seen.clear()
        recorded.clear()
        away = [True]
        if elsewhere:  # once: the call under the device is not elsewhere any more
            monkeypatch.setattr(_binding, "elsewhere", lambda t: away.pop() if away else False)
            getattr(ec, name)(*args)
            assert not away and not recorded
        else:
            getattr(ec, name)(*args, stream=Stream())
            assert {t.data_ptr() for a in args for t in _binding._tensors(a)} == set(recorded)
        assert [(n, inputs(a)) for n, a in seen] == plain and plain, name


def test_keyword_arguments_reach_the_library(stub):  # noqa: F811
    seen = []
    stub(ec_expert_route=lambda *a: (seen.append(a), ec.EC_OK)[1], ec_expert_route_backward=lambda *a: (seen.append(a), ec.EC_OK)[1])
    l, b = gpu(torch.zeros(6, 64)), gpu(torch.zeros(64))
    ids, weights = ec.expert_route(l, 3, score="sigmoid", bias=b, groups=8, top_groups=4, renormalize=False, scale=2.5)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32 and ids.shape == weights.shape == (6, 3)
    assert seen[0][:6] == (l.data_ptr(), 0, 6, 64, 64, b.data_ptr()) and seen[0][6:12] == (3, 1, 8, 4, False, 2.5)
    assert seen[0][12:14] == (ids.data_ptr(), weights.data_ptr())
    d = ec.expert_route_backward(weights, l, ids, score="sigmoid", renormalize=False, scale=2.5)
    assert seen[1][:7] == (weights.data_ptr(), l.data_ptr(), 0, 6, 64, 64, ids.data_ptr()) and seen[1][7:11] == (3, 1, False, 2.5)
    assert seen[1][11] == d.data_ptr() and d.shape == l.shape and d.dtype == l.dtype
