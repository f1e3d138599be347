"""What the binding of the 4-bit and exchange operators does around a library call, on the CPU:
the library is a stub that looks at its arguments, and tensors pass for tensors on a GPU."""
import copy
import gc
import pickle

import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from error_bounded_lossy_amd import _binding  # noqa: E402


class OnGPU(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    is_cuda = True

    def __deepcopy__(self, memo):
        return gpu(self.as_subclass(torch.Tensor).clone())


def gpu(t):
    return t.as_subclass(OnGPU)


class Stub:
    """A library whose functions do nothing but `looks[name](*args)`; sizes come from the real one."""

    def __init__(self, **looks):
        self.looks, self.calls, self.real = looks, [], ec.lib()

    def __getattr__(self, name):
        if name.endswith("_bytes") or "padded" in name:
            return getattr(self.real, name)

        def call(*args):
            self.calls.append(name)
            return self.looks[name](*args) if name in self.looks else ec.EC_OK
        return call


@pytest.fixture
def stub(monkeypatch):
    def install(**looks):
        s = Stub(**looks)
        monkeypatch.setattr(_binding, "lib", lambda: s)
        monkeypatch.setattr(_binding, "current_stream", lambda t: 0)
        monkeypatch.setattr(_binding, "elsewhere", lambda t: False)
        return s
    return install


def holder(address, size):
    """The tensors alive whose memory holds [address, address + size)."""
    held = []
    for o in gc.get_objects():
        if issubclass(type(o), torch.Tensor):
            start = o.untyped_storage().data_ptr()
            if start <= address and address + size <= start + o.untyped_storage().nbytes():
                held.append(o)
    return held


def form(*shape):
    *lead, cols = shape
    p = (cols + 127) // 128 * 128
    return ec.MXTensor(gpu(torch.zeros(*lead, p // 2, dtype=torch.uint8)),
                       gpu(torch.zeros(*lead, p // 32, dtype=torch.uint8)), cols)


# Until the call is back its kernels are not enqueued: memory that is free by then may be given to
# another thread's work on the same stream, or back to the driver.
def test_the_workspace_of_a_product_lives_through_the_call(stub):
    seen = []

    def look(*args):
        workspace, size = args[11], args[12]
        seen.append((size, len(holder(workspace, size)) if size else workspace))
        return ec.EC_OK

    stub(ec_mx_linear=look)
    ec.mx_linear(gpu(torch.zeros(100, 256)), form(40, 256))
    offsets = gpu(torch.tensor([0, 50, 100], dtype=torch.int32))
    ec.mx_experts_linear(gpu(torch.zeros(100, 256)), form(2, 40, 256), offsets)
    ec.mx_linear(gpu(torch.zeros(1, 256)), form(40, 256))
    (size, alive), (size2, alive2), (none, address) = seen
    assert size == size2 == 100 * (128 + 8) and alive and alive2
    assert none == 0 and address is None


def test_the_workspace_of_a_sort_lives_through_the_call(stub):
    seen = []

    def look(*args):
        workspace, size = args[7], args[8]
        seen.append((size, len(holder(workspace, size)) if size else workspace))
        return ec.EC_OK

    stub(ec_expert_sort=look)
    ec.expert_sort(gpu(torch.zeros(4000, 2, dtype=torch.int32)), 8)
    ec.expert_sort(gpu(torch.zeros(10, 2, dtype=torch.int32)), 8)
    (size, alive), (none, address) = seen
    assert size == 8 * 9 * 4 and alive
    assert none == 0 and address is None


def experts_saved(inference=False):
    with torch.inference_mode(inference):
        offsets = gpu(torch.tensor([0, 3, 6], dtype=torch.int32))
        offsets.add_(0)  # a version other than a new tensor's
        _, saved = ec.mx_experts_forward(gpu(torch.zeros(6, 64)), gpu(torch.zeros(2, 32, 64)), offsets)
    return offsets, saved, gpu(torch.zeros(6, 32))


# The columns are laid out by the offsets of the forward pass: with others the gradients are wrong.
def test_offsets_written_to_after_the_forward_are_refused(stub):
    s = stub()
    offsets, saved, dy = experts_saved()
    ec.mx_experts_backward(dy, saved)
    assert s.calls[-1] == "ec_mx_product_tokens"
    for other in (copy.copy(saved), copy.deepcopy(saved), pickle.loads(pickle.dumps(saved))):
        ec.mx_experts_backward(dy, other)
    calls = len(s.calls)
    kept = copy.deepcopy(saved)
    offsets[1] = 2
    for call in (lambda: ec.mx_experts_backward(dy, saved), lambda: copy.deepcopy(saved)):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == ec.EC_ERR_INVALID
    assert len(s.calls) == calls
    ec.mx_experts_backward(dy, kept)  # a copy has offsets of its own
    # a new forward pass takes the offsets as they are now
    ec.mx_experts_backward(dy, ec.mx_experts_forward(gpu(torch.zeros(6, 64)), gpu(torch.zeros(2, 32, 64)), offsets)[1])


def test_offsets_that_torch_does_not_watch_are_copied(stub):
    stub()
    offsets, saved, dy = experts_saved(inference=True)
    with torch.inference_mode():
        offsets[1] = 2
    assert saved.offsets.tolist() == [0, 3, 6]
    ec.mx_experts_backward(dy, saved)


def test_offsets_of_a_captured_forward_may_change(stub, monkeypatch):
    # a graph reads them at each replay
    stub()
    monkeypatch.setattr(_binding, "capturing", lambda t: True, raising=False)
    offsets, saved, dy = experts_saved()
    offsets[1] = 2
    ec.mx_experts_backward(dy, saved)
    assert saved.offsets.data_ptr() == offsets.data_ptr()


# ---------------------------------------------------------------- streams


CALLS = [lambda s: ec.mx_quantize(gpu(torch.zeros(4, 64)), stream=s),
         lambda s: ec.mx_product(form(4, 64), form(5, 64), stream=s),
         lambda s: ec.expert_sort(gpu(torch.zeros(4, 2, dtype=torch.int32)), 4, stream=s)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [7, object(), "stream", torch.device("cpu"), gpu(torch.zeros(1))], ids=lambda v: type(v).__name__)
def test_what_is_no_stream_is_refused(call, stream):
    with pytest.raises(ec.ECError) as e:
        call(stream)
    assert e.value.status == ec.EC_ERR_INVALID


def test_calls_without_a_tensor_are_refused():
    for call in (ec.mx_quantize, ec.mx_quantize_both, ec.mx_dequantize):
        with pytest.raises(ec.ECError) as e:
            call(None, stream=object())
        assert e.value.status == ec.EC_ERR_INVALID


# A call that fails may have enqueued a part of its work, which reads its inputs.
@pytest.mark.parametrize("fails", [False, True])
def test_inputs_stay_for_another_stream_also_when_a_call_fails(monkeypatch, fails):
    import contextlib

    recorded = []

    class Input(OnGPU):
        def record_stream(self, stream):
            recorded.append(stream)

    class Stream:
        device, stream_id = torch.device("cpu"), 1

    def call(x):
        if fails:
            raise ec.ECError(ec.EC_ERR_DEVICE, "call")
        return x

    for name in ("device", "stream"):
        monkeypatch.setattr(torch.cuda, name, lambda *a: contextlib.nullcontext())
    s = Stream()
    x = torch.zeros(3).as_subclass(Input)
    with (pytest.raises(ec.ECError) if fails else contextlib.nullcontext()):
        _binding.on_stream(call, (x,), s)
    assert recorded == [s]


# ---------------------------------------------------------------- every call, on a stream of its own


def every_call():
    r = ec.expert_sort(gpu(torch.zeros(6, 2, dtype=torch.int32)), 4)
    offsets = gpu(torch.tensor([0, 3, 6], dtype=torch.int32))
    x, w, we = gpu(torch.zeros(6, 64)), gpu(torch.zeros(32, 64)), gpu(torch.zeros(2, 32, 64))
    rows, wt = gpu(torch.zeros(12, 64)), gpu(torch.zeros(6, 2))
    dy = gpu(torch.zeros(6, 32))
    linear, experts = ec.mx_linear_forward(x, w)[1], ec.mx_experts_forward(x, we, offsets)[1]
    return {
        "mx_quantize": (x,), "mx_quantize_both": (x,), "mx_dequantize": (form(6, 64), torch.float16),
        "mx_product": (form(6, 64), form(32, 64), torch.float16), "mx_linear": (x, form(32, 64)),
        "mx_experts_linear": (x, form(2, 32, 64), offsets),
        "mx_experts_product": (form(6, 64), form(2, 32, 64), offsets, torch.float16),
        "mx_linear_forward": (x, w), "mx_linear_backward": (dy, linear),
        "mx_experts_forward": (x, we, offsets), "mx_experts_backward": (dy, experts),
        "expert_sort": (gpu(torch.zeros(6, 2, dtype=torch.int32)), 4), "expert_dispatch": (x, r),
        "expert_dispatch_mx": (x, r), "expert_dispatch_backward": (rows, r), "expert_combine": (rows, r, wt),
        "expert_combine_backward": (x, rows, r, wt),
    }


# A call on a stream, and one on tensors of a GPU that is not the current one, go through the same
# function again under that stream and device: with the same arguments in the same places.
@pytest.mark.parametrize("elsewhere", [False, True])
def test_calls_elsewhere_make_the_same_library_calls(monkeypatch, stub, elsewhere):
    import contextlib

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
    public = {n for names in ec._OPERATORS.values() for n in names if n[0].islower()}
    calls = every_call()
    assert set(calls) == public
    inputs = lambda args: [v for v in args if isinstance(v, int) and 0 <= v < 1 << 32]  # noqa: E731 (no addresses)
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
