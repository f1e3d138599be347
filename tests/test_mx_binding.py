"""What the binding of the 4-bit and exchange operators does around a library call, on the CPU:
the library is a stub that looks at its arguments, and tensors pass for tensors on a GPU."""
import gc

import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from error_bounded_lossy_amd import _binding  # noqa: E402


class OnGPU(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    is_cuda = True


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
