"""The routing's gradient takes ids and gradients of any strides, as its documentation says (on the CPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from test_mx_binding import gpu, stub  # noqa: E402, F401


def ints(address, n):
    return list((ctypes.c_int32 * n).from_address(address))


@pytest.mark.parametrize("take", [lambda t: t[:, :2], lambda t: t[:, 1:3], lambda t: t[:, ::2], lambda t: t.t()[:2, :4].t()], ids=range(4))
def test_ids_and_gradients_of_any_strides(stub, take):  # noqa: F811
    seen = []

    def look(dweights, logits, kind, tokens, stride, experts, ids, choices, *rest):
        seen.append((ints(ids, tokens * choices), ints(dweights, tokens * choices)))
        return ec.EC_OK

    stub(ec_expert_route_backward=look)
    ids = gpu(torch.arange(16, dtype=torch.int32).reshape(4, 4))
    dw = gpu(torch.arange(16.0).reshape(4, 4))
    i, d = take(ids), take(dw)
    assert not i.is_contiguous()
    ec.expert_route_backward(d, gpu(torch.zeros(4, 64)), i)
    assert seen == [(i.flatten().tolist(), d.contiguous().view(torch.int32).flatten().tolist())]
