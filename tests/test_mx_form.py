"""The 4-bit tensor as an object, on the CPU: what it hands to the library is always its own memory."""
import copy
import io
import pickle

import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from error_bounded_lossy_amd import mx  # noqa: E402


def given():
    """A form made of a caller's tensors: 6 rows of 200 elements."""
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (2, 3, 128), generator=g, dtype=torch.uint8)
    return ec.MXTensor(codes, torch.randint(1, 255, (2, 3, 8), generator=g, dtype=torch.uint8), 200)


def made():
    """A form as the library allocates it, codes and scales in one block."""
    q, like = mx._empty((2, 3), 200, torch.empty(0)), given()
    q.codes.copy_(like.codes)
    q.scales.copy_(like.scales)
    return q


def inside(address, tensor, size):
    start = tensor.untyped_storage().data_ptr()
    return start <= address and address + size <= start + tensor.untyped_storage().nbytes()


def same_and_apart(a, q):
    """a holds q's values in memory of its own, and that memory is what the library is given."""
    assert a.shape == q.shape and a.cols == q.cols and a.padded == q.padded and a.lead == q.lead
    assert torch.equal(a.codes, q.codes) and torch.equal(a.scales, q.scales)
    assert a.codes_ptr == a.codes.data_ptr() and a.scales_ptr == a.scales.data_ptr()
    for mine, other, size in ((a.codes_ptr, q.codes, 768), (a.scales_ptr, q.scales, 48)):
        assert not inside(mine, other, size)
    assert a.numel_bytes() == q.numel_bytes() == 768 + 48
    before = q.codes.clone()
    a.codes.add_(1)
    assert torch.equal(q.codes, before) and torch.equal(a.codes, before + 1)


@pytest.mark.parametrize("make", [given, made])
def test_deep_copies_have_their_own_memory(make):
    q = make()
    same_and_apart(copy.deepcopy(q), q)
    # inside of something larger, as a model is copied: an object held twice stays one
    layer = copy.deepcopy({"up": q, "again": q})
    assert layer["up"] is layer["again"]
    same_and_apart(layer["up"], q)


@pytest.mark.parametrize("make", [given, made])
def test_forms_that_were_saved(make):
    q = make()
    same_and_apart(pickle.loads(pickle.dumps(q)), q)
    f = io.BytesIO()
    torch.save({"w": q}, f)
    f.seek(0)
    same_and_apart(torch.load(f, weights_only=False)["w"], q)


@pytest.mark.parametrize("make", [given, made])
def test_a_shallow_copy_shares_its_memory(make):
    q = make()
    a = copy.copy(q)
    assert (a.codes_ptr, a.scales_ptr, a.shape) == (q.codes_ptr, q.scales_ptr, q.shape)


@pytest.mark.parametrize("make", [given, made])
def test_the_tensors_that_a_stream_has_to_keep(make):
    from error_bounded_lossy_amd import _binding
    q = make()
    for form in (q, copy.deepcopy(q)):
        held = {t.untyped_storage().data_ptr() for t in _binding._tensors(form)}
        assert held == {form.codes.untyped_storage().data_ptr(), form.scales.untyped_storage().data_ptr()}


def test_what_a_backward_needs_copies_with_it():
    saved = mx.MXLinearSaved(made(), given(), torch.tensor([0, 2, 6], dtype=torch.int32), 6, torch.bfloat16)
    for other in (copy.deepcopy(saved), pickle.loads(pickle.dumps(saved))):
        same_and_apart(other.x, saved.x)
        same_and_apart(other.w, saved.w)
        assert torch.equal(other.offsets, saved.offsets) and other.offsets.data_ptr() != saved.offsets.data_ptr()


def test_memory_that_the_caller_rebinds():
    q = given()
    codes, scales = q.codes, q.scales
    codes.data = torch.full_like(codes, 7)
    scales.data = torch.full_like(scales, 9)
    assert q.codes_ptr == q.codes.data_ptr() and bool((q.codes == 7).all())
    assert q.scales_ptr == q.scales.data_ptr() and bool((q.scales == 9).all())


@pytest.mark.parametrize("what", ["codes", "scales"])
@pytest.mark.parametrize("to", [lambda t: t[:1].clone(), lambda t: t[..., ::2].contiguous()[..., ::2],
                                lambda t: t.float(), lambda t: t.transpose(0, 1)])
def test_memory_rebound_to_another_shape_is_refused(what, to):
    # the library would read past the end of it
    q = given()
    t = getattr(q, what)
    t.data = to(t)
    with pytest.raises((ec.ECError, RuntimeError)):
        getattr(q, f"{what}_ptr")


@pytest.mark.parametrize("make", [given, made])
def test_bad_saved_state_is_refused(make):
    call, args = make().__reduce__()
    for wrong in ((args[0][..., :1], *args[1:]), (args[0].int(), *args[1:])):
        with pytest.raises(ec.ECError) as e:
            call(*wrong)
        assert e.value.status == ec.EC_ERR_INVALID


class OnGPU(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    is_cuda = True


def test_forms_of_groups_are_not_read_as_rows(monkeypatch):
    # rows of 300 elements in 3 groups are padded to 512 or more, plain ones to 384: a product would
    # read the one with the other's pitch, past its end
    from error_bounded_lossy_amd import _binding

    monkeypatch.setattr(_binding, "current_stream", lambda t: 0)
    monkeypatch.setattr(_binding, "elsewhere", lambda t: False)
    like = torch.empty(0).as_subclass(OnGPU)
    grouped = mx._empty((40,), 300, like, ec.lib().ec_mx_padded_groups(300, 3))
    plain, experts = mx._empty((40,), 300, like), mx._empty((2, 40), 300, like)
    assert grouped.padded > plain.padded and grouped.cols == plain.cols
    monkeypatch.setattr(_binding, "lib", lambda: pytest.fail("the library was reached"))
    offsets = torch.zeros(3, dtype=torch.int32).as_subclass(OnGPU)
    x = torch.zeros(5, 300).as_subclass(OnGPU)
    for call in (lambda: ec.mx_product(grouped, plain), lambda: ec.mx_product(plain, grouped),
                 lambda: ec.mx_dequantize(grouped), lambda: ec.mx_linear(x, grouped),
                 lambda: ec.mx_experts_product(grouped, experts, offsets)):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == ec.EC_ERR_INVALID


# ---------------------------------------------------------------- routings


def routing(**other):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    parts = {"order": i32(12), "place": i32(6, 2), "offsets": i32(5), "tokens": 6, "choices": 2, "experts": 4}
    return ec.Routing(**{**parts, **other})


# Its arrays go to the device as they are: with another type or size the exchange would read past them.
@pytest.mark.parametrize("wrong", [
    {"place": torch.zeros(6, 2, dtype=torch.int64)}, {"place": torch.zeros(5, 2, dtype=torch.int32)},
    {"place": torch.zeros(12, dtype=torch.int32)}, {"place": torch.zeros(2, 6, dtype=torch.int32).t()},
    {"offsets": torch.zeros(4, dtype=torch.int32)}, {"offsets": torch.zeros(5)},
    {"offsets": torch.zeros(10, dtype=torch.int32)[::2]}, {"offsets": torch.zeros(5, dtype=torch.int32, device="meta")},
    {"order": torch.zeros(11, dtype=torch.int32)}, {"order": torch.zeros(12, dtype=torch.int64)},
    {"tokens": 7}, {"choices": 3}, {"choices": 0}, {"experts": 5}, {"experts": 0}, {"place": None}],
    ids=lambda w: "-".join(f"{k}" for k in w))
def test_routings_of_other_arrays_are_refused(wrong):
    routing()
    with pytest.raises(ec.ECError) as e:
        routing(**wrong)
    assert e.value.status == ec.EC_ERR_INVALID


def test_routings_copy_with_their_arrays():
    r = routing()
    for other in (copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert other.place.data_ptr() != r.place.data_ptr() and other.experts == 4
