"""The 4-bit format, its products and the token exchange from their definitions, in 64 bits (torch,
any device), written apart from the library."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def two_to(e):
    """2^e in float64, by its bits: a library's power need not be exact on every device, and the
    rounding of middle values needs it to be."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pad(n, to=128):
    return -(-n // to) * to


def quantize(x):
    """(code [.., padded], scale byte [.., padded / 32]) of x along its last dimension."""
    x = x.double()
    x = torch.nn.functional.pad(x, (0, pad(x.shape[-1]) - x.shape[-1])).unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    _, e = torch.frexp(torch.where(torch.isfinite(top), top, torch.ones_like(top)))  # top = f 2^e
    s = torch.where(top > 0, (e - 1 + 125).clamp(min=0), torch.zeros_like(e))
    s = torch.where(torch.isfinite(top), s, torch.full_like(s, 255))
    v = (x * two_to(127 - s.clamp(max=253))[..., None]).abs()
    grid = GRID.to(x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    # a middle value goes to the even code: up from odd codes, down from even ones
    up = torch.arange(7, device=x.device) % 2 == 1
    code = ((v[..., None] > middle) | ((v[..., None] == middle) & up)).sum(-1)
    code = code + 8 * torch.signbit(x)
    return code.flatten(-2), s


def values(code, s):
    """What codes and scale bytes stand for, in float64 (NaN where the byte is 255)."""
    v = GRID.to(code.device)[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0).to(torch.float64)
    v = v.unflatten(-1, (-1, 32)) * two_to(s.int() - 127)[..., None]
    return torch.where((s == 255)[..., None], torch.full_like(v, float("nan")), v).flatten(-2)


def near(x):
    code, s = quantize(x)
    return values(code, s)[..., : x.shape[-1]]


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()


def mm_bound(a, b, dtype):
    """a b^T and how far a sum of its products in fp32, rounded once to dtype, may be off: every
    addition loses at most half a step of a partial sum, which is at most the sum of magnitudes."""
    y = a @ b.t()
    size = a.abs() @ b.abs().t()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    off = (a.shape[1] + 1) * 2.0 ** -24 * size * 1.01
    return y, off + torch.finfo(dtype).eps / 2 * (y.abs() + off) + tiny


def check(got, want, bound, what=""):
    # beyond the type's largest value, and nowhere else, an infinity is the rounding
    largest = torch.finfo(got.dtype).max
    got = got.double()
    over = torch.isinf(got) & (got * want > 0) & (want.abs() + bound >= largest)
    bad = ~(((got - want).abs() <= bound) | over)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                           f"{((got - want).abs() / bound).nan_to_num(9e9).max().item():.3g} of the bound")


def sort(ids, experts):
    flat = ids.reshape(-1).tolist()
    kept = sorted((i for i, e in enumerate(flat) if 0 <= e < experts), key=lambda i: flat[i])
    order = torch.full((len(flat),), -1, dtype=torch.int32)
    place = torch.full((len(flat),), -1, dtype=torch.int32)
    order[: len(kept)] = torch.tensor(kept, dtype=torch.int32)
    for row, i in enumerate(kept):
        place[i] = row
    counts = [0] * experts
    for i in kept:
        counts[flat[i]] += 1
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    return order, place.reshape(ids.shape), offsets
