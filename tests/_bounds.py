"""Error bounds of the operators' tests: first-order forward error analysis in 64 bits, element by element.

``U`` is half a unit in the last place of fp32, relative; ``half(dtype)`` that of the output type.
"""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(bound, ref, dtype):
    """Bound of a value known to `bound` around `ref` once it is rounded to `dtype` (fp32 values: already rounded)."""
    extra = half(dtype) if dtype != torch.float32 else 0.0
    return bound * (1 + extra) + ref.abs() * extra + torch.finfo(torch.float32).tiny


def assert_within(got, ref, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    worst = over.argmax()
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} outside the bound; worst: got "
                               f"{got.reshape(-1)[worst]:.9g} want {ref.reshape(-1)[worst]:.9g} "
                               f"bound {bound.reshape(-1)[worst]:.3g}")
