"""Scaling against 64-bit products: one rounding to fp32 and one to the
output's type, as the header says."""
import pytest
import torch

from tests.test_grad_norm_gpu import DEV, pq  # noqa: F401 (pq is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("coef", [1 / 3, 0.9999999, 1.25e-3])
def test_scaling_is_two_roundings(pq, dtype, coef):  # noqa: F811
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    t = bits.view(dtype) if dtype != torch.float32 else torch.randn(1 << 16, generator=torch.Generator().manual_seed(1))
    t = t[torch.isfinite(t)]
    c = torch.tensor([coef], device=DEV)
    got = t.to(DEV)
    pq.pq_grad_scale(pq.tensor_array([got]), c)
    exact = t.double() * c.cpu().double()
    assert torch.equal(got.cpu(), exact.float().to(dtype))
    # half a step of the type, and the fp32 product's rounding; below the
    # type's normal numbers the steps are those of the smallest
    info = torch.finfo(dtype)
    tol = exact.abs() * (info.eps / 2 + 2.0 ** -24) * (1 + info.eps) + info.tiny * info.eps / 2 + 2.0 ** -150
    assert ((got.cpu().double() - exact).abs() <= tol).all()
