"""How near the biased linears' sums are to float64, measured against float32 arithmetic: one product after the other
added to a float32 number that rounds to nearest.

A product of two bf16 numbers is a float32 number exactly, so that arithmetic has one rounding per term and no other.  An
output that many elements share its error with is compared as a whole: the count of bf16 results that are not the exact one's
rounding, or the norm of the difference.  A count of c has a standard deviation of sqrt(c); with the counts here (200 and
more on the float32 side) a factor of 1.25 is two deviations of their ratio and more.
"""
import pytest
import torch

from backward_split_linear_gb300 import binding as zb

pytestmark = pytest.mark.gpu

ROOM = 1.25


def draw(seed, t, k, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return normal(t, k).to(torch.bfloat16), (normal(n, k) * k ** -0.5).to(torch.bfloat16)


def float32_sums(x, w):
    """x w^T, term by term."""
    a, b = x.float().t().contiguous(), w.float().t().contiguous()
    out = torch.zeros(x.shape[0], w.shape[0], device="cuda")
    for k in range(x.shape[1]):
        out.addcmul_(a[k][:, None], b[k][None, :])
    return out


def misrounded(got, exact):
    return int((got != exact.to(torch.bfloat16)).sum())


@pytest.mark.parametrize("t,k,n", [(520, 2112, 2560), (1000, 640, 4096), (520, 4096, 2560), (185, 11520, 1088)])
def test_forward_with_codes(cuda_device, t, k, n):
    x, w = draw(k, t, k, n)
    exact = x.double() @ w.double().t()
    y, z = torch.empty(t, n, dtype=torch.bfloat16, device="cuda"), torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    y8 = (torch.empty(t, n, dtype=torch.uint8, device="cuda"), torch.empty(t, n // 32, dtype=torch.uint8, device="cuda"))
    zb.zb_op_linear_activation_forward(x, w, None, None, y, t, k, n, "none", z=z, y_packed=y8)
    plain = misrounded(float32_sums(x, w).to(torch.bfloat16), exact)
    got = misrounded(z, exact)
    assert got <= ROOM * plain, (got, plain)
    assert torch.equal(y, z)


@pytest.mark.parametrize("t,k,n", [(520, 14336, 2560), (1000, 4096, 4096)])
def test_forward_in_bf16(cuda_device, t, k, n):
    """Sums of 1024 terms at a time: about twice as far off as float32 arithmetic at K = 4096, nearer behind that."""
    x, w = draw(k, t, k, n)
    exact = x.double() @ w.double().t()
    y = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    zb.zb_op_linear_activation_forward(x, w, None, None, y, t, k, n, "none")
    plain = misrounded(float32_sums(x, w).to(torch.bfloat16), exact)
    got = misrounded(y, exact)
    assert got <= 2 * ROOM * plain, (got, plain)


@pytest.mark.parametrize("t,k,n", [(1, 1024, 8192), (1, 640, 16384), (1, 1984, 16384), (1, 11520, 1088)])
def test_bias_gradient(cuda_device, t, k, n):
    """One row: the bias gradient is the product itself, in float32."""
    dy, w = draw(k, t, k, n)
    exact = dy.double() @ w.double().t()
    dz = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    dbias = torch.zeros(n, device="cuda")
    scratch = torch.empty(zb.zb_op_backward_input_activation_scratch_bytes(t, n), dtype=torch.uint8, device="cuda")
    zb.zb_op_backward_input_activation(dy, w.t().contiguous(), None, dz, t, n, k, "none", dbias=dbias, scratch=scratch)
    plain = (float32_sums(dy, w).double() - exact).norm()
    got = (dbias.double() - exact[0]).norm()
    assert float(got) <= ROOM * float(plain), (float(got), float(plain))
