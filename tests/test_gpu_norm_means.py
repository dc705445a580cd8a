"""LayerNorm of rows whose mean is far larger than their spread, down to rows
of equal elements, against the formulas in float64.

Tolerances: u = 2^-24, a row's sums have no chain longer than D/32 + 16
additions. The first sweep's mean m0 is off by e0 = (D/32 + 18) u mean|s|. What
the second sweep sums is d = s - m0 (rounded: u |d|), no larger than the true
difference and e0, so c = mean(d) brings the mean to e = (D/32 + 18) u mean|d|;
the variance mean(d^2) - c^2 is off by (D/32 + 20) u mean(d^2) + 2 e |c| + e^2
and what d's rounding adds. Rows whose mean is at most 16 spreads (sqrt of the
variance and eps) stay at m0: there e = e0, at most 17 (D/32 + 18) u of the
spread, and the variance is larger by c^2 <= e^2, as mean(d) is 0 about the true
mean. An output is rounded by finfo(t).eps / 2 besides.
"""
import pytest
import torch

from tests.test_gpu_norm import forward, generator

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTHS = [7, 77, 200, 500, 700, 1000, 1023, 1024, 1500, 2000, 2500, 4099, 5000, 8192, 12_000, 16_384]


def check(x, res, gamma, beta, eps, y, mean, rstd):
    t, D = x.dtype, x.shape[1]
    s = x.double() if res is None else (x.float() + res.float()).to(t).double()
    mu = s.mean(1)
    d = s - mu[:, None]
    var = d.square().mean(1)
    inv = (var + eps).rsqrt()
    chain = (D / 32 + 18) * U
    e0 = chain * s.abs().mean(1)
    dk = d.abs() + e0[:, None]                                    # the kernel's |s - m0| at most
    e = torch.where(mu.square() <= 1.02 * 256 * (var + eps), e0, chain * dk.mean(1))   # 1.02: the kernel's own variance
    e_var = (chain + 2 * U) * dk.square().mean(1) + 2 * e * (e0 + e) + e.square()
    rel = 0.5 * e_var / (var + eps) + 4 * U
    rel = rel / (1 - 2 * rel).clamp_min(0.25)
    assert ((mean.double() - mu).abs() <= e + U * mu.abs() * 1.01).all()
    off = (rstd.double() - inv).abs() / (rel * inv)
    assert (off <= 1).all(), float(off.max())
    z, g, b = d * inv[:, None], gamma.double(), beta.double()
    want = z * g + b
    e_z = (2 * U * dk + e[:, None] + U * e0[:, None]) * inv[:, None] + z.abs() * (rel[:, None] + 3 * U)
    tol = 1.01 * g.abs() * e_z + 2 * U * (b.abs() + want.abs())
    tol = tol + torch.finfo(t).eps / 2 * (want.abs() + tol)
    off = (y.double() - want).abs() / tol
    assert (off <= 1).all(), (float(off.max()), off.argmax().item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("rows", [5, 2000])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_far_from_zero(dtype, D, rows, residual):
    """In turn: equal elements, a spread of a hundredth, a spread of one, a
    single element that differs."""
    t, gen = TYPES[dtype], generator(D + rows)
    kind = torch.arange(rows, device="cuda")[:, None] % 4
    noise = torch.randn(rows, D, device="cuda", generator=gen)
    x = 1000.1 + torch.where(kind == 1, 0.01 * noise, torch.where(kind == 2, noise, 0.0))
    x[3::4, D // 2] = 1001
    x = x.to(t)
    res = (torch.full_like(x, -333.3) + (kind == 2) * noise).to(t) if residual else None
    gamma = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen)).to(t)
    beta = (0.1 * torch.randn(D, device="cuda", generator=gen)).to(t)
    y, mean, rstd = forward(x, res, gamma, beta, 1e-5)
    check(x, res, gamma, beta, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("D", [1000, 1023, 4096, 9000])
def test_rows_of_equal_elements_of_any_size(D):
    """y = beta and rstd = 1 / sqrt(eps), whatever the elements are; NaN and infinities stay."""
    v = torch.tensor([0.0, 0.1, -3.3, 77.7, -5e3, 1.2345e5, -7.7e6, 1.1e9, float("nan"), float("inf")], device="cuda")
    x = v[:, None].repeat(1, D)
    x[8, 1:], x[9, 1:] = 1.0, 1.0                                 # one element of the row is not finite
    gamma, beta = torch.ones(D, device="cuda"), torch.full((D,), 0.25, device="cuda")
    y, mean, rstd = forward(x, None, gamma, beta, 1e-3)
    assert not torch.isfinite(y[8:]).any() and not torch.isfinite(mean[8:]).any()
    check(x[:8], None, gamma, beta, 1e-3, y[:8], mean[:8], rstd[:8])
