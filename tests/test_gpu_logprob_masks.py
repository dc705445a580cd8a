"""Token log probabilities of rows whose logits, or whose masks, lie far from
zero: finite masks of every size, whole rows beyond 2^24, and rows whose
running maximum crosses 2^24 on its way, on every path of the kernel.

Tolerances: u = 2^-24. What is checked depends on the logits' differences
alone, so they are measured against sums relative to the maximum in float64.
A term 2^y, y = (x - m) log2(e), is off by 2^-21 + 4u |x - m| of its value (the
function's 2 ulp, the roundings of the difference, of the constant and of the
product), and a sum of V of them by another (V/32 + 64) u: rows of up to 1024
run in 16 chains or more (V/16 <= V/32 + 32), longer ones in 32 or more. Below
2^24 the sums are relative to a rounded m log2(e), at most 1 away: log2 of the
sum and T / S carry it, and lose it again in their difference.
"""
import pytest
import torch

from tests.test_gpu_logprob import backward, check_backward, forward, generator

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# 8, 16 and 32 lanes; blocks of 64, 128, 256 and 512 threads; clusters of 8, 4 and 2 (the numbers of alternatives and the
# type choose among the lanes)
SHAPES = [(4, 40), (9, 1000), (1300, 2000), (1300, 8001), (612, 20_011), (8, 12_001), (320, 40_000), (100, 65_536),
          (8, 70_001), (30, 100_003), (60, 100_003)]


def check(x, tokens, K, o):
    """Rows with a finite maximum and no NaN: logp, top_logp and entropy by the differences, lse to its own places."""
    V, x64 = x.shape[1], x.double()
    m = x64.amax(1, keepdim=True)
    d = x64 - m
    e = torch.exp(d)
    S = e.sum(1)
    d0 = torch.where(e > 0, d, 0.0)
    ed = e * d0
    T = ed.sum(1)
    chain = (V / 32 + 64) * U
    term = 2.0 ** -21 + 4 * U * d0.abs()
    rel = (e * term).sum(1) / S + chain
    err_t = (ed.abs() * (term + 2 * U)).sum(1) + chain * ed.abs().sum(1)
    log_s, mean_d = S.log(), (T / S).abs()
    H = log_s - T / S
    tol = 1.05 * rel + 4 * U * (log_s + 1)
    lse = m[:, 0] + log_s
    assert ((o["lse"].double() - lse).abs() <= tol + 2 * U * lse.abs()).all()
    tol_h = 1.05 * (rel * (2 + mean_d) + err_t / S) + 4 * U * (H + log_s + mean_d + 2)
    off = (o["entropy"].double() - H).abs() / tol_h
    assert (off <= 1).all(), (float(off.max()), int(off.argmax()))

    def close(got, at):
        want = at - m - log_s[:, None]
        off = (got.double() - want).abs() / (tol[:, None] + 4 * U * (want.abs() + (at - m).abs()))
        assert (off <= 1).all(), (off.max(), got[~(off <= 1)][:4], want[~(off <= 1)][:4])

    close(o["logp"][:, None], x64.gather(1, tokens.long()[:, None]))
    if K:
        ids = (-x64).sort(dim=1, stable=True).indices[:, :K]
        assert torch.equal(o["ids"].long(), ids)
        close(o["top"], x64.gather(1, ids))


def check_all(x, gen):
    rows, V = x.shape
    tokens = torch.randint(V, (rows,), device="cuda", generator=gen, dtype=torch.int32)
    tokens[::2] = x[::2].float().argmax(1).int()
    for K in (0, 3, 20, 32) if rows * V < 2_000_000 else (0, 20):
        o = forward(x, tokens, min(K, V))
        check(x, tokens, min(K, V), o)
    return tokens, o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("mask", [-1e9, -2.0 ** 30, -1e10, -3e10, -1e12, -1e13, -1e16, -1e20, -1e29, -6e29, -1e30])
def test_finite_masks(dtype, rows, V, mask):
    """A mask is 'any value far below the others': p is 0 wherever it stands.
    In turn: rows of nothing else, a few logits allowed, a masked first half, a
    masked second half."""
    t, gen = TYPES[dtype], generator(rows + V)
    x = (2.5 * torch.randn(rows, V, device="cuda", generator=gen)).to(t)
    j, kind = torch.arange(V, device="cuda"), torch.arange(rows, device="cuda")[:, None] % 4
    some = torch.rand(rows, V, device="cuda", generator=gen) < 1 / 160
    some[:, [V // 3, V - 1]] = True
    masked = (kind == 0) | ((kind == 1) & ~some) | ((kind == 2) & (j < V // 2)) | ((kind == 3) & (j >= V // 2))
    x[masked] = torch.tensor(mask, device="cuda").to(t)
    tokens, o = check_all(x, gen)
    one = torch.ones(rows, device="cuda")
    dx = backward(x, tokens, o["lse"], o["entropy"], one, one)
    assert (dx[::4] == 0).all()                                   # nothing but a mask passes no gradient
    rest = kind[:, 0] != 0
    check_backward(x[rest], tokens[rest], o["lse"][rest], o["entropy"][rest], one[rest], one[rest], dx[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("offset", [3e6, 2.0 ** 24, 1e8, 1e9, 2.0 ** 30, 1e10, 1e20, 6e29])
def test_rows_far_from_zero(dtype, rows, V, offset):
    """Values a few steps of the type apart, on either side of zero: the
    entropy and the log probabilities are those of the differences."""
    t, gen = TYPES[dtype], generator(rows + V + 1)
    base = torch.tensor(offset, device="cuda").to(t).float()
    size = base * torch.finfo(t).eps                               # a step at the offset, or two
    steps = torch.randint(0, 3, (rows, V), device="cuda", generator=gen).float()
    steps[::3] = 0                                                 # rows of equal values
    x = (base + steps * size) * (1 - 2 * (torch.arange(rows, device="cuda")[:, None] % 2))
    check_all(x.to(t), gen)


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("order", ["any", "rising", "falling"])
@pytest.mark.parametrize("values", [(2.0 ** 24 - 2, 2.0 ** 24 - 1, 2.0 ** 24, 2.0 ** 24 + 2),
                                    (-2.0 ** 24 - 4, -2.0 ** 24 - 2, -2.0 ** 24, -2.0 ** 24 + 1),
                                    (-1e35, -1e20, -1e10, -2.0 ** 25, -1e6, -3.0, 2.0, 2.5),
                                    (-3.4e38, -1e9, 7.0, 1e5, 2.0 ** 24, 2.0 ** 24 + 2, 2.0 ** 24 + 4)])
def test_maxima_that_cross_from_near_to_far(rows, V, order, values):
    """Partial sums whose maxima lie on different sides of 2^24, joined in
    every order: all of them count."""
    gen = generator(rows + V + 2)
    at = torch.randint(0, len(values), (rows, V), device="cuda", generator=gen)
    if order != "any":
        at = at.sort(dim=1, descending=order == "falling").values
    check_all(torch.tensor(values, device="cuda")[at], gen)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 1000, 9001, 70_001])
def test_what_is_not_finite_stays_so_behind_a_mask(dtype, V):
    """NaN and +inf beside a finite mask and beside none, before and after the allowed logits."""
    t, bad = TYPES[dtype], torch.tensor([float("nan"), float("inf")], device="cuda")
    x = torch.full((8, V), -1e12, device="cuda", dtype=t)
    x[4:, V // 2] = 1.0
    x[::4, 0], x[1::4, V - 1], x[2::4, 0], x[3::4, V - 1] = bad[0], bad[0], bad[1], bad[1]
    tokens = torch.full((8,), V // 2, device="cuda", dtype=torch.int32)
    o = forward(x, tokens, 4)
    for k in ("logp", "entropy", "top"):
        assert torch.isnan(o[k]).all(), k
    assert torch.isnan(o["lse"][[0, 1, 4, 5]]).all() and not torch.isfinite(o["lse"]).any()
    assert ((o["ids"] >= 0) & (o["ids"] < V)).all()
