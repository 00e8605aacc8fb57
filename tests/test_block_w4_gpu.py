"""GPU tests of the 4-bit products where a weight of zero, an infinity or one very large activation
meets the rest of a row."""

import math

import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
DEV = "cuda"


@pytest.fixture(scope="module")
def block():
    from gemv_decode_projections_amd import block as b

    return b


def say(*a):
    print(*a, flush=True)


def weights(n, k, group, zeros, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    s = ((0.2 + torch.rand(n, k // group, generator=g)) * k ** -0.5).to(dtype)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    return q, s, z, g


def run(block, q, s, z, group, x):
    w = block.w4_prepare(q.to(DEV), s.to(DEV), None if z is None else z.to(DEV), group)
    out = torch.full((x.shape[0], q.shape[0]), math.nan, dtype=x.dtype, device=DEV)
    block.w4_run(w, x.to(DEV), out)
    torch.cuda.synchronize()
    return out


def direct(q, s, z, group, x):
    """out, and the bound of a kernel that multiplies the exact q - z: the products are exact (5 and 8 or
    11 bits), FP32 sums of k of them, each group's times its scale, err by (k + 2 k / group + 16) 2^-23
    of the magnitudes, the output is rounded once."""
    n, k = q.shape[0], 2 * q.shape[1]
    w = torch.empty(n, k, dtype=torch.float64)
    w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
    w -= torch.repeat_interleave(z.double(), group, 1) if z is not None else 8
    w *= torch.repeat_interleave(s.double(), group, 1)
    xd, u = x.double(), ref.U[x.dtype]
    out = xd @ w.t()
    return out, u * out.abs() + (1 + u) * (k + 2 * k // group + 16) * 2.0 ** -23 * (xd.abs() @ w.abs().t()) + ref.TINY[x.dtype]


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("m,n,k,group,zeros", [(1, 70, 512, 128, False), (3, 64, 4224, 64, True), (20, 33, 640, 32, True),
                                               (40, 8192, 256, 128, False)])
def test_an_infinite_activation_meets_its_weights_only(block, dtype, m, n, k, group, zeros):
    # Infinite times q - z: an infinity of its sign, NaN where q = z, as the formula has it. The other
    # tokens' rows do not notice.
    say("w4 inf", dtype, m, n, k, group, zeros)
    q, s, z, g = weights(n, k, group, zeros, dtype, 1)
    x = torch.randn(m, k, generator=g).to(dtype)
    x[0, 37] = math.inf
    if m > 2:
        x[2, k - 1] = -math.inf
    out = run(block, q, s, z, group, x)
    r, _ = direct(q, s, z, group, x)
    assert bool(torch.isinf(r[0]).any()) and bool(torch.isfinite(r[1:2]).all())
    rows = torch.isfinite(x).all(1)
    _, b = direct(q, s, z, group, torch.where(torch.isfinite(x), x, torch.zeros_like(x)))
    ref.assert_within("w4", out, r, torch.where(rows[:, None], b, torch.ones_like(b)))


@pytest.mark.parametrize("big", [2.0 ** 100, 3e38])
def test_a_very_large_activation_stays_finite(block, big):
    # 15 times the activation, times its scale, is finite; so are all sums.
    say("w4 large", big)
    q, s, _, g = weights(65, 256, 64, False, BF, 2)
    x = torch.randn(2, 256, generator=g).to(BF)
    s = (s.float() * 2.0 ** -8).to(BF)
    x[1, 100] = big
    q[:, 50] = q[:, 50] & 0xf0 | 9          # q - z = 1 there: the sum is the activation itself
    out = run(block, q, s, None, 64, x)
    r, b = direct(q, s, None, 64, x)
    assert bool(torch.isfinite(r).all())
    ref.assert_within("w4", out, r, b)


@pytest.mark.parametrize("dtype,big", [(BF, 2.0 ** 20), (FH, 32768.0)])
@pytest.mark.parametrize("m,zeros", [(1, False), (9, True), (33, True)])
def test_a_large_activation_on_zero_weights_leaves_no_trace(block, dtype, big, m, zeros):
    # Outlier channels that a row's weights leave out (q = z) contribute nothing, not even rounding.
    say("w4 outlier", dtype, m, zeros)
    n, k, group = 48, 1024, 64
    q, s, z, g = weights(n, k, group, zeros, dtype, 3)
    x = torch.randn(m, k, generator=g).to(dtype)
    for c in (200, 201, 700):
        x[:, c] = big
        zc = z[:, c // group] if z is not None else torch.full((n,), 8, dtype=torch.uint8)
        pair = q[:, c // 2]
        q[:, c // 2] = pair & 0x0f | zc << 4 if c % 2 else pair & 0xf0 | zc
    out = run(block, q, s, z, group, x)
    ref.assert_within("w4", out, *direct(q, s, z, group, x))


@pytest.mark.parametrize("m", [1, 5, 16, 17, 33, 64, 65, 100, 260])
@pytest.mark.parametrize("n,k", [(1000, 256), (4100, 64), (4112, 4096), (8200, 128), (5000, 4128), (12300, 96)])
def test_every_tile_that_the_rule_picks(block, m, n, k):
    # Row blocks on both sides of one, two and three rounds of workgroups, and token counts with and
    # without a part of a tile; the sum over a few rows is enough to see a block or tile misplaced.
    say("w4 plans", m, n, k)
    q, s, z, g = weights(n, k, 32, True, BF, 5)
    x = torch.randn(m, k, generator=g).to(BF)
    out = run(block, q, s, z, 32, x)
    rows = sorted({0, 1, 15, 16, 17, 33, 63, 64, n // 2, n - 17, n - 16, n - 15, n - 2, n - 1})
    r, b = direct(q[rows], s[rows], z[rows], 32, x)
    ref.assert_within("w4", out[:, rows], r, b)
    assert bool(torch.isfinite(out).all())
