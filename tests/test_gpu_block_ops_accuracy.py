"""Accuracy of the layer-norm and linear kernels where a plain tolerance would
hide a loss: rows whose mean is far larger than their spread, the lower tails
of the activations, and deep products. References are fp64, written so that they
keep their own digits there."""
import math

import numpy as np
import pytest
import torch

from oracle import block
from test_gpu_block_ops import CHAIN, DEV, HALF, OFFSET, SEED, Mat, _mt, np64, scratch, stream, vec, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# ---------------------------------------------------------------------------
# Layer norm of rows with a large mean
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,d", [(4, 3), (9, 257), (6, 1000), (37, 2048), (11, 2049), (5, 5120), (3, 8192)])
@pytest.mark.parametrize("times,xt", [(1e3, F32), (-1e4, F32), (1e5, F32), (100.0, BF16)])
@pytest.mark.parametrize("yt", [F32, BF16])
def test_layernorm_fwd_of_rows_with_a_large_mean(T, d, times, xt, yt):
    """A mean of `times` the spread. A first mean m, off by e <= CHAIN |mean|,
    shifts t = x - m, which is exact or off by 2^-24 of itself; the mean of t
    then takes the shift out, off by CHAIN mean |t| <= CHAIN (a + e) with a the
    mean of |x - mean|. So the bound on y grows with e^2 at most, not with the
    mean. The variance mean t^2 - shift^2 is off by CHAIN (var + e^2)."""
    mt = _mt()
    rng = np.random.default_rng(T + d)
    x = Mat(T, d, xt, 1.5 * rng.normal(size=(T, d)) + 1.5 * times * (1 + 0.1 * rng.normal(size=(T, 1))))
    g, b = vec(1 + 0.1 * rng.normal(size=d), BF16), vec(0.3 * rng.normal(size=d), BF16)
    y, m, r = Mat(T, d, yt), scratch(T), scratch(T)
    mt.mt_k_layernorm_fwd(x.ptr, x.kind, x.ld, g.data_ptr(), b.data_ptr(), y.ptr, y.kind, y.ld, m.data_ptr(), r.data_ptr(), T, d,
                          1e-5, stream())
    X, G, B = x.np(), np64(g), np64(b)
    want, wm, wr = block.layernorm_fwd(X, G, B, 1e-5)
    a, e = np.abs(X - wm[:, None]).mean(axis=1), CHAIN * np.abs(wm)
    shift = CHAIN * (a + e)
    spread = CHAIN * (1 + (e * wr) ** 2) + 2.0 ** -21  # of r, relative: half the variance's, and rsqrt's
    within(np64(m)[:T], wm, 2.0 ** -24 * np.abs(wm) * 1.001 + shift)
    within(np64(r)[:T], wr, spread * wr)
    xh = np.abs(X - wm[:, None]) * wr[:, None]
    tol = HALF[yt] * np.abs(want) + np.abs(G) * ((shift * wr)[:, None] + xh * spread[:, None]) + \
        4 * 2.0 ** -24 * (xh * np.abs(G) + np.abs(B))
    within(y.np(), want, tol)


@pytest.mark.parametrize("value", [0.1, -1234.567, 3.3e7])
@pytest.mark.parametrize("d", [3, 515, 2048, 5120])
def test_layernorm_fwd_of_a_constant_row(value, d):
    """x - mean is 0 whatever the value's digits: y is b up to the shift's own
    rounding (at most CHAIN of a shift of CHAIN |value|, times r = eps^-1/2)."""
    mt = _mt()
    x, y = Mat(2, d, F32, np.full((2, d), value)), Mat(2, d, F32)
    rng = np.random.default_rng(d)
    g, b = vec(1 + 0.1 * rng.normal(size=d), BF16), vec(0.3 * rng.normal(size=d), BF16)
    mt.mt_k_layernorm_fwd(x.ptr, 0, x.ld, g.data_ptr(), b.data_ptr(), y.ptr, 0, y.ld, 0, 0, 2, d, 1e-5, stream())
    want = np.broadcast_to(np64(b), (2, d))
    within(y.np(), want, np.abs(np64(g)) * CHAIN ** 2 * abs(value) * 1e-5 ** -0.5 + 2.0 ** -22 * np.abs(want))


def test_layernorm_fwd_statistics_of_rows_that_are_not_finite():
    """The mean of a row with infinities of one sign is that infinity, of one with
    a NaN NaN; a row whose digits' squares are beyond fp32 stays finite."""
    mt = _mt()
    T, d = 6, 300
    x = np.ones((T, d))
    x[0, 7], x[1, 0], x[2, 299], x[3, :] = np.inf, -np.inf, np.nan, 1e27
    X, y = Mat(T, d, F32, x), Mat(T, d, F32)
    g, b = vec(np.ones(d), BF16), vec(np.full(d, 0.5), BF16)
    m, r = scratch(T), scratch(T)
    mt.mt_k_layernorm_fwd(X.ptr, 0, X.ld, g.data_ptr(), b.data_ptr(), y.ptr, 0, y.ld, m.data_ptr(), r.data_ptr(), T, d, 1e-5,
                          stream())
    got, mean = y.np(), np64(m)
    assert mean[0] == np.inf and mean[1] == -np.inf and np.isnan(mean[2]) and np.isnan(mean[T])
    assert np.isnan(got[:3]).all() and (got[4:] == 0.5).all()
    assert np.isfinite(got[3]).all()


# ---------------------------------------------------------------------------
# The activations' lower tails
# ---------------------------------------------------------------------------
def gelu_parts(z):
    cdf = np.array([0.5 * math.erfc(-v / math.sqrt(2)) for v in z])
    return cdf, np.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def value_slope(z, act):
    """Value, slope, the size of the slope's terms, and the relative error that a
    term may have, in units of 2^-24. A hardware reciprocal or power of two is
    off by 4 units, a polynomial of a few terms by 8; a power's argument is off
    by a rounding or two of itself, which counts as many units as it is large:
    1.1 z^2 for exp(-z^2 / 2), |z| and 4 |u| (u itself takes three roundings) for the
    two logistic forms."""
    if act == "gelu":
        cdf, pdf = gelu_parts(z)
        return z * cdf, cdf + z * pdf, cdf + np.abs(z) * pdf, 16 + 1.1 * z * z
    if act == "silu":
        s, w = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
        return z * s, s * (1 + z * w), s * (1 + np.abs(z) * w), 16 + 1.5 * np.abs(z)
    k = math.sqrt(8 / math.pi)
    u = k * (z + 0.044715 * z ** 3)
    s, w = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u))
    du = k * (1 + 3 * 0.044715 * z * z)
    return z * s, s * (1 + z * w * du), s * (1 + np.abs(z) * w * du), 16 + 4 * np.abs(u)


@pytest.mark.parametrize("act,low", [("gelu", -12.5), ("gelu_tanh", -9.0), ("silu", -80.0)])
def test_activation_tails_keep_their_digits(act, low):
    """Value (fp32 output of a product by the identity) and slope (the bias
    gradient of one row, which is not rounded) on every bf16 number of the lower
    tail down to where the power of two leaves the normal numbers, relative to
    the value itself; and the value on the upper side."""
    mt = _mt()
    z = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(BF16).double().numpy()
    z = z[(z >= 2.0 ** -10) & (z <= -low)]
    neg, both = -z, np.concatenate([-z, z])
    kind = block.ACTS.index(act)
    n = len(both)
    A, W = Mat(1, 8, BF16, np.eye(1, 8)), Mat(n, 8, BF16, both[:, None] * np.eye(1, 8))
    C = Mat(1, n, F32)
    mt.mt_k_linear_fwd(A.ptr, A.ld, W.ptr, W.ld, 0, kind, None, 0, 0, 0, 0, C.ptr, 0, C.ld, 1, n, 8, stream())
    value, _, _, units = value_slope(both, act)
    within(C.np()[0], value, units * 2.0 ** -24 * np.abs(value))
    n = len(neg)
    _, slope, terms, units = value_slope(neg, act)
    dC, Z, dZ, db = Mat(1, n, F32, np.ones((1, n))), Mat(1, n, BF16, neg[None]), Mat(1, n, BF16), scratch(n)
    part = scratch(mt.mt_k_act_bwd_partial_floats(1, n))
    mt.mt_k_act_bwd(dC.ptr, 0, dC.ld, Z.ptr, Z.ld, kind, None, dZ.ptr, dZ.ld, part.data_ptr(), db.data_ptr(), 1, n, stream())
    within(np64(db)[:n], slope, (units + 4) * 2.0 ** -24 * terms)
    within(dZ.np()[0], slope, 2.0 ** -8 * np.abs(slope) + (units + 4) * 2.0 ** -24 * terms)


# ---------------------------------------------------------------------------
# Deep products
# ---------------------------------------------------------------------------
def far(got, want):
    return float((got.double() - want).norm())


@pytest.mark.parametrize("M,N,K", [(2309, 1948, 5504), (4000, 1300, 5000), (70, 1300, 5504)])
@pytest.mark.parametrize("fam", [0, 1, 2])
def test_fp32_outputs_of_deep_products_with_everything_in_the_epilogue(M, N, K, fam):
    """Bias, ReLU, dropout, fp32 residual and Z forward; slope, dropout and bias
    gradient back; at depths whose accumulator is added up in parts, on more
    full-width pair tiles than there are pairs (the rest cut) and on few rows.

    A part of at most 15 k-blocks on average takes 60 steps that each truncate
    half a unit, 2^-24, on average: 60 x 2^-24 of the product (relative L2). All
    344 steps of K = 5504 at once would lose 6e-6. The epilogue adds the roundings
    of the bias, the scale and the residual, 2^-24 each of what they round."""
    mt = _mt()
    g = torch.Generator(device=DEV).manual_seed(M + K)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    ld, p, unit = (N + 7) // 8 * 8 + 8, 0.25, 2.0 ** -24
    A, W, bias = r(M, K).bfloat16(), (r(N, K) / K ** 0.5).bfloat16(), (0.3 * r(N)).bfloat16()
    R, C = r(M, ld), torch.full((M + 1, ld), 77.0, device=DEV)
    Z = torch.full((M + 1, ld), 77.0, dtype=BF16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    drop = mt.mt_dropout(p, SEED, OFFSET, 0, 3)
    keep = torch.from_numpy(block.dropout_keep(M, N, p, SEED, OFFSET, 3)).to(DEV)
    was = mt.mt_k_gemm_variant(fam)
    try:
        mt.mt_k_linear_fwd(A.data_ptr(), K, W.data_ptr(), K, bias.data_ptr(), mt.MT_ACT_RELU, drop, R.data_ptr(), ld, Z.data_ptr(),
                           ld, C.data_ptr(), 0, ld, M, N, K, stream(), err.data_ptr())
        torch.cuda.synchronize()
        assert int(err) == 0
        product = A.double() @ W.double().T
        U = product + bias.double()
        kept = keep & (U > 0)
        D = torch.where(keep, U.clamp(min=0) / (1 - p), 0.0)
        want = R[:, :N].double() + D
        got = C[:M, :N]
        assert torch.equal(got[~keep], R[:, :N][~keep])  # what is dropped leaves the residual as it is
        lost = 60 * unit * float((product * kept).norm()) / (1 - p)
        assert far(got, want) <= lost + unit * float(2 * D.norm() + want.norm())
        assert bool(((Z[:M, :N].double() - U).abs() <= 2.0 ** -8 * U.abs() +
                     (K / 16 + 16) * 2.0 ** -23 * (A.double().abs() @ W.double().abs().T)).all())
        for t in (C, Z):
            assert bool((t[:, N:] == 77).all()) and bool((t[M] == 77).all())
        # back: the same depth, GELU's slope at a Z of its own
        Wk, zb = torch.zeros(K, ld, dtype=BF16, device=DEV), (1.5 * r(M, ld)).bfloat16()
        Wk[:, :N] = W.T
        dZ = torch.full((M + 1, ld), 77.0, dtype=BF16, device=DEV)
        part, db = scratch(mt.mt_k_linear_bwd_act_partial_floats(M, N)), scratch(N)
        mt.mt_k_linear_bwd_act(A.data_ptr(), K, Wk.data_ptr(), ld, zb.data_ptr(), ld, mt.MT_ACT_GELU, drop, dZ.data_ptr(), ld,
                               part.data_ptr(), db.data_ptr(), M, N, K, stream(), err.data_ptr())
        torch.cuda.synchronize()
    finally:
        mt.mt_k_gemm_variant(was)
    assert int(err) == 0
    z = zb[:, :N].double()
    slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = torch.where(keep, product * slope / (1 - p), 0.0)
    assert bool((dZ[:M, :N][~keep] == 0).all()) and bool((dZ[:, N:] == 77).all()) and bool((dZ[M] == 77).all())
    # dZ: rounded by 2^-8 at most, and by 2^-8 / sqrt 3 rms; the rest is far below
    assert far(dZ[:M, :N], want) <= 2.0 ** -8 * float(want.norm())
    # db: the product's loss is the same share of every term; the terms' own roundings (slope within 16 units, scale) and
    # the additions (32 rows, then up to 32 chains) are random
    assert far(db[:N], want.sum(0)) <= 60 * unit * float(want.sum(0).norm()) + 16 * unit * float(want.norm())
    assert bool(torch.isnan(db[N])) and bool(torch.isnan(part[-1]))


@pytest.mark.parametrize("out", [F32, BF16])
def test_products_at_the_largest_depth(out):
    """K = 2^20. fp32 outputs: parts of 60 x 2^-24 as at any depth, and some 1366
    of them added one after the other, each addition rounding by 2^-24 at random:
    sqrt(1366) = 37 units. bf16 outputs are low by about 1e-9 K = 1.1e-3 (65536
    steps of half a unit in the worst case, 2^-8) beside their own rounding."""
    mt = _mt()
    M, N, K = 5, 24, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(0)
    A, W = (torch.randn(n, K, generator=g, device=DEV).bfloat16() for n in (M, N))
    C = torch.full((M, N), 77.0, dtype=out, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    mt.mt_k_linear_fwd(A.data_ptr(), K, W.data_ptr(), K, 0, 0, None, 0, 0, 0, 0, C.data_ptr(), 0 if out == F32 else 1, N, M, N, K,
                       stream(), err.data_ptr())
    want = A.double() @ W.double().T
    assert int(err) == 0
    assert far(C, want) <= float(want.norm()) * ((60 + 37) * 2.0 ** -24 if out == F32 else 2.0 ** -8 + 2.0 ** -8)


@pytest.mark.parametrize("K", [897, 961, 1088, 1281, 1345, 1729, 1857, 2305, 5504])
@pytest.mark.parametrize("M,N", [(512, 512), (40, 2048)])
def test_fp32_outputs_stay_below_the_stated_loss(K, M, N):
    """C and the bias gradient within 1e-6 of themselves (relative L2), as the
    header says, where the accumulator is added up in two parts or a few."""
    mt = _mt()
    g = torch.Generator(device=DEV).manual_seed(K)
    ld = (K + 7) // 8 * 8
    A, W = (torch.zeros(n, ld, dtype=BF16, device=DEV) for n in (M, N))
    A[:, :K], W[:, :K] = torch.randn(M, K, generator=g, device=DEV), torch.randn(N, K, generator=g, device=DEV)
    Wk = W[:, :K].T.contiguous()
    C, dZ, db = torch.zeros(M, N, device=DEV), torch.zeros(M, N, dtype=BF16, device=DEV), torch.zeros(N, device=DEV)
    part = torch.zeros(mt.mt_k_linear_bwd_act_partial_floats(M, N), device=DEV)
    mt.mt_k_linear_fwd(A.data_ptr(), ld, W.data_ptr(), ld, 0, 0, None, 0, 0, 0, 0, C.data_ptr(), 0, N, M, N, K, stream())
    mt.mt_k_linear_bwd_act(A.data_ptr(), ld, Wk.data_ptr(), N, 0, 0, 0, None, dZ.data_ptr(), N, part.data_ptr(), db.data_ptr(), M,
                           N, K, stream())
    want = A.double() @ W.double().T
    assert far(C, want) <= 1e-6 * float(want.norm())
    assert far(db, want.sum(0)) <= 1e-6 * float(want.sum(0).norm())
