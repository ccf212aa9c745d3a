"""Layer norm, dropout, biased linear layers and the gated feed-forward part
(through the C ABI) against the fp64 definitions of oracle/block.py on the same
bf16 or fp32 inputs: ragged sizes, pitches with untouched padding, every type
combination, dropped NaN and infinities, captured graphs, two calls at once,
offsets past 2^31 elements, and the whole block run together.

Tolerances count roundings. A bf16 output is off by half a step, 2^-8 of the
value, an fp32 output by 2^-24. A product over K accumulates K / 16 steps of 16
terms on the tensor cores, each truncating to fp32: (K / 16 + 16) 2^-23 of the
sum of the terms' magnitudes. Activations: slope at most 1.13, their own error
below 2^-20 of |z| (value) or of 1 + |z| (slope): exp is off by 2 + 1.2 |z|
units, weighted by s (1 - s), erf by 2 units. Sums over rows: at most 128
additions in a chain at these sizes, 128 x 2^-24 of the sum of magnitudes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CHAIN = 128 * 2.0 ** -24
PAD = 77.0  # what the columns behind a row hold; no call may change it


def _mt():
    from host_memory_streamed_layer_b200 import mt
    return mt


def kind(t):
    return {torch.float32: 0, torch.bfloat16: 1}[t]


class Mat:
    """A matrix in a wider buffer, PAD in the columns behind it and in a row behind the last."""

    def __init__(self, rows, cols, dtype, value=None, extra=8):
        self.ld = (cols + 7) // 8 * 8 + extra
        self.buf = torch.full((rows + 1, self.ld), PAD, dtype=dtype, device=DEV)
        self.m = self.buf[:rows, :cols]
        if value is None:
            self.m.fill_(float("nan"))
        else:
            self.m.copy_(torch.as_tensor(value, dtype=torch.float32, device=DEV))
        self.ptr, self.dtype, self.kind = self.buf.data_ptr(), dtype, kind(dtype)

    def np(self):
        """The matrix as fp64, after a look at what surrounds it."""
        torch.cuda.synchronize()
        rows, cols = self.m.shape
        assert (self.buf[:, cols:] == PAD).all() and (self.buf[rows:] == PAD).all(), "written outside the matrix"
        return self.m.double().cpu().numpy()


def vec(v, dtype=torch.float32):
    return torch.as_tensor(np.asarray(v, dtype=np.float32)).to(dtype).to(DEV)


def np64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def within(got, want, tol):
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def stream():
    return torch.cuda.current_stream().cuda_stream


def scratch(n):
    return torch.full((n + 1,), float("nan"), device=DEV)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
LN = [(1, 1), (3, 7), (300, 256), (9, 257), (37, 2048), (41, 2049), (5, 5120), (129, 1000), (2, 8191), (700, 512),
      (1300, 24), (3, 8192), (7, 4097)]
TYPES = [torch.float32, torch.bfloat16]


def ln_inputs(T, d, xt, yt, seed=0):
    rng = np.random.default_rng(seed + 1000 * T + d)
    x = Mat(T, d, xt, rng.normal(0, 2, (T, d)) + 5 * rng.normal(size=(T, 1)))
    g, b = vec(1 + 0.1 * rng.normal(size=d), torch.bfloat16), vec(0.3 * rng.normal(size=d), torch.bfloat16)
    return rng, x, g, b


@pytest.mark.parametrize("T,d", LN)
@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
def test_layernorm_fwd(T, d, xt, yt):
    mt = _mt()
    _, x, g, b = ln_inputs(T, d, xt, yt)
    X = x.np()
    for shift in (True, False):
        y = Mat(T, d, yt)
        m, r = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        mt.mt_k_layernorm_fwd(x.ptr, x.kind, x.ld, g.data_ptr(), b.data_ptr() if shift else 0, y.ptr, y.kind, y.ld,
                              m.data_ptr(), r.data_ptr(), T, d, 1e-5, stream())
        B = np64(b) if shift else 0.0 * np64(b)
        want, wm, wr = block.layernorm_fwd(X, np64(g), B, 1e-5)
        size = np.abs(X).mean(axis=1, keepdims=True)
        # r's error: that of the centred squares' sum, and m's error against the row's spread
        tr = CHAIN * wr * (1 + size[:, 0] * wr)
        within(np64(m), wm, CHAIN * size[:, 0])
        within(np64(r), wr, tr)
        xh = np.abs(X - wm[:, None]) * wr[:, None]
        tol = HALF[yt] * np.abs(want) + np.abs(np64(g)) * (CHAIN * size * wr[:, None] + xh * (tr / wr)[:, None]) + \
            4 * 2.0 ** -24 * (xh * np.abs(np64(g)) + np.abs(B))
        within(y.np(), want, tol)
        x.np()  # untouched padding


def test_layernorm_fwd_without_statistics_and_bad_rows():
    """mean and rstd are optional; a row with a NaN or an infinity spoils itself
    only; a constant row gives b."""
    mt = _mt()
    T, d = 40, 515
    _, x, g, b = ln_inputs(T, d, torch.float32, torch.float32)
    x.m[3, 5], x.m[7, 0], x.m[9, :] = float("nan"), float("inf"), 4.25
    ok = [t for t in range(T) if t not in (3, 7)]
    X = x.np()
    y = Mat(T, d, torch.float32)
    mt.mt_k_layernorm_fwd(x.ptr, 0, x.ld, g.data_ptr(), b.data_ptr(), y.ptr, 0, y.ld, 0, 0, T, d, 1e-5, stream())
    want = block.layernorm_fwd(X[ok], np64(g), np64(b), 1e-5)[0]
    got = y.np()
    assert np.isnan(got[3]).all() and np.isnan(got[7]).all()
    assert np.array_equal(got[9], np64(b))
    size = np.abs(X[ok]).mean(axis=1, keepdims=True)
    others = [i for i, t in enumerate(ok) if t != 9]
    r = block.layernorm_fwd(X[ok], np64(g), np64(b), 1e-5)[2][:, None]
    tol = (CHAIN * (1 + size * r) * (2 + np.abs(X[ok]) * r)) * np.abs(np64(g)) + 2.0 ** -22 * np.abs(want)
    within(got[ok][others], want[others], tol[others])


@pytest.mark.parametrize("T,d", LN + [(5000, 136)])
@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("dyt", TYPES)
def test_layernorm_bwd(T, d, xt, dyt):
    mt = _mt()
    rng, x, g, _ = ln_inputs(T, d, xt, dyt)
    X, G = x.np(), np64(g)
    _, wm, wr = block.layernorm_fwd(X, G, 0 * G, 1e-5)
    m, r = vec(wm), vec(wr)
    M, R = np64(m), np64(r)
    dy = Mat(T, d, dyt, rng.normal(size=(T, d)))
    DY = dy.np()
    want, wdg, wdb = block.layernorm_bwd(X, G, M, R, DY)
    xh, w = (X - M[:, None]) * R[:, None], DY * G
    absolute = R[:, None] * (np.abs(w) + np.abs(w).mean(axis=1, keepdims=True) +
                             np.abs(xh) * np.abs(w * xh).mean(axis=1, keepdims=True))
    part = scratch(mt.mt_k_layernorm_bwd_partial_floats(T, d))
    for with_res in (True, False):
        res = Mat(T, d, xt, rng.normal(size=(T, d))) if with_res else None
        RES = res.np() if with_res else 0.0
        dx = Mat(T, d, xt)
        dxb = Mat(T, d, torch.bfloat16) if xt == torch.float32 else None
        dg, db = scratch(d), scratch(d)
        mt.mt_k_layernorm_bwd(x.ptr, x.kind, x.ld, g.data_ptr(), m.data_ptr(), r.data_ptr(), dy.ptr, dy.kind, dy.ld,
                              res.ptr if res else 0, res.ld if res else 0, dx.ptr, dxb.ptr if dxb else 0, dx.ld,
                              part.data_ptr(), dg.data_ptr(), db.data_ptr() if with_res else 0, T, d, stream())
        got = dx.np()
        within(got, want + RES, HALF[xt] * np.abs(want + RES) + CHAIN * (absolute + np.abs(RES)))
        if dxb:
            assert np.array_equal(dxb.np(), torch.tensor(got).bfloat16().double().numpy())  # one rounding of dx
        within(np64(dg)[:d], wdg, CHAIN * np.abs(DY * xh).sum(axis=0))
        if with_res:
            within(np64(db)[:d], wdb, CHAIN * np.abs(DY).sum(axis=0))
        else:
            assert np.isnan(np64(db)).all()
        assert np.isnan(np64(dg)[d]) and np.isnan(np64(part)[-1])


def test_layernorm_bwd_in_place_residual_and_no_rows():
    mt = _mt()
    T, d = 33, 520
    rng, x, g, _ = ln_inputs(T, d, torch.float32, torch.float32)
    m, r = vec(x.np().mean(axis=1)), vec(1 / x.np().std(axis=1))
    dy, res = Mat(T, d, torch.float32, rng.normal(size=(T, d))), rng.normal(size=(T, d))
    part = scratch(mt.mt_k_layernorm_bwd_partial_floats(T, d))
    dg, db = scratch(d), scratch(d)
    outs = []
    for inplace in (False, True):
        dx = Mat(T, d, torch.float32, res if inplace else None)
        rm = dx if inplace else Mat(T, d, torch.float32, res)
        mt.mt_k_layernorm_bwd(x.ptr, 0, x.ld, g.data_ptr(), m.data_ptr(), r.data_ptr(), dy.ptr, 0, dy.ld, rm.ptr, rm.ld,
                              dx.ptr, 0, dx.ld, part.data_ptr(), dg.data_ptr(), db.data_ptr(), T, d, stream())
        outs.append((dx.np(), np64(dg)[:d], np64(db)[:d]))
    assert all(np.array_equal(a, b) for a, b in zip(*outs))
    mt.mt_k_layernorm_bwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, dg.data_ptr(), db.data_ptr(), 0, d, stream())
    assert (np64(dg)[:d] == 0).all() and (np64(db)[:d] == 0).all()
    mt.mt_k_layernorm_fwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, d, 1e-5, stream())


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
SEED, OFFSET = 0x123456789ABCDEF, (1 << 40) + 12345


@pytest.mark.parametrize("T,d", [(1, 1), (3, 5), (100, 1376), (257, 640), (1500, 33), (64, 2050), (2000, 8)])
@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
@pytest.mark.parametrize("p", [0.1, 0.0])
def test_dropout(T, d, xt, yt, p):
    mt = _mt()
    rng = np.random.default_rng(T * d)
    x = Mat(T, d, xt, rng.normal(size=(T, d)))
    drop = mt.mt_dropout(p, SEED, OFFSET, 0, 11)
    keep = block.dropout_keep(T, d, p, SEED, OFFSET, 11)
    want = block.drop(x.np(), p, keep)
    for with_res in (True, False):
        res = Mat(T, d, yt, rng.normal(size=(T, d))) if with_res else None
        RES = res.np() if with_res else 0.0
        y = Mat(T, d, yt)
        mt.mt_k_dropout(x.ptr, x.kind, x.ld, drop, res.ptr if res else 0, res.ld if res else 0, y.ptr, y.kind, y.ld, T, d,
                        stream())
        got = y.np()
        within(got, want + RES, HALF[yt] * np.abs(want + RES) + 3 * 2.0 ** -24 * np.abs(want))
        if not with_res and p:
            assert np.array_equal(got != 0, keep & (x.np() != 0))  # the mask, exactly


def test_dropout_drops_what_is_not_finite_and_works_in_place():
    mt = _mt()
    T, d, p = 64, 200, 0.5
    keep = block.dropout_keep(T, d, p, SEED, OFFSET)
    for bad in (float("nan"), float("inf")):
        x = Mat(T, d, torch.float32, np.full((T, d), bad))
        mt.mt_k_dropout(x.ptr, 0, x.ld, mt.mt_dropout(p, SEED, OFFSET), 0, 0, x.ptr, 0, x.ld, T, d, stream())
        got = x.np()
        assert (got[~keep] == 0).all() and not np.isfinite(got[keep]).any()
    x, y = Mat(T, d, torch.bfloat16, np.ones((T, d))), Mat(T, d, torch.float32, np.full((T, d), 3.0))
    mt.mt_k_dropout(x.ptr, 1, x.ld, mt.mt_dropout(p, SEED, OFFSET), y.ptr, y.ld, y.ptr, 0, y.ld, T, d, stream())
    assert np.array_equal(y.np(), np.where(keep, 5.0, 3.0))
    mt.mt_k_dropout(0, 0, 0, mt.mt_dropout(p, SEED, OFFSET), 0, 0, 0, 0, 0, 0, d, stream())  # no rows


def test_dropout_rows_of_a_larger_matrix_and_negative_offsets():
    mt = _mt()
    T, d, p = 300, 100, 0.25
    x = Mat(T, d, torch.bfloat16, np.ones((T, d)))
    whole = Mat(T, d, torch.float32)
    mt.mt_k_dropout(x.ptr, 1, x.ld, mt.mt_dropout(p, -5, -7), 0, 0, whole.ptr, 0, whole.ld, T, d, stream())
    assert np.array_equal(whole.np() != 0, block.dropout_keep(T, d, p, -5, -7))
    a = 117
    piece = Mat(T - a, d, torch.float32)
    mt.mt_k_dropout(x.ptr + 2 * x.ld * a, 1, x.ld, mt.mt_dropout(p, -5, -7, 0, a), 0, 0, piece.ptr, 0, piece.ld, T - a, d,
                    stream())
    assert np.array_equal(piece.np(), whole.np()[a:])


def test_dropout_captured_graph_draws_anew_from_the_device_offset():
    mt = _mt()
    T, d, p = 50, 96, 0.5
    x, y = Mat(T, d, torch.bfloat16, np.ones((T, d))), Mat(T, d, torch.float32)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    drop = mt.mt_dropout(p, SEED, OFFSET, step.data_ptr())
    mt.mt_k_dropout(x.ptr, 1, x.ld, drop, 0, 0, y.ptr, 0, y.ld, T, d, stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mt.mt_k_dropout(x.ptr, 1, x.ld, drop, 0, 0, y.ptr, 0, y.ld, T, d, stream())
        step.add_(3)
    step.fill_(-4)
    for k in range(3):
        graph.replay()
        assert np.array_equal(y.np() != 0, block.dropout_keep(T, d, p, SEED, OFFSET - 4 + 3 * k))
    del graph


# ---------------------------------------------------------------------------
# Linear layers
# ---------------------------------------------------------------------------
def product_error(A, B, K):
    """Bound of the tensor cores' error of A B^T."""
    return (K / 16 + 16) * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)


SHAPES = [(1, 8, 8), (1, 1, 1), (5, 100, 40), (128, 256, 64), (300, 200, 100), (257, 1376, 256), (64, 33, 1000),
          (1000, 770, 333), (130, 5000, 72)]
LARGE = [(2600, 1400, 130), (1290, 4100, 200)]
FAMILIES = [0, 1, 2]  # automatic, single CTAs, CTA pairs


class family:
    def __init__(self, v):
        self.v = v

    def __enter__(self):
        self.was = _mt().mt_k_gemm_variant(self.v)

    def __exit__(self, *a):
        _mt().mt_k_gemm_variant(self.was)


def linear_case(M, N, K, act, out, p, res, with_z=True, bias=True, seed=0):
    mt = _mt()
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    A, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(N, K, torch.bfloat16, rng.normal(size=(N, K)) / K ** 0.5)
    b = vec(0.5 * rng.normal(size=N), torch.bfloat16)
    R = Mat(M, N, out, rng.normal(size=(M, N))) if res else None
    C, Z = Mat(M, N, out), Mat(M, N, torch.bfloat16) if with_z else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    drop = mt.mt_dropout(p, SEED, OFFSET, 0, 5) if p else None
    mt.mt_k_linear_fwd(A.ptr, A.ld, W.ptr, W.ld, b.data_ptr() if bias else 0, block.ACTS.index(act), drop,
                       R.ptr if R else 0, R.ld if R else 0, Z.ptr if Z else 0, Z.ld if Z else 0, C.ptr, C.kind, C.ld, M, N,
                       K, stream(), err.data_ptr())
    a, w = A.np(), W.np()
    assert int(err) == 0
    keep = block.dropout_keep(M, N, p, SEED, OFFSET, 5) if p else None
    r = R.np() if R else 0.0
    want, u = block.linear_fwd(a, w, np64(b) if bias else 0.0, act, p, keep, r)
    eu = product_error(a, w, K) + 2.0 ** -24 * np.abs(u)
    scale = 1 / (1 - p)
    ec = scale * (1.13 * eu + 2.0 ** -20 * np.abs(u)) + 2.0 ** -22 * (np.abs(want) + np.abs(r))
    if p:
        ec = np.where(keep, ec, 2.0 ** -24 * np.abs(r))
    within(C.np(), want, HALF[out] * np.abs(want) + ec)
    if Z:
        within(Z.np(), u, HALF[torch.bfloat16] * np.abs(u) + eu)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fam", FAMILIES)
@pytest.mark.parametrize("out", TYPES)
def test_linear_fwd_shapes(M, N, K, fam, out):
    with family(fam):
        linear_case(M, N, K, "gelu", out, 0.1, True)


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("fam", FAMILIES)
def test_linear_fwd_many_tiles(M, N, K, fam):
    with family(fam):
        linear_case(M, N, K, "silu", torch.bfloat16, 0.0, False)


@pytest.mark.parametrize("act", block.ACTS)
@pytest.mark.parametrize("p,res,with_z,bias", [(0.0, False, False, False), (0.3, True, False, True), (0.0, True, True, False),
                                               (0.3, False, True, True)])
@pytest.mark.parametrize("out", TYPES)
def test_linear_fwd_options(act, p, res, with_z, bias, out):
    linear_case(150, 203, 96, act, out, p, res, with_z, bias)


def bwd_case(M, N, K, act, p, with_db=True, inplace=False, seed=0):
    mt = _mt()
    rng = np.random.default_rng(seed + M * 5 + N * 3 + K)
    dY, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(K, N, torch.bfloat16, rng.normal(size=(K, N)) / K ** 0.5)
    Z = Mat(M, N, torch.bfloat16, 1.5 * rng.normal(size=(M, N)))
    zv = Z.np()
    dZ = Z if inplace else Mat(M, N, torch.bfloat16)
    part, db = scratch(mt.mt_k_linear_bwd_act_partial_floats(M, N)), scratch(N)
    drop = mt.mt_dropout(p, SEED, OFFSET, 0, 2) if p else None
    use_z = act != "none" or inplace
    mt.mt_k_linear_bwd_act(dY.ptr, dY.ld, W.ptr, W.ld, Z.ptr if use_z else 0, Z.ld if use_z else 0, block.ACTS.index(act),
                           drop, dZ.ptr, dZ.ld, part.data_ptr() if with_db else 0, db.data_ptr() if with_db else 0, M, N, K,
                           stream())
    dy, w = dY.np(), W.np()
    keep = block.dropout_keep(M, N, p, SEED, OFFSET, 2) if p else np.ones((M, N), bool)
    want, wdb = block.linear_bwd_act(dy, w, zv, act, p, keep)
    dh = dy @ w
    e = np.where(keep, (1.13 * product_error(dy, w.T, K) + 2.0 ** -20 * (1 + np.abs(zv)) * np.abs(dh)) / (1 - p), 0.0)
    within(dZ.np(), want, HALF[torch.bfloat16] * np.abs(want) + e)
    if with_db:
        within(np64(db)[:N], wdb, e.sum(axis=0) + CHAIN * np.abs(want).sum(axis=0))
        assert np.isnan(np64(db)[N]) and np.isnan(np64(part)[-1])


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fam", FAMILIES)
def test_linear_bwd_act_shapes(M, N, K, fam):
    with family(fam):
        bwd_case(M, N, K, "gelu", 0.1)


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("fam", FAMILIES)
def test_linear_bwd_act_many_tiles(M, N, K, fam):
    with family(fam):
        bwd_case(M, N, K, "relu", 0.0)


@pytest.mark.parametrize("act", block.ACTS)
@pytest.mark.parametrize("p,with_db,inplace", [(0.0, False, False), (0.3, True, True)])
def test_linear_bwd_act_options(act, p, with_db, inplace):
    bwd_case(150, 203, 96, act, p, with_db, inplace)


@pytest.mark.parametrize("M,N", [(1, 1), (3, 13), (100, 1376), (700, 640), (1500, 33), (65, 8200), (5000, 16)])
@pytest.mark.parametrize("act", block.ACTS)
@pytest.mark.parametrize("dct", TYPES)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_act_bwd(M, N, act, dct, p):
    mt = _mt()
    rng = np.random.default_rng(M + N)
    dC, Z = Mat(M, N, dct, rng.normal(size=(M, N))), Mat(M, N, torch.bfloat16, 1.5 * rng.normal(size=(M, N)))
    dZ, db = Mat(M, N, torch.bfloat16), scratch(N)
    part = scratch(mt.mt_k_act_bwd_partial_floats(M, N))
    use_z = act != "none"
    mt.mt_k_act_bwd(dC.ptr, dC.kind, dC.ld, Z.ptr if use_z else 0, Z.ld if use_z else 0, block.ACTS.index(act),
                    mt.mt_dropout(p, SEED, OFFSET) if p else None, dZ.ptr, dZ.ld, part.data_ptr(), db.data_ptr(), M, N,
                    stream())
    keep = block.dropout_keep(M, N, p, SEED, OFFSET) if p else np.ones((M, N), bool)
    want, wdb = block.act_bwd(dC.np(), Z.np(), act, p, keep)
    e = 2.0 ** -20 * (1 + np.abs(Z.np())) * np.abs(dC.np()) / (1 - p) * keep
    within(dZ.np(), want, HALF[torch.bfloat16] * np.abs(want) + e)
    within(np64(db)[:N], wdb, e.sum(axis=0) + CHAIN * np.abs(want).sum(axis=0))
    assert np.isnan(np64(db)[N]) and np.isnan(np64(part)[-1])


def test_dropped_elements_are_zero_whatever_the_product_holds():
    """NaN and infinite inputs make whole rows of the product NaN; the dropped
    elements of those rows are exactly zero (or the residual), forward and back."""
    mt = _mt()
    M, N, K, p = 140, 72, 64, 0.5
    rng = np.random.default_rng(0)
    keep = block.dropout_keep(M, N, p, SEED, OFFSET)
    a = rng.normal(size=(M, K))
    a[5, 3], a[77, 0] = np.nan, np.inf
    A, W = Mat(M, K, torch.bfloat16, a), Mat(N, K, torch.bfloat16, rng.normal(size=(N, K)))
    C, R = Mat(M, N, torch.float32), Mat(M, N, torch.float32, np.full((M, N), 2.0))
    drop = mt.mt_dropout(p, SEED, OFFSET)
    mt.mt_k_linear_fwd(A.ptr, A.ld, W.ptr, W.ld, 0, 0, drop, R.ptr, R.ld, 0, 0, C.ptr, 0, C.ld, M, N, K, stream())
    got = C.np()
    assert (got[~keep] == 2.0).all() and not np.isfinite(got[[5, 77]][keep[[5, 77]]]).any()
    assert np.isfinite(np.delete(got, [5, 77], axis=0)).all()
    z = rng.normal(size=(M, N))
    z[9, :] = np.nan
    Z, W2, dZ = Mat(M, N, torch.bfloat16, z), Mat(K, N, torch.bfloat16, rng.normal(size=(K, N))), Mat(M, N, torch.bfloat16)
    db, part = scratch(N), scratch(mt.mt_k_linear_bwd_act_partial_floats(M, N))
    mt.mt_k_linear_bwd_act(A.ptr, A.ld, W2.ptr, W2.ld, Z.ptr, Z.ld, mt.MT_ACT_GELU, drop, dZ.ptr, dZ.ld, part.data_ptr(),
                           db.data_ptr(), M, N, K, stream())
    got = dZ.np()
    assert (got[~keep] == 0).all() and not np.isfinite(got[[5, 9, 77]][keep[[5, 9, 77]]]).any()
    clean = [j for j in range(N) if not keep[[5, 9, 77], j].any()]
    assert clean and np.isfinite(np64(db)[clean]).all()
    mt.mt_k_act_bwd(R.ptr, 0, R.ld, Z.ptr, Z.ld, mt.MT_ACT_SILU, drop, dZ.ptr, dZ.ld,
                    scratch(mt.mt_k_act_bwd_partial_floats(M, N)).data_ptr(), db.data_ptr(), M, N, stream())
    assert (dZ.np()[~keep] == 0).all()


def test_activation_extremes():
    """Saturated and huge pre-activations, exact in bf16: the value is z or 0,
    the slope 1 or 0, and NaN stays NaN."""
    mt = _mt()
    z = np.array([-1e30, -3e4, -100.0, -0.0, 0.0, 100.0, 3e4, 1e30, 3e38, -3e38], dtype=np.float32)
    z = torch.tensor(z).bfloat16().double().numpy()
    N = len(z)
    A, W = Mat(1, 8, torch.bfloat16, np.eye(1, 8)), Mat(N, 8, torch.bfloat16, z[:, None] * np.eye(1, 8))
    for act in block.ACTS[1:]:
        C = Mat(1, N, torch.float32)
        mt.mt_k_linear_fwd(A.ptr, A.ld, W.ptr, W.ld, 0, block.ACTS.index(act), None, 0, 0, 0, 0, C.ptr, 0, C.ld, 1, N, 8,
                           stream())
        assert np.array_equal(C.np()[0], np.maximum(z, 0)), act
        dC, Z, dZ = Mat(1, N, torch.float32, np.ones((1, N))), Mat(1, N, torch.bfloat16, z[None]), Mat(1, N, torch.bfloat16)
        mt.mt_k_act_bwd(dC.ptr, 0, dC.ld, Z.ptr, Z.ld, block.ACTS.index(act), None, dZ.ptr, dZ.ld, 0, 0, 1, N, stream())
        at0 = 0.0 if act == "relu" else 0.5
        assert np.array_equal(dZ.np()[0], np.where(z > 0, 1.0, np.where(z < 0, 0.0, at0))), act
    nan = Mat(1, 8, torch.bfloat16, np.full((1, 8), np.nan))
    for act in block.ACTS:
        C = Mat(1, N, torch.float32)
        mt.mt_k_linear_fwd(nan.ptr, nan.ld, W.ptr, W.ld, 0, block.ACTS.index(act), None, 0, 0, 0, 0, C.ptr, 0, C.ld, 1, N, 8,
                           stream())
        assert np.isnan(C.np()).all(), act


# ---------------------------------------------------------------------------
# Gated feed-forward
# ---------------------------------------------------------------------------
GATED = [(1, 8, 8), (5, 104, 40), (128, 256, 64), (300, 200, 100), (257, 1376, 256), (64, 40, 1000), (1000, 776, 333),
         (13, 5504, 72)]


@pytest.mark.parametrize("M,F,K", GATED + [(2600, 712, 130)])
@pytest.mark.parametrize("fam", FAMILIES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_fwd(M, F, K, fam, act):
    mt = _mt()
    rng = np.random.default_rng(M * 7 + F * 3 + K)
    x, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(2 * F, K, torch.bfloat16, rng.normal(size=(2 * F, K)) / K ** 0.5)
    X, WW = x.np(), W.np()
    want, g, u = block.gated_fwd(X, WW[:F], WW[F:], act)
    eg, eu = product_error(X, WW[:F], K), product_error(X, WW[F:], K)
    a = block.act(g, act)
    ea = 1.13 * eg + 2.0 ** -20 * np.abs(g)
    with family(fam):
        for keep in (True, False):
            h, gu = Mat(M, F, torch.bfloat16), Mat(M, 2 * F, torch.bfloat16) if keep else None
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            mt.mt_k_gated_ffn_fwd(x.ptr, x.ld, W.ptr, W.ld, block.ACTS.index(act), gu.ptr if gu else 0, gu.ld if gu else 0,
                                  h.ptr, h.ld, M, F, K, stream(), err.data_ptr())
            within(h.np(), want, HALF[torch.bfloat16] * np.abs(want) + ea * np.abs(u) + np.abs(a) * eu + ea * eu +
                   2.0 ** -22 * np.abs(want))
            if keep:
                e = np.concatenate([eg, eu], axis=1)
                within(gu.np(), np.concatenate([g, u], axis=1), HALF[torch.bfloat16] * np.abs(np.concatenate([g, u], axis=1)) + e)
            assert int(err) == 0


@pytest.mark.parametrize("M,F,K", GATED + [(2600, 1400, 130)])
@pytest.mark.parametrize("fam", FAMILIES)
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_gated_bwd(M, F, K, fam, act):
    mt = _mt()
    rng = np.random.default_rng(M * 5 + F * 3 + K)
    dy, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(K, F, torch.bfloat16, rng.normal(size=(K, F)) / K ** 0.5)
    gu = Mat(M, 2 * F, torch.bfloat16, 1.5 * rng.normal(size=(M, 2 * F)))
    DY, WW, GU = dy.np(), W.np(), gu.np()
    g, u = GU[:, :F], GU[:, F:]
    wg, wu, wh = block.gated_bwd(DY, WW, g, u, act)
    dh, ed = DY @ WW, product_error(DY, WW.T, K)
    eg = np.abs(u) * (1.13 * ed + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(dh))
    eu = np.abs(block.act(g, act)) * ed + 2.0 ** -20 * np.abs(g) * np.abs(dh)
    want = np.concatenate([wg, wu], axis=1)
    tol = HALF[torch.bfloat16] * np.abs(want) + np.concatenate([eg, eu], axis=1) + 2.0 ** -22 * np.abs(want)
    with family(fam):
        for inplace in (False, True):
            dgu = Mat(M, 2 * F, torch.bfloat16, GU) if inplace else Mat(M, 2 * F, torch.bfloat16)
            src = dgu if inplace else gu
            h = None if inplace else Mat(M, F, torch.bfloat16)
            mt.mt_k_gated_ffn_bwd(dy.ptr, dy.ld, W.ptr, W.ld, src.ptr, src.ld, block.ACTS.index(act), dgu.ptr, dgu.ld,
                                  h.ptr if h else 0, h.ld if h else 0, M, F, K, stream())
            within(dgu.np(), want, tol)
            if h:
                within(h.np(), wh, HALF[torch.bfloat16] * np.abs(wh) + 2.0 ** -20 * np.abs(g * u))


@pytest.mark.parametrize("act", block.ACTS)
def test_gated_activations(act):
    """Every activation of the gate, against the plain products of the same weights."""
    mt = _mt()
    M, F, K = 70, 88, 48
    rng = np.random.default_rng(5)
    x, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(2 * F, K, torch.bfloat16, rng.normal(size=(2 * F, K)) / 7)
    h = Mat(M, F, torch.bfloat16)
    mt.mt_k_gated_ffn_fwd(x.ptr, x.ld, W.ptr, W.ld, block.ACTS.index(act), 0, 0, h.ptr, h.ld, M, F, K, stream())
    X, WW = x.np(), W.np()
    want, g, u = block.gated_fwd(X, WW[:F], WW[F:], act)
    ea = 1.13 * product_error(X, WW[:F], K) + 2.0 ** -20 * np.abs(g)
    eu = product_error(X, WW[F:], K)
    within(h.np(), want, (HALF[torch.bfloat16] + 2.0 ** -22) * np.abs(want) + ea * np.abs(u) + (np.abs(block.act(g, act)) + ea) * eu)


@pytest.mark.parametrize("fam", FAMILIES)
@pytest.mark.parametrize("M,N,K", [(256, 256, 13824), (300, 1000, 2056), (5, 64, 5504), (2309, 1948, 968)])
def test_fp32_outputs_keep_their_digits_at_any_depth(M, N, K, fam):
    """Long sums in fp32 outputs: the accumulator is added up after at most 15
    k-blocks of 64 on average, 60 steps that each truncate half a unit, 2^-24, on
    average: 60 x 2^-24 of the sum (relative L2). All 864 steps of K = 13824 at
    once would lose 1.6e-5."""
    mt = _mt()
    g = torch.Generator(device=DEV).manual_seed(K)
    ld = (N + 7) // 8 * 8
    A = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    W = (torch.randn(K, ld, generator=g, device=DEV) / K ** 0.5).bfloat16()
    Wt = W[:, :N].t().contiguous()
    C, dZ = torch.zeros(M, ld, device=DEV), torch.zeros(M, ld, dtype=torch.bfloat16, device=DEV)
    part, db = scratch(mt.mt_k_linear_bwd_act_partial_floats(M, N)), scratch(N)
    with family(fam):
        mt.mt_k_linear_fwd(A.data_ptr(), K, Wt.data_ptr(), K, 0, 0, None, 0, 0, 0, 0, C.data_ptr(), 0, ld, M, N, K, stream())
        mt.mt_k_linear_bwd_act(A.data_ptr(), K, W.data_ptr(), ld, 0, 0, 0, None, dZ.data_ptr(), ld, part.data_ptr(), db.data_ptr(),
                               M, N, K, stream())
    want = A.double() @ W[:, :N].double()
    for got, ref in [(C[:, :N], want), (db[:N], want.sum(0))]:
        assert float((got.double() - ref).norm() / ref.norm()) <= 60 * 2.0 ** -24
    assert float((dZ[:, :N].double() - want).norm() / want.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("fam", [0, 2])
@pytest.mark.parametrize("M,N,K", [(2309, 1948, 136), (2309, 2048, 64), (4000, 1300, 200), (19200, 264, 40)])
def test_a_last_wave_of_narrower_tiles(M, N, K, fam):
    """More 256-wide pair tiles than a 148-SM part has pairs, and some left over:
    those are cut in two or four, with parts that end inside the matrix, at its
    edge and behind it."""
    with family(fam):
        linear_case(M, N, K, "silu", torch.bfloat16, 0.1, True)
        linear_case(M, N, K, "none", torch.float32, 0.0, True)
        bwd_case(M, N, K, "gelu", 0.0)
    F = (N // 2 + 7) // 8 * 8
    test_gated_fwd(M, F, K, fam, "silu")
    test_gated_bwd(M, (N + 7) // 8 * 8, K, fam, "silu")


# ---------------------------------------------------------------------------
# Calls beside one another
# ---------------------------------------------------------------------------
def test_same_bits_again_and_on_two_streams_at_once():
    """Repeated calls, and calls in flight together on two streams with scratch
    of their own, give the bits of a call alone."""
    mt = _mt()
    M, N, K = 900, 700, 512
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    dY, W, Z = [r(M, K) for _ in range(2)], r(K, N + 4)[:, :N], r(M, N + 4)[:, :N]
    x, dy, gain = torch.randn(M, 768, generator=g, device=DEV), torch.randn(M, 768, generator=g, device=DEV), r(768)
    m, rs = x.mean(1), 1 / x.std(1)
    drop = mt.mt_dropout(0.2, SEED, OFFSET)

    def call(i, st):
        dZ, db = torch.zeros(M, N + 4, dtype=torch.bfloat16, device=DEV), torch.zeros(N, device=DEV)
        part = torch.empty(mt.mt_k_linear_bwd_act_partial_floats(M, N), device=DEV)
        dx, dg, dbeta = torch.zeros_like(x), torch.zeros(768, device=DEV), torch.zeros(768, device=DEV)
        p2 = torch.empty(mt.mt_k_layernorm_bwd_partial_floats(M, 768), device=DEV)
        st.wait_stream(torch.cuda.current_stream())
        mt.mt_k_linear_bwd_act(dY[i].data_ptr(), K, W.data_ptr(), N + 4, Z.data_ptr(), N + 4, mt.MT_ACT_SILU, drop,
                               dZ.data_ptr(), N + 4, part.data_ptr(), db.data_ptr(), M, N, K, st.cuda_stream)
        mt.mt_k_layernorm_bwd(x.data_ptr(), 0, 768, gain.data_ptr(), m.data_ptr(), rs.data_ptr(), dy.data_ptr(), 0, 768, 0, 0,
                              dx.data_ptr(), 0, 768, p2.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), M, 768, st.cuda_stream)
        return [dZ, db, dx, dg, dbeta], (part, p2)

    alone = []
    for i in range(2):
        out, _keep = call(i, torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append(out)
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in range(2)]
        both = [call(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        for want, (got, _) in zip(alone, both):
            assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_bounded_wait_ends_the_call_and_the_next_one_is_right():
    """With the main-loop wait limit at 0 a single-CTA product gives up at its
    first incomplete wait, records a code and returns; the context stays
    usable and the same call with the default limit is right."""
    mt = _mt()
    M, N, K = 128, 64, 8192
    g = torch.Generator(device=DEV).manual_seed(0)
    A, W = torch.randn(M, K, generator=g, device=DEV).bfloat16(), torch.randn(N, K, generator=g, device=DEV).bfloat16() / 90
    C, err = torch.zeros(M, N, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda: mt.mt_k_linear_fwd(A.data_ptr(), K, W.data_ptr(), K, 0, 0, None, 0, 0, 0, 0, C.data_ptr(), 0, N, M, N, K,  # noqa: E731
                                      stream(), err.data_ptr())
    with family(1):
        prev = mt.mt_k_gemm_wait_limit_ns(0)
        try:
            call()
            torch.cuda.synchronize()
            assert int(err) in (1, 2, 3, 4)
        finally:
            mt.mt_k_gemm_wait_limit_ns(prev)
        err.zero_()
        call()
        torch.cuda.synchronize()
    assert int(err) == 0
    a, w = np64(A), np64(W)
    within(np64(C), a @ w.T, product_error(a, w, K) + 2.0 ** -24 * np.abs(a @ w.T))


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (300, 200, 100), (1290, 1100, 200)])
def test_in_place_calls_give_the_bits_of_separate_buffers(M, N, K, out):
    """C over R, dZ over Z, dZ over a bf16 dC, dx over dres: what the header
    allows gives the same bits as buffers of their own."""
    mt = _mt()
    rng = np.random.default_rng(M + N)
    A, W = Mat(M, K, torch.bfloat16, rng.normal(size=(M, K))), Mat(N, K, torch.bfloat16, rng.normal(size=(N, K)))
    r, z = rng.normal(size=(M, N)), rng.normal(size=(M, N))
    drop = mt.mt_dropout(0.25, SEED, OFFSET)
    got = []
    for inplace in (False, True):
        R = Mat(M, N, out, r)
        C = R if inplace else Mat(M, N, out)
        mt.mt_k_linear_fwd(A.ptr, A.ld, W.ptr, W.ld, 0, mt.MT_ACT_SILU, drop, R.ptr, R.ld, 0, 0, C.ptr, C.kind, C.ld, M, N, K,
                           stream())
        Z, dC = Mat(M, N, torch.bfloat16, z), Mat(M, N, out, r)
        dZ = Z if inplace else Mat(M, N, torch.bfloat16)
        db = scratch(N)
        mt.mt_k_act_bwd(dC.ptr, dC.kind, dC.ld, Z.ptr, Z.ld, mt.MT_ACT_GELU, drop, dZ.ptr, dZ.ld,
                        scratch(mt.mt_k_act_bwd_partial_floats(M, N)).data_ptr(), db.data_ptr(), M, N, stream())
        got.append([C.np(), dZ.np(), np64(db)[:N]])
        if out == torch.bfloat16:
            Z, dC = Mat(M, N, torch.bfloat16, z), Mat(M, N, out, r)
            dZ = dC if inplace else Mat(M, N, torch.bfloat16)
            mt.mt_k_act_bwd(dC.ptr, dC.kind, dC.ld, Z.ptr, Z.ld, mt.MT_ACT_RELU, drop, dZ.ptr, dZ.ld, 0, 0, M, N, stream())
            got[-1].append(dZ.np())
    assert all(np.array_equal(a, b) for a, b in zip(*got))


@pytest.mark.late
def test_gated_and_backward_offsets_past_31_bits():
    """gu, dgu, Z and dZ of more than 2^31 elements: rows at both ends are right."""
    mt = _mt()
    F, K = 4096, 16
    M = (1 << 31) // F + 777
    g = torch.Generator(device=DEV).manual_seed(5)
    at = [0, 3, M - 700, M - 1]
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[at] = torch.randn(len(at), K, generator=g, device=DEV).bfloat16()
    W, Wd = torch.randn(2 * F, K, generator=g, device=DEV).bfloat16(), torch.randn(K, F, generator=g, device=DEV).bfloat16()
    gu, h = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=DEV), torch.empty(M, F, dtype=torch.bfloat16, device=DEV)
    mt.mt_k_gated_ffn_fwd(x.data_ptr(), K, W.data_ptr(), K, mt.MT_ACT_SILU, gu.data_ptr(), 2 * F, h.data_ptr(), F, M, F, K, stream())
    X, WW = np64(x[at]), np64(W)
    want, gate, up = block.gated_fwd(X, WW[:F], WW[F:], "silu")
    e = product_error(X, WW, K)
    both = np.concatenate([gate, up], axis=1)
    within(np64(gu[at]), both, 2.0 ** -8 * np.abs(both) + e)
    ea, eu = 1.13 * e[:, :F] + 2.0 ** -20 * np.abs(gate), e[:, F:]
    within(np64(h[at]), want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + ea * np.abs(up) + (np.abs(block.act(gate, "silu")) + ea) * eu)
    assert not gu[M - 699:M - 1].any() and not h[M - 699:M - 1].any()
    # back, over gu itself, and through a linear layer over Z itself
    GU = np64(gu[at])
    mt.mt_k_gated_ffn_bwd(x.data_ptr(), K, Wd.data_ptr(), F, gu.data_ptr(), 2 * F, mt.MT_ACT_SILU, gu.data_ptr(), 2 * F, 0, 0, M, F,
                          K, stream())
    wg, wu, _ = block.gated_bwd(X, np64(Wd), GU[:, :F], GU[:, F:], "silu")
    dh, ed = X @ np64(Wd), product_error(X, np64(Wd).T, K)
    tol = np.concatenate([np.abs(GU[:, F:]) * (1.13 * ed + 2.0 ** -20 * (1 + np.abs(GU[:, :F])) * np.abs(dh)),
                          np.abs(block.act(GU[:, :F], "silu")) * ed + 2.0 ** -20 * np.abs(GU[:, :F]) * np.abs(dh)], axis=1)
    want = np.concatenate([wg, wu], axis=1)
    within(np64(gu[at]), want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + tol)
    Z = np64(h[at])
    part, db = scratch(mt.mt_k_linear_bwd_act_partial_floats(M, F)), scratch(F)
    mt.mt_k_linear_bwd_act(x.data_ptr(), K, Wd.data_ptr(), F, h.data_ptr(), F, mt.MT_ACT_GELU, None, h.data_ptr(), F, part.data_ptr(),
                           db.data_ptr(), M, F, K, stream())
    want, wdb = block.linear_bwd_act(X, np64(Wd), Z, "gelu")
    e = 1.13 * ed + 2.0 ** -20 * (1 + np.abs(Z)) * np.abs(dh)
    within(np64(h[at]), want, 2.0 ** -8 * np.abs(want) + e)
    within(np64(db)[:F], wdb, e.sum(axis=0) + CHAIN * np.abs(want).sum(axis=0))  # the other rows' dY is zero


@pytest.mark.late
def test_offsets_past_31_bits():
    """Matrices of more than 2^31 elements: the last rows are right, and the
    rows in front of them too."""
    mt = _mt()
    d = 8192
    T = (1 << 31) // d + 1001
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    at = [0, 1, T - 900, T - 2, T - 1]
    x[at] = torch.randn(len(at), d, generator=g, device=DEV).bfloat16()
    y = torch.empty_like(x)
    mt.mt_k_dropout(x.data_ptr(), 1, d, mt.mt_dropout(0.5, 3, 4), 0, 0, y.data_ptr(), 1, d, T, d, stream())
    for t in at:
        keep = block.dropout_keep(1, d, 0.5, 3, 4, t)[0]
        assert np.array_equal(np64(y[t]), np.where(keep, 2 * np64(x[t]), 0.0)), t
    one, zero = torch.ones(d, dtype=torch.bfloat16, device=DEV), torch.zeros(d, dtype=torch.bfloat16, device=DEV)
    mt.mt_k_layernorm_fwd(x.data_ptr(), 1, d, one.data_ptr(), zero.data_ptr(), y.data_ptr(), 1, d, 0, 0, T, d, 1e-5, stream())
    want = block.layernorm_fwd(np64(x[at]), 1.0, 0.0, 1e-5)[0]
    within(np64(y[at]), want, 2.0 ** -8 * np.abs(want) + 2 * CHAIN * (2 + np.abs(want)))
    # a thin product with as many rows: C and Z past 2^31 elements
    K = 16
    A, W = x.view(-1)[:T * K].view(T, K), torch.randn(d, K, generator=g, device=DEV).bfloat16()
    A.zero_()
    A[at] = torch.randn(len(at), K, generator=g, device=DEV).bfloat16()
    C = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    mt.mt_k_linear_fwd(A.data_ptr(), K, W.data_ptr(), K, 0, 0, None, 0, 0, y.data_ptr(), d, C.data_ptr(), 1, d, T, d, K, stream())
    a, w = np64(A[at]), np64(W)
    within(np64(C[at]), a @ w.T, 2.0 ** -8 * np.abs(a @ w.T) + product_error(a, w, K))
    assert torch.equal(C[at], y[at]) and not C[T - 899:T - 2].any()


# ---------------------------------------------------------------------------
# The block
# ---------------------------------------------------------------------------
def test_block_forward_and_backward_captured_and_replayed():
    """out = x + drop2(W2 drop1(gelu(W1 LN(x) + b1)) + b2), forward and every
    gradient, run eagerly and as a captured graph with the masks moved on by the
    device offset between replays; against fp64 on the same bf16 weights.

    Tolerance (relative L2): the kernels round LN's output, Z, the hidden
    activations, dZ2, dZ1 and the input gradient to bf16, each by at most 2^-8 of
    a value; five such roundings in a row on the longest path (dW1 and dx), so
    5 x 2^-8 = 2 % bounds every gradient."""
    mt = _mt()
    T, d, F, p = 333, 264, 520, 0.2
    rng = np.random.default_rng(9)
    bf = torch.bfloat16
    x = torch.tensor(rng.normal(size=(T, d)) + 0.5, dtype=torch.float32, device=DEV)
    dout = torch.tensor(rng.normal(size=(T, d)), dtype=torch.float32, device=DEV)
    g, b = vec(1 + 0.1 * rng.normal(size=d), bf), vec(0.1 * rng.normal(size=d), bf)
    W1, b1 = vec(rng.normal(size=(F, d)) / d ** 0.5, bf), vec(0.3 * rng.normal(size=F), bf)
    W2, b2 = vec(rng.normal(size=(d, F)) / F ** 0.5, bf), vec(0.3 * rng.normal(size=d), bf)
    e = lambda *s, t=torch.float32: torch.full(s, float("nan"), dtype=t, device=DEV)  # noqa: E731
    n, mean, rstd, Z, h, out = e(T, d, t=bf), e(T), e(T), e(T, F, t=bf), e(T, F, t=bf), e(T, d)
    dZ2, db2, dZ1, db1, dn, dx, dg, db, dW1, dW2 = e(T, d, t=bf), e(d), e(T, F, t=bf), e(F), e(T, d), e(T, d), e(d), e(d), \
        e(F, d), e(d, F)
    parts = [e(mt.mt_k_act_bwd_partial_floats(T, d)), e(mt.mt_k_linear_bwd_act_partial_floats(T, F)),
             e(mt.mt_k_layernorm_bwd_partial_floats(T, d))]
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    drop1, drop2 = mt.mt_dropout(p, 77, 0, step.data_ptr()), mt.mt_dropout(p, 77, 1 << 32, step.data_ptr())
    P = lambda t: t.data_ptr()  # noqa: E731

    def run():
        st = stream()
        mt.mt_k_layernorm_fwd(P(x), 0, d, P(g), P(b), P(n), 1, d, P(mean), P(rstd), T, d, 1e-5, st)
        mt.mt_k_linear_fwd(P(n), d, P(W1), d, P(b1), mt.MT_ACT_GELU, drop1, 0, 0, P(Z), F, P(h), 1, F, T, F, d, st)
        mt.mt_k_linear_fwd(P(h), F, P(W2), F, P(b2), 0, drop2, P(x), d, 0, 0, P(out), 0, d, T, d, F, st)
        mt.mt_k_act_bwd(P(dout), 0, d, 0, 0, 0, drop2, P(dZ2), d, P(parts[0]), P(db2), T, d, st)
        mt.mt_k_linear_bwd_act(P(dZ2), d, P(W2), F, P(Z), F, mt.MT_ACT_GELU, drop1, P(dZ1), F, P(parts[1]), P(db1), T, F, d,
                               st)
        mt.mt_k_gemm_bf16(P(dZ2), d, 1, P(h), F, 1, P(dW2), F, mt.GEMM_OUT_F32, 0, 0, d, F, T, st)
        mt.mt_k_gemm_bf16(P(dZ1), F, 1, P(n), d, 1, P(dW1), d, mt.GEMM_OUT_F32, 0, 0, F, d, T, st)
        mt.mt_k_gemm_bf16(P(dZ1), F, 0, P(W1), d, 1, P(dn), d, mt.GEMM_OUT_F32, 0, 0, T, d, F, st)
        mt.mt_k_layernorm_bwd(P(x), 0, d, P(g), P(mean), P(rstd), P(dn), 0, d, P(dout), d, P(dx), 0, d, P(parts[2]), P(dg),
                              P(db), T, d, st)

    def check(offset):
        X, D = np64(x), np64(dout)
        k1, k2 = block.dropout_keep(T, F, p, 77, offset), block.dropout_keep(T, d, p, 77, (1 << 32) + offset)
        wn, wm, wr = block.layernorm_fwd(X, np64(g), np64(b), 1e-5)
        wh, wz = block.linear_fwd(wn, np64(W1), np64(b1), "gelu", p, k1)
        wout, _ = block.linear_fwd(wh, np64(W2), np64(b2), "none", p, k2, X)
        wdz2, wdb2 = block.act_bwd(D, 0 * D, "none", p, k2)
        wdz1, wdb1 = block.linear_bwd_act(wdz2, np64(W2), wz, "gelu", p, k1)
        wdx, wdg, wdb = block.layernorm_bwd(X, np64(g), wm, wr, wdz1 @ np64(W1))
        for name, got, want in [("out", out, wout), ("db2", db2, wdb2), ("db1", db1, wdb1), ("dW2", dW2, wdz2.T @ wh),
                                ("dW1", dW1, wdz1.T @ wn), ("dx", dx, wdx + D), ("dg", dg, wdg), ("db", db, wdb)]:
            off = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
            assert off <= 5 * 2.0 ** -8, (name, off)

    run()
    check(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        step.add_(2)
    for k in range(2):
        for t in (out, dx, dW1, dW2, dg, db, db1, db2, n, Z, h, dZ1, dZ2):
            t.fill_(float("nan"))
        graph.replay()
        check(2 * k)
    del graph


def test_gated_block_gradients():
    """y = (silu(x Wg^T) (x Wu^T)) Wd^T and every gradient with the library's
    products around the two fused kernels, against fp64 on the same weights.
    At most four bf16 roundings in a row (gate and up, dgate and dup, h, dx):
    4 x 2^-8 relative L2."""
    mt = _mt()
    T, d, F = 300, 264, 712
    rng = np.random.default_rng(4)
    bf = torch.bfloat16
    x, dy = vec(rng.normal(size=(T, d)), bf), vec(rng.normal(size=(T, d)), bf)
    Wgu, Wd = vec(rng.normal(size=(2 * F, d)) / d ** 0.5, bf), vec(rng.normal(size=(d, F)) / F ** 0.5, bf)
    e = lambda *s, t=torch.float32: torch.full(s, float("nan"), dtype=t, device=DEV)  # noqa: E731
    gu, h, h2, dgu, y, dx, dWgu, dWd = e(T, 2 * F, t=bf), e(T, F, t=bf), e(T, F, t=bf), e(T, 2 * F, t=bf), e(T, d), e(T, d), \
        e(2 * F, d), e(d, F)
    P, st = lambda t: t.data_ptr(), stream()
    mt.mt_k_gated_ffn_fwd(P(x), d, P(Wgu), d, mt.MT_ACT_SILU, P(gu), 2 * F, P(h), F, T, F, d, st)
    mt.mt_k_gemm_bf16(P(h), F, 0, P(Wd), F, 0, P(y), d, mt.GEMM_OUT_F32, 0, 0, T, d, F, st)
    mt.mt_k_gated_ffn_bwd(P(dy), d, P(Wd), F, P(gu), 2 * F, mt.MT_ACT_SILU, P(dgu), 2 * F, P(h2), F, T, F, d, st)
    mt.mt_k_gemm_bf16(P(dgu), 2 * F, 0, P(Wgu), d, 1, P(dx), d, mt.GEMM_OUT_F32, 0, 0, T, d, 2 * F, st)
    mt.mt_k_gemm_bf16(P(dgu), 2 * F, 1, P(x), d, 1, P(dWgu), d, mt.GEMM_OUT_F32, 0, 0, 2 * F, d, T, st)
    mt.mt_k_gemm_bf16(P(dy), d, 1, P(h2), F, 1, P(dWd), F, mt.GEMM_OUT_F32, 0, 0, d, F, T, st)
    X, D, W, V = np64(x), np64(dy), np64(Wgu), np64(Wd)
    wh, g, u = block.gated_fwd(X, W[:F], W[F:], "silu")
    dg, du, _ = block.gated_bwd(D, V, g, u, "silu")
    wdgu = np.concatenate([dg, du], axis=1)
    for name, got, want in [("y", y, wh @ V.T), ("dx", dx, wdgu @ W), ("dWgu", dWgu, wdgu.T @ X), ("dWd", dWd, D.T @ wh)]:
        off = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
        assert off <= 4 * 2.0 ** -8, (name, off)
