"""Accuracy of the deep products, against fp64."""
import pytest
import torch

from test_gpu_block_ops import DEV, _mt, stream

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def far(got, want):
    return float((got.double() - want).norm())


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
