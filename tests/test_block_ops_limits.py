"""Limits of the layer-norm, dropout, linear and gated feed-forward calls that
the header states, each at the border: what lies behind it is refused on the
host, before any device work (no GPU here)."""
import pytest

from test_block_ops_refusals import CONFIG, P, _mt, base, refused

I64_MAX = (1 << 63) - 1


@pytest.mark.parametrize("row0", [I64_MAX, I64_MAX - 7, I64_MAX - 8, 1 << 62, (1 << 32) - 7])
@pytest.mark.parametrize("name", ["mt_k_dropout", "mt_k_linear_fwd", "mt_k_linear_bwd_act", "mt_k_act_bwd"])
def test_rows_of_the_mask_behind_its_counter_are_refused(name, row0):
    """row0 + 8 rows must stay within 2^32, also where the sum passes 2^63."""
    refused(name, drop=_mt().mt_dropout(0.1, 1, 2, 0, row0))


def test_the_last_rows_of_the_mask_are_accepted():
    """An empty matrix of 8 rows: the arguments are checked, nothing is launched."""
    mt = _mt()
    mt.mt_k_dropout(0, 0, 0, mt.mt_dropout(0.1, 1, 2, 0, (1 << 32) - 8), 0, 0, 0, 0, 0, 8, 0)
    with pytest.raises(mt.MTError):
        mt.mt_k_dropout(0, 0, 0, mt.mt_dropout(0.1, 1, 2, 0, I64_MAX - 3), 0, 0, 0, 0, 0, 8, 0)


@pytest.mark.parametrize("name,vectors", [
    ("mt_k_layernorm_fwd", ("mean", "rstd")),
    ("mt_k_layernorm_bwd", ("mean", "rstd", "part", "dg", "db")),
    ("mt_k_linear_fwd", ("dev_err",)),
    ("mt_k_linear_bwd_act", ("part", "db", "dev_err")),
    ("mt_k_act_bwd", ("part", "db")),
    ("mt_k_gated_ffn_fwd", ("dev_err",)),
    ("mt_k_gated_ffn_bwd", ("dev_err",)),
])
def test_vectors_off_their_elements_boundary_are_refused(name, vectors):
    """fp32 vectors and dev_err between two multiples of 4 bytes, which a kernel could not read or write."""
    for v in vectors:
        for off in (1, 2):
            refused(name, **{v: P() + off})


DEEPEST = 1 << 20


@pytest.mark.parametrize("name", ["mt_k_linear_fwd", "mt_k_linear_bwd_act", "mt_k_gated_ffn_fwd", "mt_k_gated_ffn_bwd"])
@pytest.mark.parametrize("K", [DEEPEST + 1, 1 << 25, 1 << 30])
def test_depths_behind_the_largest_are_refused(name, K):
    """A product deeper than 2^20 would lose more than its output type rounds, and near 2^28 outlast its waits."""
    pitches = {k: v for k, v in dict(lda=K, ldw=K, lddy=K, ldx=K).items() if k in base(name)}
    if name in ("mt_k_linear_bwd_act", "mt_k_gated_ffn_bwd"):
        del pitches["ldw"]  # W [K, N]
    refused(name, CONFIG, K=K, **{k: (v + 7) // 8 * 8 for k, v in pitches.items()})


def test_empty_products_of_any_depth_succeed():
    mt = _mt()
    mt.mt_k_linear_fwd(0, 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 0, 0, 0, 16, 1 << 30)
    mt.mt_k_gated_ffn_fwd(0, 0, 0, 0, 4, 0, 0, 0, 0, 0, 16, 1 << 30)
