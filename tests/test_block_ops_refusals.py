"""What the layer-norm, dropout, linear and gated feed-forward calls refuse:
every bad argument is found on the host, before any device work (no GPU here),
and empty calls succeed without touching a pointer."""
import numpy as np
import pytest

ARG, CONFIG = -1, -2


def _mt():
    from host_memory_streamed_layer_b200 import mt
    return mt


def _buf():
    from host_memory_streamed_layer_b200 import arena
    return arena.aligned_empty(1 << 16)


BUF = None


def P():
    global BUF
    if BUF is None:
        BUF = _buf()
    return BUF.ctypes.data


def base(name):
    """A call that the library would launch, as keyword arguments (8 x 16, K 24)."""
    p, d = P(), _mt().mt_dropout(0.1, 1, 2)
    return {
        "mt_k_layernorm_fwd": dict(x=p, x_type=0, ldx=16, g=p, b=p, y=p, y_type=1, ldy=16, mean=p, rstd=p, T=8, d=16, eps=1e-5),
        "mt_k_layernorm_bwd": dict(x=p, x_type=0, ldx=16, g=p, mean=p, rstd=p, dy=p, dy_type=1, lddy=16, dres=p, lddres=16, dx=p,
                                   dx_bf16=p, lddx=16, part=p, dg=p, db=p, T=8, d=16),
        "mt_k_dropout": dict(x=p, x_type=0, ldx=16, drop=d, res=p, ldr=16, y=p, y_type=1, ldy=16, T=8, d=16),
        "mt_k_linear_fwd": dict(A=p, lda=24, W=p, ldw=24, bias=p, act=2, drop=d, R=p, ldr=16, Z=p, ldz=16, C=p, out_type=1,
                                ldc=16, M=8, N=16, K=24),
        "mt_k_linear_bwd_act": dict(dY=p, lddy=24, W=p, ldw=16, Z=p, ldz=16, act=2, drop=d, dZ=p, lddz=16, part=p, db=p, M=8,
                                    N=16, K=24),
        "mt_k_act_bwd": dict(dC=p, dc_type=0, lddc=16, Z=p, ldz=16, act=2, drop=d, dZ=p, lddz=16, part=p, db=p, M=8, N=16),
        "mt_k_gated_ffn_fwd": dict(x=p, ldx=24, Wgu=p, ldw=24, act=4, gu=p, ldgu=32, h=p, ldh=16, M=8, F=16, K=24),
        "mt_k_gated_ffn_bwd": dict(dy=p, lddy=24, Wd=p, ldw=16, gu=p, ldgu=32, act=4, dgu=p, lddgu=32, h=p, ldh=16, M=8, F=16,
                                   K=24),
    }[name]


BAD = [
    *[("mt_k_layernorm_fwd", c) for c in (
        dict(x=0), dict(g=0), dict(y=0), dict(x_type=2), dict(y_type=-1), dict(T=-1), dict(d=0), dict(d=-4), dict(eps=-1.0),
        dict(eps=float("nan")), dict(ldx=12), dict(ldx=18), dict(ldy=20), dict(ldy=8), dict(T=(1 << 30) + 1))],
    *[("mt_k_layernorm_bwd", c) for c in (
        dict(x=0), dict(g=0), dict(mean=0), dict(rstd=0), dict(dy=0), dict(dx=0), dict(part=0), dict(dg=0), dict(dy_type=3),
        dict(lddres=8), dict(lddx=8), dict(lddx=20), dict(lddy=20), dict(x_type=1), dict(T=-1), dict(T=0, dg=0))],
    *[("mt_k_dropout", c) for c in (
        dict(x=0), dict(y=0), dict(x_type=2), dict(ldr=8), dict(ldr=20), dict(ldx=18), dict(T=-2), dict(d=-1),
        dict(d=(1 << 30) + 1))],
    *[("mt_k_linear_fwd", c) for c in (
        dict(A=0), dict(W=0), dict(C=0), dict(act=5), dict(act=-1), dict(out_type=2), dict(K=0), dict(K=-1), dict(M=-1),
        dict(lda=16), dict(lda=28), dict(ldw=20), dict(ldr=12), dict(ldz=8), dict(ldc=8), dict(ldc=20), dict(K=25))],
    *[("mt_k_linear_bwd_act", c) for c in (
        dict(dY=0), dict(W=0), dict(dZ=0), dict(Z=0), dict(part=0), dict(act=9), dict(ldw=8), dict(lddy=16), dict(lddz=20),
        dict(ldz=8), dict(K=0), dict(N=-1))],
    *[("mt_k_act_bwd", c) for c in (
        dict(dC=0), dict(dZ=0), dict(Z=0), dict(part=0), dict(act=9), dict(dc_type=2), dict(lddc=12), dict(lddz=20), dict(ldz=8),
        dict(M=-1))],
    *[("mt_k_gated_ffn_fwd", c) for c in (
        dict(x=0), dict(Wgu=0), dict(h=0), dict(F=12), dict(F=-8), dict(K=0), dict(act=7), dict(ldgu=16), dict(ldgu=36),
        dict(ldh=8), dict(ldx=16), dict(ldw=20))],
    *[("mt_k_gated_ffn_bwd", c) for c in (
        dict(dy=0), dict(Wd=0), dict(gu=0), dict(dgu=0), dict(F=12), dict(K=0), dict(act=-2), dict(ldgu=24), dict(lddgu=16),
        dict(ldh=8), dict(ldw=8), dict(lddy=16))],
]


def refused(name, code=ARG, **change):
    mt = _mt()
    with pytest.raises(mt.MTError) as e:
        getattr(mt, name)(**{**base(name), **change})
    assert e.value.code == code, (name, change, e.value.code)


@pytest.mark.parametrize("name,change", BAD)
def test_bad_arguments_are_refused(name, change):
    refused(name, **change)


@pytest.mark.parametrize("name", ["mt_k_layernorm_fwd", "mt_k_layernorm_bwd", "mt_k_dropout", "mt_k_linear_fwd",
                                  "mt_k_linear_bwd_act", "mt_k_act_bwd", "mt_k_gated_ffn_fwd", "mt_k_gated_ffn_bwd"])
def test_misaligned_matrices_are_refused(name):
    """Every 16-byte aligned operand, one at a time."""
    p = P()
    small = {"mean", "rstd", "part", "dg", "db"}
    for k, v in base(name).items():
        if v == p and k not in small:
            refused(name, **{k: p + 8})


def test_rows_wider_than_the_layer_norm_holds():
    for name in ("mt_k_layernorm_fwd", "mt_k_layernorm_bwd"):
        refused(name, CONFIG, d=8193)
    mt = _mt()
    assert mt.mt_k_layernorm_bwd_partial_floats(8, 8193) == 0 and mt.mt_k_layernorm_bwd_partial_floats(-1, 8) == 0
    assert mt.mt_k_layernorm_bwd_partial_floats(8, 8192) >= 2 * 8192
    assert mt.mt_k_act_bwd_partial_floats(-1, 8) == 0 and mt.mt_k_linear_bwd_act_partial_floats(8, -1) == 0


@pytest.mark.parametrize("drop", [dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(p=2.0), dict(row0=-1),
                                  dict(row0=(1 << 32) - 7), dict(offset_dev=12)])
@pytest.mark.parametrize("name", ["mt_k_dropout", "mt_k_linear_fwd", "mt_k_linear_bwd_act", "mt_k_act_bwd"])
def test_bad_dropout_is_refused(name, drop):
    refused(name, drop=_mt().mt_dropout(**{**dict(p=0.1, seed=1, offset=2), **drop}))


def test_empty_calls_touch_nothing():
    mt = _mt()
    mt.mt_k_layernorm_fwd(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 16, 1e-5)
    mt.mt_k_dropout(0, 0, 0, None, 0, 0, 0, 0, 0, 0, 16)
    mt.mt_k_dropout(0, 0, 0, None, 0, 0, 0, 0, 0, 8, 0)
    mt.mt_k_linear_fwd(0, 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 0, 0, 0, 16, 24)
    mt.mt_k_linear_fwd(0, 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 0, 0, 8, 0, 24)
    mt.mt_k_linear_bwd_act(0, 0, 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 16, 24)
    mt.mt_k_act_bwd(0, 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 16)
    mt.mt_k_gated_ffn_fwd(0, 0, 0, 0, 4, 0, 0, 0, 0, 0, 16, 24)
    mt.mt_k_gated_ffn_bwd(0, 0, 0, 0, 0, 0, 4, 0, 0, 0, 0, 8, 0, 24)


def test_dropout_structure_matches_the_header():
    """p, then four 8-byte members, in the C layout."""
    mt = _mt()
    import ctypes
    assert ctypes.sizeof(mt.mt_dropout) == 40
    assert [getattr(mt.mt_dropout, n).offset for n in ("p", "seed", "offset", "offset_dev", "row0")] == [0, 8, 16, 24, 32]
    assert np.float32(mt.mt_dropout(0.1).p) == np.float32(0.1)
