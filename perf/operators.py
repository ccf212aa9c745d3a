"""The operators of a decoder block with layer norms, biased linear layers, dropout and a gated feed-forward part, as
cases to time and to compare: each in plain torch (32-bit, rounded once at the end), in 64 bits, and by this
library's kernels.

Weights and activations are bf16, the residual stream and the gradients of vectors fp32 (bf16 where a case says so),
as in the rest of the library. Sizes are those of the workloads of `synth` (widths 2048, 4096 and 5120, hidden widths
5504, 11008, 13824 and the experts' 1408, 1 to 16384 tokens) and ragged ones between them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
P_DROP = 0.1
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token through a layer norm: nothing but latency
        dict(name="ln_fwd_token", op="ln_fwd", T=1, d=5120, x="f32", y="bf16"),
        # a block's layer norm on the fp32 residual stream of 8 x 2048 tokens
        dict(name="ln_fwd", op="ln_fwd", T=16384, d=2048, x="f32", y="bf16"),
        # its gradient, with the residual's gradient added and a bf16 copy for the product before it
        dict(name="ln_bwd", op="ln_bwd", T=16384, d=2048, x="f32", y="f32"),
        # a few sequences through a small biased layer: launch latency and half-empty tiles
        dict(name="linear_small", op="linear", M=256, N=688, K=256, act="gelu", r="none", out="bf16", z=True, p=0.0),
        # the first layer of a feed-forward part in training, its pre-activation kept for the backward pass
        dict(name="linear_gelu", op="linear", M=16384, N=5504, K=2048, act="gelu", r="none", out="bf16", z=True, p=0.0),
        # the second layer: bias, dropout and the residual stream in one pass; a batch that fills no tile
        dict(name="linear_residual", op="linear", M=16333, N=2048, K=5504, act="none", r="add", out="f32", z=False, p=P_DROP),
        # back through the second layer into the first one's pre-activation, with the bias gradient
        dict(name="linear_dact", op="dact", M=16384, N=5504, K=2048, act="gelu", p=0.0),
        # dropout of a sublayer's bf16 output onto the fp32 residual stream of 2 x 4096 tokens
        dict(name="dropout_add", op="dropout", T=8192, d=5120, x="bf16", r="add", y="f32", p=P_DROP),
        # back through dropout to the sublayer's output, with the bias gradient that starts the backward pass
        dict(name="dropout_bwd", op="act_bwd", M=8191, N=5120, act="none", dc="f32", p=P_DROP),
        # the gated feed-forward part of 2 x 4096 tokens at width 5120, gate and up kept for the backward pass
        dict(name="gated", op="gated", M=8192, F=13824, K=5120, act="silu", keep=True),
        # the same part of a smaller block for a handful of tokens: bound by reading the weights
        dict(name="gated_few", op="gated", M=13, F=11008, K=4096, act="silu", keep=False),
        # back through the down projection of an expert's share of the tokens
        dict(name="gated_bwd", op="gated_bwd", M=4099, F=1408, K=2048, act="silu"),
    ]


def _size(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))
    return max(step, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "linear", "dact", "dropout", "act_bwd", "gated", "gated_bwd"])
    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    p = rng.choice([0.0, 0.0625, P_DROP, 0.5])
    act = rng.choice(ACTS)
    if op in ("ln_fwd", "ln_bwd"):
        return dict(op=op, T=_size(rng, 1, 16384), d=_size(rng, 8, 8192), x=t(), y=t())
    if op == "linear":
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 8, 5504), K=_size(rng, 8, 5504), act=act,
                    r=rng.choice(["none", "add"]), out=t(), z=rng.random() < 0.5, p=p)
    if op == "dact":
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 8, 5504), K=_size(rng, 8, 5504), act=act, p=p)
    if op == "dropout":
        return dict(op=op, T=_size(rng, 1, 16384), d=_size(rng, 8, 8192), x=t(), r=rng.choice(["none", "add"]), y=t(),
                    p=rng.choice([0.0625, P_DROP, 0.5]))
    if op == "act_bwd":
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 8, 8192), act=act, dc=t(), p=p)
    act = rng.choice(ACTS[1:])
    d = dict(op=op, M=_size(rng, 1, 8192), F=_size(rng, 8, 11008, 8), K=_size(rng, 8, 5120), act=act)
    return dict(d, keep=rng.random() < 0.5) if op == "gated" else d


# ---------------------------------------------------------------------------
# Inputs: what a program has in hand, rows padded to a pitch of 16 bytes
# ---------------------------------------------------------------------------
_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _pitch(n):
    return (n + 7) // 8 * 8


def _empty(rows, cols, dtype):
    return torch.zeros(rows, _pitch(cols), dtype=dtype, device=DEV)[:, :cols]


def _randn(g, rows, cols, dtype, std=1.0):
    out = _empty(rows, cols, dtype)
    out.copy_(torch.randn(rows, cols, generator=g, device=DEV).mul_(std))
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    rn = lambda r, c, t, std=1.0: _randn(g, r, c, _TYPE[t], std)  # noqa: E731
    vec = lambda n, mean, std: (mean + std * torch.randn(n, generator=g, device=DEV)).bfloat16()  # noqa: E731
    s = dict(case=dict(case), rng=(int(seed) * 2654435761 % (1 << 62), int(seed) % 1000 + (1 << 33)))
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, d = case["T"], case["d"]
        # a residual stream: features of unlike sizes, a few of them large, around means of their own
        x = torch.randn(T, d, generator=g, device=DEV) * (0.5 + torch.rand(d, generator=g, device=DEV))
        x += 0.3 * torch.randn(d, generator=g, device=DEV)
        x[:, :: 97] *= 8
        s["x"] = _empty(T, d, _TYPE[case["x"]])
        s["x"].copy_(x)
        s["g"], s["b"] = vec(d, 1.0, 0.1), vec(d, 0.0, 0.1)
        s["mean"], s["rstd"] = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
        if op == "ln_fwd":
            s["y"] = _empty(T, d, _TYPE[case["y"]])
            return s
        x = s["x"].float()
        s["mean"].copy_(x.mean(1))
        s["rstd"].copy_(torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS))
        s["dy"], s["dres"] = rn(T, d, case["y"]), rn(T, d, case["x"])
        s["dx"] = _empty(T, d, _TYPE[case["x"]])
        s["dxb"] = _empty(T, d, torch.bfloat16) if case["x"] == "f32" else None
        s["dg"], s["db"] = torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["W"] = rn(M, K, "bf16"), rn(N, K, "bf16", 1 / math.sqrt(K))
        s["bias"] = vec(N, 0.0, 0.3)
        s["R"] = rn(M, N, case["out"]) if case["r"] == "add" else None
        s["C"] = _empty(M, N, _TYPE[case["out"]])
        s["Z"] = _empty(M, N, torch.bfloat16) if case["z"] else None
    elif op == "dact":
        M, N, K = case["M"], case["N"], case["K"]
        s["dY"], s["W"] = rn(M, K, "bf16"), rn(K, N, "bf16", 1 / math.sqrt(K))
        s["Z"] = rn(M, N, "bf16", 1.2)
        s["dZ"], s["db"] = _empty(M, N, torch.bfloat16), torch.zeros(N, device=DEV)
    elif op == "dropout":
        T, d = case["T"], case["d"]
        s["x"] = rn(T, d, case["x"])
        s["R"] = rn(T, d, case["y"]) if case["r"] == "add" else None
        s["y"] = _empty(T, d, _TYPE[case["y"]])
    elif op == "act_bwd":
        M, N = case["M"], case["N"]
        s["dC"] = rn(M, N, case["dc"])
        s["Z"] = rn(M, N, "bf16", 1.2) if case["act"] != "none" else None
        s["dZ"], s["db"] = _empty(M, N, torch.bfloat16), torch.zeros(N, device=DEV)
    else:
        M, F, K = case["M"], case["F"], case["K"]
        s["h"] = _empty(M, F, torch.bfloat16)
        if op == "gated":
            s["x"], s["W"] = rn(M, K, "bf16"), rn(2 * F, K, "bf16", 1 / math.sqrt(K))
            s["gu"] = _empty(M, 2 * F, torch.bfloat16) if case["keep"] else None
        else:
            s["dy"], s["W"] = rn(M, K, "bf16"), rn(K, F, "bf16", 1 / math.sqrt(K))
            s["gu"] = rn(M, 2 * F, "bf16", 1.2)
            s["dgu"] = _empty(M, 2 * F, torch.bfloat16)
    if op in ("ln_bwd", "dact", "act_bwd"):
        # scratch for the column sums: a program sizes it with the library's own function, which stays below this
        rows, cols = (case["T"], case["d"]) if op == "ln_bwd" else (case["M"], case["N"])
        s["part"] = torch.empty(2 * _pitch(cols) * (rows // 32 + 1024), device=DEV)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


def _words(rows, cols, seed, offset):
    """The 32 random bits of each element: Philox4x32 with ten rounds (Salmon et al., "Parallel random numbers: as easy
    as 1, 2, 3"), counter (column / 4, row, offset), key seed; an element takes word column % 4."""
    low = 0xFFFFFFFF
    c = [torch.arange((cols + 3) // 4, device=DEV)[None, :], torch.arange(rows, device=DEV)[:, None],
         torch.tensor(offset & low, device=DEV), torch.tensor(offset >> 32, device=DEV)]
    key = [seed & low, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & low) ^ c[1] ^ key[0], b & low, ((a >> 32) & low) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    return torch.stack(torch.broadcast_tensors(*c), 2).reshape(rows, -1)[:, :cols]


def _drop(v, p, rng):
    """Where an element is dropped, zero whatever it holds; elsewhere v / (1 - p)."""
    if p == 0:
        return v
    p = float(np.float32(p))
    kept = _words(*v.shape, *rng) >= round(p * 2**32)
    return torch.where(kept, v * (1 / (1 - p)), torch.zeros_like(v))


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        y = (x - mean) * rstd * s["g"].float() + s["b"].float()
        return dict(y=y.to(_TYPE[c["y"]]), mean=mean[:, 0], rstd=rstd[:, 0])
    if op == "ln_bwd":
        rstd = s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        dy = s["dy"].float()
        dyg = dy * s["g"].float()
        dx = rstd * (dyg - dyg.mean(1, keepdim=True) - xhat * (dyg * xhat).mean(1, keepdim=True)) + s["dres"].float()
        r = dict(dx=dx.to(_TYPE[c["x"]]), dg=(dy * xhat).sum(0), db=dy.sum(0))
        return dict(r, dxb=dx.bfloat16()) if c["x"] == "f32" else r
    if op == "linear":
        z = s["A"].float() @ s["W"].float().T + s["bias"].float()
        y = _drop(_act(z, c["act"]), c["p"], s["rng"])
        y = y if s["R"] is None else s["R"].float() + y
        r = dict(c=y.to(_TYPE[c["out"]]))
        return dict(r, z=z.bfloat16()) if c["z"] else r
    if op == "dact":
        dz = _drop(s["dY"].float() @ s["W"].float(), c["p"], s["rng"]) * _act_grad(s["Z"].float(), c["act"])
        return dict(dz=dz.bfloat16(), db=dz.sum(0))
    if op == "dropout":
        y = _drop(s["x"].float(), c["p"], s["rng"])
        y = y if s["R"] is None else s["R"].float() + y
        return dict(y=y.to(_TYPE[c["y"]]))
    if op == "act_bwd":
        dz = _drop(s["dC"].float(), c["p"], s["rng"])
        dz = dz if s["Z"] is None else dz * _act_grad(s["Z"].float(), c["act"])
        return dict(dz=dz.bfloat16(), db=dz.sum(0))
    F = c["F"]
    if op == "gated":
        gu = s["x"].float() @ s["W"].float().T
        h = (_act(gu[:, :F], c["act"]) * gu[:, F:]).bfloat16()
        return dict(h=h, gu=gu.bfloat16()) if c["keep"] else dict(h=h)
    dh = s["dy"].float() @ s["W"].float()
    g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
    a = _act(g, c["act"])
    dgu = torch.cat([dh * u * _act_grad(g, c["act"]), dh * a], 1)
    return dict(dgu=dgu.bfloat16(), h=(a * u).bfloat16())


# ---------------------------------------------------------------------------
# The library's kernels
# ---------------------------------------------------------------------------
def _at(t):
    return 0 if t is None else t.data_ptr()


def _ld(t):
    return 0 if t is None else t.stride(0)


def _own(s):
    from host_memory_streamed_layer_b200 import mt
    c, op = s["case"], s["case"]["op"]
    st = torch.cuda.current_stream().cuda_stream
    kind = {"f32": mt.MT_F32, "bf16": mt.MT_BF16}
    act = getattr(mt, "MT_ACT_" + c["act"].upper()) if "act" in c else 0
    drop = mt.mt_dropout(c["p"], *s["rng"]) if c.get("p") else None
    if op == "ln_fwd":
        mt.mt_k_layernorm_fwd(_at(s["x"]), kind[c["x"]], _ld(s["x"]), _at(s["g"]), _at(s["b"]), _at(s["y"]), kind[c["y"]],
                              _ld(s["y"]), _at(s["mean"]), _at(s["rstd"]), c["T"], c["d"], EPS, st)
        return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    if op == "ln_bwd":
        mt.mt_k_layernorm_bwd(_at(s["x"]), kind[c["x"]], _ld(s["x"]), _at(s["g"]), _at(s["mean"]), _at(s["rstd"]),
                              _at(s["dy"]), kind[c["y"]], _ld(s["dy"]), _at(s["dres"]), _ld(s["dres"]), _at(s["dx"]),
                              _at(s["dxb"]), _ld(s["dx"]), _at(s["part"]), _at(s["dg"]), _at(s["db"]), c["T"], c["d"], st)
        r = dict(dx=s["dx"], dg=s["dg"], db=s["db"])
        return r if s["dxb"] is None else dict(r, dxb=s["dxb"])
    if op == "linear":
        mt.mt_k_linear_fwd(_at(s["A"]), _ld(s["A"]), _at(s["W"]), _ld(s["W"]), _at(s["bias"]), act, drop, _at(s["R"]),
                           _ld(s["R"]), _at(s["Z"]), _ld(s["Z"]), _at(s["C"]), kind[c["out"]], _ld(s["C"]), c["M"], c["N"],
                           c["K"], st)
        return dict(c=s["C"]) if s["Z"] is None else dict(c=s["C"], z=s["Z"])
    if op == "dact":
        mt.mt_k_linear_bwd_act(_at(s["dY"]), _ld(s["dY"]), _at(s["W"]), _ld(s["W"]), _at(s["Z"]), _ld(s["Z"]), act, drop,
                               _at(s["dZ"]), _ld(s["dZ"]), _at(s["part"]), _at(s["db"]), c["M"], c["N"], c["K"], st)
        return dict(dz=s["dZ"], db=s["db"])
    if op == "dropout":
        mt.mt_k_dropout(_at(s["x"]), kind[c["x"]], _ld(s["x"]), drop, _at(s["R"]), _ld(s["R"]), _at(s["y"]), kind[c["y"]],
                        _ld(s["y"]), c["T"], c["d"], st)
        return dict(y=s["y"])
    if op == "act_bwd":
        mt.mt_k_act_bwd(_at(s["dC"]), kind[c["dc"]], _ld(s["dC"]), _at(s["Z"]), _ld(s["Z"]), act, drop, _at(s["dZ"]),
                        _ld(s["dZ"]), _at(s["part"]), _at(s["db"]), c["M"], c["N"], st)
        return dict(dz=s["dZ"], db=s["db"])
    if op == "gated":
        mt.mt_k_gated_ffn_fwd(_at(s["x"]), _ld(s["x"]), _at(s["W"]), _ld(s["W"]), act, _at(s["gu"]), _ld(s["gu"]), _at(s["h"]),
                              _ld(s["h"]), c["M"], c["F"], c["K"], st)
        return dict(h=s["h"]) if s["gu"] is None else dict(h=s["h"], gu=s["gu"])
    mt.mt_k_gated_ffn_bwd(_at(s["dy"]), _ld(s["dy"]), _at(s["W"]), _ld(s["W"]), _at(s["gu"]), _ld(s["gu"]), act, _at(s["dgu"]),
                          _ld(s["dgu"]), _at(s["h"]), _ld(s["h"]), c["M"], c["F"], c["K"], st)
    return dict(dgu=s["dgu"], h=s["h"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _kept64(rows, cols, p, rng):
    """The elements that dropout keeps, with each product of two 32-bit words put together from 16-bit halves."""
    def mul(a, m):
        al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
        mid = ah * ml + (al * ml >> 16)
        mid2 = al * mh + (mid & 0xFFFF)
        return ah * mh + (mid >> 16) + (mid2 >> 16), (mid2 & 0xFFFF) << 16 | (al * ml & 0xFFFF)

    seed, offset = rng
    full = lambda v: torch.full((rows, -(-cols // 4)), v, dtype=torch.int64, device=DEV)  # noqa: E731
    x0 = full(0) + torch.arange(-(-cols // 4), device=DEV)
    x1 = full(0) + torch.arange(rows, device=DEV)[:, None]
    x2, x3 = full(offset % 2**32), full(offset // 2**32)
    for i in range(10):
        k0, k1 = (seed + i * 0x9E3779B9) % 2**32, (seed // 2**32 + i * 0xBB67AE85) % 2**32
        h0, l0 = mul(x0, 0xD2511F53)
        h1, l1 = mul(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
    bits = torch.empty(rows, 4 * x0.shape[1], dtype=torch.int64, device=DEV)
    for j, x in enumerate((x0, x1, x2, x3)):
        bits[:, j::4] = x
    return bits[:, :cols].double() >= round(float(np.float32(p)) * 2**32)


def _phi64(z, act):
    """An activation and its slope in 64 bits, by the standard normal or logistic distribution function."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        cdf = torch.sigmoid(k * (z + 0.044715 * z**3))
        return z * cdf, cdf + z * cdf * (1 - cdf) * k * (1 + 0.134145 * z**2)
    cdf = torch.sigmoid(z)
    return z * cdf, cdf + z * cdf * (1 - cdf)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    q = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k != "part"}

    def thin(v):  # v with dropout
        p = case.get("p", 0.0)
        return v if not p else torch.where(_kept64(*v.shape, p, s["rng"]), v / (1 - float(np.float32(p))), 0.0)

    if op == "ln_fwd":
        var, mean = torch.var_mean(q["x"], 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return dict(y=(q["x"] - mean[:, None]) * (rstd[:, None] * q["g"]) + q["b"], mean=mean, rstd=rstd)
    if op == "ln_bwd":
        n = case["d"]
        xc = (q["x"] - q["mean"][:, None]) * q["rstd"][:, None]
        w = q["dy"] * q["g"]
        proj = torch.einsum("td,td->t", w, xc)[:, None] / n
        dx = q["dres"] + q["rstd"][:, None] * (w - w.sum(1, True) / n - proj * xc)
        r = dict(dx=dx, dg=torch.einsum("td,td->d", q["dy"], xc), db=q["dy"].sum(0))
        return dict(r, dxb=dx) if case["x"] == "f32" else r
    if op == "linear":
        z = torch.addmm(q["bias"], q["A"], q["W"].T)
        c = thin(_phi64(z, case["act"])[0]) + q.get("R", 0)
        return dict(c=c, z=z) if case["z"] else dict(c=c)
    if op == "dact":
        dz = _phi64(q["Z"], case["act"])[1] * thin(torch.mm(q["dY"], q["W"]))
        return dict(dz=dz, db=torch.einsum("mn->n", dz))
    if op == "dropout":
        return dict(y=q.get("R", 0) + thin(q["x"]))
    if op == "act_bwd":
        dz = thin(q["dC"])
        if "Z" in q:
            dz = dz * _phi64(q["Z"], case["act"])[1]
        return dict(dz=dz, db=torch.einsum("mn->n", dz))
    if op == "gated":
        g, u = (torch.mm(q["x"], w.T) for w in q["W"].chunk(2))
        h = _phi64(g, case["act"])[0] * u
        return dict(h=h, gu=torch.cat([g, u], 1)) if case["keep"] else dict(h=h)
    g, u = q["gu"].chunk(2, 1)
    a, slope = _phi64(g, case["act"])
    dh = torch.mm(q["dy"], q["W"])
    return dict(dgu=torch.cat([dh * slope * u, dh * a], 1), h=a * u)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, d, x, y = case["T"], case["d"], size[case["x"]], size[case["y"]]
        if op == "ln_fwd":
            return dict(bytes=T * d * (x + y) + 4 * d + 8 * T, flops=8 * T * d)
        return dict(bytes=T * d * (3 * x + y + (2 if x == 4 else 0)) + 10 * d + 8 * T, flops=14 * T * d)
    if op == "linear":
        M, N, K, o = case["M"], case["N"], case["K"], size[case["out"]]
        per = o + (o if case["r"] == "add" else 0) + (2 if case["z"] else 0)
        return dict(bytes=2 * K * (M + N) + 2 * N + M * N * per, flops=2 * M * N * K)
    if op == "dact":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * K * (M + N) + 4 * N + M * N * (2 if case["act"] == "none" else 4), flops=2 * M * N * K)
    if op == "dropout":
        y = size[case["y"]]
        return dict(bytes=case["T"] * case["d"] * (size[case["x"]] + y + (y if case["r"] == "add" else 0)),
                    flops=2 * case["T"] * case["d"])
    if op == "act_bwd":
        M, N = case["M"], case["N"]
        return dict(bytes=M * N * (size[case["dc"]] + 2 + (0 if case["act"] == "none" else 2)) + 4 * N, flops=4 * M * N)
    M, F, K = case["M"], case["F"], case["K"]
    if op == "gated":
        return dict(bytes=2 * K * (M + 2 * F) + M * F * (6 if case["keep"] else 2), flops=4 * M * F * K)
    return dict(bytes=2 * K * (M + F) + 10 * M * F, flops=2 * M * F * K)
