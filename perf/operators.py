"""Measured cases of the feed-forward operators around the FP8 GEMM: the
root-mean-square norm that adds the residual and leaves in 8 bits, the gated
feed-forward product (gate and up projections, activation and product), and the
matrix product with bias, activation and residual in its epilogue; each forward
and backward.

``own`` selects between the plain form (elementary torch operations in fp32,
rounded once where the operator rounds) and the library's entry points.
FP8 tensors are uint8 codes in the operands and come back viewed as the torch
FP8 type of the same bits, so that what is compared is the values they stand for.
"""

import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
EPS = 1e-5
SCRATCH = 64 << 20  # bytes of scratch a program keeps beside each of these calls

# ---------------------------------------------------------------------------
# Cases.  hidden 4096 and feed-forward 16384 are the sizes of this library's
# linear-layer workload, 7168 the row length of its grouped one.
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token entering a layer: the residual is added and the row leaves in E4M3 with a fixed scale
        dict(name="norm_token", op="norm", rows=1, cols=4096, residual=True, blocks=False, stats=False, dtype="bf16"),
        # a ragged batch of prompt tokens in front of the grouped GEMM: a scale per 128 values
        dict(name="norm_blocks_ragged", op="norm", rows=1777, cols=7168, residual=True, blocks=True, stats=False, dtype="bf16"),
        # a training step's norm: sum, codes, reciprocal norm, and the amax for the delayed scale
        dict(name="norm_train", op="norm", rows=8192, cols=4096, residual=True, blocks=False, stats=True, dtype="bf16"),
        # its gradient, with the residual branch's gradient added
        dict(name="norm_train_backward", op="norm_backward", rows=8192, cols=4096, residual=True, dtype="bf16"),
        # one decoded token through gate and up: the weights' bytes are the bound
        dict(name="gated_token", op="gated", rows=1, hidden=4096, ffn=16384, act="silu", out="e4m3", save=False, stats=False, accum="mfma_fp8"),
        # a short ragged prompt, a narrower odd-sized layer, 16-bit output
        dict(name="gated_prompt_ragged", op="gated", rows=203, hidden=4096, ffn=5456, act="gelu", out="bf16", save=False, stats=False, accum="exact"),
        # a training step's forward: codes for the next product, amax, and gate and up kept for the gradient
        dict(name="gated_train", op="gated", rows=8192, hidden=4096, ffn=16384, act="silu", out="e4m3", save=True, stats=True, accum="exact"),
        # its gradient: both projections' gradients in E5M2 (both orientations), then the data's and the weights'
        dict(name="gated_train_backward", op="gated_backward", rows=8192, hidden=4096, ffn=16384, act="silu", accum="exact"),
        # the down projection of eight sequences decoding together, residual added
        dict(name="fused_tokens", op="fused", rows=8, inner=16384, cols=4096, bias=False, act="none", residual=True, out="bf16", save=False, stats=False, accum="mfma_fp8"),
        # a ragged prompt through an ungated up projection: bias, GELU, E4M3 for the next product
        dict(name="fused_prompt_ragged", op="fused", rows=1003, inner=4096, cols=16384, bias=True, act="gelu", residual=False, out="e4m3", save=False, stats=True, accum="exact"),
        # a training step's down projection with bias and residual, on the FP8 matrix cores
        dict(name="fused_train", op="fused", rows=8192, inner=16384, cols=4096, bias=True, act="none", residual=True, out="bf16", save=False, stats=False, accum="mfma_fp8"),
        # the gradient of a bias + GELU projection: bias gradient, codes both ways, data and weight gradients
        dict(name="fused_train_backward", op="fused_backward", rows=4096, inner=4096, cols=16384, act="gelu", accum="mfma_fp8"),
    ]


def draw(rng):
    def spread(low, high, step):
        return max(step, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step)

    op = rng.choice(["norm", "norm", "norm_backward", "gated", "gated", "gated_backward", "fused", "fused", "fused_backward"])
    if op.startswith("norm"):
        case = dict(op=op, rows=spread(1, 8192, 1), cols=spread(256, 16384, 16), residual=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "norm":
            blocks = rng.random() < 0.4
            case.update(blocks=blocks, stats=not blocks and rng.random() < 0.6)
        size = 8 if case["dtype"] == "bf16" else 16
        while case["rows"] * case["cols"] * size > 8192 * 4096 * 8:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    accum = rng.choice(["exact", "mfma_fp8"])
    if op.startswith("gated"):
        back = op == "gated_backward"
        case = dict(op=op, rows=spread(16, 8192, 16) if back else spread(1, 8192, 1), hidden=spread(256, 8192, 16), ffn=spread(256, 16384, 16),
                    act=rng.choice(["silu", "silu", "gelu", "relu"]))
        if not back:
            out = rng.choice(["e4m3", "e4m3", "bf16"])
            # the amax of a forward product is asked for where its sums are exact
            case.update(out=out, save=rng.random() < 0.4, stats=out == "e4m3" and accum == "exact" and rng.random() < 0.6)
        while case["rows"] * case["hidden"] * case["ffn"] > 8192 * 4096 * 16384:
            case["rows"] = max(16, case["rows"] // 32 * 16)
    else:
        back = op == "fused_backward"
        case = dict(op=op, rows=spread(16, 8192, 16) if back else spread(1, 8192, 1), inner=spread(256, 16384, 16), cols=spread(256, 16384, 16),
                    act=rng.choice(["gelu", "silu", "relu"] if back else ["none", "none", "gelu", "silu", "relu"]))
        if not back:
            out = rng.choice(["bf16", "bf16", "e4m3"])
            residual = rng.random() < 0.5
            case.update(bias=rng.random() < 0.6, residual=residual, out=out, save=rng.random() < 0.3,
                        stats=out == "e4m3" and accum == "exact" and rng.random() < 0.6)
        while case["rows"] * case["inner"] * case["cols"] > 8192 * 16384 * 4096:
            case["rows"] = max(16, case["rows"] // 32 * 16)
    case["accum"] = accum
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).add_(mean)

    def codes(shape, std, to):
        """A normal tensor cast with a scale that leaves its largest values near the format's top, and the inverse scale."""
        scale = TOP[to] / (6.0 * std)
        q = normal(*shape, std=std * scale).clamp_(-TOP[to], TOP[to]).to(to).view(torch.uint8)
        return q, torch.full((1,), 1.0 / scale, device=dev)

    def one(v):
        return torch.full((1,), float(v), device=dev)

    u8 = dict(dtype=torch.uint8, device=dev)
    bf = dict(dtype=torch.bfloat16, device=dev)
    s = dict(case, scratch=torch.empty(SCRATCH, **u8), amax=torch.zeros(1, device=dev))
    op = case["op"]
    if op.startswith("norm"):
        m, n = case["rows"], case["cols"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["weight"] = normal(n, std=0.1, mean=1.0).to(t)
        if op == "norm":
            s["x"] = normal(m, n).to(t)
            s["res"] = normal(m, n, std=3.0).to(t) if case["residual"] else None
            s["sum"] = torch.empty(m, n, dtype=t, device=dev) if case["residual"] else None
            s["q"] = torch.empty(m, n, **u8)
            s["rstd"] = torch.empty(m, device=dev)
            s["scale"] = one(448.0 / 6.0)
            s["scale_inv"] = torch.empty(m, (n + 127) // 128, device=dev)
        else:
            s["dy"] = normal(m, n, std=0.01).to(t)
            s["h"] = normal(m, n, std=3.0).to(t)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dres"] = normal(m, n, std=0.01).to(t) if case["residual"] else None
            s["dx"] = torch.empty(m, n, dtype=t, device=dev)
            s["dweight"] = torch.empty(n, device=dev)
    elif op.startswith("gated"):
        m, k, f = case["rows"], case["hidden"], case["ffn"]
        s["x"], s["x_inv"] = codes((m, k), 1.0, E4M3)
        s["w"], s["w_inv"] = codes((2 * f, k), 0.02, E4M3)  # the gate's rows, then the up projection's
        if op == "gated":
            s["h"] = torch.empty(m, f, **(u8 if case["out"] == "e4m3" else bf))
            s["gu"] = torch.empty(m, 2 * f, **bf) if case["save"] else None
            s["scale"] = one(16.0)
        else:
            s["dh"] = normal(m, f, std=0.01).bfloat16()
            s["gu"] = normal(m, 2 * f).bfloat16()
            s["scale"] = one(65536.0)
            s["q"], s["qt"] = torch.empty(m, 2 * f, **u8), torch.empty(2 * f, m, **u8)
            s["g_inv"] = one(1.0 / 65536.0)
            s["dx"], s["dw"] = torch.empty(m, k, **bf), torch.empty(2 * f, k, **bf)
    else:
        m, k, n = case["rows"], case["inner"], case["cols"]
        s["x"], s["x_inv"] = codes((m, k), 1.0, E4M3)
        s["w"], s["w_inv"] = codes((n, k), 0.02, E4M3)
        if op == "fused":
            s["b"] = normal(n, std=0.5).bfloat16() if case["bias"] else None
            s["res"] = normal(m, n, std=2.0).bfloat16() if case["residual"] else None
            s["y"] = torch.empty(m, n, **(u8 if case["out"] == "e4m3" else bf))
            s["z"] = torch.empty(m, n, **bf) if case["save"] else None
            s["scale"] = one(32.0)
        else:
            s["dy"] = normal(m, n, std=0.01).bfloat16()
            s["z"] = normal(m, n).bfloat16()
            s["scale"] = one(131072.0)
            s["g_inv"] = one(1.0 / 131072.0)
            s["q"], s["qt"] = torch.empty(m, n, **u8), torch.empty(n, m, **u8)
            s["db"] = torch.empty(n, device=dev)
            s["dx"], s["dw"] = torch.empty(m, k, **bf), torch.empty(n, k, **bf)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


def _norm_own(s):
    import fp8_precision_numerics_amd as fm

    if s["blocks"]:
        fm.fp8_rmsnorm_quantize_blockwise(s["x"], s["weight"], EPS, "e4m3", s["q"], s["scale_inv"], residual=s["res"], sum_out=s["sum"], rstd=s["rstd"])
        return dict(sum=s["sum"], q=s["q"].view(E4M3), scale_inv=s["scale_inv"], rstd=s["rstd"])
    if s["stats"]:
        fm.fp8_rmsnorm_quantize(s["x"], s["weight"], EPS, "e4m3", s["scale"], s["q"], residual=s["res"], sum_out=s["sum"], rstd=s["rstd"], amax=s["amax"], workspace=s["scratch"])
        return dict(sum=s["sum"], q=s["q"].view(E4M3), rstd=s["rstd"], amax=s["amax"])
    fm.fp8_rmsnorm_quantize(s["x"], s["weight"], EPS, "e4m3", s["scale"], s["q"], residual=s["res"], sum_out=s["sum"])
    return dict(sum=s["sum"], q=s["q"].view(E4M3))


def _norm_backward_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], s["dx"], dweight=s["dweight"], dresidual=s["dres"], workspace=s["scratch"])
    return dict(dx=s["dx"], dweight=s["dweight"])


def _gated_own(s):
    import fp8_precision_numerics_amd as fm

    fp8 = s["out"] == "e4m3"
    fm.fp8_gemm_gated(s["x"], "e4m3", s["w"], "e4m3", s["x_inv"], s["w_inv"], s["act"], s["h"], gu=s["gu"], out_fmt="e4m3" if fp8 else None,
                      out_scale=s["scale"] if fp8 else None, amax=s["amax"] if s["stats"] else None, accum=s["accum"], workspace=s["scratch"])
    return dict(h=s["h"].view(E4M3) if fp8 else s["h"], gu=s["gu"], amax=s["amax"] if s["stats"] else None)


def _gated_backward_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_gated_backward(s["dh"], s["gu"], s["act"], "e5m2", s["scale"], q=s["q"], q_t=s["qt"], amax=s["amax"], workspace=s["scratch"])
    fm.fp8_gemm(s["q"], "e5m2", s["w"], "e4m3", s["g_inv"], s["w_inv"], s["dx"], accum=s["accum"], b_trans=True)
    fm.fp8_gemm(s["qt"], "e5m2", s["x"], "e4m3", s["g_inv"], s["x_inv"], s["dw"], accum=s["accum"], b_trans=True)
    return dict(q=s["q"].view(E5M2), qt=s["qt"].view(E5M2), amax=s["amax"], dx=s["dx"], dw=s["dw"])


def _fused_own(s):
    import fp8_precision_numerics_amd as fm

    fp8 = s["out"] == "e4m3"
    fm.fp8_gemm_fused(s["x"], "e4m3", s["w"], "e4m3", s["x_inv"], s["w_inv"], s["y"], bias=s["b"], act=s["act"], residual=s["res"], z=s["z"], out_fmt="e4m3" if fp8 else None,
                      out_scale=s["scale"] if fp8 else None, amax=s["amax"] if s["stats"] else None, accum=s["accum"], workspace=s["scratch"])
    return dict(y=s["y"].view(E4M3) if fp8 else s["y"], z=s["z"], amax=s["amax"] if s["stats"] else None)


def _fused_backward_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_act_backward(s["dy"], s["z"], s["act"], "e5m2", s["scale"], q=s["q"], q_t=s["qt"], dbias=s["db"], amax=s["amax"], workspace=s["scratch"])
    fm.fp8_gemm(s["q"], "e5m2", s["w"], "e4m3", s["g_inv"], s["w_inv"], s["dx"], accum=s["accum"], b_trans=True)
    fm.fp8_gemm(s["qt"], "e5m2", s["x"], "e4m3", s["g_inv"], s["x_inv"], s["dw"], accum=s["accum"], b_trans=True)
    return dict(q=s["q"].view(E5M2), qt=s["qt"].view(E5M2), db=s["db"], amax=s["amax"], dx=s["dx"], dw=s["dw"])


# the plain forms: fp32 throughout, rounded where the operator rounds


def _wide(q, to):
    return q.view(to).float()


def _cast(v, scale, to):
    return (v * scale).clamp(-TOP[to], TOP[to]).to(to)


def _act(z, act):
    """(activation, derivative) of z."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    # GELU in its tanh form
    c, a = math.sqrt(2.0 / math.pi), 0.044715
    p = torch.tanh(c * (z + a * z * z * z))
    return 0.5 * z * (1.0 + p), 0.5 * (1.0 + p) + 0.5 * z * (1.0 - p * p) * c * (1.0 + 3.0 * a * z * z)


def _norm_plain(s):
    total = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    h = total.float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["weight"].float()
    out = dict(sum=total if s["res"] is not None else None)
    if s["blocks"]:
        m, n = y.shape
        b = torch.nn.functional.pad(y, (0, -n % 128)).view(m, -1, 128)
        top = b.abs().amax(2)
        scale = torch.where(top > 0, TOP[E4M3] / top, 1.0)
        q = _cast(b, scale[:, :, None], E4M3).view(torch.uint8).view(m, -1)[:, :n].contiguous().view(E4M3)
        return dict(out, q=q, scale_inv=1.0 / scale, rstd=rstd)
    out["q"] = _cast(y, s["scale"], E4M3)
    if s["stats"]:
        out.update(rstd=rstd, amax=y.abs().max().reshape(1))
    return out


def _norm_backward_plain(s):
    dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["h"].dtype), dweight=(dy * h * r).sum(0))


def _gated_plain(s):
    f = s["ffn"]
    gu = (_wide(s["x"], E4M3) @ _wide(s["w"], E4M3).t()) * (s["x_inv"] * s["w_inv"])
    h = _act(gu[:, :f], s["act"])[0] * gu[:, f:]
    return dict(h=_cast(h, s["scale"], E4M3) if s["out"] == "e4m3" else h.bfloat16(), gu=gu.bfloat16() if s["save"] else None,
                amax=h.abs().max().reshape(1) if s["stats"] else None)


def _gradients(s, d):
    """The cast gradient both ways, its amax, and the data and weight gradients from the codes."""
    q = _cast(d, s["scale"], E5M2)
    c = q.float()
    dx = (c @ _wide(s["w"], E4M3)) * (s["g_inv"] * s["w_inv"])
    dw = (c.t() @ _wide(s["x"], E4M3)) * (s["g_inv"] * s["x_inv"])
    qt = q.view(torch.uint8).t().contiguous().view(E5M2)
    return dict(q=q, qt=qt, amax=d.abs().max().reshape(1), dx=dx.bfloat16(), dw=dw.bfloat16())


def _gated_backward_plain(s):
    f = s["ffn"]
    g, u, dh = s["gu"][:, :f].float(), s["gu"][:, f:].float(), s["dh"].float()
    a, da = _act(g, s["act"])
    return _gradients(s, torch.cat([dh * u * da, dh * a], 1))


def _fused_plain(s):
    z = (_wide(s["x"], E4M3) @ _wide(s["w"], E4M3).t()) * (s["x_inv"] * s["w_inv"])
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])[0]
    if s["res"] is not None:
        y = y + s["res"].float()
    return dict(y=_cast(y, s["scale"], E4M3) if s["out"] == "e4m3" else y.bfloat16(), z=z.bfloat16() if s["save"] else None,
                amax=y.abs().max().reshape(1) if s["stats"] else None)


def _fused_backward_plain(s):
    d = s["dy"].float() * _act(s["z"].float(), s["act"])[1]
    return dict(_gradients(s, d), db=d.sum(0))


_RUN_OWN = dict(norm=_norm_own, norm_backward=_norm_backward_own, gated=_gated_own, gated_backward=_gated_backward_own,
                fused=_fused_own, fused_backward=_fused_backward_own)
_RUN_PLAIN = dict(norm=_norm_plain, norm_backward=_norm_backward_plain, gated=_gated_plain, gated_backward=_gated_backward_plain,
                  fused=_fused_plain, fused_backward=_fused_backward_plain)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    """What leaves in 8 or 16 bits is given unrounded.  A gradient's codes have no
    value here: the products that follow are defined on the rounded codes, and a
    value next to a rounding border may go either way; dx and dw tell."""
    s = prepare(case, seed)
    op, D = case["op"], torch.float64

    def val(q, to=E4M3):
        return q.view(to).to(D)

    def sigmoid(z):
        return torch.sigmoid(z)

    def phi(z):  # the tanh in GELU, as the logistic function of twice its argument
        return 2.0 * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)) - 1.0

    def act(z):
        return {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * sigmoid(z), "gelu": lambda: z * (1.0 + phi(z)) / 2.0}[case["act"]]()

    def slope(z):
        if case["act"] == "relu":
            return (z > 0).to(D)
        if case["act"] == "silu":
            return sigmoid(z) + z * sigmoid(z) * sigmoid(-z)
        return (1.0 + phi(z)) / 2.0 + z / 2.0 * (1.0 - phi(z) ** 2) * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * z ** 2)

    def grown(v, to):
        return torch.clamp(v * s["scale"].to(D), -TOP[to], TOP[to])

    def from_codes(d):
        held = grown(d, E5M2)
        # E5M2 has 2 fraction bits from 2^-14 up and a step of 2^-16 below: rounded to the step of its own power of two
        e = torch.floor(torch.log2(torch.clamp(held.abs(), min=2.0 ** -14)))
        step = torch.exp2(e - 2)
        c = torch.round(held / step) * step  # ties to even
        inv = s["g_inv"].to(D)
        return dict(q=None, qt=None, amax=d.abs().amax().reshape(1), dx=torch.matmul(c, val(s["w"])) * (inv * s["w_inv"].to(D)),
                    dw=torch.matmul(c.t().contiguous(), val(s["x"])) * (inv * s["x_inv"].to(D)))

    if op == "norm":
        h = s["x"].to(D)
        if s["res"] is not None:
            # the sum is kept in the inputs' type and the norm is taken of what is kept
            h = (h + s["res"].to(D)).to(s["x"].dtype).to(D)
        r = (h.pow(2).sum(1) / h.shape[1] + EPS).pow(-0.5)
        y = torch.einsum("mn,m,n->mn", h, r, s["weight"].to(D))
        out = dict(sum=None if s["res"] is None else s["x"].to(D) + s["res"].to(D))
        if case["blocks"]:
            n = y.shape[1]
            top = torch.stack([y[:, i:i + 128].abs().amax(1) for i in range(0, n, 128)], 1)
            wide = top.repeat_interleave(128, 1)[:, :n]
            return dict(out, q=y / wide * 448.0, scale_inv=top / 448.0, rstd=r)
        out["q"] = grown(y, E4M3)
        if case["stats"]:
            out.update(rstd=r, amax=y.abs().amax().reshape(1))
        return out
    if op == "norm_backward":
        dy, h, r, w = s["dy"].to(D), s["h"].to(D), s["rstd"].to(D), s["weight"].to(D)
        n = h.shape[1]
        hat = h * r[:, None]
        along = torch.matmul((dy * hat), w) / n  # one number a row
        dx = (dy * w - hat * along[:, None]) * r[:, None]
        return dict(dx=dx if s["dres"] is None else dx + s["dres"].to(D), dweight=torch.matmul(torch.ones(1, dy.shape[0], dtype=D, device=dy.device), dy * hat)[0])
    if op == "gated":
        f = case["ffn"]
        scale = s["x_inv"].to(D) * s["w_inv"].to(D)
        x, w = val(s["x"]), val(s["w"])
        gate, up = torch.matmul(x, w[:f].t()) * scale, torch.matmul(x, w[f:].t()) * scale
        h = act(gate) * up
        return dict(h=grown(h, E4M3) if case["out"] == "e4m3" else h, gu=torch.cat([gate, up], 1) if case["save"] else None,
                    amax=h.abs().amax().reshape(1) if case["stats"] else None)
    if op == "gated_backward":
        f = case["ffn"]
        gate, up = s["gu"].to(D).split(f, 1)
        dh = s["dh"].to(D)
        return from_codes(torch.cat([dh * up * slope(gate), dh * act(gate)], 1))
    if op == "fused":
        z = torch.matmul(val(s["x"]), val(s["w"]).t()) * (s["x_inv"].to(D) * s["w_inv"].to(D))
        z = z if s["b"] is None else z + s["b"].to(D)
        y = act(z) if s["res"] is None else act(z) + s["res"].to(D)
        return dict(y=grown(y, E4M3) if case["out"] == "e4m3" else y, z=z if case["save"] else None, amax=y.abs().amax().reshape(1) if case["stats"] else None)
    d = s["dy"].to(D) * slope(s["z"].to(D))
    return dict(from_codes(d), db=d.sum(0))


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op = case["op"]
    m = case["rows"]
    if op.startswith("norm"):
        n, b = case["cols"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            per = b + 1 + (2 * b if case["residual"] else 0)
            return dict(bytes=m * n * per + n * b + (m * 4 if case["stats"] or case["blocks"] else 0) + (m * ((n + 127) // 128) * 4 if case["blocks"] else 0), flops=6 * m * n)
        return dict(bytes=m * n * (3 * b + (b if case["residual"] else 0)) + m * 4 + n * (b + 4), flops=12 * m * n)
    if op.startswith("gated"):
        k, f = case["hidden"], case["ffn"]
        if op == "gated":
            return dict(bytes=m * k + 2 * f * k + m * f * (1 if case["out"] == "e4m3" else 2) + (m * f * 4 if case["save"] else 0), flops=2 * m * k * 2 * f)
        # dh, gate and up in; codes both ways, both gradients out; weights and activations' codes in
        return dict(bytes=m * f * (2 + 4 + 2 + 2) + 2 * f * k + m * k + 2 * (m * k + 2 * f * k), flops=2 * 2 * m * k * 2 * f)
    k, n = case["inner"], case["cols"]
    if op == "fused":
        return dict(bytes=m * k + n * k + m * n * ((1 if case["out"] == "e4m3" else 2) + (2 if case["residual"] else 0) + (2 if case["save"] else 0)) + (2 * n if case["bias"] else 0),
                    flops=2 * m * k * n)
    return dict(bytes=m * n * (2 + 2 + 1 + 1) + 4 * n + n * k + m * k + 2 * (m * k + n * k), flops=2 * 2 * m * k * n)
