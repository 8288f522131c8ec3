"""Measured cases of the operators at both ends of a model trained in FP8: layer
norm that drops values of a branch, adds the residual and leaves in 8 bits;
softmax cross entropy over a vocabulary, with the vocabulary's FP8 projection
inside and no logits kept; embedding lookup; each forward and backward.

``own`` selects between the plain form (elementary torch operations in fp32,
rounded once where the operator rounds) and the library's entry points.
FP8 tensors are uint8 codes in the operands and come back viewed as the torch
FP8 type of the same bits, so that what is compared is the values they stand for.
Dropped values are chosen by a counter-based generator (Philox4x32-10: Salmon,
Moraes, Dror and Shaw, SC 2011) from a seed and an offset that are inputs.
"""

import math

import numpy as np
import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
EPS = 1e-5
IGNORE = -100  # a target outside the vocabulary: its row takes no part
SCRATCH = 64 << 20        # bytes of scratch a program keeps beside each of these calls
SCRATCH_LOSS = 512 << 20  # and for the loss's gradient, whose pieces of the vocabulary it holds

# ---------------------------------------------------------------------------
# Cases.  hidden 4096 is this library's linear-layer workload's; 65536 and 131072
# are vocabularies of a power of two, 50021 one of no round size.
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token entering a layer: the residual is added and the row leaves in E4M3 with a fixed scale
        dict(name="norm_token", op="norm", rows=1, cols=4096, residual=True, stats=False, dropout=0.0, dtype="bf16"),
        # a training step's norm: the branch is dropped out, the sum kept, codes, mean, reciprocal deviation and amax
        dict(name="norm_train", op="norm", rows=8192, cols=4096, residual=True, stats=True, dropout=0.1, dtype="bf16"),
        # its gradient: the stream's and the branch's, with the weight's and the bias's
        dict(name="norm_train_backward", op="norm_backward", rows=8192, cols=4096, residual=True, dropout=0.1, dtype="bf16"),
        # a ragged batch in fp32 without dropout
        dict(name="norm_ragged_backward", op="norm_backward", rows=1777, cols=1040, residual=False, dropout=0.0, dtype="f32"),
        # scoring one token: the vocabulary's bytes are the bound
        dict(name="loss_token", op="loss", rows=1, hidden=4096, vocab=131072, accum="exact"),
        # a ragged evaluation batch over a vocabulary of no round size
        dict(name="loss_ragged", op="loss", rows=1003, hidden=4096, vocab=50021, accum="exact"),
        # a training step's loss
        dict(name="loss_train", op="loss", rows=8192, hidden=4096, vocab=65536, accum="exact"),
        # its gradient on the FP8 matrix cores: the hidden states' and the vocabulary weight's
        dict(name="loss_train_backward", op="loss_backward", rows=8192, hidden=4096, vocab=65536, accum="mfma_fp8"),
        # a short ragged batch of fine-tuning, exact sums
        dict(name="loss_ragged_backward", op="loss_backward", rows=219, hidden=2048, vocab=50021, accum="exact"),
        # one decoded token from a table in E4M3 (a tied head's codes)
        dict(name="embed_token", op="embed", rows=1, cols=4096, vocab=65536, table="e4m3"),
        # a training batch from a bf16 table
        dict(name="embed_train", op="embed", rows=8192, cols=4096, vocab=65536, table="bf16"),
        # the table's gradient of that batch, added to the tied head's
        dict(name="embed_train_backward", op="embed_backward", rows=8192, cols=4096, vocab=65536, base=True, dtype="bf16", out="bf16"),
    ]


def draw(rng):
    def spread(low, high, step):
        return max(step, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step)

    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "loss", "loss", "loss_backward", "loss_backward", "embed", "embed_backward"])
    if op.startswith("norm"):
        case = dict(op=op, rows=spread(1, 8192, 1), cols=spread(256, 16384, 16), residual=rng.random() < 0.7,
                    dropout=rng.choice([0.0, 0.0, 0.1, 0.25]), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "norm":
            case.update(stats=rng.random() < 0.6)
        size = 2 if case["dtype"] == "bf16" else 4
        while case["rows"] * case["cols"] * size > 8192 * 4096 * 2:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    if op.startswith("loss"):
        # the loss alone is a number of 24 bits: its products are summed exactly
        case = dict(op=op, rows=spread(1, 8192, 1), hidden=spread(256, 8192, 16), vocab=spread(1000, 131072, 1),
                    accum="exact" if op == "loss" else rng.choice(["exact", "mfma_fp8"]))
        while case["rows"] * case["hidden"] * case["vocab"] > 4096 * 4096 * 65536:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    case = dict(op=op, rows=spread(1, 32768, 1), cols=spread(256, 8192, 16), vocab=spread(1000, 131072, 1))
    if op == "embed":
        case.update(table=rng.choice(["bf16", "f32", "e4m3"]))
    else:
        case.update(base=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    while case["rows"] * case["cols"] > 8192 * 4096:
        case["rows"] = max(1, case["rows"] // 2)
    while case["vocab"] * case["cols"] * (2 if case.get("out") == "f32" else 1) > 65536 * 4096:
        case["vocab"] = case["vocab"] // 2
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).add_(mean)

    def codes(shape, std):
        """A normal tensor cast to E4M3 with a scale that leaves its largest values near the top, and the inverse scale."""
        scale = TOP[E4M3] / (6.0 * std)
        q = normal(*shape, std=std * scale).clamp_(-TOP[E4M3], TOP[E4M3]).to(E4M3).view(torch.uint8)
        return q, torch.full((1,), 1.0 / scale, device=dev)

    def one(v):
        return torch.full((1,), float(v), device=dev)

    types = dict(bf16=torch.bfloat16, f32=torch.float32)
    s = dict(case, amax=torch.zeros(1, device=dev))
    s["scratch"] = torch.empty(SCRATCH_LOSS if case["op"] == "loss_backward" else SCRATCH, dtype=torch.uint8, device=dev)
    op, m = case["op"], case["rows"]
    if op.startswith("norm"):
        n, t = case["cols"], types[case["dtype"]]
        s["weight"] = normal(n, std=0.1, mean=1.0).to(t)
        s["rng"] = torch.tensor([int(seed) * 7919 + 1, 5], dtype=torch.int64, device=dev)  # seed, and the offset of this call
        if op == "norm":
            s["bias"] = normal(n, std=0.1).to(t)
            s["x"] = normal(m, n).to(t)
            s["res"] = normal(m, n, std=3.0, mean=0.5).to(t) if case["residual"] else None
            s["sum"] = torch.empty(m, n, dtype=t, device=dev) if case["residual"] or case["dropout"] else None
            s["q"] = torch.empty(m, n, dtype=torch.uint8, device=dev)
            s["mean"], s["rstd"] = torch.empty(m, device=dev), torch.empty(m, device=dev)
            s["scale"] = one(448.0 / 6.0)
        else:
            s["dy"] = normal(m, n, std=0.01).to(t)
            s["h"] = normal(m, n, std=3.0, mean=0.5).to(t)
            h = s["h"].double()
            s["mean"] = h.mean(1).float()
            s["rstd"] = torch.rsqrt(h.var(1, unbiased=False) + EPS).float()
            s["dres"] = normal(m, n, std=0.01).to(t) if case["residual"] else None
            s["dx"] = torch.empty(m, n, dtype=t, device=dev)
            s["dbranch"] = torch.empty(m, n, dtype=t, device=dev) if case["dropout"] else None
            s["dweight"], s["dbias"] = torch.empty(n, device=dev), torch.empty(n, device=dev)
        return s
    v = case["vocab"]
    if op.startswith("loss"):
        k = case["hidden"]
        s["x"], s["x_inv"] = codes((m, k), 1.0)
        s["w"], s["w_inv"] = codes((v, k), 0.02)
        s["target"] = torch.randint(0, v, (m,), generator=g, device=dev)
        s["target"][torch.rand(m, generator=g, device=dev) < (0.05 if m > 1 else 0.0)] = IGNORE
        if op == "loss":
            s["loss"], s["lse"] = torch.empty(m, device=dev), torch.empty(m, device=dev)
        else:
            s["lse"] = torch.logsumexp(_logits(s), 1)
            s["dloss"] = torch.full((m,), 1.0 / m, device=dev)
            s["scale"], s["g_inv"] = one(16384.0 * m), one(1.0 / (16384.0 * m))  # the delayed scale and its inverse
            s["dx"] = torch.empty(m, k, dtype=torch.bfloat16, device=dev)
            s["dw"] = torch.empty(v, k, dtype=torch.bfloat16, device=dev)
        return s
    n = case["cols"]
    # common tokens are common: the density of a token falls as a power of its number
    s["tokens"] = (torch.rand(m, generator=g, device=dev, dtype=torch.float64).pow(3.0) * v).long()
    s["tokens"][torch.rand(m, generator=g, device=dev) < (0.02 if m > 1 else 0.0)] = -1  # padding
    s["factor"] = math.sqrt(n)
    if op == "embed":
        s["fmt"], s["inv"] = None, None
        if case["table"] == "e4m3":
            s["weight"], s["inv"] = codes((v, n), 0.02)
            s["fmt"] = "e4m3"
        else:
            s["weight"] = normal(v, n, std=0.02).to(types[case["table"]])
        s["out"] = torch.empty(m, n, dtype=types["f32" if case["table"] == "f32" else "bf16"], device=dev)
    else:
        s["dy"] = normal(m, n, std=0.01).to(types[case["dtype"]])
        s["base"] = normal(v, n, std=0.01).to(types[case["out"]]) if case["base"] else None
        s["dtable"] = torch.empty(v, n, dtype=types[case["out"]], device=dev)
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

    drop = dict(dropout=s["dropout"], rng=s["rng"]) if s["dropout"] else {}
    if s["stats"]:
        fm.fp8_layernorm_quantize(s["x"], s["weight"], s["bias"], EPS, "e4m3", s["scale"], s["q"], residual=s["res"], sum_out=s["sum"], mean=s["mean"], rstd=s["rstd"],
                                  amax=s["amax"], workspace=s["scratch"], **drop)
        return dict(sum=s["sum"], q=s["q"].view(E4M3), mean=s["mean"], rstd=s["rstd"], amax=s["amax"])
    fm.fp8_layernorm_quantize(s["x"], s["weight"], s["bias"], EPS, "e4m3", s["scale"], s["q"], residual=s["res"], sum_out=s["sum"], **drop)
    return dict(sum=s["sum"], q=s["q"].view(E4M3))


def _norm_backward_own(s):
    import fp8_precision_numerics_amd as fm

    drop = dict(dbranch=s["dbranch"], dropout=s["dropout"], rng=s["rng"]) if s["dropout"] else {}
    fm.fp8_layernorm_backward(s["dy"], s["h"], s["mean"], s["rstd"], s["weight"], s["dx"], dweight=s["dweight"], dbias=s["dbias"], dresidual=s["dres"],
                              workspace=s["scratch"], **drop)
    return dict(dx=s["dx"], dbranch=s["dbranch"], dweight=s["dweight"], dbias=s["dbias"])


def _loss_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_vocab_cross_entropy(s["x"], "e4m3", s["w"], "e4m3", s["x_inv"], s["w_inv"], s["target"], s["loss"], s["lse"], accum=s["accum"], workspace=s["scratch"])
    return dict(loss=s["loss"], lse=s["lse"])


def _loss_backward_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_vocab_cross_entropy_backward(s["x"], "e4m3", s["w"], "e4m3", s["x_inv"], s["w_inv"], s["target"], s["lse"], s["dloss"], "e5m2", s["scale"], s["g_inv"],
                                        dx=s["dx"], dw=s["dw"], amax=s["amax"], accum=s["accum"], workspace=s["scratch"])
    return dict(dx=s["dx"], dw=s["dw"], amax=s["amax"])


def _embed_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_embedding(s["tokens"], s["weight"], s["out"], scale=s["factor"], fmt=s["fmt"], sinv=s["inv"])
    return s["out"]


def _embed_backward_own(s):
    import fp8_precision_numerics_amd as fm

    fm.fp8_embedding_backward(s["tokens"], s["dy"], s["dtable"], scale=s["factor"], base=s["base"], workspace=s["scratch"])
    return s["dtable"]


# the plain forms: fp32 throughout, rounded where the operator rounds


def _wide(q, to=E4M3):
    return q.view(to).float()


def _cast(v, scale, to):
    return (v * scale).clamp(-TOP[to], TOP[to]).to(to)


_LOW = 0xFFFFFFFF


def _philox(groups, rng):
    """128 random bits for each counter 0 .. groups - 1, as four int64 tensors of 32 bits each."""
    n = torch.arange(groups, dtype=torch.int64, device=rng.device)
    key, offset = rng[0], rng[1]
    c = [n & _LOW, n >> 32, (offset & _LOW).expand(groups), ((offset >> 32) & _LOW).expand(groups)]
    k0, k1 = key & _LOW, (key >> 32) & _LOW
    for i in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # the products' low 64 bits are all of them
        c = [((b >> 32) & _LOW) ^ c[1] ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c[3] ^ k1, a & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c


def _keep(s, shape):
    """What each value of a tensor is multiplied with: 0 where it is dropped."""
    cut = round(s["dropout"] * 65536)
    words = torch.stack(_philox(shape[0] * shape[1] // 8, s["rng"]), 1)
    parts = torch.stack([words & 0xFFFF, words >> 16], 2).view(shape)
    return (parts >= cut).float() * (65536.0 / (65536 - cut))


def _norm_plain(s):
    total = s["x"].float()
    if s["dropout"]:
        total = total * _keep(s, total.shape)
    if s["res"] is not None:
        total = total + s["res"].float()
    total = total.to(s["x"].dtype)
    h = total.float()
    mean = h.mean(1)
    centred = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1) + EPS)
    y = centred * rstd[:, None] * s["weight"].float() + s["bias"].float()
    out = dict(sum=total if s["sum"] is not None else None, q=_cast(y, s["scale"], E4M3))
    if s["stats"]:
        out.update(mean=mean, rstd=rstd, amax=y.abs().max().reshape(1))
    return out


def _norm_backward_plain(s):
    dy, r = s["dy"].float(), s["rstd"][:, None]
    hat = (s["h"].float() - s["mean"][:, None]) * r
    g = dy * s["weight"].float()
    dx = r * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    t = s["h"].dtype
    return dict(dx=dx.to(t), dbranch=(dx * _keep(s, dx.shape)).to(t) if s["dropout"] else None, dweight=(dy * hat).sum(0), dbias=dy.sum(0))


def _logits(s):
    return (_wide(s["x"]) @ _wide(s["w"]).t()) * (s["x_inv"] * s["w_inv"])


def _loss_plain(s):
    z = _logits(s)
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    t = s["target"]
    valid = (t >= 0) & (t < s["vocab"])
    mine = z.gather(1, torch.where(valid, t, 0)[:, None])[:, 0]
    return dict(loss=torch.where(valid, lse - mine, 0.0), lse=lse)


def _loss_backward_plain(s):
    d = torch.exp(_logits(s) - s["lse"][:, None])
    t = s["target"]
    valid = (t >= 0) & (t < s["vocab"])
    d.scatter_add_(1, torch.where(valid, t, 0)[:, None], torch.full_like(d[:, :1], -1.0))
    d *= torch.where(valid, s["dloss"], 0.0)[:, None]
    amax = torch.maximum(d.amax(), -d.amin()).reshape(1)
    c = _cast(d, s["scale"], E5M2).float()
    dx = (c @ _wide(s["w"])) * (s["g_inv"] * s["w_inv"])
    dw = (c.t() @ _wide(s["x"])) * (s["g_inv"] * s["x_inv"])
    return dict(dx=dx.bfloat16(), dw=dw.bfloat16(), amax=amax)


def _embed_plain(s):
    valid = (s["tokens"] >= 0) & (s["tokens"] < s["vocab"])
    rows = s["weight"][torch.where(valid, s["tokens"], 0)]
    rows = rows.float() if s["fmt"] is None else _wide(rows) * s["inv"]
    return (rows * s["factor"] * valid[:, None]).to(s["out"].dtype)


def _embed_backward_plain(s):
    v = s["vocab"]
    valid = (s["tokens"] >= 0) & (s["tokens"] < v)
    total = torch.zeros(v + 1, s["cols"], device=s["dy"].device)  # the last row takes what has no token
    total.index_add_(0, torch.where(valid, s["tokens"], v), s["dy"].float())
    total = total[:v] * s["factor"]
    if s["base"] is not None:
        total = total + s["base"].float()
    return total.to(s["dtable"].dtype)


_RUN_OWN = dict(norm=_norm_own, norm_backward=_norm_backward_own, loss=_loss_own, loss_backward=_loss_backward_own, embed=_embed_own, embed_backward=_embed_backward_own)
_RUN_PLAIN = dict(norm=_norm_plain, norm_backward=_norm_backward_plain, loss=_loss_plain, loss_backward=_loss_backward_plain, embed=_embed_plain,
                  embed_backward=_embed_backward_plain)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------


def _random_halves(groups, seed, offset):
    """The generator again, on the host: eight numbers of 16 bits a counter."""
    full = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)

    def product(a, m):
        p = a * np.uint64(m)
        return p >> half, p & full

    n = np.arange(groups, dtype=np.uint64)
    lanes = np.zeros((4, groups), dtype=np.uint64)
    lanes[0], lanes[1], lanes[2], lanes[3] = n & full, n >> half, offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    for r in range(10):
        hi0, lo0 = product(lanes[0], 0xD2511F53)
        hi1, lo1 = product(lanes[2], 0xCD9E8D57)
        key = [np.uint64((word + r * step) % (1 << 32)) for word, step in ((seed & 0xFFFFFFFF, 0x9E3779B9), ((seed >> 32) & 0xFFFFFFFF, 0xBB67AE85))]
        lanes = np.stack([hi1 ^ lanes[1] ^ key[0], lo1, hi0 ^ lanes[3] ^ key[1], lo0])
    return np.ascontiguousarray(lanes.T.astype("<u4")).view("<u2").reshape(-1)


def exact(case, seed):
    """What leaves in 8 or 16 bits is given unrounded.  The loss's gradient is defined
    on the codes of the logits' gradient; a value next to a rounding border may go either way."""
    s = prepare(case, seed)
    op, D = case["op"], torch.float64
    dev = s["amax"].device

    def val(q):
        return q.view(E4M3).to(D)

    def factors():
        cut = int(math.floor(case["dropout"] * 65536 + 0.5))
        u = _random_halves(case["rows"] * case["cols"] // 8, *[int(x) for x in s["rng"].tolist()]).astype(np.int32)
        return torch.from_numpy(u).to(dev).reshape(case["rows"], case["cols"]).ge(cut).to(D) / (1.0 - cut / 65536.0)

    if op == "norm":
        h = s["x"].to(D)
        if case["dropout"]:
            h = h * factors()
        if s["res"] is not None:
            h = h + s["res"].to(D)
        kept = h.to(s["x"].dtype).to(D)  # the sum is kept in the inputs' type and the norm is taken of what is kept
        n = kept.shape[1]
        mean = kept.sum(1) / n
        var = (kept * kept).sum(1) / n - mean * mean
        r = (var + EPS).pow(-0.5)
        y = torch.addcmul(s["bias"].to(D), (kept - mean[:, None]) * s["weight"].to(D), r[:, None])
        out = dict(sum=h if s["sum"] is not None else None, q=torch.clamp(y * s["scale"].to(D), -448.0, 448.0))
        if case["stats"]:
            out.update(mean=mean, rstd=r, amax=y.abs().amax().reshape(1))
        return out
    if op == "norm_backward":
        n = case["cols"]
        dy, r = s["dy"].to(D), s["rstd"].to(D)
        a = (s["h"].to(D) - s["mean"].to(D)[:, None]) * r[:, None]
        g = dy * s["weight"].to(D)
        # the projection of g off the constant row and off a, divided by the deviation
        both = torch.stack([g.sum(1), (g * a).sum(1)]) / n
        dx = (g - both[0][:, None] - a * both[1][:, None]) * r[:, None]
        if s["dres"] is not None:
            dx = dx + s["dres"].to(D)
        ones = torch.ones(1, dy.shape[0], dtype=D, device=dev)
        return dict(dx=dx, dbranch=dx * factors() if case["dropout"] else None, dweight=torch.matmul(ones, dy * a)[0], dbias=torch.matmul(ones, dy)[0])
    if op.startswith("loss"):
        z = torch.matmul(val(s["x"]), val(s["w"]).t()) * (s["x_inv"].to(D) * s["w_inv"].to(D))
        inside = (s["target"] >= 0) & (s["target"] < case["vocab"])
        if op == "loss":
            lse = torch.logsumexp(z, 1)
            rows = torch.arange(case["rows"], device=dev)
            return dict(loss=torch.where(inside, lse - z[rows, s["target"].clamp(min=0)], torch.zeros_like(lse)), lse=lse)
        z -= s["lse"].to(D)[:, None]
        z.exp_()
        rows = torch.arange(case["rows"], device=dev)[inside]
        z[rows, s["target"][inside]] -= 1.0
        z *= (s["dloss"].to(D) * inside)[:, None]
        amax = torch.maximum(z.amax(), z.amin().neg()).reshape(1)
        z *= s["scale"].to(D)
        z.clamp_(-TOP[E5M2], TOP[E5M2])
        # E5M2 has 2 fraction bits from 2^-14 up and a step of 2^-16 below: rounded to the step of its own power of two
        step = torch.exp2(torch.floor(torch.log2(torch.clamp(z.abs(), min=2.0 ** -14))) - 2)
        z.div_(step).round_().mul_(step)  # ties to even
        del step
        inv = s["g_inv"].to(D)
        return dict(dx=torch.matmul(z, val(s["w"])) * (inv * s["w_inv"].to(D)), dw=torch.matmul(z.t(), val(s["x"])) * (inv * s["x_inv"].to(D)), amax=amax)
    here = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
    ids = s["tokens"][here]
    if op == "embed":
        out = torch.zeros(case["rows"], case["cols"], dtype=D, device=dev)
        out[here] = (s["weight"][ids].to(D) if s["fmt"] is None else val(s["weight"][ids]) * s["inv"].to(D)) * s["factor"]
        return out
    out = torch.zeros(case["vocab"], case["cols"], dtype=D, device=dev) if s["base"] is None else s["base"].to(D)
    return out.index_put_((ids,), s["dy"][here].to(D) * s["factor"], accumulate=True)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op, m = case["op"], case["rows"]
    if op.startswith("norm"):
        n, b, drop = case["cols"], 2 if case["dtype"] == "bf16" else 4, case["dropout"] > 0
        if op == "norm":
            per = b + 1 + (b if case["residual"] else 0) + (b if case["residual"] or drop else 0)
            return dict(bytes=m * n * per + 2 * n * b + (8 * m if case["stats"] else 0), flops=8 * m * n)
        per = 3 * b + (b if case["residual"] else 0) + (b if drop else 0)
        return dict(bytes=m * n * per + 8 * m + n * (b + 8), flops=14 * m * n)
    if op.startswith("loss"):
        k, v = case["hidden"], case["vocab"]
        if op == "loss":
            return dict(bytes=m * k + v * k + m * 16, flops=2 * m * k * v)
        # the logits again, then both gradients
        return dict(bytes=m * k + v * k + m * 16 + 2 * (m * k + v * k), flops=6 * m * k * v)
    n, v = case["cols"], case["vocab"]
    if op == "embed":
        row = n * (dict(bf16=2, f32=4, e4m3=1)[case["table"]] + (4 if case["table"] == "f32" else 2))
        return dict(bytes=m * (row + 8), flops=m * n)
    out = 2 if case["out"] == "bf16" else 4
    return dict(bytes=m * (8 + n * (2 if case["dtype"] == "bf16" else 4)) + v * n * out * (2 if case["base"] else 1), flops=2 * m * n)
