"""The operators of a pre-norm encoder layer and of a vocabulary head as measured cases: the root-mean-square norm with the
residual's addition (`norm`), also with rows in 8 bits (`norm_q8`), the projection of such rows (`linear_q8`), the gated
feed-forward (`gated`), log probabilities of given tokens with entropy and top alternatives (`logprobs`), and distillation
from a teacher's top logits (`distill`).

Each case names its operator and direction (`op`), element type and sizes. `run` computes one pass either with the
library's entry points (`own`) or in a plain form of elementary torch operations in 32 bits; `exact` computes the same
from the definitions in 64 bits.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
E4M3_MOST = 448.0  # the largest number of the 8-bit type


def listed():
    return [
        # one token's norm on its way into an 8-bit projection: serving, bound by latency
        dict(name="norm_q8_token", op="norm_q8", dtype="f16", T=1, D=1024, residual=True),
        # a training step's norm on the longest packed batch: the branch is added to the residual stream, which is kept
        dict(name="norm_long", op="norm", dtype="bf16", T=131072, D=1024, residual=True),
        # the same backwards, with the gradient that comes down the residual stream
        dict(name="norm_backward_global", op="norm_backward", dtype="bf16", T=16931, D=768, residual=True),
        # one token through an 8-bit feed-forward's first projection
        dict(name="linear_q8_token", op="linear_q8", dtype="bf16", T=1, K=1024, N=4096, act="gelu", bias=True, residual=False),
        # an offline encoding job's widest projection
        dict(name="linear_q8_local", op="linear_q8", dtype="bf16", T=72804, K=1024, N=4096, act="none", bias=True,
             residual=False),
        # one token through a gated feed-forward
        dict(name="gated_token", op="gated", dtype="bf16", T=1, K=1024, F=2624, act="gelu", bias=False, pre=False),
        # a training step's gated feed-forward; both pre-activations are kept for the backward
        dict(name="gated_long", op="gated", dtype="bf16", T=65536, K=1024, F=2624, act="gelu", bias=False, pre=True),
        # the smaller encoder's, backwards
        dict(name="gated_backward_global", op="gated_backward", dtype="f16", T=16931, K=768, F=1152, act="silu", bias=True),
        # a teacher scoring a batch and keeping its sixteen likeliest words for a student
        dict(name="logprobs_teacher", op="logprobs", dtype="bf16", T=8192, V=50000, top=16),
        # a policy's step on a few sampled tokens, with an entropy bonus; a vocabulary whose rows lie off every boundary
        dict(name="logprobs_backward_odd", op="logprobs_backward", dtype="f32", T=641, V=32003, entropy=True),
        # masked-token distillation: one token in seven has targets
        dict(name="distill_masked", op="distill", dtype="bf16", T=16931, D=768, V=50000, top=32, bias=True, temperature=1.0,
             targets=0.15),
        # a student's loss on every token, backwards
        dict(name="distill_backward_all", op="distill_backward", dtype="bf16", T=16384, D=1024, V=32768, top=16, bias=False,
             temperature=2.0, targets=1.0),
    ]


MOST_FLOPS = 6.0 * 16384 * 1024 * 32768  # of distill_backward_all, the largest listed case
MOST_ROW_ELEMENTS = 131072 * 1024        # of norm_long
MOST_LOGITS = 8192 * 50000               # of logprobs_teacher


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; in one of two cases a multiple of eight."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 16:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_backward", "linear_q8", "gated", "gated_backward", "logprobs",
                     "logprobs_backward", "distill", "distill_backward"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op.startswith("norm"):
        case.update(T=_between(rng, 1, 131072), D=_between(rng, 8, 16384), residual=rng.random() < 0.7)
        case["T"] = max(1, min(case["T"], MOST_ROW_ELEMENTS // case["D"]))
        return case
    if op.startswith("logprobs"):
        case.update(T=_between(rng, 1, 65536), V=_between(rng, 100, 200000))
        if op == "logprobs":
            case.update(top=rng.choice([0, 1, 5, 20, 64, rng.randint(1, 64)]))
        else:
            case.update(entropy=rng.random() < 0.5)
        case["T"] = max(1, min(case["T"], MOST_LOGITS // case["V"]))
        return case
    if op == "linear_q8":
        # rows of whole 16 bytes, as 8-bit weights are laid out
        case.update(T=_between(rng, 1, 131072), K=16 * _between(rng, 4, 256), N=_between(rng, 64, 4096),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
        cost = 2.0 * case["N"] * case["K"]
    elif op.startswith("gated"):
        case.update(T=_between(rng, 1, 131072), K=_between(rng, 64, 4096), F=_between(rng, 64, 4096),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5)
        if op == "gated":
            case.update(pre=rng.random() < 0.5)
        cost = (4.0 if op == "gated" else 8.0) * case["F"] * case["K"]
    else:
        case.update(T=_between(rng, 1, 65536), D=_between(rng, 64, 2048), V=_between(rng, 100, 130000), top=rng.randint(1, 64),
                    bias=rng.random() < 0.5, temperature=rng.choice([1.0, 2.0, round(rng.uniform(0.5, 4.0), 2)]),
                    targets=rng.choice([1.0, 0.9, 0.15]))
        cost = (2.0 if op == "distill" else 6.0) * case["D"] * case["V"]
    # in 64 bits and in the plain form the products are dear: no case over two fifths of the largest listed one
    case["T"] = max(1, min(case["T"], int(0.4 * MOST_FLOPS / cost)))
    if op.startswith("distill"):
        case["T"] = max(1, min(case["T"], 2 * MOST_LOGITS // case["V"]))
    return case


def _rows_with_targets(case):
    return int(round(case["targets"] * case["T"]))


def _to_e4m3(y):
    """(8-bit rows, their scales): each row's largest magnitude becomes the type's largest number."""
    scale = y.abs().amax(1) * (1.0 / E4M3_MOST)
    return (y / torch.where(scale > 0, scale, 1.0)[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dt, dev = TYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    op, T = case["op"], case["T"]
    s = dict(case=case)
    if op.startswith("norm"):
        D = case["D"]
        s["x"] = normal(T, D, std=1.5)
        s["w"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        if op == "norm_backward":
            s["dy"] = normal(T, D, std=1e-2)
            s["dh"] = normal(T, D, std=1e-2) if case["residual"] else None
        else:
            s["residual"] = normal(T, D) if case["residual"] else None
    elif op == "linear_q8":
        K, N = case["K"], case["N"]
        s["x"], s["x_scale"] = _to_e4m3(torch.randn(T, K, generator=g, device=dev))
        s["w"], s["w_scale"] = _to_e4m3(torch.randn(N, K, generator=g, device=dev) * K**-0.5)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["residual"] = normal(T, N) if case["residual"] else None
    elif op.startswith("gated"):
        K, F = case["K"], case["F"]
        s["x"] = normal(T, K)
        s["w"] = normal(2 * F, K, std=K**-0.5)
        if op == "gated":
            s["bias"] = normal(2 * F, std=0.1) if case["bias"] else None
        else:
            s["dy"] = normal(T, F, std=1e-2)
            s["pre"] = normal(T, 2 * F)
    elif op.startswith("logprobs"):
        V = case["V"]
        s["logits"] = normal(T, V, std=2.5)
        labels = torch.randint(0, V, (T,), generator=g, device=dev)
        s["labels"] = torch.where(torch.rand(T, generator=g, device=dev) < 0.1, -100, labels)
        if op == "logprobs_backward":
            p = torch.log_softmax(s["logits"].float(), 1)
            s["lse"] = torch.logsumexp(s["logits"].float(), 1)
            s["entropy"] = -(p.exp() * p).sum(1)
            s["dlogp"] = torch.randn(T, generator=g, device=dev) / T
            s["dentropy"] = -0.01 * (torch.rand(T, generator=g, device=dev) + 0.5) / T if case["entropy"] else None
    else:
        D, V, top = case["D"], case["V"], min(case["top"], case["V"])
        s["x"] = normal(T, D)
        s["w"] = normal(V, D, std=2.0 * D**-0.5)
        s["bias"] = normal(V, std=0.3) if case["bias"] else None
        # a teacher's likeliest words, the first the likeliest, with their logits; rows without a target have none
        first = torch.randint(0, V, (T, 1), generator=g, device=dev)
        idx = (first + torch.arange(top, device=dev) * (V // top)) % V
        s["values"] = (torch.randn(T, top, generator=g, device=dev) * 2.5).sort(1, descending=True).values
        order = torch.rand(T, generator=g, device=dev).argsort()
        idx[order[_rows_with_targets(case):]] = -1
        s["idx"] = idx
        if op == "distill_backward":
            rows = (idx[:, 0] >= 0).nonzero()[:, 0]
            lse = torch.zeros(T, device=dev)
            for part in rows.split(8192):
                z = s["x"][part].float() @ s["w"].float().T
                if case["bias"]:
                    z += s["bias"].float()
                lse[part] = torch.logsumexp(z / case["temperature"], 1)
            s["lse"] = lse
            s["dloss"] = (torch.rand(T, generator=g, device=dev) + 0.5) / max(1, _rows_with_targets(case))
    return s


# ------------------------------------------------------------------------------------------
# the plain form


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        h = 1.0 / (1.0 + torch.exp(-z))
        return h * (1.0 + z * (1.0 - h))
    return torch.ones_like(z)


def _plain_norm(s, dt):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
    out = {}
    if s["case"]["op"] == "norm_q8":
        out["q"], out["scale"] = _to_e4m3(y)
    else:
        out["y"] = y.to(dt)
    if s["residual"] is not None:
        out["h"] = h.to(dt)
    return out


def _plain_norm_backward(s, dt):
    h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * r
    g = dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(dt), dw=(dy * n).sum(0).to(dt))


def _plain_linear_q8(s, dt):
    z = (s["x"].float() @ s["w"].float().T) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return dict(y=y.to(dt))


def _plain_gated(s, dt):
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    gate, up = z.chunk(2, 1)
    y = (_act(gate, s["case"]["act"]) * up).to(dt)
    return dict(y=y, pre=z.to(dt)) if s["case"]["pre"] else dict(y=y)


def _plain_gated_backward(s, dt):
    gate, up = s["pre"].float().chunk(2, 1)
    dy, act = s["dy"].float(), s["case"]["act"]
    dz = torch.cat([dy * up * _act_slope(gate, act), dy * _act(gate, act)], 1)
    out = dict(dx=(dz @ s["w"].float()).to(dt), dw=(dz.T @ s["x"].float()).to(dt))
    if s["case"]["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _likeliest(z, top):
    """The indices [T, top] of the largest logits, the largest first and equal ones by their index."""
    bits = (z + 0.0).view(torch.int32).long()
    ordered = torch.where(bits < 0, -2147483648 - bits, bits)  # as the numbers are ordered
    place = torch.arange(z.shape[1], device=z.device)
    return ((1 << 20) - 1) - (ordered * (1 << 20) + ((1 << 20) - 1 - place)).topk(top, 1).values % (1 << 20)


def _plain_logprobs(s, dt):
    z, labels, top = s["logits"].float(), s["labels"], s["case"]["top"]
    most = z.max(1, keepdim=True).values
    d = z - most
    e = torch.exp(d)
    total = e.sum(1)
    rest = torch.log(total)
    picked = d.gather(1, labels.clamp(min=0)[:, None])[:, 0] - rest
    out = dict(logp=torch.where(labels >= 0, picked, 0.0), lse=most[:, 0] + rest, entropy=rest - (e * d).sum(1) / total)
    if top:
        idx = _likeliest(z, min(top, z.shape[1]))
        out.update(top_logp=d.gather(1, idx) - rest[:, None], top_idx=idx)
    return out


def _plain_logprobs_backward(s, dt):
    logp = s["logits"].float() - s["lse"][:, None]
    p = torch.exp(logp)
    has = s["labels"] >= 0
    g = torch.where(has, s["dlogp"], 0.0)
    d = -p * g[:, None]
    d.scatter_add_(1, s["labels"].clamp(min=0)[:, None], g[:, None])
    if s["dentropy"] is not None:
        d -= s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
    return dict(dlogits=d.to(dt))


def _plain_targets(s, rows):
    v = s["values"][rows] / s["case"]["temperature"]
    v = v - v.max(1, keepdim=True).values
    e = torch.exp(v)
    total = e.sum(1, keepdim=True)
    return e / total, v - torch.log(total)


def _plain_logits(s, rows):
    z = s["x"][rows].float() @ s["w"].float().T
    if s["bias"] is not None:
        z += s["bias"].float()
    return z / s["case"]["temperature"]


def _plain_distill(s, dt):
    rows = (s["idx"][:, 0] >= 0).nonzero()[:, 0]
    q, logq = _plain_targets(s, rows)
    z = _plain_logits(s, rows)
    most = z.max(1).values
    l = most + torch.log(torch.exp(z - most[:, None]).sum(1))
    logp = z.gather(1, s["idx"][rows]) - l[:, None]
    loss = torch.zeros(s["idx"].shape[0], device=z.device)
    lse = torch.zeros_like(loss)
    loss[rows] = (q * (logq - logp)).sum(1)
    lse[rows] = l
    return dict(loss=loss, lse=lse)


def _plain_distill_backward(s, dt):
    rows = (s["idx"][:, 0] >= 0).nonzero()[:, 0]
    q, _ = _plain_targets(s, rows)
    d = torch.exp(_plain_logits(s, rows).sub_(s["lse"][rows][:, None]))
    d.scatter_add_(1, s["idx"][rows], -q)
    d *= (s["dloss"][rows] / s["case"]["temperature"])[:, None]
    dx = torch.zeros(s["x"].shape, dtype=dt, device=d.device)
    dx[rows] = (d @ s["w"].float()).to(dt)
    out = dict(dx=dx, dw=(d.T @ s["x"][rows].float()).to(dt))
    if s["bias"] is not None:
        out["db"] = d.sum(0).to(dt)
    return out


PLAIN = {"norm": _plain_norm, "norm_q8": _plain_norm, "norm_backward": _plain_norm_backward, "linear_q8": _plain_linear_q8,
         "gated": _plain_gated, "gated_backward": _plain_gated_backward, "logprobs": _plain_logprobs,
         "logprobs_backward": _plain_logprobs_backward, "distill": _plain_distill, "distill_backward": _plain_distill_backward}


# ------------------------------------------------------------------------------------------
# the library's calls


def _library(s):
    import rope_cu_tile_gb300 as pk

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        if s["residual"] is None:
            return dict(y=pk.rms_norm(s["x"], s["w"], eps=EPS))
        y, h = pk.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS)
        return dict(y=y, h=h)
    if op == "norm_q8":
        if s["residual"] is None:
            q, scale = pk.rms_norm_q8(s["x"], s["w"], eps=EPS)
            return dict(q=q, scale=scale)
        q, scale, h = pk.rms_norm_q8(s["x"], s["w"], residual=s["residual"], eps=EPS)
        return dict(q=q, scale=scale, h=h)
    if op == "norm_backward":
        dx, dw = pk.rms_norm_backward(s["x"], s["w"], s["dy"], dh=s["dh"], eps=EPS)
        return dict(dx=dx, dw=dw)
    if op == "linear_q8":
        return dict(y=pk.linear_q8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], residual=s["residual"],
                                   act=case["act"], out_dtype=TYPES[case["dtype"]]))
    if op == "gated":
        got = pk.gated_linear(s["x"], s["w"], bias=s["bias"], act=case["act"], return_pre=case["pre"])
        return dict(y=got[0], pre=got[1]) if case["pre"] else dict(y=got)
    if op == "gated_backward":
        dx, dw, db = pk.gated_linear_backward(s["x"], s["w"], s["dy"], s["pre"], act=case["act"], need_db=case["bias"])
        return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)
    if op == "logprobs":
        logp, lse, entropy, top_logp, top_idx = pk.token_logprobs(s["logits"], s["labels"], top=min(case["top"], case["V"]))
        out = dict(logp=logp, lse=lse, entropy=entropy)
        return dict(out, top_logp=top_logp, top_idx=top_idx) if case["top"] else out
    if op == "logprobs_backward":
        return dict(dlogits=pk.token_logprobs_backward(s["logits"], s["labels"], s["lse"], s["entropy"], s["dlogp"],
                                                       dentropy=s["dentropy"]))
    if op == "distill":
        loss, lse = pk.distill(s["x"], s["w"], s["idx"], s["values"], bias=s["bias"], temperature=case["temperature"])
        return dict(loss=loss, lse=lse)
    dx, dw, db = pk.distill_backward(s["x"], s["w"], s["idx"], s["values"], s["lse"], s["dloss"], bias=s["bias"],
                                     temperature=case["temperature"])
    return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)


def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state, TYPES[state["case"]["dtype"]])


# ------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, e, T = case["op"], SIZE[case["dtype"]], case["T"]
    if op.startswith("norm"):
        D, r = case["D"], int(case["residual"])
        if op == "norm_backward":
            return dict(bytes=e * (T * D * (3 + r) + 2 * D), flops=10 * T * D)
        y = T * D + 4 * T if op == "norm_q8" else e * T * D
        return dict(bytes=y + e * (T * D * (1 + 2 * r) + D), flops=6 * T * D)
    if op == "linear_q8":
        K, N = case["K"], case["N"]
        return dict(bytes=T * K + N * K + 4 * (T + N) + e * (N * bool(case["bias"]) + T * N * (1 + bool(case["residual"]))),
                    flops=2 * T * N * K)
    if op.startswith("gated"):
        K, F = case["K"], case["F"]
        if op == "gated":
            return dict(bytes=e * (T * K + 2 * F * K + 2 * F * bool(case["bias"]) + T * F * (3 if case["pre"] else 1)),
                        flops=4 * T * F * K)
        return dict(bytes=e * (2 * T * K + 4 * F * K + 2 * F * bool(case["bias"]) + 3 * T * F), flops=8 * T * F * K)
    if op.startswith("logprobs"):
        V = case["V"]
        if op == "logprobs":
            return dict(bytes=e * T * V + T * (20 + 12 * min(case["top"], V)), flops=5 * T * V)
        return dict(bytes=2 * e * T * V + T * (20 + 4 * bool(case["entropy"])), flops=6 * T * V)
    D, V, A, top = case["D"], case["V"], _rows_with_targets(case), min(case["top"], case["V"])
    if op == "distill":
        return dict(bytes=e * (A * D + V * D + V * bool(case["bias"])) + 12 * A * top + 8 * T, flops=2 * A * V * D)
    return dict(bytes=e * (A * D + T * D + 2 * V * D + 2 * V * bool(case["bias"])) + 12 * A * top + 8 * T, flops=6 * A * V * D)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _wide_act(z, act):
    return {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0),
            "gelu": lambda: z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0)), "silu": lambda: z * torch.sigmoid(z)}[act]()


def _exact_norm(case, s):
    h = s["x"].double()
    if case["op"] == "norm_backward":
        h.requires_grad_(True)
        w = s["w"].double().requires_grad_(True)
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w
        value = (y * s["dy"].double()).sum()
        if s["dh"] is not None:
            value = value + (h * s["dh"].double()).sum()
        dx, dw = torch.autograd.grad(value, (h, w))
        return dict(dx=dx, dw=dw)
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].double()
    # (the 8-bit rows are a rounding of y / scale, not a number that 64 bits know better)
    out = dict(q=None, scale=y.abs().amax(1) / E4M3_MOST) if case["op"] == "norm_q8" else dict(y=y)
    return dict(out, h=h) if s["residual"] is not None else out


def _exact_linear_q8(case, s):
    z = torch.mm(s["x"].double(), s["w"].double().t()) * torch.outer(s["x_scale"].double(), s["w_scale"].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _wide_act(z, case["act"])
    return dict(y=y if s["residual"] is None else y + s["residual"].double())


def _exact_gated(case, s):
    F = case["F"]
    if case["op"] == "gated":
        z = torch.mm(s["x"].double(), s["w"].double().t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _wide_act(z[:, :F], case["act"]) * z[:, F:]
        return dict(y=y, pre=z) if case["pre"] else dict(y=y)
    z = s["pre"].double().requires_grad_(True)
    dz, = torch.autograd.grad((_wide_act(z[:, :F], case["act"]) * z[:, F:] * s["dy"].double()).sum(), z)
    out = dict(dx=torch.mm(dz, s["w"].double()), dw=torch.mm(dz.t(), s["x"].double()))
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out


def _exact_logprobs(case, s):
    parts = []
    for rows in torch.arange(case["T"], device="cuda").split(1024):
        z, labels = s["logits"][rows].double(), s["labels"][rows]
        at = labels.clamp(min=0)[:, None]
        if case["op"] == "logprobs":
            logp = torch.log_softmax(z, 1)
            got = [logp.gather(1, at)[:, 0] * (labels >= 0), torch.logsumexp(z, 1), -torch.xlogy(logp.exp(), logp.exp()).sum(1)]
            if case["top"]:
                best, idx = torch.sort(z, dim=1, descending=True, stable=True)
                top = min(case["top"], case["V"])
                got += [logp.gather(1, idx[:, :top]), idx[:, :top]]
        else:
            # with the lse and entropy that the call is given
            logp = z - s["lse"][rows].double()[:, None]
            one = torch.zeros_like(z).scatter_(1, at, 1.0)
            d = (s["dlogp"][rows].double() * (labels >= 0))[:, None] * (one - logp.exp())
            if s["dentropy"] is not None:
                d -= (s["dentropy"][rows].double())[:, None] * logp.exp() * (logp + s["entropy"][rows].double()[:, None])
            got = [d]
        parts.append(got)
    names = ["logp", "lse", "entropy", "top_logp", "top_idx"] if case["op"] == "logprobs" else ["dlogits"]
    return {name: torch.cat(list(column)) for name, column in zip(names, zip(*parts))}


def _exact_distill(case, s):
    T, tau = case["T"], case["temperature"]
    w = s["w"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dx = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    db = torch.zeros(case["V"], dtype=torch.float64, device="cuda")
    for part in torch.nonzero(s["idx"][:, 0] >= 0).flatten().split(4096):
        x, idx = s["x"][part].double(), s["idx"][part]
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        z /= tau
        logq = torch.log_softmax(s["values"][part].double() / tau, 1)
        if case["op"] == "distill":
            lse[part] = torch.logsumexp(z, 1)
            loss[part] = (logq.exp() * (logq - z.gather(1, idx) + lse[part][:, None])).sum(1)
            continue
        d = torch.exp(z - s["lse"][part].double()[:, None])
        d.scatter_add_(1, idx, -logq.exp())
        d *= s["dloss"][part].double()[:, None] / tau
        dx[part] = torch.mm(d, w)
        dw += torch.mm(d.t(), x)
        db += d.sum(0)
    if case["op"] == "distill":
        return dict(loss=loss, lse=lse)
    return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(case, s)
    if op == "linear_q8":
        return _exact_linear_q8(case, s)
    if op.startswith("gated"):
        return _exact_gated(case, s)
    return _exact_logprobs(case, s) if op.startswith("logprobs") else _exact_distill(case, s)
