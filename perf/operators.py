"""The token-row operators of a packed encoder as measured cases: the projection with its epilogue (`linear`), dropout
from a counter-based generator (`dropout`), and the softmax cross entropy over a vocabulary (`xent`).

Each case names its operator and direction (`op`), element type and sizes. `run` computes one pass either with the
library's entry points (`own`) or in a plain form of elementary torch operations in 32 bits; `exact` computes the same
from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IGNORED = -100


def listed():
    return [
        # one token through a feed-forward's first projection: serving, bound by latency and the weight's bytes
        dict(name="linear_token", op="linear", dtype="bf16", T=1, K=1024, N=4096, act="gelu", bias=True, residual=False,
             pre=False, p=0.0),
        # the smallest packed batch, in fp32: an attention's output projection back into the residual stream
        dict(name="linear_tiny_f32", op="linear", dtype="f32", T=251, K=768, N=768, act="none", bias=True, residual=True,
             pre=False, p=0.0),
        # the packed qkv of twelve heads
        dict(name="linear_qkv_global", op="linear", dtype="bf16", T=16931, K=768, N=2304, act="none", bias=True,
             residual=False, pre=False, p=0.0),
        # a feed-forward's second projection in training: dropout on the branch, then the residual stream
        dict(name="linear_down_local", op="linear", dtype="f16", T=72804, K=2048, N=768, act="none", bias=True,
             residual=True, pre=False, p=0.1),
        # a feed-forward's first projection in training, on the longest batch: the pre-activation is kept for the backward
        dict(name="linear_up_long", op="linear", dtype="bf16", T=131072, K=1024, N=4096, act="gelu", bias=True,
             residual=False, pre=True, p=0.0),
        # a small classifier's hidden layer with odd sizes
        dict(name="linear_backward_odd", op="linear_backward", dtype="f16", T=1021, K=515, N=1003, act="relu", bias=True, p=0.0),
        # the feed-forward's first projection in training, backwards
        dict(name="linear_backward_short", op="linear_backward", dtype="bf16", T=65536, K=768, N=2048, act="gelu", bias=True,
             p=0.1),
        # the gradient of a branch's dropout on the smallest batch, in fp32
        dict(name="dropout_backward_tiny", op="dropout_backward", dtype="f32", T=251, N=768, p=0.1),
        # a branch's dropout and the residual stream on the longest batch
        dict(name="dropout_long", op="dropout", dtype="bf16", T=131072, N=1024, residual=True, p=0.1),
        # scoring a small batch over an odd vocabulary
        dict(name="xent_small", op="xent", dtype="f16", T=640, D=768, V=32003, bias=False, labelled=1.0),
        # a training loss with every token labelled
        dict(name="xent_long", op="xent", dtype="bf16", T=65536, D=1024, V=32768, bias=True, labelled=1.0),
        # masked-token training: one token in seven has a label
        dict(name="xent_backward_masked", op="xent_backward", dtype="bf16", T=16931, D=768, V=50000, bias=True, labelled=0.15),
    ]


MOST_FLOPS = 2.0 * 65536 * 1024 * 32768  # of xent_long, the largest listed case
MOST_DROPPED = 131072 * 1024  # of dropout_long, the most elements a listed case draws bits for


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; in one of two cases a multiple of eight."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 16:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "dropout", "dropout_backward", "xent", "xent_backward"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]))
    p = rng.choice([0.0, round(rng.uniform(0.02, 0.5), 3)])
    if op.startswith("linear"):
        case.update(T=_between(rng, 1, 131072), K=_between(rng, 64, 4096), N=_between(rng, 64, 4096),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7, p=p)
        if op == "linear":
            case.update(residual=rng.random() < 0.5, pre=rng.random() < 0.3)
        cost = (2.0 if op == "linear" else 4.0) * case["N"] * case["K"]
    elif op.startswith("dropout"):
        case.update(T=_between(rng, 1, 131072), N=_between(rng, 1, 4096), p=p or 0.1)
        if op == "dropout":
            case.update(residual=rng.random() < 0.5)
        case["T"] = max(1, min(case["T"], MOST_DROPPED // case["N"]))
        return case
    else:
        case.update(T=_between(rng, 1, 65536), D=_between(rng, 64, 2048), V=_between(rng, 100, 130000),
                    bias=rng.random() < 0.5, labelled=rng.choice([1.0, 0.9, 0.15]))
        cost = (2.0 if op == "xent" else 6.0) * case["D"] * case["V"]
    # fp32 in 64 bits and in the plain form is the dearest: no case over a fifth of the largest listed one
    case["T"] = max(1, min(case["T"], int(0.2 * MOST_FLOPS / cost)))
    if p and "p" in case:
        case["T"] = max(1, min(case["T"], MOST_DROPPED // case["N"]))
    return case


def _labelled_rows(case):
    return int(round(case["labelled"] * case["T"]))


def prepare(case, seed):
    dt, dev = TYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    op, T = case["op"], case["T"]
    s = dict(case=case, residual=None)
    if "p" in case:
        # a training loop's generator state: one seed for the run, one offset for each layer and step
        s.update(p=case["p"], seed=(seed * 2654435761 + 12345) % (1 << 62), offset=seed % 1000003 + (5 << 33))
    if op.startswith("linear"):
        K, N = case["K"], case["N"]
        s["x"] = normal(T, K)
        s["w"] = normal(N, K, std=K**-0.5)
        if op == "linear":
            s["bias"] = normal(N, std=0.1) if case["bias"] else None
            s["residual"] = normal(T, N) if case["residual"] else None
        else:
            s["dy"] = normal(T, N, std=1e-2)
            s["pre"] = normal(T, N) if case["act"] != "none" else None
    elif op.startswith("dropout"):
        s["x"] = normal(T, case["N"], std=1.0 if op == "dropout" else 1e-2)
        s["residual"] = normal(T, case["N"]) if case.get("residual") else None
    else:
        D, V = case["D"], case["V"]
        s["x"] = normal(T, D)
        s["w"] = normal(V, D, std=2.0 * D**-0.5)
        s["bias"] = normal(V, std=0.3) if case["bias"] else None
        labels = torch.randint(0, V, (T,), generator=g, device=dev)
        order = torch.rand(T, generator=g, device=dev).argsort()
        labels[order[_labelled_rows(case):]] = IGNORED
        s["labels"] = labels
        if op == "xent_backward":
            # the forward's lse, and the gradient of a mean over the labelled rows
            rows = (labels >= 0).nonzero()[:, 0]
            lse = torch.zeros(T, device=dev)
            for part in rows.split(8192):
                z = s["x"][part].float() @ s["w"].float().T
                if case["bias"]:
                    z += s["bias"].float()
                lse[part] = torch.logsumexp(z, 1)
            s["lse"] = lse
            weight = torch.rand(T, generator=g, device=dev) + 0.5
            s["dloss"] = weight / max(1, _labelled_rows(case))
    return s


# ------------------------------------------------------------------------------------------
# the plain form


def _keep(T, N, p, seed, offset, device):
    """The truth values [T, N] of the kept elements: Philox4x32-10 at counter (col / 8, row, offset), key seed, the 16-bit
    pieces of its four words in order, kept where a piece is at least p in steps of 2^-16."""
    M32 = 0xFFFFFFFF
    c0 = torch.arange((N + 7) // 8, device=device, dtype=torch.int64)[None, :].expand(T, -1)
    c1 = torch.arange(T, device=device, dtype=torch.int64)[:, None].expand(-1, (N + 7) // 8)
    c2 = torch.full_like(c0, offset & M32)
    c3 = torch.full_like(c0, (offset >> 32) & M32)
    k0, k1 = seed & M32, (seed >> 32) & M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([c0, c1, c2, c3], -1)
    bits = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(T, -1)[:, :N]
    return bits >= _step(p)


def _step(p):
    return int(math.floor(p * 65536 + 0.5))


def _dropped(x, s):
    if _step(s["p"]) == 0:
        return x
    keep = _keep(x.shape[0], x.shape[1], s["p"], s["seed"], s["offset"], x.device)
    return torch.where(keep, x * (65536.0 / (65536 - _step(s["p"]))), torch.zeros((), device=x.device))


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
    h = 1.0 / (1.0 + torch.exp(-z))
    return h * (1.0 + z * (1.0 - h))


def _plain_linear(s, dt):
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _dropped(_act(z, s["case"]["act"]), s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return dict(y=y.to(dt), pre=z.to(dt)) if s["case"]["pre"] else dict(y=y.to(dt))


def _plain_linear_backward(s, dt):
    d = _dropped(s["dy"].float(), s)
    if s["pre"] is not None:
        d = d * _act_slope(s["pre"].float(), s["case"]["act"])
    out = dict(dx=(d @ s["w"].float()).to(dt), dw=(d.T @ s["x"].float()).to(dt))
    if s["case"]["bias"]:
        out["db"] = d.sum(0).to(dt)
    return out


def _plain_logits(s, rows):
    z = s["x"][rows].float() @ s["w"].float().T
    return z if s["bias"] is None else z.add_(s["bias"].float())


def _plain_xent(s, dt):
    labels = s["labels"]
    rows = (labels >= 0).nonzero()[:, 0]
    z = _plain_logits(s, rows)
    top = z.max(1).values
    picked = z.gather(1, labels[rows][:, None])[:, 0]
    l = top + torch.log(torch.exp(z.sub_(top[:, None])).sum(1))
    loss = torch.zeros(labels.shape[0], device=z.device)
    lse = torch.zeros_like(loss)
    loss[rows] = l - picked
    lse[rows] = l
    return dict(loss=loss, lse=lse)


def _plain_xent_backward(s, dt):
    labels = s["labels"]
    rows = (labels >= 0).nonzero()[:, 0]
    d = torch.exp(_plain_logits(s, rows).sub_(s["lse"][rows][:, None]))
    d[torch.arange(rows.shape[0], device=d.device), labels[rows]] -= 1.0
    d *= s["dloss"][rows][:, None]
    dx = torch.zeros(s["x"].shape, dtype=dt, device=d.device)
    dx[rows] = (d @ s["w"].float()).to(dt)
    out = dict(dx=dx, dw=(d.T @ s["x"][rows].float()).to(dt))
    if s["bias"] is not None:
        out["db"] = d.sum(0).to(dt)
    return out


def _plain(s):
    case = s["case"]
    dt, op = TYPES[case["dtype"]], case["op"]
    if op == "linear":
        return _plain_linear(s, dt)
    if op == "linear_backward":
        return _plain_linear_backward(s, dt)
    if op.startswith("dropout"):
        y = _dropped(s["x"].float(), s)
        return dict(y=(y if s["residual"] is None else y + s["residual"].float()).to(dt))
    return _plain_xent(s, dt) if op == "xent" else _plain_xent_backward(s, dt)


# ------------------------------------------------------------------------------------------
# the library's calls


def _library(s):
    import rope_cu_tile_gb300 as pk

    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        got = pk.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=case["act"], p=s["p"], seed=s["seed"],
                        offset=s["offset"], return_pre=case["pre"])
        return dict(y=got[0], pre=got[1]) if case["pre"] else dict(y=got)
    if op == "linear_backward":
        dx, dw, db = pk.linear_backward(s["x"], s["w"], s["dy"], pre=s["pre"], act=case["act"], p=s["p"], seed=s["seed"],
                                        offset=s["offset"], need_db=case["bias"])
        return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)
    if op == "dropout":
        return dict(y=pk.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"]))
    if op == "dropout_backward":
        return dict(y=pk.dropout_backward(s["x"], s["p"], s["seed"], s["offset"]))
    if op == "xent":
        loss, lse = pk.cross_entropy(s["x"], s["w"], s["labels"], bias=s["bias"])
        return dict(loss=loss, lse=lse)
    dx, dw, db = pk.cross_entropy_backward(s["x"], s["w"], s["labels"], s["lse"], s["dloss"], bias=s["bias"])
    return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, e, T = case["op"], SIZE[case["dtype"]], case["T"]
    if op.startswith("dropout"):
        n = T * case["N"]
        return dict(bytes=e * n * (3 if case.get("residual") else 2), flops=2 * n)
    if op == "linear":
        K, N = case["K"], case["N"]
        rows = 1 + bool(case["residual"]) + bool(case["pre"])
        return dict(bytes=e * (T * K + N * K + N * bool(case["bias"]) + rows * T * N), flops=2 * T * N * K)
    if op == "linear_backward":
        K, N = case["K"], case["N"]
        rows = 1 + (case["act"] != "none")
        return dict(bytes=e * (2 * T * K + 2 * N * K + N * bool(case["bias"]) + rows * T * N), flops=4 * T * N * K)
    D, V, A = case["D"], case["V"], _labelled_rows(case)
    if op == "xent":
        return dict(bytes=e * (A * D + V * D + V * bool(case["bias"])) + 16 * T, flops=2 * A * V * D)
    return dict(bytes=e * (A * D + T * D + 2 * V * D + 2 * V * bool(case["bias"])) + 16 * T, flops=6 * A * V * D)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _philox_word_pairs(T, N, seed, offset):
    """uint16 [T, 8 ceil(N / 8)]: the generator's pieces, in numpy's unsigned 64-bit arithmetic."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    groups = (N + 7) // 8
    x = [np.tile(np.arange(groups, dtype=u), T), np.repeat(np.arange(T, dtype=u), groups)]
    x += [np.full(T * groups, (offset >> s) & 0xFFFFFFFF, dtype=u) for s in (0, 32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        first, second = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(second >> half) ^ x[1] ^ u(key[0]), second & low, (first >> half) ^ x[3] ^ u(key[1]), first & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    out = np.empty((T * groups, 8), dtype=np.uint16)
    for i, w in enumerate(x):
        out[:, 2 * i] = (w & u(0xFFFF)).astype(np.uint16)
        out[:, 2 * i + 1] = (w >> u(16)).astype(np.uint16)
    return out.reshape(T, groups * 8)


def _factor(case, s, N):
    """float64 [T, N]: what dropout multiplies each element by; None for p = 0."""
    cut = int(math.floor(case["p"] * 65536 + 0.5))
    if cut == 0:
        return None
    kept = torch.from_numpy(_philox_word_pairs(case["T"], N, s["seed"], s["offset"])[:, :N].astype(np.int32)).cuda() >= cut
    return kept.double() / (1.0 - cut / 65536.0)


def _normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op.startswith("dropout"):
        y = s["x"].double() * _factor(case, s, case["N"])
        return dict(y=y if s["residual"] is None else y + s["residual"].double())
    if op == "linear":
        z = torch.mm(s["x"].double(), s["w"].double().t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0), "gelu": lambda: z * _normal_cdf(z),
             "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        f = _factor(case, s, case["N"])
        if f is not None:
            y = y * f
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return dict(y=y, pre=z) if case["pre"] else dict(y=y)
    if op == "linear_backward":
        dz = s["dy"].double()
        f = _factor(case, s, case["N"])
        if f is not None:
            dz = dz * f
        if s["pre"] is not None:
            z = s["pre"].double()
            if case["act"] == "relu":
                dz = torch.where(z > 0, dz, 0.0)
            elif case["act"] == "gelu":
                dz = dz * (_normal_cdf(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi))
            else:
                sg = torch.sigmoid(z)
                dz = dz * (sg + z * sg * torch.sigmoid(-z))
        out = dict(dx=torch.mm(dz, s["w"].double()), dw=torch.mm(dz.t(), s["x"].double()))
        if case["bias"]:
            out["db"] = dz.sum(0)
        return out
    # the loss, some rows at a time
    rows = torch.nonzero(s["labels"] >= 0).flatten()
    w = s["w"].double()
    b = None if s["bias"] is None else s["bias"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dx = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    db = torch.zeros(case["V"], dtype=torch.float64, device="cuda")
    for part in torch.split(rows, 4096):
        x = s["x"][part].double()
        z = torch.mm(x, w.t())
        if b is not None:
            z += b
        at = s["labels"][part]
        if op == "xent":
            lse[part] = torch.logsumexp(z, 1)
            loss[part] = lse[part] - z[torch.arange(len(part), device="cuda"), at]
            continue
        q = torch.exp(z - s["lse"][part].double()[:, None])
        q[torch.arange(len(part), device="cuda"), at] -= 1.0
        q *= s["dloss"][part].double()[:, None]
        dx[part] = torch.mm(q, w)
        dw += torch.mm(q.t(), x)
        db += q.sum(0)
    if op == "xent":
        return dict(loss=loss, lse=lse)
    return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)
