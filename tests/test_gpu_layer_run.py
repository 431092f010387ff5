"""The operators as they are used together: a teacher's batch scored and its likeliest words kept, a pre-norm encoder layer with a
gated feed-forward distilled from them, forwards and backwards against 64-bit autograd; and the layer's 8-bit form."""

import json
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

LENS = [40, 1, 70, 128, 33]
H, F, V, TOP, TAU = 2, 160, 700, 12, 2.0
D = H * 64


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def tables(dtype):
    pos, t = torch.arange(max(LENS), device="cuda").double()[:, None], torch.arange(32, device="cuda").double()
    a = pos / 10000.0 ** (t / 32)
    return a.cos().to(dtype), a.sin().to(dtype)


def weights(gen, dtype):
    p = dict(n1=1 + rand(gen, D, std=0.1), qkv=rand(gen, 3 * D, D, std=D**-0.5), o=rand(gen, D, D, std=D**-0.5), n2=1 + rand(gen, D, std=0.1),
             up=rand(gen, 2 * F, D, std=D**-0.5), down=rand(gen, D, F, std=F**-0.5), n3=1 + rand(gen, D, std=0.1),
             head=rand(gen, V, D, std=2 * D**-0.5))
    return {k: v.to(dtype) for k, v in p.items()}


def layer(x, p, cos, sin):
    """The final norm's output in 64 bits."""
    norm = lambda h, w: h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    qkv = norm(x, p["n1"]) @ p["qkv"].T
    q, k, v = (t.reshape(-1, H, 64) for t in qkv.split(D, 1))
    out, start = [], 0
    for L in LENS:
        s = slice(start, start + L)
        start += L
        c, sn = cos[:L, None].double(), sin[:L, None].double()
        rot = lambda t: torch.cat([t[..., :32] * c - t[..., 32:] * sn, t[..., :32] * sn + t[..., 32:] * c], -1)  # noqa: E731
        score = torch.einsum("ihd,jhd->hij", rot(q[s]), rot(k[s])) / 8
        out.append(torch.einsum("hij,jhd->ihd", score.softmax(-1), v[s]).reshape(L, D))
    h = x + torch.cat(out) @ p["o"].T
    g, u = (norm(h, p["n2"]) @ p["up"].T).chunk(2, 1)
    h = h + (torch.nn.functional.gelu(g) * u) @ p["down"].T
    return norm(h, p["n3"])


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-4), (torch.bfloat16, 6e-2), (torch.float16, 8e-3)])
def test_distil_a_layer(pk, dtype, tol):
    """tol: of the norm of each result. A value passes some ten roundings (u each, 2^-8, 2^-11) or, in fp32, attention held to
    1e-4, on its way and as many on the gradient's way back."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    T = sum(LENS)
    cu = torch.tensor([0] + torch.tensor(LENS).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    cos, sin = tables(dtype)
    p, x = weights(gen, dtype), rand(gen, T, D, dtype=dtype)
    # the teacher: its logits scored, the likeliest words kept where there is a token to learn
    teacher = pk.linear(rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=2 * D**-0.5, dtype=dtype))
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    logp, _, entropy, values, idx = pk.token_logprobs(teacher, labels, top=TOP)
    t64 = torch.log_softmax(teacher.double(), 1)
    assert torch.equal(idx, torch.sort(teacher.double(), dim=1, descending=True, stable=True).indices[:, :TOP])
    assert float((logp.double() - t64.gather(1, labels[:, None])[:, 0]).abs().max()) < 1e-5
    assert float((entropy.double() + (t64.exp() * t64).sum(1)).abs().max()) < 1e-5
    idx[::3] = -1
    count = int((idx[:, 0] >= 0).sum())
    # the student, forwards
    y1 = pk.rms_norm(x, p["n1"])
    qkv = pk.linear(y1, p["qkv"])
    att, alse = pk.attend(qkv, cos, sin, cu, H, 0, 0.125)
    branch = pk.linear(att, p["o"])
    y2, h = pk.rms_norm(branch, p["n2"], residual=x)
    a, pre = pk.gated_linear(y2, p["up"], act="gelu", return_pre=True)
    branch2 = pk.linear(a, p["down"])
    y3, h3 = pk.rms_norm(branch2, p["n3"], residual=h)
    loss, lse = pk.distill(y3, p["head"], idx, values, temperature=TAU)
    dloss = torch.full((T,), TAU**2 / count, device="cuda")
    # and backwards
    dy3, dhead, _ = pk.distill_backward(y3, p["head"], idx, values, lse, dloss, temperature=TAU)
    dh3, dn3 = pk.rms_norm_backward(h3, p["n3"], dy3)
    da, ddown, _ = pk.linear_backward(a, p["down"], dh3, need_db=False)
    dy2, dup, _ = pk.gated_linear_backward(y2, p["up"], da, pre, "gelu", need_db=False)
    dh, dn2 = pk.rms_norm_backward(h, p["n2"], dy2, dh=dh3)
    datt, do, _ = pk.linear_backward(att, p["o"], dh, need_db=False)
    dqkv = pk.attend_backward(qkv, cos, sin, cu, H, 0, 0.125, att, alse, datt)
    dy1, dqkv_w, _ = pk.linear_backward(y1, p["qkv"], dqkv, need_db=False)
    dx, dn1 = pk.rms_norm_backward(x, p["n1"], dy1, dh=dh)
    assert pk.last_status() == 0
    # the same in 64 bits
    P = {k: v.double().requires_grad_(True) for k, v in p.items()}
    X = x.double().requires_grad_(True)
    z = layer(X, P, cos, sin) @ P["head"].T / TAU
    q, Q, has = ref.targets(idx, values, TAU, V)
    want = (torch.xlogy(Q, Q) - Q * torch.log_softmax(z, 1)).sum(1) * has
    grads = torch.autograd.grad((want * dloss.double()).sum(), [X] + [P[k] for k in ("n1", "qkv", "o", "n2", "up", "down", "n3", "head")])
    near = lambda g, v: float((g.double() - v).norm()) <= tol * float(v.norm())  # noqa: E731
    assert near(loss, want.detach())
    for name, g, v in zip(("x", "n1", "qkv", "o", "n2", "up", "down", "n3", "head"), (dx, dn1, dqkv_w, do, dn2, dup, ddown, dn3, dhead), grads):
        assert near(g, v), name


def test_layer_in_8_bits(pk):
    """The feed-forward of a layer served in 8 bits, rows and weights: each product's operands are off by 2^-4 of an element at
    most, independently, so its result by 2^-4 sqrt(2) / sqrt(3) of its norm at worst (uniform errors); two of them in a row."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    for T in (1, 3, 200):
        p, x, r = weights(gen, torch.bfloat16), rand(gen, T, D, dtype=torch.bfloat16), rand(gen, T, D, dtype=torch.bfloat16)
        up, down = p["up"][:F].contiguous(), p["down"]
        uq, us = pk.quantize_rows(up)
        dq, ds = pk.quantize_rows(down)
        q, s, h = pk.rms_norm_q8(x, p["n1"], residual=r)
        a = pk.linear_q8(q, s, uq, us, act="gelu")
        aq, as_ = pk.quantize_rows(a)
        y = pk.linear_q8(aq, as_, dq, ds, residual=h)
        H64 = x.double() + r.double()
        n = H64 / torch.sqrt(H64.square().mean(1, keepdim=True) + 1e-6) * p["n1"].double()
        want = torch.nn.functional.gelu(n @ up.double().T) @ down.double().T
        off = float((y.double() - H64 - want).norm()) / float(want.norm())
        assert off <= 2 * 2.0**-4 * math.sqrt(2 / 3) + 2.0**-6
    assert pk.last_status() == 0


_STALL_SCRIPT = """
import json, os, sys
sys.path.insert(0, os.getcwd())
import torch
import rope_cu_tile_gb300 as pk

torch.manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
got = []
for T in (40, 3000):
    x, w = r(T, 256), r(512, 256)
    xq, xs = pk.quantize_rows(x)
    wq, ws = pk.quantize_rows(w)
    idx = torch.randint(0, 512, (T, 3), device="cuda")
    v = torch.randn(T, 3, device="cuda")
    for call in (lambda: pk.gated_linear(x, w), lambda: pk.linear_q8(xq, xs, wq, ws), lambda: pk.distill(x, w, idx, v)[0]):
        want = call()
        torch.cuda.synchronize()
        os.environ["PK_DEBUG_SKIP_ARRIVE"] = "1"
        call()
        torch.cuda.synchronize()
        del os.environ["PK_DEBUG_SKIP_ARRIVE"]
        word = pk.last_status()
        after = call()
        torch.cuda.synchronize()
        got.append([word, pk.last_status(), bool(torch.equal(after, want))])
print(json.dumps(got))
"""


def test_withheld_stage_times_out_and_the_context_stays_usable():
    env = {k: v for k, v in os.environ.items() if k != "PK_DEBUG_SKIP_ARRIVE"}
    env["PK_TIMEOUT_MS"] = "100"
    p = subprocess.run([sys.executable, "-c", _STALL_SCRIPT], env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    assert json.loads(p.stdout.strip().splitlines()[-1]) == [[6, 0, True]] * 6


def test_two_calls_at_once(pk):
    """The same operators on two streams at the same time, and two captured graphs replayed side by side: no scratch is shared."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    dt = torch.bfloat16

    def inputs():
        T = 700
        idx = torch.randint(0, V, (T, 5), generator=gen, device="cuda")
        return dict(x=rand(gen, T, D, dtype=dt), w=rand(gen, D, dtype=dt), up=rand(gen, 2 * F, D, std=D**-0.5, dtype=dt), dy=rand(gen, T, F, dtype=dt),
                    head=rand(gen, V, D, std=D**-0.5, dtype=dt), idx=idx, values=rand(gen, T, 5), g=rand(gen, T))

    def run(i):
        y = pk.rms_norm(i["x"], i["w"])
        a, pre = pk.gated_linear(y, i["up"], return_pre=True)
        dx, dw, _ = pk.gated_linear_backward(y, i["up"], i["dy"], pre)
        dn = pk.rms_norm_backward(i["x"], i["w"], dx)
        loss, lse = pk.distill(y, i["head"], i["idx"], i["values"])
        dd = pk.distill_backward(y, i["head"], i["idx"], i["values"], lse, i["g"])
        return (a, dw, *dn, loss, dd[0], dd[1])

    ins = [inputs(), inputs()]
    want = [[t.clone() for t in run(i)] for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = []
    for s, i in zip(streams, ins):
        with torch.cuda.stream(s):
            got.append(run(i))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs, outs = [], []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(i))
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w))
