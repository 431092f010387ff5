"""The token-row operators at the edges of their types: tails and infinities of the activations, values near the ends of fp16
and fp32, masked words, padding rows, long features, pieces of the vocabulary, the streams' status words, bounded waits."""

import math

import pytest

torch = pytest.importorskip("torch")

import rows_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF, NAN = float("inf"), float("nan")


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(4321)
    return g


def rounded(err, want, dtype):
    """The bound of a value off by err before its rounding to the type (fp16: half a step of its smallest numbers)."""
    return err * (1 + ref.U[dtype]) + ref.U[dtype] * want.abs() + (2.0**-25 if dtype == torch.float16 else 0.0)


# ------------------------------------------------------------------------------------------ activations


def act_of(pk, z, act, rows):
    """act at the values z: a product of nothing, z its bias."""
    x, w = torch.ones(rows, 8, dtype=z.dtype, device="cuda"), torch.zeros(z.numel(), 8, dtype=z.dtype, device="cuda")
    return pk.linear(x, w, z, act=act)


def slope_of(pk, z, act, d=1.0):
    """act' at the values z: db of one row (the sum of one dz, rounded once)."""
    n, dt = z.numel(), z.dtype
    x, w = torch.ones(1, 8, dtype=dt, device="cuda"), torch.zeros(n, 8, dtype=dt, device="cuda")
    dy = torch.full((1, n), d, dtype=dt, device="cuda")
    return pk.linear_backward(x, w, dy, z[None].contiguous(), act, need_dx=False, need_dw=False)[2]


def tail_and_density(z):
    u = z.abs()
    return 0.5 * torch.special.erfc(u / math.sqrt(2)), u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)

@pytest.mark.parametrize("dtype", TYPES)
def test_gelu_slope_keeps_its_tail(pk, dtype):
    """gelu' of z < 0 is h = Phi(-u) - u phi(u), u = -z, of z > 0 1 - h. Relative errors of the two terms, 0 <= u <= 6:
    16 bits: Phi by the fit, 2^-17; phi by an exponential whose argument's base-2 logarithm (at most 26) is off by three
    roundings, 26 * 3 * 2^-24 * ln 2 < 2^-18, and the function's 2^-22. fp32: the complementary error function's four units
    of 2^-23 and its argument's 1.5 2^-24 relative, which is 1.5 u^2 2^-24 of the value; phi as above or better."""
    z = torch.linspace(-6, 6, 4801, device="cuda").to(dtype)
    want = ref.act_slope(z.double(), "gelu")
    tail, dens = tail_and_density(z.double())
    if dtype == torch.float32:
        err = tail * (2.0**-21 + 1.5 * z.double() ** 2 * 2.0**-24) + dens * (2.0**-18 + 2.0**-22)
    else:
        err = tail * 2.0**-17 + dens * (2.0**-18 + 2.0**-22)
    err = err + 2.0**-23 * torch.where(z < 0, tail + dens, 2.0)  # the additions
    assert ref.worst(slope_of(pk, z, "gelu"), want, rounded(err, want, dtype)) <= 1
    far = torch.linspace(-60, -6, 500, device="cuda").to(dtype)
    # |gelu'(-6)| = 3.6e-8, and it falls (fp16: to the nearest multiple of 2^-24, at most half a step further)
    assert float(slope_of(pk, far, "gelu").double().abs().max()) <= 4e-8 + (2.0**-25 if dtype == torch.float16 else 0.0)

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act,value,slope", [("relu", (0.0, INF), (0.0, 1.0)), ("gelu", (0.0, INF), (0.0, 1.0)),
                                             ("silu", (0.0, INF), (0.0, 1.0))])
def test_limits_at_infinity(pk, dtype, act, value, slope):
    """Values and slopes of infinite and of the largest finite pre-activations are their limits; NaN stays NaN."""
    top = torch.finfo(dtype).max
    z = torch.tensor([-INF, INF, -top, top, NAN, 1.0], dtype=dtype, device="cuda")
    for rows in (1, 9, 300):
        y = act_of(pk, z, act, rows).float().cpu()
        assert bool((y[:, 0] == value[0]).all()) and bool((y[:, 1] == value[1]).all()), y[0]
        assert bool((y[:, 2] == 0).all()) and bool((y[:, 3] == top).all()) and bool(y[:, 4].isnan().all())
    d = slope_of(pk, z, act).float().cpu()
    assert d[0] == slope[0] and d[1] == slope[1] and d[2] == 0 and d[3] == 1 and d[4].isnan(), d
    d = slope_of(pk, z[:4], act, 0.0)
    assert bool((d == 0).all())


def test_half_precision_overflow_of_the_kept_pre_activation(pk):
    """z = -80000 is finite in fp32 and -inf in fp16: y is 0, and so is every gradient."""
    x, w = torch.full((9, 8), 200.0, device="cuda").half(), torch.full((16, 8), -50.0, device="cuda").half()
    for act in ("gelu", "silu"):
        y, pre = pk.linear(x, w, act=act, return_pre=True)
        assert bool((y == 0).all()) and bool((pre == -INF).all())
        for g in pk.linear_backward(x, w, torch.ones_like(y), pre, act, p=0.25, seed=3):
            assert bool((g == 0).all()), act

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_are_as_exact_as_their_type(pk, dtype, act):
    """Relative to the terms of each value. fp32: the complementary error function of at most four units of 2^-23 on an argument
    off by 1.5 2^-24 of itself; exponentials of at most two units, one addition and one division. 16 bits: as the fit (2^-17) and the short exponentials (2^-22, the argument
    times log2 e off by 1.5 2^-24 of itself) allow; gelu's fit holds to 6."""
    lo = 6 if act == "gelu" else 20
    z = torch.linspace(-lo, lo, 4001, device="cuda").to(dtype)
    u = z.double().abs()
    f32 = dtype == torch.float32
    want = ref.act(z.double(), act)
    slope = ref.act_slope(z.double(), act)
    if act == "gelu":
        tail, dens = tail_and_density(z.double())
        t = 2.0**-21 + 1.5 * u * u * 2.0**-24 if f32 else 2.0**-17  # of Phi(-u)
        g = 2.0**-22 + u * u * 2.0**-24 if f32 else 2.0**-18 + 2.0**-22  # of phi(u)
        err = u * tail * t + 4 * 2.0**-24 * want.abs()
        serr = tail * t + dens * g + 2.0**-23 * torch.where(z < 0, tail + dens, 2.0)
    else:
        h = torch.sigmoid(z.double())
        r = 4 * 2.0**-23 if f32 else (1.5 * u + 16) * 2.0**-24  # of h
        err = want.abs() * r
        # 1 - h: of itself in fp32, as the difference of the rounded h in 16 bits
        serr = h * ((1 + u * (1 - h)) * (r + 2.0**-22) + (0.0 if f32 else u * h * (r + 2.0**-24)))
    for rows in (1, 9):
        y = act_of(pk, z, act, rows)
        assert ref.worst(y[rows - 1], want, rounded(err, want, dtype)) <= 1
    assert ref.worst(slope_of(pk, z, act), slope, rounded(serr, slope, dtype)) <= 1

@pytest.mark.parametrize("act,p", [("none", 0.5), ("gelu", 0.0), ("silu", 0.25), ("relu", 0.4), ("relu", 0.0)])
@pytest.mark.parametrize("size", [3e-8, 1e-6, 1e-4, 2.0**-10, 0.03, 1.0, 3e4])
def test_half_precision_gradients_keep_their_range(pk, gen, act, p, size):
    """dz in fp16 is scaled by a power of two where its largest element would be past 65504, or below 2^-10 (where half a
    step of fp16's smallest numbers, 2^-25, would be over 2^-15 of it): so each element is off by 2^-11 of itself or
    2^-15 of the largest one, whichever is more, and the products as everywhere."""
    T, K, N, dt = 300, 72, 136, torch.float16
    x, w = rand(gen, T, K, std=0.05, dtype=dt), rand(gen, N, K, std=0.05, dtype=dt)
    dy = (torch.rand(T, N, generator=gen, device="cuda") * 2 - 1).mul_(2 * size).to(dt)
    pre = None if act == "none" else rand(gen, T, N, dtype=dt)
    got = pk.linear_backward(x, w, dy, pre, act, p, 5, 6)
    d = dy.double() * ref.drop_factor(T, N, p, 5, 6, "cuda")
    err = 2.0**-22 * d.abs()
    if act != "none":
        z = pre.double()
        err = err * ref.LIPSCHITZ + (2.0**-16 * (1 + z.abs()) * d.abs() if act != "relu" else 0.0)
        d = d * ref.act_slope(z, act)
    rd = err + torch.maximum(ref.U[dt] * d.abs(), 2.0**-15 * d.abs().max())
    X, W = x.double(), w.double()
    want = (d @ W, d.T @ X, d.sum(0))
    ex = rd @ W.abs() + ref.sum_bound(N, dt) * ((d.abs() + rd) @ W.abs())
    ew = rd.T @ X.abs() + ref.sum_bound(T, dt) * ((d.abs() + rd).T @ X.abs())
    eb = err.sum(0) + T * 2.0**-23 * d.abs().sum(0)
    for name, g, v, e in zip(("dx", "dw", "db"), got, want, (ex, ew, eb)):
        fits = v.abs() < 65000
        assert ref.worst(g[fits], v[fits], rounded(e, v, dt)[fits]) <= 1, name
    assert pk.last_status() == 0


def test_half_precision_gradients_beside_an_infinite_one(pk, gen):
    """One infinite dy: its own row of dx, and db and dw of its column; the rest as without it, with a dz past 65504 beside it."""
    T, K, N, dt = 40, 16, 24, torch.float16
    x, w = rand(gen, T, K, std=0.01, dtype=dt), rand(gen, N, K, std=0.01, dtype=dt)
    dy = rand(gen, T, N, dtype=dt)
    dy[2, 3] = 60000.0
    keep = torch.from_numpy(ref.keep_mask(T, N, 0.5, 1, 2)).cuda()
    dy[~keep] = 1.0
    at = int(keep[7].nonzero()[0])
    a = pk.linear_backward(x, w, dy, p=0.5, seed=1, offset=2)
    dy[7, at] = INF
    b = pk.linear_backward(x, w, dy, p=0.5, seed=1, offset=2)
    rows, cols = torch.arange(T, device="cuda") != 7, torch.arange(N, device="cuda") != at
    assert bool(a[0].isfinite().all()) and bool(a[1].isfinite().all())
    assert torch.equal(a[0][rows], b[0][rows]) and torch.equal(a[1][cols], b[1][cols]) and torch.equal(a[2][cols], b[2][cols])
    assert not bool(b[0][7].isfinite().any()) and bool(b[2][at].isinf())

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [4096, 4001])
def test_cross_entropy_bias_gradient_sums_unrounded(pk, gen, dtype, T):
    """Every word is as often a label as it is likely, so each column of dz nearly cancels: db is off by the exponentials'
    and the sum's fp32 errors (32 rows, then strided eighths of the blocks of 32, then eight), not by a rounding of dz."""
    D, V = 64, 64
    x, w = rand(gen, T, D, std=0.1, dtype=dtype), rand(gen, V, D, dtype=dtype)
    bias = torch.zeros(V, device="cuda", dtype=dtype)
    labels = torch.arange(T, device="cuda") % V
    _, lse = pk.cross_entropy(x, w, labels, bias)
    dloss = torch.ones(T, device="cuda")
    _, _, db = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    z, dz = ref.logits(x, w, bias)
    q = torch.exp(z - lse.double()[:, None])
    e = q * (dz + (z.abs() + lse.double().abs()[:, None] + 2) * 2.0**-21)
    q[torch.arange(T, device="cuda"), labels] -= 1.0
    err = e.sum(0) + (32 + T / 256 + 9 + 2) * 2.0**-24 * (q.abs() + e).sum(0)
    want = q.sum(0)
    assert ref.worst(db, want, rounded(err, want, dtype)) <= 1

def test_status_belongs_to_the_call_s_stream(pk, gen):
    """A bad label on one stream is no other stream's error; a query takes one error and leaves the other for the next."""
    x, w = torch.ones(1, 8, device="cuda"), torch.ones(2, 8, device="cuda")
    bad = torch.tensor([5], device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    pk.cross_entropy(x, w, bad, stream=a)
    a.synchronize()
    assert pk.last_status() == 0 and pk.last_status(b) == 0
    assert pk.last_status(a) == 11 and pk.last_status(a) == 0
    # the attention's error and the loss's on one stream: both are told, one after the other
    T, H = 8, 1
    qkv = torch.zeros(T, 3 * H * 64, device="cuda", dtype=torch.bfloat16)
    cos = torch.ones(16, 32, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 6, 4, 8], device="cuda", dtype=torch.int32)
    torch.cuda.synchronize()
    pk.attend(qkv, cos, torch.zeros_like(cos), cu, H, 0, 0.125, stream=b, max_len=8)
    pk.cross_entropy(x, w, bad, stream=b)
    b.synchronize()
    assert pk.last_status() == 0 and pk.last_status(a) == 0
    assert [pk.last_status(b) for _ in range(3)] == [5, 11, 0]


_MANY_STREAMS_SCRIPT = r"""
import ctypes, json, os, sys
sys.path.insert(0, os.environ["ROOT"])
import torch
import rope_cu_tile_gb300 as pk
x, w = torch.ones(1, 8, device="cuda"), torch.ones(2, 8, device="cuda")
good, bad = torch.tensor([1], device="cuda"), torch.tensor([5], device="cuda")
torch.cuda.synchronize()
streams = []
for _ in range(1030):
    p = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(p))) == 0
    streams.append(p.value)
    pk.cross_entropy(x, w, good, stream=p.value)
torch.cuda.synchronize()
got = []
for s in (streams[0], streams[500], streams[1028]):
    pk.cross_entropy(x, w, bad, stream=s)
    torch.cuda.synchronize()
    got.append([pk.last_status(), pk.last_status(streams[7]), pk.last_status(s), pk.last_status(s)])
print(json.dumps(got))
"""


def test_status_of_more_streams_than_words():
    """A device has 1024 words; the streams past them share the last. Each is still told its errors."""
    import json
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", _MANY_STREAMS_SCRIPT], env=dict(os.environ, ROOT=root), capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    assert json.loads(p.stdout.strip().splitlines()[-1]) == [[0, 0, 11, 0]] * 3

_STALL_SCRIPT = r"""
import json, os, sys, time
sys.path.insert(0, os.environ["ROOT"])
import torch
import rope_cu_tile_gb300 as pk
torch.manual_seed(3)
got = []
for T, K, N in ((300, 1024, 264), (9000, 1024, 1024)):  # one CTA a tile, and pairs; more k steps than stages
    x, w = torch.randn(T, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
    want = pk.linear(x, w)
    torch.cuda.synchronize()
    os.environ["PK_DEBUG_SKIP_ARRIVE"] = "1"
    t = time.time()
    pk.linear(x, w)
    torch.cuda.synchronize()
    t = time.time() - t
    del os.environ["PK_DEBUG_SKIP_ARRIVE"]
    word = pk.last_status()
    after = pk.linear(x, w)
    torch.cuda.synchronize()
    got.append([word, pk.last_status(), bool(torch.equal(after, want)), t])
print(json.dumps(got))
"""


def test_a_product_that_gives_up_ends_within_two_wait_bounds():
    """One bound for the wait that runs out, one for what is still on its way (bound 200 ms, and 100 ms for the host)."""
    import json
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, ROOT=root, PK_TIMEOUT_MS="200")
    env.pop("PK_DEBUG_SKIP_ARRIVE", None)
    p = subprocess.run([sys.executable, "-c", _STALL_SCRIPT], env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    for word, later, same, t in json.loads(p.stdout.strip().splitlines()[-1]):
        assert (word, later, same) == (6, 0, True) and t <= 0.5, t

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(20, 100), (300, 4099)])
def test_words_masked_by_the_lowest_value(pk, gen, dtype, T, V):
    """A bias of the type's lowest value masks words; where it masks all of them the row's lse is still its log-sum-exp (the
    lowest value, to fp32's precision) and the loss that of equal logits."""
    D = 32
    x, w = rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=D**-0.5, dtype=dtype)
    low = torch.finfo(dtype).min
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    some = torch.zeros(V, device="cuda", dtype=dtype)
    some[V // 2:] = low
    loss, lse = pk.cross_entropy(x, w, labels.clamp(max=V // 2 - 1), some)
    (wl, ws), bound = ref.cross_entropy(x, w[:V // 2].contiguous(), labels.clamp(max=V // 2 - 1), None)
    assert ref.worst(lse, ws, bound) <= 1 and ref.worst(loss, wl, 2 * bound) <= 1
    every = torch.full((V,), low, device="cuda", dtype=dtype)
    zero = torch.zeros_like(x)
    loss, lse = pk.cross_entropy(zero, w, labels, every)
    assert ref.worst(lse, torch.full_like(lse, 1.0, dtype=torch.float64) * low + math.log(V), torch.full_like(lse, abs(low) * 2.0**-23)) <= 1
    # equal logits: ln V, within the sums' errors (64 + V / 32 additions, of V ones) and the logarithm's; fp16's lowest value is
    # small enough for the logits to differ by the products' zero only
    assert ref.worst(loss, torch.full_like(loss, math.log(V), dtype=torch.float64), torch.full_like(loss, (64 + V / 32) * 2.0**-23 + 2.0**-20)) <= 1

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("labelled", [1.0, 0.6])
def test_a_word_of_infinite_weights_gets_no_gradient_from_padding(pk, gen, dtype, labelled):
    """A word whose weights are -inf has the logit -inf in every row (x > 0): probability 0, and a gradient of 0 in its row of
    dw and db. Rows that only fill a tile have x = 0 and would have a logit of 0 (-inf)."""
    T, D, V = 70, 32, 300
    x, w = rand(gen, T, D, dtype=dtype).abs() + 0.125, rand(gen, V, D, std=D**-0.5, dtype=dtype)
    w[7] = -INF
    bias = rand(gen, V, dtype=dtype)
    labels = torch.randint(8, V, (T,), generator=gen, device="cuda")
    labels[torch.rand(T, generator=gen, device="cuda") >= labelled] = -100
    _, lse = pk.cross_entropy(x, w, labels, bias)
    assert bool(lse.isfinite().all())
    _, dw, db = pk.cross_entropy_backward(x, w, labels, lse, torch.ones(T, device="cuda"), bias, need_dx=False)
    assert bool((dw[7] == 0).all()) and float(db[7]) == 0
    assert bool(dw.isfinite().all()) and bool(db.isfinite().all())

@pytest.mark.parametrize("T", [5, 16, 300])
def test_largest_fp32_operands(pk, gen, T):
    """The largest finite values round to infinity in bf16; their products with small weights are finite all the same."""
    K, N = 64, 40
    top = torch.finfo(torch.float32).max
    x, w = rand(gen, T, K), rand(gen, N, K)
    x[:, 0] = top
    x[::2, 0] = -top
    w[:, 0] = 2.0**-100
    want, _, bound, _ = ref.linear(x, w, None, None, "none", 0.0, 0, 0)
    assert ref.worst(pk.linear(x, w), want, bound) <= 1
    dy = torch.full((T, N), 2.0**-100, device="cuda")
    _, dw, _ = pk.linear_backward(x, w, dy, need_dx=False, need_db=False)
    (_, want, _), (_, bound, _) = ref.linear_backward(x, w, dy, None, "none", 0.0, 0, 0)
    assert ref.worst(dw, want, bound) <= 1
    dy = x[:, :1].expand(-1, N).contiguous()  # the gradient itself at the end of the range, through the activation
    wx = torch.full((N, K), 2.0**-100, device="cuda")
    dx, _, _ = pk.linear_backward(x, wx, dy, torch.ones(T, N, device="cuda"), "relu", need_dw=False, need_db=False)
    want = dy.double() @ wx.double()
    assert ref.worst(dx, want, (2 * ref.sum_bound(N, torch.float32) + ref.U[torch.float32]) * dy.double().abs() @ wx.double()) <= 1

@pytest.mark.parametrize("dtype,T,D,V,labelled", [(torch.float32, 300, 1100, 700, 1.0), (torch.float32, 700, 1100, 1003, 0.4),
                                                  (torch.float32, 1500, 2056, 9000, 0.9), (torch.bfloat16, 130, 16456, 300, 0.5),
                                                  (torch.float16, 300, 20000, 264, 1.0)])
def test_cross_entropy_of_long_features(pk, gen, dtype, T, D, V, labelled):
    """More terms than the tensor pipe adds up by itself: the sums are taken over in phases, for the loss and its gradient."""
    x, w = rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=2 * D**-0.5, dtype=dtype)
    bias = rand(gen, V, dtype=dtype)
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    labels[torch.rand(T, generator=gen, device="cuda") >= labelled] = -100
    loss, lse = pk.cross_entropy(x, w, labels, bias)
    (wl, ws), bound = ref.cross_entropy(x, w, labels, bias)
    assert ref.worst(lse, ws, bound) <= 1 and ref.worst(loss, wl, 2 * bound) <= 1
    # closer than the worst case of any order: the pipe truncates 2^-23 of a partial sum a step of 16, at most 1024 steps (fp32:
    # 64, and five passes 2^-8 as large) before a rounding sum takes over; a phase's partial sums are differences of two of the
    # whole's. Some rows, their partial sums in 64 bits.
    rows = (labels >= 0).nonzero()[:32, 0]
    k = D // 16 * 16
    parts = torch.einsum("tgk,vgk->tvg", x[rows, :k].double().view(len(rows), -1, 16), w[:, :k].double().view(V, -1, 16)[:, :])
    most = 2 * float(parts.cumsum(2).abs().max()) + 1
    steps = 64 * (1 + 5 * 2.0**-8) + D / 1024 + 4 if dtype == torch.float32 else 1024 + D / 16384 + 4
    zerr = steps * 2.0**-23 * most + (2.0**-24 * float((x[rows].double().abs() @ w.double().abs().T).max()) if dtype == torch.float32 else 0)
    rest = (float(ref.logits(x[rows], w, bias)[0].abs().max()) + 1) * 2.0**-21 + (64 + V / 32) * 2.0**-23 + 2.0**-22 * ws[rows].abs()
    assert ref.worst(lse[rows], ws[rows], zerr + rest) <= 1
    del parts
    dloss = torch.rand(T, generator=gen, device="cuda") + 0.5
    got = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    want, bounds = ref.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    for name, g, v, b in zip(("dx", "dw", "db"), got, want, bounds):
        assert ref.worst(g, v, b) <= 1, name
        off = float((g.double() - v).norm() / v.norm())
        assert off <= {torch.float32: 2.0**-16, torch.bfloat16: 2.0**-7, torch.float16: 2.0**-10}[dtype], (name, off)
    assert pk.last_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("labelled", [1.0, 0.3])
def test_gradient_over_several_pieces_of_the_vocabulary(pk, gen, dtype, labelled):
    """Pieces of at least 4096 words: the gradient's fp32 sums between them, fp16's scale on the last one, fp32's planes, the map
    of labelled rows, with a last piece narrower than the others. Some rows and words against 64 bits."""
    T, D, V = (40001 if dtype == torch.float32 else 131073), 40, 9001 if dtype == torch.float32 else 13001
    x, w = rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=2 * D**-0.5, dtype=dtype)
    bias = rand(gen, V, dtype=dtype)
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    labels[torch.rand(T, generator=gen, device="cuda") >= labelled] = -100
    _, lse = pk.cross_entropy(x, w, labels, bias)
    dloss = torch.rand(T, generator=gen, device="cuda") * 1e-4
    dx, dw, db = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    some = torch.arange(0, T, 1013, device="cuda")
    want, bound = ref.cross_entropy_backward(x[some], w, labels[some], lse[some], dloss[some], bias)
    assert ref.worst(dx[some], want[0], bound[0]) <= 1
    assert bool((dx[labels < 0] == 0).all())
    words = torch.tensor([0, 1, 4095, 4096, 4351, 4352, 4608, 8191, 8192, V - 300, V - 1], device="cuda")
    z, dz = ref.logits(x, w[words].contiguous(), bias[words])
    has = (labels >= 0)[:, None]
    q = torch.exp(z - lse.double()[:, None])
    e = q * (dz + (z.abs() + lse.double().abs()[:, None] + 2) * 2.0**-21)
    g = dloss.double()[:, None]
    q = torch.where(has, (q - (labels[:, None] == words[None, :]).double()) * g, 0.0)
    e = torch.where(has, e * g, 0.0) + 2.0**-22 * q.abs()
    u = ref.U[dtype] if dtype != torch.float32 else 2.0**-23
    if dtype == torch.float16:
        e = e + has * 2.0**-25 * float(dloss.max()) * 2.0**-14
    r = e + u * q.abs()  # dz as stored
    X = x.double()
    for name, got, v, b in (("dw", dw[words], q.T @ X, r.T @ X.abs() + ref.sum_bound(16384, dtype) * ((q.abs() + r).T @ X.abs())),
                            ("db", db[words], q.sum(0), r.sum(0) + 2.0**-13 * q.abs().sum(0))):
        assert ref.worst(got, v, rounded(b, v, dtype)) <= 1, name
    assert pk.last_status() == 0

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 64), (16, 64), (122, 40), (300, 2048), (9000, 64)])
def test_columns_beside_an_output_stay_as_they_were(pk, gen, dtype, T, K):
    """out as some columns of a wider matrix whose rows are whole 16 bytes: what stands left and right of them is not written,
    whatever the number of columns; alone, and as residual and output in one."""
    for N, off, wide in ((41, 0, 48), (33, 0, 40), (36, 8, 56), (34, 0, 40), (44, 0, 48), (1, 0, 8), (39, 16, 56), (589, 0, 592), (130, 8, 144),
                         (64, 0, 72), (31, 0, 32)):
        x, w = rand(gen, T, K, dtype=dtype), rand(gen, N, K, std=K**-0.5, dtype=dtype)
        want = pk.linear(x, w)
        for residual in (False, True):
            base = torch.full((T + 1, wide), 7.0, dtype=dtype, device="cuda")
            out = base[:T, off:off + N]
            if residual:
                out.copy_(rand(gen, T, N, dtype=dtype))
                want = pk.linear(x, w, residual=out.clone())
            got = pk.linear(x, w, residual=out if residual else None, out=out)
            assert torch.equal(got, want) and torch.equal(out, want), (N, off, wide)
            base[:T, off:off + N] = 7.0
            assert bool((base == 7).all()), (N, off, wide)
            got = pk.dropout(want, 0.25, 3, out=out)
            assert torch.equal(got, pk.dropout(want, 0.25, 3))
            base[:T, off:off + N] = 7.0
            assert bool((base == 7).all()), (N, off, wide)

def test_captured_calls_decide_on_the_device(pk, gen):
    """Replayed with other contents, a captured fp16 gradient takes the scale that those need, and a captured loss tells of a bad
    label in the word of the stream it was captured on."""
    T, K, N, V = 200, 64, 136, 300
    x, w, wv = rand(gen, T, K, std=0.05).half(), rand(gen, N, K, std=0.05).half(), rand(gen, V, K).half()
    dy, pre = rand(gen, T, N).half(), rand(gen, T, N).half()
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        return [*pk.linear_backward(x, w, dy, pre, "gelu", 0.5, 3, 4), *pk.cross_entropy(x, wv, labels)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for size in (1.0, 2e4, 1e-6, 0.1):
        dy.copy_((torch.rand(T, N, generator=gen, device="cuda") * 2 * size).half())
        graph.replay()
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b), size
    assert bool(got[0].isfinite().all())
    assert pk.last_status() == 0 and pk.last_status(side) == 0
    labels[3] = V
    graph.replay()
    torch.cuda.synchronize()
    assert bool(got[3][3].isnan()) and pk.last_status() == 0
    assert pk.last_status(side) == 11 and pk.last_status(side) == 0
