"""The token-row operators against their definitions in 64 bits: the projection and its gradients, dropout, the cross
entropy over a vocabulary and its gradients, at the sizes, layouts and rows where they can go wrong."""

import pytest

torch = pytest.importorskip("torch")

import rows_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
SEED, OFFSET = 0x123456789ABCDEF0, (7 << 32) + 11


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(1234)
    return g


def check_status(pk):
    assert pk.last_status() == 0


# ------------------------------------------------------------------------------------------ the projection

SIZES = [(1, 8, 8), (1, 1, 1), (1, 4096, 77), (2, 64, 40), (3, 2056, 4100), (4, 300, 33), (5, 129, 3), (8, 264, 100), (16, 256, 513), (17, 100, 264), (128, 64, 128), (129, 72, 136),
         (251, 768, 768), (300, 65, 257), (1000, 515, 1003), (513, 1024, 264), (4096, 128, 512), (20000, 64, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear(pk, gen, dtype, T, K, N):
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, N, K, std=K**-0.5, dtype=dtype)
    y = pk.linear(x, w)
    want, _, bound, _ = ref.linear(x, w, None, None, "none", 0.0, 0, 0)
    assert ref.worst(y, want, bound) <= 1
    check_status(pk)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("T,K,N", [(1, 96, 200), (9, 64, 77), (200, 328, 136), (3000, 192, 520)])
def test_linear_epilogue(pk, gen, dtype, act, T, K, N):
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, N, K, std=2 * K**-0.5, dtype=dtype)
    bias, res = rand(gen, N, dtype=dtype), rand(gen, T, N, dtype=dtype)
    y, pre = pk.linear(x, w, bias, res, act, 0.3, SEED, OFFSET, return_pre=True)
    want, z, by, bz = ref.linear(x, w, bias, res, act, 0.3, SEED, OFFSET)
    assert ref.worst(pre, z, bz) <= 1
    assert ref.worst(y, want, by) <= 1
    # each part alone gives what the whole gave
    assert torch.equal(pk.linear(x, w, bias, res, act, 0.3, SEED, OFFSET), y)
    assert torch.equal(pk.linear(x, w, bias), pre)
    pk.linear(x, w, bias, res, act, 0.3, SEED, OFFSET, out=res)  # onto the residual
    assert torch.equal(res, y)
    check_status(pk)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 200])
def test_activations_at_infinity(pk, gen, dtype, T):
    """A pre-activation of +inf, -inf or NaN (through the bias) beside finite ones: relu and gelu take their limits, NaN stays."""
    K, N = 64, 40
    x, w, bias = rand(gen, T, K, dtype=dtype), rand(gen, N, K, dtype=dtype), torch.zeros(N, dtype=dtype, device="cuda")
    bias[3], bias[4], bias[5] = float("inf"), float("-inf"), float("nan")
    ok = [i for i in range(N) if i not in (3, 4, 5)]
    for act in ("relu", "gelu"):
        y = pk.linear(x, w, bias, act=act)
        assert bool((y[:, 3] == float("inf")).all()) and bool((y[:, 4] == 0).all()) and bool(y[:, 5].isnan().all())
        assert bool(y[:, ok].isfinite().all())
    y = pk.linear(x, w, bias, act="silu")
    assert bool((y[:, 3] == float("inf")).all()) and bool(y[:, 5].isnan().all()) and bool(y[:, ok].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 7, 300])
def test_linear_strided_rows(pk, gen, dtype, T):
    """x a slice of wider rows (the v part of a packed qkv), out and the residual slices too; what lies beside is kept."""
    K, N = 128, 192
    wide = rand(gen, T, 3 * K, dtype=dtype)
    w = rand(gen, N, K, std=K**-0.5, dtype=dtype)
    for k0 in (0, 2 * K, 2 * K - 3):
        x = wide[:, k0:k0 + K]
        res_wide, out_wide = rand(gen, T, N + 5, dtype=dtype), torch.full((T, N + 9), 7.0, dtype=dtype, device="cuda")
        out = out_wide[:, 3:3 + N]
        y = pk.linear(x, w, residual=res_wide[:, 1:N + 1], out=out)
        assert y.data_ptr() == out.data_ptr()
        want, _, bound, _ = ref.linear(x, w, None, res_wide[:, 1:N + 1], "none", 0.0, 0, 0)
        assert ref.worst(out, want, bound) <= 1
        assert bool((out_wide[:, :3] == 7).all()) and bool((out_wide[:, 3 + N:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act,p", [("none", 0.0), ("none", 0.2), ("relu", 0.0), ("gelu", 0.25), ("silu", 0.5)])
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (3, 33, 50), (251, 136, 264), (1021, 515, 1003), (9000, 64, 128)])
def test_linear_backward(pk, gen, dtype, act, p, T, K, N):
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, N, K, std=K**-0.5, dtype=dtype)
    dy, pre = rand(gen, T, N, std=0.1, dtype=dtype), rand(gen, T, N, dtype=dtype)
    got = pk.linear_backward(x, w, dy, pre if act != "none" else None, act, p, SEED, OFFSET)
    want, bound = ref.linear_backward(x, w, dy, pre, act, p, SEED, OFFSET)
    for name, g, v, b in zip(("dx", "dw", "db"), got, want, bound):
        assert ref.worst(g, v, b) <= 1, name
    # one at a time: the same bits
    for i in range(3):
        need = [j == i for j in range(3)]
        one = pk.linear_backward(x, w, dy, pre, act, p, SEED, OFFSET, need_dx=need[0], need_dw=need[1], need_db=need[2])
        assert [o is not None for o in one] == need and torch.equal(one[i], got[i])
    check_status(pk)


def test_linear_gradient_against_differences(pk, gen):
    """fp32: the gradient against central differences of the library's own forward, in a random direction."""
    T, K, N = 40, 24, 32
    x, w, b = rand(gen, T, K), rand(gen, N, K, std=0.3), rand(gen, N)
    c = rand(gen, T, N)
    args = dict(act="gelu", p=0.25, seed=SEED, offset=OFFSET)
    _, pre = pk.linear(x, w, b, return_pre=True, **args)
    dx, dw, db = pk.linear_backward(x, w, c, pre, **args)
    # a step h: the third derivative's share is h^2, the rounding of the sums 2^-23 |f| sqrt(TN) / h; both below 2e-3 of |f'|
    h = 2.0**-7
    for t, g, put in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        d = rand(gen, *t.shape)

        def f(s):
            a = [x, w, b]
            a[put] = t + s * h * d
            return float((pk.linear(*a, **args).double() * c.double()).sum())

        slope, want = (f(1) - f(-1)) / (2 * h), float((g.double() * d.double()).sum())
        scale = float((g.double().abs() * d.double().abs()).sum())
        assert abs(slope - want) <= 2e-3 * scale


# ------------------------------------------------------------------------------------------ dropout


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N", [(1, 1), (1, 4096), (3, 7), (251, 768), (1000, 1003), (70000, 24)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_dropout(pk, gen, dtype, T, N, p):
    x, r = rand(gen, T, N, dtype=dtype), rand(gen, T, N, dtype=dtype)
    f = ref.drop_factor(T, N, p, SEED, OFFSET, "cuda")
    for res in (None, r):
        y = pk.dropout(x, p, SEED, OFFSET, residual=res)
        v = x.double() * f
        want = v if res is None else v + res.double()
        bound = 2.0**-23 * (v.abs() + want.abs()) + ref.U[dtype] * want.abs() + (2.0**-25 if dtype == torch.float16 else 0)
        assert ref.worst(y, want, bound) <= 1
    assert torch.equal(pk.dropout_backward(x, p, SEED, OFFSET), pk.dropout(x, p, SEED, OFFSET))
    assert torch.equal(pk.dropout(r.clone(), p, SEED, OFFSET, out=None), pk.dropout(r, p, SEED, OFFSET, out=r))  # in place


def test_dropout_draws(pk):
    """The share kept, and that neighbours in every argument draw other bits."""
    T, N, p = 4096, 1024, 0.3
    one = torch.ones(T, N, device="cuda")
    base = pk.dropout(one, p, 5, 9) != 0
    n = T * N
    assert abs(float(base.double().mean()) - (1 - p)) <= 6 * (p * (1 - p) / n) ** 0.5 + 2.0**-17
    for other in (pk.dropout(one, p, 6, 9), pk.dropout(one, p, 5, 10), pk.dropout(one, p, 5 + (1 << 32), 9),
                  pk.dropout(one, p, 5, 9 + (1 << 32)), pk.dropout(one, p, 5, 9).roll(1, 0), pk.dropout(one, p, 5, 9).roll(8, 1)):
        same = float((base == (other != 0)).double().mean())
        assert abs(same - (p * p + (1 - p) ** 2)) <= 0.01  # as independent draws agree


def test_dropout_infinities_do_not_leak(pk):
    x = torch.full((64, 64), float("inf"), device="cuda")
    y = pk.dropout(x, 0.5, 1, 2)
    keep = torch.from_numpy(ref.keep_mask(64, 64, 0.5, 1, 2)).cuda()
    assert bool((y[keep] == float("inf")).all()) and bool((y[~keep] == 0).all())


# ------------------------------------------------------------------------------------------ cross entropy

XENT = [(1, 8, 2), (1, 64, 1), (3, 33, 100), (64, 64, 257), (130, 72, 1000), (640, 128, 4099), (300, 65, 32003), (2000, 64, 264)]


def xent_case(gen, dtype, T, D, V, labelled, with_bias, std=3.0):
    x, w = rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=std * D**-0.5, dtype=dtype)
    bias = rand(gen, V, dtype=dtype) if with_bias else None
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    drop = torch.rand(T, generator=gen, device="cuda") >= labelled
    labels[drop] = -100
    return x, w, bias, labels


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("labelled", [1.0, 0.2, 0.0])
@pytest.mark.parametrize("T,D,V", XENT)
def test_cross_entropy(pk, gen, dtype, labelled, T, D, V):
    x, w, bias, labels = xent_case(gen, dtype, T, D, V, labelled, V % 2 == 0)
    loss, lse = pk.cross_entropy(x, w, labels, bias)
    (want_loss, want_lse), bound = ref.cross_entropy(x, w, labels, bias)
    assert ref.worst(lse, want_lse, bound) <= 1
    assert ref.worst(loss, want_loss, 2 * bound) <= 1
    check_status(pk)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("labelled", [1.0, 0.2, 0.0])
@pytest.mark.parametrize("T,D,V", XENT)
def test_cross_entropy_backward(pk, gen, dtype, labelled, T, D, V):
    x, w, bias, labels = xent_case(gen, dtype, T, D, V, labelled, V % 2 == 0)
    _, lse = pk.cross_entropy(x, w, labels, bias)
    dloss = torch.randn(T, generator=gen, device="cuda") / max(1, T)
    got = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    want, bound = ref.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    for name, g, v, b in zip(("dx", "dw", "db"), got, want, bound):
        if g is not None:
            assert ref.worst(g, v, b) <= 1, name
    dx, dw, _ = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias, need_dw=False)
    assert dw is None and torch.equal(dx, got[0])
    assert bool((got[0][labels < 0] == 0).all())
    check_status(pk)


def test_cross_entropy_in_pieces(pk, gen):
    """More than one piece of the vocabulary: the scratch for dz is a gigabyte, so 40000 rows over 40000 words take three."""
    T, D, V = 40000, 64, 40000
    x, w, bias, labels = xent_case(gen, torch.bfloat16, T, D, V, 1.0, True)
    _, lse = pk.cross_entropy(x, w, labels, bias)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dx, dw, db = pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    # the same rows by themselves, a few: dx does not depend on the others
    some = torch.arange(0, T, 397, device="cuda")
    want, bound = ref.cross_entropy_backward(x[some], w, labels[some], lse[some], dloss[some], bias)
    assert ref.worst(dx[some], want[0], bound[0]) <= 1
    # dw and db of some words, from their columns of dz in 64 bits
    words = torch.tensor([0, 1, 13567, 13568, 20000, 27135, 27136, 39999], device="cuda")
    q = torch.exp(x.double() @ w[words].double().T + bias[words].double() - lse.double()[:, None])
    q = (q - (labels[:, None] == words[None, :]).double()) / T
    u = ref.U[torch.bfloat16]
    rel = 2 * u + 2.0**-13  # dz's rounding and the logits' error, the sum's rounding
    assert ref.worst(dw[words], q.T @ x.double(), rel * (q.abs().T @ x.double().abs()) + u * (q.T @ x.double()).abs()) <= 1
    assert ref.worst(db[words], q.sum(0), rel * q.abs().sum(0) + u * q.sum(0).abs()) <= 1


@pytest.mark.parametrize("dtype", TYPES)
def test_cross_entropy_bad_and_extreme(pk, gen, dtype):
    T, D, V = 70, 32, 300
    x, w, bias, labels = xent_case(gen, dtype, T, D, V, 1.0, True)
    labels[3], labels[5], labels[7] = V, -1, 1 << 40
    bias[10] = float("-inf")  # a word that cannot be
    bias[11] = 60000.0 if dtype == torch.float16 else 1e30  # one that has to be
    labels[9], labels[11] = 10, 11
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = pk.cross_entropy(x, w, labels, bias, status=status)
    assert int(status) == 11  # PK_ERR_BAD_LABEL
    assert bool(loss[[3, 7]].isnan().all()) and float(loss[5]) == 0 and bool((lse[[3, 5, 7]] == 0).all())
    assert float(loss[9]) == float("inf") and abs(float(loss[11])) <= 2.0**-20 * float(bias[11].float())
    ok = [i for i in range(T) if i not in (3, 5, 7, 9)]
    assert bool(loss[ok].isfinite().all())
    dx, dw, db = pk.cross_entropy_backward(x, w, labels, lse, torch.ones(T, device="cuda"), bias, status=status)
    assert int(status) == 11
    assert bool((dx[[3, 5, 7]] == 0).all()) and bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    assert pk.last_status() == 0  # the caller's word took it
    pk.cross_entropy(x, w, labels, bias)
    assert pk.last_status() == 11 and pk.last_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [90, 3000])
def test_rows_without_a_label_do_not_leak(pk, gen, dtype, T):
    """NaN and infinities in the rows that have no label (x, lse, dloss) reach nothing."""
    D, V = 72, 700
    x, w, bias, labels = xent_case(gen, dtype, T, D, V, 0.4, True)
    _, lse = pk.cross_entropy(x, w, labels, bias)
    dloss = torch.rand(T, generator=gen, device="cuda")
    want = pk.cross_entropy(x, w, labels, bias) + pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    out = labels < 0
    x[out], lse[out], dloss[out] = float("nan"), float("inf"), float("nan")
    x[out.nonzero()[::2, 0]] = float("inf")
    got = pk.cross_entropy(x, w, labels, bias) + pk.cross_entropy_backward(x, w, labels, lse, dloss, bias)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ a run of them, streams, graphs


def encoder_step(pk, s):
    """One layer of a packed encoder and its loss, forwards and backwards, as a training step calls them."""
    H, D = s["H"], s["H"] * 64
    cu, cos, sin, x = s["cu"], s["cos"], s["sin"], s["x"]
    qkv = pk.linear(x, s["wqkv"], s["bqkv"])
    out, lse = pk.attend(qkv, cos, sin, cu, H, 0, 0.125, max_len=s["longest"])
    h = pk.linear(out, s["wo"], s["bo"], residual=x, p=0.1, seed=3, offset=1)
    a, pre = pk.linear(h, s["w1"], s["b1"], act="gelu", return_pre=True)
    y = pk.linear(a, s["w2"], s["b2"], residual=h, p=0.1, seed=3, offset=2)
    loss, l = pk.cross_entropy(y, s["wv"], s["labels"], s["bv"])
    dloss = torch.full_like(loss, 1.0 / s["count"])
    dy, dwv, dbv = pk.cross_entropy_backward(y, s["wv"], s["labels"], l, dloss, s["bv"])
    da, dw2, db2 = pk.linear_backward(a, s["w2"], dy, p=0.1, seed=3, offset=2)
    dh, dw1, db1 = pk.linear_backward(h, s["w1"], da, pre, "gelu")
    dh = dh + dy
    do, dwo, dbo = pk.linear_backward(out, s["wo"], dh, p=0.1, seed=3, offset=1)
    dqkv = pk.attend_backward(qkv, cos, sin, cu, H, 0, 0.125, out, lse, do, max_len=s["longest"])
    dx, dwqkv, dbqkv = pk.linear_backward(x, s["wqkv"], dqkv)
    return dict(loss=loss, dx=dx + dh, dwqkv=dwqkv, dbqkv=dbqkv, dwo=dwo, dbo=dbo, dw1=dw1, db1=db1, dw2=dw2, db2=db2, dwv=dwv,
                dbv=dbv)


def encoder_state(gen, dtype, H=2, V=1000, F=320, lens=(37, 64, 150, 5, 1)):
    import synth

    D, T = H * 64, sum(lens)
    c, sn = synth.rope_tables_dims(max(lens), 64, 10000.0)
    s = dict(H=H, longest=max(lens), x=rand(gen, T, D, dtype=dtype),
             cu=torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda"),
             cos=torch.from_numpy(c).cuda().to(dtype), sin=torch.from_numpy(sn).cuda().to(dtype))
    for name, n, k in (("qkv", 3 * D, D), ("o", D, D), ("1", F, D), ("2", D, F), ("v", V, D)):
        s["w" + name] = rand(gen, n, k, std=k**-0.5, dtype=dtype)
        s["b" + name] = rand(gen, n, std=0.1, dtype=dtype)
    s["labels"] = torch.randint(0, V, (T,), generator=gen, device="cuda")
    s["labels"][torch.rand(T, generator=gen, device="cuda") > 0.3] = -100
    s["count"] = int((s["labels"] >= 0).sum())
    return s


def encoder_reference(s):
    """The same step by autograd in 64 bits (the library's masks)."""
    leaves = {k: v.double().clone().requires_grad_(True) for k, v in s.items() if k == "x" or k[0] in "wb"}
    g = leaves
    H, D, T = s["H"], s["H"] * 64, s["x"].shape[0]
    qkv = g["x"] @ g["wqkv"].T + g["bqkv"]
    q, k, v = [t.view(T, H, 64) for t in qkv.split(D, 1)]
    cu = s["cu"].tolist()
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).cuda()
    c, sn = s["cos"].double()[pos][:, None], s["sin"].double()[pos][:, None]

    def rot(t):
        a, b = t[..., :32], t[..., 32:]
        return torch.cat([a * c - b * sn, a * sn + b * c], -1)

    q, k = rot(q), rot(k)
    seq = torch.bucketize(torch.arange(T, device="cuda"), s["cu"][1:].long(), right=True)
    sc = torch.einsum("ihd,jhd->hij", q, k) * 0.125
    sc = sc.masked_fill((seq[:, None] != seq[None, :])[None], float("-inf"))
    out = torch.einsum("hij,jhd->ihd", sc.softmax(-1), v).reshape(T, D)
    f = lambda off: ref.drop_factor(T, D, 0.1, 3, off, "cuda")  # noqa: E731
    h = g["x"] + f(1) * (out @ g["wo"].T + g["bo"])
    a = ref.act(h @ g["w1"].T + g["b1"], "gelu")
    y = h + f(2) * (a @ g["w2"].T + g["b2"])
    z = y @ g["wv"].T + g["bv"]
    has = s["labels"] >= 0
    loss = torch.where(has, torch.logsumexp(z, 1) - z.gather(1, s["labels"].clamp(min=0)[:, None])[:, 0], 0.0)
    (loss.sum() / s["count"]).backward()
    return dict({"d" + k: v.grad for k, v in leaves.items()}, loss=loss.detach())


@pytest.mark.parametrize("dtype", TYPES)
def test_encoder_layer_step(pk, gen, dtype):
    """Forward, loss and every gradient of a layer. The norm-relative bound: the step runs through at most twelve stored
    tensors (forward and back), each off by at most half a step u relative to its elements; products keep a relative error of their
    operands' norms up to the cancellation in them, allowed for with a factor of four."""
    s = encoder_state(gen, dtype)
    got, want = encoder_step(pk, s), encoder_reference(s)
    u = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-20}[dtype]
    for name, g in got.items():
        w = want[name]
        off = float((g.double() - w).norm() / w.norm())
        assert off <= 4 * 12 * u, (name, off)
    check_status(pk)


def test_streams_and_graphs(pk, gen):
    """On a stream of its own, in a captured and replayed graph, and two graphs replayed at the same time: the same bits."""
    s = encoder_state(gen, torch.bfloat16)

    def step():
        h, pre = pk.linear(s["x"], s["w1"], s["b1"], act="gelu", p=0.2, seed=1, offset=2, return_pre=True)
        d = pk.dropout(h, 0.3, 4, 5)
        loss, lse = pk.cross_entropy(s["x"], s["wv"], s["labels"], s["bv"])
        g = pk.linear_backward(s["x"], s["w1"], d, pre, "gelu", 0.2, 1, 2)
        e = pk.cross_entropy_backward(s["x"], s["wv"], s["labels"], lse, loss, s["bv"])
        return [h, pre, d, loss, lse, *g, *e]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = pk.linear(s["x"], s["w1"], s["b1"], act="gelu", p=0.2, seed=1, offset=2, stream=side)
    loss, _ = pk.cross_entropy(s["x"], s["wv"], s["labels"], s["bv"], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(loss, want[3])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for _, outs in graphs:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for o, w in zip(outs, want):
                assert torch.equal(o, w)
    check_status(pk)


def test_no_rows(pk):
    for dtype in TYPES:
        x, w = torch.zeros(0, 64, dtype=dtype, device="cuda"), torch.ones(40, 64, dtype=dtype, device="cuda")
        assert pk.linear(x, w).shape == (0, 40)
        dx, dw, db = pk.linear_backward(x, w, torch.zeros(0, 40, dtype=dtype, device="cuda"))
        assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
        assert pk.dropout(x, 0.5, 1).shape == (0, 64)
        labels = torch.zeros(0, dtype=torch.int64, device="cuda")
        loss, lse = pk.cross_entropy(x, w, labels)
        assert loss.shape == (0,)
        dx, dw, db = pk.cross_entropy_backward(x, w, labels, lse, loss, bias=torch.ones(40, dtype=dtype, device="cuda"))
        assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("T,K,N", [(300, 1024, 264), (130, 1100, 264), (40, 65536, 128), (2000, 40000, 520)])
def test_long_fp32_sums_do_not_drift(pk, gen, T, K, N):
    """Positive terms: an accumulator that truncates loses up to 2^-23 of the sum a step of 16. The tensor pipe adds up at
    most 64 such steps (of the largest pass; the smaller passes 2^-8 of that each) before a rounding sum takes over, so the
    result is off by at most (64 (1 + 5 2^-8) + K / 1024) 2^-23 of itself, however long it is."""
    bound = (64 * (1 + 5 * 2.0**-8) + K / 1024 + 4) * 2.0**-23
    x, w = torch.rand(T, K, generator=gen, device="cuda"), torch.rand(N, K, generator=gen, device="cuda")
    want = x.double() @ w.double().T
    assert ref.worst(pk.linear(x, w), want, bound * want) <= 1
    # the same sums as the gradients take them: over the outputs (dx) and over the rows (dw)
    dx, _, _ = pk.linear_backward(torch.zeros(T, N, device="cuda"), w.T.contiguous(), x, need_dw=False, need_db=False)
    assert ref.worst(dx, want, bound * want) <= 1
    _, dw, _ = pk.linear_backward(x.T.contiguous(), torch.zeros(N, T, device="cuda"), w.T.contiguous(), need_dx=False, need_db=False)
    want = w.double() @ x.double().T
    assert ref.worst(dw, want, bound * want) <= 1
    check_status(pk)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_long_16_bit_sums_do_not_drift(pk, gen, dtype):
    """At most 1024 truncating steps of 16 terms, 2^-23 of the sum each, before a rounding sum takes over, and the result's own
    rounding, at K = 200000 positive terms (without it: 12500 steps)."""
    K, M, N = 200000, 136, 264
    x, w = (torch.rand(K, n, generator=gen, device="cuda").mul_(0.01).to(dtype) for n in (N, M))
    _, dw, _ = pk.linear_backward(x, torch.zeros(M, N, dtype=dtype, device="cuda"), w, need_dx=False, need_db=False)
    want = w.double().T @ x.double()
    assert ref.worst(dw, want, ((1024 + 16) * 2.0**-23 + ref.U[dtype]) * want) <= 1
    check_status(pk)


def test_offsets_past_32_bits(pk, gen):
    """600000 rows of 4096: 2.4e9 elements a matrix. The last rows against the definition, the first beside them."""
    T, K, N, dtype = 600000, 32, 4096, torch.bfloat16
    rows = torch.tensor([0, 1, 299999, 524287, 524288, T - 2, T - 1], device="cuda")
    x, w, bias = rand(gen, T, K, dtype=dtype), rand(gen, N, K, std=K**-0.5, dtype=dtype), rand(gen, N, dtype=dtype)
    big = torch.empty(T, N, dtype=dtype, device="cuda").normal_(generator=gen)
    y, pre = pk.linear(x, w, bias, big, "gelu", return_pre=True)
    want, z, by, bz = ref.linear(x[rows], w, bias, big[rows], "gelu", 0.0, 0, 0)
    assert ref.worst(y[rows], want, by) <= 1 and ref.worst(pre[rows], z, bz) <= 1
    dx, dw, db = pk.linear_backward(x, w, big, pre, "gelu")
    wx, bx = ref.linear_backward(x[rows], w, big[rows], pre[rows], "gelu", 0.0, 0, 0)
    assert ref.worst(dx[rows], wx[0], bx[0]) <= 1
    dz = torch.cat([b.float() * ref.act_slope(p.float(), "gelu").float() for b, p in
                    zip(big[:, 4000:].split(100000), pre[:, 4000:].split(100000))]).double()
    u = ref.U[dtype]
    bound = u * db[4000:].double().abs() + (T * 2.0**-23 + 2.0**-16) * dz.abs().sum(0)
    assert ref.worst(db[4000:], dz.sum(0), bound) <= 1
    del y, dx, dw, db, dz
    y = pk.dropout(big, 0.25, SEED, OFFSET, residual=pre)
    keep = torch.from_numpy(ref.pieces(list(range(512)) * len(rows), [int(r) for r in rows for _ in range(512)], SEED, OFFSET)
                            .reshape(len(rows), N).astype("int32")).cuda() >= 16384
    want = big[rows].double() * keep / 0.75 + pre[rows].double()
    assert ref.worst(y[rows], want, 2.0**-22 * (want.abs() + 2 * big[rows].double().abs()) + u * want.abs()) <= 1
    del y, big, pre
    V = 5000
    x, w = x[:, :16].contiguous(), rand(gen, V, 16, dtype=dtype)
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    loss, lse = pk.cross_entropy(x, w, labels)
    (wl, ws), bound = ref.cross_entropy(x[rows], w, labels[rows], None)
    assert ref.worst(lse[rows], ws, bound) <= 1 and ref.worst(loss[rows], wl, 2 * bound) <= 1
    dloss = torch.ones(T, device="cuda")
    dx, dw, _ = pk.cross_entropy_backward(x, w, labels, lse, dloss)
    wx, bx = ref.cross_entropy_backward(x[rows], w, labels[rows], lse[rows], dloss[rows], None)
    assert ref.worst(dx[rows], wx[0], bx[0]) <= 1
    check_status(pk)


_STALL_SCRIPT = r"""
import json, os, sys
sys.path.insert(0, os.environ["ROOT"])
import torch
import rope_cu_tile_gb300 as pk
torch.manual_seed(3)
got = []
for T, K, N in ((300, 256, 264), (9000, 128, 1024)):  # one CTA a tile, and pairs
    x, w = torch.randn(T, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = pk.linear(x, w)
    os.environ["PK_DEBUG_SKIP_ARRIVE"] = "1"
    pk.linear(x, w, status=status)
    torch.cuda.synchronize()
    pk.linear(x, w)
    torch.cuda.synchronize()
    del os.environ["PK_DEBUG_SKIP_ARRIVE"]
    word = pk.last_status()
    after = pk.linear(x, w)
    torch.cuda.synchronize()
    got.append([int(status), word, pk.last_status(), bool(torch.equal(after, want))])
print(json.dumps(got))
"""


def test_withheld_stage_times_out_and_the_context_stays_usable():
    """The loading warp withholds its first arrival (test hook): every wait of the product runs out, the call ends with
    PK_ERR_TIMEOUT in the status word given or the device's, and the next call is right. Nothing traps or hangs."""
    import json
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, ROOT=root, PK_TIMEOUT_MS="100")
    env.pop("PK_DEBUG_SKIP_ARRIVE", None)
    p = subprocess.run([sys.executable, "-c", _STALL_SCRIPT], env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    assert json.loads(p.stdout.strip().splitlines()[-1]) == [[6, 6, 0, True]] * 2
