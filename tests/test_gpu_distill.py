"""Distillation from a teacher's top logits and its gradients against their definitions in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
# rows, features, words, the teacher's words
SIZES = [(1, 8, 3, 1), (1, 64, 1000, 5), (5, 33, 50, 50), (17, 100, 257, 3), (130, 72, 1003, 16), (300, 136, 5000, 33), (640, 64, 2048, 64), (2100, 96, 700, 7)]


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    return g


def case(gen, dtype, T, D, V, top, holes=True):
    """A student's rows and a teacher's words, some of them not there, some twice, some rows without any."""
    x, w = rand(gen, T, D, dtype=dtype), rand(gen, V, D, std=2 * D**-0.5, dtype=dtype)
    bias = rand(gen, V, std=0.3, dtype=dtype)
    idx = torch.randint(0, V, (T, top), generator=gen, device="cuda")
    values = rand(gen, T, top, std=2.5)
    if holes and T > 2:
        idx[torch.rand(T, top, generator=gen, device="cuda") < 0.2] = -1
        values[torch.rand(T, top, generator=gen, device="cuda") < 0.1] = float("-inf")
        idx[1] = -7
        values[2] = float("-inf")
        idx[0, 0] = idx[0, -1]
    return x, w, bias, idx, values


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D,V,top", SIZES)
def test_distill(pk, gen, dtype, T, D, V, top):
    x, w, bias, idx, values = case(gen, dtype, T, D, V, top)
    for b, tau in ((bias, 1.0), (None, 2.5)):
        loss, lse = pk.distill(x, w, idx, values, bias=b, temperature=tau)
        (wl, ws), (bl, bs) = ref.distill(x, w, idx, values, b, tau)
        assert ref.worst(lse, ws, bs) <= 1 and ref.worst(loss, wl, bl) <= 1
    assert pk.last_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D,V,top", SIZES)
def test_distill_backward(pk, gen, dtype, T, D, V, top):
    x, w, bias, idx, values = case(gen, dtype, T, D, V, top)
    dloss = rand(gen, T) / T
    for b, tau in ((bias, 0.7), (None, 3.0)):
        _, lse = pk.distill(x, w, idx, values, bias=b, temperature=tau)
        got = pk.distill_backward(x, w, idx, values, lse, dloss, bias=b, temperature=tau)
        want, bound = ref.distill_backward(x, w, idx, values, lse, dloss, b, tau)
        assert (got[2] is None) == (b is None)
        for name, g, v, e in zip(("dx", "dw", "db"), got, want, bound):
            if g is not None:
                assert ref.worst(g, v, e) <= 1, name
        if T > 2:
            assert not bool(got[0][1].any()) and not bool(got[0][2].any())
    dx, none, _ = pk.distill_backward(x, w, idx, values, lse, dloss, temperature=tau, need_dw=False)
    assert none is None and torch.equal(dx, got[0])
    none, dw, _ = pk.distill_backward(x, w, idx, values, lse, dloss, temperature=tau, need_dx=False)
    assert none is None and torch.equal(dw, got[1])
    assert pk.last_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_one_word_is_the_cross_entropy(pk, gen, dtype):
    T, D, V = 200, 64, 1500
    x, w, bias, idx, values = case(gen, dtype, T, D, V, 1, holes=False)
    idx[::5] = -1
    loss, lse = pk.distill(x, w, idx, values, bias=bias)
    want, wlse = pk.cross_entropy(x, w, idx[:, 0].contiguous(), bias=bias)
    # one arithmetic but for the joins' order: some units of 2^-24 of values below 16
    assert float((loss - want).abs().max()) < 2e-5 and float((lse - wlse).abs().max()) < 1e-5
    g = rand(gen, T) / T
    a, b = pk.distill_backward(x, w, idx, values, wlse, g, bias=bias), pk.cross_entropy_backward(x, w, idx[:, 0].contiguous(), wlse, g, bias=bias)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_several_pieces(pk, gen, dtype):
    """A vocabulary that the backward pass takes in pieces, the words of a row in all of them."""
    T, D, V, top = (40000, 64, 30000, 12) if dtype == torch.bfloat16 else (14000, 32, 30000, 12)
    x, w, bias, idx, values = case(gen, dtype, T, D, V, top)
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    keep[::40] = True
    idx[~keep] = -1  # (few rows to compute in 64 bits; the pieces go by all of them)
    tau, dloss = 1.5, rand(gen, T) / T
    _, lse = pk.distill(x, w, idx, values, bias=bias, temperature=tau)
    dx, dw, db = pk.distill_backward(x, w, idx, values, lse, dloss, bias=bias, temperature=tau)
    assert not bool(dx[~keep].any())
    want, bound = ref.distill_backward(x[keep], w, idx[keep], values[keep], lse[keep], dloss[keep], bias, tau)
    for g, v, e in zip((dx[keep], dw, db), want, bound):
        assert ref.worst(g, v, e) <= 1


def test_gradient_against_differences(pk, gen):
    T, D, V, top = 30, 24, 90, 6
    x, w, bias, idx, values = case(gen, torch.float32, T, D, V, top)
    tau, c = 1.7, rand(gen, T)
    _, lse = pk.distill(x, w, idx, values, bias=bias, temperature=tau)
    dx, dw, db = pk.distill_backward(x, w, idx, values, lse, c, bias=bias, temperature=tau)
    h = 2.0**-7  # third derivatives below h^2 of the slope's terms, roundings 2^-22 |f| / h: 2e-3 covers both
    for t, g, put in ((x, dx, 0), (w, dw, 1), (bias, db, 2)):
        d = rand(gen, *t.shape)

        def f(s):
            a = [x, w, bias]
            a[put] = t + s * h * d
            loss, _ = pk.distill(a[0], a[1], idx, values, bias=a[2], temperature=tau)
            return float((loss.double() * c.double()).sum())

        slope, want = (f(1) - f(-1)) / (2 * h), float((g.double() * d.double()).sum())
        assert abs(slope - want) <= 2e-3 * float((g.double().abs() * d.double().abs()).sum())


@pytest.mark.parametrize("top", [5, 40])
@pytest.mark.parametrize("tau", [1e-3, 0.3, 1.0, 30.0])
def test_a_constant_on_the_teachers_values(pk, gen, tau, top):
    """Values that all have the same constant added, exactly (steps of 2^-4 beside 2^18): the same loss and gradients, bit for bit."""
    T, D, V = 70, 40, 300
    x, w, bias, idx, _ = case(gen, torch.float32, T, D, V, top)
    values = torch.randint(-128, 128, (T, top), generator=gen, device="cuda").float() / 16
    values[torch.rand(T, top, generator=gen, device="cuda") < 0.1] = float("-inf")
    dloss = rand(gen, T) / T

    def run(values):
        loss, lse = pk.distill(x, w, idx, values, bias=bias, temperature=tau)
        return loss, lse, *pk.distill_backward(x, w, idx, values, lse, dloss, bias=bias, temperature=tau)

    want = run(values)
    for c in (2.0**18, -(2.0**18)):
        assert all(torch.equal(a, b) for a, b in zip(run(values + c), want))


@pytest.mark.parametrize("tau", [1e-3, 0.05, 1.0])
def test_large_values_of_the_teacher(pk, gen, tau):
    """Raw logits near 10^4: as those less their maximum (exact differences), with a bound that goes by these."""
    T, D, V, top = 60, 40, 300, 9
    x, w, bias, idx, values = case(gen, torch.float32, T, D, V, top)
    values = values * max(tau, 2.0**-6) + 1e4
    there = (idx >= 0) & ~torch.isneginf(values)
    less = values.double() - torch.where(there, values.double(), -1e30).amax(1, keepdim=True)
    loss, lse = pk.distill(x, w, idx, values, bias=bias, temperature=tau)
    (wl, ws), (bl, bs) = ref.distill(x, w, idx, less, bias, tau)
    assert ref.worst(lse, ws, bs) <= 1 and ref.worst(loss, wl, bl) <= 1
    dloss = rand(gen, T) * tau / T
    got = pk.distill_backward(x, w, idx, values, lse, dloss, bias=bias, temperature=tau)
    want, bound = ref.distill_backward(x, w, idx, less, lse, dloss, bias, tau)
    for g, v, e in zip(got, want, bound):
        assert ref.worst(g, v, e) <= 1


@pytest.mark.parametrize("tau", [1e-3, 0.5, 2.0])
def test_a_teachers_lowest_values(pk, gen, tau):
    """Words masked by the type's lowest value: no share beside others, equal ones where nothing else is there."""
    T, D, V, top = 12, 24, 200, 6
    x, w, bias, idx, values = case(gen, torch.float32, T, D, V, top, holes=False)
    low = torch.finfo(torch.float32).min
    values[0:4] = low
    values[4:8, 1:] = low
    values[8, 0], values[8, 1:] = -low, low
    same = values.clone()
    same[0:4] = 0.0
    same[4:9, 0], same[4:9, 1:] = 0.0, float("-inf")
    a, b = (pk.distill(x, w, idx, v, bias=bias, temperature=tau) for v in (values, same))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool(a[0].isfinite().all())
    g = torch.ones(T, device="cuda")
    a, b = (pk.distill_backward(x, w, idx, v, a[1], g, bias=bias, temperature=tau) for v in (values, same))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [90, 700, 20000])
def test_words_close_together(pk, gen, dtype, V):
    """Neighbouring rows with none to 64 of their words in the same 32 of the vocabulary, some more than once, the rest anywhere."""
    T, D, top = 200, 72, 64
    x, w, bias, idx, values = case(gen, dtype, T, D, V, top, holes=False)
    close = torch.arange(top, device="cuda")[None] < (torch.arange(T, device="cuda")[:, None] * 37) % 65
    near = 32 * (torch.arange(T, device="cuda") // 32 % 2)[:, None] + torch.randint(0, 32, (T, top), generator=gen, device="cuda")
    idx = torch.where(close, near, idx)
    idx[::9, ::2] = -1
    loss, lse = pk.distill(x, w, idx, values, bias=bias)
    (wl, ws), (bl, bs) = ref.distill(x, w, idx, values, bias, 1.0)
    assert ref.worst(lse, ws, bs) <= 1 and ref.worst(loss, wl, bl) <= 1
    dloss = rand(gen, T) / T
    got = pk.distill_backward(x, w, idx, values, lse, dloss, bias=bias)
    want, bound = ref.distill_backward(x, w, idx, values, lse, dloss, bias, 1.0)
    for g, v, e in zip(got, want, bound):
        assert ref.worst(g, v, e) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tau", [1e-3, 0.05, 1e3])
def test_temperatures_at_the_ends(pk, gen, dtype, tau):
    """The coldest and the hottest: probabilities all but one-hot, and all but equal; fp16's dz stays in range."""
    x, w, bias, idx, values = case(gen, dtype, 50, 40, 300, 8)
    loss, lse = pk.distill(x, w, idx, values, bias=bias, temperature=tau)
    (wl, ws), (bl, bs) = ref.distill(x, w, idx, values, bias, tau)
    assert ref.worst(lse, ws, bs) <= 1 and ref.worst(loss, wl, bl) <= 1
    dloss = rand(gen, 50) * tau
    got = pk.distill_backward(x, w, idx, values, lse, dloss, bias=bias, temperature=tau)
    want, bound = ref.distill_backward(x, w, idx, values, lse, dloss, bias, tau)
    for g, v, e in zip(got, want, bound):
        assert ref.worst(g, v, e) <= 1


def test_bad_words(pk, gen):
    x, w, bias, idx, values = case(gen, torch.bfloat16, 6, 32, 100, 4, holes=False)
    idx[2, 1], idx[4, 3] = 100, 1 << 40
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    loss, lse = pk.distill(x, w, idx, values, status=status)
    assert int(status) == 11 and pk.last_status() == 0
    assert loss.isnan().tolist() == [False, False, True, False, True, False] and float(lse[2]) == 0
    g = torch.ones(6, device="cuda")
    dx, dw, _ = pk.distill_backward(x, w, idx, values, lse, g)
    assert pk.last_status() == 11 and not bool(dx[2].any()) and not bool(dx[4].any()) and bool(dw.isfinite().all())


def test_nothing_to_learn(pk, gen):
    """No row with a target; no row at all."""
    x, w, bias, idx, values = case(gen, torch.bfloat16, 300, 32, 500, 4, holes=False)
    idx[:] = -1
    loss, lse = pk.distill(x, w, idx, values, bias=bias)
    got = pk.distill_backward(x, w, idx, values, lse, torch.ones(300, device="cuda"), bias=bias)
    assert not bool(loss.any()) and not bool(lse.any()) and not any(bool(g.any()) for g in got)
    loss, lse = pk.distill(x[:0], w, idx[:0], values[:0])
    got = pk.distill_backward(x[:0], w, idx[:0], values[:0], lse, loss, bias=bias)
    assert loss.shape == (0,) and not any(bool(g.any()) for g in got)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_streams_and_graphs(pk, gen, dtype):
    T, D, V, top = 260, 48, 900, 9
    x, w, bias, idx, values = case(gen, dtype, T, D, V, top)
    wide = rand(gen, T, 2 * D + 3, dtype=dtype)
    want = None
    for shift in (0, 8, 3):
        wide[:, shift:shift + D] = x
        view = wide[:, shift:shift + D]
        loss, lse = pk.distill(view, w, idx, values, bias=bias)
        grads = pk.distill_backward(view, w, idx, values, lse, loss, bias=bias)
        if want is None:
            want = (loss, lse, *grads)
        assert all(torch.equal(a, b) for a, b in zip((loss, lse, *grads), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pk.distill(x, w, idx, values, bias=bias, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0])
    held, words = torch.zeros_like(x), torch.full_like(idx, -1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, lse = pk.distill(held, w, words, values, bias=bias)
        grads = pk.distill_backward(held, w, words, values, lse, loss, bias=bias)
    g.replay()
    assert not bool(loss.any())
    held.copy_(x)
    words.copy_(idx)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, *grads), want))
