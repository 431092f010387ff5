"""The gated feed-forward and its gradients, and the projection of 8-bit rows, against their definitions in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
ACTS = ["none", "relu", "gelu", "silu"]
# a few rows; splits of k; a lone CTA's tile and a pair's; halves that end inside a tile, inside 16 bytes, after one column
SIZES = [(1, 8, 8), (1, 1, 1), (1, 1024, 2624), (2, 64, 40), (3, 2056, 1100), (4, 300, 33), (5, 129, 3), (8, 264, 100), (17, 1000, 264), (60, 4096, 64),
         (128, 64, 64), (129, 72, 136), (251, 768, 1152), (300, 65, 257), (1000, 515, 1003), (600, 1024, 640), (4096, 128, 512), (20000, 64, 200)]


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(777)
    return g


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,F", SIZES)
def test_gated(pk, gen, dtype, T, K, F):
    x, w, bias = rand(gen, T, K, dtype=dtype), rand(gen, 2 * F, K, std=K**-0.5, dtype=dtype), rand(gen, 2 * F, dtype=dtype)
    for act, b in (("gelu", bias), ("silu", None)):
        y, pre = pk.gated_linear(x, w, b, act=act, return_pre=True)
        (wy, wz), (by, bz) = ref.gated_linear(x, w, b, act)
        assert ref.worst(pre, wz, bz) <= 1 and ref.worst(y, wy, by) <= 1
        assert torch.equal(pk.gated_linear(x, w, b, act=act), y)
    assert pk.last_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 200, 1000])
def test_activations(pk, gen, dtype, act, T):
    x, w = rand(gen, T, 96, dtype=dtype), rand(gen, 400, 96, std=3 * 96**-0.5, dtype=dtype)
    y = pk.gated_linear(x, w, act=act)
    (wy, _), (by, _) = ref.gated_linear(x, w, None, act)
    assert ref.worst(y, wy, by) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,F", [(1, 64, 64), (3, 33, 50), (251, 136, 264), (1021, 515, 1003), (9000, 64, 128), (700, 256, 300)])
def test_gated_backward(pk, gen, dtype, act, T, K, F):
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, 2 * F, K, std=K**-0.5, dtype=dtype)
    dy, pre = rand(gen, T, F, std=0.1, dtype=dtype), rand(gen, T, 2 * F, std=1.5, dtype=dtype)
    got = pk.gated_linear_backward(x, w, dy, pre, act)
    want, bound = ref.gated_linear_backward(x, w, dy, pre, act)
    for name, g, v, b in zip(("dx", "dw", "db"), got, want, bound):
        assert ref.worst(g, v, b) <= 1, name
    for i in range(3):
        need = [j == i for j in range(3)]
        one = pk.gated_linear_backward(x, w, dy, pre, act, need_dx=need[0], need_dw=need[1], need_db=need[2])
        assert [o is not None for o in one] == need and torch.equal(one[i], got[i])
    assert pk.last_status() == 0


@pytest.mark.parametrize("std", [2.0**-14, 3000.0])
def test_fp16_gradients_out_of_range(pk, gen, std):
    """fp16: gradients whose dz would vanish among the smallest numbers, or pass the largest, keep their digits in dx and dw."""
    T, K, F = 300, 64, 136
    dtype = torch.float16
    x, w = rand(gen, T, K, dtype=dtype), rand(gen, 2 * F, K, std=K**-0.5, dtype=dtype)
    dy, pre = rand(gen, T, F, std=std, dtype=dtype), rand(gen, T, 2 * F, std=5.0, dtype=dtype)
    if std > 1:
        w, x = w * 2.0**-9, x * 2.0**-9  # so that the results themselves are numbers of fp16
    dx, dw, _ = pk.gated_linear_backward(x, w, dy, pre, "gelu")
    (wx, ww, _), _ = ref.gated_linear_backward(x, w, dy, pre, "gelu")
    # dz 2^-11 of its elements, sums of F or T of them in quadrature at worst: 2^-10 of the result's norm, its rounding 2^-11 more
    for g, v in ((dx, wx), (dw, ww)):
        tiny = 2.0**-25 * v.numel() ** 0.5
        assert float((g.double() - v).norm()) <= 2.0**-9 * float(v.norm()) + tiny


def test_gradient_against_differences(pk, gen):
    T, K, F = 40, 24, 32
    x, w, b = rand(gen, T, K), rand(gen, 2 * F, K, std=0.3), rand(gen, 2 * F)
    c = rand(gen, T, F)
    _, pre = pk.gated_linear(x, w, b, act="silu", return_pre=True)
    dx, dw, db = pk.gated_linear_backward(x, w, c, pre, "silu")
    # a step h: the third derivative's share some h^2, the roundings 2^-23 |f| sqrt(TF) / h: below 2e-3 of the slope's terms
    h = 2.0**-7
    for t, g, put in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        d = rand(gen, *t.shape)

        def f(s):
            a = [x, w, b]
            a[put] = t + s * h * d
            return float((pk.gated_linear(*a, act="silu").double() * c.double()).sum())

        slope, want = (f(1) - f(-1)) / (2 * h), float((g.double() * d.double()).sum())
        assert abs(slope - want) <= 2e-3 * float((g.double().abs() * d.double().abs()).sum())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 200, 1500])
def test_infinite_gates(pk, gen, dtype, T):
    """Gates of +inf, -inf and NaN (through the bias) beside finite ones, and their slopes."""
    K, F = 64, 40
    x, w, bias = rand(gen, T, K, dtype=dtype), rand(gen, 2 * F, K, dtype=dtype), torch.zeros(2 * F, dtype=dtype, device="cuda")
    bias[3], bias[4], bias[5] = float("inf"), float("-inf"), float("nan")
    ok = [i for i in range(F) if i not in (3, 4, 5)]
    for act in ("relu", "gelu", "silu"):
        y, pre = pk.gated_linear(x, w, bias, act=act, return_pre=True)
        assert bool((y[:, 3].abs() == float("inf")).all()) and bool((y[:, 4] == 0).all()) and bool(y[:, 5].isnan().all())
        assert bool(y[:, ok].isfinite().all())
        _, _, db = pk.gated_linear_backward(x, w, torch.ones_like(y), pre, act, need_dx=False, need_dw=False)
        assert float(db[4].abs()) == 0 and bool(db[3].isfinite()) and bool(db[5].isnan()) and bool(db[ok].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 7, 300])
def test_strided_rows(pk, gen, dtype, T):
    K, F = 128, 192
    wide = rand(gen, T, 3 * K, dtype=dtype)
    w = rand(gen, 2 * F, K, std=K**-0.5, dtype=dtype)
    for k0 in (0, 2 * K, 2 * K - 3):
        x = wide[:, k0:k0 + K]
        for f0 in (3, 8):
            out_wide = torch.full((T, F + 16), 7.0, dtype=dtype, device="cuda")
            out = out_wide[:, f0:f0 + F]
            pk.gated_linear(x, w, out=out)
            (wy, _), (by, _) = ref.gated_linear(x, w, None, "gelu")
            assert ref.worst(out, wy, by) <= 1
            assert bool((out_wide[:, :f0] == 7).all()) and bool((out_wide[:, f0 + F:] == 7).all())
        dy, pre = out_wide[:, 3:3 + F], rand(gen, T, 2 * F, dtype=dtype)
        got = pk.gated_linear_backward(x, w, dy, pre)
        want, bound = ref.gated_linear_backward(x, w, dy, pre, "gelu")
        assert all(ref.worst(g, v, b) <= 1 for g, v, b in zip(got, want, bound))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_sums(pk, gen, dtype):
    """Sums that the tensor pipe hands over in phases, for a lone CTA's tile and a pair's."""
    for T, K, F in ((150, 20000, 70), (3000, 17000 if dtype == torch.bfloat16 else 2100, 600)):
        x, w = rand(gen, T, K, dtype=dtype), rand(gen, 2 * F, K, std=K**-0.5, dtype=dtype)
        y, pre = pk.gated_linear(x, w, return_pre=True)
        (wy, wz), (by, bz) = ref.gated_linear(x, w, None, "gelu")
        assert ref.worst(pre, wz, bz) <= 1 and ref.worst(y, wy, by) <= 1


def test_no_rows(pk, gen):
    x, w = rand(gen, 0, 16), rand(gen, 20, 16)
    y, pre = pk.gated_linear(x, w, return_pre=True)
    assert y.shape == (0, 10) and pre.shape == (0, 20)
    dx, dw, db = pk.gated_linear_backward(x, w, y, pre)
    assert dx.shape == (0, 16) and not bool(dw.any()) and not bool(db.any())
    q, s = torch.zeros(0, 16, device="cuda").to(torch.float8_e4m3fn), torch.zeros(0, device="cuda")
    wq, ws = pk.quantize_rows(w)
    assert pk.linear_q8(q, s, wq, ws).shape == (0, 20)


def test_streams_and_graphs(pk, gen):
    T, K, F = 500, 256, 320
    x, w, dy = (rand(gen, *s, dtype=torch.bfloat16) for s in ((T, K), (2 * F, K), (T, F)))
    y, pre = pk.gated_linear(x, w, return_pre=True)
    grads = pk.gated_linear_backward(x, w, dy, pre)
    xq, xs = pk.quantize_rows(x)
    wq, ws = pk.quantize_rows(w)
    z = pk.linear_q8(xq, xs, wq, ws, act="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pk.gated_linear(x, w, stream=s), pk.linear_q8(xq, xs, wq, ws, act="gelu", stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], y) and torch.equal(got[1], z)
    sx = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gy, gpre = pk.gated_linear(sx, w, return_pre=True)
        ggrads = pk.gated_linear_backward(sx, w, dy, gpre)
        gq, gs = pk.quantize_rows(sx)
        gz = pk.linear_q8(gq, gs, wq, ws, act="gelu")
    sx.copy_(x)
    g.replay()
    assert torch.equal(gy, y) and torch.equal(gz, z) and all(torch.equal(a, b) for a, b in zip(ggrads, grads))


# ------------------------------------------------------------------------------------------ 8-bit rows


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 1024, 4096), (2, 528, 33), (3, 4096, 100), (4, 64, 300), (5, 32, 40), (17, 2048, 264), (129, 80, 136),
                                   (251, 768, 768), (300, 64, 257), (1000, 528, 1003), (513, 1024, 264), (4096, 128, 512), (20000, 64, 256)])
def test_linear_q8(pk, gen, dtype, T, K, N):
    xq, xs = pk.quantize_rows(rand(gen, T, K))
    wq, ws = pk.quantize_rows(rand(gen, N, K, std=K**-0.5))
    bias, res = rand(gen, N, dtype=dtype), rand(gen, T, N, dtype=dtype)
    for act, b, r in (("none", None, None), ("gelu", bias, res), ("silu", bias, None), ("relu", None, res)):
        y = pk.linear_q8(xq, xs, wq, ws, b, r, act, out_dtype=dtype)
        want, bound = ref.linear_q8(xq, xs, wq, ws, b, r, act, dtype)
        assert y.dtype == dtype and ref.worst(y, want, bound) <= 1
    assert torch.equal(pk.linear_q8(xq, xs, wq, ws, None, res, "relu", out=res), y)  # onto the residual
    assert pk.last_status() == 0


@pytest.mark.parametrize("T", [1, 300])
def test_linear_q8_strided_rows(pk, gen, T):
    K, N = 128, 96
    q, xs = pk.quantize_rows(rand(gen, T, 3 * K))
    wq, ws = pk.quantize_rows(rand(gen, N, K))
    wide = torch.full((T, N + 9), 7.0, device="cuda", dtype=torch.bfloat16)
    for k0 in (0, 144):
        x, out = q[:, k0:k0 + K], wide[:, 5:5 + N]
        pk.linear_q8(x, xs, wq, ws, out=out)
        want, bound = ref.linear_q8(x, xs, wq, ws, None, None, "none", torch.bfloat16)
        assert ref.worst(out, want, bound) <= 1
        assert bool((wide[:, :5] == 7).all()) and bool((wide[:, 5 + N:] == 7).all())


@pytest.mark.parametrize("T,K,N", [(1, 256, 70), (2, 256, 70), (4, 256, 70), (5, 8192, 130), (64, 8192, 256), (700, 256, 130), (20000, 64, 256)])
@pytest.mark.parametrize("small,large", [(1e-25, 1e-19), (1e25, 1e15), (1e-36, 1e5)])
def test_linear_q8_scales_of_any_size(pk, gen, T, K, N, small, large):
    """Scales whose product is past fp32's range though neither the scaled sum nor the result is, for few rows, splits of k and whole tiles; a row of zeros
    gives zeros."""
    xq, _ = pk.quantize_rows(rand(gen, T, K))
    wq, _ = pk.quantize_rows(rand(gen, N, K))
    if small * large > 1e38:  # small sums: one small number a row
        xq, wq = (torch.zeros_like(t.float()) for t in (xq, wq))
        xq[:, 5], wq[:, 5] = 2.0**-9, 2.0**-8
        xq, wq = xq.to(torch.float8_e4m3fn), wq.to(torch.float8_e4m3fn)
    xq.view(torch.uint8)[T // 2 :: 3] = 0
    xs, ws = (1 + torch.rand(T, generator=gen, device="cuda")) * small, (1 + torch.rand(N, generator=gen, device="cuda")) * large
    y = pk.linear_q8(xq, xs, wq, ws, out_dtype=torch.float32)
    want, bound = ref.linear_q8(xq, xs, wq, ws, None, None, "none", torch.float32)
    assert bool(want.any()) or T == 1
    assert ref.worst(y, want, bound) <= 1 and not bool(y[T // 2 :: 3].any())


@pytest.mark.parametrize("T", [2, 200])
def test_linear_q8_undefined_rows(pk, gen, T):
    """A row that could not be scaled has no value; the others keep theirs."""
    x = rand(gen, T, 64)
    x[1, 5] = float("nan")
    xq, xs = pk.quantize_rows(x)
    wq, ws = pk.quantize_rows(rand(gen, 40, 64))
    y = pk.linear_q8(xq, xs, wq, ws, out_dtype=torch.float32)
    assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all()) and bool(y[2:].isfinite().all())


def test_linear_q8_long_sums(pk, gen):
    """fp32 results of sums that the tensor pipe hands over in phases."""
    xq, xs = pk.quantize_rows(rand(gen, 700, 16384).abs())
    wq, ws = pk.quantize_rows(rand(gen, 1000, 16384).abs())
    y = pk.linear_q8(xq, xs, wq, ws, out_dtype=torch.float32)
    want = (xq.float().double() @ wq.float().double().T) * torch.outer(xs.double(), ws.double())
    # terms of one sign: at most 2048 of them in 64 steps of the pipe, each losing 2^-24 of the sum, then as few joins
    assert float(((y.double() - want) / want).abs().max()) <= 80 * 2.0**-24
