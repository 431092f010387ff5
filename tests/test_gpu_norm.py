"""The root-mean-square norm, its gradient and its 8-bit rows against their definitions in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
# rows shared out over 8 threads, a warp and blocks; odd lengths; the longest
SIZES = [(1, 1), (1, 64), (3, 8), (70, 56), (33, 65), (5, 256), (257, 200), (1, 1024), (251, 768), (1000, 1023), (77, 1032), (9, 4096),
         (300, 2623), (4, 4097), (3, 16384), (5, 16383), (20000, 64), (4099, 768)]


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(4321)
    return g


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_norm(pk, gen, dtype, T, D):
    x, r, w = rand(gen, T, D, std=1.5, dtype=dtype), rand(gen, T, D, dtype=dtype), rand(gen, D, dtype=dtype)
    y, h = pk.rms_norm(x, w, residual=r, eps=1e-5)
    (wy, wh), (by, bh), _ = ref.rms_norm(x, w, r, 1e-5)
    assert ref.worst(y, wy, by) <= 1 and ref.worst(h, wh, bh) <= 1
    y = pk.rms_norm(x, w)
    (wy, _), (by, _), _ = ref.rms_norm(x, w, None, 1e-6)
    assert ref.worst(y, wy, by) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_norm_q8(pk, gen, dtype, T, D):
    x, r, w = rand(gen, T, D, std=1.5, dtype=dtype), rand(gen, T, D, dtype=dtype), rand(gen, D, dtype=dtype)
    q, scale, h = pk.rms_norm_q8(x, w, residual=r)
    assert q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float32
    (wy, wh), (_, bh), ey = ref.rms_norm(x, w, r, 1e-6)
    ws = wy.abs().amax(1) / 448
    assert ref.worst(scale, ws, 2.0**-16 * ws) <= 1 and ref.worst(h, wh, bh) <= 1
    assert ref.worst(q.double() * scale.double()[:, None], wy, ref.e4m3_bound(wy, ey, ws)) <= 1
    assert torch.equal(q.float().abs().amax(1), torch.full((T,), 448.0, device="cuda"))
    # x itself in 8 bits
    q, scale = pk.quantize_rows(x)
    X = x.double()
    ws = X.abs().amax(1) / 448
    assert ref.worst(scale, ws, 2.0**-22 * ws) <= 1
    assert ref.worst(q.double() * scale.double()[:, None], X, ref.e4m3_bound(X, 2.0**-21 * X.abs(), ws)) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_norm_backward(pk, gen, dtype, T, D):
    h, w = rand(gen, T, D, std=1.5, dtype=dtype), rand(gen, D, dtype=dtype)
    dy, dh = rand(gen, T, D, std=0.1, dtype=dtype), rand(gen, T, D, std=0.1, dtype=dtype)
    for up in (dh, None):
        dx, dw = pk.rms_norm_backward(h, w, dy, dh=up, eps=1e-5)
        (wx, ww), (bx, bw) = ref.rms_norm_backward(h, w, dy, up, 1e-5)
        assert ref.worst(dx, wx, bx) <= 1 and ref.worst(dw, ww, bw) <= 1
    one, none = pk.rms_norm_backward(h, w, dy, eps=1e-5, need_dw=False)
    assert none is None and torch.equal(one, dx)
    none, one = pk.rms_norm_backward(h, w, dy, eps=1e-5, need_dx=False)
    assert none is None and torch.equal(one, dw)


def test_norm_gradient_against_differences(pk, gen):
    """fp32: the gradient against central differences of the library's own forward, in a random direction."""
    T, D = 30, 96
    x, r, w = rand(gen, T, D), rand(gen, T, D), rand(gen, D)
    cy, ch = rand(gen, T, D), rand(gen, T, D)
    _, h = pk.rms_norm(x, w, residual=r)
    dx, dw = pk.rms_norm_backward(h, w, cy, dh=ch)
    # a step s: the third derivative's share is some s^2, the rounding of the values 2^-23 |f| sqrt(TD) / s: both below 2e-3
    s = 2.0**-7

    def f(x, r, w):
        y, h = pk.rms_norm(x, w, residual=r)
        return float((y.double() * cy.double()).sum() + (h.double() * ch.double()).sum())

    for t, g, put in ((x, dx, 0), (r, dx, 1), (w, dw, 2)):
        d = rand(gen, *t.shape)
        at = lambda k: [v + k * s * d if i == put else v for i, v in enumerate((x, r, w))]  # noqa: E731
        slope, want = (f(*at(1)) - f(*at(-1))) / (2 * s), float((g.double() * d.double()).sum())
        assert abs(slope - want) <= 2e-3 * float((g.double().abs() * d.double().abs()).sum())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [100, 1024, 5000])
def test_special_rows(pk, gen, dtype, D):
    """Rows of zeros, of one element, of the type's largest and smallest numbers, infinite and undefined ones, beside others."""
    x, w = rand(gen, 9, D, dtype=dtype), rand(gen, D, dtype=dtype)
    most = torch.finfo(dtype).max
    x[1] = 0
    x[2] = 0
    x[2, D // 2] = 1
    x[3] = most / 4
    x[4] = torch.finfo(dtype).smallest_normal
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7, ::3] = most
    ok = [0, 1, 2, 3, 4, 7, 8]
    y = pk.rms_norm(x, w)
    (wy, _), (by, _), _ = ref.rms_norm(x[ok], w, None, 1e-6)
    # some results lie among the smallest numbers (row 7: 1 beside the largest): bf16's are 2^-133 apart, half a step is 2^-134;
    # fp32's are 2^-149 apart: h f is off by 2^-150, which is multiplied by w, and the product with w by as much again
    small = 2.0**-150 * (1 + float(w.float().abs().max())) + (2.0**-134 if dtype == torch.bfloat16 else 0.0)
    by = by + small
    assert ref.worst(y[ok], wy, by) <= 1
    assert bool(y[6].isnan().all()) and bool(y[5, 7].isnan())
    q, scale = pk.rms_norm_q8(x, w)
    assert float(scale[1]) == 0 and bool((q[1].float() == 0).all())
    assert bool(scale[5].isnan()) and bool(scale[6].isnan()) and bool(scale[ok].isfinite().all())
    q, scale = pk.quantize_rows(x)
    assert float(scale[5]) == float("inf") and bool(scale[6].isnan())
    X = x[ok].double()
    bound = ref.e4m3_bound(X, 2.0**-21 * X.abs(), X.abs().amax(1) / 448) + 2.0**-149 * 448
    assert ref.worst(q[ok].double() * scale[ok].double()[:, None], X, bound) <= 1
    dy = rand(gen, 9, D, std=0.1, dtype=dtype)
    dx, dw = pk.rms_norm_backward(x[ok].contiguous(), w, dy[ok].contiguous())
    (wx, ww), (bx, bw) = ref.rms_norm_backward(x[ok], w, dy[ok], None, 1e-6)
    # (the largest rows' gradients lie there: the difference and three products round to multiples of 2^-149 before dx does)
    assert ref.worst(dx, wx, bx + small + 4 * 2.0**-149) <= 1 and ref.worst(dw, ww, bw + small + 9 * 2.0**-149) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8192, 8189, 9000, 16384, 16377, 16383])
def test_rows_after_special_ones(pk, gen, dtype, D):
    """More long rows than there are blocks, after rows whose squares pass fp32's range (which are summed once more): every other row
    comes out as it does without them, bit for bit, and as in 64 bits."""
    T = 2500
    x, r, w = rand(gen, T, D, std=1.5, dtype=dtype), rand(gen, T, D, dtype=dtype), rand(gen, D, dtype=dtype)
    special = torch.zeros(T, dtype=torch.bool, device="cuda")
    special[3:140:7] = True
    special[700:760:3] = True
    odd = x.clone()
    odd[special] = torch.finfo(dtype).max / 4  # (past 2^64 but in fp16)
    odd[special.nonzero()[::2, 0], D // 3] = float("inf")
    want, got = pk.rms_norm_q8(x, w, residual=r), pk.rms_norm_q8(odd, w, residual=r)
    for a, b in zip(want, got):
        assert torch.equal(a[~special].view(torch.uint8), b[~special].view(torch.uint8))
    (wy, _), _, ey = ref.rms_norm(x, w, r, 1e-6)
    ws = wy.abs().amax(1) / 448
    ok = ~special
    assert ref.worst(got[1][ok], ws[ok], 2.0**-16 * ws[ok]) <= 1
    assert ref.worst(got[0][ok].double() * got[1][ok].double()[:, None], wy[ok], ref.e4m3_bound(wy[ok], ey[ok], ws[ok])) <= 1
    assert torch.equal(pk.rms_norm(odd, w)[ok], pk.rms_norm(x, w)[ok])
    assert torch.equal(pk.quantize_rows(odd)[1][ok], pk.quantize_rows(x)[1][ok])
    dx, _ = pk.rms_norm_backward(odd, w, r)
    assert torch.equal(dx[ok], pk.rms_norm_backward(x, w, r)[0][ok])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 96, 1024, 2000])
def test_strided_rows_and_in_place(pk, gen, dtype, D):
    T = 37
    for pad, shift in ((8, 0), (8, 8), (5, 3)):
        wide = [rand(gen, T, D + pad + 3, dtype=dtype) for _ in range(4)]
        x, r, out, hout = (t[:, shift:shift + D] for t in wide)
        keep = [t.clone() for t in wide]
        w = rand(gen, D, dtype=dtype)
        (wy, wh), (by, bh), _ = ref.rms_norm(x, w, r, 1e-6)
        y, h = pk.rms_norm(x, w, residual=r, out=out, h_out=hout)
        assert y.data_ptr() == out.data_ptr() and h.data_ptr() == hout.data_ptr()
        assert ref.worst(out, wy, by) <= 1 and ref.worst(hout, wh, bh) <= 1
        for t, k in zip(wide, keep):  # what lies beside
            assert torch.equal(t[:, :shift], k[:, :shift]) and torch.equal(t[:, shift + D:], k[:, shift + D:])
        # the stream updated in place, either of its two (contiguous copies: a row's sum may run in another order)
        y, h = pk.rms_norm(x.clone(), w, residual=r.clone())
        for i in (0, 1):
            a, b = x.clone(), r.clone()
            y2, h2 = pk.rms_norm(a, w, residual=b, h_out=(a, b)[i])
            assert torch.equal(y2, y) and torch.equal((a, b)[i], hout) and torch.equal(h, hout)
        q, scale, h2 = pk.rms_norm_q8(x, w, residual=r)
        assert torch.equal(h2, hout)
        dy, dh = r, x
        dx, dw = pk.rms_norm_backward(hout, w, dy, dh=dh)
        (wx, ww), (bx, bw) = ref.rms_norm_backward(hout, w, dy, dh, 1e-6)
        assert ref.worst(dx, wx, bx) <= 1 and ref.worst(dw, ww, bw) <= 1
        dx, _ = pk.rms_norm_backward(h, w, dy.clone(), dh=dh.clone())
        for i in (0, 1):
            a, b = dy.clone(), dh.clone()
            got, _ = pk.rms_norm_backward(h, w, a, dh=b, out=(a, b)[i])
            assert torch.equal(got, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D,ld,first", [(40, 131, 131, 3), (17, 1003, 1011, 0), (2, 77, 77, 5), (1, 30, 33, 1), (29, 9, 9, 7), (50, 5, 8, 2),
                                          (64, 3, 5, 1), (33, 260, 262, 2), (300, 4099, 4100, 4), (19, 16383, 16385, 1)])
def test_rows_that_begin_past_a_boundary(pk, gen, dtype, T, D, ld, first):
    """Rows `first` elements into an allocation and ld apart, equally in every matrix: what stands between and beside them (NaN here)
    is neither taken for theirs nor written."""

    def within(values=None, fill=float("nan")):
        whole = torch.full((first + T * ld + 8,), fill, device="cuda", dtype=dtype)
        view = whole[first : first + T * ld].view(T, ld)[:, :D] if ld > D else whole[first : first + T * D].view(T, D)
        if values is not None:
            view.copy_(values)
        return whole, view

    def beside(whole, view):
        rest = whole.clone()
        rest[first : first + T * ld].view(T, ld)[:, :D] = float("nan")
        assert bool(rest.isnan().all())
        return view

    x, r, w = rand(gen, T, D, std=1.5, dtype=dtype), rand(gen, T, D, dtype=dtype), rand(gen, D, dtype=dtype)
    out, h = within(), within()
    pk.rms_norm(within(x)[1], w, residual=within(r)[1], out=out[1], h_out=h[1])
    (wy, wh), (by, bh), ey = ref.rms_norm(x, w, r, 1e-6)
    assert ref.worst(beside(*out), wy, by) <= 1 and ref.worst(beside(*h), wh, bh) <= 1
    at = within(x)  # (the sum in the place of x)
    q, scale, _ = pk.rms_norm_q8(at[1], w, residual=within(r)[1], h_out=at[1])
    ws = wy.abs().amax(1) / 448
    assert ref.worst(beside(*at), wh, bh) <= 1
    assert ref.worst(q.double() * scale.double()[:, None], wy, ref.e4m3_bound(wy, ey, ws)) <= 1
    q, scale = pk.quantize_rows(within(x)[1])
    ws = x.double().abs().amax(1) / 448
    assert ref.worst(q.double() * scale.double()[:, None], x.double(), ref.e4m3_bound(x.double(), 2.0**-21 * x.double().abs(), ws)) <= 1
    dy, dh = rand(gen, T, D, std=0.1, dtype=dtype), rand(gen, T, D, std=0.1, dtype=dtype)
    at = within(dh)  # (the gradient in the place of dh)
    _, dw = pk.rms_norm_backward(within(x)[1], w, within(dy)[1], dh=at[1], out=at[1])
    (wx, ww), (bx, bw) = ref.rms_norm_backward(x, w, dy, dh, 1e-6)
    assert ref.worst(beside(*at), wx, bx) <= 1 and ref.worst(dw, ww, bw) <= 1


def test_no_rows(pk, gen):
    x, w = rand(gen, 0, 100), rand(gen, 100)
    y, h = pk.rms_norm(x, w, residual=x)
    assert y.shape == (0, 100) and h.shape == (0, 100)
    q, scale = pk.rms_norm_q8(x, w)
    assert q.shape == (0, 100) and scale.shape == (0,)
    dx, dw = pk.rms_norm_backward(x, w, x)
    assert dx.shape == (0, 100) and torch.equal(dw, torch.zeros_like(dw))


def test_past_32_bits(pk, gen):
    """A matrix past 2^32 bytes: its last rows."""
    T, D = (1 << 31) // 1024 + 300, 1024
    x, w = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), rand(gen, D, dtype=torch.bfloat16)
    x[:300], x[300:-300], x[-300:] = rand(gen, 300, D), 1.0, rand(gen, 300, D)
    y = pk.rms_norm(x, w)
    for part in (slice(0, 300), slice(T - 300, T)):
        (wy, _), (by, _), _ = ref.rms_norm(x[part], w, None, 1e-6)
        assert ref.worst(y[part], wy, by) <= 1


def test_odd_rows_past_32_bits(pk, gen):
    """The same of rows off the 16-byte grid, and their gradient."""
    T, D = (1 << 31) // 1023 + 300, 1023
    x, w = torch.ones(T, D, dtype=torch.bfloat16, device="cuda"), rand(gen, D, dtype=torch.bfloat16)
    x[:300], x[-300:] = rand(gen, 300, D), rand(gen, 300, D)
    y = pk.rms_norm(x, w)
    dx, _ = pk.rms_norm_backward(x, w, y, dh=x, need_dw=False)
    for part in (slice(0, 300), slice(T - 300, T)):
        (wy, _), (by, _), _ = ref.rms_norm(x[part], w, None, 1e-6)
        (wx, _), (bx, _) = ref.rms_norm_backward(x[part], w, y[part], x[part], 1e-6)
        assert ref.worst(y[part], wy, by) <= 1 and ref.worst(dx[part], wx, bx) <= 1


def test_streams_and_graphs(pk, gen):
    """Another stream than the tensors' own; a captured step replayed on new inputs."""
    T, D = 300, 768
    x, r, w, dy = (rand(gen, *s, dtype=torch.bfloat16) for s in ((T, D), (T, D), (D,), (T, D)))
    want = pk.rms_norm(x, w, residual=r)
    back = pk.rms_norm_backward(want[1], w, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pk.rms_norm(x, w, residual=r, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    sx, sr, sy = torch.zeros_like(x), torch.zeros_like(r), torch.zeros_like(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h = pk.rms_norm(sx, w, residual=sr)
        grads = pk.rms_norm_backward(h, w, sy)
    for a, b in ((sx, x), (sr, r), (sy, dy)):
        a.copy_(b)
    g.replay()
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and all(torch.equal(a, b) for a, b in zip(grads, back))
