"""Log probabilities of given tokens, entropy, the likeliest words and their gradient against their definitions in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
# rows in a warp's registers, a block's rows, and rows over two to eight blocks; odd lengths put rows off the 16-byte grid
SIZES = [(1, 1), (3, 2), (5, 9), (64, 100), (11, 1023), (7, 1024), (5, 1025), (400, 1031), (320, 9000), (150, 12345), (40, 32003), (3, 50000),
         (1, 131072), (2, 200001), (1, 40007)]


def rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(99)
    return g


def check(pk, z, labels, top):
    got = pk.token_logprobs(z, labels, top=top)
    want, bound = ref.token_logprobs(z, labels, top)
    for name, g, v, b in zip(("logp", "lse", "entropy"), got, want, bound):
        assert ref.worst(g, v, b) <= 1, name
    if top:
        assert got[4].dtype == torch.int64 and torch.equal(got[4], want[4])
        assert ref.worst(got[3], want[3], bound[3]) <= 1
    else:
        assert got[3] is None and got[4] is None
    assert pk.last_status() == 0
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_logprobs(pk, gen, dtype, T, V):
    z = rand(gen, T, V, std=2.5, dtype=dtype)
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    whole = check(pk, z, labels, min(64, V))
    for top in (0, 1, 5, 17):
        if top <= V:
            part = check(pk, z, labels, top)
            assert all(torch.equal(a, b) for a, b in zip(part[:3], whole[:3]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_logprobs_backward(pk, gen, dtype, T, V):
    z = rand(gen, T, V, std=2.5, dtype=dtype)
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    _, lse, entropy, _, _ = pk.token_logprobs(z, labels)
    g, h = rand(gen, T), rand(gen, T, std=0.3)
    for dent in (h, None):
        d = pk.token_logprobs_backward(z, labels, lse, entropy, g, dentropy=dent)
        want, bound = ref.token_logprobs_backward(z, labels, lse, entropy, g, dent)
        assert ref.worst(d, want, bound) <= 1
    pk.token_logprobs_backward(z, labels, lse, None, g, out=z)  # onto the logits
    assert torch.equal(z, d)


def test_gradient_against_differences(pk, gen):
    T, V = 20, 300
    z, labels = rand(gen, T, V, std=2.0), torch.randint(0, V, (T,), generator=gen, device="cuda")
    cl, ch = rand(gen, T), rand(gen, T)
    _, lse, entropy, _, _ = pk.token_logprobs(z, labels)
    d = pk.token_logprobs_backward(z, labels, lse, entropy, cl, dentropy=ch)
    s, way = 2.0**-7, rand(gen, T, V)

    def f(z):
        logp, _, entropy, _, _ = pk.token_logprobs(z, labels)
        return float((logp.double() * cl.double()).sum() + (entropy.double() * ch.double()).sum())

    # (third derivatives below s^2, roundings 2^-22 |f| / s: both below 2e-3 of the slope's terms)
    slope, want = (f(z + s * way) - f(z - s * way)) / (2 * s), float((d.double() * way.double()).sum())
    assert abs(slope - want) <= 2e-3 * float((d.double().abs() * way.double().abs()).sum())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50, 900, 6000, 70001])
def test_masked_and_equal_logits(pk, gen, dtype, V):
    """Rows of -inf but for a few words, of the type's lowest value, of equal logits, of zeros of both signs."""
    low = torch.finfo(dtype).min
    z = rand(gen, 9, V, dtype=dtype)
    z[0] = float("-inf")
    z[0, V - 1], z[0, 3] = 1.0, 2.0
    z[1] = low
    z[2] = low
    z[2, V // 2] = 0.5
    z[3] = 1.25
    z[4] = 0.0
    z[4, ::2] = -0.0
    z[5, :V - 2] = float("-inf")
    z[6] = 0.0
    z[6, V // 3] = float("-inf")
    z[7] = (torch.arange(V, device="cuda") % 3).to(dtype)
    z[8] = -z[7]
    labels = torch.tensor([3, 5, V // 2, 0, 1, V - 1, 2, V - 1, -1], device="cuda")
    top = min(64, V)
    got = check(pk, z, labels, top)
    _, lse, entropy, _, _ = got
    g, h = rand(gen, 9), rand(gen, 9)
    d = pk.token_logprobs_backward(z, labels, lse, entropy, g, dentropy=h)
    want, bound = ref.token_logprobs_backward(z, labels, lse, entropy, g, h)
    assert ref.worst(d, want, bound) <= 1
    assert bool((d[0, 4:V - 1] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [70, 5000, 70001])
def test_rows_without_a_word(pk, gen, dtype, V):
    """Every logit -inf: nothing can be, and nothing is undefined; NaN and +inf are, and the rows beside them are not touched."""
    z = rand(gen, 5, V, dtype=dtype)
    z[0] = float("-inf")
    z[1, 7] = float("nan")
    z[2, 9], z[2, 30] = float("inf"), float("nan")
    z[3, 8], z[3, 40] = float("inf"), float("inf")
    labels = torch.tensor([2, 2, 2, 8, 2], device="cuda")
    top = 12
    logp, lse, entropy, top_logp, top_idx = pk.token_logprobs(z, labels, top=top)
    ninf = float("-inf")
    assert float(lse[0]) == ninf and float(logp[0]) == ninf and float(entropy[0]) == 0 and bool((top_logp[0] == ninf).all())
    assert top_idx[0].tolist() == list(range(top))
    assert bool(lse[1:4].isnan().all()) and bool(entropy[1:4].isnan().all()) and bool(logp[1:4].isnan().all())
    key = torch.where(z.isnan(), float("inf"), z.double())
    key[2, 30] = 1e300
    key[2, 9] = 1e299  # NaN above all numbers
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(top_idx, order)
    want, bound = ref.token_logprobs(z[4:], labels[4:], top)
    assert ref.worst(lse[4:], want[1], bound[1]) <= 1 and ref.worst(top_logp[4:], want[3], bound[3]) <= 1
    g = torch.ones(5, device="cuda")
    d = pk.token_logprobs_backward(z[:1], labels[:1], lse[:1], entropy[:1], g[:1], dentropy=g[:1])
    assert bool((d[0, 3:] == 0).all()) and bool(d.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(1, 65536), (400, 65536), (700, 40000)])
def test_large_words_side_by_side(pk, gen, dtype, T, V):
    """Many candidates in few threads' words, so that their list overflows: the likeliest are still exact."""
    z = rand(gen, T, V, dtype=dtype)
    thread = (torch.arange(V, device="cuda") // 8) % 256
    z[:, thread < 40] += 30
    z[-1, thread < 40] = 40.0
    check(pk, z, torch.randint(0, V, (T,), generator=gen, device="cuda"), 64)
    z[0] = torch.arange(V, device="cuda").to(dtype) / V  # rising, and falling
    z[-1] = z[0].flip(0)
    check(pk, z, torch.randint(0, V, (T,), generator=gen, device="cuda"), 33)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,top", [(705, 64), (1000, 16), (1500, 33), (2027, 64), (2032, 5), (2033, 16)])
def test_many_rows_of_middle_length(pk, gen, dtype, V, top):
    """More rows than there are warps, off the 16-byte grid too: random ones, masked ones, equal ones, one large word in a chunk."""
    T = 2700
    z = rand(gen, T, V + 3, std=2.5, dtype=dtype)[:, 3:]
    z[0] = float("-inf")
    z[0, V - 1], z[0, 3] = 1.0, 2.0
    z[1] = torch.finfo(dtype).min
    z[2] = 1.25
    z[3, : V - 2] = float("-inf")
    z[4] = (torch.arange(V, device="cuda") % 3).to(dtype)
    z[5, : V // 2] += 30
    z[6] = torch.arange(V, device="cuda").to(dtype) / V
    z[7, ::8] = 20.0
    z[T - 1, 100:300] = 25.0
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    labels[0] = 3
    check(pk, z, labels, top)
    check(pk, z.contiguous(), labels, top)
    check(pk, z.contiguous(), labels, 0)  # (not the same bits: how a row is shared out, and so its sums' order, goes by top too)
    z[9, 7] = float("nan")
    z[2600, 9], z[2600, 30] = float("inf"), float("nan")
    _, lse, _, _, top_idx = pk.token_logprobs(z, labels, top=top)
    key = torch.where(z.isnan(), float("inf"), z.double())
    key[2600, 9] = 1e299  # NaN above all numbers
    assert torch.equal(top_idx, torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top])
    assert bool(lse[9].isnan()) and bool(lse[2600].isnan()) and bool(lse[10:2600].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(5, 8192), (36, 33000), (70, 17000), (18, 70001)])
def test_rows_over_several_blocks(pk, gen, dtype, T, V):
    """Two, four and eight blocks a row: their likeliest words all in the first block's part, in the last's, one in each, equal ones."""
    z = rand(gen, T, V, std=2.0, dtype=dtype)
    z[0, :100] += 20
    z[1, -100:] += 20
    z[2, :: V // 50] += 20
    z[3] = 0.75
    z[4] = float("-inf")
    z[4, V // 2] = 0.0
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    labels[4] = V // 2
    for top in (64, 1, 33, 0):
        check(pk, z, labels, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(300, 1040), (300, 2100), (300, 4588), (160, 8192), (64, 8192), (300, 8193)])
def test_a_block_a_row(pk, gen, dtype, T, V):
    """Rows of blocks of 64 and of 128 threads, by how many words are asked for: each against its definition (not against each other,
    whose sums' order differs), on the 16-byte grid and off it."""
    wide = rand(gen, T, V + 8, std=2.5, dtype=dtype)
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    for shift in (0, 8, 3):
        z = wide[:, shift : shift + V]
        for top in (0, 16, 32, 33, 64):
            check(pk, z, labels, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [77, 4000, 33001])
def test_strided_rows(pk, gen, dtype, V):
    wide, out = rand(gen, 6, V + 13, std=2.0, dtype=dtype), rand(gen, 6, V + 13, dtype=dtype)
    labels = torch.randint(0, V, (6,), generator=gen, device="cuda")
    for shift in (0, 1, 5, 8):
        z, o = wide[:, shift:shift + V], out[:, 3:3 + V]
        got = check(pk, z, labels, 20)
        same = pk.token_logprobs(z.clone(), labels, top=20)
        assert torch.equal(got[4], same[4])
        keep = out.clone()
        g = rand(gen, 6)
        pk.token_logprobs_backward(z, labels, got[1], got[2], g, out=o)
        want, bound = ref.token_logprobs_backward(z, labels, got[1], got[2], g, None)
        assert ref.worst(o, want, bound) <= 1
        assert torch.equal(out[:, :3], keep[:, :3]) and torch.equal(out[:, 3 + V:], keep[:, 3 + V:])


def test_large_logits_keep_their_differences(pk, gen):
    z = rand(gen, 50, 3000) + 1e4
    labels = torch.randint(0, 3000, (50,), generator=gen, device="cuda")
    logp, _, entropy, _, _ = pk.token_logprobs(z, labels)
    small = z.double() - 1e4
    want = torch.log_softmax(small, 1)
    assert float((logp.double() - want.gather(1, labels[:, None])[:, 0]).abs().max()) < 1e-5
    assert float((entropy.double() + (want.exp() * want).sum(1)).abs().max()) < 1e-5


def test_bad_labels(pk, gen):
    z = rand(gen, 4, 500)
    labels = torch.tensor([1, 500, -5, 1 << 40], device="cuda")
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    logp, lse, entropy, _, _ = pk.token_logprobs(z, labels, status=status)
    assert int(status) == 11 and pk.last_status() == 0
    assert logp.isnan().tolist() == [False, True, False, True] and float(logp[2]) == 0 and bool(lse.isfinite().all())
    pk.token_logprobs(z, labels)
    assert pk.last_status() == 11 and pk.last_status() == 0
    d = pk.token_logprobs_backward(z, labels, lse, entropy, torch.ones(4, device="cuda"))
    assert bool((d[1:] == 0).all()) and bool(d[0].any())


def test_no_rows(pk):
    z, labels = torch.zeros(0, 10, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    got = pk.token_logprobs(z, labels, top=3)
    assert [tuple(t.shape) for t in got] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    f = torch.zeros(0, device="cuda")
    assert pk.token_logprobs_backward(z, labels, f, f, f).shape == (0, 10)


def test_past_32_bits(pk, gen):
    """Logits past 2^32 bytes: the last rows."""
    V, T = 131073, 16500
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    z[-3:] = rand(gen, 3, V, std=2.0, dtype=torch.bfloat16)
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    got = pk.token_logprobs(z, labels, top=9)
    want, bound = ref.token_logprobs(z[-3:], labels[-3:], 9)
    assert torch.equal(got[4][-3:], want[4]) and ref.worst(got[0][-3:], want[0], bound[0]) <= 1
    g = rand(gen, T)
    d = pk.token_logprobs_backward(z, labels, got[1], None, g)
    want, bound = ref.token_logprobs_backward(z[-3:], labels[-3:], got[1][-3:], None, g[-3:], None)
    assert ref.worst(d[-3:], want, bound) <= 1


def test_streams_and_graphs(pk, gen):
    z, labels = rand(gen, 3, 40000, dtype=torch.bfloat16), torch.tensor([5, -1, 39999], device="cuda")
    want = pk.token_logprobs(z, labels, top=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pk.token_logprobs(z, labels, top=8, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = torch.zeros_like(z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pk.token_logprobs(held, labels, top=8)
        d = pk.token_logprobs_backward(held, labels, got[1], got[2], got[0], dentropy=got[2])
    held.copy_(z)
    for _ in range(2):
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(d, pk.token_logprobs_backward(z, labels, want[1], want[2], want[0], dentropy=want[2]))
