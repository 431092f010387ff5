"""The token-row operators' refusals, and the reference generator's published values: no GPU needed (the binding checks
shapes and types before anything reaches the library, the library its arguments before any CUDA call)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import rope_cu_tile_gb300 as pk  # noqa: E402
import rows_ref as ref  # noqa: E402


class Fake:
    """A tensor's looks on a CUDA device, without a GPU."""

    def __init__(self, t, device="cuda:0"):
        self._t, self.device, self.is_cuda = t, torch.device(device), True
        self.shape, self.dtype = t.shape, t.dtype

    def __getattr__(self, name):
        return getattr(self._t, name)


def fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return Fake(torch.zeros(*shape, dtype=dtype), device)


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pk.linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        pk.dropout(x, 0.1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pk.cross_entropy(x, w, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="dtype"):
        pk.linear(x.double(), w.double())


def test_linear_refusals():
    x, w = fake(4, 8), fake(6, 8)
    with pytest.raises(ValueError, match="w must be"):
        pk.linear(x, fake(6, 7))
    with pytest.raises(TypeError, match="w must be"):
        pk.linear(x, fake(6, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="different devices"):
        pk.linear(x, fake(6, 8, device="cuda:1"))
    with pytest.raises(ValueError, match="bias"):
        pk.linear(x, w, bias=fake(5))
    with pytest.raises(ValueError, match="residual"):
        pk.linear(x, w, residual=fake(4, 5))
    with pytest.raises(ValueError, match="act must be one of"):
        pk.linear(x, w, act="tanh")
    for p in (1.0, -0.1, float("nan"), 1 - 2.0**-18):
        with pytest.raises(ValueError, match="p must be"):
            pk.linear(x, w, p=p)
    for kw in (dict(seed=-1), dict(offset=1 << 64)):
        with pytest.raises(ValueError, match="64-bit"):
            pk.linear(x, w, p=0.5, **kw)
    with pytest.raises(ValueError, match="out must be"):
        pk.linear(x, w, out=fake(4, 7))
    with pytest.raises(ValueError, match="contiguous rows"):
        pk.linear(Fake(torch.zeros(8, 4, dtype=torch.bfloat16).T), w)
    with pytest.raises(ValueError, match="overlapping rows"):
        pk.linear(Fake(torch.zeros(1, 8, dtype=torch.bfloat16).expand(4, 8)), w)
    with pytest.raises(ValueError, match="w must be contiguous"):
        pk.linear(x, Fake(torch.zeros(6, 9, dtype=torch.bfloat16)[:, :8]))
    with pytest.raises(ValueError, match="at least one"):
        pk.linear(x, fake(0, 8))
    with pytest.raises(ValueError, match="pre-activation"):
        pk.linear_backward(x, w, fake(4, 6), act="gelu")
    with pytest.raises(ValueError, match="pre must be"):
        pk.linear_backward(x, w, fake(4, 6), pre=fake(4, 7), act="gelu")
    with pytest.raises(ValueError, match="dy must be"):
        pk.linear_backward(x, w, fake(3, 6))
    with pytest.raises(ValueError, match="status"):
        pk.linear(x, w, status=fake(2, dtype=torch.int32))

    class S:
        device = torch.device("cuda:1")

    with pytest.raises(ValueError, match="stream"):
        pk.linear(x, w, stream=S())


def test_outputs_over_inputs_are_refused():
    wide = torch.zeros(4, 32, dtype=torch.bfloat16)
    x, w = Fake(wide[:, :8]), fake(8, 8)
    with pytest.raises(ValueError, match="overlaps"):
        pk.linear(x, w, out=Fake(wide[:, 4:12]))
    with pytest.raises(ValueError, match="overlaps"):
        pk.dropout(x, 0.5, 1, out=Fake(wide[:, 1:9]))
    assert not pk._overlap(wide[:, :8], wide[:, 8:16])  # columns beside each other
    assert not pk._overlap(wide[:, 8:16], wide[:, :8])
    assert not pk._overlap(wide[:, 24:], wide[:, :8])
    assert pk._overlap(wide[:, 24:], wide[1:, :9][:, 0:9]) is False  # the next row's first columns
    assert pk._overlap(wide[:, :9], wide[:, 8:])
    assert pk._overlap(wide, wide[2:3, 4:5])
    assert not pk._overlap(wide[:2], wide[2:])


def test_cross_entropy_refusals():
    x, w, labels = fake(4, 8), fake(6, 8), fake(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="labels"):
        pk.cross_entropy(x, w, fake(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="labels"):
        pk.cross_entropy(x, w, fake(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="bias"):
        pk.cross_entropy(x, w, labels, bias=fake(6, dtype=torch.float32))
    with pytest.raises(ValueError, match="lse"):
        pk.cross_entropy_backward(x, w, labels, fake(4), fake(4, dtype=torch.float32))
    with pytest.raises(ValueError, match="dloss"):
        pk.cross_entropy_backward(x, w, labels, fake(4, dtype=torch.float32), fake(1, dtype=torch.float32))


@pytest.fixture(scope="module")
def lib():
    from rope_cu_tile_gb300 import build

    build.build()
    return pk.load()


P, ODD, NULL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001), ctypes.c_void_p(0)


def test_linear_arguments_need_no_gpu(lib):
    def fwd(**kw):
        a = dict(dtype=1, x=P, ldx=8, w=P, bias=NULL, res=NULL, ldr=6, act=0, p=0.0, seed=0, off=0, T=4, N=6, K=8, y=P, ldy=6,
                 pre=NULL, ws=NULL, wb=0, status=NULL, stream=NULL)
        a.update(kw)
        return lib.pk_linear(*a.values())

    for kw in (dict(dtype=3), dict(T=-1), dict(T=(1 << 30) + 1), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(act=4),
               dict(act=-1), dict(p=1.0), dict(p=-0.5), dict(p=float("nan")), dict(ldx=7), dict(ldy=5), dict(res=P, ldr=5),
               dict(x=NULL), dict(w=NULL), dict(y=NULL), dict(wb=-1)):
        assert fwd(**kw) == 1, kw
    for kw in (dict(x=ODD), dict(w=ODD), dict(bias=ODD), dict(res=ODD), dict(y=ODD), dict(pre=ODD), dict(ws=ODD),
               dict(status=ODD), dict(dtype=0, y=ctypes.c_void_p(0x1002))):
        assert fwd(**kw) == 2, kw
    assert fwd(T=0, x=NULL, w=NULL, y=NULL) == 0

    def bwd(**kw):
        a = dict(dtype=1, x=P, ldx=8, w=P, dy=P, lddy=6, pre=NULL, act=0, p=0.0, seed=0, off=0, T=4, N=6, K=8, dx=P, dw=P, db=P,
                 ws=NULL, wb=0, status=NULL, stream=NULL)
        a.update(kw)
        return lib.pk_linear_backward(*a.values())

    for kw in (dict(dtype=9), dict(act=2), dict(dy=NULL), dict(x=NULL), dict(w=NULL), dict(lddy=5), dict(p=2.0)):
        assert bwd(**kw) == 1, kw
    for kw in (dict(dx=ODD), dict(dw=ODD), dict(db=ODD), dict(dy=ODD), dict(pre=ODD)):
        assert bwd(**kw) == 2, kw
    n = ctypes.c_int64(-1)
    assert lib.pk_linear_workspace(1, P, 8, P, 0, 6, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.pk_linear_workspace(1, P, 7, P, 4, 6, 8, ctypes.byref(n)) == 1
    assert lib.pk_linear_backward_workspace(1, P, 8, P, P, 6, 0, 0.0, 1, 1, 1, 0, 6, 8, ctypes.byref(n)) == 0


def test_dropout_and_cross_entropy_arguments_need_no_gpu(lib):
    def drop(**kw):
        a = dict(dtype=1, x=P, ldx=6, res=NULL, ldr=6, p=0.5, seed=0, off=0, T=4, N=6, y=P, ldy=6, stream=NULL)
        a.update(kw)
        return lib.pk_dropout(*a.values())

    for kw in (dict(dtype=5), dict(T=-1), dict(N=0), dict(ldx=5), dict(ldy=5), dict(res=P, ldr=1), dict(p=1.0), dict(x=NULL),
               dict(y=NULL)):
        assert drop(**kw) == 1, kw
    assert drop(x=ODD) == 2 and drop(y=ODD) == 2 and drop(res=ODD) == 2
    assert drop(T=0, x=NULL, y=NULL) == 0

    def xent(**kw):
        a = dict(dtype=1, x=P, ldx=8, w=P, bias=NULL, labels=P, T=4, D=8, V=6, loss=P, lse=P, ws=NULL, wb=0, status=NULL,
                 stream=NULL)
        a.update(kw)
        return lib.pk_cross_entropy(*a.values())

    for kw in (dict(dtype=5), dict(T=-1), dict(D=0), dict(V=0), dict(V=(1 << 20) + 1), dict(ldx=7), dict(x=NULL), dict(w=NULL),
               dict(labels=NULL), dict(loss=NULL), dict(lse=NULL)):
        assert xent(**kw) == 1, kw
    assert xent(labels=ctypes.c_void_p(0x1004)) == 2 and xent(loss=ODD) == 2 and xent(bias=ODD) == 2
    assert xent(T=0, x=NULL, w=NULL, labels=NULL, loss=NULL, lse=NULL) == 0

    def bwd(**kw):
        a = dict(dtype=1, x=P, ldx=8, w=P, bias=NULL, labels=P, lse=P, dloss=P, T=4, D=8, V=6, dx=P, dw=P, db=P, ws=NULL, wb=0,
                 status=NULL, stream=NULL)
        a.update(kw)
        return lib.pk_cross_entropy_backward(*a.values())

    for kw in (dict(lse=NULL), dict(dloss=NULL), dict(labels=NULL), dict(dtype=-1)):
        assert bwd(**kw) == 1, kw
    assert bwd(dx=ODD) == 2 and bwd(db=ODD) == 2 and bwd(dloss=ODD) == 2


def test_reference_generator_matches_its_published_values():
    """The known answers of Philox4x32-10: counter and key all zeros, and all ones."""
    def words(c0, c1, offset, seed):
        # p just above each 16-bit piece drops it, p at it keeps it: read the pieces back through the mask
        got = []
        for j in range(8):
            lo, hi = 0, 65535
            while lo < hi:
                mid = (lo + hi + 1) // 2
                if ref.keep_mask_at(c0, c1, mid, seed, offset)[j]:
                    lo = mid
                else:
                    hi = mid - 1
            got.append(lo)
        return [got[2 * i] | got[2 * i + 1] << 16 for i in range(4)]

    assert words(0, 0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = (1 << 64) - 1
    assert words(0xFFFFFFFF, 0xFFFFFFFF, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
