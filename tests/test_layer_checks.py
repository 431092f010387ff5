"""Refusals of the norm, the 8-bit projection, the gated feed-forward, the token log probabilities and distillation: no GPU needed
(the binding checks shapes and types before anything reaches the library, the library its arguments before any CUDA call)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import rope_cu_tile_gb300 as pk  # noqa: E402
from test_rows_checks import Fake, fake  # noqa: E402

F8 = torch.float8_e4m3fn
NAN = float("nan")


def f32(*shape):
    return fake(*shape, dtype=torch.float32)


def i64(*shape):
    return fake(*shape, dtype=torch.int64)


def test_host_tensors_are_refused():
    x, w, labels = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: pk.rms_norm(x, w), lambda: pk.rms_norm_q8(x, w), lambda: pk.quantize_rows(x),
                 lambda: pk.rms_norm_backward(x, w, x), lambda: pk.gated_linear(x, torch.zeros(4, 8)),
                 lambda: pk.token_logprobs(x, labels), lambda: pk.distill(x, torch.zeros(9, 8), labels[:, None], x[:, :1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="dtype"):
        pk.rms_norm(x.double(), w.double())


def test_norm_refusals():
    x, w = fake(4, 8), fake(8)
    with pytest.raises(ValueError, match="w must be"):
        pk.rms_norm(x, fake(7))
    with pytest.raises(ValueError, match="w must be"):
        pk.rms_norm(x, fake(8, dtype=torch.float32))
    with pytest.raises(ValueError, match="residual"):
        pk.rms_norm(x, w, residual=fake(4, 9))
    with pytest.raises(TypeError, match="residual"):
        pk.rms_norm(x, w, residual=fake(4, 8, dtype=torch.float16))
    for eps in (0.0, -1e-6, NAN, float("inf"), 1e39):
        with pytest.raises(ValueError, match="eps"):
            pk.rms_norm(x, w, eps=eps)
        with pytest.raises(ValueError, match="eps"):
            pk.rms_norm_backward(x, w, x, eps=eps)
    for D in (0, 16385):
        with pytest.raises(ValueError, match="columns"):
            pk.rms_norm(fake(2, D), fake(D))
        with pytest.raises(ValueError, match="columns"):
            pk.quantize_rows(fake(2, D))
    with pytest.raises(ValueError, match="needs a residual"):
        pk.rms_norm(x, w, h_out=fake(4, 8))
    with pytest.raises(ValueError, match="out must be"):
        pk.rms_norm(x, w, out=fake(4, 7))
    with pytest.raises(ValueError, match="different devices"):
        pk.rms_norm(x, w, residual=fake(4, 8, device="cuda:1"))
    wide = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        pk.rms_norm(Fake(wide[:, :8]), w, out=Fake(wide[:, 4:12]))
    with pytest.raises(ValueError, match="overlaps"):
        pk.rms_norm(Fake(wide[:, :8]), w, residual=x, h_out=Fake(wide[:, 1:9]))
    with pytest.raises(ValueError, match="overlaps"):
        pk.rms_norm(x, w, residual=fake(4, 8), out=Fake(wide[:, :8]), h_out=Fake(wide[:, 4:12]))
    with pytest.raises(ValueError, match="dy must be"):
        pk.rms_norm_backward(x, w, fake(3, 8))
    with pytest.raises(ValueError, match="dh must be"):
        pk.rms_norm_backward(x, w, x, dh=fake(4, 7))
    with pytest.raises(ValueError, match="not needed"):
        pk.rms_norm_backward(x, w, x, need_dx=False, out=fake(4, 8))
    with pytest.raises(ValueError, match="overlaps"):
        pk.rms_norm_backward(Fake(wide[:, :8]), w, x, out=Fake(wide[:, :8]))


def test_linear_q8_refusals():
    x, xs, w, ws = fake(4, 32, dtype=F8), f32(4), fake(6, 32, dtype=F8), f32(6)
    with pytest.raises(TypeError, match="x must be"):
        pk.linear_q8(fake(4, 32), xs, w, ws)
    with pytest.raises(TypeError, match="w must be"):
        pk.linear_q8(x, xs, fake(6, 32, dtype=torch.float8_e5m2), ws)
    with pytest.raises(ValueError, match="multiple of 16"):
        pk.linear_q8(fake(4, 24, dtype=F8), xs, fake(6, 24, dtype=F8), ws)
    with pytest.raises(ValueError, match="x_scale"):
        pk.linear_q8(x, f32(5), w, ws)
    with pytest.raises(ValueError, match="w_scale"):
        pk.linear_q8(x, xs, w, fake(6))
    with pytest.raises(ValueError, match="16-byte"):
        pk.linear_q8(Fake(torch.zeros(4, 40, dtype=F8)[:, :32]), xs, w, ws)
    with pytest.raises(ValueError, match="bias"):
        pk.linear_q8(x, xs, w, ws, bias=fake(6), out_dtype=torch.float16)
    with pytest.raises(TypeError, match="dtype"):
        pk.linear_q8(x, xs, w, ws, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="act must be"):
        pk.linear_q8(x, xs, w, ws, act="tanh")


def test_gated_refusals():
    x, w = fake(4, 8), fake(12, 8)
    with pytest.raises(ValueError, match="even number"):
        pk.gated_linear(x, fake(7, 8))
    with pytest.raises(ValueError, match="w must be"):
        pk.gated_linear(x, fake(12, 9))
    with pytest.raises(ValueError, match="bias"):
        pk.gated_linear(x, w, bias=fake(6))
    with pytest.raises(ValueError, match="out must be"):
        pk.gated_linear(x, w, out=fake(4, 12))
    with pytest.raises(ValueError, match="act must be"):
        pk.gated_linear(x, w, act="swish")
    with pytest.raises(ValueError, match="dy must be"):
        pk.gated_linear_backward(x, w, fake(4, 12), fake(4, 12))
    with pytest.raises(ValueError, match="pre must be"):
        pk.gated_linear_backward(x, w, fake(4, 6), fake(4, 6))
    with pytest.raises(ValueError, match="status"):
        pk.gated_linear(x, w, status=f32(1))


def test_logprobs_refusals():
    z, labels = fake(4, 100), i64(4)
    with pytest.raises(ValueError, match="labels"):
        pk.token_logprobs(z, fake(4, dtype=torch.int32))
    for top in (-1, 65, 101):
        with pytest.raises(ValueError, match="top"):
            pk.token_logprobs(z, labels, top=top)
    with pytest.raises(ValueError, match="top"):
        pk.token_logprobs(fake(4, 10), labels, top=11)
    with pytest.raises(ValueError, match="at least one column"):
        pk.token_logprobs(fake(4, 0), labels)
    with pytest.raises(ValueError, match="contiguous rows"):
        pk.token_logprobs(Fake(torch.zeros(100, 4).T), labels)
    lse, entropy, g = f32(4), f32(4), f32(4)
    with pytest.raises(ValueError, match="lse"):
        pk.token_logprobs_backward(z, labels, fake(4), entropy, g)
    with pytest.raises(ValueError, match="entropy is needed"):
        pk.token_logprobs_backward(z, labels, lse, None, g, dentropy=g)
    with pytest.raises(ValueError, match="dlogp"):
        pk.token_logprobs_backward(z, labels, lse, entropy, f32(5))
    wide = torch.zeros(4, 250, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        pk.token_logprobs_backward(Fake(wide[:, :100]), labels, lse, entropy, g, out=Fake(wide[:, 50:150]))


def test_distill_refusals():
    x, w, idx, values = fake(4, 8), fake(60, 8), i64(4, 5), f32(4, 5)
    with pytest.raises(ValueError, match="idx must be"):
        pk.distill(x, w, i64(4, 65), f32(4, 65))
    with pytest.raises(ValueError, match="idx must be"):
        pk.distill(x, w, i64(4, 0), f32(4, 0))
    with pytest.raises(ValueError, match="idx must be"):
        pk.distill(x, w, i64(4), values)
    with pytest.raises(TypeError, match="idx must be"):
        pk.distill(x, w, fake(4, 5, dtype=torch.int32), values)
    with pytest.raises(ValueError, match="values must be"):
        pk.distill(x, w, idx, f32(4, 6))
    with pytest.raises(ValueError, match="idx must be"):
        pk.distill(x, w, i64(3, 5), values)
    for tau in (0.0, -1.0, NAN, 1e4):
        with pytest.raises(ValueError, match="temperature"):
            pk.distill(x, w, idx, values, temperature=tau)
    with pytest.raises(ValueError, match="bias"):
        pk.distill(x, w, idx, values, bias=fake(59))
    with pytest.raises(ValueError, match="lse"):
        pk.distill_backward(x, w, idx, values, f32(5), f32(4))
    with pytest.raises(ValueError, match="dloss"):
        pk.distill_backward(x, w, idx, values, f32(4), fake(4))


@pytest.fixture(scope="module")
def lib():
    from rope_cu_tile_gb300 import build

    build.build()
    return pk.load()


P, ODD, NULL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001), ctypes.c_void_p(0)
WORD = ctypes.c_void_p(0x1004)


def refuser(call, **defaults):
    def run(**kw):
        assert not set(kw) - set(defaults)
        return call(*{**defaults, **kw}.values())

    return run


def test_norm_arguments_need_no_gpu(lib):
    fwd = refuser(lib.pk_rms_norm, dtype=1, x=P, ldx=8, res=NULL, ldr=8, w=P, eps=1e-6, T=4, D=8, y=P, ldy=8, h=NULL, ldh=8, stream=NULL)
    for kw in (dict(dtype=3), dict(T=-1), dict(T=(1 << 30) + 1), dict(D=0), dict(D=16385), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN),
               dict(ldx=7), dict(ldy=7), dict(res=P, ldr=7), dict(h=P, ldh=7), dict(x=NULL), dict(w=NULL), dict(y=NULL)):
        assert fwd(**kw) == 1, kw
    for kw in (dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(y=ODD), dict(h=ODD), dict(dtype=0, x=ctypes.c_void_p(0x1002))):
        assert fwd(**kw) == 2, kw
    assert fwd(T=0, x=NULL, w=NULL, y=NULL) == 0
    q8 = refuser(lib.pk_rms_norm_q8, dtype=1, x=P, ldx=8, res=NULL, ldr=8, w=P, eps=1e-6, T=4, D=8, q=P, ldq=8, scale=P, h=NULL, ldh=8,
                 stream=NULL)
    assert q8(scale=NULL) == 1 and q8(ldq=7) == 1 and q8(scale=ODD) == 2 and q8(T=0, q=NULL, scale=NULL) == 0
    quant = refuser(lib.pk_quantize_rows, dtype=1, x=P, ldx=8, T=4, D=8, q=P, ldq=8, scale=P, stream=NULL)
    assert quant(x=NULL) == 1 and quant(D=0) == 1 and quant(x=ODD) == 2 and quant(T=0) == 0
    bwd = refuser(lib.pk_rms_norm_backward, dtype=1, h=P, ldh=8, w=P, dy=P, lddy=8, dh=NULL, lddh=8, eps=1e-6, T=4, D=8, dx=P, lddx=8, dw=P,
                  ws=NULL, wb=0, stream=NULL)
    for kw in (dict(h=NULL), dict(w=NULL), dict(dy=NULL), dict(lddy=7), dict(dh=P, lddh=7), dict(lddx=7), dict(eps=0.0), dict(wb=-1)):
        assert bwd(**kw) == 1, kw
    assert bwd(dy=ODD) == 2 and bwd(dw=ODD) == 2 and bwd(ws=ODD) == 2 and bwd(dx=NULL, dw=NULL) == 0
    n = ctypes.c_int64(-1)
    assert lib.pk_rms_norm_backward_workspace(1, 0, 8, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.pk_rms_norm_backward_workspace(1, 4, 0, 1, ctypes.byref(n)) == 1


def test_product_arguments_need_no_gpu(lib):
    tail = dict(ws=NULL, wb=0, status=NULL, stream=NULL)
    gated = refuser(lib.pk_gated_linear, dtype=1, x=P, ldx=8, w=P, bias=NULL, act=2, T=4, F=6, K=8, y=P, ldy=6, pre=NULL, **tail)
    for kw in (dict(dtype=3), dict(T=-1), dict(F=0), dict(F=(1 << 19) + 1), dict(K=0), dict(act=4), dict(ldx=7), dict(ldy=5), dict(x=NULL),
               dict(w=NULL), dict(y=NULL), dict(wb=-1)):
        assert gated(**kw) == 1, kw
    for kw in (dict(x=ODD), dict(w=ODD), dict(bias=ODD), dict(y=ODD), dict(pre=ODD), dict(ws=ODD), dict(status=ODD)):
        assert gated(**kw) == 2, kw
    assert gated(T=0, x=NULL, w=NULL, y=NULL) == 0
    back = refuser(lib.pk_gated_linear_backward, dtype=1, x=P, ldx=8, w=P, dy=P, lddy=6, pre=P, act=2, T=4, F=6, K=8, dx=P, dw=P, db=P, **tail)
    for kw in (dict(dy=NULL), dict(pre=NULL), dict(x=NULL), dict(w=NULL), dict(lddy=5), dict(act=-1)):
        assert back(**kw) == 1, kw
    assert back(dx=ODD) == 2 and back(db=ODD) == 2 and back(dy=ODD) == 2 and back(pre=ODD) == 2
    q8 = refuser(lib.pk_linear_q8, dtype=1, x=P, ldx=32, xs=P, w=P, ws_=P, bias=NULL, res=NULL, ldr=6, act=0, T=4, N=6, K=32, y=P, ldy=6, **tail)
    for kw in (dict(dtype=3), dict(K=24), dict(K=0), dict(N=0), dict(ldx=40), dict(ldx=16), dict(ldy=5), dict(res=P, ldr=5), dict(xs=NULL),
               dict(ws_=NULL), dict(x=NULL), dict(act=9)):
        assert q8(**kw) == 1, kw
    for kw in (dict(x=WORD), dict(w=WORD), dict(xs=ODD), dict(ws_=ODD), dict(bias=ODD), dict(res=ODD), dict(y=ODD)):
        assert q8(**kw) == 2, kw
    n = ctypes.c_int64(-1)
    assert lib.pk_gated_linear_workspace(1, P, 8, P, 0, 6, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.pk_gated_linear_workspace(1, P, 7, P, 4, 6, 8, ctypes.byref(n)) == 1
    assert lib.pk_gated_linear_backward_workspace(1, P, 8, P, 1, 1, 1, 0, 6, 8, ctypes.byref(n)) == 0
    assert lib.pk_linear_q8_workspace(0, 6, 32, ctypes.byref(n)) == 0 and lib.pk_linear_q8_workspace(4, 6, 33, ctypes.byref(n)) == 1


def test_vocabulary_arguments_need_no_gpu(lib):
    score = refuser(lib.pk_token_logprobs, dtype=1, z=P, ld=100, labels=P, T=4, V=100, top=5, logp=P, lse=P, entropy=P, top_logp=P, top_idx=P,
                    status=NULL, stream=NULL)
    for kw in (dict(dtype=3), dict(ld=99), dict(T=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(top=-1), dict(top=65), dict(V=4), dict(z=NULL),
               dict(labels=NULL), dict(logp=NULL), dict(lse=NULL), dict(entropy=NULL), dict(top_logp=NULL), dict(top_idx=NULL)):
        assert score(**kw) == 1, kw
    for kw in (dict(z=ODD), dict(labels=WORD), dict(logp=ODD), dict(top_idx=WORD), dict(status=ODD)):
        assert score(**kw) == 2, kw
    assert score(T=0, z=NULL, labels=NULL, logp=NULL, lse=NULL, entropy=NULL, top_logp=NULL, top_idx=NULL) == 0
    back = refuser(lib.pk_token_logprobs_backward, dtype=1, z=P, ld=100, labels=P, lse=P, entropy=P, dlogp=P, dentropy=P, T=4, V=100, dz=P,
                   lddz=100, stream=NULL)
    for kw in (dict(lse=NULL), dict(dlogp=NULL), dict(entropy=NULL), dict(dz=NULL), dict(lddz=99)):
        assert back(**kw) == 1, kw
    assert back(dz=ODD) == 2 and back(lse=ODD) == 2 and back(T=0) == 0
    tail = dict(ws=NULL, wb=0, status=NULL, stream=NULL)
    distill = refuser(lib.pk_distill, dtype=1, x=P, ldx=8, w=P, bias=NULL, idx=P, values=P, top=5, tau=1.0, T=4, D=8, V=60, loss=P, lse=P, **tail)
    for kw in (dict(dtype=3), dict(T=-1), dict(D=0), dict(V=0), dict(top=0), dict(top=65), dict(tau=0.0), dict(tau=NAN), dict(tau=2e3),
               dict(ldx=7), dict(idx=NULL), dict(values=NULL), dict(loss=NULL), dict(lse=NULL), dict(wb=-1)):
        assert distill(**kw) == 1, kw
    assert distill(idx=WORD) == 2 and distill(values=ODD) == 2 and distill(bias=ODD) == 2 and distill(T=0) == 0
    back = refuser(lib.pk_distill_backward, dtype=1, x=P, ldx=8, w=P, bias=NULL, idx=P, values=P, top=5, tau=1.0, lse=P, dloss=P, T=4, D=8,
                   V=60, dx=P, dw=P, db=P, **tail)
    for kw in (dict(lse=NULL), dict(dloss=NULL), dict(top=70), dict(tau=-1.0)):
        assert back(**kw) == 1, kw
    assert back(dx=ODD) == 2 and back(db=ODD) == 2 and back(dloss=ODD) == 2
    n = ctypes.c_int64(-1)
    assert lib.pk_distill_workspace(1, P, 8, P, 0, 0, 0, 8, 60, 5, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.pk_distill_workspace(1, P, 8, P, 1, 1, 4, 8, 60, 65, ctypes.byref(n)) == 1
