"""Refusals of the 4-bit floating-point operators and the token statistics:
every bad argument is turned away before the GPU is touched (no compute runs
here)."""

import math
import random

import pytest
import torch

import post_weight_quantization_15_amd as gq

FAKE = 0x1000      # never dereferenced: validation fails first
INV, WS = gq.GPTQ_ERR_INVALID_ARG, gq.GPTQ_ERR_WORKSPACE
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return gq.load_library()


def quantize(lib, **kw):
    a = dict(X=FAKE, dt=0, n=4, d=64, ldx=64, c=FAKE, s=FAKE, hat=None, ldh=0, st=None)
    a.update(kw)
    return lib.gptq_mx_quantize(*a.values())


def matmul(lib, **kw):
    a = dict(X=FAKE, form=0, xs=None, n=100, d=64, ldx=64, c=FAKE, s=FAKE, m=32, Y=FAKE, ydt=1,
             ldy=32, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_mx_matmul(*a.values())


def back(lib, **kw):
    a = dict(dY=FAKE, dt=0, n=100, m=32, ldy=32, c=FAKE, s=FAKE, d=64, dX=FAKE, lddx=64, ws=FAKE,
             wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_mx_matmul_t(*a.values())


def gated(lib, **kw):
    a = dict(X=FAKE, form=0, xs=None, n=100, d=64, ldx=64, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, m=32,
             act=2, Y=FAKE, ldy=32, G=None, U=None, ldg=0, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_mx_gated(*a.values())


def gated_back(lib, **kw):
    a = dict(dY=FAKE, dt=0, n=100, m=32, ldy=32, G=FAKE, U=FAKE, ldg=32, gc=FAKE, gs=FAKE, uc=FAKE,
             us=FAKE, d=64, act=2, dX=FAKE, lddx=64, dGU=FAKE, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_mx_gated_backward(*a.values())


SIZES = (dict(n=-1), dict(n=524281), dict(d=0), dict(m=0), dict(d=65536, ldx=65536, lddx=65536),
         dict(m=65536, ldy=65536, ldg=65536))


def sizes(names):
    return tuple({k: v for k, v in kw.items() if k in names} for kw in SIZES)


def test_quantize_refuses(lib):
    for kw in (dict(dt=3), dict(n=-1), dict(n=524281), dict(d=0), dict(d=65536, ldx=65536),
               dict(ldx=63), dict(hat=FAKE, ldh=63), dict(X=None), dict(c=None), dict(s=None),
               dict(c=FAKE + 8)):
        assert quantize(lib, **kw) == INV, kw
    assert quantize(lib, n=0, X=None, c=None, s=None) == gq.GPTQ_OK


def test_matmul_refuses(lib):
    for kw in sizes("n d m ldx ldy".split()) + (
            dict(form=3), dict(form=-1), dict(ydt=2), dict(ldx=63), dict(ldy=31), dict(X=None),
            dict(c=None), dict(s=None), dict(Y=None), dict(c=FAKE + 4), dict(form=2),
            dict(form=2, xs=FAKE, X=FAKE + 8)):
        assert matmul(lib, **kw) == INV, kw
    for form in range(3):
        need = lib.gptq_mx_matmul_workspace_bytes(100, 32, 64, form)
        if need:
            assert matmul(lib, form=form, xs=FAKE, wsb=need - 1) == WS
            assert matmul(lib, form=form, xs=FAKE, ws=None) == WS
            assert matmul(lib, form=form, xs=FAKE, ws=FAKE + 8) == WS
    assert matmul(lib, n=0, X=None, Y=None, c=None, ws=None, wsb=0) == gq.GPTQ_OK
    for bad in ((-1, 32, 64, 0), (4, 0, 64, 0), (4, 32, 65536, 0), (4, 32, 64, 3)):
        assert lib.gptq_mx_matmul_workspace_bytes(*bad) == 0
        assert lib.gptq_mx_gated_workspace_bytes(*bad) == 0


def test_matmul_t_refuses(lib):
    for kw in sizes("n d m lddx ldy".split()) + (
            dict(dt=1), dict(ldy=31), dict(lddx=63), dict(dY=None), dict(dX=None), dict(c=None),
            dict(s=None), dict(c=FAKE + 1)):
        assert back(lib, **kw) == INV, kw
    need = lib.gptq_mx_matmul_t_workspace_bytes(100, 32, 64)
    assert need > 0
    assert back(lib, wsb=need - 1) == WS and back(lib, ws=None) == WS and back(lib, ws=FAKE + 4) == WS
    assert back(lib, n=0, dY=None, dX=None, ws=None, wsb=0) == gq.GPTQ_OK


def test_gated_refuses(lib):
    for kw in sizes("n d m ldx ldy".split()) + (
            dict(form=3), dict(act=3), dict(act=-1), dict(ldx=63), dict(ldy=31), dict(X=None),
            dict(gc=None), dict(us=None), dict(uc=FAKE + 8), dict(Y=None), dict(G=FAKE, ldg=32),
            dict(G=FAKE, U=FAKE, ldg=31), dict(form=2)):
        assert gated(lib, **kw) == INV, kw
    need = lib.gptq_mx_gated_workspace_bytes(100, 32, 64, 0)
    if need:
        assert gated(lib, wsb=need - 1) == WS and gated(lib, ws=None) == WS
    assert gated(lib, n=0, X=None, Y=None, gc=None, ws=None, wsb=0) == gq.GPTQ_OK


def test_gated_backward_refuses(lib):
    for kw in sizes("n d m lddx ldy ldg".split()) + (
            dict(dt=1), dict(act=3), dict(ldy=31), dict(ldg=31), dict(lddx=63), dict(dY=None),
            dict(G=None), dict(U=None), dict(dGU=None), dict(dGU=FAKE + 8), dict(gc=None),
            dict(us=None)):
        assert gated_back(lib, **kw) == INV, kw
    need = lib.gptq_mx_gated_backward_workspace_bytes(100, 32, 64)
    assert need > 0
    assert gated_back(lib, wsb=need - 1) == WS and gated_back(lib, ws=None) == WS
    assert gated_back(lib, n=0, dY=None, dX=None, ws=None, wsb=0) == gq.GPTQ_OK


def test_token_statistics_refuse(lib):
    def stats(**kw):
        a = dict(z=FAKE, dt=0, n=4, V=100, ld=100, t=FAKE, T=1.0, k=5, lp=FAKE, e=FAKE, l=FAKE,
                 s=FAKE, top=FAKE, ix=FAKE, ws=FAKE, wsb=BIG, st=None)
        a.update(kw)
        return lib.gptq_token_logprobs(*a.values())

    def grad(**kw):
        a = dict(z=FAKE, dt=0, n=4, V=100, ld=100, s=FAKE, t=FAKE, T=1.0, g=FAKE, h=FAKE,
                 dz=FAKE + 4096, ldd=100, st=None)
        a.update(kw)
        return lib.gptq_token_logprobs_backward(*a.values())

    common = (dict(dt=3), dict(n=-1), dict(n=2097153), dict(V=0), dict(ld=99), dict(T=0.0),
              dict(T=-1.0), dict(T=math.inf), dict(T=math.nan), dict(z=None), dict(t=None))
    for kw in common + (dict(V=262145, ld=262145), dict(k=-1), dict(k=513, V=600, ld=600),
                        dict(k=101), dict(top=None), dict(ix=None)):
        assert stats(**kw) == INV, kw
    for kw in common + (dict(V=262145, ld=262145, ldd=262145), dict(s=None), dict(dz=None),
                        dict(ldd=99), dict(dz=FAKE, ldd=101)):
        assert grad(**kw) == INV, kw
    need = lib.gptq_token_logprobs_workspace_bytes(1, 100000, 20)
    assert need > 0
    long = dict(n=1, V=100000, ld=100000, k=20)
    assert stats(**long, wsb=need - 1) == WS and stats(**long, ws=None) == WS
    assert stats(**long, ws=FAKE + 8) == WS
    assert stats(n=0, z=None) == gq.GPTQ_OK and grad(n=0, z=None) == gq.GPTQ_OK
    for bad in ((-1, 100, 5), (4, 0, 0), (4, 100, 101), (4, 600, 513), (4, 262145, 5), (4, 100, -1)):
        assert lib.gptq_token_logprobs_workspace_bytes(*bad) == 0


def layer(m=8, nb=2):
    return torch.zeros(m, 16 * nb, dtype=torch.uint8), torch.zeros(m, nb, dtype=torch.uint8)


def test_binding_refuses_host_tensors_and_wrong_types():
    X = torch.zeros(3, 64, dtype=torch.bfloat16)
    c, s = layer()
    for call in (lambda: gq.gptq_mx_quantize(X), lambda: gq.gptq_mx_matmul(X, c, s),
                 lambda: gq.gptq_mx_matmul_t(X[:, :8], c, s, 64),
                 lambda: gq.gptq_mx_gated(X, c, s, c, s),
                 lambda: gq.gptq_mx_gated_backward(X[:, :8], X[:, :8], X[:, :8], c, s, c, s, 64),
                 lambda: gq.gptq_token_logprobs(X),
                 lambda: gq.gptq_token_logprobs_backward(X, torch.zeros(3, 3))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        gq.gptq_mx_quantize(X.double())
    with pytest.raises(TypeError):
        gq.gptq_mx_matmul(X.float(), c, s)
    with pytest.raises(ValueError, match="x_scales"):
        gq.gptq_mx_matmul(c, c, s)
    with pytest.raises(ValueError, match="x_scales"):
        gq.gptq_mx_matmul(X, c, s, x_scales=s)
    with pytest.raises(ValueError, match="activation"):
        gq.gptq_mx_gated(X, c, s, c, s, activation="gelu")
    with pytest.raises(ValueError, match="overlap"):
        gq.gptq_mx_quantize(X[:1].expand(3, 64))


def test_binding_checks_shapes():
    """The checks behind the device check, called with the host's device."""
    c, s = layer()
    dev = torch.device("cpu")
    assert gq._check_mx(c, s, "layer", 2, dev) == 8
    for bad in ((c[:, :31], s), (c, s[:, :1]), (c, s[:7]), (c[0], s)):
        with pytest.raises(ValueError):
            gq._check_mx(*bad, "layer", 2, dev)
    with pytest.raises(TypeError):
        gq._check_mx(c.int(), s, "layer", 2, dev)


def test_both_four_bit_forms_choose_alike(lib):
    """Activations rounded in the call and given as codes (whose width is known in blocks
    only) take the same kernel: few rows, without a workspace, or tiles."""
    shapes = [(36, 3125, 3828), (56, 4860, 1453), (62, 9723, 559), (18, 7719, 1633), (64, 1900, 5643)]
    rng = random.Random(3)
    shapes += [(rng.randint(17, 64), int(math.exp(rng.uniform(3, 9.4))), int(math.exp(rng.uniform(3.5, 9.4))))
               for _ in range(4000)]
    for n, m, d in shapes:
        wide = 32 * -(-d // 32)
        for need in (lib.gptq_mx_matmul_workspace_bytes, lib.gptq_mx_gated_workspace_bytes):
            assert need(n, m, d, 1) == need(n, m, wide, 2) == need(n, m, d, 2), (n, m, d)
