"""Refusals of the adapter products and the distillation loss: every bad
argument is turned away before the GPU is touched (no compute runs here)."""

import ctypes
import math

import pytest
import torch

import post_weight_quantization_15_amd as gq

FAKE = 0x1000      # never dereferenced: validation fails first
INV, WS = gq.GPTQ_ERR_INVALID_ARG, gq.GPTQ_ERR_WORKSPACE
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return gq.load_library()


def adapters(A=FAKE, B=FAKE, alpha=FAKE, row=FAKE, count=3, rank=8):
    return ctypes.byref(gq._Adapters(A, B, alpha, row, count, rank))


def lora(lib, **kw):
    a = dict(X=FAKE, xdt=0, n=4, d=64, ldx=64, qw=FAKE, sc=FAKE, sdt=1, z=FAKE, gi=FAKE, m=32,
             bits=4, g=32, sgn=0, ad=adapters(), H=None, Y=FAKE, ydt=1, ldy=32, ws=FAKE, wsb=BIG,
             st=None)
    a.update(kw)
    return lib.gptq_lora_matmul(*a.values())


def test_lora_matmul_refuses(lib):
    for kw in (dict(xdt=1), dict(ydt=2), dict(ydt=7), dict(sdt=0), dict(n=-1), dict(n=524281),
               dict(d=0), dict(m=0), dict(d=65536, ldx=65536), dict(m=65536, ldy=65536),
               dict(ldx=63), dict(ldy=31), dict(bits=5), dict(g=0), dict(g=-2), dict(sgn=2),
               dict(X=None), dict(qw=None), dict(sc=None), dict(z=None), dict(gi=None),
               dict(Y=None), dict(ad=None), dict(ad=adapters(count=0)),
               dict(ad=adapters(count=65536)), dict(ad=adapters(rank=0)),
               dict(ad=adapters(rank=129)), dict(ad=adapters(A=None)), dict(ad=adapters(B=None)),
               dict(ad=adapters(alpha=None)), dict(ad=adapters(row=None))):
        assert lora(lib, **kw) == INV, kw
    need = lib.gptq_lora_workspace_bytes(4, 32, 64, 32, 8)
    assert need > 0
    assert lora(lib, wsb=need - 1) == WS and lora(lib, ws=None) == WS
    assert lora(lib, n=0, X=None, Y=None, qw=None, ws=None, wsb=0) == gq.GPTQ_OK
    for bad in ((-1, 32, 64, 32, 8), (524281, 32, 64, 32, 8), (4, 0, 64, 32, 8),
                (4, 32, 65536, 32, 8), (4, 32, 64, 32, 0), (4, 32, 64, 32, 129), (4, 32, 64, 0, 8)):
        assert lib.gptq_lora_workspace_bytes(*bad) == 0


def backward(lib, **kw):
    a = dict(dY=FAKE, dt=0, n=4, m=32, ldy=32, X=FAKE, ldx=64, H=FAKE, qw=FAKE, sc=FAKE, sdt=1,
             z=FAKE, gi=FAKE, d=64, bits=4, g=32, sgn=0, ad=adapters(), dX=FAKE, lddx=64, dA=FAKE,
             dB=FAKE, acc=0, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_lora_backward(*a.values())


def test_lora_backward_refuses(lib):
    for kw in (dict(dt=1), dict(n=-1), dict(n=524281), dict(m=0), dict(d=0), dict(ldy=31),
               dict(ldx=63), dict(lddx=63), dict(bits=6), dict(g=0), dict(sgn=-1), dict(acc=2),
               dict(dY=None), dict(X=None), dict(H=None), dict(qw=None), dict(sc=None),
               dict(z=None), dict(gi=None), dict(sdt=0), dict(ad=None), dict(ad=adapters(rank=0)),
               dict(ad=adapters(A=None)), dict(ad=adapters(B=None)), dict(ad=adapters(row=None))):
        assert backward(lib, **kw) == INV, kw
    need = lib.gptq_lora_backward_workspace_bytes(4, 32, 64, 8, 3)
    assert need > 0
    assert backward(lib, wsb=need - 1) == WS and backward(lib, ws=None) == WS
    assert backward(lib, n=0, dA=None, dB=None, dY=None, ws=None, wsb=0) == gq.GPTQ_OK
    assert lib.gptq_lora_backward_workspace_bytes(4, 32, 64, 8, 0) == 0
    assert lib.gptq_lora_backward_workspace_bytes(4, 32, 64, 200, 3) == 0


def back(lib, **kw):
    a = dict(dY=FAKE, dt=0, n=4, m=32, ldy=32, qw=FAKE, sc=FAKE, sdt=1, z=FAKE, gi=FAKE, d=64,
             bits=4, g=32, sgn=0, dX=FAKE, lddx=64, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.gptq_dequant_matmul_t(*a.values())


def test_dequant_matmul_t_refuses(lib):
    for kw in (dict(dt=1), dict(n=-1), dict(n=524281), dict(m=0), dict(d=0), dict(m=65536, ldy=65536),
               dict(ldy=31), dict(lddx=63), dict(bits=1), dict(g=0), dict(sgn=3), dict(sdt=0),
               dict(dY=None), dict(dX=None), dict(qw=None), dict(sc=None), dict(z=None),
               dict(gi=None)):
        assert back(lib, **kw) == INV, kw
    need = lib.gptq_dequant_matmul_t_workspace_bytes(4, 32, 64)
    if need:
        assert back(lib, wsb=need - 1) == WS
    assert back(lib, n=0, dY=None, dX=None, ws=None, wsb=0) == gq.GPTQ_OK
    assert lib.gptq_dequant_matmul_t_workspace_bytes(-1, 32, 64) == 0


def test_distill_refuses(lib):
    def loss(**kw):
        a = dict(z=FAKE, dt=0, n=4, V=100, ld=100, ix=FAKE, t=FAKE, k=5, T=1.0, tl=None, w=None,
                 loss=FAKE, stats=None, dz=None, ldd=0, st=None)
        a.update(kw)
        return lib.gptq_distill_loss(*a.values())

    def grad(**kw):
        a = dict(z=FAKE, dt=0, n=4, V=100, ld=100, stats=FAKE, ix=FAKE, t=FAKE, k=5, T=1.0, tl=None,
                 w=None, g=FAKE, dz=FAKE + 4096, ldd=100, st=None)
        a.update(kw)
        return lib.gptq_distill_backward(*a.values())

    common = (dict(dt=3), dict(n=-1), dict(n=2097153), dict(V=0), dict(V=262145, ld=262145, ldd=262145),
              dict(ld=99), dict(k=0), dict(k=1025), dict(T=0.0), dict(T=-1.0), dict(T=math.inf),
              dict(T=math.nan), dict(z=None), dict(ix=None), dict(t=None))
    for kw in common + (dict(loss=None), dict(dz=FAKE + 4096, ldd=99), dict(dz=FAKE, ldd=101)):
        assert loss(**kw) == INV, kw
    for kw in common + (dict(stats=None), dict(g=None), dict(dz=None), dict(ldd=99),
                        dict(dz=FAKE, ldd=101)):
        assert grad(**kw) == INV, kw
    assert loss(n=0, z=None, loss=None) == gq.GPTQ_OK and grad(n=0, z=None) == gq.GPTQ_OK


def cpu_call():
    m, d, n, L, r = 8, 32, 3, 2, 4
    return dict(X=torch.zeros(n, d, dtype=torch.bfloat16), qw=torch.zeros(m, 4, dtype=torch.int32),
                sc=torch.ones(m, 1), z=torch.zeros(m, 1, dtype=torch.uint8),
                gi=torch.zeros(d, dtype=torch.int32), bits=4, g=32,
                A=torch.zeros(L, r, d, dtype=torch.bfloat16), B=torch.zeros(L, m, r, dtype=torch.bfloat16),
                ids=torch.zeros(n, dtype=torch.int32), alpha=torch.ones(L))


def test_binding_refuses_host_tensors_and_wrong_types():
    c = cpu_call()
    with pytest.raises(ValueError, match="GPU"):
        gq.gptq_lora_matmul(*c.values())
    with pytest.raises(ValueError, match="GPU"):
        gq.gptq_dequant_matmul_t(torch.zeros(3, 8, dtype=torch.bfloat16), *list(c.values())[1:7])
    with pytest.raises(ValueError, match="GPU"):
        gq.gptq_distill_loss(torch.zeros(2, 10), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(TypeError):
        gq.gptq_lora_matmul(*dict(c, X=c["X"].float()).values())
    with pytest.raises(ValueError, match="overlap"):
        gq.gptq_lora_matmul(*dict(c, X=torch.zeros(1, 32, dtype=torch.bfloat16).expand(3, 32)).values())
    with pytest.raises(TypeError):
        gq.gptq_distill_loss(torch.zeros(2, 10, dtype=torch.float64),
                             torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))


def test_binding_checks_shapes():
    """The checks behind the device check, called with the host's device."""
    c, dev = cpu_call(), torch.device("cpu")
    packed = (c["qw"], c["sc"], c["z"], c["gi"])
    assert gq._check_packed(*packed, 4, 32, 8, 32, dev) == gq.GPTQ_F32
    assert gq._check_packed(c["qw"], c["sc"].half(), c["z"], c["gi"], 4, 32, 8, 32, dev) == gq.GPTQ_F16
    for bits, g in ((5, 32), (4, 0), (4, -3)):
        with pytest.raises(gq.GPTQError):
            gq._check_packed(*packed, bits, g, 8, 32, dev)
    with pytest.raises(ValueError):
        gq._check_packed(*packed, 8, 32, 8, 32, dev)
    with pytest.raises(TypeError):
        gq._check_packed(c["qw"], c["sc"].double(), c["z"], c["gi"], 4, 32, 8, 32, dev)
    ad = gq._check_adapters(c["A"], c["B"], c["ids"], c["alpha"], 3, 8, 32, dev)
    assert (ad.n_adapters, ad.rank) == (2, 4)
    for key, bad in (("A", c["A"][0]), ("A", c["A"][:, :, :31]), ("B", c["B"][:, :7]),
                     ("B", c["B"].transpose(1, 2)), ("ids", c["ids"][:2]), ("alpha", c["alpha"][:1])):
        with pytest.raises(ValueError):
            k = dict(c, **{key: bad})
            gq._check_adapters(k["A"], k["B"], k["ids"], k["alpha"], 3, 8, 32, dev)
    for key, bad in (("A", c["A"].float()), ("ids", c["ids"].long()), ("alpha", c["alpha"].double())):
        with pytest.raises(TypeError):
            k = dict(c, **{key: bad})
            gq._check_adapters(k["A"], k["B"], k["ids"], k["alpha"], 3, 8, 32, dev)


def test_a_workspace_off_its_alignment_is_refused(lib):
    """The workspace's parts are read and written 16 bytes at a time."""
    for off in (1, 2, 4, 8):
        assert lora(lib, ws=FAKE + off) == WS
        assert backward(lib, ws=FAKE + off) == WS
        assert back(lib, ws=FAKE + off) == WS
    # where none is needed it is not looked at
    assert lora(lib, n=0, ws=FAKE + 4, wsb=0) == gq.GPTQ_OK
