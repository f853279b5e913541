"""What the 8-bit calls refuse, on the host before a device is touched, and
the Python checks in front of them (no GPU needed)."""
import ctypes

import pytest
import torch

from post_weight_quantization_accumulate_b200 import binding as B
from post_weight_quantization_accumulate_b200 import build as build_mod
from post_weight_quantization_accumulate_b200 import decoder, w8a8
from post_weight_quantization_accumulate_b200.layer import QuantizedLayer

P = ctypes.c_void_p
FAKE = P(1 << 20)      # never dereferenced: the checks come first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def test_quantize_tokens_refusals(lib):
    def f(Xq=FAKE, ldq=64, s=FAKE, sums=FAKE, hat=None, ldh=0, X=FAKE, ldx=50, gate=None, ldg=0, ty=0, M=3, K=50):
        return lib.gptq_quantize_tokens(Xq, ldq, s, sums, hat, ldh, X, ldx, gate, ldg, ty, M, K, None)
    for bad in (dict(M=-1), dict(M=(1 << 30) + 1), dict(K=0), dict(K=65537, ldx=1 << 17, ldq=1 << 17), dict(ty=3), dict(ty=-1),
                dict(Xq=None), dict(X=None), dict(s=None), dict(s=P((1 << 20) + 2)), dict(sums=P((1 << 20) + 2)),
                dict(Xq=P((1 << 20) + 8)), dict(ldq=60), dict(ldq=48), dict(ldx=49), dict(ldx=1 << 31),
                dict(X=P((1 << 20) + 1)), dict(ty=2, X=P((1 << 20) + 2)), dict(gate=FAKE, ldg=49),
                dict(hat=FAKE, ldh=49), dict(gate=P((1 << 20) + 1), ldg=50)):
        assert f(**bad) == 1, bad
    assert f(M=0) == 0
    assert f(M=0, X=None, s=None) == 0


def test_block_norm_refusals(lib):
    def f(so=FAKE, lds=50, out=FAKE, ldo=50, q=None, ldq=0, qs=None, qsum=None, block=FAKE, ldb=50, res=FAKE, ldr=50,
          gate=None, ldg=0, gate_rows=0, post=None, pre=None, eps=1e-6, ty=0, M=3, D=50):
        return lib.gptq_block_norm(so, lds, out, ldo, q, ldq, qs, qsum, block, ldb, res, ldr, gate, ldg, gate_rows, post, pre,
                                   1, ctypes.c_float(1.0), ctypes.c_float(eps), ty, M, D, None)
    for bad in (dict(M=-1), dict(D=0), dict(D=65537), dict(ty=5), dict(eps=-1.0), dict(eps=float("nan")),
                dict(so=None, out=None), dict(block=None, res=None), dict(lds=49), dict(ldo=49), dict(ldb=49), dict(ldr=49),
                dict(gate=FAKE, ldg=50, gate_rows=0), dict(gate=FAKE, ldg=49, gate_rows=1), dict(q=FAKE, ldq=64),
                dict(q=FAKE, ldq=50, qs=FAKE), dict(q=P((1 << 20) + 4), ldq=64, qs=FAKE), dict(post=P((1 << 20) + 2)),
                dict(pre=P((1 << 20) + 2)), dict(block=P((1 << 20) + 1)), dict(q=FAKE, ldq=64, qs=P((1 << 20) + 2)),
                dict(q=FAKE, ldq=64, qs=FAKE, qsum=P((1 << 20) + 2))):
        assert f(**bad) == 1, bad
    assert f(M=0) == 0


def test_pack_and_gemm_refusals(lib):
    def p(Wq=FAKE, ldw=64, z=FAKE, codes=FAKE, zeros=FAKE, N=3, K=50):
        return lib.gptq_w8a8_pack(Wq, ldw, z, codes, zeros, N, K, None)
    for bad in (dict(N=-1), dict(K=0), dict(K=65537, ldw=1 << 17), dict(ldw=48), dict(ldw=56), dict(Wq=None), dict(z=None),
                dict(codes=None), dict(zeros=None), dict(Wq=P((1 << 20) + 8))):
        assert p(**bad) == 1, bad
    assert p(N=0) == 0

    def g(Y=FAKE, ldy=7, ty=0, X=FAKE, ldx=64, xs=FAKE, sums=FAKE, W=FAKE, ldw=64, ws=FAKE, z=FAKE, bias=None, M=5, N=7, K=50):
        return lib.gptq_w8a8_gemm(Y, ldy, ty, X, ldx, xs, sums, W, ldw, ws, z, bias, M, N, K, None)
    for bad in (dict(M=-1), dict(N=-1), dict(M=(1 << 30) + 1), dict(M=1 << 29, N=1 << 29, ldy=1 << 29), dict(K=0),
                dict(K=65537, ldx=1 << 17, ldw=1 << 17), dict(ty=3), dict(ldy=6), dict(ldx=48), dict(ldx=56), dict(ldw=56),
                dict(X=P((1 << 20) + 8)), dict(W=P((1 << 20) + 8)), dict(Y=P((1 << 20) + 1)), dict(Y=None), dict(X=None),
                dict(xs=None), dict(W=None), dict(ws=None), dict(sums=None), dict(bias=P((1 << 20) + 2)),
                dict(z=P((1 << 20) + 2))):
        assert g(**bad) == 1, bad
    assert g(M=0) == 0
    assert g(N=0, ldy=0) == 0


def test_binding_checks():
    x = torch.zeros(3, 50, dtype=torch.bfloat16)
    q, s, n = w8a8.empty_codes(3, 50, "cpu"), torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    assert q.stride(0) == 64 and q.shape == (3, 50)
    with pytest.raises(TypeError):
        B.gptq_quantize_tokens(q, s, n, x.double())
    with pytest.raises(TypeError):
        B.gptq_quantize_tokens(q, s.double(), n, x)
    with pytest.raises(TypeError):
        B.gptq_quantize_tokens(q, s, n, x, gate=x.float())
    with pytest.raises(ValueError):
        B.gptq_quantize_tokens(q[:2], s, n, x)
    with pytest.raises(ValueError):
        B.gptq_quantize_tokens(q, s[:2], n, x)
    with pytest.raises(ValueError):
        B.gptq_quantize_tokens(q, s, n, torch.zeros(50, 3, dtype=torch.bfloat16).t())     # rows not contiguous
    with pytest.raises(ValueError):
        B.gptq_block_norm(x, x, out=x.clone(), gate=x[:1], gate_rows=0)
    with pytest.raises(ValueError):
        B.gptq_block_norm(x, x, out=x.clone(), gate=x[:1], gate_rows=2)                    # two gate rows wanted
    with pytest.raises(TypeError):
        B.gptq_block_norm(x, x.float(), out=x.clone())
    with pytest.raises(ValueError):
        B.gptq_block_norm(x, x, torch.ones(49), out=x.clone())
    w, ws, z = w8a8.empty_codes(7, 50, "cpu"), torch.zeros(7), torch.zeros(7, dtype=torch.int32)
    y = torch.zeros(3, 7, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.gptq_w8a8_gemm(y, q, s, w, ws, None, z)            # a zero point without the tokens' sums
    with pytest.raises(ValueError):
        B.gptq_w8a8_gemm(y[:, :6], q, s, w, ws)
    with pytest.raises(ValueError):
        B.gptq_w8a8_gemm(y, q, s, w[:, :40], ws)
    with pytest.raises(TypeError):
        B.gptq_w8a8_gemm(y.double(), q, s, w, ws)
    with pytest.raises(TypeError):
        B.gptq_w8a8_gemm(y, q.float(), s, w, ws)


def test_pack_needs_one_group_a_row():
    layer = QuantizedLayer(None, torch.zeros(4, 64, dtype=torch.uint8), torch.ones(4, 2), torch.zeros(4, 2),
                           torch.zeros(64, dtype=torch.int32), torch.zeros(64, dtype=torch.int32), torch.zeros(4, 64), None)
    with pytest.raises(ValueError):
        w8a8.pack(layer)
    layer.codes = None
    with pytest.raises(ValueError):
        w8a8.pack(layer)


def test_calibrate_refuses_other_activation_widths():
    with pytest.raises(ValueError):
        decoder.calibrate(torch.zeros(8, 8), {}, decoder.TINY, act_bits=4)


def test_calls_refuse_other_tensors(lib):
    """The calls that allocate their outputs refuse what is not a matrix on a
    GPU before they allocate or launch anything."""
    x = torch.zeros(3, 50, dtype=torch.bfloat16)
    t = w8a8.Tokens(w8a8.empty_codes(3, 50, "cpu"), torch.zeros(3))
    w = w8a8.Weight(w8a8.empty_codes(7, 50, "cpu"), torch.zeros(7))
    for call in (lambda: w8a8.quantize_tokens(x), lambda: w8a8.block_norm(x, x), lambda: w8a8.linear(t, w),
                 lambda: w8a8.quantize_tokens(x[0])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: w8a8.quantize_tokens(None), lambda: w8a8.block_norm(None, None),
                 lambda: w8a8.linear(w8a8.Tokens(None, torch.zeros(3)), w)):
        with pytest.raises(TypeError):
            call()
