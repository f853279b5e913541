"""What the 8-bit calls promise of each other and of arguments left out, on
the device.  Where two calls promise the same values, the bits are compared;
where a call is compared with a form in 64 bits, the bounds are those derived
in test_gpu_w8a8."""
import pytest
import torch

from post_weight_quantization_accumulate_b200 import binding as B
from post_weight_quantization_accumulate_b200 import w8a8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of float32
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _done():
    torch.cuda.synchronize()
    assert B.gptq_device_status() == 0


# -- the norm's codes -------------------------------------------------------------

@pytest.mark.parametrize("M,D", [(2048, 4096), (300, 4096), (70, 1003), (9, 11008), (5, 20000), (40, 96), (1, 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_norm_codes_next_to_the_tokens_of_its_output(M, D, weights):
    """In float32 the output holds the values whose codes are given.  The codes
    are taken of r' w, before the row's factor, by one product with 127 / t: the
    output's rounding and its maximum's are U each of the quotient, 127 / t rounded
    up 2 U, so a code is within 1/2 + 4.01 * 127 U of the output's own quotient.
    Both scales have two roundings: 4.01 U apart at most."""
    x, r = _randn(D, M, D).float().cuda(), _randn(D + 1, M, D).float().cuda()
    pre = (1 + 0.3 * _randn(D + 2, D)).float().cuda() if weights else None
    out, q = torch.empty_like(x), w8a8.empty_codes(M, D, "cuda")
    s, n = torch.empty(M, device="cuda"), torch.empty(M, dtype=torch.int32, device="cuda")
    B.gptq_block_norm(x, r, pre, out=out, q=q, q_scales=s, q_sums=n)
    want = w8a8.quantize_tokens(out)
    _done()
    ratio = 127 * out.double() / out.double().abs().amax(1, keepdim=True)
    assert ((q.double() - ratio).abs() <= 0.5 + 4.01 * 127 * U).all()
    assert (q.int() - want.codes.int()).abs().max() <= 1
    assert torch.equal(n.long(), q.long().sum(1))
    assert ((s.double() - want.scales.double()).abs() <= 4.01 * U * want.scales.double()).all()


def test_norm_and_product_repeat_their_bits():
    """The residual stream through the norm into a product, again and again:
    nothing in the chain depends on the order in which blocks run."""
    M, D, N = 2048, 4096, 11008
    g = torch.Generator("cuda").manual_seed(3)
    h, r = (torch.randn(M, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    pre = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    codes = torch.randint(-127, 128, (N, D), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    weight = w8a8.Weight(codes, torch.rand(N, generator=g, device="cuda") * 1e-3,
                         torch.randint(-20, 21, (N,), generator=g, device="cuda", dtype=torch.int32))
    first = None
    for _ in range(40):
        stream, t = w8a8.block_norm(h, r, pre, quantize=True)
        got = (stream, t.codes, t.scales, t.sums, w8a8.linear(t, weight))
        if first is None:
            first = tuple(v.clone() for v in got)
        assert all(torch.equal(u, v) for u, v in zip(first, got))
    _done()


# -- arguments left out -------------------------------------------------------------

@pytest.mark.parametrize("D", [7, 1000, 1001, 11008, 40000])
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_norm_without_a_block_takes_no_notice_of_its_factors(D, t):
    """The term of a block that is not there is 0, also where the gate or the
    weights of the norm after it hold an infinity or NaN: at every row length
    (those kept in registers, on and off their boundaries, and longer ones)."""
    r, pre = _randn(D, 6, D).to(t).cuda(), (1 + 0.3 * _randn(D + 1, D)).float().cuda()
    gate, post = torch.ones(2, D, dtype=t, device="cuda"), torch.ones(D, device="cuda")
    gate[0, D // 2], gate[1, 0], post[D - 1], post[D // 3] = float("inf"), float("nan"), -float("inf"), float("nan")
    want = w8a8.block_norm(None, r, pre)
    wt = w8a8.block_norm(None, r, pre, quantize=True)[1]
    for scale in (1.0, float("inf")):
        kw = {"post_norm": True, "post_weight": post, "gate": gate, "gate_rows": 3, "scale": scale}
        got = w8a8.block_norm(None, r, pre, **kw)
        t8 = w8a8.block_norm(None, r, pre, quantize=True, **kw)[1]
        _done()
        assert torch.equal(got[0], r) and torch.equal(got[1], want[1])
        assert torch.equal(t8.codes, wt.codes) and torch.equal(t8.scales, wt.scales) and torch.equal(t8.sums, wt.sums)
