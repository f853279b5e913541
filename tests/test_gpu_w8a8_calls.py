"""What the 8-bit calls promise of each other and of arguments left out, on
the device.  Where two calls promise the same values, the bits are compared;
where a call is compared with a form in 64 bits, the bounds are those derived
in test_gpu_w8a8."""
import math
import os
import shutil
import subprocess
import sys

import pytest
import torch

from post_weight_quantization_accumulate_b200 import binding as B
from post_weight_quantization_accumulate_b200 import decoder, w8a8
from post_weight_quantization_accumulate_b200.layer import LayerQuantizer

from test_gpu_w8a8 import _check_product, _norm_reference
from test_w8a8_launches import PRODUCTS

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


# -- the product, every kernel ---------------------------------------------------------

@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_product_by_every_kernel(M, N, K, t):
    """Sizes that are known (test_w8a8_launches) to reach every kernel of the
    product, its rings of stages and its second and third tiles."""
    _check_product(M, N, K, t, zeros=True, bias=True, seed=5)


# -- the calls that allocate their outputs -----------------------------------------------

@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("M,D,gate_rows", [(6, 1000, 4), (37, 1003, 1), (1, 4096, 1), (300, 4096, 300), (2, 40000, 2)])
def test_block_norm_with_all_of_its_arguments(M, D, gate_rows, t):
    """Every argument of w8a8.block_norm with values that none of the others
    could stand for, against the form in 64 bits."""
    block, residual = _randn(D, M, D).to(t), (2 * _randn(D + 1, M, D)).to(t)
    pre, post = (1 + 0.3 * _randn(D + 2, D)).float(), (3 + 0.5 * _randn(D + 3, D)).float()
    gate = (-1.5 + 0.3 * _randn(D + 4, -(-M // gate_rows), D)).to(t)
    scale, eps = 0.375, 0.25
    kw = {"post_norm": True, "post_weight": post.cuda(), "gate": gate.cuda(), "gate_rows": gate_rows, "scale": scale, "eps": eps}
    stream, out = w8a8.block_norm(block.cuda(), residual.cuda(), pre.cuda(), **kw)
    same, t8 = w8a8.block_norm(block.cuda(), residual.cuda(), pre.cuda(), quantize=True, **kw)
    only = w8a8.block_norm(block.cuda(), residual.cuda(), pre.cuda(), keep_stream=False, **kw)
    kept = w8a8.block_norm(block.cuda(), residual.cuda(), pre.cuda(), keep_out=False, **kw)
    _done()
    assert only[0] is None and kept[1] is None
    assert torch.equal(same, stream) and torch.equal(only[1], out) and torch.equal(kept[0], stream)
    r, size, y, ysize = _norm_reference(block, residual, pre, True, post, gate, gate_rows, scale, eps)
    d = (D / 128 + 48) * U
    half, tiny = torch.finfo(t).eps / 2, 2.0 ** -25 if t == F16 else 2.0 ** -130
    stream, out = stream.cpu().double(), out.cpu().double()
    assert ((stream - r).abs() <= d * size + half * r.abs() * (1 + d) + d * half * size + tiny).all()
    assert ((out - y).abs() <= 2 * d * ysize + half * (y.abs() + 2 * d * ysize) + tiny).all()
    top = y.abs().amax(1, keepdim=True)
    rsize = 127 * ysize / top
    codes, scales = t8.codes.cpu().double(), t8.scales.cpu().double()
    assert ((codes - 127 * y / top).abs() <= 0.5 + 2 * d * (rsize + rsize.amax(1, keepdim=True))).all()
    assert ((scales - top[:, 0] / 127).abs() <= 2 * d * ysize.amax(1) / 127 + U * top[:, 0] / 127).all()
    assert torch.equal(t8.sums.cpu().long(), t8.codes.cpu().long().sum(1))


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", [(3, 200, 333), (40, 130, 500), (300, 257, 640)])
def test_linear_with_all_of_its_arguments(M, N, K, t):
    """w8a8.linear with and without each of bias and zeros."""
    x = _randn(K, M, K).to(BF16).cuda()
    tokens = w8a8.quantize_tokens(x)
    g = torch.Generator().manual_seed(N)
    codes = w8a8.empty_codes(N, K, "cuda")
    codes.copy_(torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8))
    scales, zeros = (torch.rand(N, generator=g) * 1e-3 + 1e-4).cuda(), torch.randint(-128, 128, (N,), generator=g, dtype=torch.int32).cuda()
    bias = (5 + torch.randn(N, generator=g)).cuda()
    half, tiny = torch.finfo(t).eps / 2, 2.0 ** -25 if t == F16 else 2.0 ** -130
    for z in (None, zeros):
        for b in (None, bias):
            y = w8a8.linear(tokens, w8a8.Weight(codes, scales, z), bias=b, dtype=t)
            _done()
            assert y.dtype == t and y.shape == (M, N) and y.is_contiguous()
            w = codes.double() - (0 if z is None else z.double()[:, None])
            p = (tokens.codes.double() @ w.t()) * tokens.scales.double()[:, None] * scales.double()
            ref = p + (0 if b is None else b.double())
            bound = 3.01 * U * p.abs() * (1 + half) + (U + half * 1.01) * ref.abs() + tiny
            assert ((y.double() - ref).abs() <= bound).all()


def test_refused_calls_launch_nothing():
    x = torch.zeros(3, 50, dtype=BF16, device="cuda")
    t = w8a8.quantize_tokens(x)
    w = w8a8.Weight(w8a8.empty_codes(7, 50, "cuda").zero_(), torch.ones(7, device="cuda"), torch.zeros(7, dtype=torch.int32, device="cuda"))
    before = B.gptq_launch_count()
    for call in (lambda: w8a8.quantize_tokens(x.double()), lambda: w8a8.quantize_tokens(x.t()), lambda: w8a8.quantize_tokens(x, gate=x[:2]),
                 lambda: w8a8.block_norm(x, x.float()), lambda: w8a8.block_norm(x, x, gate=x[:1], gate_rows=2),
                 lambda: w8a8.block_norm(x, x, eps=-1.0), lambda: w8a8.linear(t, w, dtype=torch.int8),
                 lambda: w8a8.linear(w8a8.Tokens(t.codes, t.scales), w), lambda: w8a8.linear(t, w, bias=torch.ones(6, device="cuda")),
                 lambda: w8a8.linear(t, w8a8.Weight(w.codes.contiguous(), w.scales)),
                 lambda: w8a8.quantize_tokens(torch.zeros(1, 65537, dtype=BF16, device="cuda"))):
        with pytest.raises((TypeError, ValueError, B.GptqError)):
            call()
    assert B.gptq_launch_count() == before
    _done()


# -- the calibration -------------------------------------------------------------------------

@pytest.mark.parametrize("bits,gs", [(4, 128), (8, -1)])
def test_calibration_for_16_bit_inputs(bits, gs):
    """The decoder layer's calibration, written out from its formulas with the
    layer quantizer: by default, and with act_bits=16, the codes are the same."""
    shape = decoder.TINY
    W, X = decoder.synthetic_layer(shape)

    def rms(x):
        return (x * torch.rsqrt(x.pow(2).mean(dim=1, keepdim=True) + 1e-6)).to(BF16)

    def quantized(x, names):
        q = LayerQuantizer(*shape.linear_shape(names[0]), bits, gs, 128, 0.01, False)
        q.add_batch(x)
        q.prepare()
        codes, values = {}, {}
        for n in names:
            layer = q.quantize(W[n])
            codes[n], values[n] = layer.codes.clone(), layer.W_hat.to(BF16)
        return codes, values

    want, v = quantized(X, ("q", "k", "v"))
    x_o = rms((X @ v["v"].t()).float())
    codes, o = quantized(x_o, ("o",))
    want |= codes
    x_mlp = rms((X.float() + (x_o @ o["o"].t()).float()).to(BF16).float())
    codes, gu = quantized(x_mlp, ("gate", "up"))
    want |= codes
    x_down = (torch.nn.functional.silu((x_mlp @ gu["gate"].t()).float()) * (x_mlp @ gu["up"].t()).float()).to(BF16)
    want |= quantized(x_down, ("down",))[0]
    for kw in ({}, {"act_bits": 16}):
        res = decoder.calibrate(X, W, shape, bits=bits, group_size=gs, **kw)
        assert set(res.layers) == set(want) and all(torch.equal(res.layers[n].codes, want[n]) for n in want)
    # and with 8-bit inputs it is another one
    res = decoder.calibrate(X, W, shape, bits=bits, group_size=gs, act_bits=8)
    assert not all(torch.equal(res.layers[n].codes, want[n]) for n in want)
    _done()


def test_one_gate_row_for_any_number_of_rows():
    """gate_rows may be larger than the batch, up to the largest 64-bit number;
    a batch without rows has a gate without rows."""
    x, r, g = (_randn(k, 5, 64).to(BF16).cuda() for k in range(3))
    want = w8a8.block_norm(x, r, gate=g[:1], gate_rows=5)
    for rows in (6, 2 ** 31, 2 ** 63 - 5, 2 ** 63 - 1):
        got = w8a8.block_norm(x, r, gate=g[:1], gate_rows=rows)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out = torch.empty_like(x)
        B.gptq_block_norm(x, r, out=out, gate=g[:1], gate_rows=rows)
        assert torch.equal(out, want[1])
        assert w8a8.block_norm(x[:0], r[:0], gate=g[:0], gate_rows=rows)[0].shape == (0, 64)
    _done()


def test_silu_of_gates_around_its_last_value():
    """exp(87) is below 2^126, exp(88) above: there silu is taken as 0."""
    a = torch.tensor([[-87.0, -88.0, -88.7, 87.0, 0.0]], device="cuda")
    x = torch.tensor([[1e30, 1e30, 1e30, -1e-8, 1e30]], device="cuda")
    for k in (5, 40000):                              # in registers, and element by element
        g, v = torch.zeros(1, k, device="cuda"), torch.zeros(1, k, device="cuda")
        g[:, :5], v[:, :5] = a, x
        t = w8a8.quantize_tokens(v, gate=g)
        _done()
        silu = [-87.0 / (1 + math.exp(87.0)), 0.0, 0.0, 87.0, 0.0]
        want = [s * y for s, y in zip(silu, x[0].double().tolist())]
        top = max(abs(w) for w in want)
        assert t.codes[0, :5].tolist() == [round(127 * w / top) for w in want]
        # 87 log2(e) = 125.5 is rounded by 2^-18 at most, 44 U of its power of 2; log2(e) itself costs 19 U; the rest 9 U
        assert abs(t.scales.item() - top / 127) <= 100 * U * top / 127


# -- threads ---------------------------------------------------------------------------------

WAITING_LIBRARY = """
#include <unistd.h>
#define CALL(name) int name() { usleep(400000); return 0; }
CALL(gptq_quantize_tokens) CALL(gptq_block_norm) CALL(gptq_w8a8_gemm)
"""

WATCHED_CALLS = """
import sys, threading, time
import torch
sys.path.insert(0, sys.argv[1])
import _calls
x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
q, s = torch.zeros(2, 64, dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda")
turns, done = 0, False
def others():
    global turns
    while not done:
        turns += 1
        time.sleep(0.002)
thread = threading.Thread(target=others)
thread.start()
for call in (lambda: _calls.quantize_tokens(x, None, True, False),
             lambda: _calls.block_norm(x, x, None, False, None, None, 0, 1.0, 1e-6, False, True, True),
             lambda: _calls.linear(q, s, None, q, s, None, None, torch.bfloat16)):
    before = turns
    call()
    print(turns - before)
done = True
thread.join()
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    """A launch can wait for room in the stream's queue.  The calls do not hold
    the interpreter meanwhile: with a library whose calls take 0.4 s, another
    thread goes on."""
    (tmp_path / "wait.c").write_text(WAITING_LIBRARY)
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "wait.c"), "-o", str(tmp_path / "libgptq.so")], check=True)
    shutil.copy(os.path.join(os.path.dirname(B.__file__), "_calls.so"), tmp_path)
    run = subprocess.run([sys.executable, "-c", WATCHED_CALLS, str(tmp_path)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr
    turns = [int(v) for v in run.stdout.split()]
    # of 200 turns in 0.4 s on an idle machine; none while the interpreter is held
    assert len(turns) == 3 and min(turns) >= 10, turns
