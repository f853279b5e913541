"""The 8-bit calls on the device against plain forms in 64 bits.

Bounds, with u = 2^-24 (half a step of float32) and e = finfo(type).eps / 2
(half a step of the output's type):
  codes      those of x itself are the exact ones; those of a value v that is
             computed in float32 with a relative error d (and its row's
             maximum too) are within 1/2 + 2 * 127 d of 127 v / t;
  gate       silu(a) x: rounding exp's argument costs |a| u, the two
             approximations and the rest 9 u, which is below 16 u where |a|
             <= 5; farther out on the negative side |silu| is below 0.04 and
             falling, and such values are not a row's largest;
  norm       a mean of D squares summed in any order of at most D / 128 + 32
             dependent additions has a relative error of that many u, its
             root half of that; rsqrt, the products with it, the weights and
             the gate, the scale and the sum add at most 16 u;
  product    the integer sum is exact; its conversion and the products with
             two scales are 3 u of the product, the bias u of the sum.
A value y stored in the type adds e |y|; for float32 that is u."""
import numpy as np
import pytest
import torch

from post_weight_quantization_accumulate_b200 import binding as B
from post_weight_quantization_accumulate_b200 import decoder, synth, w8a8
from post_weight_quantization_accumulate_b200.layer import LayerQuantizer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _half(t):
    return torch.finfo(t).eps / 2


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), dtype=torch.float64)


def _pitched(t, pitch, fill):
    """t on the device inside rows of `pitch` elements, the rest holding `fill`."""
    wide = torch.full((t.shape[0], pitch), fill, dtype=t.dtype, device="cuda")
    wide[:, : t.shape[1]] = t.cuda()
    return wide


def _done():
    torch.cuda.synchronize()
    assert B.gptq_device_status() == 0


def _exact_codes(v):
    """(127 v / t, t) in float64."""
    t = v.abs().amax(1, keepdim=True)
    return 127.0 * v / torch.where(t > 0, t, torch.ones_like(t)), t[:, 0]


# -- tokens -------------------------------------------------------------------

def _tokens(x, gate=None, pitch=None):
    M, K = x.shape
    ld = pitch or K
    xw = _pitched(x, ld, 7.0)
    gw = _pitched(gate, ld, 7.0) if gate is not None else None
    q = torch.full((M + 1, (K + 15) // 16 * 16 + 16), 99, dtype=torch.int8, device="cuda")
    hat = torch.full((M + 1, ld + 3), 99.0, dtype=x.dtype, device="cuda")
    s = torch.full((M + 1,), 99.0, device="cuda")
    n = torch.full((M + 1,), 99, dtype=torch.int32, device="cuda")
    B.gptq_quantize_tokens(q[:M, :K], s[:M], n[:M], xw[:, :K], None if gate is None else gw[:, :K], hat[:M, :K])
    _done()
    # nothing behind a row, and no row behind the last, is written
    assert (q[M] == 99).all() and (q[:, K:] == 99).all() and (hat[M] == 99).all() and (hat[:, K:] == 99).all()
    assert s[M] == 99 and n[M] == 99
    return q[:M, :K].cpu(), s[:M].cpu(), n[:M].cpu(), hat[:M, :K].cpu()


TOKEN_SIZES = [(1, 1), (1, 4096), (3, 2), (5, 7), (2, 64), (17, 1000), (33, 1003), (300, 4096), (7, 11008), (2, 28672),
               (3, 65536), (2, 65535), (1000, 40), (300, 61), (77, 125), (33, 128), (515, 16), (2, 32761), (2, 32768)]


@pytest.mark.parametrize("M,K", TOKEN_SIZES)
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_are_exact(M, K, t):
    x = (_randn(M * 7 + K, M, K) * torch.exp(_randn(K, M, 1))).to(t)
    q, s, n, hat = _tokens(x)
    ratio, top = _exact_codes(x.double())
    want = torch.round(ratio)
    assert torch.equal(q.double(), want)
    assert torch.equal(s, (top / 127.0).float())     # a quotient of floats rounded through double is the rounded quotient
    assert torch.equal(n.long(), want.sum(1).long())
    assert torch.equal(hat, (q.float() * s[:, None]).to(t))


@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_of_strided_rows(t):
    x = _randn(3, 9, 1000).to(t)
    for pitch in (1000, 1001, 1003, 1008, 1024):
        q, s, n, hat = _tokens(x, pitch=pitch)
        assert torch.equal(q.double(), torch.round(_exact_codes(x.double())[0])), pitch


@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_ties_go_to_even(t):
    # t = 127 / 2^j: the quotients are 2^j x, with every half among them
    base = torch.cat([torch.arange(-127, 128).double(), torch.arange(-126, 127).double() + 0.5])
    for j in (0, 3, 7):
        x = (base / 2 ** j)[None].to(t)
        x = x[:, (x[0].double() * 2 ** j == base)]           # those the type holds
        q, s, n, hat = _tokens(x)
        assert torch.equal(q.double(), torch.round(x.double() * 2 ** j))


def test_tokens_ties_of_wide_maxima_float16():
    """t = 127 s 2^-j with an odd s: the quotients of v = s (2 k + 1) 2^-(j + 1) are the ties k + 1/2."""
    for s_ in (3, 5, 9, 11, 13, 15):
        for j in (0, 4, 9):
            k = torch.arange(-126, 126).double() + 0.5
            v = torch.cat([torch.tensor([127.0]).double(), k, k.round()]) * s_ / 2 ** j
            x = v[v.to(F16).double() == v][None].to(F16)
            assert x[0, 0].double() == 127 * s_ / 2 ** j and x.numel() > 100
            q, s, n, hat = _tokens(x)
            assert torch.equal(q.double(), torch.round(_exact_codes(x.double())[0]))


def test_tokens_next_to_ties_float32():
    """Values one and two steps of float32 from a tie."""
    top = torch.tensor([1.0, 3.0, 0.7, 1e-30, 3e38, 2.0 ** -149 * 12345], dtype=F32)
    rows = []
    for v in top:
        half = ((torch.arange(-126, 126).double() + 0.5) * v.double() / 127.0).float()
        near = [half, torch.nextafter(half, half + v), torch.nextafter(half, half - v)]
        rows.append(torch.cat([v[None]] + near))
    x = torch.stack(rows)
    q, s, n, hat = _tokens(x)
    # 127 x and 2 t q are exact in float64, and so is the comparison with the tie
    assert torch.equal(q.double(), torch.round(_exact_codes(x.double())[0]))


@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_of_tiny_and_huge_rows(t):
    fi = torch.finfo(t)
    x = _randn(5, 6, 500)
    x = x / x.abs().amax(1, keepdim=True)
    x = (x * torch.tensor([fi.max, fi.max / 3, fi.tiny, fi.tiny * 64, fi.tiny * 2.0 ** -4, 1.0]).double()[:, None]).to(t)
    q, s, n, hat = _tokens(x)
    ratio, top = _exact_codes(x.double())
    assert torch.equal(q.double(), torch.round(ratio))
    assert torch.equal(s, (top / 127.0).float())


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("K", [5, 1000, 4096])
def test_tokens_rows_of_zeros_and_rows_that_are_not_finite(t, K):
    x = _randn(6, 7, K).to(t)
    x[1] = 0
    x[2, K // 2] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = -0.0
    x[6, :] = float("nan")
    q, s, n, hat = _tokens(x)
    for r in (1, 5):
        assert (q[r] == 0).all() and s[r] == 0 and n[r] == 0 and (hat[r] == 0).all()
    for r in (2, 3, 4, 6):
        assert (q[r] == 0).all() and torch.isnan(s[r]) and n[r] == 0 and torch.isnan(hat[r]).all()
    assert torch.equal(q[0].double(), torch.round(_exact_codes(x[:1].double())[0])[0])


@pytest.mark.parametrize("M,K", [(1, 1), (1, 11008), (4, 1003), (129, 2048), (2, 40000)])
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_of_a_gated_activation(M, K, t):
    x, a = _randn(1 + K, M, K).to(t), (3 * _randn(2 + K, M, K)).to(t)
    q, s, n, hat = _tokens(x, a, pitch=K + (K % 8))
    v = a.double() * torch.sigmoid(a.double()) * x.double()
    ratio, top = _exact_codes(v)
    d = 16 * U
    assert ((q.double() - ratio).abs() <= 0.5 + 2 * 127 * d).all()
    assert ((s.double() - top / 127).abs() <= (d + U) * top / 127).all()
    assert torch.equal(n.long(), q.long().sum(1))
    assert torch.equal(hat, (q.float() * s[:, None]).to(t))


@pytest.mark.parametrize("M,K,pitch", [(1300, 1000, 1000), (2400, 1000, 1000), (2400, 1001, 1001), (450, 4096, 4096), (700, 4096, 4096),
                                       (700, 4099, 4100), (20, 11008, 11008), (200, 11008, 11008), (200, 11005, 11005)])
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_tokens_of_few_and_many_rows(M, K, pitch, t):
    x, a = _randn(M + K, M, K).to(t), (3 * _randn(M + K + 1, M, K)).to(t)
    q, s, n, hat = _tokens(x, pitch=pitch)
    assert torch.equal(q.double(), torch.round(_exact_codes(x.double())[0]))
    assert torch.equal(n.long(), q.long().sum(1))
    got = w8a8.quantize_tokens(x.cuda(), hat=True)           # rows without a pitch: on 16-byte boundaries where the width allows
    assert torch.equal(got.codes.cpu(), q) and torch.equal(got.hat.cpu(), hat) and torch.equal(got.sums.cpu(), n)
    got = w8a8.quantize_tokens(x.cuda(), gate=a.cuda(), hat=True)
    ratio, top = _exact_codes(a.double() * torch.sigmoid(a.double()) * x.double())
    d = 16 * U
    assert ((got.codes.cpu().double() - ratio).abs() <= 0.5 + 2 * 127 * d).all()
    assert torch.equal(got.hat, (got.codes.float() * got.scales[:, None]).to(t))


def test_tokens_of_saturated_gates():
    """silu of gates far out: x for large ones, 0 for far negative ones; an
    infinite negative gate is not a number and marks its row."""
    a = torch.tensor([[200.0, -200.0, 1e30, -1e30, 0.0, 1.0]], dtype=F32)
    x = torch.ones(1, 6, dtype=F32)
    q, s, n, hat = _tokens(x, a)
    assert q[0].tolist() == [0, 0, 127, 0, 0, 0]
    a[0, 2] = -float("inf")
    q, s, n, hat = _tokens(x, a)
    assert torch.isnan(s[0]) and (q == 0).all()


def test_tokens_in_place_and_without_codes():
    x = _randn(9, 40, 777).to(BF16).cuda()
    want = w8a8.quantize_tokens(x, hat=True)
    y = x.clone()
    s = torch.empty(40, device="cuda")
    B.gptq_quantize_tokens(None, s, None, y, hat=y)
    _done()
    assert torch.equal(y, want.hat) and torch.equal(s, want.scales)


# -- norm between blocks --------------------------------------------------------

def _norm_reference(block, residual, pre, post_norm, post, gate, gate_rows, scale, eps):
    M, D = (block if block is not None else residual).shape
    r = residual.double() if residual is not None else torch.zeros(M, D, dtype=torch.float64)
    size = r.abs()
    if block is not None:
        h = block.double()
        if post_norm:
            h = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * (1.0 if post is None else post.double())
        if gate is not None:
            h = h * gate.double()[torch.arange(M) // gate_rows]
        r = r + scale * h
        size = size + (scale * h).abs()
    rs = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    w = torch.ones(D, dtype=torch.float64) if pre is None else pre.double()
    return r, size, r * rs * w, size * rs * w.abs()


def _check_norm(M, D, t, post_norm=True, weights=True, gate_rows=1, scale=0.5, eps=1e-6, parts="br", seed=0, pitch=None, whole=False):
    sd = seed + 31 * M + D
    block = _randn(sd, M, D).to(t) if "b" in parts else None
    residual = (2 * _randn(sd + 1, M, D)).to(t) if "r" in parts else None
    pre = (1 + 0.3 * _randn(sd + 2, D)).float() if weights else None
    post = (1 + 0.3 * _randn(sd + 3, D)).float() if weights else None
    gate = (1 + 0.3 * _randn(sd + 4, -(-M // gate_rows), D)).to(t) if gate_rows else None
    ld = pitch or D
    dev = lambda a: None if a is None else _pitched(a, ld, 7.0)[:, :D]  # noqa: E731
    vec = lambda a: None if a is None else a.cuda()  # noqa: E731
    so = torch.full((M + 1, ld if whole else ld + 1), 99.0, dtype=t, device="cuda")
    out = torch.full((M + 1, ld if whole else ld + 2), 99.0, dtype=t, device="cuda")
    q = torch.full((M + 1, (D + 15) // 16 * 16 + 16), 99, dtype=torch.int8, device="cuda")
    s, n = torch.full((M + 1,), 99.0, device="cuda"), torch.full((M + 1,), 99, dtype=torch.int32, device="cuda")
    B.gptq_block_norm(dev(block), dev(residual), vec(pre), stream_out=so[:M, :D], out=out[:M, :D], q=q[:M, :D], q_scales=s[:M],
                      q_sums=n[:M], post_norm=post_norm, post_weight=vec(post), gate=dev(gate), gate_rows=gate_rows, scale=scale,
                      eps=eps)
    _done()
    for g in (so, out, q):
        assert (g[M] == 99).all() and (g[:, D:] == 99).all()
    assert s[M] == 99 and n[M] == 99
    eps = float(np.float32(eps))
    r, size, y, ysize = _norm_reference(block, residual, pre, post_norm, post, gate, gate_rows, scale, eps)
    d = (D / 128 + 48) * U
    so, out, q, s, n = (v[:M].cpu() for v in (so[:, :D], out[:, :D], q[:, :D], s, n))
    tiny = 2.0 ** -25 if t == F16 else 2.0 ** -130      # half a step of the smallest values of the type
    assert ((so.double() - r).abs() <= d * size + _half(t) * r.abs() * (1 + d) + d * _half(t) * size + tiny).all()
    # the second norm's input carries the first's error, and so does its own factor
    dy = 2 * d
    assert ((out.double() - y).abs() <= dy * ysize + _half(t) * (y.abs() + dy * ysize) + tiny).all()
    ratio, top = _exact_codes(y)
    rsize = 127 * ysize / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    big = rsize.amax(1, keepdim=True)
    assert ((q.double() - ratio).abs() <= 0.5 + dy * (rsize + big)).all()
    assert ((s.double() - top / 127).abs() <= dy * ysize.amax(1) / 127 + U * top / 127).all()
    assert torch.equal(n.long(), q.long().sum(1))


@pytest.mark.parametrize("M,D", [(1, 1), (1, 4096), (2, 3), (5, 64), (33, 1000), (3, 1003), (300, 4096), (19, 5003), (4, 11008),
                                 (2, 28672), (2, 65536), (2, 65535), (513, 72), (300, 61), (33, 128), (2, 32761)])
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_norm_sizes_and_types(M, D, t):
    _check_norm(M, D, t)


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("post_norm,weights,gate_rows,parts", [
    (False, True, 0, "br"), (True, False, 0, "br"), (False, False, 3, "br"), (True, True, 40, "br"), (True, True, 7, "br"),
    (True, True, 0, "b"), (False, True, 0, "r"), (True, True, 1, "b"), (False, False, 0, "r")])
def test_norm_forms(t, post_norm, weights, gate_rows, parts):
    _check_norm(40, 1000, t, post_norm, weights, gate_rows, parts=parts)
    _check_norm(40, 1001, t, post_norm, weights, gate_rows, parts=parts)


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("pitch", [1001, 1004, 1008, 1024])
def test_norm_strided_rows(t, pitch):
    _check_norm(7, 1000, t, pitch=pitch)


@pytest.mark.parametrize("M,D,whole", [(3, 1000, True), (1300, 1000, True), (2400, 1000, True), (2400, 1001, False), (3, 4096, True),
                                       (450, 4096, True), (700, 4096, True), (700, 4099, False), (20, 11008, True),
                                       (200, 11008, True), (200, 11005, False), (9, 64, True), (9, 384, True)])
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_norm_of_few_and_many_rows(M, D, whole, t):
    """Rows on 16-byte boundaries and off them, few for the SMs and many."""
    _check_norm(M, D, t, whole=whole)
    _check_norm(M, D, t, gate_rows=0, whole=whole)


def test_norm_scale_and_eps():
    _check_norm(9, 512, F32, scale=0.0)
    _check_norm(9, 512, F32, scale=-3.0)
    _check_norm(9, 512, F32, eps=0.0)
    _check_norm(9, 512, BF16, eps=10.0)


def test_norm_in_place():
    b, r = _randn(1, 60, 1000).to(BF16).cuda(), _randn(2, 60, 1000).to(BF16).cuda()
    want = w8a8.block_norm(b, r, post_norm=True)
    B.gptq_block_norm(b, r, stream_out=r, out=b, post_norm=True)
    _done()
    assert torch.equal(r, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("D", [7, 1000, 4096])
def test_norm_rows_of_zeros_and_rows_that_are_not_finite(D):
    b, r = _randn(1, 5, D).to(BF16), _randn(2, 5, D).to(BF16)
    b[1] = 0
    r[1] = 0
    b[2, D // 2] = float("inf")
    r[3, D - 1] = float("nan")
    x, t = w8a8.block_norm(b.cuda(), r.cuda(), quantize=True)
    y, out = w8a8.block_norm(b.cuda(), r.cuda())
    _done()
    assert (t.codes[1] == 0).all() and t.scales[1] == 0 and (out[1] == 0).all() and (y[1] == 0).all()
    for k in (2, 3):
        assert (t.codes[k] == 0).all() and torch.isnan(t.scales[k]) and t.sums[k] == 0
    assert torch.isnan(out[3]).all()
    assert torch.isfinite(out[[0, 1, 4]].float()).all() and torch.isfinite(t.scales[[0, 1, 4]]).all()


# -- product ---------------------------------------------------------------------

def _codes(seed, rows, K, extreme=False, pitch=None):
    g = _gen(seed)
    c = torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int32).to(torch.int8)
    if extreme:
        c = torch.where(torch.rand(rows, K, generator=g) < 0.5, torch.full_like(c, -128), torch.full_like(c, 127))
    return c, _pitched(c, pitch or (K + 15) // 16 * 16, 77)[:, :K]


def _check_product(M, N, K, t, zeros=True, bias=True, extreme=False, pitch_x=None, pitch_w=None, pad=0, seed=0):
    x, xd = _codes(seed + M, M, K, extreme, pitch_x)
    w, wd = _codes(seed + N + 1, N, K, extreme, pitch_w)
    g = _gen(seed + K)
    xs, ws = torch.rand(M, generator=g) * 0.1 + 1e-3, torch.rand(N, generator=g) * 0.01 + 1e-4
    z = torch.randint(-128, 128, (N,), generator=g, dtype=torch.int32) if zeros else None
    b = torch.randn(N, generator=g) if bias else None
    sums = x.sum(1, dtype=torch.int32)
    y = torch.full((M + 1, N + pad), 99.0, dtype=t, device="cuda")
    vec = lambda a: None if a is None else a.cuda()  # noqa: E731
    B.gptq_w8a8_gemm(y[:M, :N], xd, xs.cuda(), wd, ws.cuda(), sums.cuda() if zeros else None, vec(z), vec(b))
    _done()
    assert (y[M] == 99).all() and (y[:, N:] == 99).all()
    got = y[:M, :N].double()
    # sums of integers below 2^31: exact in float64
    wz = wd.double() - (z.cuda().double()[:, None] if zeros else 0.0)
    p = (xd.double() @ wz.t()) * xs.cuda().double()[:, None] * ws.cuda().double()
    ref = p + (b.cuda().double() if bias else 0.0)
    bound = 3.01 * U * p.abs() + (U + _half(t) * 1.01) * ref.abs() + _half(t) * 3.01 * U * p.abs()
    tiny = 2.0 ** -25 if t == F16 else 2.0 ** -130
    worst = ((got - ref).abs() / (bound + tiny)).max()
    assert worst <= 1.0, float(worst)
    return y


PRODUCT_SIZES = [(1, 1, 1), (1, 128, 4096), (1, 4096, 4096), (2, 77, 1003), (3, 130, 16), (4, 64, 11008), (5, 200, 96), (8, 384, 640),
                 (9, 1000, 4096), (16, 256, 768), (17, 129, 513), (31, 4096, 100), (33, 257, 2048), (64, 512, 1024),
                 (70, 260, 640), (128, 128, 4096), (129, 300, 300), (200, 1030, 1500), (256, 256, 256), (257, 511, 129),
                 (400, 4096, 256), (1000, 1003, 515), (2048, 2048, 512), (3000, 40, 1000), (200, 300, 1), (40, 130, 5), (500, 512, 2048),
                 (12, 5000, 7000), (6, 7200, 200), (700, 5000, 300)]


@pytest.mark.parametrize("M,N,K", PRODUCT_SIZES)
@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_product_sizes_and_types(M, N, K, t):
    # bounded scales keep float16 sums in range: |p| <= K 127 255 xs ws with K <= 11008
    _check_product(M, N, K, t, bias=M % 2 == 0, zeros=t != F16, seed=3)


@pytest.mark.parametrize("M", [1, 3, 20, 300])
@pytest.mark.parametrize("zeros,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_product_forms(M, zeros, bias):
    _check_product(M, 192, 320, F32, zeros, bias)
    _check_product(M, 193, 321, BF16, zeros, bias)


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_product_strided(M):
    _check_product(M, 150, 500, BF16, pitch_x=1024, pitch_w=512, pad=5)
    _check_product(M, 150, 500, F32, pitch_x=512, pitch_w=4096, pad=1)
    _check_product(M, 256, 256, BF16, pitch_x=272, pad=8)


@pytest.mark.parametrize("M", [1, 2, 33, 260])
def test_product_of_the_largest_codes(M):
    """Sums at the ends of 32 bits: the longest rows of the largest codes."""
    _check_product(M, 70, 65536, F32, extreme=True)
    K = 65536
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((70, K), -128, dtype=torch.int8, device="cuda")
    z = torch.full((70,), 127, dtype=torch.int32, device="cuda")
    s = torch.full((M,), -128 * K, dtype=torch.int32, device="cuda")
    y = torch.empty(M, 70, device="cuda")
    B.gptq_w8a8_gemm(y, x, torch.ones(M, device="cuda"), w, torch.ones(70, device="cuda"), s, z)
    _done()
    assert (y == float(K * 128 * 255)).all()


def test_product_rows_that_are_not_finite_stay_in_their_rows():
    for M in (3, 40, 300):
        x, xd = _codes(1, M, 256)
        w, wd = _codes(2, 130, 256)
        xs = torch.ones(M, device="cuda")
        xs[1] = float("nan")
        y = torch.empty(M, 130, device="cuda")
        B.gptq_w8a8_gemm(y, xd, xs, wd, torch.ones(130, device="cuda"))
        _done()
        assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


def test_empty_calls():
    z = torch.empty(0, 50, dtype=BF16, device="cuda")
    t = w8a8.quantize_tokens(z)
    w = w8a8.Weight(w8a8.empty_codes(7, 50, "cuda").zero_(), torch.ones(7, device="cuda"))
    assert w8a8.linear(t, w).shape == (0, 7)
    assert w8a8.block_norm(z, z)[1].shape == (0, 50)
    t = w8a8.quantize_tokens(torch.ones(3, 50, dtype=BF16, device="cuda"))
    assert w8a8.linear(t, w8a8.Weight(w8a8.empty_codes(0, 50, "cuda"), torch.ones(0, device="cuda"))).shape == (3, 0)
    _done()


def test_calls_refuse_what_does_not_fit():
    x = torch.zeros(3, 50, dtype=BF16, device="cuda")
    t = w8a8.quantize_tokens(x)
    w = w8a8.Weight(w8a8.empty_codes(7, 50, "cuda").zero_(), torch.ones(7, device="cuda"),
                    torch.zeros(7, dtype=torch.int32, device="cuda"))
    for call in (lambda: w8a8.quantize_tokens(x.double()), lambda: w8a8.quantize_tokens(x, gate=x.float()),
                 lambda: w8a8.block_norm(x, x.float()), lambda: w8a8.linear(t, w, dtype=torch.int8),
                 lambda: w8a8.linear(t, w8a8.Weight(w.codes, w.scales.double())),
                 lambda: w8a8.block_norm(x, x, torch.ones(50, dtype=BF16, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: w8a8.quantize_tokens(x.t()), lambda: w8a8.quantize_tokens(x, gate=x[:2]),
                 lambda: w8a8.quantize_tokens(x.cpu()), lambda: w8a8.quantize_tokens(x, gate=x.cpu()),
                 lambda: w8a8.block_norm(x, x, gate=x[:1], gate_rows=2), lambda: w8a8.block_norm(x, x, gate=x[:1]),
                 lambda: w8a8.block_norm(x, x[:, :49]), lambda: w8a8.linear(t, w8a8.Weight(w.codes[:, :49], w.scales)),
                 lambda: w8a8.linear(w8a8.Tokens(t.codes, t.scales), w), lambda: w8a8.linear(t, w, bias=torch.ones(6, device="cuda")),
                 lambda: w8a8.linear(t, w8a8.Weight(w.codes, w.scales.cpu()))):
        with pytest.raises(ValueError):
            call()
    # rows of 50 codes: not a pitch of 16 bytes, which the library refuses
    for call in (lambda: w8a8.linear(t, w8a8.Weight(w.codes.contiguous(), w.scales)),
                 lambda: w8a8.quantize_tokens(torch.zeros(1, 65537, dtype=BF16, device="cuda"))):
        with pytest.raises(B.GptqError):
            call()
    assert torch.cuda.current_stream().query() in (True, False)
    _done()


# -- together ----------------------------------------------------------------------

@pytest.mark.parametrize("N,K", [(7, 8), (130, 72), (256, 1024)])
def test_pack_keeps_the_values(N, K):
    g = _gen(N)
    codes = torch.randint(0, 256, (N, K), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
    zeros = torch.randint(0, 256, (N,), generator=g).float().cuda()
    wq = torch.full((N, (K + 15) // 16 * 16), 99, dtype=torch.int8, device="cuda")
    z = torch.empty(N, dtype=torch.int32, device="cuda")
    B.gptq_w8a8_pack(wq[:, :K], z, codes, zeros)
    _done()
    assert torch.equal(wq[:, :K].int() - z[:, None], codes.int() - zeros.int()[:, None])
    assert (wq[:, K:] == 0).all()


@pytest.mark.parametrize("d_in", [512, 520])
def test_the_quantizers_8_bit_codes_in_the_linear(d_in):
    """Quantize a layer to 8 bits, lay its codes out, multiply: X W^T with
    the values the tokens' and the weights' codes stand for."""
    d_out = 256
    W, xb = synth.random_layer(21, d_out, d_in, 1024, correlated=True)
    q = LayerQuantizer(d_out, d_in, 8, -1, 128, 0.01, False)
    x = torch.from_numpy(np.ascontiguousarray(xb).view(np.int16)).cuda().view(BF16)
    q.add_batch(x)
    layer = q.run(torch.from_numpy(W.astype(np.float32)).cuda())
    weight = w8a8.pack(layer)
    values = weight.scales[:, None].double() * (weight.codes.double() - weight.zeros[:, None].double())
    # s (q - z) is rounded to float32 once where the quantizer stores it
    assert ((values - layer.W_hat.double()).abs() <= U * values.abs() * 1.01).all()
    for M in (1, 3, 40, 300):
        t = w8a8.quantize_tokens(x[:M], hat=True)
        y = w8a8.linear(t, weight, dtype=F32)
        _done()
        # the sum in integers: products of the scaled values have 64 significant bits, and where the sum
        # cancels to 0 their rounding to float64 alone is above the bound
        p = (t.codes.double() @ (weight.codes.double() - weight.zeros[:, None].double()).t()) * (
            t.scales[:, None].double() * weight.scales.double())
        assert ((y.double() - p).abs() <= 4.01 * U * p.abs()).all()


def test_streams_and_graphs():
    """The calls together on a stream of their own, and captured into a graph
    that is replayed on new inputs."""
    M, D, N = 37, 1000, 520
    b, r = _randn(1, M, D).to(BF16).cuda(), _randn(2, M, D).to(BF16).cuda()
    _, wd = _codes(3, N, D)
    weight = w8a8.Weight(wd, torch.rand(N, device="cuda") + 0.1, torch.randint(-9, 9, (N,), device="cuda", dtype=torch.int32))

    def step():
        x, t = w8a8.block_norm(b, r, post_norm=True, quantize=True)
        y = w8a8.linear(t, weight)
        return x, y, w8a8.linear(w8a8.quantize_tokens(y, gate=y), w8a8.Weight(wd[:, :N], weight.scales))

    torch.cuda.synchronize()
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    b.copy_(_randn(5, M, D).to(BF16))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    _done()
    assert all(torch.equal(u, v) for u, v in zip(want, kept))


def test_offsets_beyond_32_bits():
    """Rows whose elements lie more than 2^31 elements into their tensors."""
    x = torch.empty(40000, 65536, dtype=BF16, device="cuda")[:, :200]        # 5 GB, pitch 65536
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    t = w8a8.quantize_tokens(x)
    out = torch.empty(40000, 65536, dtype=BF16, device="cuda")[:, :200]
    B.gptq_block_norm(None, x, out=out)
    _done()
    for at in (slice(0, 50), slice(39950, 40000)):
        want = w8a8.quantize_tokens(x[at].contiguous())
        assert torch.equal(t.codes[at], want.codes) and torch.equal(t.sums[at], want.sums)
        assert torch.equal(out[at], w8a8.block_norm(None, x[at].contiguous())[1])
    del x, out
    M = N = 47000                                                           # Y of 2.2e9 elements
    _, xd = _codes(1, M, 48)
    _, wd = _codes(2, N, 48)
    ones = torch.ones(M, device="cuda")
    y = w8a8.linear(w8a8.Tokens(xd, ones), w8a8.Weight(wd, ones))
    _done()
    assert torch.equal(y[-3:].float(), (xd[-3:].float() @ wd.float().t()).to(BF16).float())
    assert torch.equal(y[:, -3:].float(), (xd.float() @ wd[-3:].float().t()).to(BF16).float())


@pytest.mark.parametrize("M", [1, 20, 90, 300, 1500])
def test_calls_in_a_row_without_waiting(M):
    """The kernels start before the one before them ends: a chain in which each
    call reads what the last one wrote, over the same buffers, against the
    same calls with a wait after each."""
    D, N = 512, 520
    _, w1 = _codes(3, N, D)
    _, w2 = _codes(4, D, N)
    u = torch.rand(N, device="cuda") * 1e-3 + 1e-4
    a, b = w8a8.Weight(w1, u), w8a8.Weight(w2, u[:D].contiguous(), torch.randint(-9, 9, (D,), device="cuda", dtype=torch.int32))
    x0 = _randn(M, M, D).to(BF16).cuda()

    def chain(wait):
        rest = (lambda: torch.cuda.synchronize()) if wait else (lambda: None)
        x, h = x0.clone(), torch.zeros(M, D, dtype=BF16, device="cuda")
        y = torch.empty(M, N, dtype=BF16, device="cuda")
        q, s, n = w8a8.empty_codes(M, D, "cuda"), torch.empty(M, device="cuda"), torch.empty(M, dtype=torch.int32, device="cuda")
        q2 = w8a8.empty_codes(M, N, "cuda")
        rest()
        for _ in range(12):
            B.gptq_block_norm(h, x, stream_out=x, q=q, q_scales=s, q_sums=n, scale=0.5)
            rest()
            B.gptq_w8a8_gemm(y, q, s, a.codes, a.scales)
            rest()
            B.gptq_quantize_tokens(q2, s, n, y, y)
            rest()
            B.gptq_w8a8_gemm(h, q2, s, b.codes, b.scales, n, b.zeros)
            rest()
        torch.cuda.synchronize()
        return x, h, y, q, q2

    want = chain(True)
    for _ in range(3):
        got = chain(False)
        assert all(torch.equal(u, v) for u, v in zip(want, got))
    _done()


def test_products_on_two_streams_at_once():
    """Kernels that hold tensor memory, on two streams, in every size class."""
    sizes = [(20, 700, 1024), (64, 4096, 2048), (300, 600, 512), (1000, 1000, 700), (1, 4096, 512)]
    jobs = []
    for M, N, K in sizes:
        _, xd = _codes(M, M, K)
        _, wd = _codes(N, N, K)
        jobs.append((w8a8.Tokens(xd, torch.rand(M, device="cuda")), w8a8.Weight(wd, torch.rand(N, device="cuda"))))
    want = [w8a8.linear(t, w) for t, w in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for r in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append([w8a8.linear(t, w) for t, w in (jobs if i else jobs[::-1])])
    for s in streams:
        s.synchronize()
    _done()
    for k, g in enumerate(got):
        for y, v in zip(want, g if k % 2 else g[::-1]):
            assert torch.equal(y, v)


def test_decoder_layer_in_8_bits():
    """Calibrate the small decoder layer for 8-bit linears and run it in 8
    bits, against the same flow in float64 with the dequantized weights."""
    shape = decoder.TINY
    W, X = decoder.synthetic_layer(shape)
    res = decoder.calibrate(X, W, shape, bits=8, group_size=-1, act_bits=8)
    packed = decoder.pack_w8a8(res.layers)
    x = X[:300]
    got = decoder.forward_w8a8(x, packed).double()
    _done()
    w = {n: v.W_hat.double() for n, v in res.layers.items()}
    rms = lambda a: a * torch.rsqrt(a.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731

    def tok(a):
        ratio, top = _exact_codes(a)
        return torch.round(ratio) * top[:, None] / 127

    v = tok(x.double()) @ w["v"].t()
    x1 = x.double() + tok(rms(v)) @ w["o"].t()
    t = tok(rms(x1))
    gate, up = t @ w["gate"].t(), t @ w["up"].t()
    attn, mlp = x1 - x.double(), tok(torch.nn.functional.silu(gate) * up) @ w["down"].t()
    # The bf16 roundings of v, o, gate and up (2^-9 of the value each) can move a value over a border between two of its 8-bit
    # codes, a step that is not small against them: rounding noise of half a step uniform, sqrt(1 / 12), in each of the four
    # quantizations bounds what it can do in the mean.  A step is t / 127, t at most 8 root mean squares of a normed row
    # and 30 of a gated one: 8 / 127 * sqrt(1 / 6) = 0.026 and 0.1 of the branch they feed.
    err = got - (x1 + mlp)
    assert err.norm() <= 0.052 * attn.norm() + 0.13 * mlp.norm() + _half(BF16) * (x1 + mlp).norm() * 2
    # act_bits=16 is the calibration that was there
    a = decoder.calibrate(X, W, shape, bits=4, group_size=128)
    b = decoder.calibrate(X, W, shape, bits=4, group_size=128, act_bits=16)
    assert all(torch.equal(a.layers[n].codes, b.layers[n].codes) for n in a.layers)
