"""The 8-bit operators against plain float64 (tests/i8_reference.py): quantised rows and filters value by
value, scales, products and outputs within the roundings that the contract allows."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import i8_reference as ref
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of float32


@pytest.fixture(scope="module")
def cb(cuda):
    import cnn_convolution_nhwc_b200 as m
    return m


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum((i + 1) * 1009 * int(k) for i, k in enumerate(key)) % (1 << 31))


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _bytes(g, rows, C, cb, lo=-127):
    """Random 8-bit rows whose gap between C and the pitch holds garbage."""
    # a pitch of 16 bytes more than a multiple of 32 for some shapes
    pitch = (C + 15) // 16 * 16
    q = torch.full((rows, pitch), 77, dtype=torch.int8, device="cuda")[:, :C]
    q.copy_(torch.randint(lo, 128, (rows, C), generator=g, device="cuda"))
    return q


def _q(t):
    return t.cpu().numpy().astype(np.int64)


def _close(a, b, rel):
    """Scales: equal NaN places, zero equals zero, else within rel (plus the smallest float32 step)."""
    a, b = a.astype(np.float64), np.asarray(b, np.float64)
    assert np.array_equal(np.isnan(a), np.isnan(b))
    ok = ~np.isnan(b)
    assert np.all(np.abs(a[ok] - b[ok]) <= rel * np.abs(b[ok]) + 2.0 ** -149), np.max(np.abs(a[ok] - b[ok]) / np.abs(b[ok]))


# widths on both sides of every kernel's limit: a warp a row (512, 1024), a block (8192, 16384), pieces
# above; multiples of 8 and odd ones
WIDTHS = [(1, 1), (2, 8), (3, 7), (5, 64), (2, 127), (33, 512), (9, 520), (2, 1001), (4, 1024), (3, 1025), (3, 1032),
          (2, 2056), (2, 2049), (2, 4001), (7, 4096), (2, 5003), (2, 6145), (2, 8191), (1, 8192), (2, 8200), (2, 9224), (2, 10240), (2, 10248), (2, 12343),
          (3, 16384), (2, 16385), (1, 20000), (2, 40001), (1, 57001), (1, 113001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,C", WIDTHS)
def test_rmsnorm(cb, M, C, dtype):
    g = _gen(M, C)
    x, r, w = _normal(g, M, C, dtype=dtype), _normal(g, M, C, dtype=dtype), 1 + 0.2 * _normal(g, C)
    # the float32 sum of squares: at most 64 terms in a row per thread and piece of 16384 values, then ten
    # steps of tree; half of its relative error reaches the scale, plus five roundings
    rel = ((64 * (C // 16384 + 1) + 10) / 2 + 5) * U
    for residual in (None, r):
        q, scale, h = cb.rmsnorm_i8_fwd(x, w, residual, eps=1e-6)
        rq, rs, rh = ref.rmsnorm(x, w, residual)
        assert (h is None) == (residual is None)
        if h is not None:
            assert torch.equal(h.cpu(), rh)
        assert np.array_equal(_q(q), rq)
        _close(scale.cpu().numpy(), rs, rel)
    assert cb.conv_device_status() == cb.CONV_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,C", WIDTHS)
def test_quant_rows(cb, M, C, dtype):
    g = _gen(M, C, 1)
    x = _normal(g, M, C, dtype=dtype)
    q, scale = cb.quant_rows_i8_fwd(x)
    rq, rs = ref.rows(ref.f64(x))
    assert np.array_equal(_q(q), rq)
    _close(scale.cpu().numpy(), rs, U)
    # gated: the kernel's silu is off by 2^-22 + |a| 2^-23 relative, and three float32 roundings
    x = _normal(g, M, 2 * C, dtype=dtype) * 3
    q, scale = cb.quant_rows_i8_fwd(x, glu=True)
    v = ref.glu(x)
    off = (2.0 ** -22 + np.abs(ref.f64(x)[:, :C]) * 2.0 ** -23 + 2.0 ** -21) * np.abs(v)   # of v
    a = np.abs(v).max(axis=1, keepdims=True)
    s = ref.f64(scale)[:, None]
    assert np.all(np.abs(s - a / 127) <= off.max(axis=1, keepdims=True) / 127 + U * a)
    assert np.all(np.abs(_q(q) * s - v) <= s * (0.5 + 1e-6) + off + a * 2.0 ** -20)
    assert cb.conv_device_status() == cb.CONV_OK


def _special_rows(C, dtype):
    """Rows where the rounding, the range or the values are at an edge."""
    r = np.random.default_rng(5)
    rows = [np.zeros(C), -np.zeros(C), np.full(C, -3.5), np.where(np.arange(C) == C // 2, 1.0, 0.0)]
    rows.append(r.standard_normal(C) * 1e30)                          # sums of squares pass the float32 range
    rows.append(r.standard_normal(C) * 2.0 ** -130)                   # denormals
    rows.append(np.where(np.arange(C) % 3 == 0, 2.0 ** -133, 0.0))    # the smallest bf16 step
    rows.append(r.standard_normal(C) * 2.0 ** -100)
    rows.append((r.integers(-254, 255, C)) * 0.5)                     # halves of 127 / A with A = 127: ties
    rows.append(r.integers(-254, 255, C) * 2.0 ** -3)
    rows[-1][0] = rows[-2][0] = 127.0
    for bad in (np.nan, np.inf, -np.inf):
        x = r.standard_normal(C)
        x[C - 1] = bad
        rows.append(x)
    rows.append(np.full(C, 3e38))
    return torch.tensor(np.stack(rows), dtype=torch.float64).to(torch.float32).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 77, 520, 4096, 4099, 16400])
def test_special_rows(cb, C, dtype):
    x = _special_rows(C, dtype)
    q, scale = cb.quant_rows_i8_fwd(x)
    rq, rs = ref.rows(ref.f64(x))
    assert np.array_equal(_q(q), rq)
    _close(scale.cpu().numpy(), rs, U)
    w = torch.ones(C, device="cuda")
    q, scale, h = cb.rmsnorm_i8_fwd(x, w, torch.zeros_like(x))
    rq, rs, rh = ref.rmsnorm(x, w, torch.zeros_like(x))
    assert np.array_equal(_q(q), rq)
    assert np.array_equal(ref.f64(h), ref.f64(rh), equal_nan=True)
    _close(scale.cpu().numpy(), rs, ((64 * (C // 16384 + 1) + 10) / 2 + 5) * U)
    # a row that cannot be held reads back as NaN, and so does every product with it
    y = ref.f64(cb.dequant_rows_i8_fwd(q, scale, dtype=torch.float32))
    assert np.array_equal(np.isnan(y).all(axis=1), np.isnan(rs)) and np.array_equal(np.isnan(y).any(axis=1), np.isnan(rs))
    # the gate: minus infinity gives NaN (infinity times zero), large finite gates 0 or themselves
    x2 = torch.cat([x, torch.ones_like(x)], dim=1)
    q, scale = cb.quant_rows_i8_fwd(x2, glu=True)
    with np.errstate(all="ignore"):
        v = ref.glu(x2)
    assert np.array_equal(np.isnan(ref.f64(scale)), ~np.isfinite(v).all(axis=1) | (np.abs(v).max(axis=1) > 3.4028235e38))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Cin,Cout", [(1, 1), (7, 3), (64, 64), (128, 72), (129, 65), (250, 8), (1000, 1353), (1024, 512),
                                      (1025, 200), (4100, 136), (5003, 33), (9000, 72), (9100, 65), (17000, 40), (10300, 33)])
def test_quant_filter(cb, Cin, Cout, dtype):
    g = _gen(Cin, Cout)
    F = _normal(g, Cin, Cout, dtype=dtype)
    if Cout > 4:
        F[:, 1] = 0
        F[Cin // 2, 2] = float("nan")
        F[Cin - 1, 3] = float("inf")
    q, scale = cb.quant_filter_i8_fwd(F)
    rq, rs = ref.rows(np.ascontiguousarray(ref.f64(F).T))
    assert np.array_equal(_q(q), rq)
    _close(scale.cpu().numpy(), rs, U)
    q4, scale4 = cb.quant_filter_i8_fwd(F.reshape(1, 1, Cin, Cout))
    assert torch.equal(q4, q) and torch.equal(scale4.nan_to_num(), scale.nan_to_num())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,C", [(1, 1), (3, 16), (5, 33), (2, 512), (4, 528), (300, 1000), (7, 4097)])
def test_dequant(cb, M, C, dtype):
    g = _gen(M, C, 2)
    q, scale = _bytes(g, M, C, cb, lo=-128), _normal(g, M)
    y = cb.dequant_rows_i8_fwd(q, scale, dtype=dtype)
    assert torch.equal(y, (q.float() * scale[:, None]).to(dtype))


VARIANTS = ["", "pair,256", "pair,128", "split,16,1", "split,32,2", "split,64,4", "split,128,8", "split,128,1", "split,16,8"]
SHAPES = [(1, 1, 1), (1, 16, 8), (2, 17, 7), (3, 256, 128), (40, 384, 250), (90, 640, 140), (31, 1152, 300), (5, 127, 129), (16, 128, 128), (17, 129, 300), (33, 1000, 257), (64, 1024, 512),
          (65, 1030, 1000), (128, 500, 1001), (129, 4096, 136), (300, 1100, 264), (513, 272, 520), (1000, 96, 777)]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("M,Cin,Cout", SHAPES)
def test_product(cb, M, Cin, Cout, variant, monkeypatch):
    monkeypatch.setenv("CONV_B200_I8", variant)
    g = _gen(M, Cin, Cout)
    q, wq = _bytes(g, M, Cin, cb, lo=-128), _bytes(g, Cout, Cin, cb, lo=-128)
    qs, ws, bias = _normal(g, M) / 100, _normal(g, Cout) / 100, _normal(g, Cout)
    for dtype, b in ((torch.bfloat16, None), (torch.bfloat16, bias), (torch.float32, bias), (torch.float32, None)):
        guard = torch.full((M + 1, Cout), 7.0, dtype=dtype, device="cuda")
        y = cb.pointwise_i8_fwd(q, qs, wq, ws, b, y=guard[:M])
        want, mag = ref.product(q, qs, wq, ws, b)
        # the int32 sum to float32, two products and the bias: four float32 roundings; then the output's
        tol = 4 * U * mag * (1 + ref.round_half(dtype)) + ref.round_half(dtype) * np.abs(want) + 2.0 ** -149
        assert np.all(np.abs(ref.f64(y) - want) <= tol)
        assert torch.all(guard[M] == 7.0)
    assert cb.conv_device_status() == cb.CONV_OK


def test_product_rows_do_not_depend_on_the_batch(cb):
    g = _gen(31)
    for C, N in ((1000, 776), (4096, 1001)):
        q, wq = _bytes(g, 1100, C, cb), _bytes(g, N, C, cb)
        qs, ws, bias = _normal(g, 1100), _normal(g, N), _normal(g, N)
        for b in (None, bias):
            for dtype in (torch.bfloat16, torch.float32):
                y = cb.pointwise_i8_fwd(q, qs, wq, ws, b, dtype=dtype)
                for M in (1, 20, 100, 300):
                    assert torch.equal(cb.pointwise_i8_fwd(q[:M], qs[:M], wq, ws, b, dtype=dtype), y[:M])


def test_product_largest_sums(cb):
    # 131071 products of -128 * -128: 2^31 - 2^14, the largest sum that is promised
    for M in (3, 700):
        q = cb.empty_rows_i8(M, 131071).fill_(-128)
        w = cb.empty_rows_i8(5, 131071).fill_(-128)
        w[1] = 127
        one = torch.ones(M, device="cuda"), torch.ones(5, device="cuda")
        y = cb.pointwise_i8_fwd(q, one[0], w, one[1], dtype=torch.float32)
        assert torch.all(y[:, 0] == float(np.float32(131071 * 16384))) and torch.all(y[:, 1] == float(np.float32(-131071 * 128 * 127)))


def test_product_of_dead_rows_and_channels(cb):
    g = _gen(8)
    q, wq = _bytes(g, 40, 100, cb), _bytes(g, 50, 100, cb)
    qs, ws = torch.ones(40, device="cuda"), torch.ones(50, device="cuda")
    q[3] = 0
    qs[3] = float("nan")
    ws[7] = float("nan")
    y = cb.pointwise_i8_fwd(q, qs, wq, ws)
    bad = torch.zeros(40, 50, dtype=torch.bool, device="cuda")
    bad[3] = True
    bad[:, 7] = True
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("shape", [(2, 7, 7, 96, 160), (1, 1, 1, 4096, 512), (1, 1, 77, 515, 260), (8, 14, 14, 672, 112)])
def test_layer_is_its_parts(cb, shape):
    N, H, W, Cin, Cout = shape
    g = _gen(*shape)
    X, F = _normal(g, N, H, W, Cin, dtype=torch.bfloat16), _normal(g, Cin, Cout, dtype=torch.bfloat16) / Cin ** 0.5
    bias, norm = _normal(g, Cout), 1 + 0.1 * _normal(g, Cin)
    wq, ws = cb.quant_filter_i8_fwd(F)
    x = X.reshape(-1, Cin)
    for n in (None, norm):
        Y = cb.conv2d_nhwc_fwd_i8(X, wq, ws, bias, norm=n, eps=1e-5)
        # a workspace for the pitch of 32 bytes, and the smallest one, at 16
        small = torch.empty(N * H * W * ((Cin + 15) // 16 * 16 + 4), dtype=torch.uint8, device="cuda")
        assert torch.equal(Y, cb.conv2d_nhwc_fwd_i8(X, wq, ws, bias, norm=n, eps=1e-5, workspace=small))
        Y2 = torch.full_like(Y, 7.0)   # every output given: the short call
        assert cb.conv2d_nhwc_fwd_i8(X, wq, ws, bias, norm=n, eps=1e-5, Y=Y2, workspace=small) is Y2 and torch.equal(Y, Y2)
        q, s = cb.quant_rows_i8_fwd(x) if n is None else cb.rmsnorm_i8_fwd(x, n, eps=1e-5)[:2]
        assert torch.equal(Y.reshape(-1, Cout), cb.pointwise_i8_fwd(q, s, wq, ws, bias))
        # against the float layer: each operand is off by at most half a step of its scale
        v = ref.f64(x)
        if n is not None:
            v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + 1e-5) * ref.f64(n)
        y = v @ ref.f64(F) + ref.f64(bias)
        s, w = ref.f64(s)[:, None], ref.f64(F)
        off = 0.5001 * s * np.abs(w).sum(axis=0) + 0.5001 * ref.f64(ws) * (np.abs(v) + s).sum(axis=1, keepdims=True)
        assert np.all(np.abs(ref.f64(Y).reshape(-1, Cout) - y) <= off + 2.0 ** -7 * np.abs(y) + 1e-4 * np.abs(y).max())


def _feed_forward(cb, x, res, norm, w1, w2, bufs=None):
    """norm and residual -> up and gate projections -> gate -> down projection."""
    q, s, h = cb.rmsnorm_i8_fwd(x, norm, res)
    q2, s2 = cb.quant_rows_i8_fwd(cb.pointwise_i8_fwd(q, s, *w1), glu=True)
    return cb.pointwise_i8_fwd(q2, s2, *w2), h


@pytest.mark.parametrize("M", [1, 40, 700])
def test_feed_forward_run(cb, M):
    C, Fd = 512, 1360
    g = _gen(M, 3)
    x, res = _normal(g, M, C, dtype=torch.bfloat16), _normal(g, M, C, dtype=torch.bfloat16)
    norm = 1 + 0.1 * _normal(g, C)
    f1, f2 = _normal(g, C, 2 * Fd) / C ** 0.5, _normal(g, Fd, C) / Fd ** 0.5
    w1, w2 = cb.quant_filter_i8_fwd(f1), cb.quant_filter_i8_fwd(f2)
    y, h = _feed_forward(cb, x, res, norm, w1, w2)
    # against 64 bits without any quantisation: the rms of the error of 8-bit rows is about 1 / (127 sqrt(12))
    # of a row's largest value, four such roundings on the way; 5 % of the output's rms is ten times that
    hd = ref.f64(h)
    t = hd / np.sqrt((hd * hd).mean(axis=1, keepdims=True) + 1e-6) * ref.f64(norm)
    u = t @ ref.f64(f1)
    want = (u[:, :Fd] / (1 + np.exp(-u[:, :Fd])) * u[:, Fd:]) @ ref.f64(f2)
    assert np.sqrt(np.mean((ref.f64(y) - want) ** 2)) <= 0.05 * np.sqrt(np.mean(want ** 2))
    # the same run in place, on another stream, with a synchronisation after each call, and captured
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, _ = _feed_forward(cb, x, res, norm, w1, w2)
    s.synchronize()
    assert torch.equal(y2, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y3, h3 = _feed_forward(cb, x, res, norm, w1, w2)
    for _ in range(3):
        y3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and torch.equal(h3, h)
    inplace = res.clone()
    q, sc, hh = cb.rmsnorm_i8_fwd(x, norm, inplace, h=inplace)
    assert hh is inplace and torch.equal(inplace, h)
    inplace = x.clone()
    q2, sc2, _ = cb.rmsnorm_i8_fwd(inplace, norm, res, h=inplace)
    assert torch.equal(inplace, h) and torch.equal(q2, q) and torch.equal(sc2, sc)
    assert cb.conv_device_status() == cb.CONV_OK


def test_two_streams_at_once(cb):
    g = _gen(12)
    X = _normal(g, 1, 1, 300, 1024, dtype=torch.bfloat16)
    ws = [cb.quant_filter_i8_fwd(_normal(g, 1024, n)) for n in (1024, 640)]
    want = [cb.conv2d_nhwc_fwd_i8(X, *w) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(20):
        got = []
        for st, w in zip(streams, ws):
            with torch.cuda.stream(st):
                got.append(cb.conv2d_nhwc_fwd_i8(X, *w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bit_offsets(cb):
    M, C = 525000, 4104   # 2.15e9 values
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    tail = _normal(_gen(4), 3, C, dtype=torch.bfloat16)
    x[-3:] = tail
    q, scale = cb.quant_rows_i8_fwd(x)
    rq, rs = ref.rows(ref.f64(tail))
    assert np.array_equal(_q(q[-3:]), rq) and not q[0].any() and not q[M // 2].any()
    del x
    y = cb.dequant_rows_i8_fwd(q, scale)
    assert torch.equal(y[-3:], (q[-3:].float() * scale[-3:, None]).bfloat16())


def test_product_past_32_bit_offsets(cb):
    M, N = 66000, 32776   # 2.16e9 outputs
    g = _gen(6)
    q, wq = _bytes(g, M, 64, cb), _bytes(g, N, 64, cb)
    qs, ws = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = cb.pointwise_i8_fwd(q, qs, wq, ws)
    want, mag = ref.product(q[-2:], qs[-2:], wq, ws, None)
    assert np.all(np.abs(ref.f64(y[-2:]) - want) <= (4 * U + 2.0 ** -8) * mag)
    del y


def test_gap_between_rows_is_left_alone(cb):
    g = _gen(9)
    for M, C in ((5, 1000), (3, 33), (4, 5003)):
        base = torch.full((M + 1, (C + 15) // 16 * 16 + 32), 55, dtype=torch.int8, device="cuda")
        q = base[:M, :C]
        x = _normal(g, M, C, dtype=torch.bfloat16)
        cb.quant_rows_i8_fwd(x, q=q)
        assert torch.all(base[:M, C:] == 55) and torch.all(base[M] == 55)
        assert torch.equal(q, cb.quant_rows_i8_fwd(x)[0])
        F = _normal(g, C, M)
        cb.quant_filter_i8_fwd(F, q=q)
        assert torch.all(base[:M, C:] == 55) and torch.all(base[M] == 55)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,C", [(3, 40), (5, 1001), (2, 5000)])
def test_tensors_off_16_bytes(cb, M, C, dtype):
    g = _gen(M, C, 5)

    def view(n):   # starts one element into its storage
        return _normal(g, n + 1, dtype=dtype)[1:]
    x, r = view(M * C).view(M, C), view(M * C).view(M, C)
    w = 1 + 0.1 * _normal(g, C + 1)[1:]
    h = view(M * C).view(M, C)
    q, scale, h = cb.rmsnorm_i8_fwd(x, w, r, h=h)
    rq, rs, rh = ref.rmsnorm(x, w, r)
    assert torch.equal(h.cpu(), rh) and np.array_equal(_q(q), rq)
    x2 = view(M * 2 * C).view(M, 2 * C)
    for a, b in ((cb.quant_rows_i8_fwd(x), cb.quant_rows_i8_fwd(x.clone())),
                 (cb.quant_rows_i8_fwd(x2, glu=True), cb.quant_rows_i8_fwd(x2.clone(), glu=True)),
                 (cb.quant_filter_i8_fwd(x), cb.quant_filter_i8_fwd(x.clone()))):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    y = view(M * C).view(M, C)
    assert torch.equal(cb.dequant_rows_i8_fwd(q, scale, y=y), cb.dequant_rows_i8_fwd(q, scale, dtype=dtype))
    wq, ws = cb.quant_filter_i8_fwd(_normal(g, C, 64))
    y = view(M * 64).view(M, 64)
    for v in ("", "pair,256", "pair,128"):
        os.environ["CONV_B200_I8"] = v
        try:
            assert torch.equal(cb.pointwise_i8_fwd(q, scale, wq, ws, y=y), cb.pointwise_i8_fwd(q, scale, wq, ws, dtype=dtype))
        finally:
            del os.environ["CONV_B200_I8"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [3000, 9001, 17000])
def test_norm_of_tensors_that_start_apart(cb, C, dtype):
    """x, the residual and h each off 16 bytes by a different number of elements; then in place."""
    g, M = _gen(C, 6), 3

    def view(off):
        return _normal(g, M * C + off, dtype=dtype)[off:].view(M, C)
    x, r, w = view(1), view(3), 1 + 0.1 * _normal(g, C)
    rq, rs, rh = ref.rmsnorm(x, w, r)
    for h in (view(2), r, x):
        a, b = (x.clone(), r.clone()) if h is x or h is r else (x, r)
        q, scale, h = cb.rmsnorm_i8_fwd(x, w, r, h=h)
        assert torch.equal(h.cpu(), rh) and np.array_equal(_q(q), rq)
        _close(scale.cpu().numpy(), rs, ((64 * (C // 16384 + 1) + 10) / 2 + 5) * U)
        x.copy_(a)
        r.copy_(b)


def test_gates_far_from_zero(cb):
    # silu against float64 over the float32 range of gates; below -87 it counts as 0 (its size is below 1.5e-36)
    gates = torch.tensor([-3e38, -1e30, -200.0, -100.0, -88.0, -87.5, -86.0, -60.0, -20.0, -5.0, -1.0, -0.0, 0.0, 1e-30, 0.5, 5.0, 20.0,
                          88.0, 100.0, 1e30], device="cuda")
    for up in (1.0, -0.37):
        for g in gates:   # a row each, so that its own value sets the scale
            x = torch.stack([g.repeat(8), torch.full((8,), up, device="cuda")]).reshape(1, 16)
            q, s = cb.quant_rows_i8_fwd(x, glu=True)
            v, got = ref.glu(x)[0, 0], float(q[0, 0].item() * s[0].double().item())
            assert abs(got - v) <= (2.0 ** -21 + abs(float(g)) * 2.0 ** -23 if abs(float(g)) < 100 else 2.0 ** -21) * abs(v) + 1.5e-36 * abs(up)


def test_rows_of_2_27_values(cb):
    for C in (1 << 27, (1 << 27) - 3):
        x = torch.zeros(1, C, dtype=torch.bfloat16, device="cuda")
        x[0, 5], x[0, C - 1], x[0, C - 20] = 2.0, -1.0, 0.5
        q, s = cb.quant_rows_i8_fwd(x)
        assert s.item() == float(np.float32(2.0) / np.float32(127.0)) and int(q.int().abs().sum(dtype=torch.int64)) == 127 + 64 + 32
        assert q[0, 5] == 127 and q[0, C - 1] == -64 and q[0, C - 20] == 32   # -63.5 to even
        y = cb.dequant_rows_i8_fwd(q, s)
        assert y[0, C - 1] == (torch.tensor(-64.0) * s.cpu()).bfloat16().item() and int((y != 0).sum()) == 3


def test_rows_past_the_batch_are_left_alone(cb):
    g = _gen(14)
    for M, C in ((3, 1000), (5, 257), (1, 4096)):
        buf = torch.full((M + 2, C), 9.0, dtype=torch.bfloat16, device="cuda")
        scale = torch.full((M + 2,), 9.0, device="cuda")
        x, r = _normal(g, M, C, dtype=torch.bfloat16), _normal(g, M, C, dtype=torch.bfloat16)
        cb.rmsnorm_i8_fwd(x, torch.ones(C, device="cuda"), r, h=buf[1:M + 1] if (C * 2) % 16 == 0 else buf[:M], scale=scale[1:M + 1])
        first = 1 if (C * 2) % 16 == 0 else 0
        assert torch.all(buf[:first] == 9.0) and torch.all(buf[M + first:] == 9.0) and scale[0] == 9.0 and scale[M + 1] == 9.0
        q, s = cb.quant_rows_i8_fwd(x)
        y = torch.full((M + 1, C), 9.0, device="cuda")
        cb.dequant_rows_i8_fwd(q, s, y=y[:M])
        assert torch.all(y[M] == 9.0)


CHILD = r'''
import os, sys
import numpy as np
sys.path.insert(0, os.environ["CONV_TEST_ROOT"])
import cnn_convolution_nhwc_b200 as cb
from tests.test_i8_gpu import run_all
assert cb.conv_debug_bounds_build()
out = run_all(cb)
assert cb.conv_device_status() == cb.CONV_OK
assert cb.conv_debug_bounds_info() is None, cb.conv_debug_bounds_info()
np.savez(os.environ["CONV_TEST_OUT"], **out)
'''


def run_all(cb):
    out = {}
    for M, C, N in ((3, 77, 50), (40, 1032, 136), (300, 4099, 264), (2, 16640, 8)):
        g = _gen(M, C, N)
        for dtype in (torch.bfloat16, torch.float32):
            x, r = _normal(g, M, C, dtype=dtype), _normal(g, M, C, dtype=dtype)
            q, s, h = cb.rmsnorm_i8_fwd(x, 1 + 0.1 * _normal(g, C), r)
            q2, s2 = cb.quant_rows_i8_fwd(torch.cat([x, r], dim=1), glu=True)
            w, ws = cb.quant_filter_i8_fwd(_normal(g, C, N, dtype=dtype))
            ys = []
            for v in ("", "pair,256", "pair,128", "split,16,1", "split,64,1"):
                os.environ["CONV_B200_I8"] = v
                ys.append(cb.pointwise_i8_fwd(q, s, w, ws, _normal(g, N), dtype=dtype))
            os.environ.pop("CONV_B200_I8")
            for i, t in enumerate([q, s, h, q2, s2, w, ws, cb.dequant_rows_i8_fwd(q, s, dtype=dtype), *ys]):
                out[f"{M}-{C}-{dtype}-{i}"] = t.float().cpu().numpy()
    return out


def test_bounds_checked_build(cb, tmp_path):
    f = tmp_path / "out.npz"
    env = dict(os.environ, CONV_B200_DEBUG_BOUNDS="1", CONV_TEST_ROOT=ROOT, CONV_TEST_OUT=str(f))
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = np.load(f)
    for k, v in run_all(cb).items():
        assert np.array_equal(v, got[k], equal_nan=True), k


def test_short_and_checked_calls_agree(cb):
    # every output given on the current stream: the C++ path; a stream named: the checked one
    g = _gen(21)
    s = torch.cuda.current_stream()
    for M, C, N in ((1, 1024, 256), (5, 333, 70)):
        x, r = _normal(g, M, C, dtype=torch.bfloat16), _normal(g, M, C, dtype=torch.bfloat16)
        w, F, x2 = 1 + 0.1 * _normal(g, C), _normal(g, C, N), _normal(g, M, 2 * C)

        def out(rows, cols):
            return dict(q=cb.empty_rows_i8(rows, cols), scale=torch.empty(rows, device="cuda"))
        a = cb.rmsnorm_i8_fwd(x, w, r, h=torch.empty_like(x), **out(M, C))
        b = cb.rmsnorm_i8_fwd(x, w, r, stream=s)
        c = cb.quant_rows_i8_fwd(x2, glu=True, **out(M, C)) + cb.quant_filter_i8_fwd(F, **out(N, C))
        d = cb.quant_rows_i8_fwd(x2, glu=True, stream=s) + cb.quant_filter_i8_fwd(F, stream=s)
        for t, u in zip(a + c, b + d):
            assert torch.equal(t, u)
        y = torch.empty(M, N, device="cuda")
        assert torch.equal(cb.pointwise_i8_fwd(a[0], a[1], c[2], c[3], y=y), cb.pointwise_i8_fwd(a[0], a[1], c[2], c[3], dtype=torch.float32))
        y = torch.empty(M, C, device="cuda")
        assert torch.equal(cb.dequant_rows_i8_fwd(a[0], a[1], y=y), cb.dequant_rows_i8_fwd(a[0], a[1], dtype=torch.float32))
    assert cb._fast.pointwise(a[0], a[1], c[2], c[3], None, torch.empty(M, N, device="cuda")) == cb.CONV_OK


def test_binding_refuses_with_the_outputs_given(cb):
    # what the short path leaves alone reaches the checked one, which names the argument
    x = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
    q, scale, w = cb.empty_rows_i8(4, 32), torch.empty(4, device="cuda"), torch.ones(32, device="cuda")
    y = torch.empty(4, 4, device="cuda")
    with pytest.raises(ValueError, match="scale must have shape"):
        cb.quant_rows_i8_fwd(x, q=q, scale=scale[:3])
    with pytest.raises(ValueError, match="q must have shape"):
        cb.quant_rows_i8_fwd(x, q=q[:3], scale=scale)
    with pytest.raises(ValueError, match="contiguous"):
        cb.quant_rows_i8_fwd(x.t(), q=q, scale=scale)
    with pytest.raises(TypeError, match="x must be"):
        cb.quant_rows_i8_fwd(x.half(), q=q, scale=scale)
    with pytest.raises(TypeError, match="weight must be"):
        cb.rmsnorm_i8_fwd(x, w.half(), q=q, scale=scale)
    with pytest.raises(ValueError, match="residual too"):
        cb.rmsnorm_i8_fwd(x, w, h=x, q=q, scale=scale)
    with pytest.raises(ValueError, match="16-byte"):
        cb.pointwise_i8_fwd(torch.zeros(4, 40, dtype=torch.int8, device="cuda")[:, :32], scale,
                            torch.zeros(4, 33, dtype=torch.int8, device="cuda")[:, :32], scale, y=y)
    with pytest.raises(ValueError, match="columns"):
        cb.pointwise_i8_fwd(q, scale, cb.empty_rows_i8(4, 48), scale, y=y)
    with pytest.raises(ValueError, match="bias must have shape"):
        cb.pointwise_i8_fwd(q, scale, q, scale, bias=w, y=y)
    with pytest.raises(ValueError, match="CUDA"):
        cb.dequant_rows_i8_fwd(q, scale, y=torch.empty(4, 32))
    memory = torch.zeros(4 * 32, device="cuda")   # the library's own refusals: y on q's bytes, eps
    with pytest.raises(cb.ConvError):
        cb.dequant_rows_i8_fwd(memory.view(torch.int8)[:128].view(4, 32), scale, y=memory.view(4, 32))
    with pytest.raises(cb.ConvError):
        cb.rmsnorm_i8_fwd(x, w, eps=0.0, q=q, scale=scale)


def test_binding_does_not_cut_sizes_past_int(cb):
    """2^32 + 16 columns or rows, 16 in an int's bits: refused before anything is launched."""
    n = 2 ** 32 + 16
    x = torch.empty(1, n, dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    y = torch.full((1, 16), 5.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="larger than 2"):
        cb.dequant_rows_i8_fwd(x, one, y=y)
    with pytest.raises(ValueError, match="larger than 2"):
        cb.pointwise_i8_fwd(x, one, x, one, y=y[:, :1].contiguous())
    assert torch.all(y == 5.0)
    del x
    x = torch.empty(n // 2, 2, dtype=torch.bfloat16, device="cuda")   # 2^31 + 8 rows
    q, scale = cb.empty_rows_i8(16, 2), torch.full((16,), 5.0, device="cuda")
    for glu in (False, True):
        with pytest.raises(ValueError, match="larger than 2"):
            cb.quant_rows_i8_fwd(x, glu=glu, q=q, scale=scale)
        with pytest.raises(ValueError, match="larger than 2"):
            cb.quant_rows_i8_fwd(x, glu=glu)
    with pytest.raises(ValueError, match="larger than 2"):
        cb.rmsnorm_i8_fwd(x, torch.ones(2, device="cuda"), q=q, scale=scale)
    with pytest.raises(ValueError, match="larger than 2"):
        cb.quant_filter_i8_fwd(x, q=q, scale=scale)
    with pytest.raises(ValueError, match="larger than 2"):
        cb.conv2d_nhwc_fwd_i8(x.view(n // 2, 1, 1, 2), cb.empty_rows_i8(16, 2), scale)
    assert torch.all(scale == 5.0)
