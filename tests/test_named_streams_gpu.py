"""Calls on a stream named by `stream=` while another one is current: what they allocate belongs to the named
stream, so that the allocator hands it out again only behind their kernels."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cb(cuda):
    import cnn_convolution_nhwc_b200 as m
    return m


def _block_stream(ptr):
    """The stream that the allocator keeps the block at ptr for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= ptr < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not a block of the allocator")


def _bf16(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def _calls(cb):
    """Every entry point that allocates, with what it takes prepared on the current stream."""
    X, F3, F1 = _bf16(2, 12, 12, 32), _bf16(3, 3, 32, 32), _bf16(32, 48)
    x, w = torch.randn(2, 8, 14, 14, device="cuda"), torch.randn(8, 3, 3, device="cuda")
    rows, norm = _bf16(300, 32), torch.ones(32, device="cuda")
    wq, ws = cb.quant_filter_i8_fwd(F1)
    q, qs = cb.quant_rows_i8_fwd(rows)
    return {
        "dense": lambda s: cb.conv2d_nhwc_fwd(X, F3, stream=s),
        "f32": lambda s: cb.conv2d_nhwc_fwd_f32(X.float(), F3.float(), stream=s),
        "ex": lambda s: cb.conv2d_nhwc_fwd_ex(X, F3, pad=1, stream=s),
        "grouped": lambda s: cb.conv2d_nhwc_fwd_grouped(X, F3, pad=1, stream=s),
        "im2col": lambda s: cb.conv2d_nhwc_fwd_im2col(X, F3, stream=s),
        "depthwise": lambda s: cb.depthwise_fwd(x, w, stream=s),
        "dwpw": lambda s: cb.dwpw_fwd(x, w, None, F1[:8].contiguous(), pad=1, stream=s),
        "norm": lambda s: cb.rmsnorm_i8_fwd(rows, norm, rows, stream=s),
        "rows": lambda s: cb.quant_rows_i8_fwd(rows, stream=s),
        "filter": lambda s: cb.quant_filter_i8_fwd(F1, stream=s),
        "dequant": lambda s: cb.dequant_rows_i8_fwd(q, qs, stream=s),
        "product": lambda s: cb.pointwise_i8_fwd(q, qs, wq, ws, stream=s),
        "layer": lambda s: cb.conv2d_nhwc_fwd_i8(X, wq, ws, stream=s),
    }


def _tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("name", ["dense", "f32", "ex", "grouped", "im2col", "depthwise", "dwpw", "norm", "rows", "filter",
                                  "dequant", "product", "layer"])
def test_allocations_belong_to_the_named_stream(cb, name, monkeypatch):
    call = _calls(cb)[name]
    want = _tensors(call(None))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []   # every tensor of the call, the workspaces that it drops among them
    real = cb._call
    monkeypatch.setattr(cb, "_call", lambda fn, what, tensors, *a: (seen.append(tensors), real(fn, what, tensors, *a)))
    given = {t.data_ptr() for t in call.__closure__ for t in [t.cell_contents] if isinstance(t, torch.Tensor)}
    for stream in (s, s.cuda_stream):   # the stream, or its handle
        seen.clear()
        out = _tensors(call(stream))
        s.synchronize()
        own = {t.data_ptr() for t in out}
        assert own and all(_block_stream(p) == s.cuda_stream for p in own)
        if name in ("im2col", "layer"):   # Y and the workspace
            made = [t.data_ptr() for t in seen[-1] if t is not None and t.data_ptr() not in given and t.dtype == torch.uint8]
            assert len(made) == 1 and _block_stream(made[0]) == s.cuda_stream
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(_tensors(call(0)), want))   # handle 0: the default stream


@pytest.mark.parametrize("name", ["im2col", "layer"])
def test_workspace_outlives_the_call(cb, name):
    """A call without a workspace behind long kernels of its stream; meanwhile blocks of the workspace's size
    are taken and filled on the current stream."""
    if name == "layer":
        X = _bf16(4, 14, 14, 256)
        wq, ws = cb.quant_filter_i8_fwd(_bf16(256, 128))
        size = cb.lib.conv2d_nhwc_i8_workspace(4, 14, 14, 256)

        def call(s):
            return cb.conv2d_nhwc_fwd_i8(X, wq, ws, stream=s)
    else:
        X, F = _bf16(4, 14, 14, 64), _bf16(3, 3, 64, 64)
        size = cb.lib.conv2d_nhwc_im2col_workspace(4, 14, 14, 64, 3)

        def call(s):
            return cb.conv2d_nhwc_fwd_im2col(X, F, stream=s)
    want = call(None)
    q = cb.empty_rows_i8(4096, 4096).fill_(1)
    one, y = torch.ones(4096, device="cuda"), torch.empty(4096, 4096, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in streams:
            for _ in range(8):   # about half a millisecond ahead of the call
                cb.pointwise_i8_fwd(q, one, q, one, y=y, stream=streams[0])
            got.append(call(s))
            fill = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(85) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        del fill
    assert cb.conv_device_status() == cb.CONV_OK
