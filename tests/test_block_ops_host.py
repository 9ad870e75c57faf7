"""What the binding does on the host around the calls of the operators, checked
without a GPU: the library and torch's streams are stood in for."""
import contextlib
import importlib.util

import pytest
import torch

from retentive_network_scale_b200 import retention as R


class FakeLibrary:
    """Every entry point succeeds, every size is `need` bytes."""

    def __init__(self, need=64):
        self.need, self.calls = need, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return self.need if name.endswith("_size") else 0
        return call


class Made(list):
    recorded = 0


@pytest.fixture
def streams(monkeypatch):
    """Stands in for torch's streams; returns the (stream, bytes) of each allocation
    (the stream being None for the current one).  Blocks that wait for the current
    stream's work when they are let go of are counted in `recorded`."""
    inside, made, empty = [None], Made(), torch.empty

    class Stream:
        def __init__(self, handle=0, device=None):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def use(stream):
        inside.append(stream)
        yield
        inside.pop()

    def allocate(*shape, **kw):
        kw["device"] = "cpu"
        t = empty(*shape, **kw)
        made.append((inside[-1], t.numel() * t.element_size()))
        return t

    def record(t, stream):
        assert stream == "current"
        made.recorded += 1

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(R, "load_library", lambda *a: FakeLibrary())
    monkeypatch.setattr(R, "_device_of", lambda t, name: 0)
    monkeypatch.setattr(R, "_rows", lambda t, name, shape, dtype, device: (0x1000, shape[-1]))
    monkeypatch.setattr(R, "_on_stream", lambda stream, device: 0)
    return made


def test_quantize_w4_makes_its_results_on_its_stream(streams):
    W = torch.zeros(128, 8)
    side = torch.cuda.Stream(0x40)
    R.ret_quantize_w4(W, 64, zeros=True, stream=side)
    assert [s for s, _ in streams] == [side] * 3 and streams.recorded == 3
    streams.clear()
    R.ret_quantize_w4(W, 64, zeros=True, stream=0x80)           # a raw handle
    assert [s.cuda_stream for s, _ in streams] == [0x80] * 3
    streams.clear()
    R.ret_quantize_w4(W, 64)
    assert streams == [(None, 8 * 64), (None, 8 * 2 * 2)]


def test_workspaces_and_results_of_every_call_are_made_on_its_stream(streams, monkeypatch):
    """The kernels of a call on `stream` use them after the call has returned and
    let go of them."""
    monkeypatch.setattr(R, "_dev", lambda t, *a, **k: t)
    B, H, L, dk, dv, chunk, gamma = 1, 2, 8, 4, 4, 4, [0.9, 0.8]
    q, v = torch.zeros(B, H, L, dk), torch.zeros(B, H, L, dv)
    b, bv, G = q.bfloat16(), v.bfloat16(), torch.zeros(B, L, H * dv)
    x, w = torch.zeros(B, L, 8).bfloat16(), torch.zeros(8, H * (2 * dk + 2 * dv)).bfloat16()
    w_o, U = torch.zeros(H * dv, 8).bfloat16(), torch.zeros(2, B, H, dk, dv)
    # allocations of a call, and how many of them it returns
    calls = [
        (1, 0, lambda s: R.ret_parallel(q, q, v, v, gamma, stream=s)),
        (1, 0, lambda s: R.ret_chunkwise(q, q, v, gamma, chunk, O=v, stream=s)),
        (1, 0, lambda s: R.ret_chunkwise_host(q, q, v, gamma, chunk, O=v, stream=s)),
        (2, 1, lambda s: R.ret_msr_layer(x, w, w_o, gamma, chunk, dk, dv, stream=s)),
        (4, 3, lambda s: R.ret_backward(b, b, bv, bv, gamma, chunk, stream=s)),
        (2, 1, lambda s: R.ret_segment_state(b, bv, gamma, stream=s)),
        (1, 1, lambda s: R.ret_state_scan(U, [4, 4], 1, gamma, stream=s)),
        (2, 1, lambda s: R.ret_chunkwise_segmented(b, b, bv, gamma, chunk, 2, stream=s)),
    ]
    monkeypatch.setattr(R, "_stream", lambda s: R.ctypes.c_void_p(0))
    side = torch.cuda.Stream(0x40)
    for n, returned, call in calls:
        for stream in (side, None):
            streams.clear()
            streams.recorded = 0
            call(stream)
            assert [s for s, _ in streams] == [stream] * n
            assert streams.recorded == (returned if stream else 0)


def test_binding_imports_on_a_torch_without_cuda(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("retention_without_cuda", R.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    with pytest.raises(TypeError):
        module.ret_rms_norm(torch.zeros(2, 8), torch.zeros(2, 8))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: type("S", (), dict(cuda_stream=7)))
    assert module._on_stream(None, 0) == 7


def block_calls():
    """A valid call of each operator, as (function, arguments by name); host
    tensors."""
    z, bf, i8 = torch.zeros, torch.bfloat16, torch.int8
    x = z(2, 8, 64)
    return [
        (R.ret_rms_norm, dict(X=x, Y=z(2, 8, 64, dtype=i8), weight=z(64), residual=x.to(bf),
                              residual_out=x.to(bf), scales=z(2, 8, 2))),
        (R.ret_causal_conv, dict(X=x, weight=z(64, 4), Y=z(2, 8, 64), bias=z(64), lengths=z(2, dtype=torch.int32),
                                 state_in=z(2, 3, 64), state_out=z(2, 3, 64))),
        (R.ret_selective_scan, dict(U=x, delta=x, A=z(64, 16), Bm=z(2, 8, 2, 16), Cm=z(2, 8, 2, 16), Y=z(2, 8, 64),
                                    skip=z(64), Z=x, delta_bias=z(64), lengths=z(2, dtype=torch.int32),
                                    state_in=z(2, 64, 16), state_out=z(2, 64, 16))),
        (R.ret_matvec_w4, dict(X=z(3, 64, dtype=i8), Wq=z(8, 32, dtype=torch.uint8), scales=z(8, 2, dtype=bf),
                               Y=z(3, 8), zeros=z(8, 2, dtype=torch.uint8), x_scales=z(3, 1))),
        (R.ret_quantize_w4, dict(W=z(64, 8), group=32)),
    ]


@pytest.mark.parametrize("fn,args", block_calls(), ids=lambda v: getattr(v, "__name__", ""))
def test_block_calls_refuse_what_is_not_a_tensor_of_the_shape(monkeypatch, fn, args):
    lib = FakeLibrary()
    monkeypatch.setattr(R, "load_library", lambda *a: lib)
    monkeypatch.setattr(R, "_device_of", lambda t, name: -1)    # the host's number
    monkeypatch.setattr(R, "_on_stream", lambda stream, device: 0)
    fn(**args)
    assert lib.calls == [fn.__name__]
    for name, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        if name not in ("X", "U", "W"):         # those are looked at by _device_of
            for wrong in (t.numpy() if t.dtype != torch.bfloat16 else t.float().numpy(), t.tolist(), 1.0):
                with pytest.raises(TypeError):
                    fn(**dict(args, **{name: wrong}))
        for wrong in (t[..., 0] if name != "Bm" else t[..., 0, 0], t[..., None] if t.dim() < 4 else t[..., None, None],
                      torch.zeros((), dtype=t.dtype)):
            with pytest.raises(ValueError):
                fn(**dict(args, **{name: wrong}))
        if name != "W":
            with pytest.raises(TypeError):
                fn(**dict(args, **{name: t.to(torch.float64)}))
    assert lib.calls == [fn.__name__]


def test_extents_that_would_overflow_an_int_are_refused():
    """(In every machine's build: refused before any CUDA call.)"""
    from retentive_network_scale_b200 import build
    build.build()
    lib = R.load_library()
    shape, fake, limit = R.STATUS_NAMES.index("RET_ERR_SHAPE"), 0x10000, R.RET_MAX_EXTENT

    def conv(L, D):
        return lib.ret_causal_conv(1, L, D, 4, R.RET_BF16, fake, D, fake, None, 1, None, None, None, fake, None)

    def scan(L, D):
        d = R.RetScanDesc(1, L, D, 4, 1, R.RET_BF16, 1, D, D, D, 4, 4)
        return lib.ret_selective_scan(d, fake, fake, None, fake, fake, fake, None, None, None, None, None, fake, None)

    for call in (conv, scan):
        for big in (limit + 1, 2 ** 31 - 127, 2 ** 31 - 1):
            assert call(big, 1) == shape and call(1, big) == shape
    if not torch.cuda.is_available():           # valid but for the machine
        unsupported = R.STATUS_NAMES.index("RET_ERR_UNSUPPORTED")
        assert conv(limit, 1) == conv(1, limit) == scan(limit, 1) == scan(1, limit) == unsupported


def test_sizes_past_an_int_are_refused_by_the_binding(monkeypatch):
    """2^32 + 64 would arrive in the library as 64."""
    lib = FakeLibrary()
    monkeypatch.setattr(R, "load_library", lambda *a: lib)
    monkeypatch.setattr(R, "_device_of", lambda t, name: -1)
    monkeypatch.setattr(R, "_on_stream", lambda stream, device: 0)
    big = 2 ** 32 + 64
    e = lambda *shape, dtype=torch.float32: torch.empty(*shape, device="meta", dtype=dtype)  # noqa: E731
    u8, bf = torch.uint8, torch.bfloat16
    for call in (lambda: R.ret_rms_norm(e(2, big), e(2, big)),
                 lambda: R.ret_causal_conv(e(1, big, 1), e(1, 4), e(1, big, 1)),
                 lambda: R.ret_causal_conv(e(1, 1, big), e(big, 4), e(1, 1, big)),
                 lambda: R.ret_selective_scan(*[e(1, big, 1)] * 2, e(1, 1), *[e(1, big, 1)] * 3),
                 lambda: R.ret_matvec_w4(e(1, big), e(1, big // 2, dtype=u8), e(1, big // 64, dtype=bf), e(1, 1)),
                 lambda: R.ret_matvec_w4(e(1, 64), e(big, 32, dtype=u8), e(big, 1, dtype=bf), e(1, big)),
                 lambda: R.ret_quantize_w4(e(64, 8), big)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert lib.calls == []
