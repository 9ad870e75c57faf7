"""The operators around the mixers on the GPU at the ends of their ranges: tiny and
non-finite rows, layouts and lengths that take every form of each kernel, streams
that are not the current one.  References and bounds as in block_ref."""
import math

import pytest
import torch

import block_ref as ref
from retentive_network_scale_b200 import retention as R
from retentive_network_scale_b200.synth import random_tensor

pytestmark = pytest.mark.gpu
F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from retentive_network_scale_b200 import build
    build.build()
    R.load_library()
    yield
    torch.cuda.synchronize()
    assert R.ret_last_device_status() == 0


def rt(shape, seed, scale=1.0, dtype=F32):
    return random_tensor(shape, seed, scale).to(dtype)


# ------------------------------------------------------------------------ norm
def check_codes(y, sc, want, g):
    """Codes and scales of the fp64 rows `want`: the scale within the norm's
    bound, a value within half a step of its code.  4 NORM: the code is taken of a
    value and with a scale that are each off."""
    rows, d = want.shape
    top = 127.0 if y.dtype == I8 else 448.0
    scale = want.view(rows, d // g, g).abs().amax(-1) / top
    assert ref.within(sc, scale, ref.NORM * scale) <= 1
    got = (y.float().cpu().double().view(rows, d // g, g) * sc.cpu().double()[..., None]).view(rows, d)
    step = scale.repeat_interleave(g, 1)
    half = 0.5 * step if y.dtype == I8 else torch.maximum(want.abs() * 2.0 ** -4, step * 2.0 ** -10)
    assert ref.within(got, want, half + 4 * ref.NORM * (want.abs() + step)) <= 1


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("yt", [I8, E4M3])
@pytest.mark.parametrize("xs,ws,eps", [(None, 1.0, 1e-6), (1e-10, 1e-27, 0.0), (1e-16, 1.0, 1e-30),
                                       (1e12, 1e-20, 1e-5)])
def test_rms_norm_codes_of_tiny_values(group, yt, xs, ws, eps):
    """The factor between s and its code leaves fp32's range where neither does.
    (w s may be subnormal: off by 2^-150, which times 1 / rms is under 1e-6 of the
    step here.)"""
    rows, d = 3, 96
    if xs is None:                                      # scales of 2.2e-36, above the least one of 2^-119
        xs = 2.2e-36 * (127 if yt == I8 else 448) / 1.5 * eps ** 0.5
    x, w = rt((rows, d), 1).clamp(-1, 1) * xs, 1 + rt((d,), 2, 0.2).clamp(-0.5, 0.5)
    x[:, ::32] = xs                                     # every group's largest value
    x[1, 5] = 0.0
    w[::32] = 1.5
    w = w * ws
    y = torch.full((rows, d), 1.0, device="cuda").to(yt)
    sc = torch.full((rows, d // (group or d)), -1.0, device="cuda")
    R.ret_rms_norm(x.cuda(), y, weight=w.cuda(), scales=sc, eps=eps)
    _, want = ref.rms_norm(x, w, None, eps)
    check_codes(y, sc, want, group or d)
    assert float(y[1, 5].float()) == 0.0


@pytest.mark.parametrize("d,group", [(256, 64), (256, 0), (100, 0), (1056, 32)])
@pytest.mark.parametrize("yt", [I8, E4M3])
def test_rms_norm_codes_are_zero_where_the_scale_is_nan(d, group, yt):
    x = rt((6, d), 3)
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    x[3] = 0.0
    r = torch.zeros(6, d)
    r[4, 7] = float("nan")
    for eps in (1e-5, 0.0):
        y = torch.full((6, d), 1.0, device="cuda").to(yt)
        sc = torch.zeros(6, d // (group or d), device="cuda")
        R.ret_rms_norm(x.cuda(), y, residual=r.cuda(), scales=sc, eps=eps)
        s, code = sc.cpu(), y.float().cpu().view(6, sc.shape[1], -1)
        assert bool(torch.isnan(s[[1, 4]]).all())               # the sum of squares is NaN
        assert bool(torch.isnan(s[2, 40 // (group or d)]))      # infinity over an infinite norm
        assert bool(torch.isnan(s[3]).all()) == (eps == 0.0)    # 0 / 0
        assert bool(torch.isfinite(s[[0, 5]]).all())
        dead = torch.isnan(s) | (s == 0)
        assert bool((code[dead] == 0).all()) and not bool(torch.isnan(code).any())
        assert bool((code[[0, 5]].abs().amax(-1) > 0).all())


@pytest.mark.parametrize("yt", [I8, E4M3])
def test_rms_norm_least_scale(yt):
    """A scale below 2^-119 is 0, with codes 0; one above is kept."""
    d, top = 64, 127.0 if yt == I8 else 448.0
    limit = 2.0 ** -119
    x = torch.zeros(4, d)
    # eps = 1 gives y = s; 2^-20 is far above the norm's bound
    for row, f in enumerate((0.81, 1 - 2.0 ** -20, 1 + 2.0 ** -20, 1.2)):
        x[row, ::3] = limit * top * f
    y, sc = torch.full((4, d), 1.0, device="cuda").to(yt), torch.full((4, 1), -1.0, device="cuda")
    R.ret_rms_norm(x.cuda(), y, scales=sc, eps=1.0)
    codes, s = y.float().cpu(), sc.cpu()[:, 0]
    assert s[:2].tolist() == [0.0, 0.0] and bool((codes[:2] == 0).all())
    assert bool((s[2:] >= limit).all()) and bool((codes[2:, ::3] == top).all())
    assert ref.within(s[2:], x[2:, 0].double() / top, ref.NORM * x[2:, 0].double() / top) <= 1


# ------------------------------------------------------------------------ convolution, scan
def test_scan_segment_that_grows_past_fp32():
    """One segment multiplies the state by 2^140 to 2^270 (which fp32 does not
    hold), the state itself staying inside fp32; a zero state stays zero."""
    B, L, D, N = 1, 1100, 8, 16
    for grown, s0 in ((140.0, 2.0 ** -60), (200.0, -2.0 ** -100), (270.0, 2.0 ** -145), (140.0, 0.0)):
        u = torch.zeros(B, L, D)
        delta = torch.zeros(B, L, D)
        # all growth in the second of the 16 segments of 80 rows
        delta[:, 80:160] = grown / 80 * 0.6931471805599453 / 0.25
        A = torch.full((D, N), 0.25)
        bm, cm = torch.ones(B, L, 1, N), torch.ones(B, L, 1, N)
        state = torch.full((B, D, N), s0)
        y, out = torch.empty(B, L, D, device="cuda"), torch.empty(B, D, N, device="cuda")
        R.ret_selective_scan(u.cuda(), delta.cuda(), A.cuda(), bm.cuda(), cm.cuda(), y, softplus=False,
                             state_in=state.cuda(), state_out=out)
        want, last, tol, stol = ref.selective_scan(u, delta, A, bm, cm, softplus=False, state=state)
        # The bound counts roundings of normal numbers.  A subnormal state is rounded
        # to 2^-149 in every row, off by up to 2^-150, which the rows after it grow:
        # E_t = a_t E_{t-1} + 2^-150 more (2^-145 grown 2^3.4 a row ends up 3% off).
        E, sub = 0.0, torch.zeros(1, L, 1, dtype=torch.float64)
        for t in range(L):
            E = math.exp(float(delta[0, t, 0]) * 0.25) * E + (2.0 ** -150 if s0 else 0.0)
            sub[0, t] = E
        assert ref.within(out, last, stol + E) <= 1
        tol = tol + N * sub
        # (16 states of 2^125 add up to more than fp32 holds: the y that belongs there)
        past = want.abs() > torch.finfo(F32).max
        assert bool((y.cpu()[past] == want[past].sign().float() * float("inf")).all())
        got, want = torch.where(past, 0.0, y.cpu().double()), torch.where(past, 0.0, want)
        assert ref.within(got, want, tol + ref.rounded(want, F32) + 2.0 ** -149) <= 1


def test_conv_and_scan_of_the_most_rows():
    """One channel; its last rows are checked (of the scan, which would take tens of
    seconds, a short sequence in a padded batch of that many rows)."""
    L = R.RET_MAX_EXTENT
    x = torch.zeros(1, L, 1, device="cuda", dtype=BF16)
    tail, w = rt((1, 300, 1), 31, 1.0, BF16), rt((1, 2), 32)
    x[:, -300:] = tail.cuda()
    x[:, :300] = tail.cuda()
    y, end = torch.zeros_like(x), torch.empty(1, 1, 1, device="cuda", dtype=BF16)
    R.ret_causal_conv(x, w.cuda(), y, state_out=end)
    want, last, tol = ref.causal_conv(tail, w)
    assert ref.within(y[:, -300:], want, tol + ref.rounded(want, BF16)) <= 1
    assert torch.equal(end.cpu().double(), last)
    y.fill_(5.0)
    A, n = torch.full((1, 1), -0.5), torch.tensor([300], dtype=torch.int32)
    R.ret_selective_scan(x, x, A.cuda(), x, x, y, lengths=n.cuda())
    tail4 = tail[..., None]
    want, _, tol, _ = ref.selective_scan(tail, tail, A, tail4, tail4)
    assert ref.within(y[:, :300], want, tol + ref.rounded(want, BF16)) <= 1
    assert bool((y[0, 300:1000] == 5.0).all()) and bool((y[0, -1000:] == 5.0).all())


def test_conv_of_the_most_channels_a_call_takes():
    """Rows so wide that the last threads' channels lie past 2^31 unless cut."""
    D = R.RET_MAX_EXTENT - 2                    # two channels a thread
    x = torch.zeros(1, 1, D, device="cuda", dtype=BF16)
    x[0, 0, -256:] = rt((256,), 33, 1.0, BF16).cuda()
    w = torch.zeros(D, 2, device="cuda")
    w[:, 1] = 2.0
    y = torch.full_like(x, 5.0)
    R.ret_causal_conv(x, w, y, swish=False)
    assert torch.equal(y[0, 0, -256:], 2 * x[0, 0, -256:]) and bool((y[0, 0, :4096] == 0).all())


def test_scan_token_of_more_channels_than_its_threads_count():
    """Two threads a channel, whose number passes 2^31: taken by the tiles."""
    D, N, n = 2 ** 30 + 40, 5, 200
    c = {k: rt((1, 1, n), 34 + i, 1.0, BF16) for i, k in enumerate("ud")}
    A, bm = -rt((n, N), 36).abs(), rt((1, 1, 1, N), 37, 1.0, BF16)
    u, d = (torch.zeros(1, 1, D, device="cuda", dtype=BF16) for _ in range(2))
    wide = torch.zeros(D, N, device="cuda")
    u[..., -n:], d[..., -n:], wide[-n:] = c["u"].cuda(), c["d"].cuda(), A.cuda()
    y = torch.full_like(u, 5.0)
    R.ret_selective_scan(u, d, wide, bm.cuda(), bm.cuda(), y)
    want, _, tol, _ = ref.selective_scan(c["u"], c["d"], A, bm, bm)
    assert ref.within(y[..., -n:], want, tol + ref.rounded(want, BF16)) <= 1
    assert bool((y[..., :-n] == 0).all())


# ------------------------------------------------------------------------ 4-bit product
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 5, 10, 22, 64])
def test_matvec_w4_products_of_fp32_rows_are_exact(M, g):
    """Weights that pick one column each (+-1 there, times a power of two): y is x,
    bit for bit, up to the largest finite value."""
    K = 2 * g
    gen = torch.Generator().manual_seed(21)
    # all 24 bits, exponents from 2^-100 on
    x = torch.randint(1 << 23, 1 << 24, (M, K), generator=gen).double()
    x = torch.ldexp(x, torch.randint(-123, 104, (M, K), generator=gen))
    x[torch.rand(M, K, generator=gen) < 0.5] *= -1
    x[:, 3], x[:, 4] = torch.finfo(F32).max, -3.395e38
    x[:, 5] = 0.0
    x = x.float()
    sign = torch.where(torch.arange(K) % 3 == 0, -1, 1)
    q = torch.full((K, K), 8) + torch.diag(sign)
    wq = (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)
    for scale in (1.0, 2.0 ** -12):
        s = torch.full((K, 2), scale, dtype=BF16)
        y = torch.full((M, K), 7.0, device="cuda")
        R.ret_matvec_w4(x.cuda(), wq.cuda(), s.cuda(), y)
        assert torch.equal(y.cpu(), x * sign * scale)


def test_matvec_w4_keeps_infinities_and_every_nan():
    x = torch.ones(4, 64)
    x[0, 7], x[1, 7] = float("inf"), float("-inf")
    x[2:, 7] = torch.tensor([0x7f800001, -0x7fffff], dtype=torch.int32).view(F32)   # NaNs with low bits only
    wq = torch.full((8, 32), 0x99, dtype=torch.uint8)           # weights of 1
    y = torch.empty(4, 8, device="cuda")
    R.ret_matvec_w4(x.cuda(), wq.cuda(), torch.ones(8, 1, dtype=BF16).cuda(), y)
    y = y.cpu()
    assert bool((y[0] == float("inf")).all()) and bool((y[1] == float("-inf")).all())
    assert bool(torch.isnan(y[2:]).all())


def test_matvec_w4_with_the_most_columns_an_int_holds():
    """The last piece of x ends where an int does.  Everything but the first and
    the last columns is zero."""
    K, N, g = 2 ** 31 - 128, 2, 128
    gen = torch.Generator().manual_seed(22)
    ends = torch.randint(-127, 128, (1, 512), generator=gen, dtype=torch.int8)
    x = torch.zeros(1, K, device="cuda", dtype=I8)
    x[:, :256], x[:, -256:] = ends[:, :256].cuda(), ends[:, 256:].cuda()
    codes = torch.randint(0, 256, (N, 256), generator=gen, dtype=torch.uint8)
    wq = torch.zeros(N, K // 2, device="cuda", dtype=torch.uint8)
    wq[:, :128], wq[:, -128:] = codes[:, :128].cuda(), codes[:, 128:].cuda()
    s = torch.ones(N, K // g, device="cuda", dtype=BF16)
    y, xs = torch.empty(1, N, device="cuda"), torch.full((1, 1), 0.5, device="cuda")
    R.ret_matvec_w4(x, wq, s, y, x_scales=xs)
    want, _ = ref.matvec_w4(ends.float(), codes, torch.ones(N, 4, dtype=BF16))
    assert torch.equal(y.cpu().double(), want * 0.5)            # whole numbers below 2^24


def check_quantized(W, g, zeros):
    """Scales as the definition's (in fp32, rounded to bf16), codes and zero points
    exactly the nearest, ties to even, for those scales."""
    K, N = W.shape
    wq, s, z = (t if t is None else t.cpu() for t in R.ret_quantize_w4(W.cuda(), g, zeros=zeros))
    t = W.double().view(K // g, g, N)
    lo, hi = t.amin(1).clamp(max=0), t.amax(1).clamp(min=0)
    # (the range is rounded to fp32 before its division, as halves)
    scale = ((hi - lo) / 2).float() / 7.5 if zeros else torch.maximum(hi, -lo).float() / 7
    assert torch.equal(s, scale.to(BF16).t())
    d = s.double().t()
    per = lambda v: torch.where(d > 0, v / torch.where(d > 0, d, 1.0), 0.0).round()  # noqa: E731
    zp = per(-lo).clamp(0, 15) if zeros else torch.full_like(lo, 8.0)
    if zeros:
        assert torch.equal(z.double().t(), zp)
    steps = torch.where(d[:, None] > 0, t / torch.where(d > 0, d, 1.0)[:, None], 0.0).round()
    want = (steps + zp[:, None]).clamp(0, 15).view(K, N).t()
    got = torch.stack([wq & 15, wq >> 4], -1).view(N, K).double()
    assert torch.equal(got, want)


@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-37, 3e-39, 1e-40, 1e37, 8e37])
def test_quantize_w4_rounds_to_the_nearest_at_every_size(wt, zeros, size):
    K, N, g = 256, 96, 64
    W = (rt((K, N), 41).clamp(-4, 4) * size).to(wt)
    W[::7] = 0.0
    W[:g, 5] = 0.0
    check_quantized(W, g, zeros)


def test_quantize_w4_ties_go_to_even():
    """w = (k + 1/2) scale, for every mantissa of a bf16 scale."""
    scale = torch.arange(128, 256).float() / 1024                       # one column each
    steps = torch.cat([torch.tensor([7.0]), torch.arange(-7, 7) + 0.5, torch.zeros(17)])
    check_quantized(steps[:, None] * scale[None], 32, False)
    steps = torch.cat([torch.tensor([8.0, -7.0]), torch.arange(-7, 8) + 0.5, torch.zeros(15)])
    check_quantized(steps[:, None] * scale[None], 32, True)


# ------------------------------------------------------------------------ streams
def busy_then_freed(shapes):
    """Blocks of these (shape, dtype) that the allocator holds for the current
    stream, where work that writes them is still to come."""
    torch.cuda.synchronize()
    held = [torch.empty(shape, device="cuda", dtype=dtype) for shape, dtype in shapes]
    torch.cuda._sleep(int(5e7))                         # some 25 ms
    for t in held:
        t.fill_(3)


@pytest.mark.parametrize("raw", [False, True])
def test_quantize_w4_on_another_stream(raw):
    K, N, g = 1024, 2048, 64
    W = rt((K, N), 11).cuda()
    want = R.ret_quantize_w4(W, g, zeros=True)
    side = torch.cuda.Stream()
    busy_then_freed([(t.shape, t.dtype) for t in want])
    got = R.ret_quantize_w4(W, g, zeros=True, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    if raw:     # the default stream's handles
        for handle in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(want, R.ret_quantize_w4(W, g, True, stream=handle)))


@pytest.mark.parametrize("raw", [False, True])
def test_calls_with_workspaces_on_another_stream(raw):
    """A workspace or result that the call makes is neither taken from nor given
    back to the current stream while the call's kernels run elsewhere."""
    B, H, L, dk, dv, chunk, gamma = 2, 4, 512, 128, 128, 64, [0.95, 0.97, 0.98, 0.99]
    q, k = (rt((B, H, L, dk), s, dk ** -0.5, BF16).cuda() for s in (12, 13))
    v, do = (rt((B, H, L, dv), s, 1.0, BF16).cuda() for s in (14, 15))
    a, b = rt((512, 256), 16, 1.0, BF16).cuda(), rt((256, 512), 17, 1.0, BF16).cuda()
    o = torch.empty_like(v)
    calls = [lambda s: R.ret_parallel(q, k, v, o, gamma, stream=s),
             lambda s: R.ret_chunkwise(q, k, v, gamma, chunk, O=o, stream=s)[0],
             lambda s: R.ret_backward(q, k, v, do, gamma, chunk, stream=s),
             lambda s: R.ret_segment_state(k, v, gamma, stream=s),
             lambda s: R.ret_chunkwise_segmented(q, k, v, gamma, chunk, 4, stream=s)[0],
             lambda s: R.ret_gemm_bf16(a, b, stream=s)]
    side = torch.cuda.Stream()
    for call in calls:
        whole = lambda t: [x.clone() for x in (t if isinstance(t, tuple) else (t,))]  # noqa: E731
        want = whole(call(None))
        torch.cuda.synchronize()
        o.zero_()
        busy_then_freed([(t.shape, t.dtype) for t in want])
        with torch.cuda.stream(side):
            torch.cuda._sleep(int(5e7))
        got = call(side.cuda_stream if raw else side)
        # what the call has let go of must not come back here before it is done
        blocks = [torch.full((n,), 255, device="cuda", dtype=torch.uint8) for n in (1 << 14, 1 << 18, 1 << 20, 1 << 22, 1 << 24)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, whole(got)))
        del blocks


def test_result_of_another_stream_let_go_of_early():
    """The caller's stream reads a result that was made on another one, and the
    next call there may not have its memory before that."""
    W, W2 = rt((1024, 2048), 18).cuda(), rt((1024, 2048), 19).cuda()
    want = R.ret_quantize_w4(W, 64)[0].clone()
    a, b = rt((512, 256), 20, 1.0, BF16).cuda(), rt((256, 512), 21, 1.0, BF16).cuda()
    product = R.ret_gemm_bf16(a, b).clone()
    side, zero = torch.cuda.Stream(), torch.zeros_like(a)
    torch.cuda.synchronize()
    for raw in (False, True):
        stream = side.cuda_stream if raw else side
        codes, c = R.ret_quantize_w4(W, 64, stream=stream)[0], R.ret_gemm_bf16(a, b, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(int(5e7))
        got, c2 = codes.clone(), c.clone()
        del codes, c
        R.ret_quantize_w4(W2, 64, stream=stream)
        R.ret_gemm_bf16(zero, b, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(c2, product)


def test_calls_that_allocate_captured_on_two_streams():
    """A graph of calls on the capturing stream and on one that joins it."""
    W = rt((512, 256), 22).cuda()
    b = rt((256, 512), 23, 1.0, BF16).cuda()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = R.ret_quantize_w4(W, 64, zeros=True), R.ret_gemm_bf16(W.to(BF16), b)
    x, y = torch.zeros_like(W), torch.zeros_like(W.to(BF16))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        q = R.ret_quantize_w4(x, 64, zeros=True, stream=side)
        R.ret_quantize_w4(x, 32, stream=side)                   # let go of at once
        c = R.ret_gemm_bf16(y, b, stream=here)
        here.wait_stream(side)
    x.copy_(W)
    y.copy_(W)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(q, want[0])) and torch.equal(c, want[1])
