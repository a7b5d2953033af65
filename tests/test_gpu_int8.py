"""Row quantisation and int8 products through gpt2k_quantize_rows and gpt2k_matmul_i8,
against numpy in 64 bits.

Codes and scales are whole numbers and one rounding each: they are compared for
equality. The integer sums are exact, so a result differs from the 64-bit one by its
own roundings only: with u = acc sa sb, three of half a step (2^-24 each) on u, one on
the sum with the bias, one on the sum with the residual; then the rounding to the
result's type (fp32: none more; bf16: 2^-8). GELU (slope at most 1.13) passes u's error
on and adds its own: tanhf and the logistic form are within a few steps of fp32, at
most 2^-21 of |u| (bf16 results: 2^-18, ex2.approx of an argument up to 2^5), and for
u < 0 the value is a difference, hence |u| and not |gelu(u)|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _codes64(x):
    """127 x / a to the nearest whole number, ties to even, and a / 127 in fp32."""
    x = x.astype(np.float64)
    a = np.max(np.abs(x), axis=1)
    fine = np.isfinite(a)
    live = (fine & (a > 0))[:, None]
    with np.errstate(all="ignore"):
        q = np.where(live, np.rint(127.0 * x / a[:, None]), 0.0)
        scale = np.where(fine, a.astype(np.float32) / np.float32(127.0), np.float32(np.nan))
    return q.astype(np.int8), scale


def _quantize_inputs(rows, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)).astype(np.float32)
    for r in range(rows):
        kind = r % 10
        if kind == 1:
            x[r] = 0.0
        elif kind == 2:
            x[r] *= np.float32(1e-41)                       # subnormal
        elif kind == 3:
            x[r] *= np.float32(3e37)
        elif kind == 4:
            x[r] = rng.integers(-127, 127, K) * 2 + 1       # ties: a = 254 below
            x[r, 0] = 254.0
        elif kind == 5:
            x[r, K // 2] = np.nan
        elif kind == 6:
            x[r, K - 1] = -np.inf
        elif kind == 7:
            x[r, ::2] = -0.0
        elif kind == 8:
            x[r] = -x[r, 0]                                 # every value the largest
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 768), (11, 17), (30, 64), (23, 100), (13, 1600), (12, 2049),
                                    (10, 6400), (11, 8192), (10, 20011), (1030, 1024)])
@pytest.mark.parametrize("pad_x,pad_q,shift", [(0, 0, 0), (1, 3, 0), (8, 16, 8), (3, 5, 1)])
def test_quantize_rows(dtype, rows, K, pad_x, pad_q, shift):
    from decoder_only_transformer_sm_b200 import native
    x = _quantize_inputs(rows, K, dtype, rows * 31 + K)
    hold = torch.zeros(rows * (K + pad_x) + shift, dtype=dtype, device="cuda")
    dx = hold[shift:].view(rows, K + pad_x)[:, :K]
    dx.copy_(x)
    room = torch.full((rows * (K + pad_q) + shift,), 77, dtype=torch.int8, device="cuda")
    whole = room[shift:].view(rows, K + pad_q)
    scale = torch.full((rows + 1,), 5.0, device="cuda")
    native.quantize_rows(dx, whole[:, :K], scale[:rows])
    want_q, want_s = _codes64(x.float().numpy())
    np.testing.assert_array_equal(scale[:rows].cpu().numpy(), want_s)
    np.testing.assert_array_equal(whole[:, :K].cpu().numpy(), want_q)
    assert torch.all(whole[:, K:] == 77) and torch.all(room[:shift] == 77) and scale[rows] == 5.0


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -90, 2.0 ** 120, 2.0 ** -110])
def test_codes_at_borders(scale):
    """bf16: every significand of a row's largest value against every one of its elements over nine binades (with all
    their ties). fp32: the numbers next to (2 k + 1) a / 254 on both sides, for many a."""
    from decoder_only_transformer_sm_b200 import native
    tops = (np.arange(128, 256) * 2.0 ** -7 * scale)[:, None]
    x = (np.arange(128, 256)[:, None] * 2.0 ** (-7.0 - np.arange(9))).reshape(1, -1) * scale
    x = np.where(x <= tops, x, 0.0)
    rows = [np.concatenate([tops, x, -x], 1)]
    rng = np.random.default_rng(1)
    a = (rng.uniform(1.0, 2.0, 200) * scale).astype(np.float32)
    near = ((2 * np.arange(127) + 1)[None, :] * a.astype(np.float64)[:, None] / 254.0).astype(np.float32)
    up, down = np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(0))
    rows.append(np.concatenate([a[:, None], near, -near, up, -up, down, -down], 1).clip(-a[:, None], a[:, None]))
    for v, dtype in zip(rows, (torch.bfloat16, torch.float32)):
        dx = torch.from_numpy(v.astype(np.float32)).to(dtype).cuda()
        assert np.array_equal(dx.float().cpu().numpy(), v.astype(np.float32))
        R, K = dx.shape
        for pad in (0, -K % 16 + 16):
            q, s = torch.empty((R, K + pad), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
            x_in = torch.zeros((R, K + pad), dtype=dtype, device="cuda")[:, :K]
            x_in.copy_(dx)
            native.quantize_rows(x_in, q[:, :K], s)
            want_q, want_s = _codes64(v.astype(np.float32))
            np.testing.assert_array_equal(q[:, :K].cpu().numpy(), want_q)
            np.testing.assert_array_equal(s.cpu().numpy(), want_s)


def _gelu64(u):
    return 0.5 * u * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (u + 0.044715 * u ** 3)))


def _product(M, N, K, epilogue, out_dtype, pads=(0, 0, 0, 0), shift=(0, 0, 0), seed=0, extreme=False, in_place=False):
    """One product on fresh operands with guarded surroundings, checked against 64 bits."""
    from decoder_only_transformer_sm_b200 import native
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    low = -128 if extreme else -127
    A = np.full((M, K), -128) if extreme else rng.integers(low, 128, (M, K))
    B = np.full((N, K), -128) if extreme else rng.integers(low, 128, (N, K))
    if extreme and N > 1:
        B[1::2] = 127
    sa = rng.uniform(0.5, 2.0, M).astype(np.float32) * np.float32(0.02)
    sb = rng.uniform(0.5, 2.0, N).astype(np.float32) * np.float32(1e-3)
    bias = rng.standard_normal(N).astype(np.float32)
    resid = rng.standard_normal((M, N)).astype(np.float32)
    pa, pb, po, pr = pads

    def place(v, dtype, pad, at=0, fill=77):
        rows, cols = v.shape
        hold = torch.full((rows * (cols + pad) + at + 64,), fill, dtype=dtype, device="cuda")
        view = hold[at:at + rows * (cols + pad)].view(rows, cols + pad)
        view[:, :cols].copy_(torch.from_numpy(np.ascontiguousarray(v)).to(dtype))
        return hold, view

    _, a = place(A.astype(np.int8), torch.int8, pa, shift[0])
    _, b = place(B.astype(np.int8), torch.int8, pb, shift[1])
    hold, out = place(resid if in_place else np.zeros((M, N), np.float32), out_dtype, po, shift[2])
    dr = None
    if epilogue == "bias_resid":
        dr = out[:, :N] if in_place else place(resid, torch.float32, pr)[1][:, :N]
    dbias = torch.from_numpy(bias).cuda() if epilogue != "store" else None
    status = native.matmul_i8(a[:, :K], torch.from_numpy(sa).cuda(), b[:, :K], torch.from_numpy(sb).cuda(),
                              out[:, :N], epilogue=epilogue, bias=dbias, resid=dr)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    acc = A.astype(np.float64) @ B.astype(np.float64).T
    u = acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)
    err = 3 * 2.0 ** -24 * np.abs(u)
    want = u
    if epilogue != "store":
        want = u + bias
        err = err + 2.0 ** -24 * np.abs(want)
    if epilogue == "bias_gelu":
        v = want
        want = _gelu64(v)
        err = 1.13 * err + np.abs(v) * (2.0 ** -21 if out_dtype == torch.float32 else 2.0 ** -18)
    if epilogue == "bias_resid":
        want = want + resid
        err = err + 2.0 ** -24 * np.abs(want)
    if out_dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * np.abs(want) * 1.01
    got = out[:, :N].float().cpu().numpy().astype(np.float64)
    worst = np.max(np.abs(got - want) - err * 1.001)
    assert worst <= 1e-30, (worst, np.unravel_index(np.argmax(np.abs(got - want) - err), got.shape))
    # nothing around the result is touched
    left = hold.clone()
    left[shift[2]:shift[2] + M * (N + po)].view(M, N + po)[:, :N] = 77
    assert torch.all(left == 77)


SIZES = [(1, 1, 1), (1, 8, 16), (2, 100, 768), (3, 50, 31), (4, 1024, 128), (5, 77, 96), (8, 2304, 768), (8, 130, 1616),
         (9, 64, 64), (16, 8, 16), (17, 129, 144), (64, 256, 128), (127, 300, 272), (128, 128, 128), (129, 257, 160),
         (333, 1600, 1600), (256, 40, 4096), (700, 96, 32), (1, 5001, 2048), (7, 33, 5000),
         (640, 1920, 96), (1000, 2403, 144), (2305, 2310, 272)]   # more tiles than SMs at each tile width


@pytest.mark.parametrize("epilogue,out_dtype", [("store", torch.bfloat16), ("store", torch.float32),
                                                ("bias", torch.bfloat16), ("bias", torch.float32),
                                                ("bias_gelu", torch.bfloat16), ("bias_gelu", torch.float32),
                                                ("bias_resid", torch.float32)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_products(M, N, K, epilogue, out_dtype):
    """Rows of whole 16 bytes where K allows it, padded to them where it does not."""
    _product(M, N, K, epilogue, out_dtype, pads=(-K % 16, -K % 16, 0, 0))


@pytest.mark.parametrize("M,N,K", [(1, 40, 33), (3, 41, 768), (40, 70, 65), (130, 129, 257), (700, 2401, 99)])
@pytest.mark.parametrize("pads,shift", [((0, 0, 0, 0), (0, 0, 0)), ((1, 7, 3, 5), (0, 0, 0)),
                                        ((16, 32, 1, 2), (16, 32, 1)), ((0, 0, 8, 8), (3, 1, 8)),
                                        ((15, 0, 7, 1), (1, 0, 3)), ("whole", (16, 32, 0))])
def test_strides_and_starts(M, N, K, pads, shift):
    if pads == "whole":   # operands' rows of whole 16 bytes, the results' ending inside one; what pads them is not zero
        pads = (-K % 16, 16 + -K % 16, -N % 8, -N % 4)
    for epilogue, dtype in (("store", torch.bfloat16), ("bias_gelu", torch.bfloat16), ("bias_resid", torch.float32),
                            ("bias", torch.float32)):
        _product(M, N, K, epilogue, dtype, pads=pads, shift=shift)


@pytest.mark.parametrize("M", [1, 8, 9, 130])
@pytest.mark.parametrize("pad", [1, 0])
def test_largest_sums(M, pad):
    """Every code -128 against -128 and 127 at the largest K: the sums reach 2^31 - 2^14."""
    _product(M, 24, 131071, "store", torch.float32, pads=(pad, pad, 0, 0), extreme=True)


@pytest.mark.parametrize("M", [3, 20])
@pytest.mark.parametrize("odd", [0, 1])
def test_rows_far_apart(M, odd):
    """Offsets past 32 bits: rows of A, of the codes written and of the results lie over 2^31 bytes in all apart."""
    from decoder_only_transformer_sm_b200 import native
    K, N = 256, 40
    ld = (1 << 32) // M // 16 * 16 + 16 + odd
    hold = torch.empty((M - 1) * ld + K, dtype=torch.int8, device="cuda")
    q = hold.as_strided((M, K), (ld, 1))
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g)
    s = torch.empty(M, device="cuda")
    native.quantize_rows(x.cuda(), q, s)
    want_q, want_s = _codes64(x.numpy())
    assert torch.equal(q.cpu(), torch.from_numpy(want_q)) and torch.equal(s.cpu(), torch.from_numpy(want_s))
    b = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sb = torch.rand(N, generator=g).cuda()
    ldo = (1 << 31) // M // 4 * 4 + 4 + odd
    room = torch.empty((M - 1) * ldo + N, dtype=torch.bfloat16, device="cuda")
    out = room.as_strided((M, N), (ldo, 1))
    native.matmul_i8(q, s, b, sb, out)
    want = (q.double() @ b.double().t()) * s.double()[:, None] * sb.double()
    assert torch.all((out.double() - want).abs() <= (2.0 ** -8 * 1.01 + 4 * 2.0 ** -24) * want.abs())


@pytest.mark.parametrize("M,N,K", [(3, 64, 64), (150, 264, 320)])
def test_residual_in_place(M, N, K):
    _product(M, N, K, "bias_resid", torch.float32, in_place=True)


@pytest.mark.parametrize("M", [2, 40, 200])
def test_scales_that_are_nan_zero_or_tiny(M):
    """A quantised row that held a NaN has scale NaN: its results are NaN, its neighbours' are not. Scales whose
    product underflows still give the results that do not."""
    from decoder_only_transformer_sm_b200 import native
    N, K = 48, 64
    g = torch.Generator().manual_seed(M)
    a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    b = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sa, sb = torch.full((M,), 1e-20, device="cuda"), torch.full((N,), 1e-20, device="cuda")
    sa[0], sa[1] = float("nan"), 0.0
    out = torch.empty((M, N), device="cuda")
    native.matmul_i8(a, sa, b, sb, out)
    assert torch.all(torch.isnan(out[0])) and torch.all(out[1] == 0)
    if M > 2:
        want = (a[2:].double() @ b.double().t()) * sa[2:].double()[:, None] * sb.double()
        # results near 1e-37 may be subnormal: a step there is 2^-149
        assert torch.all((out[2:].double() - want).abs() <= 3 * 2.0 ** -24 * want.abs() + 2.0 ** -148)


def test_quantised_linear_layer_on_a_side_stream_and_in_a_graph():
    """quantize_rows and matmul_i8 as a layer: on another stream, and captured once and replayed on new inputs (two
    graphs interleaved), bit-equal to direct calls."""
    from decoder_only_transformer_sm_b200 import native
    M, N, K = 50, 400, 256
    g = torch.Generator().manual_seed(1)
    w = torch.randn((N, K), generator=g).cuda() * 0.02
    wq, ws = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    native.quantize_rows(w, wq, ws)
    bias = torch.randn(N, generator=g).cuda()

    class Layer:
        def __init__(self):
            self.x = torch.zeros((M, K), device="cuda", dtype=torch.bfloat16)
            self.q = torch.empty((M, K), dtype=torch.int8, device="cuda")
            self.s = torch.empty(M, device="cuda")
            self.out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def run(self, stream=None):
            native.quantize_rows(self.x, self.q, self.s, stream=stream)
            native.matmul_i8(self.q, self.s, wq, ws, self.out, epilogue="bias_gelu", bias=bias, status=self.status,
                             stream=stream)

    xs = [torch.randn((M, K), generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    want = []
    for x in xs:
        layer = Layer()
        layer.x.copy_(x)
        layer.run()
        want.append(layer.out.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer = Layer()
    layer.x.copy_(xs[0])
    side.wait_stream(torch.cuda.current_stream())
    layer.run(stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(layer.out, want[0])
    made = []
    for _ in range(2):
        layer, graph = Layer(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.run()
        made.append((layer, graph))
    for i in (0, 2):
        for j, (layer, graph) in enumerate(made):
            layer.x.copy_(xs[i + j])
            graph.replay()
        for j, (layer, _) in enumerate(made):
            assert torch.equal(layer.out, want[i + j])
    # the layer is near the unquantised one: each factor is off by at most half a code
    ref = torch.nn.functional.gelu(xs[0].double() @ w.double().t() + bias.double(), approximate="tanh")
    half = (xs[0].double().abs().amax(1, keepdim=True) / 254)
    bound = half * w.double().abs().sum(1) + (ws.double() / 2) * (xs[0].double().abs().sum(1, keepdim=True) + K * half)
    assert torch.all((want[0].double() - ref).abs() <= 1.13 * bound + 2.0 ** -7 * ref.abs() + 1e-4)


def test_pairs_of_blocks_one_product_after_another():
    """Products on pairs of blocks (256 x 256 tiles), each with the next one's blocks waiting for its SMs: a block of a
    pair stays until the other's last arrivals on its barriers. One K block, and more than the ring has stages."""
    from decoder_only_transformer_sm_b200 import native
    g = torch.Generator(device="cuda").manual_seed(0)
    for M, N, K in ((4096, 8192, 64), (4096, 4864, 784)):
        a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
        b = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
        sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(40):
            native.matmul_i8(a, sa, b, sb, outs[i % 4], status=status)
        assert int(status.item()) == 0
        want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
        for out in outs:   # three roundings of fp32, one of bf16
            assert torch.all((out.double() - want).abs() <= (2.0 ** -8 * 1.01 + 4 * 2.0 ** -24) * want.abs())


def _replay_time(call):
    """Shortest of twelve replays of a graph of ten calls, in us a call."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            call()
    best = float("inf")
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100.0)
    return best


def test_stride_of_a_single_row_does_not_matter():
    """One token's packed codes beside padded weights, and one output channel beside padded tokens: right, and no slower
    than the same operands with a padded row (20 us; the path of rows that start anywhere takes 41)."""
    from decoder_only_transformer_sm_b200 import native
    g = torch.Generator(device="cuda").manual_seed(2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    K = 763

    def operand(rows, pad):
        hold = torch.randint(-127, 128, (rows, K + pad), generator=g, dtype=torch.int8, device="cuda")
        return hold[:, :K]

    for M, N, dtype in ((1, 50304, torch.bfloat16), (1, 100, torch.float32), (300, 1, torch.float32), (5, 1, torch.bfloat16),
                        (1, 1, torch.float32)):
        a, b = operand(M, 5), operand(N, 5)
        sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
        tol = (4 * 2.0 ** -24 + (2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0.0)) * want.abs()
        times = []
        for pa, pb in ((a, b), (a.contiguous() if M == 1 else a, b.contiguous() if N == 1 else b),
                       (operand(1, 8).copy_(a) if M == 1 else a, operand(1, 8).copy_(b) if N == 1 else b)):
            out = torch.empty((M, N), dtype=dtype, device="cuda")
            native.matmul_i8(pa, sa, pb, sb, out, status=status)
            assert torch.all((out.double() - want).abs() <= tol)
            if N > 10000:
                times.append(_replay_time(lambda: native.matmul_i8(pa, sa, pb, sb, out, status=status)))
        assert not times or max(times) <= 1.4 * times[0], times
    for K_, dtype in ((6400, torch.bfloat16), (8192, torch.float32), (40, torch.bfloat16)):
        x = torch.randn((1, K_ + 3), generator=g, device="cuda").to(dtype)[:, :K_]
        room = torch.full((1, K_ + 5), 77, dtype=torch.int8, device="cuda")
        scale = torch.empty(1, device="cuda")
        native.quantize_rows(x, room[:, :K_], scale)
        want_q, want_s = _codes64(x.float().cpu().numpy())
        np.testing.assert_array_equal(room[:, :K_].cpu().numpy(), want_q)
        np.testing.assert_array_equal(scale.cpu().numpy(), want_s)
        assert torch.all(room[:, K_:] == 77)


@pytest.mark.parametrize("M,N,K", [(2500, 4001, 99), (2500, 4001, 257), (1900, 2561, 300), (1700, 3003, 385), (129, 20011, 515)])
@pytest.mark.parametrize("epilogue,out_dtype", [("bias", torch.bfloat16), ("bias_resid", torch.float32)])
@pytest.mark.parametrize("shift", [(0, 0, 0), (1, 3, 1)])
def test_rows_that_start_anywhere_over_several_tiles_a_block(M, N, K, epilogue, out_dtype, shift):
    """Packed operands, more tiles of 128 x 128 than SMs (up to 640): the ring and both accumulators are used again; one
    K block, odd and even numbers of them."""
    _product(M, N, K, epilogue, out_dtype, shift=shift)
