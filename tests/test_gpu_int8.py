"""8-bit quantizer, product and layer on the GPU against the fp64 oracle.

The codes, the scales and the products are defined to the bit (exact quotients, exact
integer sums, single roundings), so they are compared for equality.  The layer's gradients
are compared with the formula to the bit and with the real-valued layer within the bound
that half a step of every code allows.
"""

import numpy as np
import pytest
import torch

from oracle import int8

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().double().cpu().numpy()


def _matrix(rows, cols, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    M = torch.randn(rows, cols, generator=g)
    if kind == "wide":          # lines of very different size, tiny ones among them
        M = M * torch.exp(80 * (torch.rand(rows, 1, generator=g) - 0.5)) * torch.exp(4 * torch.randn(1, cols, generator=g))
    elif kind == "ties":        # quotients on half integers: 127 x / a with a = 2^e and 127 x = (2 q + 1) 2^(e - 1)
        M = torch.randint(-128, 129, (rows, cols), generator=g).float() * 0.5
        M[:, 0] = 127.0
        M[0, :] = 127.0
    elif kind == "zeros":
        M[rows // 2:] = 0
        M[:, cols // 2:] = 0
    return M.to(dtype)


def _check_quantized(q, M):
    codes, scales = int8.quantize_rows(_np(M))
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)


SHAPES = [(1, 1), (1, 16), (1, 4097), (5, 7), (3, 16), (17, 2049), (64, 256), (129, 65), (200, 1333), (513, 64), (2, 20000),
          (20000, 3)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "zeros"])
def test_quantize_matches_the_oracle(ctx, shape, dtype, kind):
    rows, cols = shape
    M = _matrix(rows, cols, dtype, rows + 31 * cols, kind).cuda()
    for want_row, want_col in ((True, False), (False, True), (True, True)):
        row = ctx.new_int8(rows, cols) if want_row else None
        col = ctx.new_int8(cols, rows) if want_col else None
        ctx.quantize_int8(M, rowwise=row, colwise=col)
        if want_row:
            _check_quantized(row, M)
        if want_col:
            _check_quantized(col, M.t())
    assert ctx.poll_device_status() == 0


@pytest.mark.parametrize("shape", [(1300, 1030), (600, 4100), (610, 8200), (600, 12000), (33, 33000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_large_matches_the_oracle(ctx, shape, dtype):
    """Row lengths of every group size, and beyond what a group holds."""
    M = _matrix(*shape, dtype, 1).cuda()
    row, col = ctx.new_int8(*shape), ctx.new_int8(*shape[::-1])
    ctx.quantize_int8(M, rowwise=row, colwise=col)
    _check_quantized(row, M)
    _check_quantized(col, M.t())
    alone = ctx.new_int8(*shape)
    ctx.quantize_int8(M, rowwise=alone)
    assert torch.equal(alone.codes, row.codes) and torch.equal(alone.scales, row.scales)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_reads_strided_rows_and_leaves_the_rest(ctx, metis_lib, dtype):
    base = _matrix(70, 411, dtype, 1).cuda()
    M = base[3:68, 5:306]                         # no row starts on 16 bytes
    rows, cols = M.shape
    rbuf = torch.full((rows + 2, 320), 99, dtype=torch.int8, device="cuda")
    cbuf = torch.full((cols + 2, 96), 98, dtype=torch.int8, device="cuda")
    row = metis_lib.Int8(rows, cols, codes=rbuf[1:-1, :cols])
    col = metis_lib.Int8(cols, rows, codes=cbuf[1:-1, 16:16 + rows])
    ctx.quantize_int8(M, rowwise=row, colwise=col)
    _check_quantized(row, M)
    _check_quantized(col, M.t())
    assert (rbuf[0] == 99).all() and (rbuf[-1] == 99).all() and (rbuf[:, cols:] == 99).all()
    assert (cbuf[0] == 98).all() and (cbuf[-1] == 98).all() and (cbuf[:, :16] == 98).all()
    assert (cbuf[:, 16 + rows:] == 98).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_non_finite_and_extreme_values(ctx, metis_lib, dtype):
    big = torch.finfo(dtype).max
    M = _matrix(40, 50, dtype, 2).cuda()
    M[1, 2], M[3, 4], M[3, 5] = float("nan"), float("inf"), -float("inf")
    M[7, :] = float("nan")
    M[8, :] = float("inf")
    M[9, :4] = torch.tensor([big, -big, big / 2, 1.0])
    M[10, :] = 0
    M[10, 0] = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    row, col = ctx.new_int8(40, 50), ctx.new_int8(50, 40)
    for kw in (dict(rowwise=row), dict(colwise=col), dict(rowwise=row, colwise=col)):
        ctx.quantize_int8(M, **kw)
        assert ctx.poll_device_status() == metis_lib.DEV_NONFINITE
        if "rowwise" in kw:
            _check_quantized(row, M)
        if "colwise" in kw:
            _check_quantized(col, M.t())


def test_quantize_more_than_two_to_the_31_elements(ctx):
    rows, cols = 131072, 16400
    M = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    M[-3:] = _matrix(3, cols, torch.bfloat16, 5).cuda()
    M[:, -2:] = _matrix(rows, 2, torch.bfloat16, 6).cuda()
    row, col = ctx.new_int8(rows, cols), ctx.new_int8(cols, rows)
    ctx.quantize_int8(M, rowwise=row)
    only = row.codes[-40:].clone()
    ctx.quantize_int8(M, rowwise=row, colwise=col)
    assert torch.equal(only, row.codes[-40:])
    want, scales = int8.quantize_rows(_np(M[-40:]))
    assert np.array_equal(row.codes[-40:].cpu().numpy(), want)
    assert np.array_equal(row.scales[-40:].cpu().numpy(), scales)
    want, scales = int8.quantize_rows(_np(M[:, -3:]).T)
    assert np.array_equal(col.codes[-3:].cpu().numpy(), want)
    assert np.array_equal(col.scales[-3:].cpu().numpy(), scales)


def _codes(rows, cols, seed, low=-128):
    g = torch.Generator().manual_seed(seed)
    ld = -(-cols // 16) * 16
    buf = torch.randint(low, 128, (rows, ld), generator=g, dtype=torch.int8)
    scales = torch.exp(4 * torch.randn(rows, generator=g))
    return buf.cuda()[:, :cols], scales.cuda()


def _bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


PRODUCTS = [(1, 1, 1), (1, 100, 3), (1, 4096, 257), (2, 131071, 3), (5, 16, 1333), (16, 129, 128), (17, 1000, 40), (33, 384, 130),
            (40, 4096, 512), (64, 128, 4100), (65, 257, 129), (100, 2000, 72), (128, 128, 128), (129, 640, 256), (256, 256, 256),
            (300, 77, 515), (515, 1000, 1333), (768, 512, 1024), (1030, 300, 520), (2048, 160, 2312), (3, 5000, 20000), (600, 1, 5000)]


@pytest.mark.parametrize("p,k,q", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_is_exact(ctx, metis_lib, p, k, q, dtype):
    a, sa = _codes(p, k, p + k)
    b, sb = _codes(q, k, q + k + 1)
    A, B = metis_lib.Int8(p, k, codes=a, scales=sa), metis_lib.Int8(q, k, codes=b, scales=sb)
    buf = torch.full((p + 2, -(-q // 8) * 8 + 8), 7.0, dtype=dtype, device="cuda")
    C = buf[1:-1, :q]
    ctx.gemm_int8(A, B, C)
    want = torch.from_numpy(int8.product(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy())).to(dtype)
    assert torch.equal(_bits(C.cpu().contiguous()), _bits(want))
    assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, q:] == 7).all()
    assert ctx.poll_device_status() == 0


# K in 2 to 8 shares (a block of 128 each up to 16 tokens, eight above), tokens that do not divide by them, and single tiles
SHARES = [(p, 128 * s - 5, q) for s in range(2, 9) for p, q in ((1, 130), (2 * s - 1, 40), (16, 257))] + \
         [(p, 1024 * s + 77, q) for s in range(2, 9) for p, q in ((17 + s, 130), (33 + 3 * s, 72), (64, 129), (60 + 8 * s, 9))] + \
         [(20, 1100, 10000), (63, 1030, 9601), (64, 1024, 18900)]


@pytest.mark.parametrize("p,k,q", SHARES)
def test_product_in_shares_is_exact(ctx, metis_lib, p, k, q):
    test_product_is_exact(ctx, metis_lib, p, k, q, torch.float32)
    test_product_is_exact(ctx, metis_lib, p, k, q, torch.bfloat16)


@pytest.mark.parametrize("p,q", [(2, 3), (70, 130), (300, 260)])
def test_product_at_the_ends_of_the_codes(ctx, metis_lib, p, q):
    """The largest sums there are: 131071 products of (-128) (-128), and of 127 (-128)."""
    k = 131071
    for x, y in ((-128, -128), (127, -128), (127, 127)):
        a = torch.full((p, 131072), x, dtype=torch.int8, device="cuda")[:, :k]
        b = torch.full((q, 131072), y, dtype=torch.int8, device="cuda")[:, :k]
        one_p, one_q = torch.ones(p, device="cuda"), torch.ones(q, device="cuda")
        C = torch.empty(p, -(-q // 4) * 4, device="cuda")[:, :q]
        ctx.gemm_int8(metis_lib.Int8(p, k, codes=a, scales=one_p), metis_lib.Int8(q, k, codes=b, scales=one_q), C)
        assert (C == float(np.float32(k * x * y))).all()


def test_product_scales_of_zero_infinity_and_nan(ctx, metis_lib):
    a, sa = _codes(20, 64, 1)
    b, sb = _codes(24, 64, 2)
    sa[3], sa[4], sb[5], sb[6] = 0.0, float("nan"), float("inf"), 2.0 ** -126
    C = torch.empty(20, 24, device="cuda")
    ctx.gemm_int8(metis_lib.Int8(20, 64, codes=a, scales=sa), metis_lib.Int8(24, 64, codes=b, scales=sb), C)
    with np.errstate(invalid="ignore"):
        want = int8.product(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy())
    assert np.array_equal(C.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("l,m,n", [(1, 4096, 1024), (7, 100, 30), (40, 512, 768), (130, 257, 129), (600, 1024, 516)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_is_the_quantizer_and_the_product(ctx, metis_lib, l, m, n, dtype):
    X = _matrix(l, m, dtype, 9).cuda()
    w, sw = _codes(n, m, 10)
    W, Xq = metis_lib.Int8(n, m, codes=w, scales=sw), ctx.new_int8(l, m)
    Y = torch.empty(l, -(-n // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :n]
    for _ in range(3):                                     # the buffers are used again
        Xq.codes.fill_(55)
        Y.fill_(3.0)
        ctx.linear_int8(X, Xq, W, Y)
        _check_quantized(Xq, X)
        codes, scales = int8.quantize_rows(_np(X))
        want = torch.from_numpy(int8.product(codes, scales, w.cpu().numpy(), sw.cpu().numpy())).bfloat16()
        assert torch.equal(_bits(Y.cpu().contiguous()), _bits(want))


def test_refusals(ctx, metis_lib):
    X = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    q, t = ctx.new_int8(4, 32), ctx.new_int8(32, 4)
    Y = torch.zeros(4, 8, device="cuda")
    w = ctx.new_int8(8, 32)

    def status(call):
        with pytest.raises(metis_lib.MetisError) as e:
            call()
        return e.value.status

    assert status(lambda: ctx.quantize_int8(X)) == 1
    assert status(lambda: ctx.quantize_int8(X, rowwise=t)) == 2
    assert status(lambda: ctx.quantize_int8(X, colwise=q)) == 2
    square = ctx.new_int8(32, 32)
    assert status(lambda: ctx.quantize_int8(torch.zeros(32, 32, device="cuda"), rowwise=square, colwise=square)) == 1
    odd = metis_lib.Int8(4, 24, codes=torch.zeros(4, 24, dtype=torch.int8, device="cuda"))
    assert status(lambda: ctx.quantize_int8(X[:, :24], rowwise=odd)) == 3             # row stride 24
    shifted = metis_lib.Int8(4, 32, codes=torch.zeros(4, 48, dtype=torch.int8, device="cuda")[:, 8:40])
    assert status(lambda: ctx.quantize_int8(X, rowwise=shifted)) == 3
    assert status(lambda: ctx.gemm_int8(q, ctx.new_int8(8, 48), Y)) == 2
    assert status(lambda: ctx.gemm_int8(q, ctx.new_int8(6, 32), torch.zeros(4, 6, device="cuda"))) == 3
    long_a, long_b = ctx.new_int8(1, 131072), ctx.new_int8(4, 131072)
    assert status(lambda: ctx.gemm_int8(long_a, long_b, torch.zeros(1, 4, device="cuda"))) == 2
    for call in (lambda: ctx.quantize_int8(X.half(), rowwise=q), lambda: ctx.quantize_int8(X.t(), rowwise=t),
                 lambda: ctx.quantize_int8(X.cpu(), rowwise=q), lambda: ctx.gemm_int8(q, w, Y.half()),
                 lambda: ctx.gemm_int8(q, w, torch.zeros(4, 12, device="cuda")),
                 lambda: ctx.quantize_int8(X[:1].expand(4, 32), rowwise=q),
                 lambda: ctx.linear_int8(X, ctx.new_int8(5, 32), w, Y)):
        with pytest.raises(ValueError):
            call()
    ctx.gemm_int8(q, w, Y)                                                             # the context is usable
    assert ctx.poll_device_status() == 0


def test_captured_and_replayed_on_new_inputs(ctx, metis_lib):
    """Two graphs of the same calls, replayed in turn on changed inputs, beside eager calls."""
    l, m, n = 40, 512, 264
    W = ctx.new_int8(n, m)
    weight = _matrix(m, n, torch.float32, 3).cuda()
    sets = []
    for i in range(2):
        X = _matrix(l, m, torch.bfloat16, 20 + i).cuda()
        Xq, row, col = ctx.new_int8(l, m), ctx.new_int8(l, m), ctx.new_int8(m, l)
        Y = torch.empty(l, n, dtype=torch.bfloat16, device="cuda")
        ctx.quantize_int8(weight, colwise=W)
        ctx.linear_int8(X, Xq, W, Y)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ctx.linear_int8(X, Xq, W, Y)
            ctx.quantize_int8(X, rowwise=row, colwise=col)
        sets.append((graph, X, row, col, Y))
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for i, (graph, X, row, col, Y) in enumerate(sets):
            X.copy_(_matrix(l, m, torch.bfloat16, 100 * rep + i))
        torch.cuda.synchronize()
        for i, (graph, *_rest) in enumerate(sets):
            with torch.cuda.stream(side[i]):
                graph.replay()
        torch.cuda.synchronize()
        for graph, X, row, col, Y in sets:
            _check_quantized(row, X)
            _check_quantized(col, X.t())
            codes, scales = int8.quantize_rows(_np(X))
            wc, ws = int8.quantize_rows(_np(weight).T)
            want = torch.from_numpy(int8.product(codes, scales, wc, ws)).bfloat16()
            assert torch.equal(_bits(Y.cpu()), _bits(want))


# ---------------------------------------------------------------------------- the layer
def _layer(m, n, seed, **kw):
    from spectral_quantized_gemm_b200.int8_linear import Int8Linear
    layer = Int8Linear(m, n, device="cuda", **kw)
    with torch.no_grad():
        layer.weight.copy_((_matrix(m, n, torch.float32, seed) / m ** 0.5).to(layer.weight.dtype))
    return layer


def _formula(x, w, dy):
    y = int8.product(*int8.quantize_rows(x), *int8.quantize_rows(w.T))
    dx = int8.product(*int8.quantize_rows(dy), *int8.quantize_rows(w))
    dw = int8.product(*int8.quantize_rows(x.T), *int8.quantize_rows(dy.T))
    return y, dx, dw


@pytest.mark.parametrize("l,m,n", [(1, 64, 48), (33, 100, 77), (256, 256, 512), (300, 515, 130), (700, 768, 264)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_matches_the_formula(metis_lib, l, m, n, dtype):
    layer = _layer(m, n, 1)
    x = _matrix(l, m, dtype, 2).cuda().requires_grad_(True)
    dy = (1e-5 * _matrix(l, n, torch.float32, 3)).bfloat16().cuda()
    y = layer(x)
    y.backward(dy)
    wy, wdx, wdw = _formula(_np(x), _np(layer.weight), _np(dy))
    assert y.dtype == torch.bfloat16 and x.grad.dtype == dtype and layer.weight.grad.dtype == torch.float32
    assert torch.equal(y.detach().cpu(), torch.from_numpy(wy).bfloat16())
    assert torch.equal(x.grad.cpu(), torch.from_numpy(wdx).to(dtype))
    assert torch.equal(layer.weight.grad.cpu(), torch.from_numpy(wdw))


@pytest.mark.parametrize("l,m,n", [(48, 96, 64), (257, 130, 72)])
def test_layer_gradients_against_differences(metis_lib, l, m, n):
    """The loss <dY, X W> is linear in X and in W, so its central difference along E is the slope
    itself; the layer's slope differs by the quantization of two operands (half a step a code),
    plus one bf16 rounding of dX."""
    layer = _layer(m, n, 4)
    x = _matrix(l, m, torch.bfloat16, 5).cuda().requires_grad_(True)
    dy = _matrix(l, n, torch.bfloat16, 6).cuda()
    layer(x).backward(dy)
    X, W, D = _np(x), _np(layer.weight), _np(dy)

    def loss(X, W):
        return float((D * (X @ W)).sum())

    rng = np.random.default_rng(0)
    for _ in range(4):
        E, F = rng.standard_normal(W.shape), rng.standard_normal(X.shape)
        slope_w = (loss(X, W + E) - loss(X, W - E)) / 2
        slope_x = (loss(X + F, W) - loss(X - F, W)) / 2
        bound_w = int8.product_error_bound(X.T, D.T, int8.quantize_rows(X.T)[1], int8.quantize_rows(D.T)[1])
        bound_x = int8.product_error_bound(D, W, int8.quantize_rows(D)[1], int8.quantize_rows(W)[1])
        bound_x = bound_x + 2.0 ** -8 * (np.abs(D @ W.T) + bound_x)
        assert abs((_np(layer.weight.grad) * E).sum() - slope_w) <= (bound_w * np.abs(E)).sum()
        assert abs((_np(x.grad) * F).sum() - slope_x) <= (bound_x * np.abs(F)).sum()


def test_layer_shapes_modes_and_zero_tokens(metis_lib):
    layer = _layer(64, 40, 7)
    x = _matrix(24, 64, torch.bfloat16, 8).cuda()
    y = layer(x)
    assert torch.equal(layer(x.reshape(2, 3, 4, 64)).reshape(24, 40), y)
    assert torch.equal(layer(x.t().contiguous().t()), y)                  # any strides
    assert torch.equal(layer(x.half().float()), layer(x.half()))          # other types go through fp32
    empty = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    out = layer(empty)
    out.backward(torch.zeros_like(out))
    assert out.shape == (0, 40) and empty.grad.shape == (0, 64) and (layer.weight.grad == 0).all()
    layer.weight.grad = None
    # only one of the gradients, and the same pass twice
    y = layer(x)
    y.backward(torch.ones_like(y), retain_graph=True)
    first = layer.weight.grad.clone()
    layer.weight.grad = None
    y.backward(torch.ones_like(y))
    assert torch.equal(first, layer.weight.grad)
    layer.weight.requires_grad_(False)
    xg = x.clone().requires_grad_(True)
    layer(xg).sum().backward()
    assert xg.grad is not None and torch.equal(layer.weight.grad, first)


def test_layer_broadcast_gradient_and_shared_weight(metis_lib):
    """A gradient expanded from one row (stride 0) and a layer used twice in one graph."""
    layer = _layer(96, 64, 9)
    x = _matrix(32, 96, torch.bfloat16, 10).cuda()
    layer(x).sum().backward()                              # dY is an expanded one
    once = layer.weight.grad.clone()
    want = _formula(_np(x), _np(layer.weight), np.ones((32, 64)))[2]
    assert torch.equal(once.cpu(), torch.from_numpy(want))
    layer.weight.grad = None
    (layer(x).sum() + layer(x).sum()).backward()
    assert torch.equal(layer.weight.grad, once + once)


@pytest.mark.parametrize("reduce", ["rows", "columns"])
def test_layer_gradient_expanded_along_one_dimension(metis_lib, reduce):
    """A mean over rows or columns hands the layer a gradient with a stride of 0."""
    layer = _layer(64, 40, 21)
    x = _matrix(24, 64, torch.bfloat16, 22).cuda().requires_grad_(True)
    w = torch.randn(40 if reduce == "rows" else 24, device="cuda", generator=torch.Generator("cuda").manual_seed(0)).bfloat16()
    (layer(x).sum(0 if reduce == "rows" else 1) * w).sum().backward()
    dy = w.expand(24, 40) if reduce == "rows" else w[:, None].expand(24, 40)
    _, dx, dw = _formula(_np(x), _np(layer.weight), _np(dy))
    assert torch.equal(x.grad.cpu(), torch.from_numpy(dx).bfloat16())
    assert torch.equal(layer.weight.grad.cpu(), torch.from_numpy(dw))


def test_layer_on_expanded_and_padded_inputs(metis_lib):
    layer = _layer(64, 40, 23)
    row = _matrix(1, 64, torch.bfloat16, 24).cuda()
    with torch.no_grad():
        want = layer(row.expand(17, 64).contiguous())
        assert torch.equal(layer(row.expand(17, 64)), want)
        wide = torch.full((17, 100), 9.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 3:67] = row
        assert torch.equal(layer(wide[:, 3:67]), want)
        layer.freeze()
        assert torch.equal(layer(row.expand(17, 64)), want)


def test_layer_pass_captured_and_replayed(metis_lib):
    layer = _layer(256, 136, 25)
    x = torch.zeros(128, 256, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    dy = torch.zeros(128, 136, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(layer(x), (x, layer.weight), dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x)
        dx, dw = torch.autograd.grad(y, (x, layer.weight), dy)
    for seed in range(3):
        with torch.no_grad():
            x.copy_(_matrix(128, 256, torch.bfloat16, 50 + seed))
            dy.copy_(_matrix(128, 136, torch.bfloat16, 60 + seed))
            layer.weight.mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        wy, wdx, wdw = _formula(_np(x), _np(layer.weight), _np(dy))
        assert torch.equal(y.detach().cpu(), torch.from_numpy(wy).bfloat16())
        assert torch.equal(dx.cpu(), torch.from_numpy(wdx).bfloat16())
        assert torch.equal(dw.cpu(), torch.from_numpy(wdw))


def test_layer_copies_and_casts(metis_lib):
    import copy
    import pickle
    layer = _layer(64, 40, 26).freeze()
    x = _matrix(5, 64, torch.bfloat16, 27).cuda()
    with torch.no_grad():
        want = layer(x)
        for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
            assert other._frozen is None and torch.equal(other(x), want)
        assert torch.equal(layer(x), want)
        half = copy.deepcopy(layer).freeze().bfloat16()
        with pytest.raises(RuntimeError):
            half(x)
        assert torch.equal(half.freeze()(x), half.unfreeze()(x))


def test_two_threads_and_two_streams(metis_lib):
    """Layers of one device share a context; passes from two threads on their own streams do not mix."""
    import threading
    layers = [_layer(256, 128, 30), _layer(128, 320, 31)]
    xs = [_matrix(64, 256, torch.bfloat16, 32).cuda(), _matrix(96, 128, torch.bfloat16, 33).cuda()]
    want = [layer(x).detach() for layer, x in zip(layers, xs)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                x = xs[i].clone().requires_grad_(True)
                y = layers[i](x)
                y.sum().backward()
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y.detach(), want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_layer_call_refusals(ctx, metis_lib):
    from spectral_quantized_gemm_b200.int8_linear import _buffers
    dev = torch.device("cuda", 0)
    X, W = torch.zeros(8, 32, device=dev), torch.zeros(32, 16, device=dev)
    Y, D = torch.zeros(8, 16, device=dev), torch.zeros(8, 16, device=dev)
    keep, (xr, wc, xc, wr, dr, dc) = _buffers(dev, ((8, 32, False), (16, 32, True), (32, 8, True), (32, 16, False), (8, 16, False), (16, 8, True)))

    def status(call):
        with pytest.raises(metis_lib.MetisError) as e:
            call()
        return e.value.status

    ctx.int8_linear_fwd(X, W, Y, xr, wc, Xcol=xc, Wrow=wr)
    assert status(lambda: ctx.int8_linear_fwd(X, W, Y, None, wc)) == 1
    assert status(lambda: ctx.int8_linear_fwd(X, W, Y, xr, wr)) in (1, 2)                     # no scratch, wrong shape
    assert status(lambda: ctx.int8_linear_fwd(X, W[:16], Y, xr, wc)) == 2
    assert status(lambda: ctx.int8_linear_fwd(X, W, Y, xr, wc, Xcol=dr)) in (1, 2)
    assert status(lambda: ctx.int8_linear_bwd(D, Drow=dr, Dcol=dc, Xcol=xc, Wrow=wr)) == 1    # nothing asked for
    wide = metis_lib.Int8Struct(xc.codes, xc.scales, 32, 8, xc.ld, wc.scratch)                # Wcol's scratch
    assert status(lambda: ctx.int8_linear_fwd(X, W, Y, xr, wc, Xcol=wide, Wrow=wr)) == 1
    wide.scratch = wc.scratch + 4 * 9 * 16 - 4                                                # its last word
    assert status(lambda: ctx.int8_linear_fwd(X, W, Y, xr, wc, Xcol=wide, Wrow=wr)) == 1
    dX, dW = torch.zeros(8, 32, device=dev), torch.zeros(32, 16, device=dev)
    assert status(lambda: ctx.int8_linear_bwd(D, Dcol=dc, Xcol=xc, dX=dX)) == 1
    assert status(lambda: ctx.int8_linear_bwd(D, Drow=dr, Wrow=wr, dW=dW)) == 1
    for call in (lambda: ctx.int8_linear_fwd(X, W, Y[:4], xr, wc), lambda: ctx.int8_linear_fwd(X.cpu(), W, Y, xr, wc),
                 lambda: ctx.int8_linear_bwd(D, Drow=dr, Wrow=wr, dX=dX[:, :16]),
                 lambda: ctx.int8_linear_bwd(D, Dcol=dc, Xcol=xc, dW=dW.bfloat16())):
        with pytest.raises(ValueError):
            call()
    ctx.int8_linear_bwd(D, Drow=dr, Dcol=dc, Xcol=xc, Wrow=wr, dX=dX, dW=dW)
    assert ctx.poll_device_status() == 0 and not dX.any() and not dW.any()
    no_scratch = metis_lib.Int8(32, 8)
    assert metis_lib._quant_i8(ctx._h, X.data_ptr(), 8, 32, 32, 0, None, metis_lib.ctypes.byref(no_scratch.struct)) == 1


def test_frozen_layer_notices_the_optimizer(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    layer = _layer(64, 40, 28).freeze()
    opt = AdamW(layer.parameters(), lr=0.1)
    x = _matrix(5, 64, torch.bfloat16, 29).cuda()
    for _ in range(3):                                     # a first step, and steps from a plan
        layer.freeze()
        layer(x).sum().backward()
        opt.step()
        with torch.no_grad(), pytest.raises(RuntimeError):
            layer(x)


def test_frozen_layer_serves_and_notices_a_changed_weight(metis_lib):
    layer = _layer(256, 136, 11)
    for rows in (1, 5, 64, 200):
        x = _matrix(rows, 256, torch.bfloat16, rows).cuda()
        with torch.no_grad():
            want = layer(x)
            layer.freeze()
            assert torch.equal(layer(x), want)
            layer.unfreeze()
    layer.freeze()
    x = _matrix(8, 256, torch.bfloat16, 1).cuda()
    with torch.no_grad():
        assert layer(x[:0]).shape == (0, 136)
        layer.weight.mul_(2)
        with pytest.raises(RuntimeError):
            layer(x)
    assert layer(x).requires_grad                          # training does not read the frozen codes
    with torch.no_grad():
        assert torch.equal(layer.freeze()(x), layer.unfreeze()(x))


@pytest.mark.parametrize("rows", [1, 24, 60, 300])
def test_served_right_after_the_weight_was_written(metis_lib, rows):
    """A new weight, its layout, its use and the next weight in the same memory, with nothing in between that
    waits: each answer belongs to its weight."""
    layer = _layer(2048, 1536, 40)
    x = _matrix(rows, 2048, torch.bfloat16, 41).cuda()
    weights = [_matrix(2048, 1536, torch.float32, 50 + i).cuda() for i in range(4)]
    want = []
    with torch.no_grad():
        for w in weights:
            layer.weight.copy_(w)
            want.append(layer(x))
            torch.cuda.synchronize()
        got = []
        for i in range(24):
            layer.weight.copy_(weights[i % 4])
            got.append(layer.freeze()(x))
        for i in range(24):
            assert torch.equal(got[i], want[i % 4]), i


def test_layer_on_another_stream(metis_lib):
    layer = _layer(512, 520, 12)
    x = _matrix(128, 512, torch.bfloat16, 13).cuda()
    want = layer(x).detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(x).detach()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


# the pair kernel's stores leave in 16 bytes: 8 bf16 or 4 fp32 columns
NARROW = [(18945, 64, q) for q in (1, 3, 4, 5, 7, 8, 12)] + [(20000, 100, 3), (19000, 1000, 7), (40000, 16, 130)]


@pytest.mark.parametrize("p,k,q", NARROW)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_many_rows_by_few_columns(ctx, metis_lib, p, k, q, dtype):
    test_product_is_exact(ctx, metis_lib, p, k, q, dtype)


@pytest.mark.parametrize("q", [1, 3, 5, 7, 8, 40])
def test_product_of_few_columns_on_few_sms(ctx, metis_lib, q):
    ctx.set_sm_count_target(2)
    try:
        for dtype in (torch.bfloat16, torch.float32):
            test_product_is_exact(ctx, metis_lib, 300, 200, q, dtype)
    finally:
        ctx.set_sm_count_target(0)


@pytest.mark.parametrize("l,m,n", [(18945, 40, 1), (18945, 3, 24), (33, 18945, 3), (18950, 5, 6)])
def test_layer_of_few_features_on_many_tokens(metis_lib, l, m, n):
    layer = _layer(m, n, 1)
    x = _matrix(l, m, torch.bfloat16, 2).cuda().requires_grad_(True)
    dy = (1e-5 * _matrix(l, n, torch.float32, 3)).bfloat16().cuda()
    y = layer(x)
    y.backward(dy)
    wy, wdx, wdw = _formula(_np(x), _np(layer.weight), _np(dy))
    assert torch.equal(y.detach().cpu(), torch.from_numpy(wy).bfloat16())
    assert torch.equal(x.grad.cpu(), torch.from_numpy(wdx).bfloat16())
    assert torch.equal(layer.weight.grad.cpu(), torch.from_numpy(wdw))
    with torch.no_grad():
        assert torch.equal(layer.freeze()(x), y)


@pytest.mark.parametrize("n", [48, 77])
@pytest.mark.parametrize("shape", [(33,), (3, 11)])
def test_layer_output_changed_in_place(metis_lib, n, shape):
    layer, bias = _layer(64, n, 5), _matrix(1, n, torch.bfloat16, 6).cuda()[0].requires_grad_(True)
    x = _matrix(33, 64, torch.bfloat16, 7).cuda().reshape(*shape, 64).requires_grad_(True)
    keep = (torch.rand(*shape, n, device="cuda", generator=torch.Generator("cuda").manual_seed(0)) > 0.5).bfloat16()
    got = {}
    for inplace in (False, True):
        y = layer(x)
        if inplace:
            y.mul_(keep)
            y += bias
            y.relu_()
        else:
            y = torch.relu(y * keep + bias)
        got[inplace] = (y.detach(), *torch.autograd.grad(y.float().square().sum(), (x, layer.weight, bias)))
    for a, b in zip(got[False], got[True]):
        assert torch.equal(a, b)
    y = torch.nn.functional.dropout(layer(x), 0.5, inplace=True)
    assert ((y == 0) | (y == 2 * layer(x))).all() and y.any()


def test_frozen_layer_notices_replaced_memory(metis_lib):
    layer = _layer(256, 136, 42)
    x = _matrix(8, 256, torch.bfloat16, 43).cuda()
    other = _matrix(256, 136, torch.float32, 44)
    with torch.no_grad():
        layer.freeze()
        for _ in range(2):
            layer.weight.data = other.cuda()
        with pytest.raises(RuntimeError):
            layer(x)


def test_frozen_layer_notices_a_round_trip_cast(metis_lib):
    layer = _layer(256, 136, 42)
    x = _matrix(8, 256, torch.bfloat16, 43).cuda()
    with torch.no_grad():
        layer.freeze()
        layer.bfloat16().float()
        with pytest.raises(RuntimeError):
            layer(x)


def test_frozen_layer_notices_another_parameter_on_its_memory(metis_lib):
    layer = _layer(256, 136, 42)
    x = _matrix(8, 256, torch.bfloat16, 43).cuda()
    with torch.no_grad():
        layer.weight = torch.nn.Parameter(layer.weight.data)
        layer.freeze()
        layer.weight.mul_(2)
        layer.weight = torch.nn.Parameter(layer.weight.data)
        with pytest.raises(RuntimeError):
            layer(x)


def test_frozen_layer_notices_a_transposed_weight(metis_lib):
    layer = _layer(64, 64, 42)
    x = _matrix(8, 64, torch.bfloat16, 43).cuda()
    with torch.no_grad():
        layer.freeze()
        layer.weight.data = layer.weight.data.t()
        with pytest.raises(RuntimeError):
            layer(x)
        assert torch.equal(layer.freeze()(x), layer.unfreeze()(x))


def test_layer_made_and_served_in_inference_mode(metis_lib):
    from spectral_quantized_gemm_b200.int8_linear import Int8Linear
    x = _matrix(8, 256, torch.bfloat16, 43).cuda()
    with torch.inference_mode():
        layer = Int8Linear(256, 136, device="cuda")
        want = layer(x)
        assert torch.equal(layer.freeze()(x), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p,q", [(513, 333), (1500, 1031)])
def test_columns_right_after_the_matrix_was_written(ctx, metis_lib, p, q, dtype):
    """A product writes a matrix whose rows are quantized from an odd column on, and the next one writes the same
    memory, with nothing in between that waits: each result belongs to its product."""
    k, n = 256, 4
    B = metis_lib.Int8(q, k, codes=_codes(q, k, 1)[0], scales=torch.ones(q, device="cuda"))
    As = [metis_lib.Int8(p, k, codes=_codes(p, k, 2 + i)[0], scales=torch.full((p,), 2.0 ** -i, device="cuda")) for i in range(n)]
    C = torch.empty(p, -(-q // 8) * 8, dtype=dtype, device="cuda")
    M = C[:, 1:q]
    want = []
    for A in As:
        ctx.gemm_int8(A, B, C[:, :q])
        torch.cuda.synchronize()
        want.append(tuple(torch.from_numpy(x).cuda() for x in int8.quantize_rows(_np(M).T)))
    got = [ctx.new_int8(q - 1, p).with_scratch() for _ in range(6 * n)]
    for i, col in enumerate(got):
        ctx.gemm_int8(As[i % n], B, C[:, :q])
        ctx.quantize_int8(M, colwise=col)
    for i, col in enumerate(got):
        assert torch.equal(col.codes, want[i % n][0]) and torch.equal(col.scales, want[i % n][1]), i


def test_frozen_weight_takes_any_number_of_tokens(metis_lib):
    layer = _layer(16, 24, 50)
    layer.weight.requires_grad_(False)
    x = _matrix(131072 + 5, 16, torch.bfloat16, 51).cuda().requires_grad_(True)
    y = layer(x)
    y.sum().backward()
    wy, wdx, _ = _formula(_np(x), _np(layer.weight), np.ones((131072 + 5, 24)))
    assert torch.equal(y.detach().cpu(), torch.from_numpy(wy).bfloat16())
    assert torch.equal(x.grad.cpu(), torch.from_numpy(wdx).bfloat16())


def test_linear_refuses_its_weight_as_the_buffer(ctx, metis_lib):
    W = ctx.new_int8(8, 32)
    X, Y = torch.zeros(8, 32, device="cuda"), torch.zeros(8, 8, device="cuda")
    with pytest.raises(metis_lib.MetisError) as e:
        ctx.linear_int8(X, W, W, Y)
    assert e.value.status == 1
    for kw in (dict(scales=W.scales), dict(codes=W.codes)):
        with pytest.raises(metis_lib.MetisError) as e:
            ctx.linear_int8(X, metis_lib.Int8(8, 32, **kw), W, Y)
        assert e.value.status == 1
