"""Layer norm on the GPU against its formulas in 64 bits.

Tolerances.  A float32 result is a short chain of operations on sums of n terms that are added in a tree
of at most 32 sequential steps per level: its error is below 64 * 2^-24 of the largest term of the
chain.  A bfloat16 result adds half a unit in the last place, up to 2^-8 of the value.
A column sum over R rows in float32 is within 2^-24 * (R / 64 + 64) of the sum of its terms' magnitudes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
UNIT = 2.0 ** -24


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_bit_quantized_gb300 as nv
    nv.reset_status()
    return nv


def close(got, want, magnitude):
    """got against the float64 value want; magnitude bounds the terms of its computation."""
    assert got.shape == want.shape
    g = got.double()
    bound = 64 * UNIT * magnitude + (2.0 ** -8 * want.abs() if got.dtype == BF16 else 0)
    worst = ((g - want).abs() - bound).max().item() if g.numel() else 0.0
    assert worst <= 0, f"off by {worst} more than the bound allows"


def case(R, C, x, y, w, seed, pitch=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mk(rows, dtype, scale=1.0, offset=0.0):
        t = torch.randn(rows, C + pitch, generator=g, device="cuda") * scale + offset
        return t.to(dtype)[:, :C]
    X, res, dy, dh = mk(R, x, 1.5, 0.3), mk(R, x), mk(R, y, 0.1), mk(R, x, 0.1)
    W, B = (1 + 0.3 * torch.randn(C, generator=g, device="cuda")).to(w), torch.randn(C, generator=g, device="cuda").to(w)
    return X, res, dy, dh, W, B


SHAPES = [(1, 1), (3, 1), (1, 2), (5, 7), (2, 31), (33, 32), (7, 33), (4, 64), (19, 100), (9, 128), (6, 255), (130, 256),
          (3, 1000), (2, 1024), (17, 1027), (300, 2048), (5, 4096), (4, 5120), (700, 5120), (3, 5127), (2, 8192), (3, 8200),
          (2, 16384), (2, 20480), (3, 20481), (2, 32768), (2, 40000), (1, 65544), (2, 70001), (2500, 96), (4000, 8)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("x,y,w", [(BF16, BF16, F32), (F32, F32, F32), (F32, BF16, BF16), (BF16, F32, BF16)])
def test_forward_and_backward_against_the_formulas(nv, R, C, x, y, w):
    X, res, dy, dh, W, B = case(R, C, x, y, w, R * 7 + C)
    for residual, bias in ((None, None), (res, B)):
        Y, mean, rstd, h = nv.layer_norm_forward(X, W, bias, eps=1e-5, residual=residual, out_dtype=y)
        assert Y.dtype == y and h.dtype == x
        hd = X.double()
        if residual is not None:
            assert torch.equal(h, (X.float() + residual.float()).to(x))
            hd = h.double()
        else:
            assert h is X
        mu = hd.mean(1, keepdim=True)
        var = (hd - mu).square().mean(1, keepdim=True)
        rs = 1 / torch.sqrt(var + 1e-5)
        xhat = (hd - mu) * rs
        top = hd.abs().amax(1, keepdim=True)
        close(mean, mu[:, 0], top[:, 0])
        # the statistics' errors pass on as top * UNIT * rstd
        close(rstd, rs[:, 0], rs[:, 0] * (1 + (top * rs)[:, 0]))
        close(Y, xhat * W.double() + (B.double() if bias is not None else 0),
              (1 + top * rs) * W.double().abs() * (1 + xhat.abs()) + (B.double().abs() if bias is not None else 0))
        # backward, at the statistics the forward pass gave
        dx, dw, db = nv.layer_norm_backward(dy, h, W, mean, rstd, dh=dh if residual is not None else None,
                                            bias=bias is not None)
        assert dx.dtype == x and dw.dtype == F32 and (db is None) == (bias is None)
        m, s = mean.double()[:, None], rstd.double()[:, None]
        xhat, g = (hd - m) * s, dy.double() * W.double()
        want = s * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        size = s * (g.abs().amax(1, keepdim=True)) * (2 + xhat.abs() * (1 + xhat.abs().amax(1, keepdim=True)))
        if residual is not None:
            want, size = want + dh.double(), size + dh.double().abs()
        close(dx, want, size * (1 + top * s))
        tree = 2.0 ** -24 * (R / 64 + 64)
        err = (dw.double() - (dy.double() * xhat).sum(0)).abs()
        assert (err <= tree * (dy.double().abs() * (xhat.abs() + top * s)).sum(0)).all()
        if bias is not None:
            err = (db.double() - dy.double().sum(0)).abs()
            assert (err <= tree * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("C", [64, 1024, 5120, 5121])
@pytest.mark.parametrize("pitch", [1, 8, 24])
def test_strided_and_unaligned_rows(nv, C, pitch):
    X, res, dy, dh, W, B = case(37, C, BF16, BF16, F32, 5, pitch)
    want = nv.layer_norm_forward(X.contiguous(), W, B, residual=res.contiguous())
    got = nv.layer_norm_forward(X, W, B, residual=res)
    for a, b in zip(got, want):
        assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-5)
    h, mean, rstd = want[3], want[1], want[2]
    hp = torch.empty(37, C + pitch, dtype=BF16, device="cuda")[:, :C].copy_(h)
    want = nv.layer_norm_backward(dy.contiguous(), h, W, mean, rstd, dh=dh.contiguous())
    got = nv.layer_norm_backward(dy, hp, W, mean, rstd, dh=dh)
    for a, b in zip(got, want):
        assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-4)
    # a weight that begins at an odd element
    off = torch.cat([W[:1], W])[1:]
    a, b = nv.layer_norm_forward(X, off, B)[0], nv.layer_norm_forward(X, W, B)[0]
    assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-5)


def test_gradients_against_differences(nv):
    """Central differences of sum(y * c), taken in float64 on the formula, for x, weight and bias."""
    R, C = 6, 96
    X, _, dy, _, W, B = case(R, C, F32, F32, F32, 3)

    def loss(x, w, b):
        mu = x.mean(1, keepdim=True)
        return (((x - mu) / torch.sqrt((x - mu).square().mean(1, keepdim=True) + 1e-5) * w + b) * dy.double()).sum()
    _, mean, rstd, h = nv.layer_norm_forward(X, W, B)
    grads = nv.layer_norm_backward(dy, h, W, mean, rstd)
    args = [X.double(), W.double(), B.double()]
    rng = np.random.default_rng(1)
    for k, grad in enumerate(grads):
        for _ in range(12):
            i = int(rng.integers(grad.numel()))
            step = torch.zeros_like(args[k]).view(-1)
            step[i] = 1e-5
            step = step.view_as(args[k])
            up, down = (loss(*[a + s * step if j == k else a for j, a in enumerate(args)]) for s in (1, -1))
            assert abs((up - down).item() / 2e-5 - grad.view(-1)[i].item()) < 1e-5   # O(step^2) + float32


def test_rows_none_constant_and_not_finite(nv):
    W = torch.ones(256, device="cuda")
    y, mean, rstd, h = nv.layer_norm_forward(torch.empty(0, 256, device="cuda", dtype=BF16), W)
    assert y.shape == (0, 256) and mean.shape == (0,)
    dx, dw, db = nv.layer_norm_backward(y, h, W, mean, rstd)
    assert dx.shape == (0, 256) and not dw.any() and not db.any()
    # constant rows: variance 0, rstd = 1 / sqrt(eps)
    x = torch.full((3, 256), 7.25, device="cuda")
    y, mean, rstd, _ = nv.layer_norm_forward(x, W, eps=1e-4)
    assert not y.any() and torch.allclose(mean, x[:, 0]) and torch.allclose(rstd, torch.full_like(rstd, 100.0))
    # a large offset does not eat the variance (no sum of squares minus square of sums)
    x = 3000.0 + torch.randn(4, 256, device="cuda")
    y = nv.layer_norm_forward(x, W)[0].double()
    xd = x.double()
    want = (xd - xd.mean(1, keepdim=True)) / torch.sqrt(xd.var(1, unbiased=False, keepdim=True) + 1e-5)
    assert (y - want).abs().max() < 64 * UNIT * 3100
    # infinities and NaN stay in their rows
    x = torch.randn(5, 256, device="cuda")
    x[1, 3], x[3, 200] = float("inf"), float("nan")
    y = nv.layer_norm_forward(x, W)[0]
    assert torch.isfinite(y[[0, 2, 4]]).all() and torch.isnan(y[[1, 3]]).any(1).all()


def test_results_repeat_and_follow_the_stream(nv):
    X, res, dy, dh, W, B = case(4099, 1536, BF16, BF16, F32, 9)
    y, mean, rstd, h = nv.layer_norm_forward(X, W, B, residual=res)
    first = nv.layer_norm_backward(dy, h, W, mean, rstd, dh=dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = nv.layer_norm_backward(dy, h, W, mean, rstd, dh=dh)
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(nv):
    """More than 2^32 bytes and 2^31 elements of rows: the last rows are normalised too."""
    R, C = 1 << 20, 2056
    x = torch.empty(R, C, dtype=BF16, device="cuda").normal_()
    W = torch.ones(C, device="cuda")
    y, mean, rstd, h = nv.layer_norm_forward(x, W)
    tail = x[-3:].double()
    want = (tail - tail.mean(1, keepdim=True)) / torch.sqrt(tail.var(1, unbiased=False, keepdim=True) + 1e-5)
    close(y[-3:], want, 1 + want.abs() * 8)
    dx, _, db = nv.layer_norm_backward(y, h, W, mean, rstd)
    alone = nv.layer_norm_backward(y[-3:], h[-3:], W, mean[-3:], rstd[-3:])[0]
    assert torch.allclose(dx[-3:].float(), alone.float(), rtol=2 ** -7, atol=1e-5)


def test_refusals(nv):
    x, W = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd, h = nv.layer_norm_forward(x, W)
    bad = [lambda: nv.layer_norm_forward(x.cpu(), W), lambda: nv.layer_norm_forward(x.half(), W),
           lambda: nv.layer_norm_forward(x.t(), W), lambda: nv.layer_norm_forward(x[0], W),
           lambda: nv.layer_norm_forward(x, W[:-1]), lambda: nv.layer_norm_forward(x, W.half()),
           lambda: nv.layer_norm_forward(x, W, W.bfloat16()), lambda: nv.layer_norm_forward(x, W, eps=-1.0),
           lambda: nv.layer_norm_forward(x, W, eps=float("nan")),
           lambda: nv.layer_norm_forward(x, W, residual=x.bfloat16()), lambda: nv.layer_norm_forward(x, W, residual=x[:2]),
           lambda: nv.layer_norm_forward(x, W, out_dtype=torch.float16), lambda: nv.layer_norm_forward(x[:, :0], W[:0]),
           lambda: nv.layer_norm_backward(y[:2], h, W, mean, rstd), lambda: nv.layer_norm_backward(y, h, W, mean[:2], rstd),
           lambda: nv.layer_norm_backward(y, h, W, mean, rstd.double()),
           lambda: nv.layer_norm_backward(y, h, W, mean, rstd, dh=h.bfloat16())]
    for f in bad:
        with pytest.raises(nv.NVFP4Error):
            f()
    assert nv.status_query() == 0


@pytest.mark.parametrize("C", [7, 64, 300, 5120, 9000, 70001])
@pytest.mark.parametrize("bias", [False, True])
def test_backward_of_no_rows_needs_only_its_outputs(nv, C, bias):
    """The C entry with rows = 0 and every operand of the rows NULL, the weight among them: the sums are zeros and nothing else is
    read, whichever kernels the width would take."""
    from nvfp4_bit_quantized_gb300 import _lib as L
    dw, db = (torch.full((C,), float("nan"), device="cuda") for _ in range(2))
    need = L.lib().nvfp4_layer_norm_backward_workspace_bytes(0, C)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    st = L.lib().nvfp4_layer_norm_backward(None, L.BF16, C, None, L.BF16, 0, C, C, None, L.F32, None, None, None, 0, None, C,
                                           dw.data_ptr(), db.data_ptr() if bias else None, ws.data_ptr(), ws.numel(),
                                           torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert not dw.any() and (torch.isnan(db).all() if not bias else not db.any())


def test_calls_of_several_widths_from_several_threads(nv):
    """One kernel serves many widths, each with its own amount of shared memory: threads that call the C entries with
    different ones, nothing between one call and the next, all get their launches, and the results are those of calls made alone."""
    import threading
    from nvfp4_bit_quantized_gb300 import _lib as L
    lib, widths = L.lib(), (8192, 4096, 6144, 2048)
    X, _, dy, _, W, B = case(3, 8192, BF16, BF16, F32, 1)

    def call(C, bufs, stream):
        y, mean, rstd, dx, dw, db, ws = (t.data_ptr() for t in bufs)
        st = lib.nvfp4_layer_norm_forward(X.data_ptr(), L.BF16, 3, C, 8192, None, 0, W.data_ptr(), B.data_ptr(), L.F32, 1e-5, y,
                                          L.BF16, C, None, 0, mean, rstd, stream)
        return st or lib.nvfp4_layer_norm_backward(dy.data_ptr(), L.BF16, 8192, X.data_ptr(), L.BF16, 3, C, 8192, W.data_ptr(),
                                                   L.F32, mean, rstd, None, 0, dx, C, dw, db, ws, bufs[6].numel(), stream)

    def buffers(C):
        f32 = dict(dtype=F32, device="cuda")
        return [torch.zeros(3, C, dtype=BF16, device="cuda"), torch.zeros(3, **f32), torch.zeros(3, **f32),
                torch.zeros(3, C, dtype=BF16, device="cuda"), torch.zeros(C, **f32), torch.zeros(C, **f32),
                torch.empty(lib.nvfp4_layer_norm_backward_workspace_bytes(3, C), dtype=torch.uint8, device="cuda")]
    want = [buffers(C) for C in widths]
    for C, b in zip(widths, want):
        assert call(C, b, torch.cuda.current_stream().cuda_stream) == 0
    got, streams = [buffers(C) for C in widths], [torch.cuda.Stream() for _ in widths]
    torch.cuda.synchronize()
    refused, gate = [], threading.Barrier(len(widths))

    def work(i):
        gate.wait()
        refused.extend(st for st in (call(widths[i], got[i], streams[i].cuda_stream) for _ in range(3000)) if st)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(widths))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[:5])
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a[:6], b[:6]))


@pytest.mark.parametrize("R,C", [(130, 64), (9, 255), (400, 1027), (400, 1024), (700, 5120), (20, 5127), (40, 8192), (40, 8200), (7, 20480),
                                 (5, 20481)])
@pytest.mark.parametrize("t", [BF16, F32])
def test_in_place(nv, R, C, t):
    """What the C interface allows to be one tensor: h = x, h = residual, y = x, dx = dh, dx = dy.  The bits are those of separate
    outputs, for rows with a pitch of their own."""
    from nvfp4_bit_quantized_gb300 import _lib as L
    lib, code, stream = L.lib(), L.F32 if t == F32 else L.BF16, torch.cuda.current_stream().cuda_stream
    X, res, dy, dh, W, B = case(R, C, t, t, F32, R + C)
    pitch = C + 8

    def rows(src=None):
        full = torch.full((R, pitch), float("nan"), dtype=t, device="cuda")
        if src is not None:
            full[:, :C] = src
        return full

    def forward(x, r, y, h):
        mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        st = lib.nvfp4_layer_norm_forward(x.data_ptr(), code, R, C, pitch, None if r is None else r.data_ptr(), pitch, W.data_ptr(),
                                          B.data_ptr(), L.F32, 1e-5, y.data_ptr(), code, pitch,
                                          None if h is None else h.data_ptr(), pitch, mean.data_ptr(), rstd.data_ptr(), stream)
        assert st == 0
        return y, mean, rstd, h

    def backward(g, x, mean, rstd, d, dx):
        dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
        ws = torch.empty(lib.nvfp4_layer_norm_backward_workspace_bytes(R, C), dtype=torch.uint8, device="cuda")
        st = lib.nvfp4_layer_norm_backward(g.data_ptr(), code, pitch, x.data_ptr(), code, R, C, pitch, W.data_ptr(), L.F32,
                                           mean.data_ptr(), rstd.data_ptr(), None if d is None else d.data_ptr(), pitch,
                                           dx.data_ptr(), pitch, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        assert st == 0
        return dx, dw, db

    def equal(got, want):
        for a, b in zip(got, want):
            if b is not None:
                assert torch.equal(a if a.dim() == 1 else a[:, :C], b if b.dim() == 1 else b[:, :C])
                assert a.dim() == 1 or torch.isnan(a[:, C:]).all()
    plain, with_res = forward(rows(X), None, rows(), None), forward(rows(X), rows(res), rows(), rows())
    x = rows(X)
    equal(forward(x, None, x, None), plain)                # y = x
    x, r = rows(X), rows(res)
    equal(forward(x, r, rows(), x), with_res)              # h = x
    x, r = rows(X), rows(res)
    equal(forward(x, r, rows(), r), with_res)              # h = residual
    x, r = rows(X), rows(res)
    equal(forward(x, r, x, r), with_res)                   # both, y = x and h = residual
    h, (mean, rstd) = rows(with_res[3][:, :C]), with_res[1:3]
    want, alone = backward(rows(dy), h, mean, rstd, rows(dh), rows()), backward(rows(dy), h, mean, rstd, None, rows())
    g, d = rows(dy), rows(dh)
    equal(backward(g, h, mean, rstd, d, d), want)          # dx = dh
    g, d = rows(dy), rows(dh)
    equal(backward(g, h, mean, rstd, d, g), want)          # dx = dy
    g = rows(dy)
    equal(backward(g, h, mean, rstd, None, g), alone)      # dx = dy, no dh
