"""Attention on the GPU against its definition in 64 bits, head by head.

Tolerances, with u = 2^-8 the unit roundoff of bf16 (8 bits of significand: between 1 and 2 its values lie 2^-7 apart,
so rounding to the nearest moves a value by up to 2^-8 of it).  out: the probabilities are rounded to bf16 (u of each, so u * sum p |v|
at most) and the result once more (u |out|); 2 u * sum(p |v|) + u |out| is allowed.  Gradients: P and dS are rounded once each (u of
each term), delta comes from the rounded out (u * sum |dout| |out|, times P), and the result is rounded (u of it); the sums of the
terms' magnitudes are computed beside the values and 2 u of them allowed (4 u for the terms with delta).  fp32 sums and the exponential
add less than 2^-16 of the same magnitudes.  lse: float32, 2^-18 * (1 + max |z|)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = 2.0 ** -8


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_bit_quantized_gb300 as nv
    nv.reset_status()
    return nv


def definition(q, k, v, dout, causal, scale, oq, ok):
    """float64 results and, for each, the sum of the magnitudes of its rounded terms."""
    T, H, D = q.shape
    S, G, _ = k.shape
    z64 = dict(dtype=torch.float64, device="cuda")
    r = {n: torch.zeros(s, **z64) for n, s in (("out", q.shape), ("dq", q.shape), ("dk", k.shape), ("dv", k.shape))}
    r.update({n + "_mag": torch.zeros_like(x) for n, x in list(r.items())})
    r["lse"] = torch.full((H, T), -math.inf, **z64)
    for a0, a1, b0, b1 in zip(oq, oq[1:], ok, ok[1:]):
        if a1 == a0 or b1 == b0:
            continue
        i, j = torch.arange(a1 - a0, device="cuda"), torch.arange(b1 - b0, device="cuda")
        seen = (j[None] <= i[:, None] + (b1 - b0) - (a1 - a0)) if causal else torch.ones(a1 - a0, b1 - b0, dtype=torch.bool,
                                                                                       device="cuda")
        for h in range(H):
            g = h // (H // G)
            Q, K, V, dO = q[a0:a1, h].double(), k[b0:b1, g].double(), v[b0:b1, g].double(), dout[a0:a1, h].double()
            z = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[:, None]).masked_fill(~seen, 0.0)
            o = p @ V
            r["out"][a0:a1, h], r["lse"][h, a0:a1] = o, lse
            r["out_mag"][a0:a1, h] = 2 * p @ V.abs() + o.abs()
            dp, delta = dO @ V.T, (dO * o).sum(1, keepdim=True)
            ds = p * (dp - delta) * scale
            mag = (2 * ds.abs() + 4 * p * abs(scale) * (dO.abs() * o.abs()).sum(1, keepdim=True))
            r["dq"][a0:a1, h] = ds @ K
            r["dq_mag"][a0:a1, h] = mag @ K.abs()
            r["dk"][b0:b1, g] += ds.T @ Q
            r["dk_mag"][b0:b1, g] += mag.T @ Q.abs()
            r["dv"][b0:b1, g] += p.T @ dO
            r["dv_mag"][b0:b1, g] += 2 * p.T @ dO.abs()
    for n in ("dq", "dk", "dv"):
        r[n + "_mag"] += r[n].abs()
    return r


def check(name, got, r):
    err = (got.double() - r[name]).abs()
    assert torch.isfinite(err).all(), name
    over = (err - (U + 2.0 ** -16) * r[name + "_mag"]).max().item() if err.numel() else 0
    assert over <= 1e-30, f"{name}: {over} more than the bound"


def make(T, S, H, G, D, seed, fused=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    if T == S and fused:
        x = rnd(T, H + 2 * G, D).to(BF16)
        q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
    else:
        q, k, v = rnd(T, H, D).to(BF16), rnd(S, G, D).to(BF16), rnd(S, G, D).to(BF16)
    return q, k, v, rnd(T, H, D).to(BF16)


def run_and_check(nv, q, k, v, dout, causal, scale, oq, ok, packed):
    D = q.shape[2]
    cu = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in (oq, ok)] if packed else (None, None)
    args = dict(causal=causal, scale=scale, cu_q=cu[0], cu_k=cu[1])
    out, lse = nv.attention_forward(q, k, v, **args)
    r = definition(q, k, v, dout, causal, D ** -0.5 if scale is None else scale, oq, ok)
    check("out", out, r)
    empty = torch.isinf(r["lse"])
    assert torch.equal(empty, torch.isinf(lse)) and (lse[empty] < 0).all()
    zmax = (q.double().norm(dim=2).max() * k.double().norm(dim=2).max() * (D ** -0.5 if scale is None else abs(scale))).item() \
        if q.numel() and k.numel() else 0
    assert ((lse.double() - r["lse"])[~empty].abs() <= 2.0 ** -18 * (1 + zmax)).all()
    assert not out.transpose(0, 1)[empty].any()
    grads = nv.attention_backward(dout, q, k, v, out, lse, **args)
    for name, g in zip(("dq", "dk", "dv"), grads):
        check(name, g, r)
    assert not grads[0].transpose(0, 1)[empty].any()
    assert nv.status_query() == 0
    return out, lse, grads


LENGTHS = [(1, 1), (1, 300), (2, 3), (64, 64), (127, 129), (128, 128), (129, 127), (200, 77), (255, 257), (256, 256),
           (300, 1), (513, 640), (1100, 1100), (0, 5), (5, 0)]


@pytest.mark.parametrize("T,S", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,G,D", [(2, 1, 128), (3, 3, 64), (4, 2, 80), (5, 1, 8)])
def test_one_sequence(nv, T, S, causal, H, G, D):
    q, k, v, dout = make(T, S, H, G, D, T * 3 + S)
    run_and_check(nv, q, k, v, dout, causal, None, [0, T], [0, S], False)


@pytest.mark.parametrize("D", range(8, 129, 8))
def test_every_head_size(nv, D):
    q, k, v, dout = make(190, 190, 2, 2, D, D)
    run_and_check(nv, q, k, v, dout, True, None, [0, 190], [0, 190], False)


@pytest.mark.parametrize("T,S,H,G,D", [(1, 5000, 2, 1, 128), (130, 4100, 4, 2, 64), (4100, 130, 4, 1, 128), (2500, 2500, 8, 1, 64),
                                       (300, 2049, 1, 1, 40), (2049, 1, 3, 1, 72)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_tiles_with_many_steps(nv, T, S, H, G, D, causal):
    """Several multiprocessors share a tile's steps: parts of every length, some of them masked away whole."""
    q, k, v, dout = make(T, S, H, G, D, T + S)
    run_and_check(nv, q, k, v, dout, causal, None, [0, T], [0, S], False)
    o = [0, T // 3, T // 3, T]
    oks = [0, S // 7, S // 2, S]
    run_and_check(nv, q, k, v, dout, causal, None, o, oks, True)


def test_forward_without_a_workspace_is_the_same_attention(nv):
    import ctypes
    from nvfp4_bit_quantized_gb300 import _lib as L
    q, k, v, dout = make(70, 3000, 2, 2, 64, 3)
    out, lse = nv.attention_forward(q, k, v)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    h = [L.HeadsC(x.data_ptr(), x.stride(0), x.stride(1)) for x in (q, k, v, o2)]
    s = L.AttentionShapeC(70, 3000, 2, 2, 64, 0, 0.125, 1, None, None)
    assert L.lib().nvfp4_attention_forward_workspace_bytes(ctypes.byref(s)) > 16      # the call above shared its tiles
    st = L.lib().nvfp4_attention_forward(ctypes.byref(s), *(ctypes.byref(x) for x in h), l2.data_ptr(),
                                         nv.dev_status().data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    r = definition(q, k, v, dout, False, 0.125, [0, 70], [0, 3000])
    check("out", o2, r)
    assert torch.allclose(l2, lse, rtol=1e-5, atol=1e-5)


PACKED = [([0, 1, 1, 130, 259, 300, 300], [0, 1, 1, 130, 259, 300, 300]),
          ([0, 0, 128, 256, 257, 700], [0, 64, 64, 320, 330, 500]),
          ([0, 5, 10, 15, 20, 25, 30, 35, 40], [0, 7, 14, 21, 28, 35, 42, 49, 56]),
          ([0, 700], [0, 20]), ([0, 0, 0, 0], [0, 3, 3, 9])]


@pytest.mark.parametrize("which", range(len(PACKED)))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_packed_sequences(nv, which, causal, D):
    oq, ok = PACKED[which]
    q, k, v, dout = make(oq[-1], ok[-1], 4, 2, D, which)
    run_and_check(nv, q, k, v, dout, causal, 0.1, oq, ok, True)


def test_many_short_sequences(nv):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 9, 700)
    o = [0] + [int(x) for x in np.cumsum(lens)]
    q, k, v, dout = make(o[-1], o[-1], 2, 1, 64, 1)
    run_and_check(nv, q, k, v, dout, True, None, o, o, True)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 8.0])
def test_scales_and_peaked_rows(nv, scale):
    """Scores from all equal to far apart: the running maximum moves by hundreds within a row."""
    q, k, v, dout = make(260, 390, 2, 2, 64, 11, fused=False)
    k[200:210] *= 4
    run_and_check(nv, q, k, v, dout, False, scale, [0, 260], [0, 390], False)
    run_and_check(nv, q, k, v, dout, True, scale, [0, 260], [0, 390], False)


def test_layouts_give_equal_results(nv):
    """Heads-first storage, sliced tokens and padded rows: the bits do not depend on the strides."""
    q, k, v, dout = (x.contiguous() for x in make(300, 300, 4, 2, 96, 2))
    out, lse = nv.attention_forward(q, k, v, causal=True)
    grads = nv.attention_backward(dout, q, k, v, out, lse, causal=True)

    def heads_first(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def padded(x):
        w = torch.full((x.shape[0], x.shape[1] + 1, x.shape[2] + 8), float("nan"), dtype=BF16, device="cuda")
        w[:, 1:, 8:] = x
        return w[:, 1:, 8:]

    def every_other(x):
        w = torch.full((2 * x.shape[0],) + x.shape[1:], float("nan"), dtype=BF16, device="cuda")
        w[::2] = x
        return w[::2]
    for lay in (heads_first, padded, every_other):
        o2, l2 = nv.attention_forward(lay(q), lay(k), lay(v), causal=True, out=lay(torch.zeros_like(q)))
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        dst = [lay(torch.zeros_like(x)) for x in (q, k, v)]
        bases = [d._base if d._base is not None else d for d in dst]
        outside = [torch.isnan(b.float()).sum().item() for b in bases]
        nv.attention_backward(lay(dout), lay(q), lay(k), lay(v), lay(out), lse, causal=True, dq=dst[0], dk=dst[1], dv=dst[2])
        for a, b in zip(dst, grads):
            assert torch.equal(a, b)
        assert outside == [torch.isnan(b.float()).sum().item() for b in bases]   # nothing beside the views was written


def test_what_lies_outside_a_sequence_does_not_reach_it(nv):
    """The neighbours of a sequence in the packed buffer hold NaN and infinities; its results are those of the sequence alone."""
    o = [0, 100, 233, 400]
    q, k, v, dout = make(400, 400, 2, 2, 64, 4, fused=False)
    for bad in (float("nan"), float("inf")):
        q2, k2, v2, d2 = (x.clone() for x in (q, k, v, dout))
        for x in (q2, k2, v2, d2):
            x[:100], x[233:] = bad, bad
        cu = torch.tensor(o, dtype=torch.int32, device="cuda")
        out, lse = nv.attention_forward(q2, k2, v2, causal=True, cu_q=cu)
        grads = nv.attention_backward(d2, q2, k2, v2, out, lse, causal=True, cu_q=cu)
        s = slice(100, 233)
        alone, l1 = nv.attention_forward(q[s], k[s], v[s], causal=True)
        want = nv.attention_backward(dout[s], q[s], k[s], v[s], alone, l1, causal=True)
        assert torch.allclose(out[s].float(), alone.float(), rtol=2 ** -7, atol=1e-3)
        for a, b in zip(grads, want):
            assert torch.isfinite(a[s].float()).all()
            assert torch.allclose(a[s].float(), b.float(), rtol=2 ** -6, atol=4e-3)


def test_bad_offsets_are_reported(nv):
    q, k, v, dout = make(300, 300, 2, 1, 64, 6)
    out, lse = nv.attention_forward(q, k, v)
    for o in ([0, 200, 100, 300], [0, 100], [5, 300], [0, 10 ** 9], [-5, 300], [0, 300, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]):
        cu = torch.tensor(o, dtype=torch.int32, device="cuda")
        nv.attention_forward(q, k, v, cu_q=cu)
        assert nv.status_query() == 1
        nv.reset_status()
        nv.attention_backward(dout, q, k, v, out, lse, cu_q=cu, causal=True)
        assert nv.status_query() == 1
        nv.reset_status()


def test_gradients_against_differences(nv):
    """Central differences, in float64 on the definition, of sum(out * dout) along single elements; the gradient is rounded to bf16
    and its terms too (the bound of the module)."""
    T, S, H, G, D = 9, 12, 2, 1, 16
    q, k, v, dout = make(T, S, H, G, D, 8)
    out, lse = nv.attention_forward(q, k, v, causal=True)
    grads = nv.attention_backward(dout, q, k, v, out, lse, causal=True)
    r = definition(q, k, v, dout, True, D ** -0.5, [0, T], [0, S])
    args = [q.double(), k.double(), v.double()]
    rng = np.random.default_rng(3)
    for n, (name, grad) in enumerate(zip(("dq", "dk", "dv"), grads)):
        for _ in range(10):
            i = int(rng.integers(grad.numel()))
            d = torch.zeros(grad.numel(), dtype=torch.float64, device="cuda")
            d[i] = 1e-4
            d = d.view(grad.shape)
            vals = [(definition(*[a + s * d if j == n else a for j, a in enumerate(args)], dout, True, D ** -0.5, [0, T],
                                [0, S])["out"] * dout.double()).sum().item() for s in (1, -1)]
            got = grad.reshape(-1)[i].item()
            assert abs((vals[0] - vals[1]) / 2e-4 - got) <= 2 * U * r[name + "_mag"].reshape(-1)[i].item() + 1e-6


def test_repeats_and_streams(nv):
    q, k, v, dout = make(1500, 1500, 6, 2, 128, 12)
    out, lse = nv.attention_forward(q, k, v, causal=True)
    grads = nv.attention_backward(dout, q, k, v, out, lse, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = nv.attention_forward(q, k, v, causal=True)
        g2 = nv.attention_backward(dout, q, k, v, out, lse, causal=True)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    for a, b in zip(grads, g2):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(nv):
    """Token strides that put the last tokens past 2^31 elements from the first."""
    T, H, D = 2200, 1, 64
    base = torch.empty(T * (1 << 20), dtype=BF16, device="cuda")
    wide = base.view(T, 1 << 20)
    q, k, v, dout = (wide[:, 64 * i:64 * i + D].view(T, 1, D) for i in range(4))
    small = make(T, T, H, H, D, 13, fused=False)
    for dst, src in zip((q, k, v, dout), small):
        dst.copy_(src)
    out, lse = nv.attention_forward(q, k, v, causal=True, out=wide[:, 512:576].view(T, 1, D))
    want, wl = nv.attention_forward(*small[:3], causal=True)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    dst = [wide[:, 1024 + 64 * i:1088 + 64 * i].view(T, 1, D) for i in range(3)]
    nv.attention_backward(dout, q, k, v, out, lse, causal=True, dq=dst[0], dk=dst[1], dv=dst[2])
    for a, b in zip(dst, nv.attention_backward(small[3], *small[:3], want, wl, causal=True)):
        assert torch.equal(a, b)


def test_refusals(nv):
    q, k, v, dout = make(64, 64, 4, 2, 64, 7, fused=False)
    out, lse = nv.attention_forward(q, k, v)
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    wide = torch.zeros(64, 4, 72, dtype=BF16, device="cuda")
    bad = [lambda: nv.attention_forward(q.float(), k, v), lambda: nv.attention_forward(q.cpu(), k, v),
           lambda: nv.attention_forward(q[0], k, v), lambda: nv.attention_forward(q, k[:, :, :56], v),
           lambda: nv.attention_forward(q, k, v[:32]), lambda: nv.attention_forward(q[:, :3], k, v),
           lambda: nv.attention_forward(q[:, :, :60], k[:, :, :60], v[:, :, :60]),
           lambda: nv.attention_forward(wide[:, :, 4:68], k, v), lambda: nv.attention_forward(q, k, v, scale=float("inf")),
           lambda: nv.attention_forward(q.transpose(1, 2), k, v), lambda: nv.attention_forward(q, k.expand(64, 2, 64)[:1].expand(64, 2, 64), v),
           lambda: nv.attention_forward(q, k, v, cu_q=cu.long()), lambda: nv.attention_forward(q, k, v, cu_q=cu[:1]),
           lambda: nv.attention_forward(q, k, v, cu_k=cu), lambda: nv.attention_forward(q, k, v, cu_q=cu.cpu()),
           lambda: nv.attention_forward(q, k, v, out=out[:32]),
           lambda: nv.attention_forward(*(torch.zeros(8, 1, 136, dtype=BF16, device="cuda"),) * 3),
           lambda: nv.attention_backward(dout, q, k, v, out, lse.double()),
           lambda: nv.attention_backward(dout, q, k, v, out, lse[:, :8]),
           lambda: nv.attention_backward(dout, q, k, v, out, lse, dq=k), lambda: nv.attention_backward(dout[:5], q, k, v, out, lse)]
    for n, f in enumerate(bad):
        with pytest.raises(nv.NVFP4Error):
            f()
            print("not refused:", n)
    assert nv.status_query() == 0


def test_calls_from_several_threads(nv):
    """Each thread's calls have their own descriptors: results are those of calls made one after another, bit for bit."""
    import threading
    cases = [make(70 + 61 * i, 130 + 40 * i, 4, 2, 64, 10 + i) for i in range(4)]

    def call(q, k, v, dout):
        out, lse = nv.attention_forward(q, k, v, causal=True)
        return (out, lse) + nv.attention_backward(dout, q, k, v, out, lse, causal=True)
    want = [call(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = call(*cases[i])
                stream.synchronize()
                bad.extend((i, n) for n, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:10]


def test_a_scale_past_fp32_is_refused(nv):
    q, k, v, _ = make(8, 8, 2, 2, 64, 3)
    for scale in (1e300, float("inf"), float("nan")):
        with pytest.raises(nv.NVFP4Error):
            nv.attention_forward(q, k, v, scale=scale)


def test_more_steps_in_parts_than_32_bits_count(nv):
    """2^25 steps of one tile of keys in 64 parts: the products of steps and part number pass 2^31, and no part's steps are lost.
    Tokens and heads overlap in memory, so that 2^32 rows of queries are small; only lse and delta are as long.  All
    probabilities are 1 / 128 (q = 0) and dout is 1, so each step adds exactly 1 to dv, each part 2^19, which fp32 holds."""
    import ctypes
    from nvfp4_bit_quantized_gb300 import _lib as L
    T, S, H, D = 1 << 23, 128, 512, 8

    def rows(value, n=T + H - 1):
        t = torch.full((n, D), value, dtype=BF16, device="cuda")
        return t, L.HeadsC(t.data_ptr(), D, D)
    zero, one, dq = rows(0.0), rows(1.0), rows(1.0)
    k, v, dk, dv = rows(0.0, S), rows(0.0, S), rows(1.0, S), rows(1.0, S)
    lse = torch.full((H, T), math.log(128), device="cuda")
    s = L.AttentionShapeC(T, S, H, 1, D, 0, 1.0, 1, None, None)
    ref = ctypes.byref
    need = L.lib().nvfp4_attention_backward_workspace_bytes(ref(s))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert need - 4 * H * T >= 2 * 64 * S * D * 4           # room for 64 parts of dV and dK
    st = L.lib().nvfp4_attention_backward(ref(s), ref(one[1]), ref(zero[1]), ref(k[1]), ref(v[1]), ref(zero[1]), lse.data_ptr(),
                                          ref(dq[1]), ref(dk[1]), ref(dv[1]), ws.data_ptr(), need,
                                          nv.dev_status().data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and nv.status_query() == 0
    assert (dv[0] == 2.0 ** 25).all() and not dk[0].any() and not dq[0].any()


@pytest.mark.parametrize("shape", [(4, 2, 0), (0, 2, 0), (4, 0, 64), (0, 0, 0)])
def test_axes_of_no_elements_are_refused(nv, shape):
    """No heads, or heads of no elements, with and without tokens: an argument error like any other."""
    x = torch.zeros(shape, dtype=BF16, device="cuda")
    lse = torch.zeros(shape[1], shape[0], device="cuda")
    for scale in (None, 1.0):
        with pytest.raises(nv.NVFP4Error):
            nv.attention_forward(x, x, x, scale=scale)
        with pytest.raises(nv.NVFP4Error):
            nv.attention_backward(x, x, x, x, x, lse, scale=scale)
    assert nv.status_query() == 0


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kind", ["mixed", "long among empty", "one more than a warp", "tiles' ends"])
def test_more_sequences_than_a_warp_holds(nv, kind, causal):
    """Past 32 sequences the tiles are found by a search: every tile of every sequence is worked on, wherever long, short and empty
    ones lie."""
    rng = np.random.default_rng(len(kind))
    lq = {"mixed": rng.integers(0, 5, 150) * rng.integers(0, 90, 150),
          "long among empty": np.where(np.arange(1100) % 300 == 299, 600, 0),
          "one more than a warp": rng.integers(1, 120, 33),
          "tiles' ends": rng.choice([0, 1, 127, 128, 129, 255, 256, 257], 40)}[kind]
    lk = np.where(rng.random(len(lq)) < 0.5, lq, rng.permutation(lq))
    o, oks = ([0] + [int(x) for x in np.cumsum(x)] for x in (lq, lk))
    q, k, v, dout = make(o[-1], oks[-1], 2, 1, 64, 5, fused=False)
    run_and_check(nv, q, k, v, dout, causal, None, o, oks, True)


def test_bad_offsets_among_many_are_reported(nv):
    good = list(range(0, 3201, 32))
    q, k, v, dout = make(3200, 3200, 2, 1, 64, 6)
    out, lse = nv.attention_forward(q, k, v)

    def statuses(o):
        cu, right = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (o, good))
        for a, b in ((cu, cu), (cu, right), (right, cu)):
            nv.attention_forward(q, k, v, cu_q=a, cu_k=b)
            yield nv.status_query()
            nv.reset_status()
            nv.attention_backward(dout, q, k, v, out, lse, cu_q=a, cu_k=b, causal=True)
            yield nv.status_query()
            nv.reset_status()
    assert set(statuses(good)) == {0}
    for at, value in ((0, 1), (0, -5), (1, 5000), (31, 1), (32, -2 ** 31), (33, 0), (64, 2 ** 31 - 1), (77, 2400), (99, 3201), (100, 3199),
                      (100, 0)):
        assert set(statuses(good[:at] + [value] + good[at + 1:])) == {1}, (at, value)


def test_the_time_grows_with_the_sequences_not_with_their_square(nv):
    """16 times the sequences of 8 tokens, 16 times the work: three times that is allowed for what does not scale."""
    def time_of(n):
        q, k, v, dout = make(8 * n, 8 * n, 4, 2, 64, n)
        cu = torch.arange(0, 8 * n + 1, 8, dtype=torch.int32, device="cuda")

        def call():
            out, lse = nv.attention_forward(q, k, v, causal=True, cu_q=cu)
            nv.attention_backward(dout, q, k, v, out, lse, causal=True, cu_q=cu)
        call()
        best = math.inf
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    few, many = time_of(1024), time_of(16384)
    assert many < 3 * 16 * few, (few, many)
    assert nv.status_query() == 0
