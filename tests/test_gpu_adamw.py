"""The AdamW step on the GPU, bit for bit against its lines in numpy float32 (each one IEEE operation), and its
32-bit form against float64.  Random words come from a separate Philox here, pinned to the oracle's."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
f = np.float32


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_bit_quantized_gb300 as nv
    nv.reset_status()
    return nv


def philox(n, stream, step, seed):
    """Word (i & 3) of Philox4x32-10 with counter (i >> 2, stream, step) for i < n."""
    low = np.uint64(0xFFFFFFFF)
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    c = [i & low, i >> np.uint64(32), np.full_like(i, stream), np.full_like(i, step)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:n].astype(np.uint32)


def e4m3_values():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))


GRID = e4m3_values()


def e4m3(x, sr, rand16):
    """Codes of float32 x: the two grid neighbours by search, the choice by position."""
    a = np.minimum(np.abs(x).astype(np.float64), 448.0)
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    gap = np.where(hi > lo, GRID[hi] - GRID[lo], 1.0)
    pos = (a - GRID[lo]) / gap
    # the conversion looks at 20 bits below the code: a position below 2^-20 of a subnormal step counts as rounded there
    pos = np.rint(pos * 2 ** 20) / 2 ** 20
    if sr:
        up = pos + rand16.astype(np.float64) / 65536 >= 1
    else:
        up = (pos > 0.5) | ((pos == 0.5) & (lo & 1 == 1))
    code = np.where(up, hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def e4m3_value(c):
    return (GRID[np.minimum(c & 127, 126)] * np.where(c & 128, -1.0, 1.0)).astype(np.float32)


def blocks_of(x):
    return np.concatenate([x, np.zeros(-len(x) % 128, np.float32)]).reshape(-1, 128)


def encode8(x, sr, rand16, floor):
    top = np.abs(blocks_of(x)).max(1) if len(x) else np.zeros(0, f)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(top > 0, np.minimum(f(448) / top, np.finfo(f).max), f(0)).astype(f)
    c = e4m3(x * np.repeat(inv, 128)[:len(x)], sr, rand16)
    if floor:
        c = np.where((x > 0) & (c == 0), 1, c).astype(np.uint8)
    return c, top * f(1 / 448)


def reference(p, g, state, bits, t, hp, gs, decay, sr, seed, i, pdtype):
    """One step of one tensor; arrays are float32 (codes uint8); returns the new p (float32) and state."""
    lr, b1, b2, eps = hp
    n = len(p)
    if bits == 8:
        m = e4m3_value(state["m"]) * np.repeat(state["m_scale"], 128)[:n]
        v = e4m3_value(state["v"]) * np.repeat(state["v_scale"], 128)[:n]
    else:
        m, v = state["m"], state["v"]
    g = g * f(gs)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    p = p * f(1 - lr * decay) - (m * f(lr / (1 - b1 ** t))) / (np.sqrt(v) * f(1 / math.sqrt(1 - b2 ** t)) + f(eps))
    assert p.dtype == f and m.dtype == f and v.dtype == f
    if pdtype == BF16:
        b = p.view(np.uint32).astype(np.uint64)
        b += (philox(n, 2 * i + 1, t, seed) & 0xFFFF) if sr else 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))
        p = (b.astype(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    if bits == 32:
        return p, {"m": m, "v": v}
    w = philox(n, 2 * i, t, seed)
    mc, ms = encode8(m, sr, w & 0xFFFF, False)
    vc, vs = encode8(v, sr, w >> 16, True)
    return p, {"m": mc, "m_scale": ms, "v": vc, "v_scale": vs}


def host(t):
    t = t.detach().cpu()
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).reshape(-1).numpy().copy()
    return t.float().reshape(-1).numpy().copy()


def test_philox_is_the_oracles(oracle_mod):
    got = philox(64, 5, 77, 0x123456789ABCDEF0)
    for grp in range(16):
        ref = oracle_mod.philox4x32_10([grp, 0, 5, 77], [0x9ABCDEF0, 0x12345678])
        assert np.array_equal(got[4 * grp:4 * grp + 4], ref)


SETS = [[1], [127, 128, 129], [0, 5, 1000, 4096], [3 * 128 * 64 + 77, 1, 130], [(48, 40), (1027,), (8, 16, 24)],
        [20480 + 8] + [33 + 5 * i for i in range(70)], [300001, 64]]


@pytest.mark.parametrize("which", range(len(SETS)))
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("pdt,gdt,sr", [(F32, BF16, True), (BF16, F32, True), (BF16, BF16, False), (F32, F32, False)])
def test_bit_for_bit(nv, which, bits, pdt, gdt, sr):
    rng = np.random.default_rng(which)
    shapes = [s if isinstance(s, tuple) else (s,) for s in SETS[which]]
    seed, hp, decay = 0xABCDEF12345, (3e-3, 0.9, 0.95, 1e-8), [0.1 * (k % 3) for k in range(len(shapes))]
    gs = torch.tensor([0.5], device="cuda")
    params = [torch.from_numpy(rng.standard_normal(s).astype(f) * f(0.05)).to(pdt).cuda() for s in shapes]
    opt = nv.AdamW(params, bits=bits, weight_decay=decay)
    ref_p = [host(p) for p in params]
    ref_s = [{k: host(v[i]) for k, v in opt.state.items()} for i in range(len(shapes))]
    for t in range(1, 4):
        grads = []
        for k, s in enumerate(shapes):
            g = rng.standard_normal(s).astype(f) * np.exp(rng.standard_normal(s) * 2).astype(f) * f(1e-3)
            if g.size > 200:
                g.reshape(-1)[130:200] *= 0.0 if t < 3 else 1e-12      # zeros, then values far below their block's largest
            grads.append(torch.from_numpy(g).to(gdt).cuda())
        opt.step(grads, lr=hp[0], betas=hp[1:3], eps=hp[3], grad_scale=gs, round=nv.SR if sr else nv.RNE, sr_seed=seed)
        assert opt.steps == t
        for i in range(len(shapes)):
            ref_p[i], ref_s[i] = reference(ref_p[i], host(grads[i]), ref_s[i], bits, t, hp, 0.5, decay[i], sr, seed, i, pdt)
            assert np.array_equal(host(params[i]), ref_p[i]), (t, i)
            for k in ref_s[i]:
                assert np.array_equal(host(opt.state[k][i]), ref_s[i][k]), (t, i, k)
    assert nv.status_query() == 0


def test_against_float64(nv):
    """32-bit states over five steps: each float32 line adds at most a unit in the last place of its terms, so after five
    steps p is within 64 * 2^-24 of |p| + the sum of the steps, and m, v within 64 * 2^-24 of their terms."""
    rng = np.random.default_rng(0)
    p0 = rng.standard_normal(5000).astype(f)
    param = torch.from_numpy(p0.copy()).cuda()
    opt = nv.AdamW([param], weight_decay=0.1)
    p, m, v, moved = p0.astype(np.float64), 0.0, 0.0, 0.0
    for t in range(1, 6):
        g = (rng.standard_normal(5000) * 0.01).astype(f)
        opt.step([torch.from_numpy(g).cuda()], lr=1e-2, betas=(0.9, 0.999), eps=1e-8)
        g = g.astype(np.float64)
        m, v = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
        step = 1e-2 * (m / (1 - 0.9 ** t)) / (np.sqrt(v / (1 - 0.999 ** t)) + 1e-8)
        p, moved = p * (1 - 1e-3) - step, moved + np.abs(step)
    assert (np.abs(host(param) - p) <= 64 * 2.0 ** -24 * (np.abs(p) + moved)).all()
    assert np.allclose(host(opt.state["v"][0]), v, rtol=64 * 2.0 ** -24, atol=0)


def test_eight_bit_states_follow_a_slow_average(nv):
    """With beta2 = 0.99 one step moves v by at most 1 % of the distance to g^2, less than half a code step (3 % of the value
    at least): rounded to nearest it stays, rounded stochastically it follows.  v starts 4 times too large; after 1000
    steps it should be 1 + 3 * 0.99^1000, almost 1.  Each element's stationary spread is at most 0.37 (code step 1/8,
    variance step^2 / 6 a step against a pull of 0.01), so the mean over 4064 elements is within 6 * 0.37 / sqrt(4064) = 0.035."""
    n = 4096
    g = torch.ones(n, device="cuda")
    g[::128] = 2.0                                          # keeps each block's scale where it is
    means = {}
    for mode in (nv.SR, nv.RNE):
        code = torch.full((n,), 448.0, device="cuda").to(torch.float8_e4m3fn)
        scale = torch.full((n // 128,), 4.0 / 448, device="cuda")
        opt = nv.AdamW([torch.zeros(n, device="cuda")], bits=8, steps=100000, state={
            "m": [torch.zeros_like(code)], "v": [code], "m_scale": [torch.zeros_like(scale)], "v_scale": [scale]})
        for _ in range(1000):
            opt.step([g], lr=0.0, betas=(0.9, 0.99), round=mode, sr_seed=3)
        v = opt.state["v"][0].float().view(-1, 128) * opt.state["v_scale"][0][:, None]
        means[mode] = v[:, 1:].mean().item()
    assert abs(means[nv.SR] - 1) < 0.035 and means[nv.RNE] > 2.5, means


def test_none_zero_steps_and_non_finite(nv):
    a, b, c = torch.ones(300, device="cuda"), torch.ones(200, device="cuda"), torch.empty(0, device="cuda")
    opt = nv.AdamW([a, b, c], bits=8, weight_decay=0.0)
    opt.step([torch.ones_like(a), None, torch.empty_like(c)], lr=0.1)
    assert torch.equal(b, torch.ones_like(b)) and not opt.state["m_scale"][1].any() and (a < 1).all()
    assert nv.status_query() == 0
    # zero gradients from zero states: nothing moves, nothing is divided by zero
    z = torch.full((256,), 3.0, device="cuda")
    opt = nv.AdamW([z], bits=8, weight_decay=0.0)
    opt.step([torch.zeros_like(z)], lr=0.1)
    assert torch.equal(z, torch.full_like(z, 3.0)) and not opt.state["m_scale"][0].any()
    for bits in (8, 32):
        w = torch.ones(512, device="cuda")
        opt = nv.AdamW([w], bits=bits)
        g = torch.ones_like(w)
        g[300] = float("inf")
        opt.step([g], lr=0.1)
        assert nv.status_query() == 7
        nv.reset_status()
        assert torch.isfinite(w[:256]).all() and torch.isfinite(w[384:]).all()
    opt = nv.AdamW([], bits=8)
    opt.step([], lr=0.1)


def test_unaligned_tensors_and_streams(nv):
    """Tensors that begin at any element give what aligned ones give; on a side stream too."""
    rng = torch.Generator().manual_seed(2)
    for bits in (8, 32):
        for off in (1, 2, 3, 5):
            base = torch.randn(3000, generator=rng).cuda()
            gr = torch.randn(3000, generator=rng).cuda()
            p1, p2 = base[off:off + 2000], base[off:off + 2000].clone()
            g1, g2 = gr[off:off + 2000].bfloat16(), gr[off:off + 2000].bfloat16()
            gbuf = torch.empty(3000, device="cuda", dtype=BF16)
            gbuf[off:off + 2000] = g1
            o1, o2 = nv.AdamW([p1], bits=bits), nv.AdamW([p2], bits=bits)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                o1.step([gbuf[off:off + 2000]], lr=1e-2, sr_seed=4)
            side.synchronize()
            o2.step([g2], lr=1e-2, sr_seed=4)
            assert torch.equal(p1, p2)
            for k in o1.state:
                assert torch.equal(o1.state[k][0].view(torch.uint8), o2.state[k][0].view(torch.uint8))


def test_refusals(nv):
    p = torch.zeros(256, device="cuda")
    g = torch.zeros_like(p)
    opt = nv.AdamW([p])
    state8 = nv.AdamW([p], bits=8).state
    bad = [lambda: nv.AdamW([p], bits=16), lambda: nv.AdamW([p.cpu()]), lambda: nv.AdamW([p.half()]),
           lambda: nv.AdamW([torch.zeros(8, 8, device="cuda").t()[1:]]), lambda: nv.AdamW([p], weight_decay=[0.1, 0.1]),
           lambda: nv.AdamW([p], state=state8), lambda: nv.AdamW([p], bits=8, state={**state8, "m": [p]}),
           lambda: nv.AdamW([p], steps=-1), lambda: opt.step([], lr=0.1), lambda: opt.step([g[:8]], lr=0.1),
           lambda: opt.step([g.half()], lr=0.1), lambda: opt.step([g.cpu()], lr=0.1),
           lambda: opt.step([torch.zeros(512, device="cuda")[::2]], lr=0.1), lambda: opt.step([g], lr=float("nan")),
           lambda: opt.step([g], lr=0.1, betas=(1.0, 0.9)), lambda: opt.step([g], lr=0.1, eps=-1.0),
           lambda: opt.step([g], lr=0.1, round=5), lambda: opt.step([g], lr=0.1, grad_scale=p)]
    for k, fn in enumerate(bad):
        with pytest.raises(nv.NVFP4Error):
            fn()
    assert opt.steps == 0 and not p.any() and nv.status_query() == 0
    moved = nv.AdamW([p])
    p.data = torch.ones(256, device="cuda")
    with pytest.raises(nv.NVFP4Error):
        moved.step([g], lr=0.1)


@pytest.mark.parametrize("bits", [8, 32])
def test_replaced_states_and_parameters_are_refused(nv, bits):
    """The step works on the tensors that the object was made with.  Others in their place, and other storage under them, are
    refused before anything is launched: neither the old tensors, which a checkpoint would not store, nor the new are touched.
    Values copied into them are the next step's."""
    def made():
        params = [torch.ones(300, device="cuda"), torch.ones(40, device="cuda")]
        opt = nv.AdamW(params, bits=bits)
        grads = [torch.ones_like(p) for p in params]
        opt.step(grads, lr=0.1)
        return opt, params, grads

    def replaced(opt, name):
        opt.state[name][1] = torch.zeros_like(opt.state[name][1])

    def storage(opt, name):
        opt.state[name][0].data = torch.zeros_like(opt.state[name][0])

    def a_list(opt, name):
        opt.state[name] = [t.clone() for t in opt.state[name]]

    def shorter(opt, name):
        opt.state[name] = opt.state[name][:1]

    def no_tensor(opt, name):
        opt.state[name][0] = None

    def parameter(opt, name):
        opt.params[1] = torch.ones(40, device="cuda")

    def no_states(opt, name):
        del opt.state[name]
    for change in (replaced, storage, a_list, shorter, no_tensor, parameter, no_states):
        for name in ("m", "v", "m_scale", "v_scale")[:4 if bits == 8 else 2]:
            opt, params, grads = made()
            before = [t.clone() for t in params]
            change(opt, name)
            with pytest.raises(nv.NVFP4Error):
                opt.step(grads, lr=0.1)
            assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(params, before))
    opt, params, grads = made()
    other, theirs, _ = made()
    other.step(grads, lr=0.1)
    for name, states in other.state.items():               # a checkpoint's values, copied in
        for a, b in zip(opt.state[name], states):
            a.copy_(b)
    opt.steps = other.steps
    for a, b in zip(params, theirs):
        a.copy_(b)
    opt.step(grads, lr=0.1)
    other.step(grads, lr=0.1)
    assert all(torch.equal(a, b) for a, b in zip(params, theirs))
    assert nv.status_query() == 0


def test_a_refused_gradient_leaves_the_next_step_whole(nv):
    """A list that is refused at its last entry has changed nothing of what the next step sees."""
    params = [torch.ones(300, device="cuda"), torch.ones(300, device="cuda")]
    want = [p.clone() for p in params]
    opt, ref = nv.AdamW(params), nv.AdamW(want)
    grads = [torch.randn(300, device="cuda") for _ in params]
    with pytest.raises(nv.NVFP4Error):
        opt.step([torch.ones(300, device="cuda", dtype=BF16), torch.ones(7, device="cuda")], lr=0.1)
    for o in (opt, ref):
        o.step([grads[0], None], lr=0.1)
        o.step([None, grads[1].bfloat16()], lr=0.1)
    assert all(torch.equal(a, b) for a, b in zip(params, want))
    assert not torch.equal(params[0], torch.ones_like(params[0])) and not torch.equal(params[1], torch.ones_like(params[1]))


def test_a_step_in_a_graph_is_refused(nv):
    """Replayed, it would be the same step number again: the same bias corrections and the same random bits."""
    p = torch.ones(300, device="cuda")
    opt, g = nv.AdamW([p], bits=8), torch.ones(300, device="cuda")
    opt.step([g], lr=0.1)
    before, side = p.clone(), torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.add_(1)
        with pytest.raises(nv.NVFP4Error):
            opt.step([g], lr=0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert opt.steps == 1 and torch.equal(p, before) and (side == 1).all()
    opt.step([g], lr=0.1)
    assert opt.steps == 2 and not torch.equal(p, before) and nv.status_query() == 0


def test_tensors_that_share_memory_are_refused(nv):
    """One launch updates all tensors at once: memory that two of them share would be updated by both, in any order.  Neighbours
    in one buffer are fine."""
    flat, other = torch.ones(600, device="cuda"), torch.ones(300, device="cuda")
    m, v = [torch.zeros(300, device="cuda") for _ in range(2)], [torch.zeros(300, device="cuda") for _ in range(2)]
    a, b = flat[:300], flat[300:]
    bad = [lambda: nv.AdamW([a, b, a]), lambda: nv.AdamW([flat, b]), lambda: nv.AdamW([a, flat[299:599]]),
           lambda: nv.AdamW([a, b], state={"m": [m[0], m[0]], "v": v}), lambda: nv.AdamW([a, b], state={"m": m, "v": m}),
           lambda: nv.AdamW([other], state={"m": [a], "v": [other]})]
    for k, fn in enumerate(bad):
        with pytest.raises(nv.NVFP4Error):
            fn()
    opt = nv.AdamW([a, b, torch.empty(0, device="cuda"), torch.empty(0, device="cuda")], state={
        "m": m + [torch.zeros(0, device="cuda")] * 2, "v": v + [torch.zeros(0, device="cuda")] * 2})
    opt.step([torch.ones_like(a), None, None, None], lr=0.1)
    assert (a < 1).all() and (b == 1).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_states_that_are_taken_over_are_the_objects_own(nv, bits):
    """Tensors given as ``state`` share their memory with the object's, which are what is updated and what a checkpoint stores, whatever
    becomes of the given ones."""
    def made(**kw):
        p = torch.ones(300, device="cuda")
        return nv.AdamW([p], bits=bits, **kw), p
    (first, p0), g = made(), torch.randn(300, device="cuda")
    first.step([g], lr=0.1)
    given = {k: [t.clone() for t in v] for k, v in first.state.items()}
    opt, p1 = made(state=given, steps=1)
    p1.copy_(p0)
    for name, states in given.items():
        assert opt.state[name][0].data_ptr() == states[0].data_ptr()
    opt, _ = made(state=given, steps=1)                    # its states are not read before the steps
    opt.params[0].copy_(p0)
    held = {name: states[0].data for name, states in given.items()}
    for name, states in given.items():
        states[0].data = torch.zeros_like(states[0])
        states[0] = None
    for o in (first, opt):
        o.step([g], lr=0.1)
    assert torch.equal(first.params[0], opt.params[0])
    for name in held:
        a, b, c = (t.view(torch.uint8) for t in (opt.state[name][0], first.state[name][0], held[name]))
        assert torch.equal(a, b) and torch.equal(a, c)
    opt.state["m"][0].data = torch.zeros_like(opt.state["m"][0])
    with pytest.raises(nv.NVFP4Error):
        opt.step([g], lr=0.1)
