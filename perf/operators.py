"""The operators around the NVFP4 linear layers of a transformer block's training step, as workloads:
layer norm (forward and backward), attention (forward, and the backward that recomputes the
probabilities) and the AdamW step over many tensors with states in 32 or 8 bits.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the calls a user makes of
``nvfp4_bit_quantized_gb300``.  ``exact`` computes the same results in 64 bits from the definitions."""
import math
import random

import torch

own = False

EPS = 1e-5                                              # layer norm
LR, BETAS, ADAM_EPS, DECAY = 3e-4, (0.9, 0.95), 1e-8, 0.1
SR_SEED = 20251


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # -- layer norm: one normalisation before a linear layer of the 5120-wide model
        # a handful of tokens (evaluation, a last short micro-batch): the launch is the cost
        dict(name="norm forward, few tokens", op="norm", back=False, rows=24, cols=5120, x="bf16", y="bf16", w="f32",
             bias=True, residual=False),
        # the residual stream of an 8192-token step: add, normalise, hand bf16 to the quantizer
        dict(name="norm forward, residual", op="norm", back=False, rows=8192, cols=5120, x="bf16", y="bf16", w="f32",
             bias=True, residual=True),
        # its gradient, with the residual branch's gradient joining at h
        dict(name="norm backward, residual", op="norm", back=True, rows=8192, cols=5120, x="bf16", y="bf16", w="f32",
             bias=True, residual=True),
        # fp32 activations of an odd width, weight only: no 16-byte rows
        dict(name="norm backward, odd fp32", op="norm", back=True, rows=4099, cols=1027, x="f32", y="f32", w="f32",
             bias=False, residual=False),
        # -- AdamW
        # one block of the 5120-wide model: the two MLP weights, the attention projections, norms; fp32
        # master weights, bf16 gradients from the Wgrad GEMM, fp32 states
        dict(name="adamw 32-bit, a block", op="adamw", bits=32, hidden=5120, ffn=20480, vectors=8, param="f32", grad="bf16"),
        # the same with 8-bit states and stochastic rounding
        dict(name="adamw 8-bit, a block", op="adamw", bits=8, hidden=5120, ffn=20480, vectors=8, param="f32", grad="bf16"),
        # only vectors of odd length (norm weights, biases) held in bf16: many small tensors, few bytes
        dict(name="adamw 8-bit, small odd tensors", op="adamw", bits=8, hidden=0, ffn=1027, vectors=48, param="bf16", grad="f32"),
        # -- attention on the fused QKV projection's output
        # 8192 tokens of one document, 40 query heads of 128 sharing 8 key heads
        dict(name="attention forward, long", op="attention", back=False, tq=8192, tk=8192, docs=1, heads=40, kv_heads=8,
             dim=128, causal=True),
        dict(name="attention backward, long", op="attention", back=True, tq=8192, tk=8192, docs=1, heads=40, kv_heads=8,
             dim=128, causal=True),
        # packed documents of uneven length, small heads
        dict(name="attention forward, packed", op="attention", back=False, tq=8192, tk=8192, docs=13, heads=32, kv_heads=32,
             dim=64, causal=True),
        dict(name="attention backward, packed", op="attention", back=True, tq=8191, tk=8191, docs=13, heads=32, kv_heads=8,
             dim=64, causal=True),
        # more queries than keys under a causal mask (the first queries see nothing), a head size that is no power of two
        dict(name="attention backward, short", op="attention", back=True, tq=213, tk=130, docs=1, heads=6, kv_heads=3,
             dim=80, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "adamw", "attention", "attention"))
    if op == "norm":
        cols = _log(rng, 33, 24000)
        if rng.random() < 0.6:
            cols = max(64, cols // 64 * 64)
        rows = _log(rng, 1, max(2, min(40000, 8192 * 5120 // cols)))
        return dict(op=op, back=rng.random() < 0.5, rows=rows, cols=cols, x=rng.choice(("bf16", "bf16", "f32")),
                    y=rng.choice(("bf16", "f32")), w=rng.choice(("f32", "bf16")), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "adamw":
        hidden = rng.choice((0, _log(rng, 100, 5000)))
        return dict(op=op, bits=rng.choice((8, 32)), hidden=hidden, ffn=_log(rng, 200, 20000), vectors=rng.randint(1, 60),
                    param=rng.choice(("f32", "bf16")), grad=rng.choice(("f32", "bf16")))
    tq = _log(rng, 1, 8000)
    kv = rng.choice((1, 2, 3, 4, 8))
    case = dict(op=op, back=rng.random() < 0.5, tq=tq, tk=tq if rng.random() < 0.7 else _log(rng, 1, 8000),
                docs=rng.choice((1, 1, rng.randint(2, 24))), heads=kv * rng.choice((1, 2, 4, 5)), kv_heads=kv,
                dim=rng.choice((16, 40, 64, 64, 72, 96, 104, 128, 128)), causal=rng.random() < 0.6)
    return case


# ----------------------------------------------------------------------------- what a case holds

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _bytes(t):
    return 4 if t == "f32" else 2


def _offsets(case):
    """Where each document begins among the queries and the keys: uneven lengths, some of them one or none."""
    r = random.Random(case["tq"] * 31 + case["docs"])

    def cut(total):
        at = sorted(r.randint(0, total) for _ in range(case["docs"] - 1))
        return [0] + at + [total]
    q = cut(case["tq"])
    return q, (q if case["tk"] == case["tq"] else cut(case["tk"]))


def _pairs(case):
    """Query-key pairs that the mask leaves."""
    oq, ok = _offsets(case)
    n = 0
    for i in range(case["docs"]):
        a, b = oq[i + 1] - oq[i], ok[i + 1] - ok[i]
        if not case["causal"]:
            n += a * b
        elif a <= b:
            n += a * b - a * (a - 1) // 2
        else:
            n += b * (b + 1) // 2
    return n


def _shapes(case):
    """Tensors of an AdamW case: a block's weights (fused QKV, attention output, MLP up and down), then vectors."""
    h, f = case["hidden"], case["ffn"]
    big = [(h + 2 * (h // 5), h), (h, h), (f, h), (h, f)] if h else []
    return big + [((h or f) + 3 * (i % 4),) for i in range(case["vectors"])]


def _sizes(case):
    return [math.prod(s) for s in _shapes(case)]


def work(case):
    if case["op"] == "norm":
        n, s = case["rows"] * case["cols"], 3 if case["back"] else 2
        per = _bytes(case["x"]) * (s - 1) + _bytes(case["y"])      # x (and dx), y or dy
        if case["residual"]:                                       # forward: residual in, h out; backward: dh in
            per += _bytes(case["x"]) * (1 if case["back"] else 2)
        vec = case["cols"] * (_bytes(case["w"]) * (1 if case["back"] else 1 + case["bias"])
                              + (4 * (1 + case["bias"]) if case["back"] else 0))
        return {"bytes": n * per + vec + 8 * case["rows"], "flops": n * (14 if case["back"] else 8)}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / 128
        return {"bytes": n * (2 * _bytes(case["param"]) + _bytes(case["grad"]) + state), "flops": n * 16}
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    q, kv = case["tq"] * hq * d, case["tk"] * hk * d
    rows = 4 * case["tq"] * hq
    if case["back"]:
        return {"bytes": 2 * (4 * q + 4 * kv) + rows, "flops": 10 * _pairs(case) * d * hq}
    return {"bytes": 2 * (2 * q + 2 * kv) + rows, "flops": 4 * _pairs(case) * d * hq}


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        xt, yt, wt = DT[case["x"]], DT[case["y"]], DT[case["w"]]
        # a residual stream: channels of unequal size, a few of them large, an offset for each token
        x = (randn(rows, cols) * (0.5 + randn(cols).abs()) + 0.3 * randn(rows, 1)).to(xt)
        s = {"case": case, "x": x, "weight": (1 + 0.2 * randn(cols)).to(wt), "bias": None, "residual": None, "dh": None}
        if case["bias"]:
            s["bias"] = (0.1 * randn(cols)).to(wt)
        if not case["back"]:
            if case["residual"]:
                s["residual"] = randn(rows, cols).to(xt)
            return s
        # the backward pass has h (x here) and the statistics that the forward pass kept
        xf = x.float()
        s["mean"] = xf.mean(1)
        s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
        s["dy"] = (1e-2 * randn(rows, cols)).to(yt)
        if case["residual"]:
            s["dh"] = (1e-2 * randn(rows, cols)).to(xt)
        return s

    if case["op"] == "adamw":
        # the tensors are views of flat buffers, as training programs keep them; each begins on a block of 128
        sizes, shapes = _sizes(case), _shapes(case)
        at, end = [], 0
        for n in sizes:
            at.append(end)
            end += (n + 127) // 128 * 128
        flat = {"param": torch.zeros(end, device="cuda"), "grad": torch.zeros(end, device="cuda"),
                "m": torch.zeros(end, device="cuda"), "v": torch.zeros(end, device="cuda")}
        for a, n in zip(at, sizes):
            flat["param"][a:a + n] = 0.02 * randn(n)
            size = 1e-3 * torch.exp(randn(n))               # gradients of unequal size, as a step in mid-training has them
            flat["grad"][a:a + n] = size * randn(n)
            flat["m"][a:a + n] = 0.3 * size * randn(n)
            flat["v"][a:a + n] = size.square() * (0.5 + torch.rand(n, generator=g, device="cuda"))
        flat["param"], flat["grad"] = flat["param"].to(DT[case["param"]]), flat["grad"].to(DT[case["grad"]])
        if case["bits"] == 8:
            for name in ("m", "v"):
                x = flat[name].view(-1, 128)
                scale = x.abs().amax(1) / 448.0
                flat[name] = (x / scale.clamp_min(1e-38)[:, None]).view(-1).to(torch.float8_e4m3fn)
                flat[name + "_scale"] = scale
        s = {"case": case, "flat": flat, "at": at, "sizes": sizes, "steps": 1000,
             "decay": [DECAY if len(sh) > 1 else 0.0 for sh in shapes], "grad_scale": torch.full((1,), 0.75, device="cuda")}
        s["begins"] = torch.tensor(at + [end], device="cuda")
        s["decays"] = torch.tensor(s["decay"], dtype=torch.float64, device="cuda")

        def views(name):
            if name.endswith("_scale"):
                return [flat[name][a // 128:(a + n + 127) // 128] for a, n in zip(at, sizes)]
            return [flat[name][a:a + n].view(sh) for a, n, sh in zip(at, sizes, shapes)]
        s["views"] = {name: views(name) for name in flat}
        if own:                                             # the optimizer object that a program keeps
            import nvfp4_bit_quantized_gb300 as nv
            s["opt"] = nv.AdamW(s["views"]["param"], bits=case["bits"], weight_decay=s["decay"], steps=s["steps"],
                                state={k: v for k, v in s["views"].items() if k not in ("param", "grad")})
        return s

    hq, hk, d, tq, tk = case["heads"], case["kv_heads"], case["dim"], case["tq"], case["tk"]
    oq, ok = _offsets(case)

    def offsets(o):
        return torch.tensor(o, dtype=torch.int32, device="cuda")

    # q, k and v are slices of one fused projection's output where queries and keys are the same tokens
    def heads(rows, n, spread):
        return (spread * randn(rows, n, d) + 0.4 * randn(n, d)).bfloat16()
    if tq == tk:
        qkv = torch.empty(tq, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q = torch.empty(tq, hq, d, dtype=torch.bfloat16, device="cuda")
        kv = torch.empty(tk, 2 * hk, d, dtype=torch.bfloat16, device="cuda")
        k, v = kv[:, :hk], kv[:, hk:]
    q.copy_(heads(tq, hq, 1.4)), k.copy_(heads(tk, hk, 1.2)), v.copy_(heads(tk, hk, 1.0))
    s = {"case": case, "q": q, "k": k, "v": v, "scale": 1 / math.sqrt(d)}
    many = case["docs"] > 1
    s["cu_q"], s["cu_k"] = (offsets(oq), offsets(ok)) if many else (None, None)
    if case["back"]:                                        # what the forward pass kept, and the gradient that arrives
        s["out"], s["lse"] = _attention(s)
        s["dout"] = (1e-2 * randn(tq, hq, d)).bfloat16()
        if tq == tk:                                        # the gradients fill one buffer: the projection's dY
            s["grads"] = {"dqkv": torch.empty_like(qkv)}
            w = s["grads"]["dqkv"]
            s["dq"], s["dk"], s["dv"] = w[:, :hq], w[:, hq:hq + hk], w[:, hq + hk:]
        else:
            s["dq"], dkv = torch.empty_like(q), torch.empty_like(kv)
            s["grads"] = {"dq": s["dq"], "dkv": dkv}
            s["dk"], s["dv"] = dkv[:, :hk], dkv[:, hk:]
    return s


# ----------------------------------------------------------------------------- the plain forms

def _norm(s):
    x = s["x"].float()
    h = x
    if s["residual"] is not None:
        h = (x + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(1) + EPS)
    y = centred * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"y": y.to(DT[s["case"]["y"]]), "mean": mean, "rstd": rstd}
    return dict(out, h=h) if s["residual"] is not None else out


def _norm_backward(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    out = {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0)}
    return dict(out, dbias=dy.sum(0)) if s["bias"] is not None else out


def random_words(group, stream, step):
    """The random inputs of stochastic rounding: the four 32-bit words of Philox4x32-10 (Salmon et al., SC'11) with
    counter (group, stream, step), for elements 4 group .. 4 group + 3 of the tensor that the stream belongs to."""
    low = 0xFFFFFFFF
    c = [group & low, group >> 32, stream + torch.zeros_like(group), torch.full_like(group, step)]
    k0, k1 = SR_SEED & low, SR_SEED >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, 1).view(-1)


def _to_e4m3(x, rand16, floor):
    """Values of the E4M3 grid's range, stochastically rounded to it: scaled by 2^-120 the grid's exponents and its
    subnormals are fp32's, so the code is the top of the fp32 word."""
    bits = (x.abs() * 2.0 ** -120).view(torch.int32)
    code = torch.clamp((bits + (rand16 << 4).int()) >> 20, max=126)
    if floor:
        code = torch.where((x > 0) & (code == 0), 1, code)
    return (code | torch.where(torch.signbit(x), 128, 0)).to(torch.uint8).view(torch.float8_e4m3fn)


def _quantize8(x, rand16, floor):
    blocks = x.view(-1, 128)
    top = blocks.abs().amax(1)
    inv = torch.where(top > 0, torch.clamp(torch.full_like(top, 448.0) / top, max=torch.finfo(torch.float32).max), 0.0)
    return _to_e4m3((blocks * inv[:, None]).view(-1), rand16, floor), top * (1 / 448)


def _dequantize8(code, scale):
    return (code.float().view(-1, 128) * scale[:, None]).view(-1)


def _adamw(s):
    """Over the flat buffers: what lies between the tensors is zero and stays zero."""
    case, flat = s["case"], s["flat"]
    s["steps"] += 1
    t, (b1, b2) = s["steps"], BETAS
    size, unbias = LR / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
    ends = s["begins"][1:]
    owner = torch.searchsorted(ends, torch.arange(0, flat["param"].numel(), 4, device="cuda"), right=True)
    group = torch.arange(len(owner), device="cuda") - s["begins"][owner] // 4
    keep = (1 - LR * s["decays"])[owner].repeat_interleave(4).float()
    g = flat["grad"].float() * s["grad_scale"]
    if case["bits"] == 8:
        m, v = _dequantize8(flat["m"], flat["m_scale"]), _dequantize8(flat["v"], flat["v_scale"])
    else:
        m, v = flat["m"], flat["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    new = flat["param"].float() * keep - m * size / (v.sqrt() * unbias + ADAM_EPS)
    if case["param"] == "bf16":
        bits = new.view(torch.int32) + (random_words(group, 2 * owner + 1, t) & 0xFFFF).int()
        new = (bits & -65536).view(torch.float32).bfloat16()
    flat["param"].copy_(new)
    if case["bits"] == 8:
        w = random_words(group, 2 * owner, t)
        for name, x, rand, floor in (("m", m, w & 0xFFFF, False), ("v", v, w >> 16, True)):
            code, scale = _quantize8(x, rand, floor)
            flat[name].copy_(code), flat[name + "_scale"].copy_(scale)
    else:
        flat["m"].copy_(m), flat["v"].copy_(v)
    return {name: x for name, x in flat.items() if name != "grad"}


def _mask(s):
    """[tq, tk]: which pairs attend."""
    case = s["case"]
    q, k = (torch.arange(case[t], device="cuda") for t in ("tq", "tk"))
    if s["cu_q"] is None:
        return (k[None] - case["tk"] <= q[:, None] - case["tq"]) if case["causal"] else torch.ones(
            len(q), len(k), dtype=torch.bool, device="cuda")
    dq, dk = (torch.searchsorted(s[c][1:].long(), x, right=True) for c, x in (("cu_q", q), ("cu_k", k)))
    same = dq[:, None] == dk[None]
    if not case["causal"]:
        return same
    # positions counted from the end of their document: a query sees the keys that are no later than itself
    return same & ((k - s["cu_k"][1:].long()[dk])[None] <= (q - s["cu_q"][1:].long()[dq])[:, None])


def _logits(s):
    """Scaled scores [heads, tq, tk] with minus infinity where nothing attends; keys repeated for their heads."""
    share = s["case"]["heads"] // s["case"]["kv_heads"]
    q = s["q"].float().transpose(0, 1)
    k, v = (s[n].float().transpose(0, 1).repeat_interleave(share, 0) for n in ("k", "v"))
    scores = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    return q, k, v, torch.where(_mask(s), scores, -torch.inf)


def _attention(s):
    _, _, v, scores = _logits(s)
    top = scores.amax(2, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out.transpose(0, 1).to(torch.bfloat16), (torch.log(total) + top).squeeze(2)


def _attention_backward(s):
    case = s["case"]
    share = case["heads"] // case["kv_heads"]
    q, k, v, scores = _logits(s)
    do, out = s["dout"].float().transpose(0, 1), s["out"].float().transpose(0, 1)
    lse = torch.where(s["lse"] == -torch.inf, 0.0, s["lse"])
    p = torch.exp(scores - lse[:, :, None])
    del scores
    delta = (do * out).sum(2, keepdim=True)
    dv = torch.matmul(p.transpose(1, 2), do)
    ds = p * (torch.matmul(do, v.transpose(1, 2)) - delta) * s["scale"]
    del p
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(1, 2), q)
    dk, dv = (x.view(-1, share, *x.shape[1:]).sum(1) for x in (dk, dv))
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        s[name].copy_(x.transpose(0, 1))
    return s["grads"]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "adamw":
            return _adamw(s)
        if case["op"] == "norm":
            return _norm_backward(s) if case["back"] else _norm(s)
        if case["back"]:
            return _attention_backward(s)
        out, lse = _attention(s)
        return {"out": out, "lse": lse}
    import nvfp4_bit_quantized_gb300 as nv
    if case["op"] == "adamw":
        s["opt"].step(s["views"]["grad"], lr=LR, betas=BETAS, eps=ADAM_EPS, grad_scale=s["grad_scale"], round=nv.SR,
                      sr_seed=SR_SEED)
        return {name: x for name, x in s["flat"].items() if name != "grad"}
    if case["op"] == "norm":
        if case["back"]:
            dx, dw, db = nv.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dh=s["dh"],
                                                bias=case["bias"])
            return {"dx": dx, "dweight": dw, "dbias": db} if case["bias"] else {"dx": dx, "dweight": dw}
        y, mean, rstd, h = nv.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"],
                                                 out_dtype=DT[case["y"]])
        out = {"y": y, "mean": mean, "rstd": rstd}
        return dict(out, h=h) if case["residual"] else out
    mask = dict(causal=case["causal"], scale=s["scale"], cu_q=s["cu_q"], cu_k=s["cu_k"])
    if not case["back"]:
        out, lse = nv.attention_forward(s["q"], s["k"], s["v"], **mask)
        return {"out": out, "lse": lse}
    nv.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], dq=s["dq"], dk=s["dk"], dv=s["dv"], **mask)
    return s["grads"]


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "adamw":
        # the largest tensors would take over 20 seconds in 64 bits with their random words
        return None if sum(s["sizes"]) > 3e8 else _exact_adamw(s)
    return _exact_attention(s)


def _exact_norm(s):
    case, x, w = s["case"], s["x"].double(), s["weight"].double()
    if not case["back"]:
        h = None
        if case["residual"]:
            h = (x + s["residual"].double()).to(s["x"].dtype)     # the statistics are those of the stored sum
            x = h.double()
        mean = x.mean(1)
        var = ((x - mean[:, None]) ** 2).mean(1)
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * w + (s["bias"].double() if case["bias"] else 0)
        out = {"y": y, "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
        return dict(out, h=h.double()) if case["residual"] else out
    # through the Jacobian of the normalisation at the statistics that came in
    dy, n = s["dy"].double(), case["cols"]
    rstd, centred = s["rstd"].double()[:, None], x - s["mean"].double()[:, None]
    a = dy * w
    dx = a * rstd - rstd * a.sum(1, keepdim=True) / n - centred * rstd ** 3 * (a * centred).sum(1, keepdim=True) / n
    if case["residual"]:
        dx = dx + s["dh"].double()
    out = {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, centred * rstd)}
    return dict(out, dbias=dy.sum(0)) if case["bias"] else out


def _grid(value, rand16, floor):
    """Stochastic rounding of values to the E4M3 grid {0, k 2^-9, ...}: up where position + rand16 / 2^16 reaches the
    next grid point."""
    a = value.abs().clamp(max=448.0)
    exponent = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    spacing = torch.exp2(exponent - 3)
    steps = a / spacing
    up = torch.floor(steps) + ((steps - torch.floor(steps)) + rand16.double() / 65536 >= 1).double()
    q = (up * spacing).clamp(max=448.0)
    if floor:
        q = torch.where((a > 0) & (q == 0), 2.0 ** -9, q)
    return torch.copysign(q, value)


def _exact_adamw(s):
    case, views, out = s["case"], s["views"], {}
    total = s["flat"]["param"].numel()
    for name, x in s["flat"].items():
        if name != "grad":
            out[name] = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    t, (b1, b2) = s["steps"] + 1, BETAS
    for i, (a, n, decay) in enumerate(zip(s["at"], s["sizes"], s["decay"])):
        def get(name):
            return views[name][i].reshape(-1).float().double()
        g = get("grad") * 0.75
        blocks, groups = torch.arange(n, device="cuda") // 128, torch.arange((n + 3) // 4, device="cuda")
        if case["bits"] == 8:
            m, v = get("m") * get("m_scale")[blocks], get("v") * get("v_scale")[blocks]
        else:
            m, v = get("m"), get("v")
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
        step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM_EPS)
        p = get("param")
        p = p - LR * decay * p - LR * step
        if case["param"] == "bf16":                          # bf16 keeps 8 bits of the significand
            spacing = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
            k = p.abs() / spacing
            frac = k - torch.floor(k)
            k = torch.floor(k) + (frac + (random_words(groups, 2 * i + 1, t)[:n] & 0xFFFF).double() / 65536 >= 1)
            p = torch.copysign(k * spacing, p)
        out["param"][a:a + n] = p
        if case["bits"] == 8:
            w = random_words(groups, 2 * i, t)[:n]
            for name, x, rand, floor in (("m", m, w & 0xFFFF, False), ("v", v, w >> 16, True)):
                top = torch.zeros((n + 127) // 128, dtype=torch.float64, device="cuda")
                top.scatter_reduce_(0, blocks, x.abs(), "amax")
                out[name + "_scale"][a // 128:a // 128 + len(top)] = top / 448
                out[name][a:a + n] = _grid(x / (top / 448).clamp(min=1e-300)[blocks], rand, floor)
        else:
            out["m"][a:a + n], out["v"][a:a + n] = m, v
    assert total == s["flat"]["param"].numel()
    return out


def _exact_attention(s):
    """Head by head from the definition: softmax of the scaled scores over the keys of the query's document, no later
    than the query where causal, both counted from the document's end."""
    case = s["case"]
    share, oq, ok = case["heads"] // case["kv_heads"], *_offsets(case)
    out = torch.zeros(case["tq"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], case["tq"]), -torch.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(case["tk"], case["kv_heads"], case["dim"], dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for i in range(case["docs"]):
        a, b = slice(oq[i], oq[i + 1]), slice(ok[i], ok[i + 1])
        rows, cols = oq[i + 1] - oq[i], ok[i + 1] - ok[i]
        if not rows or not cols:
            continue
        hidden = None
        if case["causal"]:
            hidden = torch.arange(cols, device="cuda")[None] > torch.arange(rows, device="cuda")[:, None] + cols - rows
        for h in range(case["heads"]):
            q, k, v = s["q"][a, h].double(), s["k"][b, h // share].double(), s["v"][b, h // share].double()
            z = q @ k.T * s["scale"]
            if hidden is not None:
                z.masked_fill_(hidden, -torch.inf)
            norm = torch.logsumexp(z, 1)
            p = torch.exp(z - norm[:, None])
            if hidden is not None:
                p.masked_fill_(hidden, 0.0)                   # also the rows that see nothing
            o = p @ v
            out[a, h], lse[h, a] = o, norm
            if case["back"]:
                do = s["dout"][a, h].double()
                dv[b, h // share] += p.T @ do
                dp = do @ v.T
                dz = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                dq[a, h] = dz @ k
                dk[b, h // share] += dz.T @ q
    if not case["back"]:
        return {"out": out, "lse": lse}
    if case["tq"] == case["tk"]:
        return {"dqkv": torch.cat([dq, dk, dv], 1)}
    return {"dq": dq, "dkv": torch.cat([dk, dv], 1)}
