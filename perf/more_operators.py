"""The 8-bit layers, the router's balance loss and the LM head's cross entropy: cases, plain forms and calls.

Five operators are covered, each by the call that a training or serving
program makes of it:

  quantize         8-bit images of a list of matrices with a scale for each
                   block of 128, read back as the values they stand for;
  linear           y = x W^T with x quantised on the way and W held in 8 bits;
  linear_backward  dx and dW of that layer from dy and the saved images;
  balance          the balance loss of a router, its experts' counts, and the
                   gradient for the router's logits;
  cross_entropy    the softmax cross entropy of an LM head from its input and
                   its weights, with the gradients of both.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` is the definition in 64
bits.  The 8-bit format: blocks of 128 along a row (in a square image: of 128
rows by 128 columns) share a power of two 2^e, e the smallest integer, at least
-127, with max|x| <= 448 2^e, stored as e + 127 in a byte; an element is an
e4m3 number (1 sign, 4 exponent and 3 mantissa bits, subnormals, largest 448),
rounded to nearest, ties to even.  An image of [R, C] is codes [R, 128 nb] (nb =
ceil(C / 128)) and scales [R, 16 ceil(nb / 16)]; padding is zero.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------- cases
def listed():
    """The measured cases, from single tokens to whole layers and batches."""
    return [
        # one token's activations on their way into an 8-bit layer: pure latency
        {"name": "quantize_one_token", "op": "quantize", "shapes": "1x2048", "dtype": "bf16", "both": False, "square": False},
        # the matrices of 8 experts, both orientations, as after an optimizer step
        {"name": "quantize_experts", "op": "quantize", "dtype": "f32", "both": True, "square": True,
         "shapes": ",".join(["2048x1408,2048x1408,1408x2048"] * 8)},
        # decoding one sequence through the large model's wide matrix: the weights' bytes are all there is
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "n": 28672, "k": 8192, "dtype": "bf16", "out": "bf16"},
        # a ragged batch of sequences through an expert, odd sizes on every axis
        {"name": "linear_ragged_batch", "op": "linear", "tokens": 77, "n": 1407, "k": 2045, "dtype": "bf16", "out": "f32"},
        # prefill or a training forward of the large model's wide matrix
        {"name": "linear_large", "op": "linear", "tokens": 8192, "n": 28672, "k": 8192, "dtype": "bf16", "out": "bf16"},
        # a training backward of the 1.5B model's MLP
        {"name": "backward_mlp", "op": "linear_backward", "tokens": 8192, "n": 5632, "k": 2048, "dtype": "bf16", "out": "bf16"},
        # an expert's backward over the odd number of tokens that the router sent it
        {"name": "backward_expert_odd", "op": "linear_backward", "tokens": 997, "n": 1408, "k": 2048, "dtype": "f32", "out": "f32"},
        # the router's choices of a few tokens, some of them padding
        {"name": "balance_few_tokens", "op": "balance", "tokens": 37, "experts": 64, "top": 6, "pad": 0, "dtype": "bf16"},
        # a training batch of sequences through the router of 64 experts
        {"name": "balance_batch", "op": "balance", "tokens": 65536, "experts": 64, "top": 6, "pad": 0, "dtype": "f32"},
        # scoring the next token of a few sequences while serving: no gradients, the head is read once
        {"name": "cross_entropy_few_rows", "op": "cross_entropy", "rows": 3, "hidden": 2048, "vocab": 32000, "pad": 0, "x": "bf16",
         "w": "bf16", "dw": "bf16", "grad": False},
        # the LM head of a training batch
        {"name": "cross_entropy_batch", "op": "cross_entropy", "rows": 8192, "hidden": 2048, "vocab": 32000, "pad": 0, "x": "bf16",
         "w": "bf16", "dw": "bf16", "grad": True},
        # a ragged batch against a long odd vocabulary held in 32 bits, whose gradient an optimizer takes in 32 bits
        {"name": "cross_entropy_long_odd", "op": "cross_entropy", "rows": 1021, "hidden": 2045, "vocab": 129283, "pad": 3, "x": "bf16",
         "w": "f32", "dw": "f32", "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["quantize", "linear", "linear", "linear_backward", "balance", "cross_entropy", "cross_entropy"])
    if op == "quantize":
        shapes = []
        for _ in range(rng.randint(1, 6)):
            r, c = _log(rng, 1, 8192), _log(rng, 16, 8192)
            shapes.append("%dx%d" % (r, c))
        return {"op": op, "shapes": ",".join(shapes), "dtype": rng.choice(["f32", "bf16"]), "both": rng.random() < 0.5,
                "square": rng.random() < 0.5}
    if op in ("linear", "linear_backward"):
        tokens, n, k = _log(rng, 1, 8192), _log(rng, 64, 16384 if op == "linear" else 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:
            n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64
        return {"op": op, "tokens": tokens, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"])}
    if op == "balance":
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": min(_log(rng, 1, 262144), (1 << 23) // experts), "experts": experts,
                "top": rng.randint(1, min(8, experts)), "pad": rng.choice([0, 0, 1, 8]), "dtype": rng.choice(["f32", "bf16"])}
    vocab, hidden = _log(rng, 500, 160000), _log(rng, 64, 8192)
    if rng.random() < 0.5:
        hidden = (hidden + 63) // 64 * 64
    rows = max(1, min(_log(rng, 1, 8192), 8192 * 2048 * 32000 // (vocab * hidden)))
    w = rng.choice(["bf16", "bf16", "f32"])
    return {"op": op, "rows": rows, "hidden": hidden, "vocab": vocab, "pad": rng.choice([0, 0, 1, 16]),
            "x": rng.choice(["bf16", "bf16", "f32"]), "w": w, "dw": rng.choice(["bf16", "f32"]), "grad": rng.random() < 0.75}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _image_bytes(r, c):
    return r * (c + -(-c // 128))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, t, c, dt):
    """Normal values whose channels differ in scale, a few of them strongly."""
    s = torch.exp(0.5 * torch.randn(c, generator=g, device="cuda"))
    s = torch.where(torch.rand(c, generator=g, device="cuda") < 0.01, s * 20.0, s)
    return (torch.randn(t, c, generator=g, device="cuda") * s).to(dt)


def prepare(case, seed):
    """Inputs on the GPU and the 8-bit images that a program keeps between calls."""
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        dt = _DT[case["dtype"]]
        st["mats"] = [(torch.randn(r, c, generator=g, device="cuda") * 0.02).to(dt) for r, c in _shapes(case)]
    elif op == "linear":
        st["x"] = _activations(g, case["tokens"], case["k"], _DT[case["dtype"]])
        st["w"] = _pack(torch.randn(case["n"], case["k"], generator=g, device="cuda") * 0.02, True)
    elif op == "linear_backward":
        dt = _DT[case["dtype"]]
        st["dy"] = (torch.randn(case["tokens"], case["n"], generator=g, device="cuda") * 1e-3).to(dt)
        st["x_t"] = _pack(_activations(g, case["tokens"], case["k"], dt).float().t().contiguous(), False)
        st["w_t"] = _pack(torch.randn(case["k"], case["n"], generator=g, device="cuda") * 0.02, True)
    elif op == "balance":
        t, e, k = case["tokens"], case["experts"], case["top"]
        z = torch.randn(t, e + case["pad"], generator=g, device="cuda") * (0.5 + torch.rand(t, 1, generator=g, device="cuda"))
        z[:, :e] += torch.randn(e, generator=g, device="cuda")             # experts that are liked more than others
        st["z"] = z.to(_DT[case["dtype"]])[:, :e]
        _, idx = torch.topk(st["z"].float() + 0.1 * torch.randn(t, e, generator=g, device="cuda"), k, dim=1)
        r = torch.rand(t, 1, generator=g, device="cuda")
        idx = torch.where(r < 0.04, torch.full_like(idx, -1), idx)         # positions behind a sequence's end
        idx[:, -1:] = torch.where((r > 0.98) & (k > 1), torch.full_like(idx[:, -1:], -1), idx[:, -1:])   # a dropped choice
        st["idx"] = idx.contiguous()
        st["g"] = torch.full((), 0.5, device="cuda")
    else:
        t, h, v = case["rows"], case["hidden"], case["vocab"]
        w = torch.randn(v, h, generator=g, device="cuda") * 0.02
        st["w"] = w.to(_DT[case["w"]])
        tgt = torch.randint(0, v, (t,), generator=g, device="cuda")
        x = torch.randn(t, h + case["pad"], generator=g, device="cuda")
        lift = torch.rand(t, 1, generator=g, device="cuda") * 12.0          # from surprising to certain tokens
        x[:, :h] += w[tgt] * (lift / (4e-4 * h))
        st["x"] = x.to(_DT[case["x"]])[:, :h]
        skip = torch.rand(t, generator=g, device="cuda") < 0.03             # prompts and padding
        skip[0] = False
        st["t"] = torch.where(skip, torch.full_like(tgt, -1), tgt)
        st["g"] = torch.full((t,), 1.0 / max(1, t - int(skip.sum())), device="cuda")
        # the buffer that the head's gradient goes to, where it is not of the weights' type
        st["dw"] = torch.empty(v, h, dtype=_DT[case["dw"]], device="cuda") if case["grad"] and case["dw"] != case["w"] else None
    if own:
        import matrix_orthogonalizing_optimizer_amd as mo
        for name, cols in (("w", case.get("k")), ("x_t", case.get("tokens")), ("w_t", case.get("n"))):
            if isinstance(st.get(name), tuple):
                st[name] = mo.Fp8Matrix(st[name][0], st[name][1], cols)
    return st


# -------------------------------------------------------------- plain forms
def _two_to(e):
    """2^e of integers in [-127, 127], exactly (a pow is not), from its bits."""
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _scales(x, square):
    """Exponent of each block of 128 of [r, c] (fp32), [r, nb]."""
    r, c = x.shape
    nb, rb = -(-c // 128), -(-r // 128)
    p = torch.zeros(rb * 128 if square else r, nb * 128, dtype=torch.float32, device=x.device)
    p[:r, :c] = x
    if square:
        a = p.view(rb, 128, nb, 128).abs().amax((1, 3)).repeat_interleave(128, 0)[:r]
    else:
        a = p.view(r, nb, 128).abs().amax(2)
    m, e = torch.frexp(a)                                   # a = m 2^e with m in [0.5, 1); 448 = 0.875 2^9
    e = e - 9 + (m > 0.875).int()
    return torch.where(a == 0, torch.full_like(e, -127), e).clamp(min=-127), p[:r]


def _rounded(x, square):
    """(e4m3 values of the scaled elements [r, nb, 128], exponents [r, nb])."""
    e, p = _scales(x, square)
    t = p.view(x.shape[0], -1, 128) * _two_to(-e)[:, :, None]
    step = _two_to(torch.frexp(t)[1].clamp(min=-5) - 4)      # 8 steps to a binade, subnormals below 2^-6
    return torch.round(t / step) * step, e


def _quantized(x, square=False):
    v, e = _rounded(x.float(), square)
    return (v * _two_to(e)[:, :, None]).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _pack(x, square):
    """The stored image of [r, c]."""
    v, e = _rounded(x, square)
    m = v.abs()
    ex = torch.frexp(m)[1].clamp(min=-5)                     # binade 2^(ex - 1), -5 for the subnormals' step too
    man = (m / _two_to(ex - 4)).int()                        # 8 to 15, less than 8 for subnormals
    code = torch.where(man >= 8, ((ex + 6) << 3) + man - 8, man) + (torch.signbit(v).int() << 7)
    r, nb = e.shape
    scales = torch.zeros(r, -(-nb // 16) * 16, dtype=torch.uint8, device=x.device)
    scales[:, :nb] = (e + 127).to(torch.uint8)
    return code.to(torch.uint8).view(r, nb * 128), scales


def _stored_values(image, cols):
    codes, scales = image
    r, nb = codes.shape[0], -(-cols // 128)
    c = codes.view(r, nb, 128).int()
    ex, man = (c >> 3) & 15, c & 7
    v = torch.where(ex > 0, man + 8, man).float() * _two_to(ex.clamp(min=1) - 10)
    v = torch.where(c >= 128, -v, v) * _two_to(scales[:, :nb].int() - 127)[:, :, None]
    return v.reshape(r, -1)[:, :cols]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        out = []
        for x in st["mats"]:
            out.append(_quantized(x, case["square"]).to(torch.bfloat16))
            if case["both"]:
                out.append(_quantized(x.t(), case["square"]).to(torch.bfloat16))
        return out
    if op == "linear":
        return _quantized(st["x"]).matmul(_stored_values(st["w"], case["k"]).t()).to(_DT[case["out"]])
    if op == "linear_backward":
        dy = st["dy"]
        dx = _quantized(dy).matmul(_stored_values(st["w_t"], case["n"]).t())
        dw = _quantized(dy.t()).matmul(_stored_values(st["x_t"], case["tokens"]).t())
        return dx.to(_DT[case["out"]]), dw
    if op == "balance":
        z, idx = st["z"].float(), st["idx"]
        e = z.shape[1]
        live = (idx >= 0).any(1)
        n = live.sum().clamp(min=1).float()
        counts = torch.zeros(e + 1, dtype=torch.int64, device=z.device)
        counts.scatter_add_(0, torch.where(idx < 0, torch.full_like(idx, e), idx).view(-1), torch.ones_like(idx).view(-1))
        counts = counts[:e]
        f = counts.float() * e / counts.sum().clamp(min=1).float()
        ex = torch.exp(z - z.amax(1, keepdim=True))
        p = torch.where(live[:, None], ex / ex.sum(1, keepdim=True), torch.zeros_like(z))
        loss = 0.01 * (f * (p.sum(0) / n)).sum()
        grad = p * (f - (p * f).sum(1, keepdim=True)) * (0.01 * st["g"] / n)
        return loss, counts, grad.to(st["z"].dtype)
    x, w = st["x"].bfloat16().float(), st["w"].bfloat16().float()           # the products take 16-bit operands
    t = st["t"]
    live = t >= 0
    at = t.clamp(min=0)[:, None]
    z = x.matmul(w.t())
    m = z.amax(1, keepdim=True)
    ex = torch.exp(z - m)
    s = ex.sum(1, keepdim=True)
    loss = (m + torch.log(s) - z.gather(1, at))[:, 0]
    loss = torch.where(live, loss, torch.zeros_like(loss))
    if not case["grad"]:
        return loss
    p = ex / s
    p.scatter_add_(1, at, torch.full_like(s, -1.0))
    p = p * torch.where(live, st["g"], torch.zeros_like(loss))[:, None]
    return loss, p.matmul(w).to(st["x"].dtype), p.t().matmul(x).to(_DT[case["dw"]])


def _own(st):
    import matrix_orthogonalizing_optimizer_amd as mo
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q = mo.fp8_quantize(st["mats"], images="both" if case["both"] else "rows", square=case["square"])
        return mo.fp8_dequantize([i for pair in q for i in pair] if case["both"] else q)
    if op == "linear":
        return mo.fp8_linear(st["x"], st["w"], out_dtype=_DT[case["out"]])
    if op == "linear_backward":
        return mo.fp8_linear_backward(st["dy"], st["x_t"], st["w_t"], dx_dtype=_DT[case["out"]])
    if op == "balance":
        r = mo.balance_loss(st["z"], st["idx"], weight=0.01, grad_loss=st["g"])
        return r.loss, r.counts, r.grad
    if not case["grad"]:
        return mo.linear_cross_entropy(st["x"], st["w"], st["t"], grad=False)[0]
    return mo.linear_cross_entropy(st["x"], st["w"], st["t"], grad_loss=st["g"], dw=st["dw"])


def run(state):
    """One pass through the case's operator."""
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    if op == "quantize":
        s, b, f = _SIZE[case["dtype"]], 0, 0
        for r, c in _shapes(case):
            b += r * c * s + _image_bytes(r, c) + 2 * r * c
            f += 4 * r * c
            if case["both"]:
                b += _image_bytes(c, r) + 2 * r * c
                f += 4 * r * c
        return {"bytes": b, "flops": f}
    if op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": t * k * _SIZE[case["dtype"]] + _image_bytes(n, k) + t * n * _SIZE[case["out"]], "flops": 2 * t * n * k}
    if op == "linear_backward":
        t, n, k = case["tokens"], case["n"], case["k"]
        b = t * n * _SIZE[case["dtype"]] + _image_bytes(k, t) + _image_bytes(k, n) + t * k * _SIZE[case["out"]] + n * k * 4
        return {"bytes": b, "flops": 4 * t * n * k}
    if op == "balance":
        t, e = case["tokens"], case["experts"]
        return {"bytes": t * (2 * e * _SIZE[case["dtype"]] + 8 * case["top"]) + 8 * e, "flops": 10 * t * e}
    t, h, v = case["rows"], case["hidden"], case["vocab"]
    b = t * h * _SIZE[case["x"]] + v * h * _SIZE[case["w"]] + 12 * t
    if case["grad"]:
        b += t * h * _SIZE[case["x"]] + v * h * _SIZE[case["dw"]] + 4 * t
    return {"bytes": b, "flops": (6 if case["grad"] else 2) * t * v * h}


# ------------------------------------------------- the definition in 64 bits
def _exact_two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_table(device):
    """The 127 magnitudes that are numbers, in the order of their codes."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7) for c in range(127)],
                        dtype=torch.float64, device=device)


def _exact_quantized(x, square=False):
    """Blocks scaled, each element to the nearer of its neighbours in the table, halves to the even code."""
    x = x.double()
    r, c = x.shape
    p = torch.nn.functional.pad(x, (0, -c % 128, 0, (-r % 128) if square else 0))
    k = 128 if square else 1
    b = p.reshape(p.shape[0] // k, k, -1, 128)
    a = b.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448.0))
    e = torch.where(448.0 * _exact_two_to(e - 1) >= a, e - 1, e)             # log2 next to a whole number
    e = torch.where(448.0 * _exact_two_to(e) < a, e + 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, -127.0)).clamp(min=-127)
    t = b / _exact_two_to(e)
    table = _e4m3_table(x.device)
    hi = torch.searchsorted(table, t.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = t.abs() - table[lo], table[hi] - t.abs()
    take = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    v = torch.sign(t) * table[take] * _exact_two_to(e)
    return v.reshape(p.shape)[:r, :c]


def _exact_stored(image, cols):
    codes, scales = (image.codes, image.scales) if hasattr(image, "codes") else image
    table = _e4m3_table(codes.device)
    c = codes[:, :cols].long()
    s = _exact_two_to(scales.long() - 127).repeat_interleave(128, dim=1)[:, :cols]
    return torch.where(c < 128, table[c % 128], -table[c % 128]) * s


def exact(case, seed):
    """What ``run`` returns, from the definition in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = []
        for x in st["mats"]:
            out.append(_exact_quantized(x, case["square"]))
            if case["both"]:
                out.append(_exact_quantized(x.t(), case["square"]))
        return out
    if op == "linear":
        return torch.matmul(_exact_quantized(st["x"]), _exact_stored(st["w"], case["k"]).t())
    if op == "linear_backward":
        dx = torch.matmul(_exact_quantized(st["dy"]), _exact_stored(st["w_t"], case["n"]).t())
        dw = torch.matmul(_exact_quantized(st["dy"].t()), _exact_stored(st["x_t"], case["tokens"]).t())
        return dx, dw
    if op == "balance":
        idx, e = st["idx"], case["experts"]
        live = (idx >= 0).any(1)
        counts = torch.bincount(idx[idx >= 0], minlength=e)
        f = counts.double() * e / max(1, int(counts.sum()))
        n = max(1, int(live.sum()))
        p = torch.softmax(st["z"].double(), dim=1).masked_fill(~live[:, None], 0.0)
        w = 0.01 * float(st["g"]) / n
        return (p * f).sum() * 0.01 / n, counts, w * (p * f - p * (p * f).sum(1, keepdim=True))
    x, w = st["x"].bfloat16().double(), st["w"].bfloat16().double()
    tgt = st["t"]
    skip = tgt < 0
    logp = torch.log_softmax(torch.matmul(x, w.t()), dim=1)
    loss = -logp.gather(1, tgt.clamp(min=0)[:, None])[:, 0].masked_fill(skip, 0.0)
    if not case["grad"]:
        return loss
    d = logp.exp_()
    d[torch.arange(tgt.shape[0], device=d.device), tgt.clamp(min=0)] -= 1.0
    d *= st["g"].double().masked_fill(skip, 0.0)[:, None]
    return loss, torch.matmul(d, w), torch.matmul(d.t(), x)
