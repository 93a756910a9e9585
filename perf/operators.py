"""The 4-bit and distillation operators: cases, plain forms and calls.

Five operators are covered, each by the call that a training or serving
program makes of it:

  quantize         4-bit microscaled images of a list of matrices, read back
                   as the values they stand for;
  linear           y = x W^T with x quantised on the way and W held in 4 bits;
  linear_backward  dx and dW of that layer from dy and the saved images;
  logprobs         log probabilities of given tokens, entropy, alternatives;
  distill          loss and gradient against a teacher's top logits.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` is the definition in 64
bits.  The 4-bit format: blocks of 32 along a row share a power-of-two scale
2^e, e = floor(log2 max|x|) - 2, stored as e + 127 in a byte; an element is a
sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, rounded to nearest, ties to the
even code, saturating at 6.  An image of [R, C] is codes [R, 16 nb] (nb =
ceil(C / 32), even column in the low half of a byte) and scales [R, 4
ceil(nb / 4)]; padding is zero.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# midpoints of the grid, and whether a value on the midpoint goes up (to the even code)
_MID = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


# ------------------------------------------------------------------- cases
def listed():
    """The measured cases, from single tokens to whole layers and batches."""
    return [
        # one token's activations on their way into a 4-bit layer: pure latency
        {"name": "quantize_one_token", "op": "quantize", "shapes": "1x2048", "dtype": "bf16", "both": False},
        # the matrices of two layers of the 1.5B dense model, both orientations, as after an optimizer step
        {"name": "quantize_two_layers", "op": "quantize", "dtype": "f32", "both": True,
         "shapes": ",".join(["2048x2048,2048x2048,2048x512,2048x512,2048x5632,2048x5632,5632x2048"] * 2)},
        # decoding one sequence through the large model's wide matrix: the weights' bytes are all there is
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "n": 28672, "k": 8192, "dtype": "bf16", "out": "bf16"},
        # a ragged batch of sequences through an expert, odd sizes on every axis
        {"name": "linear_ragged_batch", "op": "linear", "tokens": 77, "n": 1407, "k": 2045, "dtype": "bf16", "out": "f32"},
        # prefill or a training forward of the large model's wide matrix
        {"name": "linear_large", "op": "linear", "tokens": 8192, "n": 28672, "k": 8192, "dtype": "bf16", "out": "bf16"},
        # a training backward of the 1.5B model's MLP
        {"name": "backward_mlp", "op": "linear_backward", "tokens": 8192, "n": 5632, "k": 2048, "dtype": "bf16", "out": "f32"},
        # an expert's backward over the odd number of tokens that the router sent it
        {"name": "backward_expert_odd", "op": "linear_backward", "tokens": 997, "n": 1408, "k": 2048, "dtype": "f32", "out": "f32"},
        # scoring the next token of a few sequences while serving
        {"name": "logprobs_few_rows", "op": "logprobs", "rows": 3, "vocab": 32000, "pad": 0, "dtype": "f32", "top": 20, "tau": 1.0},
        # a teacher's answers over a training batch: what the distillation loss reads
        {"name": "logprobs_teacher", "op": "logprobs", "rows": 4096, "vocab": 32000, "pad": 0, "dtype": "bf16", "top": 64, "tau": 1.0},
        # the same over a long odd vocabulary whose rows are padded
        {"name": "logprobs_long_odd", "op": "logprobs", "rows": 501, "vocab": 129283, "pad": 61, "dtype": "bf16", "top": 8, "tau": 0.7},
        # the student's loss and gradient over a training batch
        {"name": "distill_batch", "op": "distill", "rows": 8192, "vocab": 32000, "pad": 0, "dtype": "bf16", "top": 64, "tau": 1.0},
        # a small step over a long odd vocabulary in 32 bits, few alternatives
        {"name": "distill_long_odd", "op": "distill", "rows": 13, "vocab": 100003, "pad": 5, "dtype": "f32", "top": 7, "tau": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["quantize", "linear", "linear", "linear_backward", "logprobs", "distill"])
    if op == "quantize":
        shapes = []
        for _ in range(rng.randint(1, 6)):
            r, c = _log(rng, 1, 8192), _log(rng, 16, 8192)
            shapes.append("%dx%d" % (r, c))
        return {"op": op, "shapes": ",".join(shapes), "dtype": rng.choice(["f32", "bf16"]), "both": rng.random() < 0.5}
    if op in ("linear", "linear_backward"):
        tokens, n, k = _log(rng, 1, 8192), _log(rng, 64, 16384 if op == "linear" else 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:
            n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64
        return {"op": op, "tokens": tokens, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"])}
    vocab = _log(rng, 1000, 160000)
    rows = min(_log(rng, 1, 8192), 262144000 // vocab)
    return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 1, 32, 77]), "dtype": rng.choice(["f32", "bf16"]),
            "top": rng.randint(1, 64), "tau": rng.choice([1.0, 1.0, 0.5, 2.0])}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _image_bytes(r, c):
    return r * (-(-c // 32)) * 17


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


def _logits(g, rows, vocab, pad, dt):
    """Rows from flat to peaked, in a buffer whose rows may be longer than the vocabulary."""
    z = torch.randn(rows, vocab + pad, generator=g, device="cuda")
    z.mul_(1.0 + 3.0 * torch.rand(rows, 1, generator=g, device="cuda"))
    hot = torch.randint(0, vocab, (rows, 4), generator=g, device="cuda")
    z.scatter_(1, hot, 10.0 + 6.0 * torch.rand(rows, 4, generator=g, device="cuda"))
    return z.to(dt)[:, :vocab]


def prepare(case, seed):
    """Inputs on the GPU and the 4-bit images that a program keeps between calls."""
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    st = {"case": case}
    if op == "quantize":
        st["mats"] = [(torch.randn(r, c, generator=g, device="cuda") * 0.02).to(dt) for r, c in _shapes(case)]
    elif op == "linear":
        st["x"] = _activations(g, case["tokens"], case["k"], dt)
        st["w"] = _pack(torch.randn(case["n"], case["k"], generator=g, device="cuda") * 0.02)
    elif op == "linear_backward":
        st["dy"] = (torch.randn(case["tokens"], case["n"], generator=g, device="cuda") * 1e-3).to(dt)
        st["x_t"] = _pack(_activations(g, case["tokens"], case["k"], dt).float().t().contiguous())
        st["w_t"] = _pack((torch.randn(case["k"], case["n"], generator=g, device="cuda") * 0.02))
    else:
        rows, vocab = case["rows"], case["vocab"]
        z = _logits(g, rows, vocab, case["pad"], dt)
        st["z"] = z
        if op == "logprobs":
            banned = torch.randint(0, vocab, (max(1, vocab // 100),), generator=g, device="cuda")
            z[:, banned] = -math.inf                       # tokens that the sampler may not take
            tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
            ok = torch.isfinite(z.gather(1, tok[:, None])[:, 0].float())
            best = z.float().argmax(1)
            st["tokens"] = torch.where(ok, tok, best)
            # positions that are not scored (padding behind a sequence)
            st["tokens"][torch.rand(rows, generator=g, device="cuda") < 0.03] = -1
        else:
            k = case["top"]
            idx = torch.empty(rows, k, dtype=torch.int64, device="cuda")
            val = torch.empty(rows, k, device="cuda")
            for a in range(0, rows, 512):                   # the teacher: near the student, its best k
                t = z[a:a + 512].float()
                t = t + 0.5 * torch.randn(t.shape, generator=g, device="cuda")
                v, i = torch.topk(t, k, dim=1)
                val[a:a + 512], idx[a:a + 512] = v, i
            short = torch.randint(1, k + 1, (rows, 1), generator=g, device="cuda")
            keep = torch.rand(rows, 1, generator=g, device="cuda") < 0.9
            slot = torch.arange(k, device="cuda")[None, :]
            idx = torch.where(keep | (slot < short), idx, torch.full_like(idx, -1))
            empty = torch.rand(rows, 1, generator=g, device="cuda") < 0.05   # padding positions: no teacher
            idx = torch.where(empty, torch.full_like(idx, -1), idx)
            st["idx"], st["val"] = idx.contiguous(), val
            n = max(1, int((idx[:, 0] >= 0).sum()))
            st["g"] = torch.full((rows,), 1.0 / n, device="cuda")
    if own:
        import matrix_orthogonalizing_optimizer_amd as mo
        for name, cols in (("w", case.get("k")), ("x_t", case.get("tokens")), ("w_t", case.get("n"))):
            if name in st:
                st[name] = mo.Mx4Matrix(st[name][0], st[name][1], cols)
    return st


# -------------------------------------------------------------- plain forms
def _two_to(e):
    """2^e of integers in [-127, 127], exactly (a pow is not), from its bits."""
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _blocks(x):
    r, c = x.shape
    nb = -(-c // 32)
    p = torch.zeros(r, nb * 32, dtype=torch.float32, device=x.device)
    p[:, :c] = x
    return p.view(r, nb, 32)


def _codes(x):
    """(codes, scale bytes) of [r, c] in 32 bits: block scales and grid indices by comparisons."""
    b = _blocks(x)
    a = b.abs().amax(2, keepdim=True)
    e = torch.frexp(a)[1] - 3                               # floor(log2 a) - 2
    e = torch.where(a == 0, torch.full_like(e, -127), e).clamp(min=-127)
    t = b * _two_to(-e)
    m = t.abs()
    code = torch.zeros(b.shape, dtype=torch.uint8, device=x.device)
    for mid, up in _MID:
        code += (m >= mid) if up else (m > mid)
    code += (t < 0).to(torch.uint8) * 8
    return code, (e[:, :, 0] + 127).to(torch.uint8)


def _pack(x):
    """The stored image of [r, c]."""
    code, s = _codes(x)
    r, nb = s.shape
    code = code.view(r, nb * 16, 2)
    scales = torch.zeros(r, -(-nb // 4) * 4, dtype=torch.uint8, device=x.device)
    scales[:, :nb] = s
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous(), scales


def _values(code, s, cols):
    """What codes [r, nb, 32] and scale bytes [r, nb] stand for, fp32 [r, cols]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float32, device=code.device)
    v = grid[code.int()]
    v = v * _two_to(s.int() - 127)[:, :, None]
    return v.reshape(code.shape[0], -1)[:, :cols]


def _stored_values(image, cols):
    codes, scales = image
    r = codes.shape[0]
    nb = -(-cols // 32)
    code = torch.stack((codes & 15, codes >> 4), dim=2).view(r, nb, 32)
    return _values(code, scales[:, :nb], cols)


def _quantized(x):
    code, s = _codes(x.float())
    return _values(code, s, x.shape[1])


def _order(z):
    """Integers that order as the values do (negative zero equal to zero)."""
    b = (z.float() + 0.0).view(torch.int32)
    return torch.where(b < 0, b ^ 0x7fffffff, b).long()


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        out = []
        for x in st["mats"]:
            out.append(_quantized(x).to(torch.bfloat16))
            if case["both"]:
                out.append(_quantized(x.t()).to(torch.bfloat16))
        return out
    if op == "linear":
        return _quantized(st["x"]).matmul(_stored_values(st["w"], case["k"]).t()).to(_DT[case["out"]])
    if op == "linear_backward":
        dy = st["dy"]
        dx = _quantized(dy).matmul(_stored_values(st["w_t"], case["n"]).t())
        dw = _quantized(dy.t()).matmul(_stored_values(st["x_t"], case["tokens"]).t())
        return dx.to(_DT[case["out"]]), dw
    z = st["z"].float() / case["tau"]
    m = z.amax(1, keepdim=True)
    ex = torch.exp(z - m)
    s = ex.sum(1, keepdim=True)
    lse = m + torch.log(s)
    if op == "logprobs":
        tok = st["tokens"]
        lp = z.gather(1, tok.clamp(min=0)[:, None])[:, 0] - lse[:, 0]
        lp = torch.where(tok < 0, torch.zeros_like(lp), lp)
        ent = torch.log(s[:, 0]) + torch.where(ex > 0, ex * (m - z), torch.zeros_like(ex)).sum(1) / s[:, 0]
        key = (_order(st["z"]) << 20) + (z.shape[1] - 1 - torch.arange(z.shape[1], device=z.device))
        idx = z.shape[1] - 1 - (torch.topk(key, case["top"], dim=1)[0] & 0xfffff)
        return lp, ent, z.gather(1, idx) - lse, idx
    idx, tau = st["idx"], case["tau"]
    here = idx >= 0
    t = torch.where(here, st["val"] / tau, torch.full_like(st["val"], -math.inf))
    some = here.any(1, keepdim=True)
    tm = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(m))
    p = torch.exp(t - tm)
    ts = torch.where(some, p.sum(1, keepdim=True), torch.ones_like(m))
    p = p / ts
    logp = t - tm - torch.log(ts)
    logq = z.gather(1, idx.clamp(min=0)) - lse
    loss = tau * tau * torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
    grad = ex / s
    grad.scatter_add_(1, idx.clamp(min=0), -p)
    grad = torch.where(some, grad * (tau * st["g"])[:, None], torch.zeros_like(grad))
    return loss, grad.to(st["z"].dtype)


def _own(st):
    import matrix_orthogonalizing_optimizer_amd as mo
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q = mo.mx4_quantize(st["mats"], images="both" if case["both"] else "rows")
        return mo.mx4_dequantize([i for pair in q for i in pair] if case["both"] else q)
    if op == "linear":
        return mo.mx4_linear(st["x"], st["w"], out_dtype=_DT[case["out"]])
    if op == "linear_backward":
        return mo.mx4_linear_backward(st["dy"], st["x_t"], st["w_t"], dx_dtype=_DT[case["out"]])
    if op == "logprobs":
        r = mo.token_logprobs(st["z"], st["tokens"], top=case["top"], temperature=case["tau"])
        return r.logprob, r.entropy, r.top_logprob, r.top_index
    return mo.distill_loss(st["z"], st["idx"], st["val"], temperature=case["tau"], grad_loss=st["g"])


def run(state):
    """One pass through the case's operator."""
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op, s = case["op"], _SIZE[case["dtype"]]
    if op == "quantize":
        b = f = 0
        for r, c in _shapes(case):
            b += r * c * s + _image_bytes(r, c) + 2 * r * c
            f += 4 * r * c
            if case["both"]:
                b += _image_bytes(c, r) + 2 * r * c
                f += 4 * r * c
        return {"bytes": b, "flops": f}
    if op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": t * k * s + _image_bytes(n, k) + t * n * _SIZE[case["out"]], "flops": 2 * t * n * k}
    if op == "linear_backward":
        t, n, k = case["tokens"], case["n"], case["k"]
        b = t * n * s + _image_bytes(k, t) + _image_bytes(k, n) + t * k * _SIZE[case["out"]] + n * k * 4
        return {"bytes": b, "flops": 4 * t * n * k}
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    if op == "logprobs":
        return {"bytes": rows * (vocab * s + 16 + 12 * top), "flops": 6 * rows * vocab}
    return {"bytes": rows * (2 * vocab * s + 8 + 12 * top), "flops": 6 * rows * vocab}


# ------------------------------------------------- the definition in 64 bits
def _exact_two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantized(x):
    """Scaled to the block's power of two, rounded by the step of its binade, halves to even."""
    x = x.double()
    r, c = x.shape
    out = torch.nn.functional.pad(x, (0, -c % 32)).reshape(r, -1, 32)
    a = out.abs().max(dim=2, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = torch.where(_exact_two_to(e + 1) <= a, e + 1, e)   # log2 of a value next to a power of two
    e = torch.where(_exact_two_to(e) > a, e - 1, e)
    e = torch.where(a > 0, e - 2, torch.zeros_like(e)).clamp(min=-127)
    t = out / _exact_two_to(e)
    m = t.abs()
    step = torch.where(m < 2, torch.full_like(m, 0.5), torch.where(m < 4, torch.ones_like(m), torch.full_like(m, 2.0)))
    q = (torch.round(m / step) * step).clamp(max=6.0) * torch.sign(t)
    return (q * _exact_two_to(e)).reshape(r, -1)[:, :c]


def _exact_stored(image, cols):
    codes, scales = (image.codes, image.scales) if hasattr(image, "codes") else image
    r = codes.shape[0]
    both = torch.stack((codes % 16, codes // 16), dim=2).reshape(r, -1).to(torch.int64)
    mag, sign = both % 8, 1.0 - 2.0 * (both // 8).double()
    ex, man = mag // 2, (mag % 2).double()                  # two exponent bits, one mantissa bit
    v = torch.where(ex == 0, 0.5 * man, _exact_two_to(ex - 1) * (1.0 + 0.5 * man)) * sign
    s = _exact_two_to(scales.to(torch.int64) - 127).repeat_interleave(32, dim=1)[:, :v.shape[1]]
    return (v * s)[:, :cols]


def exact(case, seed):
    """What ``run`` returns, from the definition in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = []
        for x in st["mats"]:
            out.append(_exact_quantized(x))
            if case["both"]:
                out.append(_exact_quantized(x.t()))
        return out
    if op == "linear":
        return torch.matmul(_exact_quantized(st["x"]), _exact_stored(st["w"], case["k"]).t())
    if op == "linear_backward":
        dx = torch.matmul(_exact_quantized(st["dy"]), _exact_stored(st["w_t"], case["n"]).t())
        dw = torch.matmul(_exact_quantized(st["dy"].t()), _exact_stored(st["x_t"], case["tokens"]).t())
        return dx, dw
    z = st["z"].double() / case["tau"]
    logq = torch.log_softmax(z, dim=1)
    if op == "logprobs":
        tok = st["tokens"]
        lp = torch.where(tok < 0, torch.zeros_like(z[:, 0]), logq.gather(1, tok.clamp(min=0)[:, None])[:, 0])
        q = logq.exp()
        ent = -torch.where(q > 0, q * logq, torch.zeros_like(q)).sum(1)
        idx = torch.sort(st["z"].double(), dim=1, descending=True, stable=True)[1][:, :case["top"]].contiguous()
        return lp, ent, logq.gather(1, idx), idx
    idx, tau = st["idx"], case["tau"]
    t = (st["val"].double() / tau).masked_fill(idx < 0, -math.inf)
    none = (idx < 0).all(1, keepdim=True)
    logp = torch.log_softmax(t.masked_fill(none, 0.0), dim=1)
    p = logp.exp().masked_fill(none, 0.0)
    terms = p * (logp - logq.gather(1, idx.clamp(min=0)))
    loss = tau ** 2 * terms.masked_fill(idx < 0, 0.0).sum(1)
    q = torch.zeros_like(z).scatter_add_(1, idx.clamp(min=0), p)
    grad = tau * st["g"].double()[:, None] * (logq.exp() - q)
    return loss, grad.masked_fill(none, 0.0)
