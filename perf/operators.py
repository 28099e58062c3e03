"""Cases of the low-rank adapters, the gradient norm and the AdamW step.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and through the package's entry points:

  adapters_forward   y_t += s_a B_a (A_a x_t) for the adapter a of each token's segment
  adapters_backward  gradients of the same onto x, A and B
  grad_norm          global 2-norm of many gradients and the clipping coefficient
  adamw              AdamW over many tensors, states in 32 or in 8 bits

Sizes: the decoder layer of hidden 2048 and 5632 and the 11008 x 4096
projection, sequences of 256 tokens, 24 layers.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256                 # values that share an exponent byte in the 8-bit states
DEV = "cuda"
ALPHA_POS, ALPHA_STEP = 0xC13FA9A9, 0x91E10DA5   # the dither's two irrationals, times 2^32
HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)
STEP0 = 100                 # steps already taken when a case starts


# ---- the cases -------------------------------------------------------------------------------------------

def listed():
    return [
        # serving, one request's next token: latency alone
        dict(name="fwd token", op="adapters_forward", m=2048, n=2048, tokens=1, segs=1, adapters=1, rank=16,
             ranks="same", lens="even", dtype="bf16"),
        # serving, the next token of 64 requests, each with an adapter of its own among 32
        dict(name="fwd 64 requests", op="adapters_forward", m=5632, n=2048, tokens=64, segs=64, adapters=32, rank=64,
             ranks="mixed", lens="even", dtype="bf16"),
        # prompts of many lengths beside single tokens, some requests without an adapter
        dict(name="fwd prompts", op="adapters_forward", m=2048, n=5632, tokens=4099, segs=23, adapters=8, rank=32,
             ranks="mixed", lens="ragged", dtype="bf16"),
        # training, 32 sequences of 256 tokens over four adapters
        dict(name="fwd 8192 tokens", op="adapters_forward", m=5632, n=2048, tokens=8192, segs=32, adapters=4, rank=16,
             ranks="same", lens="even", dtype="bf16"),
        # single precision with odd widths and ranks, as the small parity layers have them
        dict(name="bwd odd f32", op="adapters_backward", m=600, n=520, tokens=333, segs=5, adapters=3, rank=12,
             ranks="mixed", lens="ragged", dtype="f32"),
        # a ragged training batch
        dict(name="bwd ragged", op="adapters_backward", m=2048, n=2048, tokens=2001, segs=11, adapters=4, rank=64,
             ranks="mixed", lens="ragged", dtype="bf16"),
        # training, 32 sequences of 256 tokens on the large projection
        dict(name="bwd 8192 tokens", op="adapters_backward", m=11008, n=4096, tokens=8192, segs=32, adapters=4, rank=16,
             ranks="same", lens="even", dtype="bf16"),
        # clipping the adapters of one decoder layer: many small tensors
        dict(name="norm adapters", op="grad_norm", layers=1, hidden=2048, ffn=5632, block=0, rank=16, grad="bf16"),
        # clipping the generators of 24 decoder layers
        dict(name="norm generators", op="grad_norm", layers=24, hidden=2048, ffn=5632, block=256, rank=0, grad="f32"),
        # the adapters of 24 decoder layers: fp32 master values with the bf16 copy that the products read
        dict(name="adamw 32 adapters", op="adamw", bits=32, layers=24, hidden=2048, ffn=5632, block=0, rank=16,
             param="f32", grad="f32", copy=True),
        # bf16 adapters of one small layer, odd widths: the smallest step
        dict(name="adamw 8 small", op="adamw", bits=8, layers=1, hidden=520, ffn=601, block=0, rank=5, param="bf16",
             grad="bf16", copy=False),
        # generators and adapters of 24 decoder layers, states in 8 bits
        dict(name="adamw 8 all", op="adamw", bits=8, layers=24, hidden=2048, ffn=5632, block=256, rank=16, param="f32",
             grad="f32", copy=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters_forward", "adapters_forward", "adapters_backward", "adapters_backward", "grad_norm",
                     "adamw", "adamw"])
    if op.startswith("adapters"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        tokens = _log(rng, 1, 8192) if op == "adapters_forward" else _log(rng, 32, 8192)
        m, n = _log(rng, 256, 11008), _log(rng, 256, 5632)
        if rng.random() < 0.7:      # most projections are whole multiples of 64 wide
            m, n = -(-m // 64) * 64, -(-n // 64) * 64
        if dtype == "f32":
            tokens, m, n = min(tokens, 2048), min(m, 2048), min(n, 2048)
        lens = rng.choice(["ragged", "ragged", "even"])
        segs = tokens if rng.random() < 0.25 and tokens <= 256 else min(tokens, _log(rng, 1, 64))
        return dict(op=op, m=m, n=n, tokens=tokens, segs=segs, adapters=_log(rng, 1, 32),
                    rank=rng.choice([8, 16, 16, 32, 64, _log(rng, 1, 96)]), ranks=rng.choice(["same", "mixed"]),
                    lens=lens, dtype=dtype)
    hidden = _log(rng, 128, 2048)
    case = dict(op=op, layers=_log(rng, 1, 20), hidden=hidden, ffn=int(hidden * rng.uniform(1, 2.75)),
                block=rng.choice([0, 32, 64, 128]), rank=_log(rng, 1, 64), grad=rng.choice(["f32", "f32", "bf16"]))
    if op == "adamw":
        param = rng.choice(["f32", "f32", "bf16"])
        case.update(bits=rng.choice([8, 32]), param=param, copy=param == "f32" and rng.random() < 0.5)
    return case


def _ranks(case):
    r, count = case["rank"], case["adapters"]
    return [r if case["ranks"] == "same" else max(1, (r, r // 2, r // 4, r - 3)[i % 4]) for i in range(count)]


def _numels(case):
    """Sizes of the tensors a step sees: for every projection of a layer, its generators (both sides) and its adapter."""
    h, f, b, r = case["hidden"], case["ffn"], case["block"], case["rank"]
    shapes = [(h, h)] * 4 + [(f, h)] * 2 + [(h, f)]
    one = []
    for m, n in shapes:
        if b:
            one += [(k // b) * (b * (b - 1) // 2) for k in (m, n) if k >= b]
        if r:
            one += [r * n, m * r]
    return one * case["layers"]


def work(case):
    if case["op"].startswith("adapters"):
        es = 2 if case["dtype"] == "bf16" else 4
        m, n, N = case["m"], case["n"], case["tokens"]
        weights = sum(_ranks(case)) * (n + m)
        if case["op"] == "adapters_forward":
            return {"bytes": es * (N * (n + 2 * m) + min(weights, N * max(_ranks(case)) * (n + m))),
                    "flops": 2.0 * N * case["rank"] * (n + m)}
        return {"bytes": es * (N * (3 * n + m) + weights) + 4 * weights, "flops": 2.0 * N * case["rank"] * (3 * n + 2 * m)}
    count = sum(_numels(case))
    g = 4 if case["grad"] == "f32" else 2
    if case["op"] == "grad_norm":
        return {"bytes": g * count, "flops": 2.0 * count}
    p = 8 if case["param"] == "f32" else 4
    state = 16 if case["bits"] == 32 else 4 + 4    # 8 bits: both moments read and written, then returned in bf16
    return {"bytes": count * (g + p + state + (2 if case["copy"] else 0)), "flops": 12.0 * count}


# ---- inputs ----------------------------------------------------------------------------------------------

def _segments(case, rng):
    N, S = case["tokens"], case["segs"]
    if case["lens"] == "even":
        cuts = [N * i // S for i in range(S + 1)]
    else:                       # lengths over several orders of magnitude, single tokens and empty ones among them
        w = np.exp(rng.uniform(0, math.log(700), S))
        cuts = [0] + [int(x) for x in np.floor(np.cumsum(w) / w.sum() * N + 0.5)]
        cuts[-1] = N
    count = case["adapters"]
    which = rng.integers(0, count, S)
    if case["lens"] == "ragged":
        which[rng.random(S) < 0.1] = -1
    if count <= S:              # every adapter has a request, as a batch is put together
        which[rng.permutation(S)[:count]] = np.arange(count)
    return cuts, which


def _prepare_adapters(case, seed):
    rng = np.random.default_rng([7, seed])
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    m, n, N = case["m"], case["n"], case["tokens"]
    ranks = _ranks(case)

    def normal(shape, sigma):
        return (torch.randn(shape, generator=gen, device=DEV) * sigma).to(dt)

    cuts, which = _segments(case, rng)
    A = [normal((r, n), n ** -0.5) for r in ranks]
    B = [normal((m, r), 0.05) for r in ranks]
    scales = [float(2.0 ** rng.integers(-1, 2)) for _ in ranks]
    s = dict(case=case, A=A, B=B, scales=scales, ranks=ranks, X=normal((N, n), 1.0),
             seg_start=torch.tensor(cuts, dtype=torch.int32, device=DEV),
             seg_adapter=torch.tensor(which, dtype=torch.int32, device=DEV),
             # per row of the adapters stacked on each other: its adapter and its scale
             row_adapter=torch.tensor(np.repeat(np.arange(len(ranks)), ranks), dtype=torch.int32, device=DEV),
             row_scale=torch.tensor(np.repeat(scales, ranks), dtype=torch.float32, device=DEV))
    if case["op"] == "adapters_forward":
        s["Y"] = normal((N, m), 1.0)            # what the shared projection gave
    else:
        s["dY"] = normal((N, m), 1.0)
        s["dX"] = normal((N, n), 1.0)           # what the shared projection's backward gave
        s["dA"] = torch.zeros(sum(ranks) * n, device=DEV)
        s["dB"] = torch.zeros(sum(ranks) * m, device=DEV)
    if own:
        import orthogonal_reparameterized_poetx_amd as P
        grads = {}
        if case["op"] == "adapters_backward":
            grads = dict(dA=[t.view(r, n) for t, r in zip(s["dA"].split([r * n for r in ranks]), ranks)],
                         dB=[t.view(m, r) for t, r in zip(s["dB"].split([r * m for r in ranks]), ranks)])
        s["set"] = P.AdapterSet(m, n, A, B, scales, **grads)
    return s


def _prepare_tensors(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    numels = _numels(case)
    blocks = [-(-x // BLOCK) for x in numels]
    total = sum(blocks) * BLOCK
    gdt = torch.bfloat16 if case["grad"] == "bf16" else torch.float32
    offs = (np.cumsum([0] + blocks[:-1]) * BLOCK).tolist()
    real = torch.zeros(total, dtype=torch.bool, device=DEV)     # not the padding after a tensor
    for o, x in zip(offs, numels):
        real[o:o + x] = True

    def normal(sigma):
        return torch.where(real, torch.randn(total, generator=gen, device=DEV) * sigma, 0.0)

    def views(flat):
        return [flat[o:o + x] for o, x in zip(offs, numels)]

    # every tensor's gradients have a size of their own, some values far smaller than the rest
    size = torch.exp(torch.randn(len(numels), generator=gen, device=DEV) * 1.5 - 6.0)
    per_block = torch.repeat_interleave(size, torch.tensor(blocks, device=DEV))
    g = (normal(1.0).view(-1, BLOCK) * per_block[:, None]).view(-1)
    g = torch.where(torch.rand(total, generator=gen, device=DEV) < 0.1, g * 1e-3, g)
    s = dict(case=case, g=g.to(gdt))
    if case["op"] == "grad_norm":
        s["max_norm"] = 1.0
        if own:
            import orthogonal_reparameterized_poetx_amd as P
            s["norm"] = P.GradNorm(views(s["g"]))
        return s
    s["p"] = normal(0.03).to(torch.bfloat16 if case["param"] == "bf16" else torch.float32)
    s["copy"] = s["p"].to(torch.bfloat16) if case["copy"] else None
    s["coef"] = torch.full((1,), 0.75, device=DEV)              # as the clipping left it
    s["step"] = STEP0
    # every other tensor takes decay and half the learning rate
    lr_mul = [0.5 if i % 2 else 1.0 for i in range(len(numels))]
    decay = [0.1 if i % 2 else 0.0 for i in range(len(numels))]
    reps = torch.tensor(blocks, device=DEV)
    s["lr_mul"] = torch.repeat_interleave(torch.tensor(lr_mul, device=DEV), reps)[:, None]
    s["decay"] = torch.repeat_interleave(torch.tensor(decay, device=DEV), reps)[:, None]
    mom = g * torch.rand(total, generator=gen, device=DEV) * 0.5
    sec = g * g * (0.5 + torch.rand(total, generator=gen, device=DEV))
    if case["bits"] == 32:
        state = dict(m=mom, v=sec)
    else:
        state = {}
        state["m"], state["m_exp"] = _encode(mom, torch.zeros((), dtype=torch.int32, device=DEV), True)
        state["v"], state["v_exp"] = _encode(sec, torch.zeros((), dtype=torch.int32, device=DEV), False)
    s["state"] = state
    if own:
        import orthogonal_reparameterized_poetx_amd as P
        s["opt"] = P.AdamW(views(s["p"]), views(s["g"]), lr_mul=lr_mul, weight_decay=decay, state_bits=case["bits"],
                           copies=views(s["copy"]) if case["copy"] else None, state=state, step=STEP0, **HYPER)
    return s


def prepare(case, seed):
    return _prepare_adapters(case, seed) if case["op"].startswith("adapters") else _prepare_tensors(case, seed)


# ---- the plain forms -------------------------------------------------------------------------------------

def _row_weights(s):
    """[tokens][stacked rows]: the scale where the row belongs to the token's adapter, else 0."""
    N = s["case"]["tokens"]
    of_token = torch.repeat_interleave(s["seg_adapter"], s["seg_start"].diff(), output_size=N)
    return (of_token[:, None] == s["row_adapter"][None, :]) * s["row_scale"]


def _plain_adapters_forward(s):
    A, B = torch.cat(s["A"]).float(), torch.cat(s["B"], 1).float()
    T = s["X"].float() @ A.t() * _row_weights(s)
    s["Y"].copy_(s["Y"].float() + T @ B.t())
    return {"Y": s["Y"]}


def _plain_adapters_backward(s):
    A, B = torch.cat(s["A"]).float(), torch.cat(s["B"], 1).float()
    X, dY, w = s["X"].float(), s["dY"].float(), _row_weights(s)
    T, U = X @ A.t() * w, dY @ B * w
    s["dA"].copy_((U.t() @ X).view(-1))
    s["dB"].copy_(torch.cat([t.reshape(-1) for t in (dY.t() @ T).split(s["ranks"], 1)]))
    s["dX"].copy_(s["dX"].float() + U @ A)
    return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}


def _plain_norm(s):
    norm = (s["g"].float() * s["g"].float()).sum().sqrt()
    return {"norm": norm, "coef": (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)}


def _dither(total, step):
    """20 bits for each moment from the fractional parts of pos alpha + step beta (a Weyl sequence)."""
    wrap = lambda c: c - (1 << 32) if c >= 1 << 31 else c   # noqa: E731
    h = torch.arange(total, dtype=torch.int32, device=DEV) * wrap(ALPHA_POS) + wrap(step * ALPHA_STEP & 0xFFFFFFFF)
    return (h >> 12) & 0xFFFFF, (h >> 5) & 0xFFFFF, (h >> 16) & 0xFFFF


def _encode(x, u, signed):
    """8-bit codes of x and the exponent byte of each block: 3 mantissa bits, 4 (signed) or 5 exponent bits."""
    low, fixed = (15, 271) if signed else (31, 287)
    bits = x.view(torch.int32) & 0x7FFFFFFF
    exp = ((bits.view(-1, BLOCK).amax(1) + 0xFFFFF) >> 23).clamp(40, 254)
    e = exp[:, None].expand(-1, BLOCK).reshape(-1)
    normal = ((bits + u) >> 20) - ((e - low) << 3)
    unit = ((fixed - e) << 23).view(torch.float32)
    tiny = torch.floor(bits.view(torch.float32) * unit + u.float() * 2.0 ** -20).to(torch.int32)
    code = torch.where((bits >> 23) - e + low >= 1, normal, tiny)
    if signed:
        code = code.clamp(max=127) | torch.where(x < 0, 128, 0)
    else:
        code = torch.where(bits > 0, code.clamp(1, 255), 0)
    return code.to(torch.uint8), exp.to(torch.uint8)


def _decode(code, exp, signed):
    low = 15 if signed else 31
    c, top = code.to(torch.int32), exp.to(torch.int32)[:, None].expand(-1, BLOCK).reshape(-1)
    e, f = (c >> 3) & low, c & 7
    normal = ((top - low + e) << 23 | f << 20).view(torch.float32)
    tiny = f.float() * ((top - low - 2) << 23).view(torch.float32)
    value = torch.where(e > 0, normal, tiny)
    return torch.where(c >= 128, -value, value) if signed else value


def _plain_adamw(s):
    st, case = s["state"], s["case"]
    s["step"] += 1
    b1, b2 = (float(np.float32(b)) for b in HYPER["betas"])
    bc1, bc2 = 1.0 - b1 ** s["step"], 1.0 - b2 ** s["step"]
    g = s["g"].float() * s["coef"]
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m, v = _decode(st["m"], st["m_exp"], True), _decode(st["v"], st["v_exp"], False)
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g * g * (1.0 - b2)
    p = s["p"].float().view(-1, BLOCK)
    upd = ((m / bc1) / (torch.sqrt(v / bc2) + HYPER["eps"])).view(-1, BLOCK)
    p = (p - (HYPER["lr"] * s["lr_mul"]) * (s["decay"] * p + upd)).view(-1)
    um, uv, up = _dither(m.numel(), s["step"])
    if case["param"] == "bf16":     # rounded by the dither: small updates are kept on average
        s["p"].copy_(((p.view(torch.int32) + up) & -65536).view(torch.float32))
    else:
        s["p"].copy_(p)
    out = {"p": s["p"]}
    if case["copy"]:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return dict(out, m=st["m"], v=st["v"])
    for k, x, u, signed in (("m", m, um, True), ("v", v, uv, False)):
        code, exp = _encode(x, u, signed)
        st[k].copy_(code)
        st[k + "_exp"].copy_(exp)
    # what the codes stand for has at most 4 significant bits: bf16 holds it exactly
    return dict(out, m=_decode(st["m"], st["m_exp"], True).to(torch.bfloat16),
                v=_decode(st["v"], st["v_exp"], False).to(torch.bfloat16))


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"adapters_forward": _plain_adapters_forward, "adapters_backward": _plain_adapters_backward,
                "grad_norm": _plain_norm, "adamw": _plain_adamw}[op](s)
    if op == "adapters_forward":
        s["set"].forward(s["X"], s["Y"], s["seg_start"], s["seg_adapter"])
        return {"Y": s["Y"]}
    if op == "adapters_backward":
        s["set"].backward(s["X"], s["dY"], s["seg_start"], s["seg_adapter"], dX=s["dX"])
        return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}
    if op == "grad_norm":
        norm, coef = s["norm"](s["max_norm"])
        return {"norm": norm, "coef": coef}
    opt = s["opt"]
    opt.step(coef=s["coef"])
    out = {"p": s["p"]}
    if s["case"]["copy"]:
        out["copy"] = s["copy"]
    out["m"], out["v"] = opt.moments()
    return out


# ---- the same from the definitions in 64 bits ------------------------------------------------------------

def _exact_adapters(s):
    X = s["X"].double()
    cuts, which = s["seg_start"].tolist(), s["seg_adapter"].tolist()
    fwd = s["case"]["op"] == "adapters_forward"
    out = (s["Y"] if fwd else s["dX"]).double()
    dA, dB = [torch.zeros_like(a, dtype=torch.float64) for a in s["A"]], [torch.zeros_like(b, dtype=torch.float64)
                                                                          for b in s["B"]]
    for lo, hi, a in zip(cuts, cuts[1:], which):
        if a < 0 or lo == hi:
            continue
        A, B, c = s["A"][a].double(), s["B"][a].double(), s["scales"][a]
        x = X[lo:hi]
        if fwd:
            out[lo:hi] += (x @ A.t() * c) @ B.t()
            continue
        dy = s["dY"][lo:hi].double()
        u = dy @ B * c
        out[lo:hi] += u @ A
        dA[a] += u.t() @ x
        dB[a] += dy.t() @ (x @ A.t() * c)
    if fwd:
        return {"Y": out}
    return {"dX": out, "dA": torch.cat([t.reshape(-1) for t in dA]), "dB": torch.cat([t.reshape(-1) for t in dB])}


def _fraction(total, step, shift, bits):
    h = (torch.arange(total, dtype=torch.int64, device=DEV) * ALPHA_POS + step * ALPHA_STEP) % 2 ** 32
    return ((h // 2 ** shift) % 2 ** bits).double() / 2 ** bits


def _exact_round(x, u, exponents):
    """x on the grid of its block: 8 steps to an octave, the lowest octave's steps below it; up where the fraction plus u reaches 1."""
    a = x.abs().view(-1, BLOCK)
    top = torch.frexp(a.amax(1) * (1 + 0.0625 - 2.0 ** -40))[1] - 1        # the octave of the largest code
    top = torch.where(a.amax(1) > 0, top, -87).clamp(-87, 127)
    low = (top - (2 ** exponents - 2))[:, None]
    octave = torch.maximum(torch.frexp(a)[1] - 1, low)
    step = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), octave - 3)
    r = torch.floor(a / step + u.view(-1, BLOCK)) * step
    if exponents == 5:
        r = torch.where((a > 0) & (r == 0), torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), low - 3), r)
    return torch.sign(x) * r.view(-1)


def _exact_codes(code, exp, mant_exp):
    """The value of each code, from a table in 64 bits."""
    c = np.arange(256)
    sign = np.where((c >= 128) & (mant_exp == 4), -1.0, 1.0)
    e, f = (c >> 3) % 2 ** mant_exp, c & 7
    grid = sign * np.where(e > 0, (1 + f / 8) * 2.0 ** (e - (2 ** mant_exp - 1)), f / 8 * 2.0 ** (2 - 2 ** mant_exp))
    t = torch.tensor(grid, dtype=torch.float64, device=DEV)[code.long()]
    return torch.ldexp(t.view(-1, BLOCK), exp.to(torch.int32)[:, None] - 127).reshape(-1)


def _exact_adamw(s):
    st, case, step = s["state"], s["case"], STEP0 + 1
    b1, b2 = (float(np.float32(b)) for b in HYPER["betas"])
    g, p = s["g"].double() * s["coef"].double(), s["p"].double()
    if case["bits"] == 32:
        m, v = st["m"].double(), st["v"].double()
    else:
        m, v = _exact_codes(st["m"], st["m_exp"], 4), _exact_codes(st["v"], st["v_exp"], 5)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
    lr = (HYPER["lr"] * s["lr_mul"].double()).expand(-1, BLOCK).reshape(-1)
    decay = s["decay"].double().expand(-1, BLOCK).reshape(-1)
    p = p - lr * (decay * p + m / (1 - b1 ** step) / ((v / (1 - b2 ** step)) ** 0.5 + HYPER["eps"]))
    out = {"copy": p} if case["copy"] else {}
    if case["param"] == "bf16":
        unit = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), torch.frexp(p)[1] - 8)
        p = torch.sign(p) * torch.floor(p.abs() / unit + _fraction(p.numel(), step, 16, 16)) * unit
    if case["bits"] == 8:
        m = _exact_round(m, _fraction(m.numel(), step, 12, 20), 4)
        v = _exact_round(v, _fraction(v.numel(), step, 5, 20), 5)
    return dict(out, p=p, m=m, v=v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("adapters"):
        return _exact_adapters(s)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    norm = s["g"].double().square().sum().sqrt()
    return {"norm": norm, "coef": torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)}
