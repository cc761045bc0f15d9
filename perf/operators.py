"""Benchmark cases of the int8 products and of the Muon optimizer's operators.

    quantize_i8    rows (or columns) of a matrix to int8, one scale each
    gemm_i8        C = A B^T in int8 with a scale per token and per channel
    linear_i8      y = x W^T and its two gradients, all three products in int8
    newton_schulz  orthogonalisation of a matrix (or a batch) by Newton-Schulz products
    muon_step      momentum, orthogonalisation and the stochastically rounded weight update

``run`` computes each in plain torch operations where ``own`` is false, and
through the package's entry points where it is true. ``exact`` gives the
same from the definitions in binary64. Hidden size 4096, MLP width 14336 and
key/value width 1024 are those of the benchmark's Llama-3-8B-shaped list.
"""

import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
NS_STEPS = 5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's activations, quantised before the next product
        dict(name="quantize_token", op="quantize_i8", rows=1, cols=4096, dtype="bf16",
             transpose=False, rounding="rn"),
        # the gradient of 8,192 tokens, quantised by stochastic rounding along the tokens
        dict(name="quantize_grad_columns", op="quantize_i8", rows=8192, cols=4096, dtype="bf16",
             transpose=True, rounding="sr"),
        # one decoded token through an MLP's up projection: bound by reading the weights
        dict(name="gemm_token", op="gemm_i8", m=1, n=14336, k=4096, rounding="rn"),
        # a ragged batch through an odd-sized projection, stochastically rounded
        dict(name="gemm_ragged", op="gemm_i8", m=333, n=1009, k=1111, rounding="sr"),
        # the up projection of 8,192 tokens
        dict(name="gemm_prefill", op="gemm_i8", m=8192, n=14336, k=4096, rounding="rn"),
        # a small model's layer in training
        dict(name="linear_small", op="linear_i8", m=67, n=512, k=256),
        # a training step's up projection: forward and both gradients
        dict(name="linear_train", op="linear_i8", m=4096, n=14336, k=4096),
        # one small square matrix: a chain of dependent small products
        dict(name="ns_small", op="newton_schulz", batch=1, rows=128, cols=128, dtype="bf16"),
        # odd sides, f32 gradient, taller than wide
        dict(name="ns_odd", op="newton_schulz", batch=1, rows=517, cols=333, dtype="f32"),
        # the key projections of eight layers at once
        dict(name="ns_kv_batch", op="newton_schulz", batch=8, rows=1024, cols=4096, dtype="bf16"),
        # a small model's matrices
        dict(name="muon_small", op="muon_step", shapes="64x64 64x256 256x64", copies=2),
        # the matrices of one transformer layer of the Llama-3-8B-shaped list
        dict(name="muon_layer", op="muon_step",
             shapes="4096x4096 1024x4096 14336x4096 4096x14336", copies=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize_i8", "gemm_i8", "linear_i8", "newton_schulz", "muon_step"])
    if op == "quantize_i8":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 8, 8192),
                    dtype=rng.choice(["bf16", "f32"]), transpose=rng.random() < 0.5,
                    rounding=rng.choice(["rn", "sr"]))
    if op == "gemm_i8":
        return dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 16, 14336), k=_log(rng, 16, 8192),
                    rounding=rng.choice(["rn", "sr"]))
    if op == "linear_i8":
        return dict(op=op, m=_log(rng, 1, 2048), n=_log(rng, 64, 8192), k=_log(rng, 64, 4096))
    if op == "newton_schulz":
        return dict(op=op, batch=rng.choice([1, 1, 2, 3, 5]), rows=_log(rng, 16, 2048),
                    cols=_log(rng, 16, 4096), dtype=rng.choice(["bf16", "f32"]))
    shapes = ["%dx%d" % (_log(rng, 16, 2048), _log(rng, 16, 2048))
              for _ in range(rng.randint(1, 4))]
    return dict(op=op, shapes=" ".join(shapes), copies=rng.randint(1, 3))


def _shapes(case):
    one = [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split()]
    return one * case["copies"]


def work(case):
    op = case["op"]
    if op == "quantize_i8":
        n = case["rows"] * case["cols"]
        groups = case["cols"] if case["transpose"] else case["rows"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (size + 1) + 4 * groups, "flops": 3 * n}
    if op == "gemm_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 2 * m * n + 4 * (m + n), "flops": 2 * m * n * k}
    if op == "linear_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * n * k}

    def ns_flops(rows, cols):
        # the products with a symmetric result need one half of it
        s, t = min(rows, cols), max(rows, cols)
        return NS_STEPS * (s * (s + 1) * t + s * s * (s + 1) + 2 * s * s * t)

    if op == "newton_schulz":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2),
                "flops": case["batch"] * ns_flops(case["rows"], case["cols"])}
    total = sum(r * c for r, c in _shapes(case))
    # gradient read, momentum read and written, weight read and written
    return {"bytes": total * (2 + 8 + 4),
            "flops": sum(ns_flops(r, c) for r, c in _shapes(case))}


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _activations(gen, rows, cols):
    """Normal values with every 64th or so channel ten times as large."""
    gain = torch.ones(cols, device="cuda")
    gain[torch.rand(cols, generator=gen, device="cuda") < 1 / 64] = 10.0
    return _normal(gen, (rows, cols), 1.0) * gain


def _gradient(gen, batch, rows, cols):
    """A few strong directions over a broad floor, as a weight's gradient has."""
    rank = max(1, min(rows, cols) // 16)
    left, right = _normal(gen, (batch, rows, rank), 1.0), _normal(gen, (batch, rank, cols), 1.0)
    strength = torch.logspace(0, -1, rank, device="cuda")
    strong = torch.bmm(left * strength, right) * (2.0 / math.sqrt(rank))
    return (strong + _normal(gen, (batch, rows, cols), 0.5)) * 1e-3


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(case, seed):
    gen, op = _generator(seed), case["op"]
    key = dict(seed=seed & 0xFFFFFFFF, step=3, base_index=4 * (seed % 1000))
    if op == "quantize_i8":
        x = _activations(gen, case["rows"], case["cols"]).to(_dtype(case["dtype"]))
        return dict(x=x, **key)
    if op == "gemm_i8":
        def codes(rows, cols):
            # rows padded to 16 bytes, as the quantiser lays them out
            full = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device="cuda")
            view = full[:, :cols]
            view.copy_(_normal(gen, (rows, cols), 32.0).round().clamp(-127, 127))
            return view

        m, n, k = case["m"], case["n"], case["k"]
        scale_a = torch.rand(m, generator=gen, device="cuda") * 0.05 + 0.01
        scale_b = torch.rand(n, generator=gen, device="cuda") * 0.001 + 0.0002
        return dict(a=codes(m, k), b=codes(n, k), scale_a=scale_a, scale_b=scale_b, **key)
    if op == "linear_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(x=_activations(gen, m, k).bfloat16(),
                    w=_normal(gen, (n, k), 0.02).bfloat16(),
                    dy=_normal(gen, (m, n), 1e-3).bfloat16(), **key)
    if op == "newton_schulz":
        g = _gradient(gen, case["batch"], case["rows"], case["cols"])
        return dict(g=g.to(_dtype(case["dtype"])))
    shapes = _shapes(case)
    sizes = [r * c for r, c in shapes]
    return dict(params=[_normal(gen, s, 0.02).bfloat16() for s in shapes],
                grads=[_gradient(gen, 1, *s)[0].bfloat16() for s in shapes],
                momenta=[_gradient(gen, 1, *s)[0] * 5 for s in shapes],
                bases=[sum(sizes[:i]) for i in range(len(sizes))],
                seed=key["seed"], step=3)


HYPER = dict(lr=0.01, momentum=0.95, weight_decay=0.1)


def prepare(case, seed):
    return dict(case=case, **_inputs(case, seed))


# ------------------------------------------------------------ plain forms
def _wide_product(c, constant):
    """High and low 32 bits of c * constant, c in [0, 2**32) held in int64."""
    low, high = c * (constant & 0xFFFF), c * (constant >> 16)
    return ((low >> 16) + high) >> 16, (low + ((high << 16) & 0xFFFFFFFF)) & 0xFFFFFFFF


def _random16(n, seed, step, base):
    """The stream's 16 random bits of positions base .. base + n - 1."""
    first, last = base // 4, (base + n - 1) // 4
    j = torch.arange(first, last + 1, device="cuda", dtype=torch.int64)
    c = [j & 0xFFFFFFFF, j >> 32, torch.zeros_like(j), torch.zeros_like(j)]
    k0, k1 = seed, step
    for _ in range(10):
        ah, al = _wide_product(c[0], 0xD2511F53)
        bh, bl = _wide_product(c[2], 0xCD9E8D57)
        c = [bh ^ c[1] ^ k0, bl, ah ^ c[3] ^ k1, al]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack(c, 1).reshape(-1) & 0xFFFF
    return words[base - 4 * first:base - 4 * first + n]


def _round_bf16(x, rounding, s, base=None):
    """f32 x to bf16, to nearest or by adding 16 random bits and truncating."""
    if rounding == "rn":
        return x.to(torch.bfloat16)
    bits = x.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    r = _random16(x.numel(), s["seed"], s["step"], s["base_index"] if base is None else base)
    high = (bits + r.view(x.shape)) >> 16
    return (high - ((high >> 15) << 16)).to(torch.int16).view(torch.bfloat16)


def _quantize(x, rounding, s, transpose=False):
    """int8 codes and f32 scales of the rows (transpose: of the columns) of x."""
    r = None
    if rounding == "sr":
        r = _random16(x.numel(), s["seed"], s["step"], s["base_index"]).view(x.shape)
    if transpose:
        x, r = x.t(), None if r is None else r.t()
    x = x.float()
    # 64 bits: torch divides by a number as a product with its reciprocal, and
    # next to a border between two codes 32 bits do not tell the side
    scale = (x.abs().amax(1).double() / 127.0).float()
    t = x.abs().double() / scale[:, None].double()
    q = torch.round(t) if r is None else torch.floor(t + r.double() / 65536.0)
    return (torch.sign(x) * q.clamp(max=127).float()).to(torch.int8), scale


def _product_i8(a, b, scale_a, scale_b):
    return (a.float() @ b.float().t()) * scale_a[:, None] * scale_b


def _orthogonal(g, f):
    """Newton-Schulz on a batch of f32 matrices, in the type f."""
    x = g.transpose(1, 2) if g.shape[1] > g.shape[2] else g
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x.to(f) / (norm + EPS).to(f)).contiguous()
    a, b, c = COEFFS
    for _ in range(NS_STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if g.shape[1] > g.shape[2] else x


def _step_size(rows, cols):
    return HYPER["lr"] * math.sqrt(max(1.0, rows / cols))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize_i8":
        return _quantize(s["x"], case["rounding"], s, case["transpose"])
    if op == "gemm_i8":
        y = _product_i8(s["a"], s["b"], s["scale_a"], s["scale_b"])
        return _round_bf16(y, case["rounding"], s)
    if op == "linear_i8":
        (qx, sx), (qw, sw) = _quantize(s["x"], "rn", s), _quantize(s["w"], "rn", s)
        y = _product_i8(qx, qw, sx, sw)
        (qd, sd), (qwt, swt) = _quantize(s["dy"], "sr", s), _quantize(s["w"], "rn", s, True)
        dx = _product_i8(qd, qwt, sd, swt)
        (qdt, sdt), (qxt, sxt) = _quantize(s["dy"], "sr", s, True), _quantize(s["x"], "rn", s, True)
        dw = _product_i8(qdt, qxt, sdt, sxt)
        return y.bfloat16(), dx.bfloat16(), dw.bfloat16()
    if op == "newton_schulz":
        return _orthogonal(s["g"].float(), torch.float32).bfloat16()
    mu = HYPER["momentum"]
    for p, g, m, base in zip(s["params"], s["grads"], s["momenta"], s["bases"]):
        m.mul_(mu).add_(g.float())
        o = _orthogonal((g.float() + mu * m)[None], torch.float32)[0]
        new = p.float() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - _step_size(*p.shape) * o
        p.copy_(_round_bf16(new, "sr", s, base))
    return s["params"] + s["momenta"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def _own(s):
    from adamw_optimizer_stochastic_amd import linear_i8, ops
    case = s["case"]
    op = case["op"]
    if op == "quantize_i8":
        return ops.quantize_i8(s["x"], transpose=case["transpose"], rounding=case["rounding"],
                               seed=s["seed"], step=s["step"], base_index=s["base_index"])
    if op == "gemm_i8":
        return ops.gemm_i8(s["a"], s["b"], s["scale_a"], s["scale_b"], rounding=case["rounding"],
                           seed=s["seed"], step=s["step"], base_index=s["base_index"])
    if op == "linear_i8":
        x, w = s["x"].detach().requires_grad_(), s["w"].detach().requires_grad_()
        y = linear_i8(x, w, seed=s["seed"], step=s["step"], base_index=s["base_index"])
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"])
        return y.detach(), dx, dw
    if op == "newton_schulz":
        return ops.newton_schulz(s["g"], steps=NS_STEPS, coefficients=COEFFS, eps=EPS)
    ops.muon_step(s["params"], s["grads"], s["momenta"], s["bases"], lr=HYPER["lr"],
                  momentum=HYPER["momentum"], nesterov=True, weight_decay=HYPER["weight_decay"],
                  ns_steps=NS_STEPS, ns_coefficients=COEFFS, eps=EPS, adjust_lr="original",
                  step=s["step"], seed=s["seed"], rounding="sr")
    return s["params"] + s["momenta"]


# ------------------------------------------- the definitions in binary64
# (a bf16 output's value before it is rounded, to nearest or stochastically)
def _exact_bits(n, seed, step, base):
    """Philox4x32-10 by 8-bit limbs of the constants, 16 low bits a position."""
    pos = torch.arange(base, base + n, device="cuda", dtype=torch.int64)
    call = torch.unique_consecutive(pos >> 2)
    mask = 0xFFFFFFFF

    def times(v, constant):
        low = torch.zeros_like(v)
        high = torch.zeros_like(v)
        for shift in (0, 8, 16, 24):
            part = v * ((constant >> shift) & 0xFF)         # below 2**40
            low = low + ((part << shift) & mask)
            high = high + (part >> (32 - shift))
        return (high + (low >> 32)) & mask, low & mask

    w0, w1 = call & mask, call >> 32
    w2, w3 = torch.zeros_like(call), torch.zeros_like(call)
    for r in range(10):
        ka, kb = (seed + r * 0x9E3779B9) & mask, (step + r * 0xBB67AE85) & mask
        (h0, l0), (h2, l2) = times(w0, 0xD2511F53), times(w2, 0xCD9E8D57)
        w0, w1, w2, w3 = h2 ^ w1 ^ ka, l2, h0 ^ w3 ^ kb, l0
    at = (pos >> 2) - call[0]
    lane = pos & 3
    out = torch.where(lane == 0, w0[at], torch.where(lane == 1, w1[at],
                      torch.where(lane == 2, w2[at], w3[at])))
    return (out & 0xFFFF).double() / 65536.0


def _exact_codes(x, transpose, share):
    x = x.double().t() if transpose else x.double()
    scale = (x.abs().amax(1) / 127.0).float()               # the scale is a binary32 number
    t = x.abs() / scale.double()[:, None]
    q = torch.floor(t + (share.t() if transpose else share)) if share is not None else t.round()
    return torch.sign(x) * q.clamp(max=127.0), scale.double()


def exact(case, seed):
    op, s = case["op"], _inputs(case, seed)

    def share(shape):
        n = shape[0] * shape[1]
        return _exact_bits(n, s["seed"], s["step"], s["base_index"]).view(shape)

    if op == "quantize_i8":
        x = s["x"]
        q, _ = _exact_codes(x, case["transpose"], share(x.shape) if case["rounding"] == "sr" else None)
        top = x.double().abs().amax(0 if case["transpose"] else 1) / 127.0
        return q.to(torch.int8), top
    if op == "gemm_i8":
        y = s["a"].double() @ s["b"].double().t()
        return y * s["scale_a"].double()[:, None] * s["scale_b"].double()[None, :]
    if op == "linear_i8":
        bits = share(s["dy"].shape)

        def product(left, right):
            return (left[0] @ right[0].t()) * torch.outer(left[1], right[1])

        x, w, dy = s["x"], s["w"], s["dy"]
        y = product(_exact_codes(x, False, None), _exact_codes(w, False, None))
        dx = product(_exact_codes(dy, False, bits), _exact_codes(w, True, None))
        dw = product(_exact_codes(dy, True, bits), _exact_codes(x, True, None))
        return y, dx, dw

    def polar(g):
        wide = g.shape[-2] <= g.shape[-1]
        z = g.double() if wide else g.double().mT
        z = z / (torch.sqrt((z * z).sum(dim=(-1, -2), keepdim=True)) + EPS)
        one = torch.eye(z.shape[-2], dtype=torch.float64, device=z.device)
        for _ in range(NS_STEPS):
            h = z @ z.mT
            z = (COEFFS[0] * one + h @ (COEFFS[1] * one + COEFFS[2] * h)) @ z
        return z if wide else z.mT

    if op == "newton_schulz":
        return polar(s["g"])
    mu, new_p, new_m = HYPER["momentum"], [], []
    for p, g, m in zip(s["params"], s["grads"], s["momenta"]):
        buf = mu * m.double() + g.double()
        o = polar(g.double() + mu * buf)
        v = p.double() * (1.0 - HYPER["lr"] * HYPER["weight_decay"])
        v = v - HYPER["lr"] * max(1.0, p.shape[0] / p.shape[1]) ** 0.5 * o
        new_p.append(v)
        new_m.append(buf)
    return new_p + new_m
