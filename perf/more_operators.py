"""Benchmark cases of the layers between the products, and of activations kept in 8 bits.

    pack_i8     a matrix to 8-bit codes, one scale a block of 128 columns, and back
    layer_norm  normalised rows with weight and bias; gradients of all three
    silu_mul    silu(gate) * up of a gated MLP; both gradients
    linear_i8   y = x W^T and its gradients in int8, x kept for them in 8 bits
    embedding   rows of a table, scaled; the table's gradient in a fixed order

``run`` computes each in plain torch operations where ``own`` is false, and
through the package's entry points where it is true. ``exact`` gives the
same from the definitions in binary64. Hidden size 4096, MLP width 14336 and
the vocabulary of 128256 are those of the benchmark's Llama-3-8B-shaped list.
"""

import math

import torch

own = False

BLOCK = 128
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's activations before a projection
        dict(name="norm_token", op="layer_norm", rows=1, cols=4096, dtype="bf16", wdtype="bf16",
             train=False, saved="input"),
        # a training step's norm over 8,192 tokens, its input kept
        dict(name="norm_train", op="layer_norm", rows=8192, cols=4096, dtype="bf16",
             wdtype="bf16", train=True, saved="input"),
        # the same with the normalised rows kept in 8 bits, an odd width and f32 weights
        dict(name="norm_odd_i8", op="layer_norm", rows=2047, cols=1111, dtype="bf16",
             wdtype="f32", train=True, saved="i8"),
        # a gated MLP's activation for one decoded token
        dict(name="silu_token", op="silu_mul", rows=1, cols=14336, dtype="bf16", joint=True,
             train=False, saved="inputs"),
        # the same in a training step over 8,192 tokens, its inputs kept in 8 bits
        dict(name="silu_train_i8", op="silu_mul", rows=8192, cols=14336, dtype="bf16", joint=True,
             train=True, saved="i8"),
        # a small model's activations in f32, packed by stochastic rounding
        dict(name="pack_small", op="pack_i8", rows=67, cols=512, dtype="f32", rounding="sr"),
        # the MLP activations of 8,192 tokens, packed and unpacked
        dict(name="pack_large", op="pack_i8", rows=8192, cols=14336, dtype="bf16", rounding="rn"),
        # a small model's layer in training, its input kept in 8 bits
        dict(name="linear_small_i8", op="linear_i8", m=67, n=512, k=256),
        # a training step's up projection, its input kept in 8 bits
        dict(name="linear_train_i8", op="linear_i8", m=4096, n=14336, k=4096),
        # a decoding batch's tokens
        dict(name="embed_tokens", op="embedding", tokens=16, vocab=128256, dim=4096, dtype="bf16",
             ids="int64", pad=False, scale=1.0, train=False),
        # a small model with an odd width, scaled by sqrt(dim), rows of padding among the tokens
        dict(name="embed_small", op="embedding", tokens=777, vocab=1009, dim=333, dtype="f32",
             ids="int32", pad=True, scale=math.sqrt(333.0), train=True),
        # a training step's 8,192 tokens over the large vocabulary
        dict(name="embed_train", op="embedding", tokens=8192, vocab=128256, dim=4096, dtype="bf16",
             ids="int64", pad=False, scale=1.0, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "silu_mul", "pack_i8", "linear_i8", "embedding"])
    train = rng.random() < 0.75
    if op == "layer_norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 8, 8192), dtype=dtype,
                    wdtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), train=train,
                    saved=rng.choice(["input", "i8"]))
    if op == "silu_mul":
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 8, 14336),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), joint=rng.random() < 0.5,
                    train=train, saved=rng.choice(["inputs", "i8"]))
    if op == "pack_i8":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 8, 8192),
                    dtype=rng.choice(["bf16", "f32"]), rounding=rng.choice(["rn", "sr"]))
    if op == "linear_i8":
        return dict(op=op, m=_log(rng, 1, 2048), n=_log(rng, 64, 8192), k=_log(rng, 64, 4096))
    dim = _log(rng, 8, 4096)
    return dict(op=op, tokens=_log(rng, 1, 32768 if dim <= 1024 else 8192),
                vocab=_log(rng, 2, 128256), dim=dim,
                dtype=rng.choice(["bf16", "f32"]) if dim <= 2048 else "bf16",
                ids=rng.choice(["int64", "int32"]), pad=rng.random() < 0.5,
                scale=rng.choice([1.0, math.sqrt(dim)]), train=train)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op = case["op"]
    if op == "linear_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * n * k}
    if op == "embedding":
        n, vocab, dim, size = case["tokens"], case["vocab"], case["dim"], _size(case["dtype"])
        index = n * (8 if case["ids"] == "int64" else 4)
        if not case["train"]:
            return {"bytes": index + 2 * min(n, vocab) * dim * size
                    + max(0, n - vocab) * dim * size, "flops": n * dim}
        # rows read (no more than there are) and written, the gradient read, the table's written
        return {"bytes": index + (min(n, vocab) + 2 * n + vocab) * dim * size,
                "flops": 3 * n * dim}
    n, size = case["rows"] * case["cols"], _size(case["dtype"])
    if op == "pack_i8":
        # the values read, and written as they come back
        return {"bytes": 2 * n * size, "flops": 4 * n}
    if op == "layer_norm":
        params = case["cols"] * _size(case["wdtype"])
        if not case["train"]:
            return {"bytes": 2 * n * size + 2 * params, "flops": 8 * n}
        return {"bytes": 4 * n * size + 4 * params, "flops": 22 * n}
    if not case["train"]:
        return {"bytes": 3 * n * size, "flops": 6 * n}
    return {"bytes": 6 * n * size, "flops": 18 * n}


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _activations(gen, rows, cols, offset=0.0):
    """Normal values, every 64th or so channel ten times as large."""
    gain = torch.ones(cols, device="cuda")
    gain[torch.rand(cols, generator=gen, device="cuda") < 1 / 64] = 10.0
    return (_normal(gen, (rows, cols), 1.0) + offset) * gain


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _tokens(gen, n, vocab, pad):
    """Ids with the frequencies of text (the k-th most frequent about 1/k), spread over
    the table; where there is padding, the last tenth is id 0."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp(0, vocab - 1)
    ids = (rank * 7919 + 13) % vocab
    if pad:
        ids[n - n // 10:] = 0
    return ids


def _inputs(case, seed):
    gen, op = _generator(seed), case["op"]
    key = dict(seed=seed & 0xFFFFFFFF, step=3, base_index=4 * (seed % 1000))
    if op == "linear_i8":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(x=_activations(gen, m, k).bfloat16(), w=_normal(gen, (n, k), 0.02).bfloat16(),
                    dy=_normal(gen, (m, n), 1e-3).bfloat16(), **key)
    f = _dtype(case["dtype"])
    if op == "embedding":
        n, dim = case["tokens"], case["dim"]
        ids = _tokens(gen, n, case["vocab"], case["pad"])
        return dict(ids=ids if case["ids"] == "int64" else ids.int(),
                    w=_normal(gen, (case["vocab"], dim), 0.02).to(f),
                    dy=_normal(gen, (n, dim), 1e-3).to(f))
    rows, cols = case["rows"], case["cols"]
    if op == "pack_i8":
        return dict(x=_activations(gen, rows, cols).to(f), **key)
    if op == "layer_norm":
        wf = _dtype(case["wdtype"])
        return dict(x=_activations(gen, rows, cols, 0.1).to(f),
                    w=(1.0 + _normal(gen, (cols,), 0.1)).to(wf), b=_normal(gen, (cols,), 0.1).to(wf),
                    dy=_normal(gen, (rows, cols), 1e-3).to(f))
    dy = _normal(gen, (rows, cols), 1e-3).to(f)
    if case["joint"]:
        return dict(gate=_activations(gen, rows, 2 * cols).to(f), up=None, dy=dy)
    return dict(gate=_activations(gen, rows, cols).to(f), up=_activations(gen, rows, cols).to(f),
                dy=dy)


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


def _codes(x, r=None):
    """int8 codes (as f32) and f32 scales of x's last dimension, r the random bits."""
    # 64 bits: next to a border between two codes 32 bits do not tell the side
    scale = (x.abs().amax(-1).double() / 127.0).float()
    t = x.abs().double() / scale[..., None].double()
    q = torch.round(t) if r is None else torch.floor(t + r.double() / 65536.0)
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q))
    return (torch.sign(x) * q.clamp(max=127.0)).float(), scale


def _blocks(x):
    rows, cols = x.shape
    pad = -cols % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros((rows, pad))], 1)
    return x.view(rows, -1, BLOCK)


def _through_8_bits(x, r=None):
    """What the codes of x stand for, in f32, one scale a block of 128 columns."""
    q, scale = _codes(_blocks(x), None if r is None else _blocks(r))
    return (q * scale[..., None]).view(x.shape[0], -1)[:, :x.shape[1]]


def _plain_linear(s):
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    r = _random16(dy.numel(), s["seed"], s["step"], s["base_index"]).view(dy.shape)
    (qx, sx), (qw, sw) = _codes(x), _codes(w)
    y = (qx @ qw.t()) * sx[:, None] * sw
    (qd, sd), (qwt, swt) = _codes(dy, r), _codes(w.t())
    dx = (qd @ qwt.t()) * sd[:, None] * swt
    qz, sz = _codes((dy * sx[:, None]).t(), r.t())
    dw = (qz @ qx) * sz[:, None]
    return y.bfloat16(), dx.bfloat16(), dw.bfloat16()


def _plain_norm(s):
    case, x, w, b = s["case"], s["x"].float(), s["w"].float(), s["b"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    xh = (x - mean) * rstd
    y = (xh * w + b).to(s["x"].dtype)
    if not case["train"]:
        return y
    if case["saved"] == "i8":
        # 64 bits: the rows' values next to a border between two codes
        x = s["x"].double()
        x = x - x.mean(1, keepdim=True)
        xh = _through_8_bits(x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS))
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return (y, dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["w"].dtype),
            dy.sum(0).to(s["b"].dtype))


def _plain_silu(s):
    case, f, cols = s["case"], s["gate"].dtype, s["case"]["cols"]
    gate = s["gate"].float()
    gate, up = (gate[:, :cols], gate[:, cols:]) if case["joint"] else (gate, s["up"].float())
    y = (gate / (1.0 + torch.exp(-gate)) * up).to(f)
    if not case["train"]:
        return y
    if case["saved"] == "i8":
        gate, up = _through_8_bits(gate), _through_8_bits(up)
    dy = s["dy"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgate, dup = dy * up * sig * (1.0 + gate * (1.0 - sig)), dy * gate * sig
    if case["joint"]:
        return y, torch.cat([dgate, dup], 1).to(f)
    return y, dgate.to(f), dup.to(f)


def _plain_embedding(s):
    case, w, ids = s["case"], s["w"], s["ids"].long()
    y = (w[ids].float() * case["scale"]).to(w.dtype)
    if not case["train"]:
        return y
    dw = torch.zeros(w.shape, dtype=torch.float32, device="cuda")
    dw.index_add_(0, ids, s["dy"].float())
    if case["pad"]:
        dw[0] = 0.0
    return y, (dw * case["scale"]).to(w.dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "linear_i8":
        return _plain_linear(s)
    if op == "layer_norm":
        return _plain_norm(s)
    if op == "silu_mul":
        return _plain_silu(s)
    if op == "embedding":
        return _plain_embedding(s)
    x = s["x"]
    r = None
    if s["case"]["rounding"] == "sr":
        r = _random16(x.numel(), s["seed"], s["step"], s["base_index"]).view(x.shape)
    return _through_8_bits(x.float(), r).to(x.dtype)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def _own(s):
    from adamw_optimizer_stochastic_amd import embedding, layer_norm, linear_i8, ops, silu_mul
    case = s["case"]
    op = case["op"]
    if op == "pack_i8":
        q, scale = ops.pack_i8(s["x"], rounding=case["rounding"], seed=s["seed"], step=s["step"],
                               base_index=s["base_index"])
        return ops.unpack_i8(q, scale, dtype=s["x"].dtype)
    if op == "linear_i8":
        x, w = s["x"].detach().requires_grad_(), s["w"].detach().requires_grad_()
        y = linear_i8(x, w, seed=s["seed"], step=s["step"], base_index=s["base_index"],
                      saved="i8")
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"])
        return y.detach(), dx, dw
    if op == "layer_norm":
        if not case["train"]:
            return layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        leaves = [s[name].detach().requires_grad_() for name in ("x", "w", "b")]
        y = layer_norm(*leaves, eps=EPS, saved=case["saved"])
        return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"]))
    if op == "silu_mul":
        if not case["train"]:
            return silu_mul(s["gate"], s["up"])
        leaves = [t.detach().requires_grad_() for t in (s["gate"], s["up"]) if t is not None]
        y = silu_mul(*leaves, saved=case["saved"])
        return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"]))
    padding = 0 if case["pad"] else None
    if not case["train"]:
        return embedding(s["ids"], s["w"], scale=case["scale"], padding_idx=padding)
    w = s["w"].detach().requires_grad_()
    y = embedding(s["ids"], w, scale=case["scale"], padding_idx=padding)
    return y.detach(), *torch.autograd.grad(y, w, s["dy"])


# ------------------------------------------- the definitions in binary64
# (an output's value before it is rounded to the output's type)
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


def _exact_codes(x, share=None):
    """Codes of binary64 rows, and their scales: binary32 numbers by definition."""
    scale = (x.abs().amax(1) / 127.0).float().double()
    t = x.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = t.round() if share is None else torch.floor(t + share)
    return torch.sign(x) * q.clamp(max=127.0), scale


def _exact_through(x, share=None):
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        part = slice(c, min(c + BLOCK, x.shape[1]))
        q, scale = _exact_codes(x[:, part], None if share is None else share[:, part])
        out[:, part] = q * scale[:, None]
    return out


def exact(case, seed):
    op, s = case["op"], _inputs(case, seed)
    if op == "pack_i8":
        x = s["x"].double()
        share = None
        if case["rounding"] == "sr":
            share = _exact_bits(x.numel(), s["seed"], s["step"], s["base_index"]).view(x.shape)
        return _exact_through(x, share)
    if op == "linear_i8":
        x, w, dy = (s[name].double() for name in ("x", "w", "dy"))
        share = _exact_bits(dy.numel(), s["seed"], s["step"], s["base_index"]).view(dy.shape)
        (qx, sx), (qw, sw) = _exact_codes(x), _exact_codes(w)
        y = (qx @ qw.t()) * torch.outer(sx, sw)
        (qd, sd), (qwt, swt) = _exact_codes(dy, share), _exact_codes(w.t())
        dx = (qd @ qwt.t()) * torch.outer(sd, swt)
        # the weighted gradient is a binary32 number by definition
        z = (dy * sx[:, None]).float().double()
        qz, sz = _exact_codes(z.t(), share.t())
        return y, dx, (qz @ qx) * sz[:, None]
    if op == "embedding":
        ids, scale = s["ids"].long(), case["scale"]
        y = s["w"].double()[ids] * scale
        if not case["train"]:
            return y
        order = torch.argsort(ids, stable=True)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        dw.index_put_((ids[order],), s["dy"].double()[order] * scale, accumulate=True)
        if case["pad"]:
            dw[0] = 0.0
        return y, dw
    if op == "layer_norm":
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        xh = (x - mean) / (var + EPS).sqrt()
        y = b + w * xh
        if not case["train"]:
            return y
        if case["saved"] == "i8":
            xh = _exact_through(xh)
        dy, n = s["dy"].double(), x.shape[1]
        dxh = dy * w
        dx = n * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True)
        return y, dx / (n * (var + EPS).sqrt()), torch.einsum("rc,rc->c", dy, xh), dy.sum(0)
    gate = s["gate"].double()
    gate, up = gate.chunk(2, 1) if case["joint"] else (gate, s["up"].double())
    y = gate * torch.sigmoid(gate) * up
    if not case["train"]:
        return y
    if case["saved"] == "i8":
        gate, up = _exact_through(gate), _exact_through(up)
    dy, sig = s["dy"].double(), torch.sigmoid(gate)
    slope = sig + gate * sig * (1.0 - sig)
    if case["joint"]:
        return y, torch.cat([dy * up * slope, dy * gate * sig], 1)
    return y, dy * up * slope, dy * gate * sig
