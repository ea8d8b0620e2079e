"""The operators around 8-bit activation checkpoints, as cases to time and to compare.

A training step keeps the input of each linear layer for the backward pass.  Here it is kept in
8 bits: codes of one byte and one power-of-two scale for each group of 32 columns of a row.  The
RMS norm writes its normalised row in that form, the weight gradient of the layer behind it and
the norm's own backward pass read it, and both gradients are fp32, as the gradient compressor
takes them.

``run`` computes each operator in elementary torch operations, or, where ``own`` is true, through
the framework.  Sizes are those of the repository's workloads (Llama-2-7B: 4096 and 11008,
BERT-large: 1024), rows are tokens, and odd sizes stand for ragged batches and other models.
"""
import numpy as np
import torch

own = False

GROUP = 32
LOWEST, HIGHEST, BAD = 7, 248, 255     # biased exponents of the scales; BAD: the group is NaN
SEED, STEP = 0x1234567890, 3
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST_ELEMENTS = 8192 * 11008           # the largest matrix of the memory-bound operators
MOST_FLOPS = 2 * 8192 * 11008 * 4096   # the largest weight gradient


def listed():
    return [
        # one new token of a served model: latency
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True,
             weight="bf16", stochastic=False),
        # the norm in front of the attention or the MLP, 8192 tokens of a 7B model
        dict(name="norm_train", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True,
             weight="bf16", stochastic=False),
        # a ragged batch in full precision, without a residual stream, rounded stochastically
        dict(name="norm_odd_fp32", op="norm", rows=1537, cols=1023, dtype="fp32", residual=False,
             weight="fp32", stochastic=True),
        # that norm's backward pass, with the gradient of the residual stream joined
        dict(name="norm_grad_train", op="norm_grad", rows=8192, cols=4096, dtype="bf16",
             residual=True, weight="bf16"),
        # a ragged batch in half precision
        dict(name="norm_grad_odd_fp16", op="norm_grad", rows=515, cols=1000, dtype="fp16",
             residual=False, weight="fp32"),
        # the input of one layer kept and read back: a short odd one, in full precision
        dict(name="keep_small_fp32", op="keep", rows=77, cols=333, dtype="fp32",
             stochastic=False),
        # the MLP's hidden activations of 8192 tokens
        dict(name="keep_mlp", op="keep", rows=8192, cols=11008, dtype="bf16", stochastic=False),
        # stochastic rounding, which keeps the gradient's expectation, in half precision
        dict(name="keep_random_fp16", op="keep", rows=2048, cols=4096, dtype="fp16",
             stochastic=True),
        # one sequence of a BERT-large-sized layer: few tiles, a short sum
        dict(name="wgrad_short", op="wgrad", rows=512, cols=1024, n_out=1024, dtype="bf16",
             scale=False),
        # an attention projection of a 7B model behind its norm (the norm's weight scales columns)
        dict(name="wgrad_proj", op="wgrad", rows=4096, cols=4096, n_out=4096, dtype="bf16",
             scale=True),
        # an MLP matrix of a 7B model: the largest
        dict(name="wgrad_mlp", op="wgrad", rows=8192, cols=4096, n_out=11008, dtype="bf16",
             scale=True),
        # nothing divides anything, gradients in full precision
        dict(name="wgrad_odd_fp32", op="wgrad", rows=1531, cols=1000, n_out=1025, dtype="fp32",
             scale=False),
    ]


def _size(rng, low, high, multiple):
    """A size between low and high, even over its logarithm; a multiple of `multiple` or any."""
    v = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 0.5:
        v = max(multiple, v // multiple * multiple)
    return v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "keep", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    rows = _size(rng, 1, 16384, 64)
    cols = _size(rng, 48, 11008, 64)
    if op == "wgrad":
        n_out = _size(rng, 48, 11008, 64)
        rows = max(1, min(rows, MOST_FLOPS // (2 * cols * n_out)))
        return dict(op=op, rows=rows, cols=cols, n_out=n_out, dtype=dtype,
                    scale=rng.random() < 0.5)
    rows = max(1, min(rows, MOST_ELEMENTS // 4 // cols))
    if op == "keep":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, stochastic=rng.random() < 0.3)
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7,
                weight=rng.choice([dtype, "fp32"]))
    if op == "norm":
        case["stochastic"] = rng.random() < 0.3
    return case


def _layout(cols):
    groups = (cols + GROUP - 1) // GROUP
    return groups * GROUP, groups


def _activations(gen, rows, cols, dtype):
    """Activations with a few strong columns and rows of unlike size, as hidden states have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    strong = torch.rand(cols, generator=gen, device="cuda") < 0.01
    x *= torch.where(strong, 12.0, 1.0)
    return x.to(dtype)


def _gradients(gen, rows, cols, dtype):
    """Gradients that arrive from the layer above: small, of unlike size from token to token."""
    d = torch.randn(rows, cols, generator=gen, device="cuda")
    d *= 2e-3 * torch.exp(0.7 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return d.to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rows, cols, dtype = case["rows"], case["cols"], TYPES[case["dtype"]]
    pitch, groups = _layout(cols)
    st = dict(case, eps=1e-5)
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    st["codes"] = empty(rows, pitch, dtype=torch.int8)
    st["exps"] = empty(rows, groups, dtype=torch.uint8)
    if case["op"] in ("norm", "norm_grad"):
        w = 1.0 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
        st["w"] = w.to(TYPES[case["weight"]])
    if case["op"] == "norm":
        st["x"] = _activations(gen, rows, cols, dtype)
        st["res"] = _activations(gen, rows, cols, dtype) if case["residual"] else None
        st["h"] = empty(rows, cols, dtype=dtype) if case["residual"] else None
        st["y"] = empty(rows, cols, dtype=dtype)
        st["rstd"] = empty(rows, dtype=torch.float32)
        st["z"] = empty(rows, cols, dtype=dtype)
    elif case["op"] == "keep":
        st["x"] = _activations(gen, rows, cols, dtype)
        st["z"] = empty(rows, cols, dtype=dtype)
    else:
        x = _activations(gen, rows, cols, torch.float32)
        rstd = torch.rsqrt((x * x).mean(1) + st["eps"])
        codes, exps = _quantise(x * rstd[:, None])
        st["codes"].copy_(codes)
        st["exps"].copy_(exps)
        if case["op"] == "norm_grad":
            st["rstd"] = rstd
            st["dy"] = _gradients(gen, rows, cols, dtype)
            st["dres"] = _gradients(gen, rows, cols, dtype) if case["residual"] else None
            st["dx"] = empty(rows, cols, dtype=dtype)
            st["dw"] = empty(cols, dtype=torch.float32)
        else:
            n_out = case["n_out"]
            st["dy"] = _gradients(gen, rows, n_out, dtype)
            st["scale_k"] = None
            if case["scale"]:
                st["scale_k"] = 1.0 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
            st["dw"] = empty(n_out, cols, dtype=torch.float32)
    return st


# ------------------------------------------------------------------ plain forms
def _product32(a, m):
    """High and low 32 bits of a * m (both below 2^32), in int64."""
    p, q = (a & 0xFFFF) * m, (a >> 16) * m
    return (q + (p >> 16)) >> 16, (p + (q << 16)) & 0xFFFFFFFF


def _draws(rows, pitch, device):
    """24 random bits for each element: Philox4x32-10 at (block lo, block hi, step, 0x54), a block
    for four consecutive elements."""
    block = torch.arange(rows * pitch // 4, device=device)
    c0, c1 = block & 0xFFFFFFFF, block >> 32
    c2, c3 = torch.full_like(block, STEP), torch.full_like(block, 0x54)
    k0, k1 = SEED & 0xFFFFFFFF, SEED >> 32
    for _ in range(10):
        h0, l0 = _product32(c0, 0xD2511F53)
        h1, l1 = _product32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return (torch.stack((c0, c1, c2, c3), 1) >> 8).reshape(rows, pitch)


def _quantise(x, stochastic=False):
    """Codes and biased exponents of the fp32 matrix x."""
    rows, cols = x.shape
    pitch, groups = _layout(cols)
    x = torch.nn.functional.pad(x, (0, pitch - cols)).view(rows, groups, GROUP)
    bits = x.abs().amax(2).view(torch.int32)
    e = (((bits + 0x1FFFF) >> 23) - 6).clamp(min=LOWEST)
    bad = e > HIGHEST
    inverse = ((254 - e.clamp(max=HIGHEST)) << 23).view(torch.float32)
    a = x * inverse[:, :, None]
    if stochastic:
        u = _draws(rows, pitch, x.device).view(rows, groups, GROUP)
        down = a.abs().floor()
        up = u.float() < (a.abs() - down) * 16777216.0
        q = torch.copysign(down + up, a)
    else:
        q = a.round()
    q = torch.where(bad[:, :, None], 0.0, q)
    return q.to(torch.int8).view(rows, pitch), torch.where(bad, BAD, e).to(torch.uint8)


def _restore(codes, exps, cols):
    """The fp32 values that codes and exponents stand for."""
    rows, groups = exps.shape
    scale = (exps.int() << 23).view(torch.float32)
    return (codes.view(rows, groups, GROUP).float() * scale[:, :, None]).view(rows, -1)[:, :cols]


def _run_plain(st):
    op = st["op"]
    if op == "keep":
        x = st["x"]
        codes, exps = _quantise(x.float(), st["stochastic"])
        return [_restore(codes, exps, st["cols"]).to(x.dtype)]
    if op == "norm":
        h = st["x"]
        if st["res"] is not None:
            h = (h.float() + st["res"].float()).to(h.dtype)
        # the mean square in 64 bits: the codes next to a rounding border depend on rstd's last bit
        mean = (h.double() * h.double()).mean(1)
        rstd = (1.0 / torch.sqrt(mean + st["eps"])).float()
        z = h.float() * rstd[:, None]
        y = (z * st["w"].float()).to(h.dtype)
        codes, exps = _quantise(z, st["stochastic"])
        out = [y, rstd, _restore(codes, exps, st["cols"]).to(h.dtype)]
        return out + [h] if st["res"] is not None else out
    z = _restore(st["codes"], st["exps"], st["cols"])
    dy = st["dy"].float()
    if op == "norm_grad":
        t = dy * st["w"].float()
        c = (t * z).mean(1, keepdim=True)
        dx = st["rstd"][:, None] * (t - z * c)
        if st["dres"] is not None:
            dx = dx + st["dres"].float()
        return [dx.to(st["dy"].dtype), (dy * z).sum(0)]
    dw = dy.t() @ z
    if st["scale_k"] is not None:
        dw = dw * st["scale_k"]
    return [dw]


def _run_own(st):
    import gradient_compression_amd as gca
    op = st["op"]
    if op == "keep":
        gca.act_quant(st["x"], st["codes"], st["exps"], stochastic=st["stochastic"], seed=SEED,
                      step=STEP)
        gca.act_restore(st["codes"], st["exps"], st["z"])
        return [st["z"]]
    if op == "norm":
        gca.rmsnorm(st["x"], weight=st["w"], eps=st["eps"], residual=st["res"], h=st["h"],
                    y=st["y"], rstd=st["rstd"], codes=st["codes"], exps=st["exps"],
                    stochastic=st["stochastic"], seed=SEED, step=STEP)
        gca.act_restore(st["codes"], st["exps"], st["z"])
        out = [st["y"], st["rstd"], st["z"]]
        return out + [st["h"]] if st["res"] is not None else out
    if op == "norm_grad":
        gca.rmsnorm_backward(st["dy"], st["codes"], st["exps"], st["rstd"], st["dx"],
                             weight=st["w"], dres=st["dres"], dweight=st["dw"])
        return [st["dx"], st["dw"]]
    gca.act_weight_grad(st["dy"], st["codes"], st["exps"], st["dw"], col_scale=st["scale_k"])
    return [st["dw"]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    rows, cols, s = case["rows"], case["cols"], SIZE[case["dtype"]]
    pitch, groups = _layout(cols)
    n, kept = rows * cols, rows * (pitch + groups)
    if case["op"] == "keep":       # x in, the checkpoint out, the restored values out
        return {"bytes": 2 * n * s + kept, "flops": 6 * n}
    if case["op"] == "norm":       # x (and the residual) in; y (and h), the checkpoint, its values out
        passes = 5 if case["residual"] else 3
        return {"bytes": passes * n * s + kept + 4 * rows + cols * SIZE[case["weight"]],
                "flops": 12 * n}
    if case["op"] == "norm_grad":  # dy, the checkpoint (and the residual's gradient) in; dx, dw out
        passes = 3 if case["residual"] else 2
        return {"bytes": passes * n * s + kept + 4 * rows + cols * (4 + SIZE[case["weight"]]),
                "flops": 10 * n}
    n_out = case["n_out"]
    return {"bytes": rows * n_out * s + kept + 4 * n_out * cols + (4 * cols if case["scale"] else 0),
            "flops": 2 * rows * cols * n_out}


# ------------------------------------------------------------------ 64 bits
def _philox_numpy(blocks):
    """Philox4x32-10 with unsigned 64-bit arithmetic: [blocks, 4] words."""
    i = np.arange(blocks, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    c = [i & low, i >> np.uint64(32), np.full_like(i, STEP), np.full_like(i, 0x54)]
    key = [SEED & 0xFFFFFFFF, SEED >> 32]
    for r in range(10):
        k = [np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF),
             np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ k[0], q & low, (p >> np.uint64(32)) ^ c[3] ^ k[1],
             p & low]
    return np.stack(c, 1)


def _power64(e):
    """2^e in 64 bits, from its bits: pow and exp2 may be off in the last one."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept64(x, stochastic):
    """The values (64 bits) that the checkpoint of x (64 bits, finite) holds."""
    rows, cols = x.shape
    pad = -cols % GROUP
    g = torch.cat((x, x.new_zeros(rows, pad)), 1).view(rows, -1, GROUP)
    frac, power = torch.frexp(g.abs().amax(2, keepdim=True) / 127.0)
    power = torch.where(frac == 0.5, power - 1, power).clamp(min=-120)
    unit = _power64(power)
    a = g / unit
    if stochastic:
        words = _philox_numpy(rows * (cols + pad) // 4) >> np.uint64(8)
        u = torch.from_numpy(words.astype(np.float64)).to(x.device).view_as(a) / 2.0 ** 24
        m = a.abs()
        q = torch.sign(a) * (m.floor() + (u < m - m.floor()))
    else:
        q = torch.round(a)
    return (q * unit).view(rows, -1)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op, eps = case["op"], st["eps"]
    if case.get("stochastic") and case["rows"] * case["cols"] > 1 << 25:
        return None
    if op == "keep":
        return [_kept64(st["x"].double(), case["stochastic"])]
    if op == "norm":
        h = st["x"].double()
        if st["res"] is not None:
            # the norm is of the stream as it is stored
            h = (h + st["res"].double()).to(st["x"].dtype).double()
        rstd = (h.square().sum(1) / case["cols"] + eps).rsqrt()
        # what is kept is, by definition, the product of h and rstd, each in 32 bits, in 32 bits
        kept = _kept64((h * rstd.float().double().unsqueeze(1)).float().double(),
                       case["stochastic"])
        out = [h * rstd.unsqueeze(1) * st["w"].double(), rstd, kept]
        return out + [st["x"].double() + st["res"].double()] if st["res"] is not None else out
    unit = _power64(st["exps"].long() - 127).repeat_interleave(GROUP, 1)
    z = (st["codes"].double() * unit)[:, :case["cols"]]
    dy = st["dy"].double()
    if op == "norm_grad":
        t = dy * st["w"].double()
        inner = (t * z).sum(1, keepdim=True) / case["cols"]
        dx = (t - z * inner) * st["rstd"].double().unsqueeze(1)
        if st["dres"] is not None:
            dx = dx + st["dres"].double()
        return [dx, torch.einsum("mk,mk->k", dy, z)]
    dw = torch.matmul(z.t().contiguous(), dy).t()
    return [dw * st["scale_k"].double() if st["scale_k"] is not None else dw]
