"""The gated feed-forward block, its backward pass, and the clipping of a model's gradients by their
global norm, as cases to time and to compare.

The block takes the rows behind a norm (cols wide) through two projections of n columns each, the
gate's activation and the product: h = act(x Wg^T) * (x Wu^T).  Its backward pass starts from h's
gradient and the kept gate and up rows, and ends in their gradients (which the weight gradients are
formed from) and in the gradient of x.  The gradients of all tensors of the model are then scaled by
one factor, so that their norm is at most max_norm, and laid into the flat fp32 buffer that the
gradient compressor takes; or looked at where they lie, and left alone where the norm is small enough.

``run`` computes each operator in elementary torch operations, or, where ``own`` is true, through
the framework.  Sizes are those of the repository's workloads (Llama-2-7B: 4096 and 11008,
BERT-large: 1024 and 4096, the tensors of ResNet-50, BERT-large and Llama-2-7B), rows are tokens, and
odd sizes stand for ragged batches and other models.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST_PRODUCTS = 8192 * 4096 * 11008    # rows * cols * n of the largest block
MOST_GRADIENTS = 1 << 29               # elements of the largest drawn set of gradients


def listed():
    return [
        # one new token of a served 7B model: its weights are read once, latency counts
        dict(name="block_token", op="block", rows=1, cols=4096, n=11008, dtype="bf16", act="silu",
             keep=False),
        # an odd batch of served sequences, a token each
        dict(name="block_batch", op="block", rows=27, cols=4096, n=11008, dtype="bf16", act="silu",
             keep=False),
        # one sequence of a BERT-large-sized block in half precision: few tiles
        dict(name="block_short_fp16", op="block", rows=512, cols=1024, n=4096, dtype="fp16",
             act="gelu_tanh", keep=True),
        # 8192 tokens of a 7B model in training, gate and up kept for the backward pass: the largest
        dict(name="block_train", op="block", rows=8192, cols=4096, n=11008, dtype="bf16",
             act="silu", keep=True),
        # nothing divides anything, in full precision
        dict(name="block_odd_fp32", op="block", rows=515, cols=1001, n=2731, dtype="fp32",
             act="gelu", keep=True),
        # the backward pass of one BERT-large-sized sequence: few tiles, a long sum
        dict(name="block_grad_short", op="block_grad", rows=512, cols=1024, n=4096, dtype="bf16",
             act="gelu_tanh"),
        # that of 8192 tokens of a 7B model
        dict(name="block_grad_train", op="block_grad", rows=8192, cols=4096, n=11008, dtype="bf16",
             act="silu"),
        # a ragged batch in half precision, rows that start at any element
        dict(name="block_grad_odd_fp16", op="block_grad", rows=1537, cols=1001, n=2731,
             dtype="fp16", act="gelu"),
        # the 161 tensors of ResNet-50, most of them small, looked at where they lie: too small a
        # norm to clip, as in most steps
        dict(name="clip_small_kept", op="clip", model="resnet50", layers=4, dtype="fp32",
             clip=False, flat=False),
        # the 391 tensors of BERT-large, matrices in bf16 and vectors in fp32, into the flat gradient
        dict(name="clip_mixed", op="clip", model="bert_large", layers=24, dtype="bf16", clip=True,
             flat=True),
        # embedding, head and four layers of Llama-2-7B, into the flat gradient
        dict(name="clip_large", op="clip", model="llama2_7b", layers=4, dtype="bf16", clip=True,
             flat=True),
        # a gradient that is flat and in full precision already, as one tensor: nothing to clip
        dict(name="clip_flat_kept", op="clip", model="one", layers=1, dtype="fp32", clip=False,
             flat=False, elements=335141888),
    ]


def _size(rng, low, high, multiple):
    """A size between low and high, even over its logarithm; a multiple of `multiple` or any."""
    v = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 0.5:
        v = max(multiple, v // multiple * multiple)
    return v


def draw(rng):
    op = rng.choice(["block", "block_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "clip":
        case = dict(op=op, model="drawn", layers=rng.randint(1, 400), dtype=dtype,
                    clip=rng.random() < 0.6, flat=rng.random() < 0.6, sizes=rng.randrange(1 << 30),
                    most=_size(rng, 64, 1 << 26, 64))
        # clipped where they lie, the gradients would be other ones in the next pass
        case["flat"] = case["flat"] or case["clip"]
        return case
    rows, cols, n = _size(rng, 1, 8192, 64), _size(rng, 48, 8192, 64), _size(rng, 48, 11008, 64)
    rows = max(1, min(rows, MOST_PRODUCTS // (cols * n) // (16 if dtype == "fp32" else 1)))
    case = dict(op=op, rows=rows, cols=cols, n=n, dtype=dtype,
                act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    if op == "block":
        case["keep"] = rng.random() < 0.6
    return case


# ------------------------------------------------------------------ inputs
def _shapes(case):
    """The elements of each tensor of a model, and whether it is a matrix."""
    model, layers = case["model"], case["layers"]
    if model == "one":
        return [(case["elements"], True)]
    if model == "drawn":      # a spread of sizes from the case's own number; tensors of none among them
        sizes, state, left = [], case["sizes"], MOST_GRADIENTS
        for _ in range(layers):
            state = (state * 6364136223846793005 + 1442695040888963407) % (1 << 64)
            part = (state >> 33) / (1 << 31)
            n = min(left, int(case["most"] ** part) if part > 0.02 or not sizes else 0)
            left -= n
            sizes.append((n, (state >> 20) % 3 > 0))
        return sizes
    if model == "resnet50":
        out, planes_in = [(64 * 3 * 49, True), (64, False), (64, False)], 64
        for planes, blocks in [(64, 3), (128, 4), (256, 6), (512, 3)][:layers]:
            for b in range(blocks):
                out += [(planes * planes_in, True), (planes, False), (planes, False),
                        (planes * planes * 9, True), (planes, False), (planes, False),
                        (planes * 4 * planes, True), (planes * 4, False), (planes * 4, False)]
                if b == 0:
                    out += [(planes * 4 * planes_in, True), (planes * 4, False), (planes * 4, False)]
                planes_in = planes * 4
        return out + [(1000 * 2048, True), (1000, False)]
    if model == "bert_large":
        h, f = 1024, 4096
        out = [(30522 * h, True), (512 * h, True), (2 * h, True), (h, False), (h, False)]
        for _ in range(layers):
            out += [(h * h, True), (h, False)] * 4 + [(h, False), (h, False)]
            out += [(f * h, True), (f, False), (h * f, True), (h, False), (h, False), (h, False)]
        return out + [(h * h, True), (h, False)]
    h, f = 4096, 11008
    out = [(32000 * h, True)]
    for _ in range(layers):
        out += [(h * h, True)] * 4 + [(f * h, True)] * 3 + [(h, False)] * 2
    return out + [(h, False), (32000 * h, True)]


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols, dtype):
    """Normalised rows with a few strong columns, as behind a norm."""
    strong = torch.rand(cols, generator=gen, device="cuda") < 0.01
    return (_normal(gen, rows, cols) * torch.where(strong, 6.0, 0.9)).to(dtype)


def _prepare_clip(case, gen):
    shapes = _shapes(case)
    # matrices in the case's type, vectors in fp32, as mixed-precision programs keep them; of unlike
    # size from tensor to tensor
    scale = (1e-3 * torch.exp(0.7 * _normal(gen, len(shapes)))).tolist()
    kinds = [TYPES[case["dtype"]] if matrix else torch.float32 for _, matrix in shapes]
    st = dict(case, buckets=[])
    if case["flat"]:
        grads = [torch.empty(n, dtype=k, device="cuda") for (n, _), k in zip(shapes, kinds)]
    else:                     # back to back in a bucket for each type, as data-parallel programs have them
        parts = {k: [n if k == kind else 0 for (n, _), kind in zip(shapes, kinds)] for k in set(kinds)}
        held = {k: torch.empty(sum(n), dtype=k, device="cuda") for k, n in parts.items()}
        views = {k: held[k].split(n) for k, n in parts.items()}
        grads = [views[k][i] for i, k in enumerate(kinds)]
        st["buckets"] = [held[k] for k in TYPES.values() if k in held]
    for t, s in zip(grads, scale):
        t.normal_(0.0, s, generator=gen)
    expected = math.sqrt(sum(n * s * s for (n, _), s in zip(shapes, scale)))
    st["grads"], st["max_norm"] = grads, (0.37 if case["clip"] else 3.0) * expected + 1e-9
    st["norm"] = torch.empty(1, device="cuda")
    st["norms"] = torch.empty(len(grads), device="cuda")
    st["out"] = torch.empty(sum(n for n, _ in shapes), device="cuda") if case["flat"] else None
    return st


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, gen)
    rows, cols, n, dtype = case["rows"], case["cols"], case["n"], TYPES[case["dtype"]]
    empty = lambda *shape: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    st = dict(case)
    st["wg"] = (_normal(gen, n, cols) * (1.2 / math.sqrt(cols))).to(dtype)
    st["wu"] = (_normal(gen, n, cols) * (1.0 / math.sqrt(cols))).to(dtype)
    if case["op"] == "block":
        st["x"] = _activations(gen, rows, cols, dtype)
        st["h"] = empty(rows, n)
        st["gate"], st["up"] = (empty(rows, n), empty(rows, n)) if case["keep"] else (None, None)
    else:
        st["gate"] = (1.5 * _normal(gen, rows, n)).to(dtype)
        st["up"] = _normal(gen, rows, n).to(dtype)
        # gradients that arrive from the layer above: small, of unlike size from token to token
        st["dh"] = (2e-3 * _normal(gen, rows, n) * torch.exp(0.7 * _normal(gen, rows, 1))).to(dtype)
        st["dgate"], st["dup"], st["dx"] = empty(rows, n), empty(rows, n), empty(rows, cols)
    return st


# ------------------------------------------------------------------ plain forms
def _act32(name, g):
    """(act(g), act'(g)) in 32 bits."""
    if name == "silu":
        s, t = torch.sigmoid(g), torch.sigmoid(-g)
        return g * s, s * (1.0 + g * t)
    if name == "gelu":
        phi = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = 2.0 * math.sqrt(2.0 / math.pi)
    inner = c * (g + 0.044715 * g * g * g)
    s, t = torch.sigmoid(inner), torch.sigmoid(-inner)
    return g * s, s + g * s * t * (c * (1.0 + 0.134145 * g * g))


def _run_plain(st):
    if st["op"] == "clip":
        # the squares of long sums in 64 bits
        squares = torch.stack([t.float().square().sum(dtype=torch.float64) for t in st["grads"]])
        norm = squares.sum().sqrt().float()
        f = torch.where(norm > st["max_norm"], st["max_norm"] / norm, 1.0)
        if st["flat"]:
            return [norm.view(1), squares.sqrt().float(),
                    torch.cat([t.float() for t in st["grads"]]).mul_(f)]
        [t.mul_(f) for t in st["grads"]]
        return [norm.view(1), squares.sqrt().float(), *st["buckets"]]
    wg, wu = st["wg"].float(), st["wu"].float()
    if st["op"] == "block":
        x, dtype = st["x"].float(), st["x"].dtype
        gate, up = x @ wg.t(), x @ wu.t()
        out = [(_act32(st["act"], gate)[0] * up).to(dtype)]
        return out + [gate.to(dtype), up.to(dtype)] if st["keep"] else out
    dh, dtype = st["dh"].float(), st["dh"].dtype
    act, slope = _act32(st["act"], st["gate"].float())
    dgate, dup = (dh * st["up"].float() * slope).to(dtype), (dh * act).to(dtype)
    # dx is of the gradients as they are stored, which the weight gradients are formed from too
    return [dgate, dup, (dgate.float() @ wg + dup.float() @ wu).to(dtype)]


def _run_own(st):
    import gradient_compression_amd as gca
    if st["op"] == "clip":
        gca.clip_grad_norm(st["grads"], st["max_norm"], st["norm"], out=st["out"],
                           norms=st["norms"])
        out = [st["out"]] if st["flat"] else st["buckets"]
        return [st["norm"], st["norms"], *out]
    if st["op"] == "block":
        gca.gated_linear(st["x"], st["wg"], st["wu"], st["h"], gate=st["gate"], up=st["up"],
                         activation=st["act"])
        return [st["h"], st["gate"], st["up"]] if st["keep"] else [st["h"]]
    gca.gated_linear_backward(st["dh"], st["gate"], st["up"], st["dgate"], st["dup"],
                              w_gate=st["wg"], w_up=st["wu"], dx=st["dx"], activation=st["act"])
    return [st["dgate"], st["dup"], st["dx"]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"] == "clip":
        shapes = _shapes(case)
        n = sum(m for m, _ in shapes)
        held = sum(m * (s if matrix else 4) for m, matrix in shapes)
        # read once; the flat gradient is written, what lies where it is is left
        return {"bytes": held + (4 * n if case["flat"] else 0) + 4 * len(shapes) + 4,
                "flops": 3 * n if case["flat"] else 2 * n}
    rows, cols, n = case["rows"], case["cols"], case["n"]
    if case["op"] == "block":      # x and both weights in; h (and gate and up) out
        return {"bytes": s * (rows * cols + 2 * n * cols + rows * n * (3 if case["keep"] else 1)),
                "flops": 4 * rows * cols * n + 8 * rows * n}
    # dh, gate, up and both weights in; dgate, dup and dx out
    return {"bytes": s * (5 * rows * n + 2 * n * cols + rows * cols),
            "flops": 4 * rows * cols * n + 16 * rows * n}


# ------------------------------------------------------------------ 64 bits
def _logistic64(v):
    """(sigmoid, its complement) without cancellation, from the exponential of -|v|."""
    e = (-v.abs()).exp()
    large, small = 1.0 / (1.0 + e), e / (1.0 + e)
    return torch.where(v >= 0, large, small), torch.where(v >= 0, small, large)


def _act64(name, g):
    if name == "gelu":
        cumulative = torch.special.ndtr(g)
        density = (g.square() / -2.0).exp() / math.sqrt(2.0 * math.pi)
        return g * cumulative, cumulative + g * density
    if name == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        k = math.sqrt(8.0 / math.pi)
        v, dv = k * g * (1.0 + 0.044715 * g.square()), k * (1.0 + 3 * 0.044715 * g.square())
    p, q = _logistic64(v)
    return g * p, p + g * p * q * dv


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norms = torch.stack([torch.linalg.vector_norm(t, dtype=torch.float64) for t in st["grads"]])
        norm = torch.linalg.vector_norm(norms)
        f = min(1.0, st["max_norm"] / norm.item()) if norm.item() > 0 else 1.0
        if case["flat"]:
            return [norm.view(1), norms, torch.cat([t.double() for t in st["grads"]]) * f]
        return [norm.view(1), norms, *[t.double() * f for t in st["buckets"]]]
    wg, wu = st["wg"].double(), st["wu"].double()
    if case["op"] == "block":
        x = st["x"].double()
        gate, up = torch.mm(wg, x.t()).t(), torch.mm(wu, x.t()).t()
        h = _act64(case["act"], gate)[0] * up
        return [h, gate, up] if case["keep"] else [h]
    dh = st["dh"].double()
    act, slope = _act64(case["act"], st["gate"].double())
    dgate, dup = dh * slope * st["up"].double(), dh * act
    # dx is, by definition, of dgate and dup as they are stored
    dtype = st["dh"].dtype
    stored = torch.cat((dgate.to(dtype), dup.to(dtype)), 1).double()
    return [dgate, dup, torch.mm(stored, torch.cat((wg, wu), 0))]
