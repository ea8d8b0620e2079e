"""The activation operators on the GPU against plain implementations.

The checkpoint is compared bit for bit with the CPU oracle.  The norm is compared bit for bit with
its definition in numpy from the GPU's own rstd (which is within one ulp: its square sum is a double
sum in an unspecified order).  The backward pass and the weight gradient are compared with their
formulas in 64 bits; each tolerance counts the roundings that the definition allows (u = 2^-24, half
a step of fp32), and integer data, whose sums are exact in fp32, has to come out equal.
"""
import numpy as np
import pytest
import torch

import gradient_compression_amd as gca
import oracle
from tests.gpu_helpers import assert_bitwise, log

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
# below the normal numbers the step no longer shrinks with the value: 2^-24 for fp16 (2^-14 with 10
# bits behind the point), so half a step is 2^-25 there
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative


def f32(t):
    return t.detach().float().cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def strided(t, pad, shift=0):
    """The matrix in a wider buffer of sevens (rows `pad` elements apart, `shift` elements off the
    buffer's start), and the buffer."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=t.dtype, device=t.device)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view, buf


def untouched(buf, view):
    """The buffer outside the view still holds its sevens."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[mask] == 7.0).all())


def checkpoint(rows, cols, fill=99):
    pitch, groups = gca.act_layout(cols)
    # a canary row behind each
    codes = torch.full((rows + 1, pitch), fill, dtype=torch.int8, device="cuda")
    exps = torch.full((rows + 1, groups), fill, dtype=torch.uint8, device="cuda")
    return codes, exps


def activations(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_t(4, (rows, cols)) * np.exp(rng.normal(size=(rows, 1)))
    return torch.from_numpy(x.astype(np.float32)).to("cuda").to(TYPES[dtype])


def kept(rows, cols, seed):
    """A checkpoint on the GPU and its values in 64 bits."""
    codes, exps = oracle.act_quant(f32(activations(rows, cols, "f32", seed)))
    z = oracle.act_restore(codes, exps, cols).astype(np.float64)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda(), z


# ---------------------------------------------------------------- the checkpoint
SHAPES = [(1, 1), (1, 32), (3, 33), (7, 31), (5, 8), (2, 1000), (17, 333), (1, 11008), (300, 48),
          (33, 512), (9, 513), (70, 4096), (1, 100003)]


def check_quant(x, random, label):
    rows, cols = x.shape
    codes, exps = checkpoint(rows, cols)
    gca.act_quant(x, codes[:rows], exps[:rows], stochastic=random, seed=0x123456789A, step=77)
    torch.cuda.synchronize()
    want_c, want_e = oracle.act_quant(f32(x).copy(), random=random, seed=0x123456789A, step=77)
    assert_bitwise(exps[:rows], want_e, f"{label} exponents")
    assert_bitwise(codes[:rows], want_c, f"{label} codes")
    assert bool((codes[rows] == 99).all()) and bool((exps[rows] == 99).all())
    return codes[:rows], exps[:rows]


@pytest.mark.parametrize("random", [False, True], ids=["nearest", "stochastic"])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_quant_and_restore_match_the_oracle(dtype, random):
    for n, (rows, cols) in enumerate(SHAPES):
        label = f"{dtype} {rows}x{cols}"
        log(f"[act] {label}")
        x = activations(rows, cols, dtype, n)
        codes, exps = check_quant(x, random, label)
        back = oracle.act_restore(codes.cpu().numpy(), exps.cpu().numpy(), cols)
        for name, t in TYPES.items():
            out, buf = strided(torch.zeros(rows, cols, dtype=t, device="cuda"), 3, 1)
            gca.act_restore(codes, exps, out)
            torch.cuda.synchronize()
            want = torch.from_numpy(back).to(t)
            assert torch.equal(out.cpu(), want), f"{label} restored as {name}"
            assert untouched(buf, out)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (0, 1), (8, 8), (24, 3)])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_quant_of_strided_and_unaligned_rows(dtype, pad, shift):
    for rows, cols in ((5, 64), (4, 1003), (3, 520)):
        x, _ = strided(activations(rows, cols, dtype, rows), pad, shift)
        check_quant(x, False, f"{dtype} {rows}x{cols}+{pad} at {shift}")


def test_quant_ends_of_the_range():
    x = torch.zeros(9, 96)
    x[0, 3], x[1, 95], x[2, 0] = float("inf"), float("nan"), -float("inf")
    x[3, :32] = torch.linspace(-3.3e38, 3.3e38, 32)
    x[4, :3] = torch.tensor([127.0, 0.5, -1.5])
    x[5, :3] = torch.tensor([127.00001, 1.0, 3.0])
    x[6, :4] = torch.tensor([1e-45, 2.0 ** -126, -(2.0 ** -121), 2.0 ** -120])
    x[7] = -0.0
    x[8, :2] = torch.tensor([1.6909e38, 1.0])
    for random in (False, True):
        codes, exps = check_quant(x.cuda(), random, "range")
    out = torch.empty(9, 96, device="cuda")
    gca.act_restore(codes, exps, out)
    nan = torch.isnan(out).cpu()
    assert nan[0, :32].all() and nan[1, 64:].all() and nan[2, :32].all() and nan[3, :32].all()
    assert nan.sum() == 128


def test_every_exponent_is_read_back_exactly():
    """All scales that are written, with all codes, through each reader: the restored matrix, the
    norm's weight gradient and the weight gradient of one row of ones."""
    codes = torch.arange(-127, 129, dtype=torch.int16).clamp(max=127).to(torch.int8).cuda()
    for e in list(range(7, 12)) + [60, 120, 127, 128, 200] + list(range(244, 249)):
        c = codes.view(1, 256)
        x = torch.full((1, 8), e, dtype=torch.uint8, device="cuda")
        want = torch.from_numpy(oracle.act_restore(c.cpu().numpy(), x.cpu().numpy(), 256))
        assert torch.isfinite(want).all()
        for t in (torch.float32, torch.bfloat16):
            out = torch.empty(1, 256, dtype=t, device="cuda")
            gca.act_restore(c, x, out)
            assert torch.equal(out.float().cpu(), want), f"exponent {e} as {t}"
        one = torch.ones(1, 256, device="cuda")
        dx, dw = torch.empty_like(one), torch.empty(256, device="cuda")
        gca.rmsnorm_backward(one, c, x, one[0, :1], dx, dweight=dw)
        assert torch.equal(dw.cpu(), want[0]), f"exponent {e} in the norm"
        for t in TYPES.values():
            dl = torch.empty(3, 256, device="cuda")
            gca.act_weight_grad(one[:, :3].to(t), c, x, dl)
            assert torch.equal(dl.cpu(), want.expand(3, 256)), f"exponent {e} in the product of {t}"


def test_quant_of_leading_dimensions_and_empty():
    x = activations(6, 70, "bf16", 4)
    codes, exps = check_quant(x, False, "flat")
    c2, e2 = checkpoint(6, 70)
    gca.act_quant(x.view(2, 3, 70), c2[:6], e2[:6])
    assert torch.equal(c2[:6], codes) and torch.equal(e2[:6], exps)
    empty = torch.empty(0, 70, device="cuda")
    gca.act_quant(empty, codes[:0], exps[:0])
    gca.act_restore(codes[:0], exps[:0], empty)
    gca.act_quant(torch.empty(4, 0, device="cuda"), codes[:0], exps[:0])
    with pytest.raises(ValueError):
        gca.act_quant(x.view(2, 3, 70).transpose(0, 1), c2[:6], e2[:6])
    with pytest.raises(ValueError):
        gca.act_quant(x[:, ::2], c2[:6], e2[:6])
    with pytest.raises(ValueError):
        gca.act_quant(x[:1].expand(6, 70), c2[:6], e2[:6])
    with pytest.raises(TypeError):
        gca.act_quant(x.double(), c2[:6], e2[:6])
    with pytest.raises(ValueError):
        gca.act_quant(x, c2, e2[:6])


# ---------------------------------------------------------------- the norm
def check_norm(x, res, w, eps, dtype, h=None, y=None, rstd=None, random=False, label=""):
    """Runs the norm into the given outputs and compares with its definition."""
    rows, cols = x.shape
    hx, hr = f32(x), None if res is None else f32(res)
    hw = np.ones(cols, np.float32) if w is None else f32(w)
    codes, exps = checkpoint(rows, cols)
    rstd = torch.empty(rows, device="cuda") if rstd is None else rstd
    gca.rmsnorm(x, weight=w, eps=eps, residual=res, h=h, y=y, rstd=rstd, codes=codes[:rows],
                exps=exps[:rows], stochastic=random, seed=11, step=5)
    torch.cuda.synchronize()
    want_h = hx if hr is None else f32(torch.from_numpy(hx + hr).to(TYPES[dtype]))
    got = rstd.cpu().numpy()
    with np.errstate(all="ignore"):
        sq = (want_h.astype(np.float64) ** 2).sum(1) / cols + np.float64(np.float32(eps))
        want_r = (1.0 / np.sqrt(sq)).astype(np.float32)
        both = np.isfinite(want_r)
        assert np.array_equal(both, np.isfinite(got)), f"{label} rstd finite"
        assert (np.abs(got - want_r)[both] <= np.spacing(want_r[both])).all(), f"{label} rstd"
        z = want_h * got[:, None]
        want_y = torch.from_numpy(z * hw).to(TYPES[dtype])
    if h is not None:
        assert torch.equal(h.cpu().float(), torch.from_numpy(want_h)), f"{label} h"
    if y is not None and y.data_ptr() not in (x.data_ptr(),):
        assert torch.equal(torch.nan_to_num(y.cpu(), 3.0), torch.nan_to_num(want_y, 3.0)), f"{label} y"
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want_y))
    want_c, want_e = oracle.act_quant(np.ascontiguousarray(z), random=random, seed=11, step=5)
    assert_bitwise(exps[:rows], want_e, f"{label} exponents")
    assert_bitwise(codes[:rows], want_c, f"{label} codes")
    assert bool((codes[rows] == 99).all()) and bool((exps[rows] == 99).all())
    return want_y


NORM_SHAPES = [(1, 1), (3, 33), (5, 512), (4, 513), (2, 1000), (9, 1025), (3, 2048), (2, 2049),
               (3, 4096), (2, 4104), (2, 8192), (3, 8200), (2, 16384), (1, 16385), (2, 32768), (530, 64)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_norm_matches_its_definition(dtype):
    for n, (rows, cols) in enumerate(NORM_SHAPES):
        label = f"{dtype} {rows}x{cols}"
        log(f"[norm] {label}")
        x, res = activations(rows, cols, dtype, n), activations(rows, cols, dtype, 100 + n)
        w = torch.rand(cols, device="cuda") + 0.5
        w = w if n % 2 else w.to(TYPES[dtype])
        h, y = torch.empty_like(x), torch.empty_like(x)
        check_norm(x, res, w, 1e-5, dtype, h=h, y=y, label=label)
        check_norm(x, None, None, 1e-6, dtype, y=y, random=True, label=label + " plain")


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_norm_strided_and_in_place(dtype):
    for rows, cols in ((4, 96), (3, 1003), (2, 4100)):
        x, res = activations(rows, cols, dtype, 1), activations(rows, cols, dtype, 2)
        w = torch.rand(cols, device="cuda") + 0.5
        xs, _ = strided(x, 3, 1)
        rs, _ = strided(res, 8, 0)
        (h, hb), (y, yb) = strided(torch.zeros_like(x), 5, 2), strided(torch.zeros_like(x), 16, 8)
        want = check_norm(xs, rs, w, 1e-5, dtype, h=h, y=y, label="strided")
        assert untouched(hb, h) and untouched(yb, y)
        # the stream updated in place, the branch's input overwritten by the norm
        x2, r2 = x.clone(), res.clone()
        gca.rmsnorm(x2, weight=w, eps=1e-5, residual=r2, h=r2, y=x2)
        assert torch.equal(x2.cpu(), want) and torch.equal(r2, h.contiguous())
        x3, r3 = x.clone(), res.clone()
        gca.rmsnorm(x3, weight=w, eps=1e-5, residual=r3, h=x3, y=r3)
        assert torch.equal(r3.cpu(), want) and torch.equal(x3, h.contiguous())
        x4 = x.clone()
        gca.rmsnorm(x4, residual=x4, y=x4, eps=1e-5)      # h = 2 x
        y4 = torch.empty_like(x)
        gca.rmsnorm(x + x, y=y4, eps=1e-5)
        assert torch.equal(x4, y4)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_norm_outputs_are_optional_and_shapes_have_leading_dimensions(dtype):
    shape, cols = (3, 5, 130), 130
    x, res = (activations(15, cols, dtype, i).view(shape) for i in (1, 2))
    w = torch.rand(cols, device="cuda").to(torch.float16)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(3, 5, device="cuda")
    codes, exps = checkpoint(14, cols)
    gca.rmsnorm(x, weight=w, residual=res, h=h, y=y, rstd=rstd, codes=codes, exps=exps)
    for only in (("y",), ("codes", "exps"), ("h", "y"), ("codes", "exps", "rstd"), ("h", "codes", "exps")):
        got = dict(h=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty_like(rstd),
                   codes=torch.empty_like(codes), exps=torch.empty_like(exps))
        gca.rmsnorm(x, weight=w, residual=res, **{k: got[k] for k in only})
        for k in only:
            assert torch.equal(got[k], dict(h=h, y=y, rstd=rstd, codes=codes, exps=exps)[k]), (only, k)
    with pytest.raises(gca.GCError):
        gca.rmsnorm(x, h=h)
    with pytest.raises(ValueError):
        gca.rmsnorm(x, codes=codes)
    with pytest.raises(ValueError):
        gca.rmsnorm(x, y=y.view(15, cols))
    with pytest.raises(TypeError):
        gca.rmsnorm(x, y=y, residual=res.double())
    with pytest.raises(ValueError):
        gca.rmsnorm(x, y=y, weight=w[:-1])
    dx, dw, flat = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(15, cols, dtype=x.dtype, device="cuda")
    dw2 = torch.empty_like(dw)
    gca.rmsnorm_backward(y, codes, exps, rstd, dx, weight=w, dres=h, dweight=dw)
    gca.rmsnorm_backward(y.view(15, cols), codes, exps, rstd, flat, weight=w, dres=h.view(15, cols), dweight=dw2)
    assert torch.equal(dx.view(15, cols), flat) and torch.equal(dw, dw2)
    dl, dl2 = torch.empty(70, cols, device="cuda"), torch.empty(70, cols, device="cuda")
    gca.act_weight_grad(x[..., :70], codes, exps, dl)
    gca.act_weight_grad(x.reshape(15, cols)[:, :70].contiguous(), codes, exps, dl2)
    assert torch.equal(dl, dl2)


@pytest.mark.parametrize("gap", [0, 1, 6])
def test_norm_between_column_blocks_of_one_buffer(gap):
    """x, the residual, h and y side by side in the rows of one buffer: they share no byte."""
    rows, cols = 7, 75
    wide = torch.full((rows, 4 * (cols + gap)), 7.0, device="cuda")
    x, res, h, y = (wide[:, i * (cols + gap):i * (cols + gap) + cols] for i in (2, 0, 3, 1))
    x.copy_(activations(rows, cols, "f32", 1))
    res.copy_(activations(rows, cols, "f32", 2))
    want_h, want_y = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    gca.rmsnorm(x.contiguous(), residual=res.contiguous(), h=want_h, y=want_y)
    gca.rmsnorm(x, residual=res, h=h, y=y)
    assert torch.equal(h, want_h) and torch.equal(y, want_y)
    assert bool((wide.view(rows, 4, -1)[:, :, cols:] == 7.0).all())
    with pytest.raises(gca.GCError):
        gca.rmsnorm(x, residual=res, y=wide[:, 1:1 + cols])


def test_norm_of_rows_without_a_norm():
    # zeros, huge, tiny, Inf and NaN rows next to an ordinary one
    x = torch.randn(8, 100, generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] *= 1e37
    x[2] *= 1e-37
    x[3, 7] = float("inf")
    x[4, 99] = float("nan")
    x[5] = 1e-30
    x[6, 1:] = 0.0
    x = x.cuda()
    for eps in (1e-5, 0.0):
        y = torch.empty_like(x)
        check_norm(x, None, None, eps, "f32", y=y, label=f"eps {eps}")
        bad = torch.isnan(y).any(1).cpu().tolist()
        assert bad == [eps == 0.0, False, False, True, True, False, False, False]


# ---------------------------------------------------------------- its backward pass
def check_backward(rows, cols, dtype, seed, residual=True, weight="f32", accumulate=False,
                   pad=None, alias=None):
    codes, exps, z = kept(rows, cols, seed)
    rng = np.random.default_rng(seed + 1)
    t = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda()  # noqa: E731
    rstd = torch.rand(rows, device="cuda") + 0.5
    dy = (t(rows, cols) * 1e-2).to(TYPES[dtype])
    dres = (t(rows, cols) * 1e-2).to(TYPES[dtype]) if residual else None
    w = None if weight is None else (t(cols) * 0.2 + 1.0).to(TYPES[weight])
    start = t(cols)
    flat = torch.cat((torch.full((3,), 7.0, device="cuda"), start,
                      torch.full((3,), 7.0, device="cuda")))
    dw = flat[3:3 + cols]                        # 4-byte aligned only, as a segment may be
    dx, buf = torch.empty_like(dy), None
    h_dy, h_dres = f64(dy), 0.0 if dres is None else f64(dres)
    if pad is not None:
        dy, _ = strided(dy, pad, 1)
        dx, buf = strided(dx, pad + 1)
        dres = dres if dres is None else strided(dres, pad + 2)[0]
    if alias == "dy":
        dx = dy
    if alias == "dres":
        dx = dres
    gca.rmsnorm_backward(dy, codes, exps, rstd, dx, weight=w, dres=dres, dweight=dw,
                         accumulate=accumulate)
    torch.cuda.synchronize()
    hw = np.ones(cols) if w is None else f64(w)
    r = f64(rstd)[:, None]
    tt = h_dy * hw
    c = (tt * z).mean(1, keepdims=True)
    want = r * (tt - z * c) + h_dres
    # t one rounding, c at most 64 sums deep (32 a lane, 6 in the wave, 16 waves) and its terms and
    # quotient, the difference, the product and the sum one each: every term's share of u
    c_err = 70 * U * np.abs(tt * z).mean(1, keepdims=True)
    tol = (r * (4 * U * (np.abs(tt) + np.abs(z * c)) + np.abs(z) * c_err)
           + 2 * U * np.abs(want) + U * np.abs(h_dres) + HALF[dtype] * np.abs(want) * 1.01
           + SMALLEST[dtype] / 2)
    off = np.abs(f64(dx) - want)
    assert (off <= tol).all(), f"dx off by {np.max(off / tol)} of its tolerance"
    if buf is not None and alias is None:
        assert untouched(buf, dx)
    want_w = (h_dy * z).sum(0) + (f64(start) if accumulate else 0.0)
    # a worker's rows, the workers of a slice, 32 slices, and the last addition
    deep = rows / max(1, min(rows, 1024)) + rows / 32 + 34
    tol_w = (min(deep, rows + 34) * U * (np.abs(h_dy * z).sum(0) + np.abs(f64(start)) * accumulate)
             + U * np.abs(want_w) + 1e-30)
    off = np.abs(f64(dw) - want_w)
    assert (off <= tol_w).all(), f"dw off by {np.max(off / tol_w)} of its tolerance"
    assert bool((flat[:3] == 7.0).all()) and bool((flat[3 + cols:] == 7.0).all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_norm_backward_matches_the_formula(dtype):
    for n, (rows, cols) in enumerate(NORM_SHAPES + [(2500, 96), (1100, 1030)]):
        log(f"[norm grad] {dtype} {rows}x{cols}")
        check_backward(rows, cols, dtype, n, residual=n % 3 != 0,
                       weight=(None, "f32", dtype)[n % 3], accumulate=n % 2 == 0)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_norm_backward_strided_and_in_place(dtype):
    for rows, cols in ((40, 100), (5, 4096), (1030, 2056)):
        check_backward(rows, cols, dtype, 7, pad=3)
        check_backward(rows, cols, dtype, 8, pad=8)
        check_backward(rows, cols, dtype, 9, alias="dy")
        check_backward(rows, cols, dtype, 10, alias="dres")


def test_norm_backward_without_rows_or_weight_gradient():
    dw = torch.full((50,), 5.0, device="cuda")
    codes, exps, _ = kept(3, 50, 0)
    none = torch.empty(0, 50, device="cuda")
    gca.rmsnorm_backward(none, codes[:0], exps[:0], dw[:0], none, dweight=dw, accumulate=True)
    assert bool((dw == 5.0).all())
    gca.rmsnorm_backward(none, codes[:0], exps[:0], dw[:0], none, dweight=dw)
    assert bool((dw == 0.0).all())
    dy = torch.randn(3, 50, device="cuda")
    rstd = torch.ones(3, device="cuda")
    a, b = torch.empty_like(dy), torch.empty_like(dy)
    gca.rmsnorm_backward(dy, codes, exps, rstd, a)
    gca.rmsnorm_backward(dy, codes, exps, rstd, b, dweight=dw)
    assert torch.equal(a, b)


def test_norm_backward_of_bad_groups():
    codes, exps, _ = kept(4, 70, 3)
    exps[1, 2] = 255                       # the short last group of row 1
    codes[1, 64:] = 0
    dy, rstd = torch.randn(4, 70, device="cuda"), torch.ones(4, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(70, device="cuda")
    gca.rmsnorm_backward(dy, codes, exps, rstd, dx, dweight=dw)
    assert torch.isnan(dx).all(1).tolist() == [False, True, False, False]
    assert not torch.isnan(dx[[0, 2, 3]]).any()
    assert torch.isnan(dw).tolist() == [False] * 64 + [True] * 6


# ---------------------------------------------------------------- the weight gradient
WGRAD_SHAPES = [(1, 1, 1), (1, 64, 64), (5, 3, 33), (31, 130, 200), (32, 128, 128), (33, 129, 127),
                (64, 257, 96), (100, 64, 1000), (257, 300, 320), (700, 96, 640), (1000, 512, 257),
                (4100, 40, 70), (2049, 384, 512), (65, 1000, 31), (513, 768, 1280)]


def exact_case(rows, n_out, cols, dtype, seed):
    """Integer gradients and codes of scale 1: every partial sum is below 2^24, so any order of the
    sums gives the same bits."""
    rng = np.random.default_rng(seed)
    most = min(2047 if dtype == "f16" else 255 if dtype == "bf16" else 1 << 20,
               max(1, (1 << 24) // (127 * rows)))
    dy = rng.integers(-most, most + 1, (rows, n_out))
    pitch, groups = gca.act_layout(cols)
    codes = rng.integers(-127, 128, (rows, pitch)).astype(np.int8)
    codes[:, cols:] = 0
    if (most == 1) and rows * 127 > 1 << 24:
        raise ValueError("too many rows for exact sums")
    want = dy.T.astype(np.float64) @ codes[:, :cols].astype(np.float64)
    exps = np.full((rows, groups), 127, np.uint8)
    return (torch.from_numpy(dy.astype(np.float32)).cuda().to(TYPES[dtype]),
            torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda(), want)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_weight_grad_of_integers_is_exact(dtype):
    for n, (rows, n_out, cols) in enumerate(WGRAD_SHAPES):
        log(f"[wgrad] {dtype} {rows} {n_out}x{cols}")
        dy, codes, exps, want = exact_case(rows, n_out, cols, dtype, n)
        flat = torch.full((n_out * cols + 2,), 7.0, device="cuda")
        dw = flat[1:-1].view(n_out, cols)
        gca.act_weight_grad(dy, codes, exps, dw)
        torch.cuda.synchronize()
        assert np.array_equal(f64(dw), want), f"{rows} {n_out}x{cols}"
        gca.act_weight_grad(dy, codes, exps, dw, accumulate=True)
        assert np.array_equal(f64(dw), 2 * want)
        assert flat[0] == 7.0 and flat[-1] == 7.0


def check_wgrad(rows, n_out, cols, dtype, seed, scale=None, pad=None, accumulate=False):
    codes, exps, z = kept(rows, cols, seed)
    rng = np.random.default_rng(seed + 5)
    t = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda()  # noqa: E731
    dy = (t(rows, n_out) * np.float32(1e-2)).to(TYPES[dtype])
    sc = None if scale is None else (t(cols) * 0.2 + 1.0).to(TYPES[scale])
    start = t(n_out, cols)
    dw = start.clone()
    h = f64(dy)
    if pad is not None:
        dy, _ = strided(dy, *pad)
    gca.act_weight_grad(dy, codes, exps, dw, col_scale=sc, accumulate=accumulate)
    torch.cuda.synchronize()
    s = np.ones(cols) if sc is None else f64(sc)
    want = (h.T @ z) * s + (f64(start) if accumulate else 0.0)
    # at most three exact parts a row, added one after the other in fp32: u for each addition,
    # twice that where the matrix core cuts off instead of rounding; two more for the scale and the sum
    n = {"bf16": 1, "f16": 2, "f32": 3}[dtype] * rows
    tol = 2 * (n + 20) * U * (np.abs(h).T @ np.abs(z)) * np.abs(s) + 2 * U * np.abs(want) + 1e-30
    got = f64(dw)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {np.max(off / tol)} of the tolerance"
    # the same roundings, as errors of either sign: far below that worst case
    assert np.linalg.norm(got - want) <= 4e-7 * np.sqrt(n + 20) * (
        np.linalg.norm(want) + np.linalg.norm(np.sqrt((h ** 2).T @ (z ** 2)) * np.abs(s))) + 1e-30


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_weight_grad_matches_the_formula(dtype):
    for n, (rows, n_out, cols) in enumerate(WGRAD_SHAPES):
        log(f"[wgrad] {dtype} {rows} {n_out}x{cols}")
        check_wgrad(rows, n_out, cols, dtype, n, scale=(None, "f32", dtype)[n % 3],
                    accumulate=n % 2 == 0)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_weight_grad_of_many_tiles(dtype):
    """Matrices that fill the GPU with the largest tiles, whole and ragged ones, sums of no, one, two
    and several steps."""
    for n, (rows, n_out, cols) in enumerate([(1, 3600, 3400), (70, 3585, 3600), (129, 3840, 3328),
                                             (200, 8200, 1800), (64, 300, 30000), (4000, 600, 520),
                                             (3000, 1030, 1500)]):
        log(f"[wgrad] {dtype} {rows} {n_out}x{cols}")
        dy, codes, exps, want = exact_case(rows, n_out, cols, dtype, n)
        dw = torch.ones(n_out, cols, device="cuda")
        if n % 2:
            dy, _ = strided(dy, 5, 3)
        gca.act_weight_grad(dy, codes, exps, dw, accumulate=True)
        torch.cuda.synchronize()
        assert np.array_equal(f64(dw), want + 1.0), f"{rows} {n_out}x{cols}"


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_weight_grad_of_strided_and_unaligned_rows(dtype):
    for pad in ((3, 0), (8, 0), (0, 1), (8, 8), (40, 5)):
        check_wgrad(150, 200, 100, dtype, 3, pad=pad)
        check_wgrad(40, 136, 264, dtype, 4, pad=pad)


def test_weight_grad_parts_of_full_precision():
    # one row: the product of a 24-bit gradient and a code, at most three roundings of fp32
    codes, exps, z = kept(1, 64, 2)
    dy = torch.randn(1, 300, device="cuda") * torch.exp(4 * torch.randn(1, 300, device="cuda"))
    for t in (torch.float32, torch.float16):
        d = dy.to(t)
        dw = torch.empty(300, 64, device="cuda")
        gca.act_weight_grad(d, codes, exps, dw)
        with np.errstate(invalid="ignore"):
            want = f64(d).T @ z              # a gradient past fp16's range is Inf, Inf * 0 is NaN
        got, fine = f64(dw), np.isfinite(want)
        assert (np.abs(got[fine] - want[fine]) <= 6 * U * np.abs(want[fine])).all()
        assert np.array_equal(got[~fine], want[~fine], equal_nan=True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_weight_grad_of_inf_nan_and_range(dtype):
    codes, exps, z = kept(40, 96, 6)
    codes[:, 5] = 3                       # no zero times Inf in this column
    codes[7, 32:64], exps[7, 1] = 0, 255  # NaN in columns 32..63
    dy = torch.randn(40, 70, device="cuda").to(TYPES[dtype])
    dy[3, 10], dy[5, 20] = float("inf"), float("nan")
    dw = torch.empty(70, 96, device="cuda")
    gca.act_weight_grad(dy, codes, exps, dw)
    got = dw.cpu()
    assert torch.isnan(got[:, 32:64]).all() and torch.isnan(got[20]).all()
    assert got[10, 5] == float("inf")
    assert not torch.isfinite(got[10]).any()
    rest = torch.ones(70, dtype=torch.bool)
    rest[[10, 20]] = False
    assert torch.isfinite(got[rest][:, :32]).all() and torch.isfinite(got[rest][:, 64:]).all()
    # a NaN whose payload sits in the low bits only, and values at the type's ends
    if dtype == "f32":
        d = torch.zeros(1, 4, device="cuda")
        d.view(torch.int32)[0, 0] = 0x7F800001
        d[0, 1], d[0, 2] = 3.4e38, -3.4028234e38
        c, e = torch.ones(1, 32, dtype=torch.int8, device="cuda"), torch.full((1, 1), 127, dtype=torch.uint8, device="cuda")
        w = torch.empty(4, 32, device="cuda")
        gca.act_weight_grad(d, c, e, w)
        assert torch.isnan(w[0]).all() and bool((w[1] == 3.4e38).all())
        assert bool((w[2] == -3.4028234e38).all()) and bool((w[3] == 0).all())


def test_weight_grad_without_rows():
    dw = torch.full((4, 40), 5.0, device="cuda")
    codes, exps, _ = kept(1, 40, 0)
    dy = torch.empty(0, 4, device="cuda")
    gca.act_weight_grad(dy, codes[:0], exps[:0], dw, accumulate=True)
    assert bool((dw == 5.0).all())
    gca.act_weight_grad(dy, codes[:0], exps[:0], dw)
    assert bool((dw == 0.0).all())


def test_weight_grad_with_the_callers_workspace():
    rows, n_out, cols = 4100, 100, 70
    need = gca.act_weight_grad_workspace(rows, n_out, cols, torch.bfloat16)
    dy, codes, exps, want = exact_case(rows, n_out, cols, "bf16", 1)
    buf = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
    dw = torch.empty(n_out, cols, device="cuda")
    gca.act_weight_grad(dy, codes, exps, dw, workspace=buf[:need])
    assert np.array_equal(f64(dw), want) and bool((buf[need:] == 77).all())
    with pytest.raises(gca.GCError):
        gca.act_weight_grad(dy, codes, exps, dw, workspace=buf[:need - 4])
    with pytest.raises(gca.GCError):
        gca.act_weight_grad(dy, codes, exps, dw, workspace=buf[4:])


# ---------------------------------------------------------------- streams and graphs
def test_two_streams_at_once_and_repeats_give_the_same_bits():
    dy = activations(2000, 300, "bf16", 1)
    codes, exps, _ = kept(2000, 260, 2)
    first = torch.empty(300, 260, device="cuda")
    gca.act_weight_grad(dy, codes, exps, first)
    d = activations(2000, 260, "bf16", 3)
    rstd = torch.rand(2000, device="cuda")
    dx, dw = torch.empty_like(d), torch.empty(260, device="cuda")
    gca.rmsnorm_backward(d, codes, exps, rstd, dx, dweight=dw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for r in range(6):
        s = streams[r % 2]
        a, b, c = torch.empty_like(first), torch.empty_like(dx), torch.empty_like(dw)
        s.wait_stream(torch.cuda.current_stream())
        if r < 3:
            with torch.cuda.stream(s):
                gca.act_weight_grad(dy, codes, exps, a)
                gca.rmsnorm_backward(d, codes, exps, rstd, b, dweight=c)
        else:
            gca.act_weight_grad(dy, codes, exps, a, stream=s)
            gca.rmsnorm_backward(d, codes, exps, rstd, b, dweight=c, stream=s)
        outs.append((a, b, c))
    torch.cuda.synchronize()
    for a, b, c in outs:
        assert torch.equal(a, first) and torch.equal(b, dx) and torch.equal(c, dw)


def test_graph_replays_match_eager_calls():
    rows, cols, n_out = 700, 320, 200
    x, res = activations(rows, cols, "bf16", 1), activations(rows, cols, "bf16", 2)
    dy_out = activations(rows, n_out, "bf16", 3)
    w = torch.rand(cols, device="cuda") + 0.5
    pitch, groups = gca.act_layout(cols)

    def buffers():
        return dict(h=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(rows, device="cuda"),
                    codes=torch.empty(rows, pitch, dtype=torch.int8, device="cuda"),
                    exps=torch.empty(rows, groups, dtype=torch.uint8, device="cuda"),
                    dx=torch.empty_like(x), dw=torch.zeros(cols, device="cuda"),
                    dl=torch.zeros(n_out, cols, device="cuda"), z=torch.empty_like(x))

    def step(b):
        gca.rmsnorm(x, weight=w, residual=res, h=b["h"], y=b["y"], rstd=b["rstd"],
                    codes=b["codes"], exps=b["exps"], stochastic=True, seed=3, step=4)
        gca.act_restore(b["codes"], b["exps"], b["z"])
        gca.act_weight_grad(dy_out, b["codes"], b["exps"], b["dl"], col_scale=w, accumulate=True)
        gca.rmsnorm_backward(b["y"], b["codes"], b["exps"], b["rstd"], b["dx"], weight=w,
                             dres=b["h"], dweight=b["dw"], accumulate=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buffers())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    captured, eager = buffers(), buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    scratch = torch.zeros(1 << 20, device="cuda")
    for t in range(4):
        x.copy_(activations(rows, cols, "bf16", 10 + t))
        dy_out.copy_(activations(rows, n_out, "bf16", 20 + t))
        scratch.add_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        log(f"[act graph] replay {t}")
        for name in captured:
            assert torch.equal(captured[name], eager[name]), f"replay {t} {name}"
    del graph
