"""Refused calls of the operators over many tensors and of the gated block leave everything as it was."""
from types import SimpleNamespace

import pytest
import torch

import gradient_compression_amd as gca

pytestmark = pytest.mark.gpu


class Call:
    """Arguments of a clip_grad_norm call, all outputs at 7."""

    def __init__(self):
        gen = torch.Generator("cuda").manual_seed(1)
        self.ts = [torch.randn(n, generator=gen, device="cuda").to(t) for n, t in (
            (1000, torch.float32), (77, torch.bfloat16), (5000, torch.float16))]
        self.norm, self.norms, self.factors, self.flat = (
            torch.full((n,), 7.0, device="cuda") for n in (1, 3, 2, 6077))

    def tensors(self):
        return [*self.ts, self.norm, self.norms, self.factors, self.flat]


@pytest.mark.parametrize("what", ["negative", "nan", "text", "none", "short", "type", "kind", "count",
                                  "sizes", "over_input", "over_norm", "factors_type", "factors_kind",
                                  "factors_over_norm", "factors_over_tensor", "in_place_twice"])
def test_a_refused_clip_grad_norm_writes_nothing(what):
    """Its norm is not written before the scaling's arguments are looked at."""
    c = Call()
    limit, ts, more = 1.0, c.ts, dict(norms=c.norms, out=c.flat, factors=c.factors)
    if what in ("negative", "nan", "text", "none"):
        limit = {"negative": -1.0, "nan": float("nan"), "text": "one", "none": None}[what]
    elif what == "short":
        more["out"] = c.flat[1:]
    elif what == "type":
        more["out"] = c.flat.double()
    elif what == "kind":
        more["out"] = 3
    elif what == "count":
        more["out"] = [c.flat]
    elif what == "sizes":
        more["out"] = list(c.flat.split([1000, 78, 4999]))
    elif what == "over_input":
        ts = [*c.ts[:2], c.flat[10:5010]]
    elif what == "over_norm":
        more["out"] = torch.cat((c.flat, c.norm))[:-1]
        c.norm = more["out"][5:6].fill_(7.0)
    elif what == "factors_type":
        more["factors"] = c.factors.half()
    elif what == "factors_kind":
        more["factors"] = [1.0]
    elif what == "factors_over_norm":
        more["factors"] = c.norm
    elif what == "factors_over_tensor":
        more["factors"] = c.ts[0][:2]
    elif what == "in_place_twice":
        ts, more["out"] = [c.ts[0], c.ts[1], c.ts[0]], None
    before = [t.clone() for t in c.tensors()]
    versions = [t._version for t in c.tensors()]
    with pytest.raises((ValueError, TypeError, gca.GCError)):
        gca.clip_grad_norm(ts, limit, c.norm, **more)
    torch.cuda.synchronize()
    for t, b, v in zip(c.tensors(), before, versions):
        assert torch.equal(t, b) and t._version == v


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """The workspace would be allocated there, and the kernels would run there."""
    c = Call()
    x, w = torch.full((300, 64), 0.5, device="cuda"), torch.full((520, 64), 0.5, device="cuda")
    h, g, u = (torch.full((300, 520), 7.0, device="cuda") for _ in range(3))
    other = SimpleNamespace(device_index=torch.cuda.current_device() + 1, cuda_stream=0)
    everything = [*c.tensors(), x, w, h, g, u]
    before = [t.clone() for t in everything]
    allocated = []
    monkeypatch.setattr(gca, "_workspace", lambda *a: allocated.append(a) or (None, 0, None))
    for call in (lambda: gca.grad_norm(c.ts, c.norm, norms=c.norms, stream=other),
                 lambda: gca.grad_clip(c.ts, 1.0, c.norm, factors=c.factors, stream=other),
                 lambda: gca.clip_grad_norm(c.ts, 1.0, c.norm, out=c.flat, stream=other),
                 lambda: gca.gated_linear(x, w, w, h, stream=other),
                 lambda: gca.gated_linear_backward(h, g, u, g, u, w_gate=w, w_up=w, dx=x,
                                                   stream=other)):
        with pytest.raises(ValueError, match="stream is on"):
            call()
    torch.cuda.synchronize()
    assert not allocated
    assert all(torch.equal(t, b) for t, b in zip(everything, before))


def test_inputs_among_the_outputs_in_any_order():
    """Tensors and results that lie between each other in one buffer, and share no element, are taken."""
    buf = torch.arange(1.0, 601.0, device="cuda")
    parts = list(buf.split(50))
    for order in ((0, 1, 2, 3, 4, 5), (3, 0, 5, 1, 4, 2)):
        ts, outs = [parts[2 * i] for i in order], [parts[2 * i + 1] for i in order]
        norm = torch.empty(1, device="cuda")
        want = [t.clone() for t in ts]
        gca.clip_grad_norm(ts, 10.0, norm, out=outs)
        f = torch.tensor(10.0, device="cuda") / norm
        assert all(torch.equal(o, w * f) and torch.equal(t, w) for o, t, w in zip(outs, ts, want))
        with pytest.raises(gca.GCError):
            gca.clip_grad_norm(ts, 10.0, norm, out=[*outs[:-1], buf[50 * 2 * order[-1] + 1:][:50]])
