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
