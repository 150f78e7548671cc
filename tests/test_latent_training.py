"""A training step over latent rows that are key and value, as the README
writes it: norm and rotation, forward, backward, and back through both."""
import os
import re

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES, half_step, table
from parity_util import REL_TOL

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
EPS = 1e-6


def _step():
    """The README's block that trains on latent rows."""
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "norm_rope_grad(" in b)


def _inputs(tokens, heads, keys, dtype, device):
    g = torch.Generator().manual_seed(0)
    t = DTYPES[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t).to(device)  # noqa: E731
    n = (1, tokens)
    return dict(c=r(*n, 1, 512), kr0=r(*n, 1, 64), q0=r(*n, heads, 512), qr0=r(*n, heads, 64),
                w=(1 + 0.1 * r(512)).to(t), wq=(1 + 0.1 * r(512)).to(t), d_out=r(*n, heads, 512),
                positions=torch.arange(tokens, dtype=torch.int32, device=device)[None],
                cos_sin=table(tokens, device),
                indices=torch.stack([torch.randperm(tokens, generator=g)[:keys] for _ in range(tokens)]).int()
                .view(1, tokens, 1, keys).to(device), scale=576 ** -0.5)


def _loss(x, p):
    """sum(out * d_out) in 64 bits of the parameters p (c, kr0, q0, qr0, w, wq)."""
    def normed(v, w):
        return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    def turned(v):
        cs = x["cos_sin"].double()[x["positions"].long()][..., None, :]
        a, b, co, si = v[..., 0::2], v[..., 1::2], cs[..., :32], cs[..., 32:]
        return torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)

    k = normed(p["c"], p["w"])[0, :, 0]
    row = torch.cat((k, turned(p["kr0"])[0, :, 0]), -1)
    q = torch.cat((normed(p["q0"], p["wq"]), turned(p["qr0"])), -1)[0]
    at = x["indices"][0, :, 0].long()
    s = torch.einsum("thd,tkd->thk", q, row[at]) * x["scale"]
    out = torch.einsum("thk,tkd->thd", s.softmax(-1), k[at])
    return (out * x["d_out"][0].double()).sum()


NAMES = {"c": "dc", "kr0": "dkr0", "q0": "dq0", "qr0": "dqr0", "w": "dw", "wq": "dwq"}


def test_documented_step_names_every_gradient():
    step = _step()
    for name in NAMES.values():
        assert re.search(rf"\b{name}\b", step), name
    for call in ("sfa.norm_rope(", "sfa.fwd(", "sfa.grad("):
        assert call in step, call


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dtype", [(16, "bf16"), (128, "fp16")])
def test_training_step_on_latent_rows(heads, dtype):
    """Relative errors, by root mean squares; r = u / sqrt(3) for one rounding
    of half a step u.  The rows' rounding moves scores of size one by sqrt(2) r
    and so P, and dP and D by r each: dS 2 r in all, and with the queries' own
    rounding 3 r.  dk, dv, their sum and the gradient of the row are rounded
    once each, 4 r.  7 r is below 5 u; the backward itself may be off by its
    tolerance for given inputs."""
    x = _inputs(96, heads, 40, dtype, "cuda")
    got = dict(x, sfa=sfa)
    exec(_step(), got)
    p = {n: x[n].double().requires_grad_() for n in NAMES}
    loss = _loss(x, p)
    want = dict(zip(NAMES, torch.autograd.grad(loss, list(p.values()))))
    tol = REL_TOL[dtype] + 5 * half_step(DTYPES[dtype])
    for n, name in NAMES.items():
        d = got[name].double().view(want[n].shape)
        assert float((d - want[n]).norm() / want[n].norm()) <= tol, name
        # the loss's difference along the gradient is its length (h^2 of the
        # third derivative is below the tolerance by far)
        h = 1e-4
        step = d / d.norm()
        up, dn = ({m: v.detach() + (h * s * step if m == n else 0) for m, v in p.items()} for s in (1, -1))
        slope = float((_loss(x, up) - _loss(x, dn)) / (2 * h))
        assert abs(slope - float(d.norm())) <= 2 * tol * float(d.norm()), name
