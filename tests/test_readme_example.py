"""The readme's example, run on the CPU with the oracle in place of the kernels: what its delta-rule layer makes of
queries and keys is what the rule is meant for.
"""
from __future__ import annotations

import builtins
import os
import re
import sys
from unittest.mock import MagicMock

import torch

from oracle import delta_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G, K, H, V, L = 16, 128, 32, 64, 5


class _Names(dict):
    """What the example takes from the program around it."""

    def __missing__(self, name):
        if name.startswith("__") or name == "torch" or hasattr(builtins, name):
            raise KeyError(name)
        self[name] = MagicMock(name=name)
        return self[name]


def _norm(x, weight=None, bias=None, *, groups=1, gate=None, eps=1e-5):
    f = lambda t: None if t is None else t.flatten(0, -2)
    return orc.group_norm(f(x), weight, bias, f(gate), groups, "plain" if gate is None else "gated", False, eps).reshape(x.shape)


def test_queries_and_keys_have_length_one(monkeypatch):
    with open(os.path.join(ROOT, "README.md")) as fh:
        code = re.search(r"```python\n(.*?)```", fh.read(), re.S).group(1)
    seen = []

    def rule(q, k, v, g, beta, **kw):
        seen.append((q, k))
        return torch.zeros(1, L, H, V), MagicMock()

    m2 = MagicMock(name="m2")
    m2.conv_fwd.return_value = m2.ssm_fwd.return_value = (MagicMock(), MagicMock())
    m2.group_norm_fwd.side_effect = _norm
    m2.delta_fwd.side_effect = rule
    monkeypatch.setitem(sys.modules, "bwd_mamba2_scan_amd", m2)
    gen = torch.Generator().manual_seed(0)
    size = torch.tensor([0.03, 0.3, 1.0, 30.0, 0.0]).reshape(1, L, 1)  # of a convolution's output: small, large, none
    draw = lambda n: torch.randn(1, L, n, generator=gen) * size
    names = _Names(u_q=draw(G * K), u_k=draw(G * K), norm_weight=torch.ones(V), z=torch.zeros(1, L, H * V), device="cpu")
    exec(compile(code, "README.md", "exec"), {}, names)
    assert len(seen) == 1
    for t in seen[0]:
        assert t.shape == (1, L, G, K)
        length = t.norm(dim=-1)
        assert float((length[:, :4] - 1).abs().max()) < 1e-3 and float(length[:, 4].abs().max()) == 0
