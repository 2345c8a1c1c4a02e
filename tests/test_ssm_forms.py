"""The selective scan's launch forms and the GPU cases that reach them (CPU)."""
from __future__ import annotations

import itertools

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd.layer import Seqs, SsmDims
from tests.ssm_forms import HEADS, SEGMENTS, plan, sizes, workspaces


def test_rules_are_the_librarys():
    L = m2.lib()
    for length, batch, packed, (H, G), P, N in itertools.product(
            (0, 1, 64, 65, 256, 257, 384, 385, 640, 641, 1400, 5000, 100000), (1, 2, 3, 7, 40, 520), (False, True),
            ((1, 1), (3, 1), (12, 2), (32, 1), (24, 8)), (8, 32, 72, 128), (8, 64, 72, 128)):
        q, d = Seqs(batch, length, 0x1000 if packed else None), SsmDims(1, 1, H, P, G, N, 1)
        args = length, batch, packed, H, P, G, N
        assert (L.mamba2_ssm_fwd_workspace_bytes(q, d), L.mamba2_ssm_bwd_workspace_bytes(q, d)) == workspaces(*args), args


def test_cases_reach_every_form():
    heads = [(plan(*sizes(c)), c) for c in HEADS]
    assert all(p["run"] > 1 for p, _ in heads)
    for typ in ("f32", "bf16"):
        some = [(p, c[4]) for p, c in heads if c[5] == typ]
        assert any(p["splits"] == 1 for p, _ in some) and any(p["splits"] > 1 for p, _ in some)
        assert any(p["slices"] > 1 for p, _ in some) and any(p["ratio"] % p["run"] for p, _ in some)
        assert {1 if n <= 32 else 2 if n <= 64 else 4 for _, n in some} >= ({1, 4} if typ == "f32" else {1, 2, 4})
        assert any(p["run"] > 2 for p, _ in some)           # the ring of three decays comes round
    assert any(p["segments"] for p, _ in heads)
    reached = set()
    for c in SEGMENTS:
        p = plan(*sizes(c))
        assert p["segments"]
        reached.add((c[5], sizes(c)[2], p["fold"]))
    for typ, packed in itertools.product(("f32", "bf16"), (False, True)):
        assert {(typ, packed, False), (typ, packed, True)} <= reached, (typ, packed)
    # a sequence of more segments than the carry has in flight
    assert any(not plan(*sizes(c))["fold"] and sizes(c)[0] > 9 * plan(*sizes(c))["seg"] for c in SEGMENTS)
