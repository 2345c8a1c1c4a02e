"""Cases of the selective scan that reach its launch forms, and the library's rules for them.

The rules (segments, the pass that carries states across them, the heads of a
backward work-group) are host code inside the library; `plan` states them again
so that a CPU test can say which form a case reaches.  That the statement holds
is checked against the workspace sizes, which follow from it.
"""
from __future__ import annotations

CUS, STEP = 256, 64


def _ceil(a, b):
    return -(-a // b)


def _units_of(length, run):
    return max(1, _ceil(length, run))


def plan(length, batch, packed, H, P, G, N, bwd=True):
    """length: tokens of a sequence, or all rows of a packed call."""
    waves = 1 if P <= 16 else 2 if P <= 32 else 4
    slices = _ceil(P, 16 * waves)
    want = max(1, CUS * (2 if N > 64 else 3) // (H * slices * (1 if packed else batch)))
    few = STEP * (10 if bwd else min(6 * batch, 10) if packed else 6)
    seg = length if length <= few else _ceil(length, want)
    seg = max(2 * STEP, _ceil(seg, STEP) * STEP)
    units = lambda run: length // run + batch if packed else _units_of(length, run) * batch
    steps, ratio = units(STEP), H // G
    run = _ceil(ratio, min(ratio, _ceil(2 * CUS, steps * G)))
    return dict(waves=waves, slices=slices, seg=seg, units=units(seg), steps=steps, ratio=ratio, run=run,
                splits=_ceil(ratio, run), segments=length > seg,
                fold=_units_of(length, seg) <= (4 if N > 64 else 6) * (min(batch, 4) if packed else 1))


def workspaces(length, batch, packed, H, P, G, N):
    """Bytes of the forward's and the backward's workspace."""
    p, f = (plan(length, batch, packed, H, P, G, N, bwd) for bwd in (True, False))
    pad4 = lambda n: _ceil(n, 4) * 4
    states = p["units"] * H * N * P
    fwd = _ceil(f["units"] * H * (N * P + 1) * 4, 16) * 16 if f["segments"] else 0
    keep = p["steps"] * H * _ceil(P, 16) * _ceil(N, 16) * 256
    rows = length * (1 if packed else batch)
    part_bc = pad4(p["splits"] * rows * G * N) if p["splits"] > 1 else 0
    seg = pad4(states) + pad4(p["units"] * H) if p["segments"] else 0
    return fwd, 4 * (2 * (keep + seg + part_bc) + pad4(p["steps"] * H * 4))


def _every(n, step):
    return [i * step for i in range(n + 1)]


# Backward work-groups with several heads.  (offsets or (batch, L), H, P, G, N, type, dt type)
HEADS = [
    ((140, 70), 3, 24, 1, 40, "bf16", "bf16"),                  # runs of two heads and of one
    ((100, 130), 12, 16, 2, 24, "f32", "f32"),                  # one run of six per group
    (_every(300, 5), 8, 40, 2, 24, "bf16", "f32"),              # one run of four: d_B and d_C stored directly
    ((260, 3), 15, 32, 1, 72, "f32", "bf16"),                   # runs of eight and of seven heads
    ([0, 1, 1, 90] + [90 + i for i in range(1, 520)], 5, 64, 1, 128, "bf16", "bf16"),   # one run of five, an odd number
    ((130, 67), 3, 72, 1, 104, "bf16", "bf16"),                 # two slices of columns
    ((130, 66), 6, 128, 2, 128, "f32", "f32"),                  # two slices, the states in two parts
    (_every(530, 2), 3, 88, 1, 120, "f32", "f32"),              # the same in one run of three
    ((2, 2050), 16, 64, 1, 128, "bf16", "bf16"),                # runs of two behind segments
]

# Segments, with the carry pass and without.
SEGMENTS = [
    ((2, 1400), 2, 16, 1, 16, "f32", "f32"),                    # eleven segments: the carry's second round
    ((1, 2600), 3, 64, 1, 128, "bf16", "bf16"),
    ((3, 1290), 1, 72, 1, 24, "f32", "bf16"),
    ([0, 100, 2900, 2900, 3400], 2, 24, 2, 40, "f32", "f32"),   # packed, a carry over 22 segments
    ([5, 2905, 3300, 3301], 4, 64, 1, 72, "bf16", "bf16"),
    ([0, 1390], 2, 32, 1, 32, "bf16", "f32"),                   # one packed sequence
    ([0, 2990, 2990, 3000], 2, 40, 1, 24, "f32", "f32"),        # one long sequence among three
    ([0, 900, 1990], 3, 16, 3, 88, "bf16", "bf16"),
    # from here on the segments add up the states before them
    ([0, 2290, 2290, 2300], 2, 40, 1, 24, "f32", "f32"),        # 18 in one sequence
    ([9, 700, 1020], 3, 64, 1, 96, "bf16", "bf16"),
    ((2, 760), 4, 24, 2, 48, "bf16", "f32"),                    # six
    ((1, 700), 3, 72, 1, 16, "f32", "f32"),
]


def sizes(case):
    """Arguments of plan()."""
    lead, H, P, G, N = case[:5]
    if isinstance(lead, tuple):
        return lead[1], lead[0], False, H, P, G, N
    return lead[-1], len(lead) - 1, True, H, P, G, N
