"""Tables of rotary frequencies for fp8_rope: radians a position for each pair of a head,
as they were trained or scaled for contexts longer than those.  Computed once, on the host, in
64 bits; the table is FP32."""

import math

SCALINGS = (None, "linear", "base", "parts")


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, trained=None, fast=32.0, slow=1.0, device="cuda"):
    """(freq f32 [rot / 2], amplitude) of pairs i = 0 .. rot / 2 - 1, unscaled base ** (-2 i / rot).

    scaling="linear"  every frequency divided by `factor` (positions interpolated)
    scaling="base"    the base times factor ** (rot / (rot - 2)): the fastest pair stays, the
                      slowest is divided by `factor`
    scaling="parts"   by how often a pair turns in the `trained` positions: at least `fast` times
                      stays, at most `slow` times is divided by `factor`, linear in
                      between; the amplitude is 0.1 ln(factor) + 1, so that its square scales the scores
                      (Peng et al., "YaRN: Efficient Context Window Extension of Large Language
                      Models", 2023, section 3)
    """
    import torch
    if rot <= 0 or rot % 2 != 0:
        raise ValueError(f"rot must be a positive even number, got {rot}")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}, got {scaling!r}")
    if not base > 0 or not factor >= 1:
        raise ValueError(f"base {base} must be positive and factor {factor} at least 1")
    if scaling == "base":
        if rot == 2:
            raise ValueError("scaling='base' needs two pairs or more")
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    amplitude = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        if trained is None or not fast > slow:
            raise ValueError("scaling='parts' needs the trained length and fast > slow")
        keep = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        amplitude = 0.1 * math.log(factor) + 1
    return torch.tensor(f, dtype=torch.float64).to(torch.float32).to(device), amplitude
