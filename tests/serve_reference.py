"""Plain 64-bit definitions of the serving-step calls, and the error each call
may make, both written from the formulas (torch on the CPU, test plumbing)."""
from __future__ import annotations

import math

import torch

from oracle import rope as orope

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}           # half a step: finfo.eps / 2
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.uint8}


def stored_values(cache_dtype: str, x):
    """fp64 values of stored cache elements (unscaled)."""
    if cache_dtype == "e4m3":
        return x.view(torch.float8_e4m3fn).to(torch.float64)
    return x.to(torch.float64)


def extend(seq, new, free, head, table, bs, num_blocks, max_tokens):
    """Python integers; valid requests only."""
    table = [list(r) for r in table]
    slots, pos, start, out = [], [], [0], []
    for r, (n, m) in enumerate(zip(seq, new)):
        for j in range(-(-n // bs), -(-(n + m) // bs)):
            table[r][j] = free[head]
            head += 1
        for p in range(n, n + m):
            b = table[r][p // bs]
            slots.append(b * bs + p % bs if 0 <= b < num_blocks else -1)
            pos.append(p)
        start.append(start[-1] + m)
        out.append(n + m)
    return table, slots + [-1] * (max_tokens - len(slots)), pos, start, out, head


def axis_of_pair(half: int, sections, interleaved: bool):
    if sections is None or len(sections) == 1:
        return [0] * half
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    owner = [0] * half
    for a in range(1, len(sections)):
        for j in range(sections[a]):
            owner[a + j * len(sections)] = a
    return owner


def rotate(x, positions, spec, sections=None, interleaved=False):
    """x [T][heads][D] in fp64, positions [axes][T]; spec: dict of oracle.rope.inv_freq
    arguments plus style.  Returns the rotated rows and, per element, |a| + |b| of its pair."""
    D = x.shape[-1]
    w = torch.tensor(orope.inv_freq(D, spec["theta"], *spec.get("scaling", ())))
    p = positions.to(torch.float64)
    ang = torch.stack([p[a] * w[i] for i, a in enumerate(axis_of_pair(D // 2, sections, interleaved))], -1)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if spec["style"] == 0:
        a, b = x[..., : D // 2], x[..., D // 2:]
        mag = (a.abs() + b.abs()).repeat(1, 1, 2)
        return torch.cat([a * c - b * s, b * c + a * s], -1), mag
    a, b = x[..., 0::2], x[..., 1::2]
    mag = (a.abs() + b.abs()).repeat_interleave(2, -1)
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), mag


# The turns of an angle are reduced in fp32: at most 2^-24.5 of a turn off
# (the sum's rounding at 1/2 is 2^-26, the low part's product 2^-27, its own
# rounding 2^-27, the fp32 difference's 2^-26), so 2 pi 2^-24.5 < 2^-21.8 in the
# angle; sin and cos are then within 2 units of 2^-24 and two fp32 roundings
# follow: together below 2^-20.5 of |a| + |b|.
ROTATE = 2.0 ** -20


def rotated_tolerance(y, mag, dtype: str):
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0                       # half the smallest f16 step
    return U[dtype] * y.abs() * (1 + 2.0 ** -10) + tiny + ROTATE * mag


def e4m3_tolerance(y, err):
    """y: the scaled fp64 value before rounding, err: its fp32 error.  Half a step: 2^-4
    relative, 2^-10 among the subnormals; values past 448 saturate."""
    return 2.0 ** -4 * y.abs().clamp(max=448) + 2.0 ** -10 + (1 + 2.0 ** -4) * (err + 2.0 ** -22 * y.abs())


def attend(q, seq, k, v, named, scale, window):
    """One request: q [n][Hq][D] fp64; k, v [S][H][D] fp64 of positions 0..S-1; named [S] bool
    (the table names the position).  Returns out, lse, sum_j p_j |v_j|, and the largest
    sum_d |q_d k_d| * scale and number of keys seen per (row, head)."""
    n, Hq, D = q.shape
    S, H = k.shape[0], k.shape[1]
    G = Hq // H
    p = torch.arange(seq - n, seq)[:, None]
    j = torch.arange(S)[None]
    see = (j <= p) & named[None]
    if window:
        see &= j > p - window
    seen = see.sum(1).to(torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    out, spread = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    heft = torch.zeros(n, Hq, dtype=torch.float64)
    if S == 0:
        return out, lse, spread, heft, seen
    some = seen > 0
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kk.T * scale).masked_fill(~see, -math.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        w = torch.where(some[:, None], torch.exp(s - lse[:, h, None]), torch.zeros(()).double())
        out[:, h], spread[:, h] = w @ vv, w @ vv.abs()
        heft[:, h] = (q[:, h].abs() @ kk.abs().T).masked_fill(~see, 0.0).amax(1) * abs(scale)
    return out, lse, spread, heft, seen


def attend_tolerance(dtype, cache_dtype, D, out, lse, spread, heft, seen, vmax):
    """A weight is off by the fp32 sum of its logit (D products; heft is the sum of their
    magnitudes; 8 more roundings scale it and take the maximum off), the hardware exp2
    (2^-21 covers it), and, for 16-bit queries, its rounding to 16 bits (U; in fp16, also half
    of the smallest step, 2^-25, against a largest weight of at least 1).  A wrong weight
    counts once in the numerator and once in the sum.  The fp32 sums over the keys add one
    rounding a key; the output is rounded once."""
    delta = (D + 8) * 2.0 ** -24 * heft + 2.0 ** -21
    acc = (seen[:, None] + 16) * 2.0 ** -24
    math16 = None if dtype == "f32" else ("f16" if cache_dtype == "e4m3" else dtype)
    w = 0.0 if math16 is None else U[math16]
    tol = (w + 2 * delta + 2 * acc)[..., None] * spread * 1.01 + U[dtype] * 1.01 * out.abs()
    if math16 == "f16":
        tol = tol + (seen * 2.0 ** -25)[:, None, None] * vmax
    if dtype == "f16":
        tol = tol + 2.0 ** -25
    lse_tol = delta + acc + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0) + 2.0 ** -22
    return tol, lse_tol
