"""Plain 64-bit definitions of the calls over a scaled cache, and the error each
may make, both written from the formulas (torch on the CPU, test plumbing)."""
from __future__ import annotations

import torch

from tests import serve_reference as ref

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.uint8}
SMALLEST, LARGEST = 2.0 ** -40, 2.0 ** 40


def numbers(cache: str, codes):
    """fp64 values of codes, in their block's scale."""
    return (codes.view(torch.float8_e4m3fn) if cache == "e4m3" else codes).to(torch.float64)


def encode(cache: str, x):
    """Codes of numbers in their block's scale: nearest even, saturated."""
    if cache == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8)


def quantised(cache: str, x, held=None):
    """A whole cache's codes and fp32 scales of x [2][NB][bs][H][D] (fp64); held: rows of each block that count."""
    size = x.abs()
    if held is not None:
        size = size * (torch.arange(x.shape[2])[None] < held[:, None])[None, :, :, None, None]
    scales = (size.amax((2, 4)) / QMAX[cache]).clamp(SMALLEST, LARGEST).to(torch.float32)
    return encode(cache, x / scales.double()[:, :, None, :, None]), scales


def code_tolerance(cache: str, y, err):
    """y: fp64 numbers in the scale's units before rounding, err: their fp32 error.  Half a step, and where the
    product with the reciprocal is rounded (two roundings of 2^-24) or err carries it over a border, that much more."""
    if cache == "e4m3":
        return ref.e4m3_tolerance(y, err)
    return 0.5 + err + 2.0 ** -22 * y.abs().clamp(max=256)


def groups(slots, bs: int, n_slots: int):
    """(block, tokens) of each run of adjacent tokens in one block."""
    found, last = [], -1
    for t, slot in enumerate(slots.tolist()):
        b = slot // bs if 0 <= slot < n_slots else -1
        if b >= 0 and b == last:
            found[-1][1].append(t)
        elif b >= 0:
            found.append((b, [t]))
        last = b
    return found


def check_write(cache, bs, slots, refused, rows, err, before, after):
    """rows, err [2][T][H][D]: keys and values in fp64 and their fp32 error; refused [T]: not written.  before, after:
    (codes, scales) of the cache.  Every code and scale of the cache is looked at."""
    (c0, s0), (c1, s1) = before, after
    NB = s0.shape[1]
    want_same = torch.ones(c0.shape[:3], dtype=torch.bool)
    same_scale = torch.ones(s0.shape[:2], dtype=torch.bool)
    n0, n1 = numbers(cache, c0), numbers(cache, c1)
    for b, tokens in groups(slots, bs, NB * bs):
        live = [t for t in tokens if not refused[t]]
        if not live:
            continue
        low = min(int(slots[t]) % bs for t in tokens)
        at = [int(slots[t]) % bs for t in live]
        want_same[:, b, at] = False
        same_scale[:, b] = False
        for kv in range(2):
            y, e = rows[kv, live], err[kv, live]
            e = torch.where(y.isfinite(), e, torch.zeros(()).double())   # the others have no error: they saturate, or are NaN
            finite = torch.where(y.isfinite(), y.abs(), torch.zeros(()).double())
            top = finite.amax((0, 2))                                # [H]
            new = (top / QMAX[cache]).clamp(SMALLEST, LARGEST)
            slack = e.amax((0, 2)) / QMAX[cache] + 2.0 ** -23 * new
            old = s0[kv, b].double()
            want = torch.maximum(old, new) if low else new
            got = s1[kv, b].double()
            assert bool(((got - want).abs() <= slack).all()), (kv, b, got, want)
            if low:
                assert bool((got >= old).all())
                kept = got == old
                held = slice(0, low)
                want_same[kv, b, held] = False
                assert torch.equal(c0[kv, b, held][:, kept], c1[kv, b, held][:, kept])
                was = n0[kv, b, held][:, ~kept] * (old / got)[~kept, None]
                tol = code_tolerance(cache, was, 2.0 ** -22 * was.abs())
                ok = ((n1[kv, b, held][:, ~kept] - was).abs() <= tol) | (was.isnan() & n1[kv, b, held][:, ~kept].isnan())
                assert bool(ok.all())
            x = y / got[:, None]
            tol = code_tolerance(cache, x, e / got[:, None])
            x = x.clamp(-QMAX[cache], QMAX[cache])                   # infinities and what the largest scale leaves out
            have = n1[kv, b, at]
            if cache == "int8":
                x = x.nan_to_num(nan=0.0)
                tol = tol.nan_to_num(nan=0.0, posinf=0.0)
            ok = ((have - x).abs() <= tol.nan_to_num(nan=0.0, posinf=1.0)) | (x.isnan() & have.isnan())
            assert bool(ok.all()), (kv, b, float((have - x).abs().nan_to_num(0).max()))
    assert torch.equal(c0[want_same], c1[want_same])
    assert torch.equal(s0.view(torch.int32)[same_scale], s1.view(torch.int32)[same_scale])


def attend_tolerance(dtype, D, out, lse, spread, heft, seen, scales, qmax):
    """As for a cache with one scale (codes are exact in fp16), and: a weight holds its key's V scale as a power of two,
    whose exponent log2 is rounded (one step of it) and added to the logit (half a step), and whose reciprocal is
    rounded, the sum taking it back.  fp16 steps of the faintest weights, 2^-25 beside a largest of at least 1, are
    relative to weight times V scale, so they are worth the largest V scale times the largest code each."""
    lv = float(torch.log2(scales.double()).abs().max())
    extra = 3 * 2.0 ** -24 * (lv + 2)
    tol, lse_tol = ref.attend_tolerance(dtype, "e4m3", D, out, lse, spread, heft, seen, qmax * float(scales.max()))
    return tol + 2 * extra * spread, lse_tol + 2 * extra
