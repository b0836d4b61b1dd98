"""The serving step over a scaled cache on the GPU: is_append_scaled,
is_move_scaled, is_read_scaled and is_attend_scaled against their plain 64-bit
definitions, at the sizes, masks and layouts where they can go wrong, and all of
them together behind an injection."""
import math

import numpy as np
import pytest
import torch

from kv_cache_injection_gb300 import _lib, api
from tests import gpu_helpers as gh
from tests import scaled_reference as sref
from tests import serve_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
PLAIN = dict(theta=1e4, style=0)
LLAMA = dict(theta=5e5, style=0, scaling=(1, 8.0, 1.0, 4.0, 8192))
CACHES = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def built():
    gh.ensure_built()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def rope_of(spec):
    return api.make_rope(spec["theta"], spec["style"], *spec.get("scaling", ()))


def packed_slots(reqs, bs, g, spare=3):
    """Slots and positions of the last m of each request's n tokens (n, m), blocks in random order; blocks, the rows
    each block holds before, and each request's table."""
    need = [-(-n // bs) for n, _ in reqs]
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=g).tolist()
    slots, pos, held, tables = [], [], torch.zeros(nb, dtype=torch.int64), []
    for (n, m), k in zip(reqs, need):
        table = [ids.pop() for _ in range(k)]
        tables.append(table)
        for p in range(n - m, n):
            slots.append(table[p // bs] * bs + p % bs)
            pos.append(p)
        for j, b in enumerate(table):
            held[b] = min(bs, max(0, n - m - j * bs))
    return torch.tensor(slots, dtype=torch.int64), torch.tensor(pos, dtype=torch.int32), nb, held, tables


def random_cache(cache, nb, bs, H, D, g, held=None, gain=1.0):
    """Codes and scales as if rows `held` of each block had been written (all: None); what lies behind is noise."""
    x = gain * torch.randn(2, nb, bs, H, D, generator=g).double() * 2.0 ** torch.randint(-3, 4, (2, 1, 1, H, 1), generator=g)
    codes, scales = sref.quantised(cache, x, held)
    if held is not None:
        scales[:, held == 0] = math.nan                  # a block that holds nothing: its scale means nothing
    return codes, scales


# ---------------------------------------------------------------- is_append_scaled

def append_case(reqs, Hq, H, D, dtype, cache, spec=PLAIN, sections=None, interleaved=False, bs=16, seed=0, gain=1.0, skip=(),
                shift=0, values=None, far=None, split=True):
    g = torch.Generator().manual_seed(seed)
    td = ref.TORCH[dtype]
    slots, pos, nb, held, _ = packed_slots(reqs, bs, g)
    T = len(slots)
    qkv = (gain * torch.randn(T, Hq + 2 * H, D, generator=g)).to(td)
    if values is not None:
        values(qkv, Hq, H)
    axes = 1 if sections is None else len(sections)
    pos = torch.stack([pos + shift + 3 * a * (pos % 5) for a in range(axes)]).to(torch.int32)
    if far is not None:
        pos[:, -1] = far
    for t in skip:
        slots[t] = -1
    c0, s0 = random_cache(cache, nb, bs, H, D, g, held)
    codes, scales = c0.to(DEV), s0.to(DEV)
    dev = qkv.to(DEV)
    q, k, v = dev[:, :Hq], dev[:, Hq: Hq + H], dev[:, Hq + H:]
    if not split:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = torch.full((T, Hq, D), math.nan, dtype=td, device=DEV)
    status = ints([0])
    ax = api.make_axes(sections, interleaved) if sections else None
    api.is_append_scaled(q if Hq else None, k, v, pos.to(DEV), slots.to(DEV), rope_of(spec), api.make_cache_desc(bs, nb, cache),
                         codes, scales, q_out if Hq else None, status, axes=ax)
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    x = qkv.double()
    y, mag = ref.rotate(x[:, Hq: Hq + H], pos, spec, sections, interleaved)
    rows = torch.stack([y, x[:, Hq + H:]])
    err = torch.stack([mag * ref.ROTATE, torch.zeros_like(mag)])
    refused = slots < 0
    sref.check_write(cache, bs, slots, refused, rows, err, (c0, s0), (codes.cpu(), scales.cpu()))
    if Hq:                                               # the queries are is_append's, bit for bit
        plain, same = torch.zeros(2, nb, bs, H, D, dtype=td, device=DEV), torch.full_like(q_out, math.nan)
        api.is_append(q, k, v, pos.to(DEV), slots.to(DEV), rope_of(spec), api.make_cache_desc(bs, nb, dtype), plain, same,
                      status, axes=ax)
        i = {2: torch.int16, 4: torch.int32}[q_out.element_size()]
        assert torch.equal(q_out.view(i), same.view(i))
    return codes, scales


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("reqs,Hq,H,D,style", [
    ([(1, 1)], 4, 2, 64, 0), ([(18, 1), (33, 1), (16, 1)], 28, 4, 128, 0), ([(40, 33)], 8, 8, 64, 1), ([(5, 3)], 1, 1, 16, 0),
    ([(3, 2), (50, 17)], 6, 2, 32, 1), ([(20, 4)], 5, 1, 256, 0), ([(23, 7)], 0, 3, 128, 0), ([(17, 2)], 2, 1, 128, 1),
    ([(160, 150), (70, 70)], 32, 8, 128, 0), ([(9, 5)], 3, 17, 64, 0)])
def test_append(reqs, Hq, H, D, style, dtype, cache):
    append_case(reqs, Hq, H, D, dtype, cache, dict(theta=1e4, style=style), seed=len(reqs))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("bs", [1, 5, 7, 24, 31, 32, 64, 130, 1000])
def test_append_block_sizes(bs, cache):
    """Groups shorter and longer than a warp's tile, than 31 tokens and than the block."""
    append_case([(7, 7), (2 * bs + 3, bs + 2), (bs, 1), (bs + 1, 1)], 4, 2, 64, "bf16", cache, bs=bs)
    append_case([(300, 280), (90, 1)], 2, 1, 256, "bf16", cache, bs=bs, seed=1)
    append_case([(200, 150)], 2, 1, 32, "f32", cache, bs=bs, seed=2)


def test_append_widest_head():
    append_case([(21, 9)], 2, 1, 512, "bf16", "int8")


@pytest.mark.parametrize("sections,interleaved,style", [
    ([16, 24, 24], False, 0), ([24, 20, 20], True, 0), ([40, 24], False, 1), ([0, 0, 64], False, 0)])
def test_append_axes(sections, interleaved, style):
    append_case([(40, 21)], 6, 2, 128, "bf16", "int8", dict(theta=1e6, style=style), sections, interleaved)


@pytest.mark.parametrize("spec", [PLAIN, LLAMA])
def test_append_far_positions(spec):
    append_case([(40, 40)], 4, 2, 128, "f32", "int8", spec, far=(1 << 24) - 1)
    append_case([(40, 40)], 4, 2, 128, "bf16", "e4m3", spec, [16, 24, 24], far=(1 << 24) - 1)


def test_append_padding_and_separate_tensors():
    append_case([(50, 30), (20, 5)], 8, 2, 64, "bf16", "int8", bs=7, skip=(33, 34), split=False)
    append_case([(9, 9)], 8, 2, 64, "f16", "e4m3", skip=tuple(range(9)))


@pytest.mark.parametrize("cache", CACHES)
def test_append_of_many_magnitudes(cache):
    """Zeros, elements around the smallest and largest scales, and rows far above and below what the block holds."""
    append_case([(20, 4)], 2, 2, 64, "f32", cache, gain=0.0)
    for gain in (1e-38, 1e-13, 1e-4, 3e3, 1e13, 1e20):
        append_case([(20, 4), (33, 1), (5, 5)], 2, 2, 64, "f32", cache, gain=gain, seed=7)


@pytest.mark.parametrize("cache", CACHES)
def test_append_what_is_not_finite(cache):
    """Infinities saturate and NaN stays NaN or becomes 0; neither counts for the scale.  In values, which are not rotated."""
    def spoil(qkv, Hq, H):
        v = qkv[:, Hq + H:]
        v[1, 0, 3], v[2, 1, 5], v[3, 0, 0] = math.inf, -math.inf, math.nan
    append_case([(12, 8)], 2, 2, 64, "bf16", cache, values=spoil)

    def spoil_keys(qkv, Hq, H):                          # of head 0: what head 1 gets is as ever
        k = qkv[:, Hq: Hq + H]
        k[1, 0, 3], k[2, 0, 40], k[5, 0, 0] = math.inf, -math.inf, math.nan
    append_case([(12, 8)], 2, 2, 64, "bf16", cache, values=spoil_keys)
    append_case([(40, 40)], 2, 2, 64, "f16", cache, values=spoil_keys, bs=8)


@pytest.mark.parametrize("cache", CACHES)
def test_append_rows_in_any_order(cache):
    """The tokens of a block in another order than its rows; the lowest row says what is held."""
    g = torch.Generator().manual_seed(13)
    bs, H, D, nb = 16, 2, 64, 3
    rows = [21, 19, 24, 22] + [32 + r for r in (7, 0, 3)]          # block 1 from row 3 on, block 2 afresh
    slots, T = torch.tensor(rows), len(rows)
    k, v = (torch.randn(T, H, D, generator=g) for _ in range(2))
    c0, s0 = random_cache(cache, nb, bs, H, D, g)
    codes, scales, status = c0.to(DEV), s0.to(DEV), ints([0])
    api.is_append_scaled(None, k.to(DEV), v.to(DEV), ints([0] * T), slots.to(DEV), rope_of(PLAIN), api.make_cache_desc(bs, nb, cache),
                         codes, scales, None, status)
    both = torch.stack([k, v]).double()
    sref.check_write(cache, bs, slots, torch.zeros(T, dtype=torch.bool), both, torch.zeros_like(both), (c0, s0),
                     (codes.cpu(), scales.cpu()))
    assert status.tolist() == [0]


@pytest.mark.parametrize("cache", CACHES)
def test_append_token_by_token(cache):
    """A block filled one token at a time: its scale ends as that of all tokens together, and what was rounded anew each
    time it grew is off by half a step of each scale that it had."""
    g = torch.Generator().manual_seed(12)
    bs, H, D, n = 16, 2, 64, 37
    k, v = (torch.randn(n, H, D, generator=g) * torch.linspace(0.2, 3, n)[:, None, None] for _ in range(2))
    nb, order = 3, [2, 0, 1]
    codes = torch.full((2, nb, bs, H, D), 77, dtype=sref.CODES[cache], device=DEV)
    scales, status = torch.full((2, nb, H), math.nan, device=DEV), ints([0])
    cd, zero = api.make_cache_desc(bs, nb, cache), ints([0])
    steps = torch.zeros(2, n, H)                         # the sum of the scales a row was rounded under
    for p in range(n):
        b = order[p // bs]
        before = scales.cpu()
        api.is_append_scaled(None, k[p: p + 1].to(DEV), v[p: p + 1].to(DEV), zero, ints([b * bs + p % bs], torch.int64),
                             rope_of(PLAIN), cd, codes, scales, None, status)
        s = scales.cpu()[:, b]
        steps[:, p] = s
        first = p // bs * bs
        grew = s != before[:, b]
        if p > first:
            steps[:, first:p] += (grew * s)[:, None]
    assert status.tolist() == [0]
    half = {"int8": 0.5, "e4m3": 16.0}[cache]            # half of the largest step, in the scale's units
    at = torch.tensor([order[p // bs] * bs + p % bs for p in range(n)])
    s = scales.cpu().double()
    got = sref.numbers(cache, codes.cpu()).view(2, nb * bs, H, D)[:, at] * s[:, at // bs, :, None]
    want = torch.stack([k, v]).double()
    assert bool(((got - want).abs() <= half * steps[..., None] * (1 + 2.0 ** -10)).all())
    for j in range(3):
        part = want[:, j * bs: (j + 1) * bs].abs().amax((1, 3)) / sref.QMAX[cache]
        assert bool(((s[:, order[j]] - part).abs() <= 2.0 ** -23 * part).all())


def test_append_skips_bad_tokens():
    """Bad slots and positions: nothing is written for them; a block with earlier rows and no scale keeps its codes."""
    x = torch.ones(6, 1, 64, device=DEV)
    codes, scales = torch.full((2, 3, 16, 1, 64), 99, dtype=torch.int8, device=DEV), torch.ones(2, 3, 1, device=DEV)
    scales[1, 2] = 0.0
    out, status = torch.full((6, 1, 64), math.nan, device=DEV), ints([0])
    api.is_append_scaled(x, x.clone(), x.clone(), ints([0, -1, 1 << 24, 3, 4, 5]), ints([0, 1, 2, 48, -2, 35], torch.int64),
                         rope_of(PLAIN), api.make_cache_desc(16, 3, "int8"), codes, scales, out, status)
    assert status.tolist() == [_lib.IS_ST_POSITION | _lib.IS_ST_BLOCK_ID | _lib.IS_ST_SCALE]
    good = [0, 5]
    assert bool(torch.isfinite(out[good]).all()) and bool(out[1:5].isnan().all())
    assert bool((codes[:, 0, 0] != 99).any()) and bool((codes[:, 0, 1:] == 99).all()) and bool((codes[:, 1] == 99).all())
    assert bool((codes[0, 2, 3] != 99).any()) and bool((codes[1, 2] == 99).all()) and float(scales[1, 2]) == 0.0
    codes2, scales2 = codes.clone(), scales.clone()      # nothing but refused tokens: nothing changes
    api.is_append_scaled(x[:2], x[:2].clone(), x[:2].clone(), ints([-1, -1]), ints([16, 17], torch.int64), rope_of(PLAIN),
                         api.make_cache_desc(16, 3, "int8"), codes, scales, out[:2], ints([0]))
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


def test_append_many_tokens_in_one_block():
    """One block of thousands of rows, as a cache without paging has it."""
    append_case([(3000, 2500)], 2, 2, 64, "bf16", "int8", bs=4096)


# ---------------------------------------------------------------- is_move_scaled

@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dtype,H,D,bs,fbs,reqs", [
    ("bf16", 8, 128, 16, 16, [(100, 100), (45, 20), (16, 16)]), ("f16", 2, 64, 32, 5, [(70, 33)]), ("f32", 2, 64, 16, 16, [(33, 30)]),
    ("bf16", 1, 16, 7, 3, [(20, 13)]), ("f32", 1, 256, 64, 8, [(100, 90)]), ("bf16", 3, 512, 16, 16, [(20, 20)]), ("bf16", 9, 32, 1, 16, [(5, 5)])])
def test_move(dtype, H, D, bs, fbs, reqs, cache):
    g = torch.Generator().manual_seed(3)
    slots, _, nb, held, _ = packed_slots(reqs, bs, g)
    T = len(slots)
    fnb = -(-T // fbs) + 2
    source = torch.randn(2, fnb, fbs, H, D, generator=g).to(ref.TORCH[dtype])
    from_slots = torch.randperm(fnb * fbs, generator=g)[:T]
    from_slots[T // 2] = -1                              # padding on either side
    slots[T - 1] = -1
    c0, s0 = random_cache(cache, nb, bs, H, D, g, held)
    codes, scales, status = c0.to(DEV), s0.to(DEV), ints([0])
    api.is_move_scaled(api.make_cache_desc(fbs, fnb, dtype), source.to(DEV), from_slots.to(DEV), api.make_cache_desc(bs, nb, cache),
                       codes, scales, slots.to(DEV), status)
    assert status.tolist() == [0]
    rows = source.double().view(2, fnb * fbs, H, D)[:, from_slots.clamp(min=0)]
    sref.check_write(cache, bs, slots, (slots < 0) | (from_slots < 0), rows, torch.zeros_like(rows), (c0, s0),
                     (codes.cpu(), scales.cpu()))


def test_move_skips_bad_slots():
    source = torch.ones(2, 1, 4, 1, 64, device=DEV)
    codes, scales, status = torch.zeros(2, 2, 4, 1, 64, dtype=torch.int8, device=DEV), torch.ones(2, 2, 1, device=DEV), ints([0])
    api.is_move_scaled(api.make_cache_desc(4, 1, "f32"), source, ints([0, 4, -3, 1, 2], torch.int64), api.make_cache_desc(4, 2, "int8"),
                       codes, scales, ints([0, 1, 2, 9, 4], torch.int64), status)
    assert status.tolist() == [_lib.IS_ST_BLOCK_ID]
    assert bool((codes[:, :, 0] == 127).all()) and bool((codes[:, :, 1:] == 0).all())


# ---------------------------------------------------------------- is_read_scaled

@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,D,bs,style,sections", [
    (1, 2, 64, 16, None, None), (77, 8, 128, 16, 0, None), (130, 3, 32, 7, 1, None), (20, 1, 16, 1, 0, None), (33, 2, 256, 24, 0, None),
    (40, 4, 128, 32, 0, [16, 24, 24]), (9, 5, 128, 16, 1, [40, 24]), (700, 4, 64, 16, None, None)])
def test_read(T, H, D, bs, style, sections, dtype, cache):
    g = torch.Generator().manual_seed(T)
    td, nb = ref.TORCH[dtype], -(-T // bs) + 2
    codes, scales = random_cache(cache, nb, bs, H, D, g)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if T > 5:
        slots[3] = -1
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, 1 << 20, (axes, T), generator=g, dtype=torch.int32)
    k_out, v_out, status = (torch.full((T, H, D), 7.0, dtype=td, device=DEV) for _ in range(2)), None, ints([0])
    k_out, v_out = k_out
    kw = {} if style is None else dict(positions=pos.to(DEV), rope=api.make_rope(1e6, style),
                                       axes=None if sections is None else api.make_axes(sections))
    cd, dev_codes, dev_scales = api.make_cache_desc(bs, nb, cache), codes.to(DEV), scales.to(DEV)
    api.is_read_scaled(slots.to(DEV), cd, dev_codes, dev_scales, k_out, v_out, status, **kw)
    assert status.tolist() == [0]
    at, keep = slots.clamp(min=0), slots >= 0
    x = sref.numbers(cache, codes).view(2, nb * bs, H, D)[:, at] * scales.double()[:, at // bs, :, None]
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    v_tol = ref.U[dtype] * x[1].abs() * (1 + 2.0 ** -10) + 2.0 ** -24 * x[1].abs() + tiny
    assert bool(((v_out.cpu().double() - x[1]).abs() <= v_tol)[keep].all())
    k, k_tol = x[0], ref.U[dtype] * x[0].abs() * (1 + 2.0 ** -10) + 2.0 ** -24 * x[0].abs() + tiny
    if style is not None:                                # turned back: the rotation by -p
        k, mag = ref.rotate(x[0], -pos, dict(theta=1e6, style=style), sections)
        k_tol = ref.rotated_tolerance(k, mag, dtype) + 2.0 ** -23 * mag
    assert bool(((k_out.cpu().double() - k).abs() <= k_tol)[keep].all())
    assert bool((k_out.cpu()[~keep] == 7).all()) and bool((v_out.cpu()[~keep] == 7).all())
    only = torch.full((T, H, D), 7.0, dtype=td, device=DEV)
    api.is_read_scaled(slots.to(DEV), cd, dev_codes, dev_scales, None, only, status)
    assert torch.equal(only, v_out)


def test_read_skips_bad_tokens():
    codes, scales = torch.ones(2, 2, 4, 2, 64, dtype=torch.int8, device=DEV), torch.ones(2, 2, 2, device=DEV)
    scales[0, 1, 1] = math.inf
    k, v, status = torch.zeros(5, 2, 64, device=DEV), torch.zeros(5, 2, 64, device=DEV), ints([0])
    api.is_read_scaled(ints([0, 8, -2, 5, 1], torch.int64), api.make_cache_desc(4, 2, "int8"), codes, scales, k, v, status,
                       positions=ints([0, 1, 2, 0, -1]), rope=rope_of(PLAIN))
    assert status.tolist() == [_lib.IS_ST_BLOCK_ID | _lib.IS_ST_POSITION | _lib.IS_ST_SCALE]
    assert bool((k[0] == 1).all()) and bool((k[3, 0] == 1).all()) and bool((k[3, 1] == 0).all()) and bool((v[3] == 1).all())
    assert bool((k[[1, 2, 4]] == 0).all()) and bool((v[[1, 2, 4]] == 0).all())


def test_write_and_read_back_facts():
    """Keys before the rotation come back from the cache that their rotated form was written to."""
    g = torch.Generator().manual_seed(4)
    T, H, D, bs = 90, 4, 128, 16
    k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    pos, slots, nb = torch.arange(T, dtype=torch.int32) + 777, torch.arange(T), 6
    codes, scales, status = torch.zeros(2, nb, bs, H, D, dtype=torch.int8, device=DEV), torch.zeros(2, nb, H, device=DEV), ints([0])
    cd = api.make_cache_desc(bs, nb, "int8")
    api.is_append_scaled(None, k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), rope_of(LLAMA), cd, codes, scales, None, status)
    k2, v2 = torch.empty(T, H, D, device=DEV), torch.empty(T, H, D, device=DEV)
    api.is_read_scaled(slots.to(DEV), cd, codes, scales, k2, v2, status, positions=pos.to(DEV), rope=rope_of(LLAMA))
    assert status.tolist() == [0]
    s = scales.cpu().double()[:, slots // bs][..., None]
    # half a step of each of a pair's two codes, turned back: sqrt(2) halves at most
    assert bool(((k2.cpu().double() - k.double()).abs() <= s[0] * (0.5 * math.sqrt(2) + 0.01)).all())
    assert bool(((v2.cpu().double() - v.double()).abs() <= s[1] * 0.501).all())


# ---------------------------------------------------------------- is_attend_scaled

def attend_case(reqs, Hq, H, D, dtype, cache, bs=16, window=0, scale=None, seed=0, before=0, behind=0, holes=(), bad=(),
                use_start=True, max_q=None, spread_q=False, gain=1.0, extra_width=2, spread_scales=0, run=None):
    """reqs: (seq_len, query rows); holes: (request, block, id) table entries overwritten; bad: (request, block, kv, scale)
    scales overwritten; spread_scales: powers of two between blocks' magnitudes.  Unused blocks have NaN scales and
    unused rows the largest codes (E4M3: NaN), so what is read but should not count shows.  Checks every row."""
    g = torch.Generator().manual_seed(seed)
    td = ref.TORCH[dtype]
    R = len(reqs)
    need = [-(-n // bs) for n, _ in reqs]
    nb = sum(need) + 3
    ids = torch.randperm(nb, generator=g).tolist()
    table = torch.full((R, max(max(need), 1) + extra_width), -1, dtype=torch.int32)
    held = torch.zeros(nb, dtype=torch.int64)
    for r, k in enumerate(need):
        for j in range(k):
            table[r, j] = ids.pop()
            held[table[r, j]] = min(bs, reqs[r][0] - j * bs)
    x = gain * torch.randn(2, nb, bs, H, D, generator=g).double()
    x = x * 2.0 ** torch.randint(-spread_scales, spread_scales + 1, (2, nb, 1, H, 1), generator=g)
    if spread_scales:                                    # keys of one magnitude, so that many count
        x[0] /= x[0].abs().amax((1, 3), keepdim=True)
    codes, scales = sref.quantised(cache, x, held)
    unused = torch.arange(bs)[None] >= held[:, None]
    codes[:, unused] = 127                               # E4M3: 0x7f is NaN
    scales[:, held == 0] = math.nan
    named = [torch.ones(n, dtype=torch.bool) for n, _ in reqs]
    want_bits = 0
    k, v, used = [], [], [torch.ones(1)]
    for r, (n, _) in enumerate(reqs):
        j = torch.arange(n)
        b = table[r].long()[j // bs]
        k.append(sref.numbers(cache, codes[0, b, j % bs]) * scales[0, b].double()[..., None])
        v.append(sref.numbers(cache, codes[1, b, j % bs]) * scales[1, b].double()[..., None])
        used.append(scales[1, b].flatten())
    used = torch.cat(used[1:]) if sum(n for n, _ in reqs) else used[0]
    for r, b, kv, s in bad:
        scales[kv, table[r, b]] = s
        codes[:, table[r, b]] = 127                      # E4M3: NaN
        named[r][b * bs: (b + 1) * bs] = False
        want_bits |= _lib.IS_ST_SCALE
    for r, b, i in holes:
        table[r, b] = i
        named[r][b * bs: (b + 1) * bs] = False
        want_bits |= _lib.IS_ST_BLOCK_ID
    starts = np.cumsum([before] + [m for _, m in reqs]).tolist()
    row = starts.pop()
    q = (gain * torch.randn(row + behind, Hq, D, generator=g)).to(td)
    qd = q.to(DEV)
    if spread_q:
        wide = torch.full((q.shape[0], Hq + 3, D), math.nan, dtype=td, device=DEV)
        wide[:, 1: 1 + Hq] = qd
        qd = wide[:, 1: 1 + Hq]
    out = torch.full((q.shape[0], Hq, D), 7.0, dtype=td, device=DEV)
    lse, status = torch.full((q.shape[0], Hq), 7.0, device=DEV), ints([0])
    scale = D ** -0.5 if scale is None else scale
    kw = dict(q_start=ints(starts + [row]) if use_start else None, max_q_len=max_q or max(1, max(m for _, m in reqs)), scale=scale,
              window=window, lse_out=lse)
    args = (qd, ints([n for n, _ in reqs]), table.to(DEV), api.make_cache_desc(bs, nb, cache), codes.to(DEV), scales.to(DEV), out,
            api.attend_workspace(), status)
    if run is None:
        api.is_attend_scaled(*args, **kw)
    else:
        run(args, kw)
    torch.cuda.synchronize()
    assert status.item() == want_bits
    out, lse = out.cpu(), lse.cpu()
    owned = torch.zeros(q.shape[0], dtype=torch.bool)
    for r, (n, m) in enumerate(reqs):
        if m == 0:
            continue
        rows = slice(starts[r], starts[r] + m)
        owned[rows] = True
        o, ls, spread, heft, seen = ref.attend(q[rows].double(), n, k[r], v[r], named[r], scale, window)
        tol, ltol = sref.attend_tolerance(dtype, D, o, ls, spread, heft, seen, used, sref.QMAX[cache])
        err = (out[rows].double() - o).abs()
        assert bool((err <= tol).all()), (r, float((err / tol.clamp(min=1e-30)).max()))
        none = seen == 0
        assert bool((lse[rows][none] == -math.inf).all()) and bool((out[rows][none] == 0).all())
        lerr = (lse[rows].double() - ls).abs()[~none]
        assert bool((lerr <= ltol[~none]).all()), (r, float((lerr / ltol[~none]).max()))
    assert bool((out[~owned] == 7.0).all()) and bool((lse[~owned] == 7.0).all())


TYPES = [("bf16", "int8"), ("bf16", "e4m3"), ("f16", "int8"), ("f16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (7, 1, 128), (4, 4, 128), (6, 2, 256), (20, 1, 64)])
def test_decode_ragged(Hq, H, D, dtype, cache):
    attend_case([(n, 1) for n in (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300)], Hq, H, D, dtype, cache)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_one_long_request_is_split(dtype, cache):
    attend_case([(9001, 1)], 4, 1, 128, dtype, cache)
    attend_case([(3000, 1), (1, 1), (7777, 1)], 8, 2, 64, dtype, cache)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bs", [1, 5, 8, 24, 64, 1000])
def test_decode_block_sizes(bs, dtype, cache):
    attend_case([(n, 1) for n in (1, 5, 49, 200, 333)], 4, 2, 64, dtype, cache, bs=bs)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1 << 30])
def test_windows(window, dtype, cache):
    attend_case([(1, 1), (16, 1), (17, 1), (130, 1), (500, 1)], 4, 2, 64, dtype, cache, window=window)
    attend_case([(60, 33), (5, 5), (300, 70)], 4, 2, 128, dtype, cache, window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (7, 1, 128), (4, 2, 256)])
def test_few_and_many_rows(Hq, H, D, dtype, cache):
    attend_case([(40, 2), (3, 3), (100, 0), (257, 4), (0, 0), (9, 1)], Hq, H, D, dtype, cache, before=2, behind=3)
    attend_case([(140, 129), (64, 64), (200, 1), (77, 31)], Hq, H, D, dtype, cache, behind=5)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,bs,window", [(4, 1, 64, 16, 0), (7, 1, 64, 24, 0), (4, 2, 128, 16, 0), (4, 1, 128, 5, 0),
                                              (2, 1, 256, 16, 0), (4, 1, 64, 8, 700), (4, 1, 128, 128, 900), (4, 1, 128, 40, 0)])
def test_long_prompts(Hq, H, D, bs, window, dtype, cache):
    attend_case([(3333, 200), (70, 70), (5000, 129), (1999, 1)], Hq, H, D, dtype, cache, bs=bs, window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_rows_that_see_nothing(dtype, cache):
    attend_case([(3, 5), (0, 4), (0, 1), (2, 1)], 4, 2, 64, dtype, cache)
    attend_case([(10, 90), (0, 70)], 4, 1, 128, dtype, cache)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("cache", CACHES)
def test_unnamed_blocks_and_bad_scales_are_hidden(cache, rows):
    attend_case([(100, rows), (47, min(rows, 47)), (70, rows)], 4, 2, 64, "bf16", cache, holes=((0, 2, -1), (1, 0, -5), (2, 4, 1 << 30)))
    for s in (0.0, -1.0, math.nan, math.inf, 2.0 ** -41, 2.0 ** 41):
        for kv in (0, 1):
            attend_case([(100, rows), (50, rows)], 4, 2, 128, "bf16", cache, bad=((0, 1, kv, s), (1, 3, kv, s)))
    attend_case([(16, 1), (100, rows)], 4, 2, 128, "f16", cache, bad=((0, 0, 1, 0.0),))        # nothing left


@pytest.mark.parametrize("rows", [1, 6, 50])
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scales_far_apart(dtype, cache, rows):
    """Blocks whose values lie up to 2^24 (fp16 output: 2^12) and 2^70 apart, in one request."""
    attend_case([(300, rows), (77, rows)], 8, 2, 64, dtype, cache, spread_scales=6 if dtype == "f16" else 12)
    if dtype == "bf16":
        attend_case([(500, rows)], 4, 1, 128, dtype, cache, spread_scales=30)


@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("cache", CACHES)
def test_large_logits(cache, rows):
    """Logits in the thousands: one key takes all weight, or nearly."""
    attend_case([(200, rows), (61, rows)], 4, 2, 128, "bf16", cache, gain=30.0, scale=0.5)
    attend_case([(200, rows), (61, rows)], 4, 2, 64, "f16", cache, gain=8.0, scale=1.0)


@pytest.mark.parametrize("Hq,H", [(16, 1), (33, 1), (71, 1), (8, 8)])
def test_wide_groups(Hq, H):
    attend_case([(40, 1), (300, 1)], Hq, H, 64, "bf16", "int8")
    attend_case([(90, 40), (300, 5)], Hq, H, 128, "bf16", "int8")


@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_odd_scales(scale, rows):
    attend_case([(100, rows), (33, min(rows, 33))], 4, 2, 64, "bf16", "int8", scale=scale)


def test_thousands_of_requests():
    attend_case([(1 + i % 37, 1) for i in range(4096)], 2, 1, 64, "bf16", "int8")


def test_many_requests_without_q_start_and_strided_q():
    attend_case([(5 + 3 * i, 1) for i in range(130)], 4, 2, 64, "bf16", "int8", use_start=False, spread_q=True)
    attend_case([(90, 50), (60, 20)], 4, 2, 128, "f16", "e4m3", spread_q=True)


def test_single_tokens_under_a_large_bound():
    attend_case([(40, 1), (333, 1), (1, 1)], 4, 2, 128, "bf16", "int8", max_q=100)


@pytest.mark.parametrize("rows", [1, 80])
def test_same_call_gives_the_same_bits(rows):
    got = []

    def run(args, kw):
        for _ in range(3):
            args[6].fill_(7.0)
            args[7].fill_(0xFF)                          # what the workspace holds means nothing
            api.is_attend_scaled(*args, **kw)
            got.append(args[6].clone())
    attend_case([(4000, rows), (100, min(rows, 100)), (2500, rows)], 8, 2, 128, "bf16", "int8", run=run)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_unit_scales_match_an_fp8_cache():
    """E4M3 codes under scales of 1 are an FP8 cache of is_attend: the same products, in the same order."""
    g = torch.Generator().manual_seed(9)
    nb, H, Hq, D, bs = 40, 2, 8, 128, 16
    codes = (torch.randn(2, nb, bs, H, D, generator=g) * 3).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    for rows in (1, 70):
        q = torch.randn(rows, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
        outs = [torch.empty_like(q) for _ in range(2)]
        table, status, ws = torch.arange(nb, dtype=torch.int32, device=DEV)[None], ints([0]), api.attend_workspace()
        kw = dict(q_start=ints([0, rows]), max_q_len=rows)
        cd = api.make_cache_desc(bs, nb, "e4m3")
        api.is_attend(q, ints([600]), table, cd, codes, outs[0], ws, status, **kw)
        api.is_attend_scaled(q, ints([600]), table, cd, codes, torch.ones(2, nb, H, device=DEV), outs[1], ws, status, **kw)
        assert status.tolist() == [0]
        assert bool(((outs[0].float() - outs[1].float()).abs() <= 2.0 ** -7 * outs[0].float().abs() + 2.0 ** -9).all())


def test_cache_past_32_bits():
    """A layer of 4.6 GB of codes whose used blocks lie at its end: byte offsets pass 2^32."""
    H, D, bs, nb = 8, 128, 16, 140000
    g = torch.Generator(device=DEV).manual_seed(4)
    n, used = 40, [nb - 1, 3, nb - 2]
    big = torch.empty((2, nb, bs, H, D), dtype=torch.int8, device=DEV), torch.ones((2, nb, H), device=DEV)
    small = torch.empty((2, 3, bs, H, D), dtype=torch.int8, device=DEV), torch.ones((2, 3, H), device=DEV)
    qkv = torch.randn((n, 32 + 2 * H, D), generator=g, device=DEV).to(torch.bfloat16)
    got = []
    for (codes, scales), ids in ((big, used), (small, [0, 1, 2])):
        t = torch.arange(n, device=DEV)
        slots = ints(ids, torch.int64)[t // bs] * bs + t % bs
        q, status = torch.empty((n, 32, D), dtype=torch.bfloat16, device=DEV), ints([0])
        cd = api.make_cache_desc(bs, codes.shape[1], "int8")
        api.is_append_scaled(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], t.to(torch.int32), slots, rope_of(LLAMA), cd, codes, scales,
                             q, status)
        for rows in (1, n):
            out = torch.empty((rows, 32, D), dtype=torch.bfloat16, device=DEV)
            api.is_attend_scaled(q[n - rows:], ints([n]), ints([ids]), cd, codes, scales, out, api.attend_workspace(), status,
                                 q_start=ints([0, rows]), max_q_len=rows)
            got.append(out.cpu())
        k, v = (torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        api.is_read_scaled(slots, cd, codes, scales, k, v, status)
        got += [k.cpu(), v.cpu()]
        assert status.tolist() == [0]
    assert all(torch.equal(a, b) for a, b in zip(got[:4], got[4:]))


@pytest.mark.parametrize("rows", [1, 60])
def test_graphs_and_streams(rows):
    """Two captured graphs of a write, an attention and a read, a workspace each, replay on two streams at once, over
    tensors made on another; replays read the buffers' new contents."""
    H, Hq, D, bs, nb = 2, 8, 128, 16, 200
    g = torch.Generator(device=DEV).manual_seed(6)
    sets = []
    for i in range(2):
        n = 1400 + 300 * i
        x = torch.randn((rows, Hq + 2 * H, D), generator=g, device=DEV).to(torch.bfloat16)
        codes = torch.randint(-127, 128, (2, nb, bs, H, D), generator=g, device=DEV, dtype=torch.int8)
        table = torch.randperm(nb, generator=g, device=DEV)[:120].to(torch.int32)[None].contiguous()
        pos = torch.arange(n - rows, n, device=DEV)
        t = dict(x=x, seq=ints([n]), table=table, codes=codes, scales=torch.full((2, nb, H), 0.01, device=DEV),
                 pos=pos.to(torch.int32), slots=table[0, pos // bs].long() * bs + pos % bs, q=torch.zeros_like(x[:, :Hq]).contiguous(),
                 ws=api.attend_workspace(), status=ints([0]), start=ints([0, rows]))
        t.update(out=torch.zeros_like(t["q"]), k=torch.zeros(rows, H, D, dtype=torch.bfloat16, device=DEV),
                 v=torch.zeros(rows, H, D, dtype=torch.bfloat16, device=DEV))
        sets.append(t)
    cd = api.make_cache_desc(bs, nb, "int8")

    def call(t):
        x = t["x"]
        api.is_append_scaled(x[:, :Hq], x[:, Hq: Hq + H], x[:, Hq + H:], t["pos"], t["slots"], rope_of(LLAMA), cd, t["codes"],
                             t["scales"], t["q"], t["status"])
        api.is_attend_scaled(t["q"], t["seq"], t["table"], cd, t["codes"], t["scales"], t["out"], t["ws"], t["status"],
                             q_start=t["start"], max_q_len=rows)
        api.is_read_scaled(t["slots"], cd, t["codes"], t["scales"], t["k"], t["v"], t["status"], positions=t["pos"],
                           rope=rope_of(LLAMA))
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for t, s in zip(sets, streams):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                call(t)
        graphs.append(graph)
    for turn in range(2):
        for t in sets:
            if turn:
                t["x"].normal_(generator=g).mul_(3.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        for t in sets:
            got = {name: t[name].clone() for name in ("out", "k", "v", "codes", "scales")}
            for name in ("out", "k", "v"):
                t[name].zero_()
            call(t)                                      # the same tokens once more: nothing grows, nothing changes
            torch.cuda.synchronize()
            assert all(torch.equal(t[name], got[name]) for name in got) and bool(got["out"].any()) and t["status"].tolist() == [0]


# ---------------------------------------------------------------- all of them behind an injection

@pytest.mark.parametrize("cache_dtype", CACHES)
def test_step_behind_an_injected_segment(cache_dtype):
    """A segment is injected into a 16-bit cache and moved into a scaled one; a prompt follows it, then single tokens;
    attention at each step against one fp64 attention over what the cache holds; what was written is read back, stored
    as facts, retrieved and injected again."""
    H, D, Hq, bs, L = 4, 64, 8, 16, 1
    g = torch.Generator().manual_seed(8)
    lens = [7, 19, 30, 4, 11]
    cfg = api.make_config(num_layers=L, num_kv_heads=H, head_dim=D, emb_dim=64, kv_dtype="bf16", emb_dtype="f16", max_facts=8,
                          max_tokens=200, max_users=2, max_queries=4, max_k=4)
    with api.is_store_create(cfg, 0) as store:
        fk, fv = (torch.randn(sum(lens), L, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
        api.is_store_add_facts(store, 0, lens, fk.to(DEV), fv.to(DEV), torch.randn(5, 64, generator=g).half().to(DEV))
        facts = [[2, 0], [4, 1], [3]]
        segs = [sum(lens[f] for f in fs) for fs in facts]
        R, W, nb = 3, 8, 40
        status = ints([0])
        # the segments, in a 16-bit cache with a table of its own
        plain, pd = torch.full((L, 2, 12, bs, H, D), math.nan, dtype=torch.bfloat16, device=DEV), api.make_cache_desc(bs, 12, "bf16")
        from_slots = torch.full((sum(segs),), -1, dtype=torch.int64, device=DEV)
        api.is_inject(store, ints([f + [-1] * (2 - len(f)) for f in facts], torch.int64), ints([len(f) for f in facts]),
                      ints([0] * R), rope_of(LLAMA), ints([[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]]), pd, plain,
                      slot_mapping_out=from_slots)
        assert api.is_get_status(store) == 0
        # blocks and slots in the scaled one
        codes = torch.full((2, nb, bs, H, D), 127, dtype=sref.CODES[cache_dtype], device=DEV)
        scales, cd = torch.full((2, nb, H), math.nan, device=DEV), api.make_cache_desc(bs, nb, cache_dtype)
        table, free = torch.full((R, W), -1, dtype=torch.int32, device=DEV), torch.randperm(nb, generator=g).to(torch.int32).to(DEV)
        seq, head = ints([0] * R), ints([0])

        def extend(new):
            nonlocal seq, head
            T = sum(new)
            slots, pos = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
            start, seq2, head2 = ints([0] * (R + 1)), torch.empty_like(seq), torch.empty_like(head)
            api.is_extend_block_table(seq, ints(new), free, bs, nb, table, slots, pos, start, seq2, status, free_head=head,
                                      free_head_out=head2)
            seq, head = seq2, head2
            return slots, pos, start
        slots, seg_pos, _ = extend(segs)
        seg_slots = slots
        api.is_move_scaled(pd, plain[0], from_slots, cd, codes, scales, slots, status)
        ws = api.attend_workspace()
        for new in ([9, 1, 40], [1, 1, 1], [1, 0, 1], [17, 1, 3]):
            T = sum(new)
            x = torch.randn(T, Hq + 2 * H, D, generator=g).to(torch.bfloat16).to(DEV)
            slots, pos, start = extend(new)
            q, out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
            c0, s0 = codes.cpu(), scales.cpu()
            api.is_append_scaled(x[:, :Hq], x[:, Hq: Hq + H], x[:, Hq + H:], pos, slots, rope_of(LLAMA), cd, codes, scales, q, status)
            api.is_attend_scaled(q, seq, table, cd, codes, scales, out, ws, status, q_start=start, max_q_len=max(new))
            c1, s1 = codes.cpu(), scales.cpu()
            y, mag = ref.rotate(x[:, Hq: Hq + H].cpu().double(), pos.cpu()[None], LLAMA)
            sref.check_write(cache_dtype, bs, slots.cpu(), torch.zeros(T, dtype=torch.bool), torch.stack([y, x[:, Hq + H:].cpu().double()]),
                             torch.stack([mag * ref.ROTATE, mag * 0]), (c0, s0), (c1, s1))
            st, tb = start.tolist(), table.cpu().long()
            for r in range(R):
                if new[r] == 0:
                    continue
                n = int(seq[r])
                j = torch.arange(n)
                b = tb[r][j // bs]
                k, v = (sref.numbers(cache_dtype, c1[kv, b, j % bs]) * s1[kv, b].double()[..., None] for kv in range(2))
                rows = slice(st[r], st[r + 1])
                o, ls, spread, heft, seen = ref.attend(q[rows].cpu().double(), n, k, v, torch.ones(n, dtype=torch.bool), D ** -0.5, 0)
                tol, _ = sref.attend_tolerance("bf16", D, o, ls, spread, heft, seen, s1[:, b], sref.QMAX[cache_dtype])
                assert bool(((out[rows].cpu().double() - o).abs() <= tol).all())
        # the first request's segment, read back with its keys turned back, as one new fact of another user
        n = segs[0]
        k, v = (torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        api.is_read_scaled(seg_slots[:n].contiguous(), cd, codes, scales, k, v, status, positions=seg_pos[:n].contiguous(),
                           rope=rope_of(LLAMA))
        emb = torch.randn(1, 64, generator=g).half().to(DEV)
        api.is_store_capture_begin(store, 1, [0], [n], emb)
        api.is_store_capture_layer(store, 0, k, v)
        new_id = api.is_store_capture_end(store, 1)
        again = torch.zeros(L, 2, 4, bs, H, D, dtype=torch.bfloat16, device=DEV)
        ids = torch.empty(1, 1, dtype=torch.int64, device=DEV)
        api.is_retrieve_and_inject(store, ints([1]), emb, 1, ints([0]), rope_of(LLAMA), ints([[0, 1, 2, 3]]),
                                   api.make_cache_desc(bs, 4, "bf16"), again, ids_out=ids)
        assert api.is_get_status(store) == 0 and ids.tolist() == [new_id.tolist()] and status.tolist() == [0]
        got, want = again[0].cpu().double().view(2, 64, H, D)[:, :n], plain[0].cpu().double().view(2, -1, H, D)[:, from_slots[:n].cpu()]
        b = seg_slots[:n].cpu() // bs
        unit = scales.cpu().double()[:, b][..., None]
        # a code's half step (its block's scale has grown at most four times since: five roundings), for keys of a pair's
        # two codes, and three roundings to bf16: read, rotated again, and the first copy's own
        half = {"int8": 0.5, "e4m3": 16.0}[cache_dtype] * 5 * math.sqrt(2)
        size = want.abs().amax(-1, keepdim=True) * math.sqrt(2) + half * unit
        assert bool(((got - want).abs() <= half * unit + 3 * 2.0 ** -8 * size).all())


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("dtype,cache,D,bs", [("bf16", "int8", 128, 16), ("f16", "e4m3", 64, 8), ("bf16", "e4m3", 64, 16), ("f16", "int8", 128, 40)])
def test_waits_that_run_out(dtype, cache, D, bs):
    """A prompt with limits of its waits that it cannot keep ends with IS_ST_TIMEOUT and nothing else, and the next call on
    the same stream and workspace gives the bits that it gave before."""
    g = torch.Generator().manual_seed(61)
    H, Hq, lens, start = 2, 8, [3333, 900, 70], [0, 200, 300, 370]
    need = [-(-n // bs) for n in lens]
    nb = sum(need)
    table, at = torch.full((3, max(need)), -1, dtype=torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = torch.arange(at, at + n)
        at += n
    codes, scales = random_cache(cache, nb, bs, H, D, g)
    q = torch.randn(start[-1], Hq, D, generator=g).to(ref.TORCH[dtype]).to(DEV)
    args = (q, ints(lens), table.to(DEV), api.make_cache_desc(bs, nb, cache), codes.to(DEV), scales.to(DEV))
    ws, status = api.attend_workspace(), ints([0])

    def call(**kw):
        out = torch.zeros_like(q)
        api.is_attend_scaled(*args, out, ws, status, q_start=ints(start), max_q_len=200, **kw)
        torch.cuda.synchronize()
        bits = status.item()
        status.zero_()
        return out.cpu(), bits

    want, bits = call()
    assert bits == 0 and bool(want.isfinite().all())
    seen = 0
    for budget in (0, 0, 500, 2000, 10000, 100000):
        out, bits = call(budget_ns=budget)
        assert bits in (0, _lib.IS_ST_TIMEOUT) and (bits or torch.equal(out, want))
        seen |= bits
        out, bits = call()
        assert bits == 0 and torch.equal(out, want)
    assert seen == _lib.IS_ST_TIMEOUT


# ---------------------------------------------------------------- many short groups in a call

@pytest.mark.parametrize("cache,D,bs", [("int8", 64, 16), ("e4m3", 128, 16), ("int8", 128, 32), ("int8", 128, 64), ("e4m3", 256, 8)])
def test_append_many_requests(cache, D, bs):
    """Hundreds of requests with one to a few new tokens each, so that a CTA has many groups, some in new blocks and some
    that raise a block's scale, with padding between requests."""
    reqs = [(1 + (37 * i) % 90, 1 + (i % 7 == 0) * (i % 5)) for i in range(700)]
    reqs = [(n, min(n, m)) for n, m in reqs]
    at = np.cumsum([0] + [m for _, m in reqs])
    skip = [int(at[r]) for r in range(0, 700, 53) if reqs[r][1] == 1]       # a block's tokens stay adjacent
    append_case(reqs, 4, 3, D, "bf16", cache, bs=bs, skip=skip)


@pytest.mark.parametrize("Hq,H,D", [(2, 32, 64), (33, 9, 64), (4, 3, 128)])
def test_append_long_prompts(Hq, H, D):
    """More CTAs than fit at once, of which those of the queries are fewer or more than those of the groups."""
    append_case([(1700, 1650), (90, 1), (1301, 1300), (2000, 1999)], Hq, H, D, "bf16", "int8")
