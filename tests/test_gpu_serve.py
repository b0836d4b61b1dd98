"""The serving step around the segment on the GPU: is_extend_block_table,
is_append and is_attend against their plain 64-bit definitions, at the lengths,
masks, strides and layouts where they can go wrong, and all of them behind an
injection.  Unused cache rows hold NaN (FP8: NaN bytes), so a row read that
should not be shows."""
import math

import numpy as np
import pytest
import torch

from kv_cache_injection_gb300 import _lib, api
from synth import staging, workloads
from tests import gpu_helpers as gh
from tests import serve_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    gh.ensure_built()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def bits_of(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[x.element_size()])


def nan_cache(shape, cache):
    if cache == "e4m3":
        return torch.full(shape, 0x7F, dtype=torch.uint8)
    return torch.full(shape, math.nan, dtype=ref.TORCH[cache])


def quantise(x, cache, scale):
    if cache == "e4m3":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(ref.TORCH[cache])


# ---------------------------------------------------------------- is_extend_block_table

def run_extend(seq, new, table, free, bs, num_blocks, head=None, capacity=None, num_free=None):
    R = len(seq)
    cap = capacity or max(1, sum(max(0, m) for m in new) + 3)
    t = dict(table=ints(table), slots=torch.full((cap,), -9, dtype=torch.int64, device=DEV),
             pos=torch.full((cap,), -9, dtype=torch.int32, device=DEV),
             start=torch.full((R + 1,), -9, dtype=torch.int32, device=DEV),
             out=torch.full((R,), -9, dtype=torch.int32, device=DEV), head_out=ints([-9]), status=ints([0]))
    api.is_extend_block_table(ints(seq), ints(new), ints(free), bs, num_blocks, t["table"], t["slots"], t["pos"],
                              t["start"], t["out"], t["status"], free_head=None if head is None else ints([head]),
                              free_head_out=t["head_out"])
    return {k: v.cpu().tolist() for k, v in t.items()}


@pytest.mark.parametrize("R,bs,lens,news", [
    (1, 16, [0], [1]), (1, 16, [16], [1]), (1, 16, [15], [2]), (3, 16, [0, 0, 5], [0, 0, 0]), (4, 1, [0, 1, 2, 3], [1, 0, 3, 2]),
    (5, 7, [6, 7, 8, 0, 13], [1, 1, 0, 15, 2]), (2, 16, [33, 1], [5000, 4096]), (2, 1 << 24, [5, 0], [3, 9])])
def test_extend_small(R, bs, lens, news):
    rng = np.random.default_rng(R * 31 + bs)
    need = [-(-(n + m) // bs) for n, m in zip(lens, news)]
    have = [-(-n // bs) for n in lens]
    nb = sum(need) + 7
    ids = rng.permutation(nb).tolist()
    W = max(need) + 2
    table = [[-1] * W for _ in lens]
    for r in range(R):
        for j in range(have[r]):
            table[r][j] = ids.pop()
    for head in (None, 3):
        got = run_extend(lens, news, table, ids, bs, nb, head)
        want = ref.extend(lens, news, ids, head or 0, table, bs, nb, len(got["slots"]))
        total = sum(news)
        assert got["table"] == want[0]
        assert got["slots"] == want[1]
        assert got["pos"] == want[2] + [-9] * (len(got["pos"]) - total)
        assert got["start"] == want[3] and got["out"] == want[4] and got["head_out"] == [want[5]]
        assert got["status"] == [0]


@pytest.mark.parametrize("R", [255, 256, 257, 1000, 4096])
def test_extend_many_requests(R):
    rng = np.random.default_rng(R)
    bs = 16
    lens, news = rng.integers(0, 200, R).tolist(), rng.integers(0, 40, R).tolist()
    need = [-(-(n + m) // bs) for n, m in zip(lens, news)]
    ids = rng.permutation(sum(need) + 11).tolist()
    table = [[-1] * (max(need) + 1) for _ in lens]
    for r in range(R):
        for j in range(-(-lens[r] // bs)):
            table[r][j] = ids.pop()
    got = run_extend(lens, news, table, ids, bs, sum(need) + 11, 2)
    want = ref.extend(lens, news, ids, 2, table, bs, sum(need) + 11, len(got["slots"]))
    assert got["table"] == want[0] and got["slots"] == want[1] and got["start"] == want[3]
    assert got["out"] == want[4] and got["head_out"] == [want[5]] and got["status"] == [0]


def test_extend_refuses_on_the_device():
    """Each refused request keeps its packed tokens (slot and position -1), takes no block and keeps its length."""
    table = [[-1] * 3 for _ in range(7)]
    table[0][0], table[6][0] = 5, 5
    lens = [3, -1, 2, 1 << 24, 0, 0, 4]
    news = [2, 2, -5, 1, 49, 17, 1]
    got = run_extend(lens, news, table, [9], 16, 64)
    #        fits   bad length  bad count  position  row too short  two blocks of a list of one  fits
    assert got["start"] == [0, 2, 4, 4, 5, 54, 71, 72]
    assert got["out"] == [5, -1, 2, 1 << 24, 0, 0, 5]
    assert got["slots"][:2] == [83, 84] and got["slots"][71] == 84
    assert set(got["slots"][2:71]) == {-1} and set(got["pos"][2:71]) == {-1}
    assert got["pos"][:2] == [3, 4] and got["pos"][71] == 4
    assert got["table"] == table and got["head_out"] == [0]
    assert got["status"] == [_lib.IS_ST_COUNT | _lib.IS_ST_POSITION | _lib.IS_ST_BLOCK_TABLE | _lib.IS_ST_FREE_LIST]


def test_extend_free_list_runs_out_behind_earlier_requests():
    got = run_extend([0, 0, 0, 15], [16, 40, 16, 1], [[-1] * 4] * 3 + [[7, -1, -1, -1]], [3, 1], 16, 8)
    assert got["head_out"] == [1] and got["table"][0] == [3, -1, -1, -1] and got["table"][1] == [-1] * 4
    assert got["out"] == [16, 0, 0, 16] and got["status"] == [_lib.IS_ST_FREE_LIST]
    assert got["slots"][72] == 7 * 16 + 15            # needs no block, so it goes on
    assert got["slots"][56:72] == [-1] * 16


@pytest.mark.parametrize("head", [-1, 3])
def test_extend_bad_head_takes_nothing(head):
    got = run_extend([0], [1], [[-1]], [0, 1], 16, 4, head)
    assert got["status"] == [_lib.IS_ST_FREE_LIST] and got["slots"][0] == -1 and got["table"] == [[-1]]


def test_extend_bad_block_ids_and_full_slot_map():
    got = run_extend([3, 16], [2, 1], [[64, -1], [1, -1]], [99], 16, 64, capacity=2)
    assert got["slots"] == [-1, -1] and got["pos"] == [3, 4]
    assert got["status"] == [_lib.IS_ST_BLOCK_ID | _lib.IS_ST_COUNT]
    assert got["start"] == [0, 2, 3] and got["out"] == [5, 17]


def test_extend_without_optional_outputs():
    slots, status = torch.full((4,), -9, dtype=torch.int64, device=DEV), ints([0])
    api.is_extend_block_table(ints([3]), ints([2]), torch.empty(0, dtype=torch.int32, device=DEV), 16, 8,
                              ints([[6]]), slots, status_out=status)
    assert slots.tolist() == [99, 100, -1, -1] and status.tolist() == [0]


# ---------------------------------------------------------------- is_append

PLAIN = dict(theta=1e4, style=0)
LLAMA = dict(theta=5e5, style=0, scaling=(1, 8.0, 1.0, 4.0, 8192))


def rope_of(spec):
    return api.make_rope(spec["theta"], spec["style"], *spec.get("scaling", ()))


def append_case(T, Hq, H, D, dtype, cache, spec, sections=None, interleaved=False, bs=16, scales=(1.0, 1.0), seed=0,
                fused=True, high=4000, skip=()):
    g = torch.Generator().manual_seed(seed)
    td = ref.TORCH[dtype]
    qkv = torch.randn(T, Hq + 2 * H, D, generator=g).to(td)
    dev = qkv.to(DEV)
    if fused:
        q, k, v = dev[:, :Hq], dev[:, Hq: Hq + H], dev[:, Hq + H:]
    else:
        q, k, v = (x.contiguous() for x in (dev[:, :Hq], dev[:, Hq: Hq + H], dev[:, Hq + H:]))
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, high, (axes, T), generator=g, dtype=torch.int32)
    pos[:, -1] = high - 1
    nb = -(-T // bs) + 3
    slots = torch.randperm(nb * bs, generator=g)[:T]
    for t in skip:
        slots[t] = -1
    store = nan_cache((2, nb, bs, H, D), cache)
    lc = store.to(DEV)
    q_out = torch.full((T, Hq, D), math.nan, dtype=td, device=DEV)
    status = ints([0])
    api.is_append(q if Hq else None, k, v, pos.to(DEV), slots.to(DEV), rope_of(spec),
                  api.make_cache_desc(bs, nb, cache, *scales), lc, q_out if Hq else None, status,
                  axes=api.make_axes(sections, interleaved) if sections else None)
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    keep = slots >= 0
    x = qkv.double()
    got_q, got = q_out.cpu(), lc.cpu().view(2, nb * bs, H, D)
    if Hq:
        y, mag = ref.rotate(x[:, :Hq], pos, spec, sections, interleaved)
        tol = ref.rotated_tolerance(y, mag, dtype)
        assert bool(((got_q.double() - y).abs() <= tol)[keep].all())
        assert bool(got_q[~keep].isnan().all())
    y, mag = ref.rotate(x[:, Hq: Hq + H], pos, spec, sections, interleaved)
    yk, yv, at = y[keep], x[:, Hq + H:][keep], slots[keep]
    gk, gv = got[0, at], got[1, at]
    if cache == "e4m3":
        for have, want, err, sc in ((gk, yk, mag[keep] * ref.ROTATE, scales[0]), (gv, yv, yv.abs() * 0, scales[1])):
            want = want / sc
            tol = ref.e4m3_tolerance(want, err / sc)
            assert bool(((ref.stored_values("e4m3", have) - want.clamp(-448, 448)).abs() <= tol).all())
    else:
        tol = ref.rotated_tolerance(yk, mag[keep], dtype)
        assert bool(((gk.double() - yk).abs() <= tol).all())
        assert torch.equal(gv.double(), yv)
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(bits_of(got)[:, rest], bits_of(store.view(2, nb * bs, H, D))[:, rest])
    return got_q, got


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("T,Hq,H,D,style", [
    (1, 4, 2, 64, 0), (5, 28, 4, 128, 0), (33, 8, 8, 64, 1), (3, 1, 1, 16, 0), (2, 6, 2, 32, 1), (4, 5, 1, 256, 0),
    (7, 0, 3, 128, 0), (2, 2, 1, 128, 1), (150, 32, 8, 128, 0)])
def test_append(T, Hq, H, D, style, dtype, cache):
    scales = (0.02, 0.5) if cache == "e4m3" else (1.0, 1.0)
    append_case(T, Hq, H, D, dtype, cache, dict(theta=1e4, style=style), scales=scales, seed=T)


def test_append_widest_head():
    append_case(3, 2, 1, 512, "bf16", "bf16", PLAIN)


@pytest.mark.parametrize("sections,interleaved,style", [
    ([16, 24, 24], False, 0), ([24, 20, 20], True, 0), ([16, 24, 24], False, 1), ([40, 24], False, 0),
    ([32, 32], True, 1), ([64, 0, 0], False, 0), ([0, 0, 64], False, 0), ([64, 0, 0], True, 0)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_axes(sections, interleaved, style, cache):
    append_case(21, 6, 2, 128, "bf16", cache, dict(theta=1e6, style=style), sections, interleaved, scales=(0.1, 0.1)
                if cache == "e4m3" else (1.0, 1.0))


@pytest.mark.parametrize("spec", [PLAIN, LLAMA])
def test_append_far_positions(spec):
    """Positions up to the last one, 2^24 - 1."""
    append_case(40, 4, 2, 128, "f32", "f32", spec, high=1 << 24)
    append_case(40, 4, 2, 128, "bf16", "bf16", spec, [16, 24, 24], high=1 << 24)


def test_append_separate_tensors_odd_blocks_and_padding():
    append_case(50, 8, 2, 64, "bf16", "bf16", LLAMA, bs=7, fused=False, skip=(0, 13, 48, 49))
    append_case(9, 8, 2, 64, "f16", "e4m3", PLAIN, bs=1, scales=(0.3, 3.0), skip=tuple(range(9)))


def test_append_in_place_matches():
    g = torch.Generator().manual_seed(3)
    q, kv = torch.randn(6, 4, 64, generator=g).to(DEV), torch.randn(2, 6, 2, 64, generator=g).to(DEV)
    pos, slots = torch.arange(6, dtype=torch.int32, device=DEV), torch.arange(6, device=DEV)
    cd, outs = api.make_cache_desc(16, 1, "f32"), []
    for place in (False, True):
        mine, lc, status = q.clone(), torch.zeros(2, 1, 16, 2, 64, device=DEV), ints([0])
        out = mine if place else torch.empty_like(q)
        api.is_append(mine, kv[0], kv[1], pos, slots, rope_of(PLAIN), cd, lc, out, status)
        outs.append((out.cpu(), lc.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_append_equal_axes_rotate_as_text():
    """A token whose positions agree on all axes is rotated bit for bit as with one axis."""
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(9, 8, 128, generator=g).to(torch.bfloat16).to(DEV)
    p = torch.randint(0, 5000, (9,), generator=g, dtype=torch.int32).to(DEV)
    got = []
    for axes, pos in ((None, p), (api.make_axes([16, 24, 24]), p.repeat(3, 1)),
                      (api.make_axes([24, 20, 20], True), p.repeat(3, 1))):
        lc, out = torch.zeros(2, 1, 16, 2, 128, dtype=torch.bfloat16, device=DEV), torch.empty_like(qkv[:, :4])
        out = out.contiguous()
        api.is_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, torch.arange(9, device=DEV), rope_of(LLAMA),
                      api.make_cache_desc(16, 1, "bf16"), lc, out, ints([0]), axes=axes)
        got.append((out.cpu(), lc.cpu()))
    for a in got[1:]:
        assert torch.equal(a[0], got[0][0]) and torch.equal(a[1], got[0][1])


def test_append_skips_bad_tokens():
    x = torch.ones(5, 1, 64, device=DEV)
    lc, out, status = torch.full((2, 1, 16, 1, 64), math.nan, device=DEV), torch.full((5, 1, 64), math.nan, device=DEV), ints([0])
    api.is_append(x, x.clone(), x.clone(), ints([0, -1, 1 << 24, 3, 4]), ints([0, 1, 2, 16, -2], torch.int64),
                  rope_of(PLAIN), api.make_cache_desc(16, 1, "f32"), lc, out, status)
    assert status.tolist() == [_lib.IS_ST_POSITION | _lib.IS_ST_BLOCK_ID]
    assert bool(torch.isfinite(out[0]).all()) and bool(out[1:].isnan().all())
    assert bool(torch.isfinite(lc[:, 0, 0]).all()) and bool(lc[:, 0, 1:].isnan().all())


# ---------------------------------------------------------------- is_attend

def attend_case(reqs, Hq, H, D, dtype, cache, bs=16, window=0, scale=None, scales=(1.0, 1.0), seed=0, before=0, behind=0, holes=(),
                use_start=True, max_q=None, spread_q=False, gain=1.0, extra_width=2, run=None):
    """reqs: (seq_len, query rows) of each request; before, behind: rows of no request; holes: (request,
    block index, id) table entries overwritten.  Checks every row."""
    g = torch.Generator().manual_seed(seed)
    td = ref.TORCH[dtype]
    R = len(reqs)
    need = [-(-n // bs) for n, _ in reqs]
    nb = sum(need) + 3
    ids = torch.randperm(nb, generator=g).tolist()
    width = max(max(need), 1) + extra_width
    table = torch.full((R, width), -1, dtype=torch.int32)
    for r, n in enumerate(need):
        for j in range(n):
            table[r, j] = ids.pop()
    k = [gain * torch.randn(n, H, D, generator=g) for n, _ in reqs]
    v = [gain * torch.randn(n, H, D, generator=g) for n, _ in reqs]
    store = nan_cache((2, nb, bs, H, D), cache)
    flat = store.view(2, nb * bs, H, D)
    for r, (n, _) in enumerate(reqs):
        j = torch.arange(n)
        at = table[r].long()[j // bs] * bs + j % bs
        flat[0, at], flat[1, at] = quantise(k[r], cache, scales[0]), quantise(v[r], cache, scales[1])
        k[r] = ref.stored_values(cache, flat[0, at]) * scales[0]
        v[r] = ref.stored_values(cache, flat[1, at]) * scales[1]
    named = [torch.ones(n, dtype=torch.bool) for n, _ in reqs]
    want_bits = 0
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
    lse = torch.full((q.shape[0], Hq), 7.0, device=DEV)
    status = ints([0])
    scale = D ** -0.5 if scale is None else scale
    kw = dict(q_start=ints(starts + [row]) if use_start else None,
              max_q_len=max_q or max(1, max(m for _, m in reqs)), scale=scale, window=window, lse_out=lse)
    args = (qd, ints([n for n, _ in reqs]), table.to(DEV), api.make_cache_desc(bs, nb, cache, *scales), store.to(DEV),
            out, api.attend_workspace(), status)
    if run is None:
        api.is_attend(*args, **kw)
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
        vmax = float(v[r].abs().max()) if n else 0.0
        tol, ltol = ref.attend_tolerance(dtype, cache, D, o, ls, spread, heft, seen, vmax)
        err = (out[rows].double() - o).abs()
        assert bool((err <= tol).all()), (r, float((err / tol.clamp(min=1e-30)).max()))
        none = seen == 0
        assert bool((lse[rows][none] == -math.inf).all()) and bool((out[rows][none] == 0).all())
        lerr = (lse[rows].double() - ls).abs()[~none]
        assert bool((lerr <= ltol[~none]).all()), (r, float((lerr / ltol[~none]).max()))
    assert bool((out[~owned] == 7.0).all()) and bool((lse[~owned] == 7.0).all())


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")]
SCALES = {"e4m3": (0.02, 0.05)}


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (7, 1, 128), (4, 4, 128), (6, 2, 256), (20, 1, 64)])
def test_decode_ragged(Hq, H, D, dtype, cache):
    reqs = [(n, 1) for n in (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300)]
    attend_case(reqs, Hq, H, D, dtype, cache, scales=SCALES.get(cache, (1.0, 1.0)))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_decode_one_long_request_is_split(dtype, cache):
    attend_case([(9001, 1)], 4, 1, 128, dtype, cache, scales=SCALES.get(cache, (1.0, 1.0)))
    attend_case([(3000, 1), (1, 1), (7777, 1)], 8, 2, 64, dtype, cache, scales=SCALES.get(cache, (1.0, 1.0)))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bs", [1, 5, 8, 24, 64, 1000])
def test_decode_block_sizes(bs, dtype, cache):
    attend_case([(n, 1) for n in (1, 5, 49, 200, 333)], 4, 2, 64, dtype, cache, bs=bs, scales=SCALES.get(cache, (1.0, 1.0)))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1 << 30])
def test_windows(window, dtype, cache):
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(1, 1), (16, 1), (17, 1), (130, 1), (500, 1)], 4, 2, 64, dtype, cache, window=window, scales=sc)
    attend_case([(60, 33), (5, 5), (300, 70)], 4, 2, 128, dtype, cache, window=window, scales=sc)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (7, 1, 128), (4, 2, 256)])
def test_few_and_many_rows(Hq, H, D, dtype, cache):
    """Two to a few hundred rows a request, causal; requests without rows; rows behind the last request."""
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(40, 2), (3, 3), (100, 0), (257, 4), (0, 0), (9, 1)], Hq, H, D, dtype, cache, before=2, behind=3, scales=sc)
    attend_case([(140, 129), (64, 64), (200, 1), (77, 31)], Hq, H, D, dtype, cache, behind=5, scales=sc)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,bs,window", [(4, 1, 64, 16, 0), (7, 1, 64, 24, 0), (4, 2, 128, 16, 0), (4, 1, 128, 5, 0),
                                              (2, 1, 256, 16, 0), (4, 1, 64, 8, 700), (4, 1, 128, 128, 900)])
def test_long_prompts(Hq, H, D, bs, window, dtype, cache):
    """Dozens of key tiles a request, so that every ring of the pipeline goes round many times; several items a CTA
    and items cut between CTAs."""
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(3333, 200), (70, 70), (5000, 129), (1999, 1)], Hq, H, D, dtype, cache, bs=bs, window=window, scales=sc)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_rows_that_see_nothing(dtype, cache):
    """More rows than tokens: the first ones stand before position 0.  Empty caches."""
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(3, 5), (0, 4), (0, 1), (2, 1)], 4, 2, 64, dtype, cache, scales=sc)
    attend_case([(10, 90), (0, 70)], 4, 1, 128, dtype, cache, scales=sc)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_unnamed_blocks_are_hidden(dtype, cache):
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(100, 1), (16, 1), (70, 1)], 4, 2, 64, dtype, cache, holes=((0, 2, -1), (1, 0, -5), (2, 4, 1 << 30)), scales=sc)
    attend_case([(100, 40), (16, 16)], 4, 2, 128, dtype, cache, holes=((0, 2, -1), (1, 0, 9999)), scales=sc)


def test_positions_past_the_table_are_hidden():
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(2, 2, 16, 1, 64, generator=g)
    q = torch.randn(1, 1, 64, generator=g)
    out, status, lse = torch.empty(1, 1, 64, device=DEV), ints([0]), torch.empty(1, 1, device=DEV)
    api.is_attend(q.to(DEV), ints([50]), ints([[1, 0]]), api.make_cache_desc(16, 2, "f32"), rows.to(DEV), out,
                  api.attend_workspace(), status, lse_out=lse)
    k, v = (torch.cat([rows[i, 1], rows[i, 0]]).double() for i in (0, 1))
    o, ls, spread, heft, seen = ref.attend(q.double(), 50, k, v, torch.ones(32, dtype=torch.bool), 0.125, 0)
    tol, ltol = ref.attend_tolerance("f32", "f32", 64, o, ls, spread, heft, seen, 9.0)
    assert status.tolist() == [_lib.IS_ST_BLOCK_TABLE]
    assert bool(((out.cpu().double() - o).abs() <= tol).all()) and bool(((lse.cpu().double() - ls).abs() <= ltol).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_large_logits(dtype, cache):
    """Logits of hundreds: the softmax is one key's, the running maximum moves often."""
    attend_case([(333, 1), (90, 40)], 4, 2, 64, dtype, cache, gain=4.0, scale=1.0, scales=SCALES.get(cache, (1.0, 1.0)))
    attend_case([(200, 1)], 4, 2, 128, dtype, cache, scale=-0.1, scales=SCALES.get(cache, (1.0, 1.0)))
    attend_case([(200, 1)], 4, 2, 128, dtype, cache, scale=0.0, scales=SCALES.get(cache, (1.0, 1.0)))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bs", [16, 24])
def test_nan_before_the_window(bs, dtype, cache):
    """Positions before the window of every row hold NaN: single tokens and a prompt."""
    g = torch.Generator().manual_seed(11)
    H, Hq, D, n, sc = 2, 8, 64, 700, SCALES.get(cache, (1.0, 1.0))
    nb = -(-n // bs)
    for rows, window in ((1, 90), (20, 250)):
        store = nan_cache((2, nb, bs, H, D), cache)
        flat = store.view(2, nb * bs, H, D)
        see = slice(n - rows - window + 1, n)
        x = [torch.zeros(n, H, D, dtype=torch.float64) for _ in range(2)]
        for i in range(2):
            flat[i, see] = quantise(torch.randn(rows + window - 1, H, D, generator=g), cache, sc[i])
            x[i][see] = ref.stored_values(cache, flat[i, see]) * sc[i]
        q = torch.randn(rows, Hq, D, generator=g).to(ref.TORCH[dtype])
        out, lse, status = torch.empty_like(q, device=DEV), torch.empty(rows, Hq, device=DEV), ints([0])
        api.is_attend(q.to(DEV), ints([n]), ints([list(range(nb))]), api.make_cache_desc(bs, nb, cache, *sc), store.to(DEV), out,
                      api.attend_workspace(), status, q_start=ints([0, rows]), max_q_len=rows, window=window, lse_out=lse)
        o, ls, spread, heft, seen = ref.attend(q.double(), n, *x, torch.ones(n, dtype=torch.bool), D ** -0.5, window)
        tol, ltol = ref.attend_tolerance(dtype, cache, D, o, ls, spread, heft, seen, float(x[1].abs().max()))
        assert bool(((out.cpu().double() - o).abs() <= tol).all()) and bool(((lse.cpu().double() - ls).abs() <= ltol).all())
        assert status.tolist() == [0]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H", [(64, 1), (100, 1), (33, 3)])
def test_wide_groups(Hq, H, dtype, cache):
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(200, 1), (33, 3), (150, 9)], Hq, H, 64, dtype, cache, scales=sc)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-40, 1e-30])
def test_odd_scales(scale, dtype, cache):
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(200, 60), (130, 1)], 4, 2, 64, dtype, cache, scales=sc, scale=scale)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_single_tokens_under_a_large_bound(dtype, cache):
    """max_q_len far above the rows there are."""
    sc = SCALES.get(cache, (1.0, 1.0))
    attend_case([(n, 1) for n in (1, 16, 17, 127, 128, 129, 400, 2000, 3, 0, 77, 256, 600)], 4, 1, 128, dtype, cache, scales=sc,
                max_q=1000)
    attend_case([(900, 1)] * 20, 8, 2, 64, dtype, cache, scales=sc, max_q=64, use_start=True, window=100)


@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rows_of_any_magnitude(rows, cache):
    """bf16 query rows from 1e-35 to 1e30, and zeros: an FP8 cache's products are taken in fp16, on scaled rows."""
    g = torch.Generator().manual_seed(12)
    H, Hq, D, n, bs, sc = 1, 4, 64, 300, 16, SCALES.get(cache, (1.0, 1.0))
    nb = -(-n // bs)
    store = nan_cache((2, nb, bs, H, D), cache)
    flat, x = store.view(2, nb * bs, H, D), []
    for i in range(2):
        flat[i, :n] = quantise(torch.randn(n, H, D, generator=g), cache, sc[i])
        x.append(ref.stored_values(cache, flat[i, :n]) * sc[i])
    size = torch.tensor([1e-35, 1e-3, 0.0, 1e30])
    for scale in (1e-30, 1.0):
        q = (torch.randn(rows, Hq, D, generator=g) * size[:, None]).to(torch.bfloat16)
        out, lse, status = torch.empty_like(q, device=DEV), torch.empty(rows, Hq, device=DEV), ints([0])
        api.is_attend(q.to(DEV), ints([n]), ints([list(range(nb))]), api.make_cache_desc(bs, nb, cache, *sc), store.to(DEV), out,
                      api.attend_workspace(), status, q_start=ints([0, rows]), max_q_len=rows, scale=scale, lse_out=lse)
        use = slice(0, 4 if scale < 1 else 3)         # 1e30 at scale 1: one key takes all, ties of 2^100 apart decided in fp32
        o, ls, spread, heft, seen = ref.attend(q.double(), n, *x, torch.ones(n, dtype=torch.bool), scale, 0)
        tol, ltol = ref.attend_tolerance("bf16", cache, D, o, ls, spread, heft, seen, float(x[1].abs().max()))
        assert bool(((out.cpu().double() - o).abs() <= tol)[:, use].all())
        assert bool(((lse.cpu().double() - ls).abs() <= ltol)[:, use].all()) and status.tolist() == [0]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_prompts_of_different_magnitudes(D, dtype):
    """Items of one or two key tiles behind one another in a CTA, over an FP8 cache, each request's query rows of
    a magnitude of their own."""
    g = torch.Generator().manual_seed(5)
    R, H, Hq, bs, m, n, sc = 1200, 1, 4, 16, 20, 128, SCALES["e4m3"]
    nb = R * (n // bs)
    store = nan_cache((2, nb, bs, H, D), "e4m3")
    flat = store.view(2, nb * bs, H, D)
    x = []
    for i in range(2):
        flat[i] = quantise(torch.randn(nb * bs, H, D, generator=g), "e4m3", sc[i])
        x.append(ref.stored_values("e4m3", flat[i]) * sc[i])
    table = torch.arange(nb, dtype=torch.int32).reshape(R, n // bs)
    size = 2.0 ** ((torch.arange(R) * 5) % 8 - 7).double()          # 2^-7 .. 1
    q = (torch.randn(R * m, Hq, D, generator=g) * size.repeat_interleave(m)[:, None, None]).to(ref.TORCH[dtype])
    out, lse, status = torch.empty_like(q, device=DEV), torch.empty(R * m, Hq, device=DEV), ints([0])
    api.is_attend(q.to(DEV), ints([n] * R), table.to(DEV), api.make_cache_desc(bs, nb, "e4m3", *sc), store.to(DEV), out,
                  api.attend_workspace(), status, q_start=ints([m * r for r in range(R + 1)]), max_q_len=m, scale=D ** -0.5,
                  lse_out=lse)
    assert status.tolist() == [0]
    out, lse = out.cpu().double(), lse.cpu().double()
    for r in range(R):
        rows, keys = slice(m * r, m * r + m), slice(n * r, n * r + n)
        k, v = x[0][keys], x[1][keys]
        o, ls, spread, heft, seen = ref.attend(q[rows].double(), n, k, v, torch.ones(n, dtype=torch.bool), D ** -0.5, 0)
        tol, ltol = ref.attend_tolerance(dtype, "e4m3", D, o, ls, spread, heft, seen, float(v.abs().max()))
        assert bool(((out[rows] - o).abs() <= tol).all()), r
        assert bool(((lse[rows] - ls).abs() <= ltol).all()), r


def test_thousands_of_requests():
    attend_case([(1 + (53 * r) % 40, (r * 7) % 3) for r in range(2500)], 2, 1, 64, "bf16", "bf16")
    attend_case([(1 + (53 * r) % 40, (r * 7) % 19) for r in range(600)], 4, 1, 64, "f16", "f16")


def test_many_requests_without_q_start_and_strided_q():
    attend_case([(1 + (37 * r) % 90, 1) for r in range(300)], 4, 2, 64, "bf16", "bf16", use_start=False)
    attend_case([(50, 3), (20, 20)], 4, 2, 64, "bf16", "bf16", spread_q=True)
    attend_case([(150, 1)] * 3, 28, 4, 128, "f16", "f16", spread_q=True, use_start=False)


def test_bad_requests_are_left_out():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(6, 2, 64, generator=g).to(DEV)
    lc = torch.randn(2, 4, 16, 1, 64, generator=g).to(DEV)
    out, status = torch.full((6, 2, 64), 7.0, device=DEV), ints([0])
    table = ints([[0, 1], [2, 3], [0, 1], [1, 2]])
    #          good    4 rows of 3 allowed   negative length   rows past T
    api.is_attend(q, ints([5, 9, -1, 8]), table, api.make_cache_desc(16, 4, "f32"), lc, out, api.attend_workspace(),
                  status, q_start=ints([0, 1, 5, 5, 9]), max_q_len=3)
    assert status.tolist() == [_lib.IS_ST_COUNT]
    assert bool((out[1:] == 7.0).all()) and bool((out[0] != 7.0).all())


def test_cache_past_32_bits():
    """A layer cache of 4.5 GB whose used blocks lie at its end: byte offsets pass 2^32, elements 2^31."""
    H, D, bs, nb = 8, 128, 16, 70000
    lc = torch.empty((2, nb, bs, H, D), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    n, used = 40, [nb - 1, 3, nb - 2]
    small = torch.empty((2, 3, bs, H, D), dtype=torch.bfloat16, device=DEV)
    qkv = torch.randn((n, 32 + 2 * H, D), generator=g, device=DEV).to(torch.bfloat16)
    outs = []
    for cache, ids in ((lc, used), (small, [0, 1, 2])):
        t = torch.arange(n, device=DEV)
        slots = ints(ids, torch.int64)[t // bs] * bs + t % bs
        q, status = torch.empty((n, 32, D), dtype=torch.bfloat16, device=DEV), ints([0])
        cd = api.make_cache_desc(bs, cache.shape[1], "bf16")
        api.is_append(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], t.to(torch.int32), slots, rope_of(LLAMA), cd, cache, q, status)
        for rows in (1, n):
            out = torch.empty((rows, 32, D), dtype=torch.bfloat16, device=DEV)
            api.is_attend(q[n - rows:], ints([n]), ints([ids]), cd, cache, out, api.attend_workspace(), status,
                          q_start=ints([0, rows]), max_q_len=rows)
            outs.append(out.cpu())
        assert status.tolist() == [0]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    del lc


@pytest.mark.parametrize("rows", [1, 3, 80])
def test_same_call_gives_the_same_bits(rows):
    got = []

    def run(args, kw):
        for _ in range(3):
            args[5].fill_(7.0)
            args[6].fill_(0xFF)              # what the workspace holds means nothing
            api.is_attend(*args, **kw)
            got.append(args[5].clone())
    attend_case([(4000, rows), (100, min(rows, 100)), (2500, rows)], 8, 2, 128, "bf16", "bf16", run=run)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("rows", [1, 60])
def test_graphs_and_streams(rows):
    """Two captured graphs with a workspace each replay on two streams at once; replays read the buffers' new
    contents."""
    H, Hq, D, bs, nb = 2, 8, 128, 16, 200
    g = torch.Generator(device=DEV).manual_seed(6)
    sets = []
    for i in range(2):
        n = 1400 + 300 * i
        cache = torch.randn((2, nb, bs, H, D), generator=g, device=DEV).to(torch.bfloat16)
        q = torch.randn((rows, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
        t = dict(q=q, seq=ints([n]), table=torch.randperm(nb, generator=g, device=DEV)[:120].to(torch.int32)[None].contiguous(),
                 cache=cache, out=torch.zeros_like(q), ws=api.attend_workspace(), status=ints([0]), start=ints([0, rows]))
        sets.append(t)
    cd = api.make_cache_desc(bs, nb, "bf16")

    def call(t, out):
        api.is_attend(t["q"], t["seq"], t["table"], cd, t["cache"], out, t["ws"], t["status"], q_start=t["start"],
                      max_q_len=rows)
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for t, s in zip(sets, streams):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                call(t, t["out"])
        graphs.append(graph)
    for turn in range(2):
        for t in sets:
            if turn:
                t["q"].normal_(generator=g)
                t["seq"].sub_(777)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        for t in sets:
            want = torch.zeros_like(t["out"])
            call(t, want)
            torch.cuda.synchronize()
            assert torch.equal(want, t["out"]) and bool(want.any()) and t["status"].tolist() == [0]


# ---------------------------------------------------------------- all of them behind an injection

@pytest.mark.parametrize("cache_dtype", ["bf16", "e4m3"])
def test_step_behind_an_injected_segment(cache_dtype):
    """Blocks for three requests' segments and prompts, injection of their facts, the prompts' K/V, attention from
    the prompts, then two single-token steps: against one fp64 attention over all tokens' keys and values."""
    L, H, D, Hq, bs = 2, 4, 64, 8, 16
    g = torch.Generator().manual_seed(8)
    lens = [7, 19, 30, 4, 11]
    cfg = api.make_config(num_layers=L, num_kv_heads=H, head_dim=D, emb_dim=64, kv_dtype="bf16", emb_dtype="f16",
                          max_facts=8, max_tokens=100, max_users=1, max_queries=4, max_k=4)
    sc = (0.05, 0.02) if cache_dtype == "e4m3" else (1.0, 1.0)
    with api.is_store_create(cfg, 0) as store:
        fk, fv = (torch.randn(sum(lens), L, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
        api.is_store_add_facts(store, 0, lens, fk.to(DEV), fv.to(DEV), torch.randn(5, 64, generator=g).half().to(DEV))
        facts, head0, prompt = [[2, 0], [4, 1], [3]], [5, 0, 2], [9, 1, 40]
        segs = [sum(lens[f] for f in fs) for fs in facts]
        R, W, nb = 3, 8, 40
        table, free = torch.full((R, W), -1, dtype=torch.int32, device=DEV), torch.randperm(nb, generator=g).to(torch.int32).to(DEV)
        status, cache = ints([0]), nan_cache((L, 2, nb, bs, H, D), cache_dtype).to(DEV)
        cd = api.make_cache_desc(bs, nb, cache_dtype, *sc)
        spec = LLAMA
        base = fk.double(), fv.double()
        off = np.concatenate([[0], np.cumsum(lens)])
        keys = [[] for _ in range(R)]                 # (pre-rotation K, V [.][L][H][D]) in order
        for r in range(R):
            keys[r].append(tuple(torch.randn(head0[r], L, H, D, generator=g).to(torch.bfloat16).double() for _ in range(2)))
            for f in facts[r]:
                keys[r].append(tuple(b[off[f]: off[f + 1]] for b in base))
        seq, head = ints([0, 0, 0]), ints([0])

        def extend(new):
            nonlocal seq, head
            T = sum(new)
            slots, pos, start = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV), ints([0] * (R + 1))
            seq2, head2 = torch.empty_like(seq), torch.empty_like(head)
            api.is_extend_block_table(seq, ints(new), free, bs, nb, table, slots, pos, start, seq2, status, free_head=head,
                                      free_head_out=head2)
            seq, head = seq2, head2
            return slots, pos, start

        def step(new, x):
            """x: per request (q, k, v) rows; appends and attends, returns the checked outputs."""
            slots, pos, start = extend(new)
            q, k, v = (torch.cat([y[i] for y in x]).to(DEV) for i in range(3))
            for layer in range(L):
                qr = torch.empty_like(q[:, layer]).contiguous()
                api.is_append(q[:, layer], k[:, layer], v[:, layer], pos, slots, rope_of(spec), cd, cache[layer], qr, status)
                if not Hq:
                    continue
                out = torch.empty_like(qr)
                api.is_attend(qr, seq, table, cd, cache[layer], out, api.attend_workspace(), status, q_start=start,
                              max_q_len=max(new))
                yield layer, out.cpu(), start.cpu().tolist()

        def rows(n):
            return [torch.randn(n, L, h, D, generator=g).to(torch.bfloat16) for h in (Hq, H, H)]

        first = [rows(n) for n in head0]              # the system prefix
        for r in range(R):
            keys[r][0] = (first[r][1].double(), first[r][2].double())
        list(step(head0, first))
        before = seq.clone()
        extend(segs)
        fact_ids = ints([f + [-1] * (2 - len(f)) for f in facts], torch.int64)
        got_len = ints([0] * R)
        api.is_inject(store, fact_ids, ints([len(f) for f in facts]), before, rope_of(spec), table, cd, cache,
                      seg_len_out=got_len)
        assert api.is_get_status(store) == 0 and got_len.tolist() == segs
        for new in (prompt, [1, 1, 1], [1, 0, 1]):
            x = [rows(n) for n in new]
            for r in range(R):
                keys[r].append((x[r][1].double(), x[r][2].double()))
            for layer, out, start in step(new, x):
                for r in range(R):
                    if new[r] == 0:
                        continue
                    k = torch.cat([a[0] for a in keys[r]])[:, layer]
                    v = torch.cat([a[1] for a in keys[r]])[:, layer]
                    n = k.shape[0]
                    kr, kmag = ref.rotate(k, torch.arange(n)[None], spec)
                    qr, qmag = ref.rotate(x[r][0][:, layer].double(), torch.arange(n - new[r], n)[None], spec)
                    named = torch.ones(n, dtype=torch.bool)
                    o, ls, spread, heft, seen = ref.attend(qr, n, kr, v, named, D ** -0.5, 0)
                    # stored keys, values and rotated queries are rounded: each logit moves by at most the relative
                    # steps of q and k times sum |q k|, each value by its own step
                    step_k = (2.0 ** -4 if cache_dtype == "e4m3" else ref.U["bf16"]) * 1.01
                    step_v = 2.0 ** -4 * 1.01 if cache_dtype == "e4m3" else 0.0
                    drift = heft * (step_k + ref.U["bf16"] * 1.01) + 2.0 ** -10
                    if cache_dtype == "e4m3":         # subnormal steps of the stored key: 2^-10 each, times scale and |q|
                        drift = drift + qr.abs().sum(-1) * 2.0 ** -10 * sc[0] * D ** -0.5
                    tol, _ = ref.attend_tolerance("bf16", cache_dtype, D, o, ls, spread, heft, seen, float(v.abs().max()))
                    tol = tol + (torch.expm1(2 * drift) + step_v)[..., None] * (spread + o.abs()) + 2.0 ** -10 * sc[1]
                    err = (out[start[r]: start[r + 1]].double() - o).abs()
                    assert bool((err <= tol).all()), (layer, r, float((err / tol).max()))
        assert status.tolist() == [0]
