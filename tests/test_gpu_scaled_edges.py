"""The scaled cache at its edges on the GPU: factors past the smallest number, tokens left out inside a block, waits that
run out."""
import math

import pytest
import torch

from kv_cache_injection_gb300 import _lib, api
from tests import gpu_helpers as gh
from tests import scaled_reference as sref
from tests import serve_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def built():
    gh.ensure_built()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


# ---------------------------------------------------------------- keys of the smallest scale

@pytest.mark.parametrize("rows", [1, 8, 9, 40, 90])
@pytest.mark.parametrize("dtype,cache,D,bs,window,scale,gain", [
    ("bf16", "int8", 64, 16, 0, 1e-30, 1.0), ("bf16", "e4m3", 128, 8, 0, 1e-30, 1.0), ("bf16", "e4m3", 64, 16, 20, 1e-36, 1.0),
    ("f16", "int8", 128, 16, 0, 1e-36, 1.0), ("f16", "e4m3", 64, 24, 33, 1e-38, 1.0), ("bf16", "int8", 128, 16, 0, None, 1e-30),
    ("bf16", "e4m3", 64, 40, 50, None, 1e-37), ("bf16", "int8", 256, 16, 0, 1e-30, 1.0), ("bf16", "int8", 64, 16, 0, 1.0, 1.0)])
def test_zero_keys_under_the_smallest_factor(dtype, cache, D, bs, window, scale, gain, rows):
    """Blocks of zero keys have the smallest K scale; with a small scale, or queries that are small, its product with the
    row's factor lies below the smallest number.  What is hidden stays hidden, and all that is seen weighs the same."""
    g = torch.Generator().manual_seed(31)
    H, Hq, lens = 2, 8, [300, 97, 131]
    ms = [min(rows, n) for n in lens]
    need = [-(-n // bs) for n in lens]
    nb = sum(need)
    ids = torch.randperm(nb, generator=g).to(torch.int32)
    table, at = torch.full((3, max(need)), -1, dtype=torch.int32), 0
    for r, k in enumerate(need):
        table[r, :k] = ids[at: at + k]
        at += k
    x = torch.randn(2, nb, bs, H, D, generator=g).double()
    x[0, torch.rand(nb, generator=g) < 0.5] = 0.0
    x[0, table[0, 0]] = 0.0                              # the first blocks, and the last ones, which the causal mask cuts
    x[0, table[0, need[0] - 1]] = 0.0
    x[0, table[2, need[2] - 1]] = 0.0
    codes, scales = sref.quantised(cache, x)
    assert float(scales[0].min()) == sref.SMALLEST
    q = (gain * torch.randn(sum(ms), Hq, D, generator=g)).to(ref.TORCH[dtype])
    starts = [0]
    for m in ms:
        starts.append(starts[-1] + m)
    out, lse, status = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(q.shape[:2], device=DEV), ints([0])
    scale = D ** -0.5 if scale is None else scale
    api.is_attend_scaled(q.to(DEV), ints(lens), table.to(DEV), api.make_cache_desc(bs, nb, cache), codes.to(DEV), scales.to(DEV), out,
                         api.attend_workspace(), status, q_start=ints(starts), max_q_len=max(ms), scale=scale, window=window, lse_out=lse)
    assert status.tolist() == [0]
    for r, n in enumerate(lens):
        rng = slice(starts[r], starts[r + 1])
        j = torch.arange(n)
        b = table[r].long()[j // bs]
        k, v = (sref.numbers(cache, codes[kv, b, j % bs]) * scales[kv, b].double()[..., None] for kv in range(2))
        o, ls, spread, heft, seen = ref.attend(q[rng].double(), n, k, v, torch.ones(n, dtype=torch.bool), scale, window)
        tol, ltol = sref.attend_tolerance(dtype, D, o, ls, spread, heft, seen, scales[1, b], sref.QMAX[cache])
        assert bool(((out[rng].cpu().double() - o).abs() <= tol).all()) and bool(((lse[rng].cpu().double() - ls).abs() <= ltol).all())


# ---------------------------------------------------------------- tokens left out inside a block

def with_holes(n, holes, pad, g):
    """Where n tokens come to lie when holes[i] skipped ones follow token i, and the length with `pad` in front."""
    at, t = [], pad
    for i in range(n):
        at.append(t)
        t += 1 + holes.get(i, 0)
    return torch.tensor(at), t


def cache_of(cache, nb, bs, H, D, g):
    codes, scales = sref.quantised(cache, torch.randn(2, nb, bs, H, D, generator=g).double() * 0.5)
    return codes.to(DEV), scales.to(DEV)


HOLES = [{2: 1}, {0: 29}, {0: 30}, {0: 31}, {5: 32}, {3: 95}, {3: 127}, {3: 128}, {3: 129}, {7: 700}, {i: 1 for i in range(60)},
         {i: (i * 7) % 5 for i in range(60)}, {i: 40 for i in range(0, 60, 3)}, {59: 300}, {10: 3, 11: 33, 12: 130, 40: 600}]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("bs", [1, 7, 16, 64, 1000])
@pytest.mark.parametrize("pad", [0, 1, 40, 500])
def test_skipped_tokens_between_those_of_a_block(cache, bs, pad):
    """However many tokens without a slot, or with a slot outside the cache, lie between a block's tokens, the call writes
    what it writes without them."""
    g = torch.Generator().manual_seed(bs + pad)
    H, Hq, D, n, nb = 3, 4, 64, 61, 64 if bs < 64 else 3
    order = torch.randperm(nb, generator=g)
    first = 3 if bs > 3 else 0                           # the first block holds rows already
    p = first + torch.arange(n)
    slots = order[p // bs] * bs + p % bs
    x = (3 * torch.randn(n, Hq + 2 * H, D, generator=g)).to(torch.bfloat16).to(DEV)
    rope, cd = api.make_rope(1e4), api.make_cache_desc(bs, nb, cache)
    source = torch.randn(2, 8, 16, H, D, generator=g).to(torch.bfloat16).to(DEV)
    from_slots = torch.randperm(128, generator=g)[:n].to(DEV)
    c0, s0 = cache_of(cache, nb, bs, H, D, g)

    def append(at, T, bad):
        codes, scales, status = c0.clone(), s0.clone(), ints([0])
        rows = torch.full((T, Hq + 2 * H, D), math.nan, dtype=torch.bfloat16, device=DEV)
        where = torch.full((T,), bad, dtype=torch.int64)
        pos = torch.full((T,), -7, dtype=torch.int32)    # what is skipped may have any position
        rows[at.to(DEV)], where[at], pos[at] = x, slots, p.to(torch.int32)
        q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        api.is_append_scaled(rows[:, :Hq], rows[:, Hq: Hq + H], rows[:, Hq + H:], pos.to(DEV), where.to(DEV), rope, cd, codes, scales,
                             q, status)
        return codes, scales, q[at.to(DEV)], status

    def move(at, T, bad):
        codes, scales, status = c0.clone(), s0.clone(), ints([0])
        where, source_at = torch.full((T,), bad, dtype=torch.int64), torch.full((T,), 5, dtype=torch.int64, device=DEV)
        where[at], source_at[at.to(DEV)] = slots, from_slots
        api.is_move_scaled(api.make_cache_desc(16, 8, "bf16"), source, source_at, cd, codes, scales, where.to(DEV), status)
        return codes, scales, status

    for call in (append, move):
        want = call(torch.arange(n), n, -1)
        assert want[-1].tolist() == [0] and not torch.equal(want[1], s0)
        for holes in HOLES:
            at, T = with_holes(n, holes, pad, g)
            for bad, bits in ((-1, 0), (nb * bs, _lib.IS_ST_BLOCK_ID), (-2, _lib.IS_ST_BLOCK_ID)):
                got = call(at, T, bad)
                assert got[-1].tolist() == [bits if T > n else 0]
                assert all(torch.equal(a, b) for a, b in zip(got[:-1], want[:-1])), (call.__name__, holes, bad)


@pytest.mark.parametrize("T,window", [(5000, 0), (9000, 64), (700, 7)])
def test_skipped_tokens_in_long_batches(T, window):
    """Many requests' tokens with random ones left out, several tokens a CTA."""
    g = torch.Generator().manual_seed(T)
    H, D, bs, nb = 4, 128, 16, T // 16 + 1
    slots = torch.randperm(nb, generator=g).repeat_interleave(bs)[:T] * bs + torch.arange(T) % bs
    keep = torch.rand(T, generator=g) < 0.6
    if window:
        keep &= (torch.arange(T) // window) % 3 != 1     # whole stretches too
    source = torch.randn(2, nb, bs, H, D, generator=g).to(torch.bfloat16).to(DEV)
    c0, s0 = cache_of("int8", nb, bs, H, D, g)
    cd, fd, got = api.make_cache_desc(bs, nb, "int8"), api.make_cache_desc(bs, nb, "bf16"), []
    for at, from_slots in ((torch.where(keep, slots, -1), torch.arange(T)), (slots[keep], torch.arange(T)[keep])):
        codes, scales, status = c0.clone(), s0.clone(), ints([0])
        api.is_move_scaled(fd, source, from_slots.to(DEV), cd, codes, scales, at.to(DEV), status)
        assert status.tolist() == [0]
        got.append((codes, scales))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("bad,bits", [(-1, 0), (64, _lib.IS_ST_BLOCK_ID), (-3, _lib.IS_ST_BLOCK_ID)])
def test_moved_tokens_without_a_source_count_for_nothing(cache, bad, bits):
    """A row whose token has no source is none of the call's rows: below the others it is held, and keeps its value when the
    scale grows; as a block's row 0 it does not make the block a fresh one."""
    g = torch.Generator().manual_seed(17)
    H, D, bs, nb = 2, 64, 16, 4
    source = (4 * torch.randn(2, 4, 16, H, D, generator=g)).to(torch.bfloat16).to(DEV)
    c0, s0 = cache_of(cache, nb, bs, H, D, g)
    cd, fd = api.make_cache_desc(bs, nb, cache), api.make_cache_desc(16, 4, "bf16")

    def move(slots, from_slots, s=s0):
        codes, scales, status = c0.clone(), s.clone(), ints([0])
        api.is_move_scaled(fd, source, ints(from_slots, torch.int64), cd, codes, scales, ints(slots, torch.int64), status)
        return codes, scales, status.item()

    for slots, from_slots in (([5, 6], [bad, 9]), ([0, 1], [bad, 9]), ([0, 1, 2, 3], [bad, bad, bad, 9]), ([7, 6, 8], [9, bad, 3]),
                              ([16 + 15, 33, 32, 34], [4, 5, bad, 7]), ([3] * 40 + [4], [bad] * 40 + [1]), ([0, 16, 32], [bad] * 3)):
        live = [i for i, f in enumerate(from_slots) if f != bad]
        got = move(slots, from_slots)
        want = move([slots[i] for i in live], [from_slots[i] for i in live])
        assert got[2] == bits and want[2] == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    codes, scales, _ = move([5, 6], [bad, 9])            # row 5 was held: half a step of the new scale off at most
    assert bool((scales[:, 0] > s0[:, 0]).all())
    was, now = (sref.numbers(cache, c[:, 0, 5].cpu()) * s[:, 0, :, None].cpu().double() for c, s in ((c0, s0), (codes, scales)))
    half = {"int8": 0.5, "e4m3": 16.0}[cache]
    assert bool(((was - now).abs() <= half * (1 + 2.0 ** -10) * scales[:, 0, :, None].cpu().double()).all())
    none = s0.clone()
    none[:, 0] = math.nan                                # row 0 is not written, so the block is not fresh: its scale is missed
    codes, scales, status = move([0, 1], [bad, 9], none)
    assert status == bits | _lib.IS_ST_SCALE and torch.equal(codes, c0)


def test_random_moves_without_some_sources():
    g = torch.Generator().manual_seed(18)
    for T, H, D, bs in ((300, 2, 64, 16), (2000, 3, 128, 7), (6000, 4, 64, 64)):
        nb = -(-T // bs) + 1
        slots = torch.randperm(nb, generator=g).repeat_interleave(bs)[:T] * bs + torch.arange(T) % bs
        keep = torch.rand(T, generator=g) < 0.7
        source = torch.randn(2, nb, bs, H, D, generator=g).to(torch.bfloat16).to(DEV)
        c0, s0 = cache_of("int8", nb, bs, H, D, g)
        cd, fd, got = api.make_cache_desc(bs, nb, "int8"), api.make_cache_desc(bs, nb, "bf16"), []
        for at, from_slots in ((slots, torch.where(keep, torch.arange(T), -1)), (slots[keep], torch.arange(T)[keep])):
            codes, scales, status = c0.clone(), s0.clone(), ints([0])
            api.is_move_scaled(fd, source, from_slots.to(DEV), cd, codes, scales, at.to(DEV), status)
            assert status.tolist() == [0]
            got.append((codes, scales))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("dtype,cache,H,D,bs,T", [("bf16", "int8", 8, 128, 16, 3000), ("f16", "e4m3", 3, 64, 32, 900),
                                                  ("f32", "int8", 2, 256, 8, 400), ("bf16", "e4m3", 4, 128, 16, 40)])
def test_writes_whose_waits_run_out(dtype, cache, H, D, bs, T):
    """With limits that it cannot keep a write ends with IS_ST_TIMEOUT: each head of a block is as it was or as the whole
    call writes it, and writing the same tokens again gives what one call gives."""
    g = torch.Generator().manual_seed(23)
    nb = -(-(T + 5) // bs) + 2
    order = torch.randperm(nb, generator=g)
    p = 5 + torch.arange(T)                              # the first block holds rows already
    slots = (order[p // bs] * bs + p % bs).to(DEV)
    c0, s0 = cache_of(cache, nb, bs, H, D, g)
    cd, fd, td = api.make_cache_desc(bs, nb, cache), api.make_cache_desc(16, nb * bs // 16 + 1, dtype), ref.TORCH[dtype]
    x = (2 * torch.randn(T, 2 * H, D, generator=g)).to(td).to(DEV)
    source = torch.randn(2, nb * bs // 16 + 1, 16, H, D, generator=g).to(td).to(DEV)
    from_slots = torch.randperm(nb * bs, generator=g)[:T].to(DEV)

    def append(codes, scales, status, **kw):
        api.is_append_scaled(None, x[:, :H], x[:, H:], p.to(torch.int32).to(DEV), slots, api.make_rope(1e4), cd, codes, scales, None,
                             status, **kw)

    def move(codes, scales, status, **kw):
        api.is_move_scaled(fd, source, from_slots, cd, codes, scales, slots, status, **kw)

    def of_heads(codes, scales):                         # a row of numbers for each K or V, block and head
        return torch.cat([codes.transpose(2, 3).reshape(2, nb, H, -1).to(torch.int64), scales.view(torch.int32)[..., None].long()], -1)

    for call in (append, move):
        status, seen = ints([0]), 0
        want_codes, want_scales = c0.clone(), s0.clone()
        call(want_codes, want_scales, status)
        assert status.item() == 0
        before, want = of_heads(c0, s0), of_heads(want_codes, want_scales)
        for budget in (0, 0, 300, 600, 1000, 2000, 5000, 0):
            codes, scales = c0.clone(), s0.clone()
            torch.cuda.synchronize()
            call(codes, scales, status, budget_ns=budget)
            bits = status.item()
            seen |= bits
            got = of_heads(codes, scales)
            written = (got == want).all(-1)
            assert bits in (0, _lib.IS_ST_TIMEOUT) and bool((written | (got == before).all(-1)).all())
            assert bits or bool(written.all())
            status.zero_()
            call(codes, scales, status)
            assert status.item() == 0 and torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
        assert seen == _lib.IS_ST_TIMEOUT or call is append   # whose rows may land while its sines are computed


def test_waits_of_a_long_group_that_run_out():
    """A block that gets more rows than fit a round, whose tokens come twice: left half-way, it is as it should be after the
    same call again."""
    g = torch.Generator().manual_seed(24)
    H, D, bs, T = 2, 128, 1024, 900
    c0, s0 = cache_of("int8", 2, bs, H, D, g)
    source = (3 * torch.randn(2, 64, 16, H, D, generator=g)).to(torch.bfloat16).to(DEV)
    args = api.make_cache_desc(16, 64, "bf16"), source, torch.randperm(1024, generator=g)[:T].to(DEV), api.make_cache_desc(bs, 2, "int8")
    slots, status = (bs + 40 + torch.arange(T)).to(DEV), ints([0])
    want_codes, want_scales = c0.clone(), s0.clone()
    api.is_move_scaled(*args, want_codes, want_scales, slots, status)
    assert status.item() == 0
    for budget in (0, 500, 700, 900, 1200, 1500, 2000, 3000):
        codes, scales = c0.clone(), s0.clone()
        api.is_move_scaled(*args, codes, scales, slots, status, budget_ns=budget)
        assert status.item() in (0, _lib.IS_ST_TIMEOUT)
        status.zero_()
        api.is_move_scaled(*args, codes, scales, slots, status)
        assert status.item() == 0 and torch.equal(codes, want_codes) and torch.equal(scales, want_scales)


# ---------------------------------------------------------------- far holes, graphs and streams

@pytest.mark.parametrize("gap", [1023, 1024, 1025, 2047, 2048, 2049, 6000])
def test_holes_further_off_than_a_look(gap):
    """More skipped tokens than a CTA looks at in one go: between a block's tokens, before the first and behind the last."""
    g = torch.Generator().manual_seed(gap)
    H, D, bs, nb = 2, 64, 16, 6
    slots = torch.tensor([35, 36, 37, 40, 64, 65, 80, 8, 9])         # blocks 2 (from row 3), 4, 5 and 0
    source = torch.randn(2, 2, 16, H, D, generator=g).to(torch.bfloat16).to(DEV)
    c0, s0 = cache_of("int8", nb, bs, H, D, g)
    cd, fd, n = api.make_cache_desc(bs, nb, "int8"), api.make_cache_desc(16, 2, "bf16"), len(slots)

    def move(at, T):
        codes, scales, status = c0.clone(), s0.clone(), ints([0])
        where = torch.full((T,), -1, dtype=torch.int64)
        from_slots = torch.full((T,), 3, dtype=torch.int64)
        where[at], from_slots[at] = slots, torch.arange(n) + 5
        api.is_move_scaled(fd, source, from_slots.to(DEV), cd, codes, scales, where.to(DEV), status)
        assert status.tolist() == [0]
        return codes, scales

    want = move(torch.arange(n), n)
    for holes, pad, behind in (({1: gap}, 0, 0), ({3: gap, 4: gap}, 7, gap), ({0: gap, 1: gap, 7: 40}, gap, 1), ({}, gap, gap)):
        at, T = with_holes(n, holes, pad, g)
        assert all(torch.equal(a, b) for a, b in zip(move(at, T + behind), want))


def test_writes_with_holes_in_graphs_on_two_streams():
    """Captured writes, one a stream, whose buffers' slots change between replays: skipped tokens come and go."""
    g = torch.Generator().manual_seed(41)
    H, Hq, D, bs, nb, T = 2, 4, 64, 16, 24, 300
    rope, cd, fd = api.make_rope(1e4), api.make_cache_desc(bs, nb, "e4m3"), api.make_cache_desc(16, 20, "bf16")
    order = torch.randperm(nb, generator=g)
    slots = order[torch.arange(T) // bs] * bs + torch.arange(T) % bs
    c0, s0 = cache_of("e4m3", nb, bs, H, D, g)
    x = torch.randn(T, Hq + 2 * H, D, generator=g).to(torch.bfloat16).to(DEV)
    source = torch.randn(2, 20, 16, H, D, generator=g).to(torch.bfloat16).to(DEV)
    pos, from_slots = torch.arange(T, dtype=torch.int32, device=DEV), torch.randperm(320, generator=g)[:T].to(DEV)

    def state():
        return dict(codes=c0.clone(), scales=s0.clone(), at=slots.to(DEV), q=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV),
                    status=ints([0]))

    def call(kind, t, stream=None):
        if kind:
            api.is_move_scaled(fd, source, from_slots, cd, t["codes"], t["scales"], t["at"], t["status"], stream=stream)
        else:
            api.is_append_scaled(x[:, :Hq], x[:, Hq: Hq + H], x[:, Hq + H:], pos, t["at"], rope, cd, t["codes"], t["scales"], t["q"],
                                 t["status"], stream=stream)
    states, streams, graphs = [state(), state()], [torch.cuda.Stream() for _ in range(2)], []
    for kind in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[kind]):
            call(kind, states[kind], streams[kind])
        graphs.append(graph)
    for share in (0.0, 0.5, 0.9, 0.99, 1.0):
        skip = torch.rand(T, generator=g) < share
        for t in states:
            t["at"].copy_(torch.where(skip, -1, slots))
            t["codes"].copy_(c0)
            t["scales"].copy_(s0)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for kind, t in enumerate(states):
            want = state()
            want["at"].copy_(t["at"])
            call(kind, want)
            assert all(torch.equal(want[name].view(torch.uint8), t[name].view(torch.uint8)) for name in ("codes", "scales"))
            assert t["status"].tolist() == [0] and (share < 1.0 or torch.equal(t["codes"], c0))
