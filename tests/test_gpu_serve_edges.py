"""The serving step's calls at their edges, against the plain 64-bit definitions."""
import time

import pytest
import torch

from kv_cache_injection_gb300 import _lib, api
from tests import gpu_helpers as gh
from tests import serve_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")]
SCALES = {"e4m3": (0.02, 0.05)}


@pytest.fixture(scope="module", autouse=True)
def built():
    gh.ensure_built()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def stored(x, cache, scale):
    """x as the cache holds it, and the fp64 values that stands for."""
    if cache == "e4m3":
        x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = x.to(ref.TORCH[cache])
    return x, ref.stored_values(cache, x) * scale


# ---------------------------------------------------------------- blocks freed behind a window

@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bs", [8, 16, 24, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_before_the_window_need_no_name(D, bs, dtype, cache):
    """An engine takes back the blocks that lie before every row's window and leaves -1, or an id of no block, in the
    table: single tokens and prompts answer as if they were there, and report nothing."""
    g = torch.Generator().manual_seed(21)
    H, Hq, n, sc = 2, 8, 700, SCALES.get(cache, (1.0, 1.0))
    nb = -(-n // bs)
    for rows, window in ((1, 90), (1, 300), (20, 250), (70, 5), (200, 40)):
        kv = [stored(torch.randn(nb * bs, H, D, generator=g), cache, sc[i]) for i in range(2)]
        lc = torch.stack([s for s, _ in kv]).view(2, nb, bs, H, D)
        table = torch.arange(nb, dtype=torch.int32)
        first = n - rows - window + 1                  # the first position that a row sees
        table[: first // bs: 2], table[1: first // bs: 2] = -1, nb + 5
        q = torch.randn(rows, Hq, D, generator=g).to(ref.TORCH[dtype])
        out, lse, status = torch.empty_like(q, device=DEV), torch.empty(rows, Hq, device=DEV), ints([0])
        api.is_attend(q.to(DEV), ints([n]), table[None].to(DEV), api.make_cache_desc(bs, nb, cache, *sc), lc.to(DEV), out,
                      api.attend_workspace(), status, q_start=ints([0, rows]), max_q_len=rows, window=window, lse_out=lse)
        k, v = (x[:n] for _, x in kv)
        o, ls, spread, heft, seen = ref.attend(q.double(), n, k, v, torch.ones(n, dtype=torch.bool), D ** -0.5, window)
        tol, ltol = ref.attend_tolerance(dtype, cache, D, o, ls, spread, heft, seen, float(v.abs().max()))
        assert status.tolist() == [0], (rows, window)
        assert bool(((out.cpu().double() - o).abs() <= tol).all()) and bool(((lse.cpu().double() - ls).abs() <= ltol).all())


# ---------------------------------------------------------------- the largest slot map

@pytest.mark.parametrize("requests", [3, 600])
def test_slot_map_of_2_31_entries(requests):
    """The largest slot map that max_tokens can name (17 GB), nearly all of it padding: the kernel has as many threads."""
    bs, cap = 16, (1 << 31) - 1
    lens, news = [7 * r % 50 for r in range(requests)], [1 + 5 * r % 40 for r in range(requests)]
    need = [-(-(n + m) // bs) for n, m in zip(lens, news)]
    have = [-(-n // bs) for n in lens]
    ids = list(range(sum(need) + 3))[::-1]
    table = [[ids.pop() if j < have[r] else -1 for j in range(7)] for r in range(requests)]
    want = ref.extend(lens, news, ids, 0, table, bs, len(ids) + sum(have), sum(news))
    t, status, head = ints(table), ints([0]), ints([-9])
    slots = torch.full((cap,), -9, dtype=torch.int64, device=DEV)
    api.is_extend_block_table(ints(lens), ints(news), ints(ids), bs, len(ids) + sum(have), t, slots, status_out=status,
                              free_head_out=head)
    assert t.tolist() == want[0] and head.tolist() == [want[5]] and status.tolist() == [0]
    assert slots[: sum(news)].tolist() == want[1]
    assert all(bool((slots[i: i + (1 << 28)] == -1).all()) for i in range(sum(news), cap, 1 << 28))


# ---------------------------------------------------------------- faint weights

@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("dtype,cache", [("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128])
def test_faint_weights_beside_a_strong_one(D, dtype, cache, rows):
    """A first key that takes nearly all weight and whose value is 0: the output is what the other 2999 keys add, each
    with about 2^-26 of the first one's weight.  Weights are kept in fp16 with at least 2^7 for the largest, so that
    a step of the smallest ones is 2^-24, half of it 2^-32 of the largest: that times |v| a key is the bound on what
    their rounding may change."""
    g = torch.Generator().manual_seed(31)
    H, Hq, n, bs, R, sc = 1, 4, 3000, 16, 600 if rows == 1 else 64, SCALES.get(cache, (1.0, 1.0))
    nb = -(-n // bs)
    k = 0.3 * torch.randn(nb * bs, H, D, generator=g) * (64 / D) ** 0.5
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = 2.28125
    v = 1.0 + 0.2 * torch.randn(nb * bs, H, D, generator=g)
    v[0] = 0.0
    (ks, k), (vs, v) = stored(k, cache, sc[0]), stored(v, cache, sc[1])
    k, v = k[:n], v[:n]
    q = 0.25 * torch.randn(R * rows, Hq, D, generator=g)
    q[:, :, 0] = 8.0
    q = q.to(ref.TORCH[dtype])
    out, lse, status = torch.empty_like(q, device=DEV), torch.empty(R * rows, Hq, device=DEV), ints([0])
    api.is_attend(q.to(DEV), ints([n] * R), torch.arange(nb, dtype=torch.int32).repeat(R, 1).to(DEV),
                  api.make_cache_desc(bs, nb, cache, *sc), torch.stack([ks, vs]).view(2, nb, bs, H, D).to(DEV), out,
                  api.attend_workspace(), status, q_start=ints([rows * r for r in range(R + 1)]), max_q_len=rows, scale=1.0,
                  lse_out=lse)
    assert status.tolist() == [0]
    out, lse = out.cpu().double(), lse.cpu().double()
    for r in range(0, R, 1 if rows == 1 else 4):
        mine = slice(rows * r, rows * (r + 1))
        o, ls, spread, heft, seen = ref.attend(q[mine].double(), n, k, v, torch.ones(n, dtype=torch.bool), 1.0, 0)
        tol, ltol = ref.attend_tolerance(dtype, cache, D, o, ls, spread, heft, seen, float(v.abs().max()) * 2.0 ** -7)
        err = (out[mine] - o).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()), float((err / o.abs()).max()))
        assert bool(((lse[mine] - ls).abs() <= ltol).all())

# ---------------------------------------------------------------- logits without bounds

@pytest.mark.parametrize("rows", [1, 5, 60])
@pytest.mark.parametrize("dtype,cache,size", [("bf16", "bf16", 1e30), ("bf16", "e4m3", 1e30), ("f32", "f32", 1e30),
                                              ("f16", "f16", 6e4), ("f16", "e4m3", 6e4), ("bf16", "bf16", 1e9)])
def test_logits_past_every_step(dtype, cache, size, rows):
    """Logits of 2^24 to 2^110, whose fp32 steps are larger than any softmax is wide.  One key's is positive and all
    others' are negative, so that one takes all weight: the output is its value, rounded."""
    g = torch.Generator().manual_seed(51)
    H, Hq, D, n, bs, sc = 1, 4, 64, 400, 16, SCALES.get(cache, (1.0, 1.0))
    nb = -(-n // bs)
    big = 900.0 if cache == "f16" else 4.0
    k = -big * torch.rand(nb * bs, H, D, generator=g)
    k[17] = -k[17]
    (ks, k), (vs, v) = stored(k, cache, sc[0]), stored(torch.randn(nb * bs, H, D, generator=g), cache, sc[1])
    q = (size * (0.5 + 0.5 * torch.rand(rows, Hq, D, generator=g))).to(ref.TORCH[dtype])
    out, lse, status = torch.empty_like(q, device=DEV), torch.empty(rows, Hq, device=DEV), ints([0])
    api.is_attend(q.to(DEV), ints([n]), ints([list(range(nb))]), api.make_cache_desc(bs, nb, cache, *sc),
                  torch.stack([ks, vs]).view(2, nb, bs, H, D).to(DEV), out, api.attend_workspace(), status,
                  q_start=ints([0, rows]), max_q_len=rows, scale=1.0, lse_out=lse)
    o, ls, spread, heft, seen = ref.attend(q.double(), n, k[:n], v[:n], torch.ones(n, dtype=torch.bool), 1.0, 0)
    # The others' weights are exactly 0, so only the value's scale, its weight (1 over itself) and the output round.
    tol = (ref.U[dtype] * 1.01 + 2.0 ** -20) * o.abs() + (2.0 ** -25 if dtype == "f16" else 0.0)
    lse_tol = (D + 16) * 2.0 ** -24 * heft + 2.0 ** -22 * ls.abs()
    assert status.tolist() == [0]
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert bool(((lse.cpu().double() - ls).abs() <= lse_tol).all())


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("dtype,cache,D,bs,window", [
    ("bf16", "bf16", 64, 16, 0), ("bf16", "bf16", 128, 16, 0), ("f16", "f16", 128, 8, 250), ("bf16", "bf16", 128, 24, 0),
    ("f16", "f16", 256, 16, 0), ("bf16", "e4m3", 128, 16, 0), ("f16", "e4m3", 64, 16, 0)])
def test_waits_that_run_out(dtype, cache, D, bs, window):
    """An ordinary prompt with limits of its waits that it cannot keep: the call ends at once (its own copies in flight
    have landed by then), reports IS_ST_TIMEOUT and nothing else, and the next call on the same stream and workspace,
    which needs the tensor memory back, gives the bits that it gave before."""
    g = torch.Generator().manual_seed(61)
    H, Hq, lens, rows, sc = 2, 8, [3333, 900, 70], [200, 100, 70], SCALES.get(cache, (1.0, 1.0))
    need = [-(-n // bs) for n in lens]
    nb = sum(need)
    table, at = torch.full((3, max(need)), -1, dtype=torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = torch.arange(at, at + n)
        at += n
    lc = torch.stack([stored(torch.randn(nb * bs, H, D, generator=g), cache, sc[i])[0] for i in range(2)])
    q = torch.randn(sum(rows), Hq, D, generator=g).to(ref.TORCH[dtype]).to(DEV)
    start = [0, 200, 300, 370]
    args = (q, ints(lens), table.to(DEV), api.make_cache_desc(bs, nb, cache, *sc), lc.view(2, nb, bs, H, D).to(DEV))
    ws, status = api.attend_workspace(), ints([0])

    def call(**kw):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        t = time.perf_counter()
        api.is_attend(*args, out, ws, status, q_start=ints(start), max_q_len=200, window=window, **kw)
        torch.cuda.synchronize()
        bits = status.item()
        status.zero_()
        return out.cpu(), bits, time.perf_counter() - t

    want, bits, _ = call()
    assert bits == 0 and bool(want.isfinite().all())
    seen = 0
    for budget in (0, 0, 500, 2000, 10000, 100000):
        out, bits, took = call(budget_ns=budget)
        assert bits in (0, _lib.IS_ST_TIMEOUT) and took < 1.0
        assert bits or torch.equal(out, want)
        seen |= bits
        out, bits, _ = call()
        assert bits == 0 and torch.equal(out, want)
    assert seen == _lib.IS_ST_TIMEOUT


# ---------------------------------------------------------------- arguments left out

def test_q_start_without_max_q_len():
    """Requests of several rows are answered although their largest number is not given."""
    g = torch.Generator().manual_seed(41)
    H, Hq, D, bs, nb = 1, 2, 64, 16, 6
    lc = torch.randn(2, nb, bs, H, D, generator=g)
    q = torch.randn(24, Hq, D, generator=g)
    for starts, lens in (([0, 5, 24], [30, 40]), ([0, 1, 2], [30, 40]), ([0, 0, 24], [9, 24])):
        got = []
        for kw in (dict(), dict(max_q_len=24)):
            out, status = torch.full((24, Hq, D), 7.0, device=DEV), ints([0])
            api.is_attend(q.to(DEV), ints(lens), ints([[0, 1, 2], [3, 4, 5]]), api.make_cache_desc(bs, nb, "f32"), lc.to(DEV),
                          out, api.attend_workspace(), status, q_start=ints(starts), **kw)
            assert status.tolist() == [0]
            got.append(out.cpu())
        assert torch.equal(*got)
        assert bool((got[0][: starts[-1]] != 7.0).all()) and bool((got[0][starts[-1]:] == 7.0).all())


# ---------------------------------------------------------------- query rows of a wide spread

@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale,zero", [(0.125, True), (2.0 ** -26, False)])
def test_one_large_element_a_query_row(D, rows, scale, zero):
    """bf16 rows with one element of 2^26 over an FP8 cache, whose keys are 0 there (the others decide) or not.  The
    products are taken in fp16 with the largest element in [2^14, 2^15), where rounding changes an element by half of
    the smallest step, 2^-25, at most: 2^-39 of the largest element, times |k| and the scale in a logit."""
    g = torch.Generator().manual_seed(71)
    H, Hq, n, bs, sc = 1, 4, 500, 16, SCALES["e4m3"]
    nb = -(-n // bs)
    k = torch.randn(nb * bs, H, D, generator=g)
    if zero:
        k[:, :, 0] = 0.0
    (ks, k), (vs, v) = stored(k, "e4m3", sc[0]), stored(torch.randn(nb * bs, H, D, generator=g), "e4m3", sc[1])
    k, v = k[:n], v[:n]
    q = torch.randn(rows, Hq, D, generator=g)
    q[:, :, 0] = 2.0 ** 26
    q = q.to(torch.bfloat16)
    out, lse, status = torch.empty_like(q, device=DEV), torch.empty(rows, Hq, device=DEV), ints([0])
    api.is_attend(q.to(DEV), ints([n]), ints([list(range(nb))]), api.make_cache_desc(bs, nb, "e4m3", *sc),
                  torch.stack([ks, vs]).view(2, nb, bs, H, D).to(DEV), out, api.attend_workspace(), status,
                  q_start=ints([0, rows]), max_q_len=rows, scale=scale, lse_out=lse)
    o, ls, spread, heft, seen = ref.attend(q.double(), n, k, v, torch.ones(n, dtype=torch.bool), scale, 0)
    lost = 2.0 ** -39 * 2.0 ** 26 * float(k.abs().sum(-1).max()) * scale
    tol, ltol = ref.attend_tolerance("bf16", "e4m3", D, o, ls, spread, heft + lost / ((D + 8) * 2.0 ** -24), seen,
                                     float(v.abs().max()))
    assert status.tolist() == [0] and lost < 0.01
    assert bool(((out.cpu().double() - o).abs() <= tol).all()) and bool(((lse.cpu().double() - ls).abs() <= ltol).all())


# ---------------------------------------------------------------- single tokens' weights

@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (7, 1, 128), (4, 2, 256)])
def test_single_tokens_weights_keep_their_bits(Hq, H, D, dtype, cache):
    """A single token's weights are multiplied with what their rounding took off: they keep 2^-16 (bf16) or 2^-22 (fp16;
    2^-32 of the largest among the faintest), so that the output's rounding is all that 16 bits cost."""
    g = torch.Generator().manual_seed(81)
    lens, bs, sc = [1, 17, 130, 900, 2500] * 20, 16, SCALES.get(cache, (1.0, 1.0))
    nb = -(-max(lens) // bs)
    kv = [stored(torch.randn(nb * bs, H, D, generator=g), cache, sc[i]) for i in range(2)]
    k, v = (x for _, x in kv)
    q = torch.randn(len(lens), Hq, D, generator=g).to(ref.TORCH[dtype])
    out, status = torch.empty_like(q, device=DEV), ints([0])
    api.is_attend(q.to(DEV), ints(lens), torch.arange(nb, dtype=torch.int32).repeat(len(lens), 1).to(DEV),
                  api.make_cache_desc(bs, nb, cache, *sc), torch.stack([s for s, _ in kv]).view(2, nb, bs, H, D).to(DEV), out,
                  api.attend_workspace(), status)
    assert status.tolist() == [0]
    for r, n in enumerate(lens):
        o, ls, spread, heft, seen = ref.attend(q[r: r + 1].double(), n, k[:n], v[:n], torch.ones(n, dtype=torch.bool), D ** -0.5, 0)
        tol, _ = ref.attend_tolerance("f32", "f32", D, o, ls, spread, heft, seen, 0.0)
        tol = tol + (2.0 ** -16 if dtype == "bf16" else 2.0 ** -22) * 1.01 * spread + ref.U[dtype] * 1.01 * o.abs()
        if dtype == "f16":
            tol = tol + n * 2.0 ** -32 * float(v[:n].abs().max()) + 2.0 ** -25
        err = (out[r: r + 1].cpu().double() - o).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()))
