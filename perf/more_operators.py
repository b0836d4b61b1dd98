"""The serving step over a paged cache held in 8 bits with a scale for each block and KV head.

Codes [2][blocks][block][kv_heads][dim] (INT8, or FP8 E4M3) and scales fp32
[2][blocks][kv_heads]; an element is its code times its block's scale.  The
scales follow the data: a block's first tokens set them, later ones may raise
them, and then what the block holds already is rounded anew.  Cases of five
kinds:

  append   is_append_scaled: rotary positions, K/V quantised as they are written
  move     is_move_scaled: tokens of a 16-bit cache (an injected segment) into it
  read     is_read_scaled: tokens read back as rows, keys turned back if wanted
  decode   is_attend_scaled with one new token per request
  prompt   is_attend_scaled with a ragged chunk of new tokens per request, causal

`run` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64), or, where `own` is set, by the framework's call.  Codes
come back as the numbers they are, beside their scales.
"""
import math
import random

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SMALLEST, LARGEST = 2.0 ** -40, 2.0 ** 40             # of a scale
WORKSPACE = 64 << 20                                  # bytes of scratch an engine keeps for attention


# ---------------------------------------------------------------- cases

def listed():
    llama = dict(heads=32, kv_heads=8, dim=128)       # also the Mistral-7B shape
    qwen = dict(heads=28, kv_heads=4, dim=128)
    return [
        # The single new token of one request, inside a block: nothing but latency.
        dict(name="append_one_token", op="append", requests=1, shortest=1313, longest=1313, new_min=1, new_max=1,
             dtype="bf16", cache="e4m3", axes=1, style=0, theta=5e5, block=16, pad=0, **llama),
        # One step of 100 users, some at a block's first row, some raising a block's scale.
        dict(name="append_step_100", op="append", requests=100, shortest=300, longest=2048, new_min=1, new_max=1,
             dtype="bf16", cache="e4m3", axes=1, style=0, theta=1e6, block=16, pad=0, **qwen),
        # Prompts of several requests together: whole blocks, and ragged first and last ones.
        dict(name="append_prompts", op="append", requests=5, shortest=1700, longest=1900, new_min=1500, new_max=1700,
             dtype="bf16", cache="int8", axes=1, style=0, theta=5e5, block=16, pad=0, **llama),
        # One user's injected segment of 50 facts, from the 16-bit cache that it was injected into.
        dict(name="move_segment", op="move", requests=1, shortest=1276, longest=1276, new_min=1276, new_max=1276,
             dtype="bf16", cache="int8", block=16, pad=0, **llama),
        # The segments of many users at once.
        dict(name="move_segments_40", op="move", requests=40, shortest=900, longest=1400, new_min=900, new_max=1400,
             dtype="bf16", cache="e4m3", block=32, pad=0, **llama),
        # A conversation read back with its keys turned back, to be stored as new facts.
        dict(name="read_conversation", op="read", requests=1, shortest=1300, longest=1300, new_min=700, new_max=700,
             dtype="bf16", cache="int8", axes=1, style=0, theta=5e5, turned=1, block=16, pad=0, **llama),
        # What many users have in the cache, for an engine that works on dense rows.
        dict(name="read_users", op="read", requests=40, shortest=300, longest=2048, new_min=300, new_max=2048,
             dtype="bf16", cache="e4m3", axes=1, style=0, theta=1e6, turned=0, block=16, pad=0, **llama),
        # One request right behind an injected segment of 50 facts.
        dict(name="decode_one", op="attend", requests=1, shortest=1313, longest=1313, new_min=1, new_max=1, window=0,
             dtype="bf16", cache="int8", block=16, **llama),
        # 100 users, ragged lengths, a group of seven query heads.
        dict(name="decode_users_100", op="attend", requests=100, shortest=300, longest=2048, new_min=1, new_max=1,
             window=0, dtype="bf16", cache="int8", block=16, **qwen),
        # Few rows over very long caches: the length has to be split.
        dict(name="decode_long", op="attend", requests=4, shortest=60000, longest=131072, new_min=1, new_max=1,
             window=0, dtype="bf16", cache="int8", block=16, **llama),
        # The users' questions behind their injected segments, several requests packed.
        dict(name="prompt_questions", op="attend", requests=16, shortest=900, longest=2000, new_min=20, new_max=100,
             window=0, dtype="bf16", cache="e4m3", block=16, **llama),
        # Long prompts behind long segments: compute-bound.
        dict(name="prompt_long", op="attend", requests=2, shortest=6000, longest=8192, new_min=2000, new_max=2500,
             window=0, dtype="bf16", cache="int8", block=16, **llama),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "move", "read", "decode", "decode", "prompt"])
    block = rng.choice([16, 16, 32, 8, 64, 24, 7])
    heads = rng.choice([dict(heads=32, kv_heads=8, dim=128), dict(heads=28, kv_heads=4, dim=128),
                        dict(heads=40, kv_heads=8, dim=128), dict(heads=8, kv_heads=8, dim=64),
                        dict(heads=16, kv_heads=2, dim=64), dict(heads=16, kv_heads=1, dim=128),
                        dict(heads=8, kv_heads=4, dim=256)])
    dtype, cache = rng.choice(["bf16", "bf16", "f16"]), rng.choice(["int8", "int8", "e4m3"])
    if op in ("append", "move", "read"):
        if rng.random() < 0.15:
            dtype, heads = "f32", dict(heads=4, kv_heads=2, dim=64)
        requests = _log(rng, 1, 200)
        new = 1 if op == "append" and rng.random() < 0.4 else _log(rng, 1, 6000 // requests)
        longest = new + rng.choice([0, _log(rng, 1, 2000)])
        return dict(op=op, requests=requests, shortest=new, longest=longest, new_min=rng.choice([1, max(1, new // 2)]),
                    new_max=new, dtype=dtype, cache=cache, axes=rng.choice([1, 1, 2, 3]), style=rng.choice([0, 0, 1]),
                    theta=rng.choice([1e4, 5e5, 1e6]), turned=rng.choice([0, 1]), block=block, pad=rng.choice([0, 0, 3]),
                    **heads)
    if op == "decode":
        requests = _log(rng, 1, 300)
        longest = _log(rng, 30, max(100, min(120000, 400000 // requests)))
        new = rng.choice([1, 1, 1, 2, 4])
    else:
        requests = _log(rng, 1, 24)
        longest = _log(rng, 400, max(500, 16000 // requests))
        new = _log(rng, 8, 2000 // requests)
    return dict(op="attend", requests=requests, shortest=_log(rng, 1, longest), longest=longest, new_min=1,
                new_max=min(new, longest), window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype=dtype, cache=cache,
                block=block, **heads)


def _lengths(case):
    """(length, new tokens of it) of each request: the case's own, whatever the seed; the first has the largest."""
    rng = random.Random(case["requests"] * 1000003 + case["longest"])
    got = [(case["longest"], case["new_max"])]
    while len(got) < case["requests"]:
        got.append((rng.randint(case["shortest"], case["longest"]), rng.randint(case["new_min"], case["new_max"])))
    return [(n, min(n, m)) for n, m in got]


def _blocks_touched(case):
    """Blocks that hold new tokens."""
    bs = case["block"]
    return sum(-(-n // bs) - (n - m) // bs for n, m in _lengths(case))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"append": _prepare_append, "move": _prepare_move, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, g)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, dtype=TORCH[dtype], device="cuda")


def _values(case, codes):
    """Codes as numbers."""
    return codes.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else codes


def _encode(case, x):
    """fp32 numbers in a scale's units to codes: nearest even, saturated."""
    if case["cache"] == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.nan_to_num(nan=0.0).round().clamp(-127, 127).to(torch.int8)


def _scaled_cache(g, case, blocks, held=None):
    """N(0, 1) keys and values, heads of different magnitude.  held [blocks]: rows that count for a block's scale."""
    H, D, bs = case["kv_heads"], case["dim"], case["block"]
    x = torch.randn((2, blocks, bs, H, D), generator=g, dtype=torch.bfloat16, device="cuda")
    x *= 2.0 ** torch.randint(-2, 3, (2, 1, 1, H, 1), generator=g, device="cuda").to(torch.bfloat16)
    size = x.abs()
    if held is not None:
        size = size * (torch.arange(bs, device="cuda")[None] < held[:, None])[None, :, :, None, None]
    scales = (size.amax((2, 4)).float() / QMAX[case["cache"]]).clamp(SMALLEST, LARGEST)
    codes = torch.cat([_encode(case, x[kv:kv + 1].float() / scales[kv:kv + 1, :, None, :, None]) for kv in (0, 1)])
    return codes, scales


def _tokens(g, case):
    """Slots and positions of the requests' new tokens, requests back to back, and per block the rows held before."""
    lens, bs = _lengths(case), case["block"]
    n, m = _ints([a for a, _ in lens], torch.int64), _ints([b for _, b in lens], torch.int64)
    taken = (n + bs - 1) // bs
    blocks = sum(-(-a // bs) for a, _ in lens) + 4
    ids = torch.randperm(blocks, generator=g, device="cuda")
    T = sum(b for _, b in lens)
    r = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), m, output_size=T)
    position = torch.arange(T, device="cuda") - (m.cumsum(0) - m)[r] + (n - m)[r]
    first_block = taken.cumsum(0) - taken
    slots = ids[first_block[r] + position // bs] * bs + position % bs
    held = torch.zeros(blocks, dtype=torch.int64, device="cuda")
    held[ids[first_block + (n - m) // bs]] = torch.where(m > 0, (n - m) % bs, 0)
    if case["pad"]:                                   # a padded batch: its last tokens have no slot
        slots[max(1, T - case["pad"]):] = -1
    return blocks, slots, position, held


def _axes_of(g, case, position):
    """[axes][T]: text, or an image of 32 columns behind the first positions."""
    image, cell = (position % 1024) >= 256, (position % 1024) - 256
    shift = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
    axis = [position, torch.where(image, position - cell + cell // 32, position),
            torch.where(image, position - cell + cell % 32, position)]
    return (torch.stack(axis[: case["axes"]]) + shift).to(torch.int32).contiguous()


def _sections(case):
    half = case["dim"] // 2
    if case["axes"] == 1:
        return [half]
    if case["axes"] == 2:
        return [half - half // 2, half // 2]
    side = 3 * half // 8
    return [half - 2 * side, side, side]


def _prepare_append(case, g):
    H, D = case["kv_heads"], case["dim"]
    blocks, slots, position, held = _tokens(g, case)
    T = slots.shape[0]
    # one projection's output holds the queries, keys and values of a token side by side
    qkv = _randn(g, (T, case["heads"] + 2 * H, D), case["dtype"])
    codes, scales = _scaled_cache(g, case, blocks, held)
    s = dict(case=case, qkv=qkv, q=qkv[:, : case["heads"]], k=qkv[:, case["heads"]: case["heads"] + H],
             v=qkv[:, case["heads"] + H:], slots=slots, positions=_axes_of(g, case, position), codes=codes, scales=scales,
             q_out=torch.zeros((T, case["heads"], D), dtype=TORCH[case["dtype"]], device="cuda"), status=_ints([0]))
    if own:                                           # the arguments a serving loop marshals once
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_append_scaled(
            s["q"], s["k"], s["v"], s["positions"], slots, api.make_rope(case["theta"], case["style"]),
            api.make_cache_desc(case["block"], blocks, case["cache"]), codes, scales, s["q_out"], s["status"],
            axes=api.make_axes(_sections(case)))
    return s


def _prepare_move(case, g):
    H, D, bs = case["kv_heads"], case["dim"], case["block"]
    blocks, slots, _, held = _tokens(g, case)
    T = slots.shape[0]
    from_blocks = -(-T // 16) + 3                     # the engine's 16-bit cache has blocks of 16
    order = torch.randperm(from_blocks, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    codes, scales = _scaled_cache(g, case, blocks, held)
    s = dict(case=case, source=_randn(g, (2, from_blocks, 16, H, D), case["dtype"]), slots=slots,
             from_slots=order[t // 16] * 16 + t % 16, codes=codes, scales=scales, status=_ints([0]))
    if own:
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_move_scaled(
            api.make_cache_desc(16, from_blocks, case["dtype"]), s["source"], s["from_slots"],
            api.make_cache_desc(bs, blocks, case["cache"]), codes, scales, slots, s["status"])
    return s


def _prepare_read(case, g):
    H, D = case["kv_heads"], case["dim"]
    blocks, slots, position, _ = _tokens(g, case)
    codes, scales = _scaled_cache(g, case, blocks)
    rows = (slots.shape[0], H, D)
    s = dict(case=case, slots=slots, positions=_axes_of(g, case, position), codes=codes, scales=scales,
             k_out=torch.zeros(rows, dtype=TORCH[case["dtype"]], device="cuda"),
             v_out=torch.zeros(rows, dtype=TORCH[case["dtype"]], device="cuda"), status=_ints([0]))
    if own:
        from kv_cache_injection_gb300 import api
        turn = dict(positions=s["positions"], rope=api.make_rope(case["theta"], case["style"]),
                    axes=api.make_axes(_sections(case))) if case["turned"] else {}
        s["call"] = api.prepare_read_scaled(slots, api.make_cache_desc(case["block"], blocks, case["cache"]), codes, scales,
                                            s["k_out"], s["v_out"], s["status"], **turn)
    return s


def _prepare_attend(case, g):
    lens = _lengths(case)
    bs, T = case["block"], sum(m for _, m in lens)
    taken = [-(-n // bs) for n, _ in lens]
    width, blocks = max(taken) + 3, sum(taken) + 4
    codes, scales = _scaled_cache(g, case, blocks)
    ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < _ints(taken)[:, None]] = ids[: sum(taken)]
    starts = [0]
    for _, m in lens:
        starts.append(starts[-1] + m)
    s = dict(case=case, q=_randn(g, (T, case["heads"], case["dim"]), case["dtype"]), codes=codes, scales=scales,
             table=table, seq_len=_ints([n for n, _ in lens]), start=_ints(starts),
             out=torch.zeros((T, case["heads"], case["dim"]), dtype=TORCH[case["dtype"]], device="cuda"),
             lse=torch.zeros((T, case["heads"]), dtype=torch.float32, device="cuda"), status=_ints([0]),
             workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda"))
    if own:
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_attend_scaled(
            s["q"], s["seq_len"], table, api.make_cache_desc(bs, blocks, case["cache"]), codes, scales, s["out"],
            s["workspace"], s["status"], q_start=s["start"], max_q_len=case["new_max"], scale=case["dim"] ** -0.5,
            window=case["window"], lse_out=s["lse"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    else:
        {"append": _plain_append, "move": _plain_move, "read": _plain_read, "attend": _plain_attend}[op](s)
    if op == "attend":
        return s["out"], s["lse"]
    if op == "read":
        return s["k_out"], s["v_out"]
    codes = _values(s["case"], s["codes"])
    if s["case"]["cache"] == "int8":                  # as numbers: whole ones that a bf16 holds
        codes = codes.to(torch.bfloat16)
    return (codes, s["scales"], s["q_out"]) if op == "append" else (codes, s["scales"])


def _turn(s):
    """cos and sin [T][1][D / 2] of the tokens' positions."""
    case, half = s["case"], s["case"]["dim"] // 2
    pair = torch.arange(half, device="cuda", dtype=torch.float64)
    frequency = case["theta"] ** (-2.0 * pair / case["dim"])
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), _ints(_sections(case)), output_size=half)
    angle = s["positions"].double()[axis].T * frequency
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin, style):
    """x [T][heads][D] in 32 bits, cos and sin [T][1][D / 2]."""
    if style == 0:
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_write(s, rows):
    """rows [2][T][H][D] in 32 bits to the tokens' slots, quantised."""
    case, codes, scales, slots = s["case"], s["codes"], s["scales"], s["slots"]
    bs, blocks, H, D = case["block"], scales.shape[1], case["kv_heads"], case["dim"]
    put = slots >= 0
    at = torch.where(put, slots, blocks * bs)         # tokens without a slot go to a block behind the last
    block, row = at // bs, at % bs
    top = torch.zeros((2, blocks + 1, H), device="cuda")
    top.index_reduce_(1, block, rows.abs().amax(-1), "amax")
    low = torch.full((blocks + 1,), bs, dtype=torch.int64, device="cuda").index_reduce_(0, block, row, "amin")[:blocks]
    fresh = (top[:, :blocks] / QMAX[case["cache"]]).clamp(SMALLEST, LARGEST)
    touched = low < bs
    scale = torch.where(touched[:, None], torch.where((low == 0)[:, None], fresh, torch.maximum(scales, fresh)), scales)
    ratio = scales / scale                            # what a block holds already is rounded anew where its scale grows
    grown = touched[None, :, None] & (low > 0)[None, :, None] & (scale > scales)
    old = (torch.arange(bs, device="cuda")[None] < low[:, None])[None, :, :, None] & grown[:, :, None]
    again = _encode(case, _values(case, codes).float() * ratio[:, :, None, :, None])
    flat = torch.where(old[..., None], again, codes).view(2, blocks * bs, H, D)
    flat = torch.cat([flat, flat[:, :1]], 1)          # a place for the tokens without a slot
    inverse = torch.cat([1.0 / scale, torch.ones_like(scale[:, :1])], 1)
    flat[:, at] = _encode(case, rows * inverse[:, block, :, None])
    codes.copy_(flat[:, : blocks * bs].view(codes.shape))
    scales.copy_(scale)


def _plain_append(s):
    cos, sin = _turn(s)
    style, put = s["case"]["style"], (s["slots"] >= 0)[:, None, None]
    q = _rotate(s["q"].float(), cos, sin, style).to(s["q_out"].dtype)
    s["q_out"].copy_(torch.where(put, q, s["q_out"]))
    _plain_write(s, torch.stack([_rotate(s["k"].float(), cos, sin, style), s["v"].float()]))


def _plain_move(s):
    source = s["source"]
    _plain_write(s, source.view(2, -1, *source.shape[3:])[:, s["from_slots"]].float())


def _plain_read(s):
    case, put = s["case"], (s["slots"] >= 0)[:, None, None]
    at, H, D = s["slots"].clamp(min=0), case["kv_heads"], case["dim"]
    rows = _values(case, s["codes"].view(2, -1, H, D)[:, at]).float() * s["scales"][:, at // case["block"], :, None]
    k, v = rows[0], rows[1]
    if case["turned"]:
        cos, sin = _turn(s)
        k = _rotate(k, cos, -sin, case["style"])
    s["k_out"].copy_(torch.where(put, k.to(s["k_out"].dtype), s["k_out"]))
    s["v_out"].copy_(torch.where(put, v.to(s["v_out"].dtype), s["v_out"]))


def _plain_attend(s):
    case = s["case"]
    bs, D, H = case["block"], case["dim"], case["kv_heads"]
    G, R, N, T = case["heads"] // H, case["requests"], case["new_max"], s["q"].shape[0]
    table, seq, start = s["table"], s["seq_len"].long(), s["start"].long()
    key = torch.arange(table.shape[1] * bs, device="cuda")
    block = table[:, key // bs].long()
    at = block.clamp(min=0) * bs + key % bs           # [R][S]
    rows, scales = s["codes"].view(2, -1, H, D), s["scales"][:, block.clamp(min=0), :, None]
    k = _values(case, rows[0][at]).float() * scales[0]
    v = _values(case, rows[1][at]).float() * scales[1]
    count = start[1:] - start[:-1]
    i = torch.arange(N, device="cuda")
    q = s["q"][(start[:-1, None] + i).clamp(max=T - 1)].float().view(R, N, H, G, D)
    position = (seq - count)[:, None] + i             # [R][N]
    seen = (key <= position[..., None]) & (block >= 0)[:, None]
    if case["window"]:
        seen &= key > position[..., None] - case["window"]
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(R, H, G * N, D), k.permute(0, 2, 3, 1)) * D ** -0.5
    score = score.view(R, H, G, N, -1).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, H, G * N, -1), v.permute(0, 2, 1, 3)).view(R, H, G, N, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(R, N, H * G, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(R, N, H * G)
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(start[1:], t, right=True)
    s["out"], s["lse"] = o[r, t - start[r]].to(s["q"].dtype), lse[r, t - start[r]]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    lens = _lengths(case)
    H, D, e = case["kv_heads"], case["dim"], SIZE[case["dtype"]]
    T = sum(m for _, m in lens)
    scales = 8 * H * _blocks_touched(case)            # K's and V's, once
    if case["op"] == "append":
        return {"bytes": T * (D * (2 * case["heads"] * e + 2 * H * e + 2 * H) + 8 + 4 * case["axes"]) + 2 * scales,
                "flops": 3 * T * D * (case["heads"] + H)}
    if case["op"] == "move":
        return {"bytes": T * (2 * H * D * (e + 1) + 16) + scales, "flops": 0}
    if case["op"] == "read":
        return {"bytes": T * (2 * H * D * (1 + e) + 8 + case["turned"] * 4 * case["axes"]) + scales,
                "flops": case["turned"] * 3 * T * D * H}
    reach = case["window"] or 1 << 40
    pairs = sum(min(n - m + i + 1, reach) for n, m in lens for i in range(m))
    keys = sum(min(n, m - 1 + reach) for n, m in lens if m)
    return {"bytes": 2 * keys * H * (D + 4 / case["block"]) + T * case["heads"] * (2 * D * e + 4),
            "flops": 4 * pairs * case["heads"] * D}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "move": _exact_move, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)


def _numbers(case, codes):
    return (codes.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else codes).to(torch.float64)


def _unit_turns(case, s, sign):
    D = case["dim"]
    owner = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
    i = torch.arange(D // 2, dtype=torch.float64, device="cuda")
    angle = sign * s["positions"].to(torch.float64)[owner] * torch.exp(-math.log(case["theta"]) * 2 * i / D)[:, None]
    return torch.polar(torch.ones_like(angle), angle).T[:, None]     # [T][1][D / 2]


def _turned(case, x, unit):
    D, x = case["dim"], x.to(torch.float64)
    if case["style"] == 1:
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], D // 2, 2)) * unit).flatten(-2)
    z = torch.complex(x[..., : D // 2], x[..., D // 2:]) * unit
    return torch.cat([z.real, z.imag], -1)


def _exact_write(case, s, k, v):
    """Codes before their rounding, and scales.  INT8 codes are whole numbers, a hundredth off what they stand for by
    their nature: they are compared with the plain form's alone."""
    bs, largest = case["block"], {"int8": 127, "e4m3": 448}[case["cache"]]
    codes, scales = _numbers(case, s["codes"]), s["scales"].to(torch.float64)
    slotted = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][slotted]
    ids, which = torch.unique(at // bs, return_inverse=True)
    spread = which[:, None].expand(-1, case["kv_heads"])
    low = torch.full(ids.shape, bs, device="cuda").scatter_reduce(0, which, at % bs, "amin")
    below = torch.arange(bs, device="cuda") < low[:, None]
    for kv, rows in enumerate((k[slotted], v[slotted])):
        size = rows.abs().amax(-1)
        size = torch.zeros((len(ids), case["kv_heads"]), dtype=torch.float64, device="cuda").scatter_reduce(0, spread, size, "amax")
        new = torch.clamp(size / largest, 2.0 ** -40, 2.0 ** 40)
        before = scales[kv, ids]
        now = torch.where(low[:, None] > 0, torch.maximum(before, new), new)
        held = codes[kv, ids]
        codes[kv, ids] = torch.where(below[..., None, None], held * (before / now)[:, None, :, None], held)
        codes[kv].view(-1, *rows.shape[1:])[at] = rows / now[which][..., None]
        scales[kv, ids] = now
    return codes if case["cache"] == "e4m3" else None, scales


def _exact_append(case, s):
    unit = _unit_turns(case, s, 1.0)
    codes, scales = _exact_write(case, s, _turned(case, s["k"], unit), s["v"].to(torch.float64))
    return codes, scales, torch.where((s["slots"] >= 0)[:, None, None], _turned(case, s["q"], unit), s["q_out"].double())


def _exact_move(case, s):
    k, v = (half.flatten(0, 1)[s["from_slots"]].to(torch.float64) for half in s["source"])
    return _exact_write(case, s, k, v)


def _exact_read(case, s):
    slotted = torch.nonzero(s["slots"] >= 0)[:, 0]
    block, row = s["slots"][slotted] // case["block"], s["slots"][slotted] % case["block"]
    outs = []
    for kv, out in enumerate((s["k_out"], s["v_out"])):
        x = _numbers(case, s["codes"][kv, block, row]) * s["scales"][kv, block].to(torch.float64)[..., None]
        if kv == 0 and case["turned"]:
            x = _turned(case, x, _unit_turns(case, s, -1.0)[slotted])
        whole = out.to(torch.float64)
        whole[slotted] = x
        outs.append(whole)
    return tuple(outs)


def _exact_attend(case, s):
    H, D, bs = case["kv_heads"], case["dim"], case["block"]
    G = case["heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["q"].shape[0], case["heads"]), dtype=torch.float64, device="cuda")
    begin = 0
    for r, (n, m) in enumerate(_lengths(case)):
        if m == 0:
            continue
        first = max(0, n - m + 1 - case["window"]) if case["window"] else 0
        at = torch.arange(first, n, device="cuda")
        block = s["table"][r, at // bs].long()
        k, v = (_numbers(case, s["codes"][kv, block, at % bs]) * s["scales"][kv, block].double()[..., None] for kv in (0, 1))
        mine = torch.arange(n - m, n, device="cuda")[:, None]
        hidden = at > mine
        if case["window"]:
            hidden |= at <= mine - case["window"]
        for h in range(H):
            q = s["q"][begin: begin + m, h * G: (h + 1) * G].double()
            logit = torch.einsum("mgd,sd->mgs", q, k[:, h]) / math.sqrt(D)
            logit.masked_fill_(hidden[:, None], -math.inf)
            norm = torch.logsumexp(logit, -1)
            lse[begin: begin + m, h * G: (h + 1) * G] = norm
            out[begin: begin + m, h * G: (h + 1) * G] = torch.exp(logit - norm[..., None]) @ v[:, h]
        begin += m
    return out, lse
