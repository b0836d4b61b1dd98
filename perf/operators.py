"""The serving step around the injected memory segment, operator by operator.

A serving engine that injects a memory segment into the paged cache next makes
room for the tokens that follow it (a block table and a slot map from the
requests' lengths), rotates their queries and keys and writes their keys and
values behind the segment, and attends from them over the whole paged cache.
Cases of four kinds measure that:

  blocks   is_extend_block_table: blocks, slots and positions of the new tokens
  append   is_append: rotary positions of one or three axes, paged K/V write
  decode   is_attend with one new token per request
  prompt   is_attend with a ragged chunk of new tokens per request, causal

`run` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64), or, where `own` is set, by the framework's call.
"""
import math
import random

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.uint8}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
WORKSPACE = 64 << 20          # bytes of scratch an engine keeps for attention


# ---------------------------------------------------------------- cases

def listed():
    llama = dict(heads=32, kv_heads=8, dim=128)       # also the Mistral-7B shape
    qwen = dict(heads=28, kv_heads=4, dim=128)
    return [
        # One decode step of 100 users: a block is taken when a length crosses a block's end.
        dict(name="blocks_step_100", op="blocks", requests=100, shortest=300, longest=2000, new_min=1, new_max=1,
             block=16),
        # Admission of many users at once: each gets blocks for its segment and prompt.
        dict(name="blocks_admit_4096", op="blocks", requests=4096, shortest=0, longest=700, new_min=0, new_max=300,
             block=16),
        # The single new token of one Llama-3.1-8B request: nothing but latency.
        dict(name="append_one_token", op="append", tokens=1, dtype="bf16", cache="bf16", axes=1, style=0, theta=5e5,
             block=16, pad=0, **llama),
        # One step of 100 users into an FP8 cache.
        dict(name="append_step_fp8", op="append", tokens=100, dtype="bf16", cache="e4m3", axes=1, style=0, theta=1e6,
             block=16, pad=0, **qwen),
        # Prompts with images: three position axes, tokens of several requests together.
        dict(name="append_prompt_3axes", op="append", tokens=8192, dtype="bf16", cache="bf16", axes=3, style=0,
             theta=1e6, block=16, pad=0, **llama),
        # One request right behind an injected segment of 50 facts.
        dict(name="decode_one", op="attend", requests=1, shortest=1313, longest=1313, new_min=1, new_max=1, window=0,
             dtype="bf16", cache="bf16", block=16, **llama),
        # 100 users, ragged lengths, a group of seven query heads.
        dict(name="decode_users_100", op="attend", requests=100, shortest=300, longest=2048, new_min=1, new_max=1,
             window=0, dtype="bf16", cache="bf16", block=16, **qwen),
        # A large batch over an FP8 cache.
        dict(name="decode_fp8_64", op="attend", requests=64, shortest=500, longest=8000, new_min=1, new_max=1,
             window=0, dtype="bf16", cache="e4m3", block=16, **llama),
        # Few rows over very long caches: the length has to be split.
        dict(name="decode_long", op="attend", requests=4, shortest=60000, longest=131072, new_min=1, new_max=1,
             window=0, dtype="bf16", cache="bf16", block=16, **llama),
        # The fp32 cache of the small checkable model.
        dict(name="decode_f32", op="attend", requests=32, shortest=17, longest=1500, new_min=1, new_max=1, window=0,
             dtype="f32", cache="f32", block=16, heads=4, kv_heads=2, dim=64),
        # The users' questions behind their injected segments, several requests packed.
        dict(name="prompt_questions", op="attend", requests=16, shortest=900, longest=2000, new_min=20, new_max=100,
             window=0, dtype="bf16", cache="bf16", block=16, **llama),
        # Long prompts behind long segments: compute-bound.
        dict(name="prompt_long", op="attend", requests=2, shortest=6000, longest=8192, new_min=2000, new_max=2500,
             window=0, dtype="bf16", cache="bf16", block=16, **llama),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["blocks", "append", "decode", "decode", "prompt"])
    block = rng.choice([16, 16, 32, 8, 64])
    heads = rng.choice([dict(heads=32, kv_heads=8, dim=128), dict(heads=28, kv_heads=4, dim=128),
                        dict(heads=40, kv_heads=8, dim=128), dict(heads=8, kv_heads=8, dim=64),
                        dict(heads=16, kv_heads=2, dim=64), dict(heads=16, kv_heads=1, dim=128),
                        dict(heads=8, kv_heads=4, dim=256)])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    if op == "blocks":
        new = rng.choice([1, _log(rng, 2, 300)])
        return dict(op=op, requests=_log(rng, 1, 4096), shortest=0, longest=_log(rng, 20, 4000),
                    new_min=min(new, rng.choice([0, 1])), new_max=new, block=block)
    if op == "append":
        if rng.random() < 0.15:
            dtype = cache = "f32"
            heads = dict(heads=4, kv_heads=2, dim=64)
        return dict(op=op, tokens=_log(rng, 1, 6000), dtype=dtype, cache=cache, axes=rng.choice([1, 1, 2, 3]),
                    style=rng.choice([0, 0, 1]), theta=rng.choice([1e4, 5e5, 1e6]), block=block,
                    pad=rng.choice([0, 0, 3]), **heads)
    if rng.random() < 0.12:
        dtype = cache = "f32"
        heads = dict(heads=4, kv_heads=2, dim=64)
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
    """(length, new tokens) of each request: the case's own, whatever the seed; the first request has the largest."""
    rng = random.Random(case["requests"] * 1000003 + case["longest"])
    got = [(case["longest"], case["new_max"])]
    while len(got) < case["requests"]:
        got.append((rng.randint(case["shortest"], case["longest"]), rng.randint(case["new_min"], case["new_max"])))
    if case["op"] == "attend":                        # lengths there count the new tokens
        got = [(n, min(n, m)) for n, m in got]
    return got


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"blocks": _prepare_blocks, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, g)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, dtype=TORCH[dtype], device="cuda")


def _random_cache(g, case, blocks):
    """[2][blocks][block][kv_heads][dim]: N(0, 1) keys and values, an FP8 cache with scales of its own."""
    shape = (2, blocks, case["block"], case["kv_heads"], case["dim"])
    if case["cache"] != "e4m3":
        return _randn(g, shape, case["cache"]), 1.0, 1.0
    x = _randn(g, shape, "bf16")
    x[0] /= 0.02
    x[1] /= 0.03
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), 0.02, 0.03


def _prepare_blocks(case, g):
    lens = _lengths(case)
    bs, tokens = case["block"], sum(m for _, m in lens)
    taken = [-(-n // bs) for n, _ in lens]
    missing = [-(-(n + m) // bs) - t for (n, m), t in zip(lens, taken)]
    width = max(t + k for t, k in zip(taken, missing)) + 2
    total = sum(taken) + sum(missing) + 5
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(width, device="cuda")[None] < _ints(taken)[:, None]
    table[have] = ids[: sum(taken)]
    capacity = tokens + 7                             # a padded batch: the last slots stay -1
    s = dict(case=case, seq_len=_ints([n for n, _ in lens]), new_len=_ints([m for _, m in lens]), table=table,
             free=ids[sum(taken):].contiguous(), head=_ints([2]), num_blocks=total,
             slots=torch.empty(capacity, dtype=torch.int64, device="cuda"),
             positions=torch.zeros(capacity, dtype=torch.int32, device="cuda"),
             start=torch.empty(len(lens) + 1, dtype=torch.int32, device="cuda"),
             seq_out=torch.empty(len(lens), dtype=torch.int32, device="cuda"),
             head_out=torch.empty(1, dtype=torch.int32, device="cuda"), status=_ints([0]))
    if own:                                           # the arguments a serving loop marshals once
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_extend_block_table(
            s["seq_len"], s["new_len"], s["free"], bs, total, s["table"], s["slots"], s["positions"], s["start"],
            s["seq_out"], s["status"], free_head=s["head"], free_head_out=s["head_out"])
    return s


def _sections(case):
    half = case["dim"] // 2
    if case["axes"] == 1:
        return [half]
    if case["axes"] == 2:
        return [half - half // 2, half // 2]
    side = 3 * half // 8
    return [half - 2 * side, side, side]


def _prepare_append(case, g):
    T, H, D, bs = case["tokens"], case["kv_heads"], case["dim"], case["block"]
    blocks = -(-T // bs) + 4
    # one projection's output holds the queries, keys and values of a token side by side
    qkv = _randn(g, (T, case["heads"] + 2 * H, D), case["dtype"])
    cache, k_scale, v_scale = _random_cache(g, case, blocks)
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:T]
    if case["pad"]:                                   # a padded batch: its last tokens have no slot
        slots[max(1, T - case["pad"]):] = -1
    t = torch.arange(T, device="cuda")
    start = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
    image = (t % 1024) >= 256                         # text, then an image of 32 columns
    cell = (t % 1024) - 256
    axis = [start + t, torch.where(image, start + t - cell + cell // 32, start + t),
            torch.where(image, start + t - cell + cell % 32, start + t)]
    positions = torch.stack(axis[: case["axes"]]).to(torch.int32).contiguous()
    s = dict(case=case, qkv=qkv, q=qkv[:, : case["heads"]], k=qkv[:, case["heads"]: case["heads"] + H],
             v=qkv[:, case["heads"] + H:], slots=slots, positions=positions, cache=cache, k_scale=k_scale,
             v_scale=v_scale, q_out=torch.zeros((T, case["heads"], D), dtype=TORCH[case["dtype"]], device="cuda"),
             status=_ints([0]))
    if own:
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_append(
            s["q"], s["k"], s["v"], positions, slots, api.make_rope(case["theta"], case["style"]),
            api.make_cache_desc(bs, blocks, case["cache"], k_scale, v_scale), cache, s["q_out"], s["status"],
            axes=api.make_axes(_sections(case)))
    return s


def _prepare_attend(case, g):
    lens = _lengths(case)
    bs, T = case["block"], sum(m for _, m in lens)
    taken = [-(-n // bs) for n, _ in lens]
    width, blocks = max(taken) + 3, sum(taken) + 4
    cache, k_scale, v_scale = _random_cache(g, case, blocks)
    ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < _ints(taken)[:, None]] = ids[: sum(taken)]
    starts = [0]
    for _, m in lens:
        starts.append(starts[-1] + m)
    s = dict(case=case, q=_randn(g, (T, case["heads"], case["dim"]), case["dtype"]), cache=cache, k_scale=k_scale,
             v_scale=v_scale, table=table, seq_len=_ints([n for n, _ in lens]), start=_ints(starts),
             out=torch.zeros((T, case["heads"], case["dim"]), dtype=TORCH[case["dtype"]], device="cuda"),
             lse=torch.zeros((T, case["heads"]), dtype=torch.float32, device="cuda"), status=_ints([0]),
             workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda"))
    if own:
        from kv_cache_injection_gb300 import api
        s["call"] = api.prepare_attend(
            s["q"], s["seq_len"], table, api.make_cache_desc(bs, blocks, case["cache"], k_scale, v_scale), cache,
            s["out"], s["workspace"], s["status"], q_start=s["start"], max_q_len=case["new_max"],
            scale=case["dim"] ** -0.5, window=case["window"], lse_out=s["lse"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        if op == "blocks":
            return s["table"], s["slots"], s["positions"], s["start"], s["seq_out"], s["head_out"]
        if op == "append":
            return s["q_out"], _cache_values(s["case"], s["cache"])
        return s["out"], s["lse"]
    return {"blocks": _plain_blocks, "append": _plain_append, "attend": _plain_attend}[op](s)


def _cache_values(case, cache):
    return cache.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else cache


def _plain_blocks(s):
    bs, table, seq, new = s["case"]["block"], s["table"], s["seq_len"], s["new_len"]
    have, need = (seq + bs - 1) // bs, (seq + new + bs - 1) // bs
    missing = need - have
    first = s["head"] + torch.cumsum(missing, 0) - missing
    column = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (column >= have[:, None]) & (column < need[:, None])
    take = (first[:, None] + column - have[:, None]).clamp(0, s["free"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free"][take], table))
    end = torch.cumsum(new, 0)
    start = torch.cat([torch.zeros_like(end[:1]), end]).to(torch.int32)
    t = torch.arange(s["slots"].shape[0], device="cuda")
    r = torch.searchsorted(end, t, right=True).clamp(max=seq.shape[0] - 1)
    position = seq[r] + t - start[r]
    inside = t < end[-1]
    at = torch.where(inside, position, 0)
    slots = torch.where(inside, table[r, at // bs].long() * bs + at % bs, -1)
    s["positions"].copy_(torch.where(inside, position, s["positions"]))
    return table, slots, s["positions"], start, (seq + new).to(torch.int32), (s["head"] + missing.sum()).to(torch.int32)


def _rotate(x, cos, sin, style):
    """x [T][heads][D] in 32 bits, cos and sin [T][D / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    if style == 0:
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_append(s):
    case = s["case"]
    D, half = case["dim"], case["dim"] // 2
    pair = torch.arange(half, device="cuda", dtype=torch.float64)
    frequency = case["theta"] ** (-2.0 * pair / D)
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), _ints(_sections(case)), output_size=half)
    angle = s["positions"].double()[axis].T * frequency          # [T][half]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    put = s["slots"] >= 0
    q = _rotate(s["q"].float(), cos, sin, case["style"]).to(s["q_out"].dtype)
    s["q_out"].copy_(torch.where(put[:, None, None], q, s["q_out"]))
    k, v = _rotate(s["k"].float(), cos, sin, case["style"]), s["v"].float()
    flat = s["cache"].view(2, -1, case["kv_heads"], D)
    spare = flat.shape[1] - 1
    at = torch.where(put, s["slots"], spare)          # unslotted tokens write back what the last slot holds
    if case["cache"] == "e4m3":
        k = (k * (1.0 / s["k_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v * (1.0 / s["v_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = put[:, None, None]
    if case["pad"]:
        hold = (at == spare) & put                    # the last slot may be some token's own
        own_k = torch.where(hold[:, None, None], k.to(flat.dtype), 0).sum(0, dtype=torch.float32).to(flat.dtype)
        own_v = torch.where(hold[:, None, None], v.to(flat.dtype), 0).sum(0, dtype=torch.float32).to(flat.dtype)
        flat[0, spare] = torch.where(hold.any(), own_k, flat[0, spare])
        flat[1, spare] = torch.where(hold.any(), own_v, flat[1, spare])
    flat[0, at] = torch.where(keep, k.to(flat.dtype), flat[0, spare])
    flat[1, at] = torch.where(keep, v.to(flat.dtype), flat[1, spare])
    return s["q_out"], _cache_values(case, s["cache"])


def _plain_attend(s):
    case = s["case"]
    bs, D, H = case["block"], case["dim"], case["kv_heads"]
    G, R, N, T = case["heads"] // H, case["requests"], case["new_max"], s["q"].shape[0]
    table, seq, start = s["table"], s["seq_len"].long(), s["start"].long()
    key = torch.arange(table.shape[1] * bs, device="cuda")
    block = table[:, key // bs].long()
    at = block.clamp(min=0) * bs + key % bs           # [R][S]
    rows = _cache_values(case, s["cache"]).view(2, -1, H, D)
    if case["cache"] == "e4m3":
        rows = rows.view(torch.uint8)
        k = rows[0][at].view(torch.float8_e4m3fn).float() * s["k_scale"]
        v = rows[1][at].view(torch.float8_e4m3fn).float() * s["v_scale"]
    else:
        k, v = rows[0][at].float(), rows[1][at].float()
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
    return o[r, t - start[r]].to(s["q"].dtype), lse[r, t - start[r]]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "blocks":
        lens = _lengths(case)
        tokens, bs = sum(m for _, m in lens), case["block"]
        fresh = sum(-(-(n + m) // bs) - -(-n // bs) for n, m in lens)
        return {"bytes": 12 * (tokens + 7) + 8 * fresh + 20 * len(lens) + 8, "flops": 0}
    H, D = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        T, e, f = case["tokens"], SIZE[case["dtype"]], SIZE[case["cache"]]
        return {"bytes": T * (D * (2 * case["heads"] * e + 2 * H * e + 2 * H * f) + 8 + 4 * case["axes"]),
                "flops": 3 * T * D * (case["heads"] + H)}
    lens = _lengths(case)
    reach = case["window"] or 1 << 40
    pairs = sum(min(n - m + i + 1, reach) for n, m in lens for i in range(m))
    keys = sum(min(n, m - 1 + reach) for n, m in lens if m)
    tokens = sum(m for _, m in lens)
    return {"bytes": 2 * keys * H * D * SIZE[case["cache"]] + tokens * case["heads"] * (2 * D * SIZE[case["dtype"]] + 4),
            "flops": 4 * pairs * case["heads"] * D}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "blocks":
        return None                                   # whole numbers
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_attend(case, s)


def _as_double(case, stored):
    if case["cache"] == "e4m3":
        return stored.view(torch.float8_e4m3fn).to(torch.float64)
    return stored.to(torch.float64)


def _exact_append(case, s):
    D = case["dim"]
    owner = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
    i = torch.arange(D // 2, dtype=torch.float64, device="cuda")
    turn = s["positions"].to(torch.float64)[owner] * torch.exp(-math.log(case["theta"]) * 2 * i / D)[:, None]
    unit = torch.polar(torch.ones_like(turn), turn).T[:, None]   # [T][1][D / 2]

    def turned(x):
        x = x.to(torch.float64)
        if case["style"] == 1:
            return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], D // 2, 2)) * unit).flatten(-2)
        z = torch.complex(x[..., : D // 2], x[..., D // 2:]) * unit
        return torch.cat([z.real, z.imag], -1)

    slotted = torch.nonzero(s["slots"] >= 0)[:, 0]
    q = s["q_out"].to(torch.float64)
    q[slotted] = turned(s["q"])[slotted]
    cache = _as_double(case, s["cache"])
    rows = cache.view(2, -1, case["kv_heads"], D)
    rows[0, s["slots"][slotted]] = turned(s["k"])[slotted] / s["k_scale"]
    rows[1, s["slots"][slotted]] = s["v"].to(torch.float64)[slotted] / s["v_scale"]
    return q, cache


def _exact_attend(case, s):
    H, D, bs = case["kv_heads"], case["dim"], case["block"]
    G = case["heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for r, (n, m) in enumerate(_lengths(case)):
        if m == 0:
            continue
        first = max(0, n - m + 1 - case["window"]) if case["window"] else 0
        at = torch.arange(first, n, device="cuda")
        slot = s["table"][r, at // bs].long() * bs + at % bs
        k, v = (_as_double(case, half.reshape(-1, H, D)[slot]) * f
                for half, f in zip(s["cache"], (s["k_scale"], s["v_scale"])))
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
