"""is_append_scaled, is_move_scaled, is_read_scaled and is_attend_scaled refuse bad
arguments on the host, before anything reaches a device (no GPU is needed)."""
import ctypes

import pytest

from kv_cache_injection_gb300 import _lib, api, build
from tests.test_serve_refusals import INVALID, UNSUPPORTED, addr, append_args, attend_args

CODES = api.make_cache_desc(16, 8, "int8")
SCALES = addr(20)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def fields(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def move_args(**kw):
    return fields(_lib.MoveArgs(3, 2, 64, _lib.IS_BF16, *[addr(i) for i in range(6)], api.make_cache_desc(16, 8, "bf16"),
                                CODES, (ctypes.c_int32 * 2)(0, 0)), kw)


def read_args(**kw):
    return fields(_lib.ReadArgs(3, 2, 64, _lib.IS_BF16, 1, 0, *[addr(i) for i in range(7)], api.make_rope(1e4),
                                api.make_axes(), CODES, 0), kw)


def call(lib, name, args, scales=SCALES):
    ref = ctypes.byref(args) if args is not None else None
    if name in ("is_append_scaled", "is_attend_scaled"):
        return getattr(lib, name)(ref, scales, None)
    if name == "is_attend_scaled_within":
        return lib.is_attend_scaled_within(ref, scales, 5, None)
    return getattr(lib, name)(ref, None)


@pytest.mark.parametrize("name", ["is_append_scaled", "is_move_scaled", "is_read_scaled", "is_attend_scaled",
                                  "is_attend_scaled_within"])
def test_null_args(lib, name):
    assert call(lib, name, None) == INVALID


BAD_CACHES = [(api.make_cache_desc(16, 8, "bf16"), INVALID), (api.make_cache_desc(16, 8, 7), INVALID),
              (api.make_cache_desc(0, 8, "int8"), INVALID), (api.make_cache_desc(16, 0, "e4m3"), INVALID),
              (api.make_cache_desc((1 << 24) + 1, 8, "int8"), INVALID), (api.make_cache_desc(16, 8, "int8", 0.5), INVALID),
              (api.make_cache_desc(16, 8, "e4m3", 1.0, 2.0), INVALID)]


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_bad_caches(lib, cache, status):
    assert call(lib, "is_append_scaled", append_args(cache=cache)) == status
    assert call(lib, "is_move_scaled", move_args(cache=cache)) == status
    assert call(lib, "is_read_scaled", read_args(cache=cache)) == status
    assert call(lib, "is_attend_scaled", attend_args(cache=cache)) == status
    assert lib.is_last_error_message()


def test_plain_calls_refuse_int8(lib):
    assert lib.is_append(ctypes.byref(append_args(cache=CODES)), None) == INVALID
    assert lib.is_attend(ctypes.byref(attend_args(cache=CODES)), None) == INVALID


@pytest.mark.parametrize("field", ["q", "k", "v", "positions", "slot_mapping", "q_out", "layer_cache", "status_out"])
def test_append_needs_its_pointers(lib, field):
    assert call(lib, "is_append_scaled", append_args(cache=CODES, **{field: None})) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(dtype=4), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(q_stride=500), INVALID),
    (dict(layer_cache=addr(6) + 8), INVALID), (dict(q_out=addr(1)), INVALID), (dict(rope=api.make_rope(0.5)), INVALID),
    (dict(axes=api.make_axes([8, 8, 8])), INVALID), (dict(k=SCALES), INVALID), (dict(layer_cache=SCALES - 2 * 8 * 16 * 2 * 64 + 16), INVALID)])
def test_append_refuses(lib, kw, status):
    assert call(lib, "is_append_scaled", append_args(**{"cache": CODES, **kw})) == status
    assert lib.is_last_error_message()


def test_scales_are_needed(lib):
    assert call(lib, "is_append_scaled", append_args(cache=CODES), SCALES + 2) == INVALID
    assert call(lib, "is_attend_scaled", attend_args(cache=CODES), SCALES + 1) == INVALID
    assert call(lib, "is_move_scaled", move_args(scales=SCALES + 2)) == INVALID
    assert call(lib, "is_read_scaled", read_args(scales=SCALES + 2)) == INVALID
    assert call(lib, "is_append_scaled", append_args(cache=CODES), None) == INVALID
    assert call(lib, "is_attend_scaled", attend_args(cache=CODES), None) == INVALID
    assert call(lib, "is_attend_scaled", attend_args(cache=CODES, out=SCALES)) == INVALID


@pytest.mark.parametrize("field", ["from_slots", "slot_mapping", "from_cache", "layer_cache", "scales", "status_out"])
def test_move_needs_its_pointers(lib, field):
    assert call(lib, "is_move_scaled", move_args(**{field: None})) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=48), UNSUPPORTED), (dict(dtype=3), INVALID),
    (dict(dtype=_lib.IS_F16), INVALID), (dict(from_=api.make_cache_desc(16, 8, "e4m3")), UNSUPPORTED),
    (dict(from_=api.make_cache_desc(0, 8, "bf16")), INVALID), (dict(from_cache=addr(2) + 8), INVALID),
    (dict(layer_cache=addr(3) + 4), INVALID), (dict(scales=addr(3) + 64), INVALID), (dict(layer_cache=addr(2)), INVALID),
    (dict(status_out=addr(4) + 4), INVALID), (dict(reserved=(ctypes.c_int32 * 2)(0, 1)), INVALID),
    (dict(dtype=_lib.IS_F32, head_dim=512, from_=api.make_cache_desc(16, 8, "f32")), UNSUPPORTED)])
def test_move_refuses(lib, kw, status):
    assert call(lib, "is_move_scaled", move_args(**kw)) == status
    assert lib.is_last_error_message()


@pytest.mark.parametrize("field", ["slot_mapping", "positions", "layer_cache", "scales", "status_out"])
def test_read_needs_its_pointers(lib, field):
    assert call(lib, "is_read_scaled", read_args(**{field: None})) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=8), UNSUPPORTED), (dict(dtype=4), INVALID),
    (dict(unrotate=2), INVALID), (dict(reserved=1), INVALID), (dict(reserved2=1), INVALID), (dict(k_out=None, v_out=None), INVALID),
    (dict(k_out=addr(4) + 8), INVALID), (dict(v_out=addr(4)), INVALID), (dict(v_out=addr(2)), INVALID),
    (dict(rope=api.make_rope(1e4, style=2)), INVALID), (dict(axes=_lib.RopeAxes(0)), INVALID),
    (dict(dtype=_lib.IS_F32, head_dim=512), UNSUPPORTED), (dict(rope=api.make_rope(1e4, style=1), head_dim=512), UNSUPPORTED)])
def test_read_refuses(lib, kw, status):
    assert call(lib, "is_read_scaled", read_args(**kw)) == status
    assert lib.is_last_error_message()


def test_calls_of_nothing_are_ok(lib):
    assert call(lib, "is_append_scaled", append_args(num_tokens=0, cache=CODES, k=None)) == 0
    assert call(lib, "is_move_scaled", move_args(num_tokens=0, from_cache=None, layer_cache=None)) == 0
    assert call(lib, "is_read_scaled", read_args(num_tokens=0, k_out=None, unrotate=0, rope=_lib.RopeParams())) == 0
    assert call(lib, "is_attend_scaled", attend_args(num_tokens=0, cache=CODES)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=_lib.IS_F32), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(out=addr(5) + 16), INVALID), (dict(q=None), INVALID),
    (dict(workspace_bytes=_lib.IS_ATTEND_WORKSPACE_BYTES - 1), INVALID), (dict(reserved=1), INVALID)])
def test_attend_refuses(lib, kw, status):
    assert call(lib, "is_attend_scaled", attend_args(**{"cache": CODES, **kw})) == status
    assert lib.is_last_error_message()


@pytest.mark.parametrize("budget", [-1, 2_000_000_001])
def test_attend_within_refuses_budgets(lib, budget):
    args = attend_args(num_tokens=0, cache=CODES)
    assert lib.is_attend_scaled_within(ctypes.byref(args), SCALES, budget, None) == INVALID
    assert lib.is_attend_scaled_within(ctypes.byref(args), SCALES, 0, None) == 0


def test_host_tensors_are_refused_by_the_binding():
    import torch
    x = torch.zeros(1, 2, 64)
    i, sc = torch.zeros(1, dtype=torch.int32), torch.ones(2, 8, 2)
    codes = torch.zeros(2, 8, 16, 2, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        api.is_append_scaled(x, x, x, i, i.long(), api.make_rope(1e4), CODES, codes, sc, x, i)
    with pytest.raises(ValueError):
        api.is_move_scaled(api.make_cache_desc(16, 8, "f32"), codes.float(), i.long(), CODES, codes, sc, i.long(), i)
    with pytest.raises(ValueError):
        api.is_read_scaled(i.long(), CODES, codes, sc, x, x, i)
    with pytest.raises(ValueError):
        api.is_attend_scaled(x, i, i.view(1, 1), CODES, codes, sc, x, i, i)


def test_struct_layouts():
    assert [ctypes.sizeof(c) for c in (_lib.MoveArgs, _lib.ReadArgs)] == [112, 176]
