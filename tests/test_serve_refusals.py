"""is_extend_block_table, is_append and is_attend refuse bad arguments on the
host, before anything reaches a device (no GPU is needed)."""
import ctypes

import pytest

from kv_cache_injection_gb300 import _lib, api, build

INVALID, UNSUPPORTED = 1, 8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# Fake device addresses, 1 GiB apart: nothing reads them.
def addr(i):
    return (i + 1) << 30


def extend_args(**kw):
    a = _lib.ExtendArgs(4, 10, 16, 64, 8, 32, *[addr(i) for i in range(11)])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append_args(**kw):
    a = _lib.AppendArgs(3, 8, 2, 64, _lib.IS_BF16, 0, 512, 128, 128, *[addr(i) for i in range(8)],
                        api.make_rope(1e4), api.make_axes(), api.make_cache_desc(16, 8, "bf16"), 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend_args(**kw):
    a = _lib.AttendArgs(3, 3, 1, 8, 2, 64, _lib.IS_BF16, 4, 0, 0.125, 512, *[addr(i) for i in range(8)],
                        _lib.IS_ATTEND_WORKSPACE_BYTES, addr(8), api.make_cache_desc(16, 8, "bf16"), 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def status_of(lib, name, args):
    return getattr(lib, name)(ctypes.byref(args) if args is not None else None, None)


@pytest.mark.parametrize("name", ["is_extend_block_table", "is_append", "is_attend"])
def test_null_args(lib, name):
    assert status_of(lib, name, None) == INVALID


@pytest.mark.parametrize("field", ["seq_len", "new_len", "free_blocks", "block_table", "slot_mapping_out", "status_out"])
def test_extend_needs_its_pointers(lib, field):
    assert status_of(lib, "is_extend_block_table", extend_args(**{field: None})) == INVALID


@pytest.mark.parametrize("kw", [
    dict(num_requests=0), dict(num_requests=4097), dict(num_free=-1), dict(block_size=0), dict(num_blocks=0),
    dict(block_size=(1 << 24) + 1), dict(max_blocks_per_seq=0), dict(max_tokens=0),
    dict(seq_len_out=addr(0)), dict(free_head_out=addr(3)), dict(positions_out=addr(5) + 8),
    dict(status_out=addr(4) + 4)])
def test_extend_refuses(lib, kw):
    assert status_of(lib, "is_extend_block_table", extend_args(**kw)) == INVALID
    assert lib.is_last_error_message()


@pytest.mark.parametrize("field", ["q", "k", "v", "positions", "slot_mapping", "q_out", "layer_cache", "status_out"])
def test_append_needs_its_pointers(lib, field):
    assert status_of(lib, "is_append", append_args(**{field: None})) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(num_q_heads=-1), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=9), INVALID), (dict(reserved=1), INVALID), (dict(reserved2=1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=8), UNSUPPORTED), (dict(head_dim=1024), UNSUPPORTED),
    (dict(dtype=_lib.IS_F16), INVALID), (dict(q_stride=500), INVALID), (dict(k_stride=132), INVALID),
    (dict(v_stride=120), INVALID), (dict(q=addr(0) + 2), INVALID), (dict(layer_cache=addr(6) + 8), INVALID),
    (dict(q_out=addr(1)), INVALID), (dict(q_out=addr(0) + 16), INVALID), (dict(status_out=addr(6) + 64), INVALID),
    (dict(q_out=addr(0), q_stride=1024), INVALID),
    (dict(cache=api.make_cache_desc(0, 8, "bf16")), INVALID), (dict(cache=api.make_cache_desc(16, 0, "bf16")), INVALID),
    (dict(cache=api.make_cache_desc(16, 8, "e4m3", 0.0, 1.0)), INVALID),
    (dict(cache=api.make_cache_desc(16, 8, "e4m3", 1.0, float("inf"))), INVALID),
    (dict(cache=api.make_cache_desc(16, 8, "f16")), INVALID),
    (dict(dtype=_lib.IS_F32, cache=api.make_cache_desc(16, 8, "e4m3")), UNSUPPORTED),
    (dict(rope=api.make_rope(0.5)), INVALID), (dict(rope=api.make_rope(1e4, style=2)), INVALID),
    (dict(rope=api.make_rope(1e4, style=1), head_dim=512, q_stride=4096, k_stride=1024, v_stride=1024), UNSUPPORTED),
    (dict(axes=_lib.RopeAxes(0)), INVALID), (dict(axes=_lib.RopeAxes(4)), INVALID),
    (dict(axes=api.make_axes([8, 8, 8])), INVALID), (dict(axes=api.make_axes([40, -8])), INVALID),
    (dict(axes=api.make_axes([0, 32], interleaved=True)), INVALID),
    (dict(axes=_lib.RopeAxes(1, 2)), INVALID)])
def test_append_refuses(lib, kw, status):
    assert status_of(lib, "is_append", append_args(**kw)) == status
    assert lib.is_last_error_message()


def test_append_of_nothing_is_ok(lib):
    assert status_of(lib, "is_append", append_args(num_tokens=0, k=None, v=None, q=None)) == 0


def test_append_checks_a_changed_axis_table_again(lib):
    """The turns of the last parameters are kept by value: a refusal in between does not leak into them."""
    ok, bad = append_args(num_tokens=0), append_args(num_tokens=0, axes=api.make_axes([1, 2, 3]))
    assert [status_of(lib, "is_append", a) for a in (ok, bad, ok, bad)] == [0, INVALID, 0, INVALID]


@pytest.mark.parametrize("field", ["q", "seq_len", "block_table", "layer_cache", "out", "workspace", "status_out"])
def test_attend_needs_its_pointers(lib, field):
    assert status_of(lib, "is_attend", attend_args(**{field: None})) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=0), INVALID), (dict(num_requests=4097), INVALID), (dict(num_tokens=-1), INVALID),
    (dict(max_q_len=0), INVALID), (dict(num_q_heads=7), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(dtype=3), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(head_dim=32), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED), (dict(q_stride=508), INVALID),
    (dict(q=addr(0) + 8), INVALID), (dict(out=addr(5) + 4), INVALID), (dict(workspace=addr(7) + 8), INVALID),
    (dict(out=addr(5) + 16), INVALID), (dict(workspace=addr(7) + 16), INVALID),
    (dict(workspace_bytes=_lib.IS_ATTEND_WORKSPACE_BYTES - 1), INVALID), (dict(out=addr(0)), INVALID),
    (dict(lse_out=addr(5)), INVALID), (dict(workspace=addr(4)), INVALID), (dict(reserved=2), INVALID),
    (dict(q_start=None, num_requests=4), INVALID), (dict(cache=api.make_cache_desc(16, 8, "f32")), INVALID),
    (dict(dtype=_lib.IS_F32, cache=api.make_cache_desc(16, 8, "e4m3")), UNSUPPORTED),
    (dict(cache=api.make_cache_desc(1 << 25, 8, "bf16")), INVALID)])
def test_attend_refuses(lib, kw, status):
    assert status_of(lib, "is_attend", attend_args(**kw)) == status
    assert lib.is_last_error_message()


def test_attend_of_no_rows_is_ok(lib):
    assert status_of(lib, "is_attend", attend_args(num_tokens=0)) == 0


def test_host_tensors_are_refused_by_the_binding():
    import torch
    x = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.is_extend_block_table(x, x, x, 16, 4, x.view(1, 2), torch.zeros(3, dtype=torch.int64), status_out=x[:1])
    with pytest.raises(ValueError):
        api.make_axes([1, 2, 3, 4])
    with pytest.raises(ValueError):
        api.is_attend(torch.zeros(1, 2, 64), x, x.view(2, 1), api.make_cache_desc(16, 1, "f32"),
                      torch.zeros(2, 1, 16, 2, 64), torch.zeros(1, 2, 64), x, x[:1])


def test_struct_layouts():
    assert [ctypes.sizeof(c) for c in (_lib.RopeAxes, _lib.ExtendArgs, _lib.AppendArgs, _lib.AttendArgs)] == \
        [24, 112, 208, 152]
