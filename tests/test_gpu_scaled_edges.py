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
