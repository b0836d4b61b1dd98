"""How a write into a scaled cache is spread over CTAs: the host code of the library, compiled by itself (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

from kv_cache_injection_gb300 import build

FIELDS = ["window", "heads_of", "rows", "share", "group_ctas", "query_ctas", "turns", "smem"]
SHELL = """
#include "scaled_plan.h"
extern "C" void plan(int T, int Hq, int H, int D, int bytes, int bs, int sms, int rotate, long long* out) {
  const isk::scaled::WritePlan w = isk::scaled::plan_write(T, Hq, H, D, bytes, bs, sms, rotate != 0);
  const long long v[] = {w.window, w.heads_of, w.rows, w.share, w.group_ctas, w.query_ctas, w.turns, (long long)w.smem};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SHELL)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", build.CSRC,
                    str(at / "plan.cpp"), "-o", str(at / "plan.so")], check=True)
    lib = ctypes.CDLL(str(at / "plan.so"))

    def call(T, Hq, H, D, bytes=2, bs=16, sms=152, rotate=True):
        out = (ctypes.c_longlong * 8)()
        lib.plan(T, Hq, H, D, bytes, bs, sms, int(rotate), out)
        return dict(zip(FIELDS, out))
    return call


SHAPES = [(Hq, H, D, b) for Hq, H, D in ((32, 8, 128), (28, 4, 128), (0, 8, 128), (1, 1, 16), (8, 8, 64), (3, 17, 64), (8, 4, 256), (2, 1, 512))
          for b in (2, 4) if D * b <= 1024]
LENGTHS = [1, 2, 31, 100, 151, 152, 153, 160, 190, 303, 304, 400, 1000, 2400, 8000, 44000, 1 << 20]


def test_a_device_whose_sms_are_not_known(plan):
    """No division by their number: a plan for one SM."""
    for T in LENGTHS:
        assert plan(T, 32, 8, 128, sms=0) == plan(T, 32, 8, 128, sms=-1) == plan(T, 32, 8, 128, sms=1)


@pytest.mark.parametrize("bs", [1, 7, 16, 32, 64, 130, 1 << 24])
@pytest.mark.parametrize("rotate", [True, False])
def test_every_plan_covers_the_call(plan, bs, rotate):
    for Hq, H, D, b in SHAPES:
        for T in LENGTHS:
            for sms in (1, 152):
                w = plan(T, Hq if rotate else 0, H, D, b, bs, sms, rotate)
                assert 1 <= w["window"] <= 30 and w["heads_of"] in (1, 2, 4) and 4 <= w["rows"] <= 128
                windows = -(-T // w["window"])
                assert w["group_ctas"] == windows * -(-H // w["heads_of"])
                assert w["query_ctas"] == (-(-T * w["share"] // 4) if Hq and rotate else 0)
                assert 0 <= w["turns"] <= min(w["group_ctas"], w["query_ctas"])
                # a round's rows, a largest element for each of their units, their sines; four warps' sines of queries
                need = w["rows"] * (2 * w["heads_of"] * (D * b + 4) + (4 * D if rotate else 0))
                assert w["rows"] * 2 * w["heads_of"] * D * b <= 32768 and w["smem"] >= max(need, 16 * D if rotate else 0)
                assert w["smem"] + 4096 <= 227 * 1024


def places(heads_of, D, bytes, rotate, sms=152):
    """CTAs that 228 KB of shared memory an SM and 64 K registers hold: 92 and 76 registers a thread come in eights."""
    rows = min(128, 32768 // (2 * heads_of * D * bytes))
    smem = max(rows * (2 * heads_of * (D * bytes + 4) + (4 * D if rotate else 0)), 16 * D if rotate else 0)
    return sms * min(65536 // (128 * (96 if rotate else 80)), 228 * 1024 // (smem + 4096))


@pytest.mark.parametrize("Hq,H,D", [(32, 8, 128), (28, 4, 128), (8, 8, 64), (8, 4, 256), (0, 8, 128)])
def test_few_heads_only_where_their_ctas_fit(plan, Hq, H, D):
    """Two heads a CTA where all CTAs fit at once, the queries' beside them, or the groups' take two thirds of the places."""
    for rotate in (True, False):
        for T in list(range(1, 400, 7)) + LENGTHS:
            for bs in (8, 16):
                w = plan(T, Hq if rotate else 0, H, D, bs=bs, rotate=rotate)
                assert w["heads_of"] in ((2, 4) if D * 2 * 4 * bs * 2 <= 32768 else (2,))
                if w["heads_of"] == 2 and D * 2 * 4 * bs * 2 <= 32768:
                    most = places(2, D, 2, rotate)
                    assert w["group_ctas"] <= most
                    assert w["group_ctas"] + w["query_ctas"] <= 5 * 152 or w["query_ctas"] == 0 or 3 * w["group_ctas"] <= 2 * most
            w = plan(T, Hq if rotate else 0, H, D, bs=64, rotate=rotate)
            if w["heads_of"] == 1:
                assert w["window"] > 1 and w["group_ctas"] <= (10 if rotate else 12) * 152


def test_decode_steps_keep_to_the_form_that_fits(plan):
    """Steps of single tokens, 32 + 8 heads: with two heads a CTA 160 of them needed a second wave of CTAs."""
    assert [plan(T, 32, 8, 128)["heads_of"] for T in (1, 100, 120, 140, 160, 190, 305, 1000)] == [2, 2, 2, 4, 4, 4, 4, 4]
    assert [plan(T, 0, 8, 128, rotate=False)["heads_of"] for T in (1, 1276, 3000, 44000)] == [2, 2, 2, 4]
    assert [plan(T, 32, 8, 128, bs=64)["heads_of"] for T in (100, 1276, 8000)] == [2, 1, 2]
