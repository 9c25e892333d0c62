"""The plan of the embedding gradient's sort on devices of any number of SMs
(a partition of a GPU has few): only rows that a helper clears count as cleared,
the cluster fits the device, and it holds all tokens or the call is refused."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
THREADS, MOST_ITEMS = 1024, 16


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("needs a C++ compiler")
    from collective_reduction_math_gb300 import _build
    so = str(tmp_path_factory.mktemp("native") / "sort_plan.so")
    subprocess.run([cc, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, "-o", so,
                    os.path.join(HERE, "native", "sort_plan.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.sort_plan.argtypes = [ctypes.c_size_t] * 5 + [ctypes.c_int] * 3 + [ctypes.c_void_p]

    def call(rows, vocab=131072, hidden=256, g_bytes=2, table_bytes=4, accumulate=0, sms=152, most=16):
        out = (ctypes.c_int * 5)()
        lib.sort_plan(rows, vocab, hidden, g_bytes, table_bytes, accumulate, sms, most, out)
        return dict(zip(("cluster", "items", "helpers", "ahead", "cleared"), out))
    return call


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 76, 152])
@pytest.mark.parametrize("most", [8, 16])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_any_device(plan, sms, most, accumulate):
    for rows in (0, 1, 777, 1024, 1025, 8192, 16384, 32768, 32769, 65536, 131072, 131073, 262144):
        p = plan(rows, sms=sms, most=most, accumulate=accumulate)
        if p["cluster"] == 0:
            # as many CTAs as there may be, with all that they hold, are not enough
            widest = max(c for c in (1, 2, 4, 8, 16) if c <= min(sms, most if rows > 32768 else 8))
            assert rows > THREADS * widest * MOST_ITEMS
            continue
        assert p["cluster"] <= min(sms, most)
        assert p["cluster"] * p["items"] * THREADS >= rows
        assert 0 <= p["helpers"] <= sms // p["cluster"] - 1
        # who clears or asks ahead is there
        assert p["helpers"] > 0 or (p["cleared"] == 0 and p["ahead"] == 0)
        assert p["cleared"] % 8 == 0 and p["cleared"] * 256 * 4 <= 48 << 20
        assert accumulate == 0 or p["cleared"] == 0
        assert p["ahead"] <= rows


def test_whole_device(plan):
    """152 SMs with clusters of 16: what the sizes of the calls call for."""
    assert plan(0) == {"cluster": 1, "items": 1, "helpers": 151, "ahead": 0, "cleared": 49152}
    assert plan(16384) == {"cluster": 8, "items": 2, "helpers": 18, "ahead": 16384, "cleared": 49152}
    assert plan(32769) == {"cluster": 16, "items": 4, "helpers": 8, "ahead": 32769, "cleared": 49152}
    assert plan(262144, accumulate=1) == {"cluster": 16, "items": 16, "helpers": 8, "ahead": 262144, "cleared": 0}
    # without clusters of 16, half of the rows
    assert plan(131072, most=8)["cluster"] == 8 and plan(131073, most=8)["cluster"] == 0
    # rows too large for either
    assert plan(777, hidden=(1 << 31) - 1) == {"cluster": 1, "items": 1, "helpers": 0, "ahead": 0, "cleared": 0}
