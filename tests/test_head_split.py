"""How the normed heads' kernels share a token's heads among their threads: checked with the host compiler, without a GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_decoder_layer_llama_gb300", "csrc")
SOURCE = """
#include "head_split.h"
extern "C" void split(int lanes, int heads, int per_thread, int threads, int* out) {
    const ll::HeadSplit s = ll::head_split(lanes, heads, per_thread, threads);
    out[0] = s.lanes; out[1] = s.width; out[2] = s.rows; out[3] = s.parts; out[4] = s.slots; out[5] = s.threads;
}
extern "C" int first(int rows, int part, int row, int per_thread) {
    ll::HeadSplit s{};
    s.rows = rows;
    return ll::first_head(s, part, row, per_thread);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("split")
    (d / "split.cc").write_text(SOURCE)
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", CSRC, str(d / "split.cc"), "-o", str(d / "split.so")],
                   check=True)
    return ctypes.CDLL(str(d / "split.so"))


def split(lib, *args):
    out = (ctypes.c_int * 6)()
    lib.split(*args, out)
    return dict(zip(("lanes", "width", "rows", "parts", "slots", "threads"), out))


@pytest.mark.parametrize("per_thread,threads", [(3, 256), (6, 256), (2, 128), (4, 128)])
def test_every_head_is_some_threads(lib, per_thread, threads):
    """Every head belongs to one (turn, group, place), within a CTA's threads."""
    for lanes in (1, 4, 5, 9, 17, 31, 32):
        for heads in [*range(1, 140), 255, 295, 540, 541, 1000, 1261, 4095, 4096]:
            s = split(lib, lanes, heads, per_thread, threads)
            assert s["lanes"] <= s["width"] <= 32 and s["slots"] * s["rows"] * s["width"] <= s["threads"] <= threads
            part, row, u = np.meshgrid(range(s["parts"]), range(s["rows"]), range(per_thread), indexing="ij")
            h = part * s["rows"] * per_thread + row + u * s["rows"]
            assert sorted(h[h < heads].tolist()) == list(range(heads))
            last = s["parts"] - 1
            assert lib.first(s["rows"], last, s["rows"] - 1, per_thread) == h[last, -1, 0]


@pytest.mark.parametrize("lanes,heads,per_thread", [(32, 127, 3), (16, 541, 3), (32, 295, 6), (16, 1261, 6)])
def test_groups_without_a_head(lib, lanes, heads, per_thread):
    """The last turn of these has groups whose first head is behind the last: what they would read for it (a gain that the
    call does not have) must not be read.  They are the smallest such sizes of their forms."""
    def none(n):
        s = split(lib, lanes, n, per_thread, 256)
        return lib.first(s["rows"], s["parts"] - 1, s["rows"] - 1, per_thread) >= n
    assert none(heads) and not any(none(n) for n in range(1, heads))
