"""The rules by which la_delta_extend lays a batch over the SMs (la_delta_plan.h), for any number of SMs:
compiled by the host's compiler, without CUDA and without a GPU."""
import ctypes
import os
import subprocess

import pytest

from lightning_attention_gb300 import _build

SHIM = r"""
#include "la_delta_plan.h"
extern "C" void schedule(long long B, long long T, long long H, long long max_seqlen, int sms, int *r) {
    const la::Schedule s = la::make_schedule(B, T, H, max_seqlen, sms);
    r[0] = s.planned;
    r[1] = s.cut.segs;
    r[2] = s.cut.ratio;
    r[3] = s.ranked;
}
extern "C" int last_segment(int segs, int ratio, int nchunks) {
    return la::split_last(la::Cut{segs, ratio}, nchunks);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cc").write_text(SHIM)
    so = os.path.join(d, "shim.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-Werror", "-I", _build.CSRC,
                    str(d / "shim.cc"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.schedule.argtypes = [ctypes.c_longlong] * 4 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    lib.schedule.restype = None

    def schedule(B, T, H, max_seqlen=None, sms=152):
        r = (ctypes.c_int * 4)()
        lib.schedule(B, T, H, T if max_seqlen is None else max_seqlen, sms, r)
        return dict(planned=bool(r[0]), segs=r[1], ratio=r[2], ranked=bool(r[3]))

    schedule.last_segment = lib.last_segment
    return schedule


@pytest.mark.parametrize("sms", [1, 18, 19, 40, 75, 76, 100, 152])
def test_a_split_batch_is_never_ranked(plan, sms):
    """The join finds a chain's segments by the request's place in the batch, so a batch that is split has
    to keep its order whatever the number of SMs; a batch is split, planned or taken whole, and only whole
    chains are ranked."""
    split = 0
    for B in (1, 2, 3, 7, 38, 76, 129):
        for H in (1, 2, 10, 38, 76):
            for longest in (64, 1216, 1217, 2300, 5000, 40000):
                s = plan(B, longest + 40 * (B - 1), H, longest, sms)
                assert not (s["ranked"] and (s["segs"] > 1 or s["planned"])), (B, H, longest, s)
                assert not (s["planned"] and s["segs"] > 1)
                split += s["segs"] > 1
                if s["segs"] == 1 and not s["planned"]:
                    assert s["ranked"] == (B > 1 and B * H > sms), (B, H, longest, s)
    assert split > 40


@pytest.mark.parametrize("chains,first", [(1, 1217), (8, 1217), (16, 1217), (32, 1473), (51, 2753), (76, 2753)])
def test_onset_of_a_split(plan, chains, first):
    """From which length on a request is cut into segments, as the header states it: only lengths within 400
    tokens above the first stay whole."""
    segs = lambda n: plan(1, n, chains)["segs"]  # noqa: E731
    assert all(segs(n) == 1 for n in range(1, first, 7)) and segs(first - 1) == 1
    assert segs(first) > 1
    assert all(segs(n) > 1 for n in range(first + 400, 40000, 61))
    assert plan(77, 40000, 1, 1217)["segs"] == 1 and plan(1, 40000, 77)["segs"] == 1


def test_onset_of_a_plan(plan):
    """A skewed batch of more than 76 pairs and 2 to 128 requests is planned from 1,985 tokens on."""
    assert not plan(100, 1984 + 99, 1, 1984)["planned"] and plan(100, 1985 + 99, 1, 1985)["planned"]
    assert not plan(129, 4000, 1, 3000)["planned"] and plan(128, 4000, 1, 3000)["planned"]
    assert not plan(1, 40000, 128)["planned"] and not plan(2, 40000, 38)["planned"]
    # at least twice the SMs' share of all chunks, 8 added to it
    for rest in range(0, 60000, 500):
        s = plan(100, 4096 + rest, 4, 4096)
        assert s["planned"] == (64 * 152 >= 2 * (4 * ((4096 + rest + 63) // 64) + 8 * 152)), rest
