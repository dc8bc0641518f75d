"""CPU-side checks of the gated-delta-rule and packed-store entry points: every refusal happens on the
host before anything is launched, so it runs the same with or without a GPU."""
import ctypes

import pytest
import torch

import lightning_attention_gb300 as la
from lightning_attention_gb300 import _build, binding

OK, BAD16, BAD4 = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8), ctypes.c_void_p(4096 + 2)
N = None


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def extend(lib, q=OK, k=OK, v=OK, rs=(0, 0, 0), g=OK, beta=OK, pool=OK, slots=4, idx=OK, cu=OK, pm=OK,
           out=OK, B=1, T=8, H=2, Hk=1, D=128, ms=8, ws=OK, nbytes=1 << 30):
    return lib.la_delta_extend(q, k, v, *rs, g, beta, pool, slots, idx, cu, pm, out, B, T, H, Hk, D, ms, 0, ws,
                               nbytes, N)


def decode(lib, q=OK, k=OK, v=OK, rs=(0, 0, 0), g=OK, beta=OK, pool=OK, slots=4, idx=OK, out=OK, B=2, H=2,
           Hk=1, D=128):
    return lib.la_delta_decode(q, k, v, *rs, g, beta, pool, slots, idx, out, B, H, Hk, D, 0, N)


def verify(lib, q=OK, k=OK, v=OK, rs=(0, 0, 0), g=OK, beta=OK, pool=OK, slots=4, idx=OK, inter=OK, out=OK,
           B=2, n=3, H=2, Hk=1, D=128):
    return lib.la_delta_verify_chain(q, k, v, *rs, g, beta, pool, slots, idx, inter, out, B, n, H, Hk, D, 0, N)


def pack(lib, pool=OK, slots=4, idx=OK, codes=OK, scales=OK, entries=4, sidx=OK, B=1, H=1, D=128):
    return lib.la_pack_states(pool, slots, idx, codes, scales, entries, sidx, B, H, D, N)


def unpack(lib, pool=OK, slots=4, idx=OK, codes=OK, scales=OK, entries=4, sidx=OK, B=1, H=1, D=128):
    return lib.la_unpack_states(codes, scales, entries, sidx, pool, slots, idx, B, H, D, N)


def test_sizes_and_heads(lib):
    for call in (extend, decode, verify):
        for kw in ({"B": -1}, {"H": 0}, {"Hk": 0}, {"H": 3, "Hk": 2}, {"slots": 0}, {"D": 0}, {"H": 1, "Hk": 2}):
            assert call(lib, **kw) == 1, (call, kw)
        assert call(lib, D=64) == 2
    assert extend(lib, T=-1) == 1 and extend(lib, ms=-1) == 1
    assert verify(lib, n=0) == 1 and verify(lib, B=1 << 20, n=1 << 20) == 1
    for call in (pack, unpack):
        for kw in ({"B": -1}, {"H": 0}, {"slots": 0}, {"entries": 0}, {"D": 0}):
            assert call(lib, **kw) == 1, (call, kw)
        assert call(lib, D=64) == 2


def test_empty_batch_is_a_no_op(lib):
    none = dict(q=N, k=N, v=N, g=N, beta=N, pool=N, idx=N, out=N, B=0)
    assert extend(lib, **none, cu=N, pm=N, T=0) == 0
    assert decode(lib, **none) == 0
    assert verify(lib, **none, inter=N) == 0
    for call in (pack, unpack):
        assert call(lib, pool=N, idx=N, codes=N, scales=N, sidx=N, B=0) == 0


def test_null_and_misaligned_pointers(lib):
    for call, more16, more4 in ((extend, (), ("cu",)), (decode, (), ()), (verify, ("inter",), ())):
        for name in ("q", "k", "v", "pool", "out") + more16:
            assert call(lib, **{name: BAD16}) == 1, (call, name)
            assert call(lib, **{name: N}) == 1, (call, name)
        for name in ("g", "beta", "idx") + more4:
            assert call(lib, **{name: BAD4}) == 1, (call, name)
            assert call(lib, **{name: N}) == 1, (call, name)
    assert extend(lib, pm=N) == 1
    assert extend(lib, ws=N) == 1 and extend(lib, ws=BAD16) == 1
    assert extend(lib, nbytes=la.delta_extend_workspace_size(1, 8, 2, 128) - 1) == 1
    for call in (pack, unpack):
        for name, bad in (("pool", BAD16), ("codes", BAD16), ("scales", BAD4), ("idx", BAD4), ("sidx", BAD4)):
            assert call(lib, **{name: bad}) == 1, (call, name)
            assert call(lib, **{name: N}) == 1, (call, name)


def test_row_strides(lib):
    for call in (extend, decode, verify):
        for rs in ((120, 0, 0), (0, 132, 0), (0, 0, 128), (-128, 0, 0), (0, 0, 260)):
            assert call(lib, rs=rs) == 1, (call, rs)
        assert call(lib, rs=(1 << 40, 0, 0)) == 2


def _cpu(rows=4, Hk=1, H=2):
    bf = lambda w: torch.zeros(rows, w, dtype=torch.bfloat16)  # noqa: E731
    return (bf(Hk * 128), bf(Hk * 128), bf(H * 128), torch.zeros(rows, H), torch.zeros(rows, H),
            torch.zeros(3, H, 128, 128), torch.zeros(rows, dtype=torch.int32))


def test_workspace_size(lib):
    nb = ctypes.c_size_t(7)
    size = lib.la_delta_extend_workspace_size
    assert size(1, 1, 1, 64, ctypes.byref(nb)) == 2
    assert size(-1, 1, 1, 128, ctypes.byref(nb)) == 1 and size(1, -1, 1, 128, ctypes.byref(nb)) == 1
    assert size(1, 1, 0, 128, ctypes.byref(nb)) == 1 and size(1, 1, 1, 128, None) == 1
    assert size(0, 0, 1, 128, ctypes.byref(nb)) == 0 and nb.value == 0
    one = la.delta_extend_workspace_size(1, 64, 1, 128)
    assert one > 0 and la.delta_extend_workspace_size(3, 1000, 4, 128) % 16 == 0
    # enough slots for every way to cut T tokens into B requests
    for lens in ([1, 1, 1], [64, 64, 64], [63, 65, 1], [0, 0, 129], [128, 127, 2]):
        base = [sum(lens[:b]) // 64 + b for b in range(3)]
        chunks = [-(-n // 64) for n in lens]
        ends = [x + y for x, y in zip(base, chunks)]
        assert all(e <= s for e, s in zip(ends, base[1:] + [sum(lens) // 64 + 3]))
    # segments of long requests take room where there are few chains, and only there
    slots = lambda B, T, H: (T // 64 + B) * H * 21520 + (4 * B + 4 + 15) // 16 * 16  # noqa: E731
    assert la.delta_extend_workspace_size(2, 1216, 4, 128) == slots(2, 1216, 4)
    assert la.delta_extend_workspace_size(1, 8192, 3, 128) == slots(1, 8192, 3) + 3 * 61 * 65536
    assert la.delta_extend_workspace_size(2, 8192, 38, 128) == slots(2, 8192, 38) + 304 * 65536
    # a plan for up to 128 requests of which one may be far longer than the others
    assert la.delta_extend_workspace_size(7, 8192, 11, 128) == slots(7, 8192, 11) + 6208 + 512 * 65536
    assert la.delta_extend_workspace_size(7, 1984, 11, 128) == slots(7, 1984, 11)
    assert la.delta_extend_workspace_size(129, 8192, 11, 128) == slots(129, 8192, 11)
    assert la.delta_extend_workspace_size(7, 8192, 512, 128) == slots(7, 8192, 512)
    # more (chunk, head) pairs than a grid has CTAs
    assert size(1, 2 ** 31 - 1, 65, 128, ctypes.byref(nb)) == 2
    assert size(2 ** 31 - 1, 0, 2 ** 31 - 1, 128, ctypes.byref(nb)) == 2


def test_binding_refuses_before_the_library():
    q, k, v, g, beta, pool, idx = _cpu()
    with pytest.raises(ValueError):  # host tensors
        la.delta_decode(q, k, v, g, beta, pool, idx)
    with pytest.raises(TypeError):
        la.delta_decode(None, k, v, g, beta, pool, idx)
    with pytest.raises(ValueError):
        la.delta_verify_chain(q, k, v, g, beta, pool, idx, 0)
    with pytest.raises(ValueError):
        la.pack_states(pool, idx, torch.zeros(1, 2, 128, 128, dtype=torch.int8),
                       torch.zeros(1, 2, 128, 4, dtype=torch.uint8), idx)
    rows = torch.zeros(4, 300, dtype=torch.bfloat16)
    cpu = torch.device("cpu")
    assert binding._need_rows(rows[:, :128].contiguous(), "q", cpu, 4, 128) == 128
    with pytest.raises(ValueError):  # 300 is no multiple of 8
        binding._need_rows(rows[:, :128], "q", cpu, 4, 128)
    assert binding._need_rows(torch.zeros(4, 304).bfloat16()[:, 8:136], "q", cpu, 4, 128) == 304
    with pytest.raises(ValueError):
        binding._need_rows(torch.zeros(1, 128).bfloat16().expand(4, 128), "q", cpu, 4, 128)
    with pytest.raises(ValueError):
        binding._need_rows(torch.zeros(128, 4).bfloat16().t(), "q", cpu, 4, 128)
    with pytest.raises(TypeError):
        binding._need_rows(torch.zeros(4, 128), "q", cpu, 4, 128)
    with pytest.raises(ValueError):
        binding._need_rows(torch.zeros(4, 128).bfloat16(), "q", cpu, 4, 256)
