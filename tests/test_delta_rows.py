"""Row strides of the gated-delta-rule calls at a single row, on the host: the refusal that is looked for comes
before any launch."""
import ctypes

from lightning_attention_gb300 import _build, binding


def test_strides_of_a_single_row_are_ignored():
    """Any row stride passes for a single row; 2^30 heads are refused (LA_ERR_UNSUPPORTED) behind that check."""
    _build.build()
    lib = binding.load()
    p, H = ctypes.c_void_p(4096), 1 << 30
    for rs in ((0, 0, 0), (-128, 3, 1), (1, -1, 8), (1 << 40, 0, -(1 << 40))):
        assert lib.la_delta_decode(p, p, p, *rs, p, p, p, 4, p, p, 1, H, 1, 128, 0, None) == 2, rs
        assert lib.la_delta_extend(p, p, p, *rs, p, p, p, 4, p, p, p, p, 1, 1, H, 1, 128, 1, 0, p, 1 << 30, None) == 2
        assert lib.la_delta_verify_chain(p, p, p, *rs, p, p, p, 4, p, p, p, 1, 1, H, 1, 128, 0, None) == 2
