"""seg_la on GB300: Bailing-style segmented lightning attention behind a C ABI.

The computation runs in hand-written sm_103a CUDA kernels (csrc/), reached through the C ABI of
include/la.h; this package holds the ctypes binding (binding.py), the in-tree build (_build.py)
and the seeded synthetic workloads (workloads.py).
"""
from .binding import (LAError, commit_accepted, decode, decode_gqa, delta_decode, delta_extend,  # noqa
                      delta_extend_workspace_size, delta_verify_chain, extend, extend_gqa, extend_gqa_workspace_size,
                      extend_noalloc, extend_workspace_size, load, pack_states, poll_error,
                      set_balanced, set_column_split, set_persistent, set_wait_limit, slopes,
                      unpack_states, verify_chain, verify_tree)
