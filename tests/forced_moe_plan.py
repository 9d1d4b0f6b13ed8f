"""The experts' products with tile and parts chosen by the test:
`with forced(tile, part):` puts tests/helpers/_build/libforced_moe_plan.so (the
library's own sources and a plan that the test sets) behind the binding.

tile 256, 192 (256 x 128), 128 or 64, or 0 for the library's own choice; a weight
gradient sums at most `part` rows of an expert at a time (0: the library's own
choice)."""
import contextlib
import ctypes
import os

import sharded_optimizer_step_adamw_amd as z

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "helpers", "_build", "libforced_moe_plan.so")
TILES = [256, 192, 128, 64]
_own = None


class _Library:
    """The entry points that the forced library has, and the others of libzopt."""

    def __init__(self):
        real = z.lib()
        self.real, self.forced = real, ctypes.CDLL(PATH)
        for name in ("zopt_moe_forward", "zopt_moe_backward", "zopt_moe_plan"):
            f = getattr(self.forced, name)
            f.argtypes, f.restype = getattr(real, name).argtypes, ctypes.c_int
            setattr(self, name, f)

    def __getattr__(self, name):
        return getattr(self.real, name)


@contextlib.contextmanager
def forced(tile, part=0):
    global _own
    if _own is None:
        _own = _Library()
    assert _own.forced.force_moe_plan(tile, part) == 0
    z._lib = _own
    try:
        yield
    finally:
        z._lib = _own.real
