"""The gradient operators with tile and split chosen by the test:
`with forced(tile, splits, rest):` puts tests/helpers/_build/libforced_plan.so
(the library's own sources and a plan that the test sets) behind the binding.

tile 256, 192 (256 x 128), 128 or 64, or 0 for the library's own choice; the
reduction of all tiles (rest 2), half of them (1) or none (0) is split."""
import contextlib
import ctypes
import os

import sharded_optimizer_step_adamw_amd as z

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "helpers", "_build", "libforced_plan.so")
TILES = [256, 192, 128, 64]
SPLITS = [(1, 0), (3, 2), (2, 1)]  # whole; all split; half of the tiles split
_own = None


class _Library:
    """The entry points that the forced library has, and the others of libzopt."""

    def __init__(self):
        real = z.lib()
        self.real, self.forced = real, ctypes.CDLL(PATH)
        for name in ("zopt_linear_xent", "zopt_act8_pack", "zopt_act8_unpack", "zopt_act8_wgrad",
                     "zopt_glu_forward", "zopt_glu_backward"):
            f = getattr(self.forced, name)
            f.argtypes, f.restype = getattr(real, name).argtypes, ctypes.c_int
            setattr(self, name, f)

    def __getattr__(self, name):
        return getattr(self.real, name)


@contextlib.contextmanager
def forced(tile, splits=1, rest=0):
    global _own
    if _own is None:
        _own = _Library()
    assert _own.forced.force_plan(tile, splits, rest) == 0
    z._lib = _own
    try:
        yield
    finally:
        z._lib = _own.real
