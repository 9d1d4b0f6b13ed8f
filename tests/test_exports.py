"""What `from sharded_optimizer_step_adamw_amd import *` gives."""
import re

import sharded_optimizer_step_adamw_amd as z


def test_every_entry_point_of_the_module_is_exported():
    listed = re.findall(r"^  (\w+)(?: / (\w+))?(?: / (\w+))?", z.__doc__[z.__doc__.index("Entry points"):], re.M)
    names = {n for row in listed for n in row if n}
    assert {"linear_xent_grad", "glu_backward", "act8_wgrad", "MuonGraph", "grad_sq_norm"} <= names
    assert names <= set(z.__all__), sorted(names - set(z.__all__))


def test_every_public_function_is_exported_and_exists():
    own = {n for n, v in vars(z).items()
           if not n.startswith("_") and callable(v) and getattr(v, "__module__", "") == z.__name__}
    assert own <= set(z.__all__), sorted(own - set(z.__all__))
    assert len(set(z.__all__)) == len(z.__all__) and all(hasattr(z, n) for n in z.__all__)
