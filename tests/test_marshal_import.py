"""The marshalling module is needed by the calls that use it, not by the import (no GPU needed)."""
import subprocess
import sys

from block_sparse_full_b200 import ssa

_BLOCKED = """
import sys

class Block:
    def find_spec(self, name, path=None, target=None):
        if name == "block_sparse_full_b200._marshal":
            raise ImportError("undefined symbol: from another torch")

sys.meta_path.insert(0, Block())
import torch
from block_sparse_full_b200 import ssa

assert ssa.ssa_version() >> 16 == 1
p = ssa.make_params(1, 2, 256, 64, 64, 2, torch.float32)
assert ssa.ssa_workspace_size(p, 0) != ssa.ctypes.c_size_t(-1).value
t = torch.zeros(1, 2, 8, 64)
for call in (lambda: ssa.window_params_for(t, t, 4), lambda: ssa.window_fwd(None, t, t, t)):
    try:
        call()
    except ImportError as e:
        assert "python -m block_sparse_full_b200.build" in str(e) and "undefined symbol" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_earlier_calls_do_not_need_it():
    r = subprocess.run([sys.executable, "-c", _BLOCKED], capture_output=True, text=True, timeout=300,
                       cwd=ssa.os.path.dirname(ssa.os.path.dirname(ssa.__file__)))
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_it_is_the_module_itself_after_the_first_call():
    import torch

    t = torch.zeros(1, 2, 8, 64)
    ssa.window_params_for(t, t, 4)
    assert type(ssa._marshal) is type(sys) and ssa._marshal.__name__.endswith("_marshal")
