"""What can be imported and called without PyTorch."""
import subprocess
import sys

import pytest

from partial_activation_sync_caat_b200 import build as B


@pytest.mark.parametrize("module", ["caat", "build", "tp"])
def test_imports_without_torch(module):
    """Host-only calls and the build need no PyTorch, and importing the binding does not load it."""
    code = ("import sys; sys.modules['torch'] = None\n"
            f"import partial_activation_sync_caat_b200.{module} as m\n"
            "if m.__name__.endswith('caat'): print(m.caat_sync_mask(8, 0.5)[1], m.caat_rope_frequencies(4)[0][0])")
    run = subprocess.run([sys.executable, "-c", code], cwd=B.ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    if module == "caat":
        assert run.stdout.split() == ["4", "1.0"]


def test_the_marshalling_is_bound_whichever_comes_first():
    for order in ("import torch\nC.lib()", "C.lib()\nassert C._marshal is None and 'torch' not in sys.modules\nimport torch"):
        code = f"import sys\nfrom partial_activation_sync_caat_b200 import caat as C\n{order}\nassert C._fast() is C._marshal is not None"
        run = subprocess.run([sys.executable, "-c", code], cwd=B.ROOT, capture_output=True, text=True)
        assert run.returncode == 0, run.stderr
