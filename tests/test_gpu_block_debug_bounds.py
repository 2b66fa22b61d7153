"""The tests of the operators around the scan once more through the
debug-bounds library (every global index checked), in a process of its own:
the bounds word is read after every test."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_block_operators_stay_in_bounds_under_the_debug_build():
    from selective_state_space_25_b200 import build as libbuild
    libbuild.build(debug_bounds=True)
    env = dict(os.environ, SSM_DEBUG_BOUNDS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join(HERE, "test_gpu_block.py")], env=env, capture_output=True, text=True,
                       timeout=900, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]


@pytest.mark.parametrize("name", ["random", "rounds", "eps", "ends", "nonfinite", "closed"])
def test_more_block_operators_stay_in_bounds_under_the_debug_build(name):
    """The other sizes, too: seeded random ones, many rounds, odd row counts."""
    from selective_state_space_25_b200 import build as libbuild
    libbuild.build(debug_bounds=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join(HERE, f"test_gpu_block_{name}.py")],
                       env=dict(os.environ, SSM_DEBUG_BOUNDS="1"), capture_output=True, text=True,
                       timeout=900, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
