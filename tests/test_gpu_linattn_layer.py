"""The operators together, as the example layer uses them."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("args", [["--T", "300"], ["--hidden", "520", "--ffn", "264", "--Hk", "1", "--Hv", "3", "--B", "1",
                                                  "--T", "2500", "--new", "9"]])
def test_prompt_then_tokens_equals_a_longer_prompt(args):
    r = subprocess.run([sys.executable, "-m", "gated_deltanet_mixer_gb300.linattn_layer", *args], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
