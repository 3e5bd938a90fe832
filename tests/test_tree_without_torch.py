"""The tree operators' binding in a process that has not imported torch (no GPU needed)."""
import subprocess
import sys

import pytest

import bit_quantized_token_gb300 as bq
from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()


@pytest.mark.parametrize("call", ["bq.tree_status()", "bq.tree_status(None)",
                                  "bq.KVView(np.zeros((1, 1, 4, 64), np.float32), np.zeros((1, 1, 4, 64), np.float32))"])
def test_errors_are_the_librarys(call):
    """A status without trouble, or an LlmError: no GPU here, or arrays that are no tensors of the library's types."""
    code = ("import sys\nimport numpy as np\nimport bit_quantized_token_gb300 as bq\nassert 'torch' not in sys.modules\n"
            f"try:\n    {call}\nexcept bq.LlmError:\n    pass\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)
