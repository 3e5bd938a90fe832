"""read_kv's two outputs (no GPU needed)."""
import pytest

import bit_quantized_token_gb300 as bq
from test_serve_args import Fake, read


def test_one_tensor_for_both():
    """It would hold parts of either."""
    bq.build()
    k = Fake((1, 3, 2, 64))
    with pytest.raises(bq.LlmError, match="k and v are the same memory"):
        read(k=k, v=k)
    with pytest.raises(bq.LlmError, match="not memory of the current device|current device"):
        read(k=k, v=Fake((1, 3, 2, 64), at=1 << 30))
