"""The block-sparse attention example runs and agrees with plain attention."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,steps", [(500, 70), (64, 1)])
def test_example(tokens, steps):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import block_sparse_attention as E
    finally:
        sys.path.pop(0)
    E.main(["--tokens", str(tokens), "--steps", str(steps)])
