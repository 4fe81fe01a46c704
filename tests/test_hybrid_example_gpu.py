"""The example that runs the operators together: prompts, then rounds of draft, verify and commit.  The
committed pools have to be those of the same texts fed as prompts from nothing, up to the rounding of
bf16 activations along different kernels (each layer's input and output are rounded to 2^-8 a few times:
a few 2^-8; a wrong step, slot or count is off by the states themselves)."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_committed_pools_are_the_texts_states():
    import hybrid_serving
    assert hybrid_serving.main() < 0.05
