"""The example runs: training lowers the loss, and the served batch agrees with each user's
adapter applied alone."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu


def test_example():
    ex = runpy.run_path(os.path.join(os.path.dirname(__file__), "..", "examples", "many_adapters.py"))
    layer, pool, first, last = ex["train"](d_out=256, d_in=256, users=3, tokens=200, steps=40)
    print(f"[example] loss {first:.4f} -> {last:.4f}", flush=True)
    assert last < 0.5 * first
    # two bf16 results of one product, the single-adapter one with another rounding per block
    assert ex["serve"](layer, pool) < 0.006
