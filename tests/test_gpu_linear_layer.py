"""The example layer: a prompt and single tokens through projections, linear attention and the
MoE-FFN step give what one longer prompt gives.

Both runs round activations to bf16 at the same places, but the prompt's q, k, v of a token come
from the same 4-bit sums in another order, so a value may fall on the other side of a rounding
(2^-8 relative). A layer has four such roundings between x and its output (norm, q/k/v, k's
normalisation, o) and the batched FFN path rounds its activations to f16 (1e-3 measured for that
path against float64): 4 * 2^-8 + 2e-3 < 2e-2."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompt,tokens,sequences", [(90, 6, 3), (20, 3, 1)])
def test_prompt_and_tokens_against_one_prompt(prompt, tokens, sequences):
    spec = importlib.util.spec_from_file_location("linear_layer", os.path.join(ROOT, "examples", "linear_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    rate, worst = mod.run(prompt, tokens, sequences, check=True)
    assert rate > 0
    assert worst < 2e-2, worst
