"""Chunks of prompts over a paged cache: hundreds of new tokens as one chain behind the
earlier ones, with a window and with one of 2^30 tokens, which hides nothing.  Against the
fp64 oracle; tolerances as in tests/test_gpu_masked_values.py."""
import pytest
import torch

from tests.test_gpu_masked import rf  # noqa: F401
from tests.test_gpu_masked_values import compare
from tests.test_gpu_paged import BF16, Batch, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("d,Hkv,G,ps,Tq,window,sinks", [
    (128, 1, 5, 64, 300, 2**30, 0), (128, 2, 1, 16, 513, 2**30, 7), (64, 1, 4, 32, 700, 2**30, 0),
    (128, 1, 8, 128, 257, 100, 4), (64, 2, 2, 16, 400, 129, 0), (64, 1, 7, 64, 100, 1000, 200)])
def test_chunks(rf, kind, d, Hkv, G, ps, Tq, window, sinks):  # noqa: F811
    # a chunk alone, behind others, longer than its sequence (its first rows read nothing), none
    lens = [Tq, Tq + 700, Tq - 90, 0, Tq + 1, 1]
    bt = Batch(kind, lens, Hkv, d, ps, seed=1700 + Tq).garbage()
    q = torch.randn(len(lens), Tq, Hkv * G, d, generator=_gen(1701 + Tq)).to(BF16)
    compare(rf, bt, q, d ** -0.5, f"chunks of {Tq}", window, sinks)
