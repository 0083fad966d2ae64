"""Attention over the 8-bit cache where it can go wrong: the ends of its ranges, masked places, captured calls.

Tolerances are those of test_gpu_kv_cache.py (its docstring), with what the range of the weights adds named at the
test that is about it."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, TYPES, check_attention, fp4, gen, kv, make_table, on_gpu, random_cache, scaled  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,fmt", [(2, "e4m3"), (8, "e4m3"), (8, "int8")])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
def test_attention_largest_windows(kv, group, fmt, window):
    """A window past every length is none, on both kernels, for sequences shorter than their queries too."""
    lens = [0, 1, 2, 3, 4, 5, 100, 300]
    g = gen(group)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), fmt)
    q = torch.randn(len(lens), 4, 2 * group, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16", window=window)
