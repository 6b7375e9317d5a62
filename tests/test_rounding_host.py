"""The bound that include/eagle3.h states for prompt_attn's weights, against every bf16 rounding."""
import os
import re

import numpy as np
import torch

HEADER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "eagle3.h")


def test_stated_error_of_bf16_weights():
    """Weights are rounded to bf16, to the nearest: all of a binade's fp32 values that lie midway between two bf16 ones, and their
    neighbours, are within what the header states, and some of them at no less than half of it."""
    with open(HEADER) as f:
        text = f.read()
    at = text.index("prompt_attn: causal attention")
    stated = 2.0 ** -int(re.search(r"weights good to 2\^-(\d+)", text[at:]).group(1))
    mid = (0x3F80 + np.arange(128, dtype=np.uint32)) << np.uint32(16)
    x = np.concatenate([mid + np.uint32(0x8000 + d) for d in (-1, 0, 1)]).astype(np.uint32).view(np.float32)
    err = np.abs(torch.from_numpy(x).bfloat16().double().numpy() - x.astype(np.float64)) / x
    assert err.max() <= stated < 2 * err.max() * (1 + 2.0 ** -7)
