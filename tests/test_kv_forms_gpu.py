"""The attentions over both caches by the form that a call's sizes lead to."""
import numpy as np
import pytest
import torch

import test_kv4_attention_gpu as four
import test_kv8_gpu as eight
from test_kv4_gpu import BF16, F32, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,rows,length,T,D,KVH,G", [
    (1, 128, 4000, 64, 128, 5, 4), (3, 256, 1777, 32, 64, 8, 2), (1, 500, 1777, 32, 64, 8, 2),
    (17, 500, 2049, 16, 128, 2, 4), (0, 128, 4000, 64, 128, 5, 4), (1, 128, 700, 128, 64, 5, 4)])
def test_fewer_rows_than_the_call(gpu, n, rows, length, T, D, KVH, G, dtype, bits):
    """A lone sequence that brings a few of the rows that its call has room for: cut into
    parts, or not where its keys are few; the rows behind are left."""
    if bits == 4:
        four.check_filled(gpu, make(150, [n], [length], T, D, KVH, dtype, G, behind=rows - n))
        return
    s = eight.make(150, [n], [length], T, D, KVH, dtype, G, behind=rows - n)
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    used = eight.check_attention(s, eight.attend(gpu, d, out=out))
    assert (out.cpu().float().numpy()[~used] == 77.0).all()
    assert np.count_nonzero(used) == n * KVH * G * D
