"""Paged-cache calls on drawn sizes, types, layouts and masks against the
definitions.  SPECVERIFY_RANDOM_PAGED_CASES sets how many, SPECVERIFY_RANDOM_OFFSET
which seeds."""
import os
import random

import pytest
import torch

import draft_token_verification_vocab_amd as sv
import test_gpu_tree as tree

pytestmark = pytest.mark.gpu
CASES = int(os.environ.get("SPECVERIFY_RANDOM_PAGED_CASES", "60"))
OFFSET = int(os.environ.get("SPECVERIFY_RANDOM_OFFSET", "0"))


@pytest.mark.parametrize("seed", range(OFFSET, OFFSET + CASES))
def test_tree_attention(seed):
    r = random.Random(seed)
    dt = r.choice([tree.BF16, tree.F16, tree.F32])
    kv, G = r.choice([1, 2, 3, 8, 33]), r.choice([1, 2, 3, 4, 7, 8, 16])
    T = r.choice([1, 1, 2, 5, 9, 17, r.randint(1, 128)])
    D = 8 * r.randint(1, 32) if r.random() < 0.5 else r.choice([64, 128, 128, 256])
    page = r.choice([8, 16, 32, 64, 128, 256])
    B = r.randint(1, 6)
    high = int(2 ** r.uniform(0, 11.5))
    low = r.randint(0, high)
    c = tree.make(seed, dt, B, T, kv * G, kv, D, page, low, high, tree=r.random() < 0.5,
                  least=r.choice([None, 0, T]), extra=r.choice([0, 1, 40]))
    if r.random() < 0.2:
        c["table"][r.randrange(B), r.randrange(c["table"].shape[1])] = -1
    scale = r.choice([None, None, 0.3])
    d = tree.on_gpu(c, r.choice(["heads", "heads", "slots", "both"]), r.random() < 0.5)
    tree.check(c, tree.call(d, lse=True, scale=scale), scale)
