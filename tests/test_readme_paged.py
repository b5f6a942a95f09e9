"""The README's paged-cache example, run as it is printed, against what the calls
promise."""
import os
import re

import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")

# a tree may be shipped without its documents
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(README), reason="README.md is not here")]


def example():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "tree_attention" in b]
    assert len(found) == 1
    return found[0]


def test_example():
    g = torch.Generator().manual_seed(3)
    B, T, H, kv, dim, page, P, N, layers = 3, 6, 4, 2, 64, 16, 9, 60, 2

    def ints(x):
        return torch.as_tensor(x, dtype=torch.int32).cuda()

    def floats(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()

    start, nodes = [20, 0, 47], [6, 2, 5]
    names = dict(sv=sv, torch=torch, B=B, P=P, page=page, layers=layers,
                 pools=[floats(N, kv, page, dim) for _ in range(2 * layers)],
                 table=torch.full((B, P), -1, dtype=torch.int32, device="cuda"),
                 refs=torch.zeros(N, dtype=torch.int32, device="cuda"), lengths=ints(start),
                 num_nodes=ints(nodes), parents=ints([[-1, 0, 0, 1, 2, 4]] * B),
                 tokens=ints([[9, 1, 2, 3, 4, 5]] * B), chosen=ints([[2, 0, 4, 0, 5, 7]] * B),
                 q=[floats(B, T, H, dim) for _ in range(layers)],
                 k=[floats(B, T, kv, dim) for _ in range(layers)],
                 v=[floats(B, T, kv, dim) for _ in range(layers)])
    sv.pages_reserve(names["table"], torch.zeros_like(names["lengths"]), names["refs"], page,
                     names["lengths"])
    exec(example(), names)
    assert names["r"]["missing"].item() == 0
    # the path 0 2 4 5 as far as the nodes reach
    assert names["path"]["path"].cpu().tolist() == [[0, 2, 4, 5, -1, -1], [0] + 5 * [-1],
                                                    [0, 2, 4] + 3 * [-1]]
    assert names["path"]["tokens"].cpu().tolist() == [[2, 4, 5, 7, -1, -1], [2] + 5 * [-1],
                                                      [2, 4, 5] + 3 * [-1]]
    lengths = names["lengths"].cpu()
    assert lengths.tolist() == [24, 1, 50]
    # kept positions hold their nodes' keys and values
    table = names["table"].cpu()
    for b in range(B):
        for i, node in enumerate([0, 2, 4, 5][:int(lengths[b]) - start[b]]):
            p = start[b] + i
            at = int(table[b, p // page])
            for n in range(layers):
                for new, pool in ((names["k"], names["pools"][2 * n]),
                                  (names["v"], names["pools"][2 * n + 1])):
                    assert torch.equal(pool[at, :, p % page], new[n][b, node])
    # what is behind them was given back, what is left has three holders
    held = [-(-int(n) // page) for n in lengths]
    want = np.full((B, P), -1)
    refs = np.zeros(N, dtype=int)
    for b in range(B):
        want[b, :held[b]] = table[b, :held[b]].tolist()
        refs[want[b, :held[b]]] = 3
    assert (table.numpy() == want).all()
    assert (names["branches"].cpu().numpy() == want[:, None]).all()
    assert (names["used"].cpu() == lengths[:, None]).all()
    assert (names["refs"].cpu().numpy() == refs).all()
    # an attention of the last layer over the whole example's cache, by its definition
    chain = sv.tree_attention(names["q"][1], names["pools"][2], names["pools"][3], names["table"],
                              names["lengths"] - 1, num_nodes=torch.ones_like(names["lengths"]))
    keys, values = (names["pools"][i].cpu() for i in (2, 3))
    for b in range(B):
        n = int(lengths[b])
        rows = [torch.stack([x[int(table[b, p // page]), :, p % page] for p in range(n)])
                for x in (keys, values)]
        for h in range(H):
            z = rows[0][:, h // 2].double() @ names["q"][1][b, 0, h].cpu().double() * dim ** -0.5
            o = torch.softmax(z, 0) @ rows[1][:, h // 2].double()
            # weights and result rounded to 8 bits, of values up to about 4
            assert (chain[b, 0, h].cpu().double() - o).abs().max() <= 2 * 2 ** -8 * 4
