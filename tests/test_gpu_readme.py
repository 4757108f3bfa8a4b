"""The README's Python examples run, and leave the page pool and the caches as a server
would need them."""
import os
import re

import pytest
import torch

import linear_attention_blocked_b200 as la

pytestmark = pytest.mark.gpu


def test_examples():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    n = {}
    for block in blocks[:2]:  # (the third needs several ranks)
        exec(block, n)
    assert la.get_device_status() == la.LA_OK
    pool, ids, child = n["pool"], n["ids"], n["child"]
    # prompts of 1000 and 3096 tokens, then one token each; the child is the first one's copy
    assert [pool.length(r) for r in (*ids, child)] == [1001, 3097, 1001]
    for cache, new in ((n["kc"], n["k"]), (n["vc"], n["v"])):
        for r, want in ((ids[0], torch.cat([new[:1000], new[:1]])), (ids[1], torch.cat([new[1000:], new[1:2]])),
                        (child, torch.cat([new[:1000], new[:1]]))):
            at = torch.arange(pool.length(r), device="cuda")
            page = torch.tensor(pool.pages(r), device="cuda")[at // 64]
            assert torch.equal(cache[page, :, at % 64], want)
