"""The README's loop for a budget of positions, run as it stands there: sequences above their budget are cut to it, and
those below it keep their length and their pages."""
import os
import textwrap

import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def block(having):
    """The indented block of the README that has this line."""
    with open(README) as f:
        blocks, now = [], []
        for line in f.read().split("\n") + ["end"]:
            if line.startswith("    ") or (now and not line.strip()):
                now.append(line)
            elif now:
                blocks.append("\n".join(now))
                now = []
    found = [b for b in blocks if having in b]
    assert len(found) == 1
    return textwrap.dedent(found[0])


def test_sequences_below_their_budget_stay_as_they_are():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()
    layers, B, Hkv, D, ps, max_pages, pages, l = 1, 4, 2, 64, 16, 8, 40, 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    old, lens, most = [39, 99, 6, 64], [40, 100, 7, 65], [64, 64, 64, 64]
    k, v = (torch.randn(layers, pages, ps, Hkv, D, device="cuda").to(torch.bfloat16) for _ in "kv")
    count, table, short = ne.pages_resize(torch.zeros(pages, dtype=torch.int32, device="cuda"),
                                          torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda"), i32([0] * B), i32(lens), k, v)
    new_lens, budget, cu_new, longest = i32(lens), i32(most), i32(range(B + 1)), 1
    q = torch.randn(B, 4, D, device="cuda").to(torch.bfloat16)
    o, lse = ne.paged_attn(q, k[l], v[l], table, new_lens, cu_new, max_new=longest)
    names = dict(globals(), **locals())
    exec(block("ne.pages_evict("), names)
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    keep = [min(a, b) for a, b in zip(lens, most)]
    assert int(names["short"]) == 0
    assert int(names["count"].sum()) == sum(-(-n // ps) for n in keep)
    assert [int(n) for n in (names["table"] >= 0).sum(1)] == [-(-n // ps) for n in keep]
    assert names["offset"].tolist() == [a - b for a, b in zip(lens, keep)]
    assert names["cut"].tolist() == keep                   # what the next step begins with
    assert [int(n) for n in (names["weights"][0, :, 0] > 0).sum(1)] == keep
