"""The barrier protocol of the attention over shared prefixes at two terms per weight and head_dim 64 (and 32, which
runs as 64): P lies over S as at head_dim 128, over a ring of twelve slots.  The model is test_paged_protocol_model's, with P
as one barrier; the kernel's two halves of P are two, each with one phase per tile like the modelled one."""
import random

import pytest

import test_paged_protocol_model as model


@pytest.mark.parametrize("seed", range(300))
def test_two_terms_over_a_long_ring(seed):
    rng = random.Random(1000 + seed)
    model.simulate(model.draw_parts(rng), False, 12, rng)
