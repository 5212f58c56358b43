"""The tests' account of how attention calls are cut, against the library's workspaces."""

import random

import pytest
import torch

import attn_shapes
import chunked_gated_delta_rule_amd as gdn


@pytest.mark.parametrize("seed", range(4))
def test_workspaces_follow_from_the_shapes(seed):
    rng = random.Random(seed)
    cus = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 256
    split = 0
    for _ in range(500):
        hkv = rng.choice([1, 2, 3, 8])
        n = rng.choice([1, 2, 7, 64, 65, 256, 257, 1000])
        c = gdn.make_attn_config(int(2 ** rng.uniform(0, 15)), n, hkv * rng.choice([1, 2, 4, 5, 17, 24]),
                                 hkv, rng.choice([128, 256]), page_size=rng.choice([16, 64, 256]),
                                 n_pages=9, max_pages=int(2 ** rng.uniform(0, 12)),
                                 tk_max=rng.choice([0, int(2 ** rng.uniform(0, 16))]),
                                 shared_max=rng.choice([0, int(2 ** rng.uniform(4, 16))]))
        assert gdn.gdn_attn_workspace_size(c) == attn_shapes.workspace_size(c, cus)
        split += attn_shapes.shape(c, attn_shapes.ROWS, cus).splits > 1
    assert split > 20
