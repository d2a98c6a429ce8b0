"""Which arrays of layers kvq_tree_commit refuses, where no GPU is needed to tell."""
import pytest

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import KvqLayer
from test_draft_host import ALIGN, INVALID, LAYER, commit, config

PAGED = dict(page_tokens=128, n_pages=8)


@pytest.mark.parametrize("over,layers", [
    ({}, (LAYER, KvqLayer(160, 16, 320, 48))),                       # the same key scales
    ({}, (LAYER, KvqLayer(160, 176, 320, 48))),                      # the same value scales
    (dict(kv_format=kvq.KVQ_FMT_TENSOR), (LAYER, KvqLayer(160, 16, 32, 48))),
    ({}, (KvqLayer(16, 16, 32, 48, 64), KvqLayer(16, 16, 32, 48, 80))),   # not paged: tables are not read
    (PAGED, (KvqLayer(16, 16, 32, 48, 64), KvqLayer(160, 160, 320, 320, 80), KvqLayer(16, 16, 32, 48, 64)))])
def test_commit_refuses_layers_of_the_same_rows(over, layers):
    assert commit(cfg=config(**over), layers=layers) == INVALID


@pytest.mark.parametrize("over,layers", [
    (dict(kv_format=kvq.KVQ_FMT_TENSOR), (LAYER, KvqLayer(160, 16, 320, 48))),   # scales are not moved
    (dict(k_bits=16, v_bits=16), (KvqLayer(16, None, 32, None), KvqLayer(160, None, 320, None))),
    (PAGED, (KvqLayer(16, 16, 32, 48, 64), KvqLayer(16, 16, 32, 48, 80), KvqLayer(16, 16, 32, 48, 96)))])
def test_commit_takes_layers_that_share_other_things(over, layers):
    # the last layer is misaligned, which is found after those before it were taken
    assert commit(cfg=config(**over), layers=layers + (KvqLayer(24, 8, 24, 8, 128),)) == ALIGN
