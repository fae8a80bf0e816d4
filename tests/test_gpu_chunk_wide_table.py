"""The cases of test_gpu_chunk with block tables wider than their sequences need: the
forms of the attention for long contexts, which the table's width chooses, on short
and odd lengths."""
import pytest

import test_gpu_chunk
from chunk_util import Problem
from test_gpu_chunk import (  # noqa: F401  (collected here as well)
    _lib, test_a_chunk_in_pieces_equals_the_chunk, test_bad_pages_are_skipped,
    test_bad_sequences_are_skipped, test_few_rows, test_head_groups, test_host_resident_cache,
    test_more_heads_per_kv_head_than_a_tile_has_rows, test_no_rows_at_all, test_page_sizes,
    test_ragged, test_repeats_bit_for_bit_and_in_a_graph, test_rows_that_see_nothing,
    test_running_maximum_moves, test_scales, test_unseen_8_bit_vectors_do_not_reach_a_row,
    test_unseen_keys_do_not_reach_a_row, test_unseen_tokens_do_not_reach_a_row)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[1500, 4500])
def _wide(monkeypatch, request):
    class Wide(Problem):
        def __init__(self, dtype, hq, hkv, ps, *args, **kw):
            kw["extra_pages"] = request.param // ps
            super().__init__(dtype, hq, hkv, ps, *args, **kw)

    monkeypatch.setattr(test_gpu_chunk, "Problem", Wide)
