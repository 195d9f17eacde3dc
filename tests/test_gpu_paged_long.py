"""The paged cache's attention tests once more, with page tables wide enough for long sequences: a call is
planned by the keys that its sequences may have, so the same short ones then go to the kernels of long caches."""
import numpy as np  # noqa: F401
import pytest

import test_gpu_paged as T
from test_gpu_paged import (kvb, test_a_bad_page_is_absent_and_reported, test_a_mapped_prefix_is_decoded_from,  # noqa: F401
                            test_a_query_that_is_not_finite_stays_in_its_row, test_both_caches_attentions_share_a_context,
                            test_contexts_of_their_own_on_two_streams, test_long_cache_split_over_ctas_joins_and_repeats_bit_for_bit,
                            test_many_rows, test_new_tokens_that_are_not_finite_stay_hidden_from_earlier_ones,
                            test_on_another_stream_and_captured_while_the_cache_grows, test_one_token_over_ragged_lengths,
                            test_rows_of_tokens_that_no_sequence_owns_are_left_alone, test_rows_that_see_nothing_and_cache_lengths,
                            test_scale_layers_and_no_lse, test_scores_near_the_ends_of_fp32, test_scores_that_rise_and_fall_over_the_tiles,
                            test_several_tokens_are_causal)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def widen(P, keys=2 ** 18):
    """Columns without pages after a pool's own."""
    more = keys // P.page - P.dtab.shape[1]
    P.dtab = torch.nn.functional.pad(P.dtab, (0, max(more, 0)), value=-1).contiguous()


@pytest.fixture(autouse=True)
def wide_tables(monkeypatch):
    init = T.Pool.__init__

    def wider(self, *args, **kw):
        init(self, *args, **kw)
        widen(self)

    monkeypatch.setattr(T.Pool, "__init__", wider)
