"""The workspace of cross_entropy_bwd, on the CPU: the sizes that the query
names, and what the C entry point and the binding take and refuse.  (A call
that is taken would launch, so the C entry point is only shown what it
refuses.)"""
import time

import pytest
import torch

from test_activation_refusals import INVAL, call
from test_vocabulary_refusals import LOSS_BWD, coat  # noqa: F401  (the fixture)


def test_search_for_the_pieces_is_short(coat):  # noqa: F811
    """A workspace too small for any number of pieces: the vocabulary's 16384 pieces of 256 rows make 255 different
    sizes, and each is looked at once."""
    def best(vocab):
        times = []
        for _ in range(30):
            start = time.perf_counter()
            assert call(coat, "cross_entropy_bwd", coat.CrossEntropyBwdArgs, LOSS_BWD, rows=70, vocab=vocab,
                        workspace_bytes=1000) == INVAL
            times.append(time.perf_counter() - start)
        return min(times)

    assert best(1 << 22) < 60 * best(256)
