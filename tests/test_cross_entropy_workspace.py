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


SHAPES = [(8192, 8192, 4096), (8192, 1000, 2048), (8192, 300, 4096), (64, 300, 4096), (65, 300, 4096), (5000, 32000, 2048),
          (1, 32000, 4096), (300, 131072, 256), (2047, 50001, 2048), (70, 1000, 128), (100, 257, 64 * 1024), (4096, 8192, 8192),
          (1, 1, 128), (200, 1 << 20, 128)]


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,vocab,cols", SHAPES)
def test_every_query_is_taken(coat, rows, vocab, cols, f32, codes):  # noqa: F811
    """A workspace of the size that a query names passes the binding's check (and is refused for its device alone);
    larger pieces never ask for less; the least of all is what the C entry point takes, and less is refused."""
    def query(piece):
        return coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=piece, codes=codes, f32=f32)

    sizes = []
    for piece in sorted({1, 256, 257, 512, 1000, 4096, 8192, 16384, max(1, vocab // 3), max(1, vocab - 1), vocab, 1 << 40}):
        sizes.append(query(piece))
        kind = torch.uint8 if codes else torch.bfloat16
        with pytest.raises(ValueError, match="device"):
            coat.cross_entropy_bwd(meta(rows, dtype=torch.float32), meta(rows, cols, dtype=kind), meta(vocab, cols, dtype=kind),
                                   meta(rows, dtype=torch.int64), meta(rows, dtype=torch.float32), meta(rows, cols),
                                   meta(vocab, cols, dtype=torch.float32 if f32 else torch.bfloat16),
                                   workspace=meta(sizes[-1], dtype=torch.uint8))
    assert sizes == sorted(sizes) and sizes[-1] == query(vocab)
    ops = dict(x=None, weight=None, x_codes=1 << 20, weight_codes=1 << 20) if codes else {}
    out = dict(dw_bf16=None, dw_f32=1 << 20) if f32 else {}
    assert call(coat, "cross_entropy_bwd", coat.CrossEntropyBwdArgs, {**LOSS_BWD, **ops, **out}, rows=rows, vocab=vocab,
                cols=cols, workspace_bytes=sizes[0] - 1) == INVAL
    with pytest.raises(ValueError, match="workspace holds"):
        coat.cross_entropy_bwd(meta(rows, dtype=torch.float32), meta(rows, cols, dtype=kind), meta(vocab, cols, dtype=kind),
                               meta(rows, dtype=torch.int64), meta(rows, dtype=torch.float32), meta(rows, cols),
                               meta(vocab, cols, dtype=torch.float32 if f32 else torch.bfloat16),
                               workspace=meta(sizes[0] - 1, dtype=torch.uint8))
