"""Sizes that the library's C types do not hold are refused, not cut to the bits that they do hold.  No GPU needed."""

import pytest


@pytest.fixture(scope="module")
def ops():
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


@pytest.mark.parametrize("name,args", [
    ("FeedForward", (2, 2 ** 32 + 64, 64)), ("FeedForward", (2 ** 32 + 2, 64, 64)), ("FeedForward", (2, 64, 2 ** 64 + 5)),
    ("FeedForward", (2, -2 ** 32 + 64, 64)), ("FeedForward", (-2 ** 40 + 2, 64, 64)), ("Checkpoint", (2 ** 32 + 64,)),
    ("BlockNorm", (2, 2 ** 32 + 64)), ("BlockNorm", (2 ** 32 + 2, 64)), ("VocabHead", (2, 2 ** 64 + 5)),
    ("VocabHead", (2 ** 32 + 2, 50))])
def test_sizes_that_would_wrap(ops, name, args):
    with pytest.raises(ValueError, match="out of range"):
        getattr(ops, name)(*args)


@pytest.mark.parametrize("name,args", [("FeedForward", (2, 2 ** 31 - 1, 64)), ("FeedForward", (33, 64, 64)),
                                       ("FeedForward", (2, 64, 2 ** 62)), ("Checkpoint", (-1,)), ("BlockNorm", (-1, 64))])
def test_sizes_out_of_the_library_s_range(ops, name, args):
    """What fits the types is the library's to refuse."""
    with pytest.raises(ops.RAError):
        getattr(ops, name)(*args)
