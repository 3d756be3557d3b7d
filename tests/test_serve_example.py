"""What the example server refuses, without a GPU: no step is taken."""
import os
import sys
import types

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_step as E  # noqa: E402


class Stepped(Exception):
    pass


def model(pages, cols):
    def step(*args, **kw):
        raise Stepped
    return types.SimpleNamespace(table=torch.zeros(2, cols), batch=2, free_pages=torch.zeros(pages), step=step)


@pytest.mark.parametrize("pages, cols, length, answer, fits", [(64, 20, 300, 20, True), (64, 20, 300, 21, False), (64, 20, 321, 1, False),
                                                               (19, 20, 300, 20, False), (1, 1, 1, 15, True), (1, 1, 1, 16, False), (9, 9, 3, 0, False)])
def test_requests_that_do_not_fit_are_refused(pages, cols, length, answer, fits):
    """A request that a row of the table, or the cache, cannot hold would be given no slots for ever; without an answer none ends."""
    with pytest.raises(Stepped if fits else AssertionError, match=None if fits or not answer else "no request may need more pages"):
        E.serve(model(pages, cols), [[1] * min(5, length), [1] * length], answer)
