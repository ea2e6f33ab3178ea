"""What block.Head refuses ahead of any call: given tokens that are not rows of the buffers' M.  No GPU needed."""
from types import SimpleNamespace

import pytest
import torch

blk = pytest.importorskip("w4a4_outlier_split_amd.block", reason="libosc.so not built")


class Called(Exception):
    pass


@pytest.fixture
def head(monkeypatch):
    def call(*args):
        raise Called(args)

    monkeypatch.setattr(blk, "osc_logprobs", call)
    return blk.Head(SimpleNamespace(N=100), None)


def bufs(M):
    return dict(M=M, K=1, logits=None, lp=None, ent=None, topv=None, topi=None, ws=None)


@pytest.mark.parametrize("M,shape", [(2, (4, 3)), (2, (4, 1)), (3, (4, 2)), (1, (1, 4)), (0, (4, 1)), (0, (4,)), (2, (9,)), (1, (2, 4, 2)), (2, ())])
def test_given_tokens_of_another_width_are_refused(head, M, shape):
    with pytest.raises(ValueError):
        head.logprobs(4, bufs(M), torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("M,ids", [(2, (4, 2)), (2, (9, 2)), (1, (4, 1)), (1, (4,)), (1, (9,)), (2, (8,)), (2, (7,)), (2, (3, 2)), (2, None), (0, None), (0, (4, 0)), (2, 0x10000)])
def test_given_tokens_reach_the_call(head, M, ids):
    """(which refuses those of too few bytes)"""
    ids = torch.zeros(ids, dtype=torch.int32) if isinstance(ids, tuple) else ids
    with pytest.raises(Called) as e:
        head.logprobs(4, bufs(M), ids)
    given = e.value.args[0]
    assert given[6] is ids and given[7] == (0 if ids is None else M)
