"""The status word of dense products."""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("M", [1, 40, 300, 3000])
def test_a_status_word_changes_nothing_and_stays_clear(M):
    moe = lib()
    x = torch.randn((M, 512), device=DEV).to(BF)
    w = torch.randn((256, 512), device=DEV).to(BF)
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    want = moe.linear(x, w)
    assert torch.equal(moe.linear(x, w, status=status), want)
    assert torch.equal(moe.linear(x, w, status=status, stream=torch.cuda.current_stream()), want)
    assert moe.check_status(status) == 0 and moe.linear_status() == 0
    assert moe.linear_status(stream=torch.cuda.Stream()) == 0


def test_status_words_that_are_refused():
    moe = lib()
    x, w = torch.zeros((4, 64), dtype=BF, device=DEV), torch.zeros((8, 64), dtype=BF, device=DEV)
    for status in (torch.zeros(1, device=DEV, dtype=torch.uint8),
                   torch.zeros(1, device=DEV, dtype=torch.int64), torch.zeros(1, dtype=torch.int32),
                   torch.zeros(0, device=DEV, dtype=torch.int32)):
        with pytest.raises(ValueError, match="status"):
            moe.linear(x, w, status=status)
