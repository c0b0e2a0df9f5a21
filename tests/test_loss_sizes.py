"""Sizes that the vocabulary loss refuses, before anything is launched (nothing is launched here)."""
import pytest

from test_loss_abi import _backward, _forward, lib  # noqa: F401 (lib: the fixture)


@pytest.mark.parametrize("M,V,K", [
    (1 << 30, 1, 1 << 16),   # dH alone has 2^30 tiles of 256 x 256
    (1, 1 << 30, 1 << 16),   # dW alone
    (1 << 30, 1 << 16, 8),   # the logits
])
def test_more_tiles_than_the_schedule_counts(lib, M, V, K):  # noqa: F811
    assert _backward(lib, M=M, V=V, K=K, wsb=1 << 62) == 4
    assert _forward(lib, M=M, V=V, K=K, wsb=1 << 62) == 4
    assert lib.sru_softmax_loss_workspace_bytes(M, V, K, 1) == 0
