"""Host-side argument checks of the vocabulary loss (nothing is launched)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import parallelizable_recurrence_b200 as m
    from parallelizable_recurrence_b200 import build
    return m.load_library(build.build())


FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
BIG = 1 << 40


def _forward(lib, **kw):
    a = dict(H=FAKE, W=FAKE, t=FAKE, loss=FAKE, lse=FAKE, M=16, V=100, K=64, ws=FAKE, wsb=BIG, st=None)
    a.update(kw)
    return lib.sru_softmax_loss(*a.values())


def _backward(lib, **kw):
    a = dict(H=FAKE, W=FAKE, t=FAKE, lse=FAKE, g=FAKE, dH=FAKE, ht=0, dW=FAKE, wt=1, M=16, V=100, K=64, ws=FAKE,
             wsb=BIG, st=None)
    a.update(kw)
    return lib.sru_softmax_loss_backward(*a.values())


@pytest.mark.parametrize("call", [_forward, _backward])
def test_refusals(lib, call):
    for name in ("H", "W", "t", "lse", "ws"):
        assert call(lib, **{name: None}) == 1, name
        assert call(lib, **{name: ODD}) == 1, name
    assert call(lib, M=-1) == 1
    assert call(lib, V=0) == 1
    assert call(lib, K=0) == 1
    assert call(lib, K=12) == 4
    assert call(lib, M=1 << 31) == 4
    assert call(lib, V=1 << 31) == 4
    assert call(lib, M=(1 << 31) - 1, V=(1 << 31) - 1) == 4  # more tiles than an int counts
    assert call(lib, wsb=100) == 1


def test_backward_refusals(lib):
    assert _backward(lib, g=None) == 1
    assert _backward(lib, dH=ODD) == 1
    assert _backward(lib, dW=ODD) == 1
    assert _backward(lib, ht=2) == 1
    assert _backward(lib, wt=7) == 1
    assert _backward(lib, dH=None, dW=None) == 0  # nothing asked for
    assert _backward(lib, M=0, dW=None) == 0
    assert _forward(lib, M=0) == 0


def test_workspace_sizes(lib):
    size = lib.sru_softmax_loss_workspace_bytes
    assert size(0, 100, 64, 1) == 0 and size(16, 100, 12, 1) == 0 and size(16, 0, 64, 0) == 0
    # 8 bytes per row and 256 classes, and the target's logit
    assert size(1000, 1000, 64, 0) >= 1000 * (4 * 8 + 4)
    # the gradients hold one piece of dz, not the logits
    assert size(1000, 1000, 64, 1) >= 1000 * 1000 * 2
    assert size(1 << 20, 200000, 1024, 1) < 1 << 34


def test_binding_refuses_host_and_mixed_tensors():
    import parallelizable_recurrence_b200 as sru
    H, W = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    t, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError):
        sru.sru_softmax_loss(H, W, t, f, f)
    with pytest.raises(ValueError):
        sru.sru_softmax_loss(H, W[:, :4], t, f, f)
    with pytest.raises(ValueError):
        sru.sru_softmax_loss_backward(H, W, t, f, f, dH=torch.zeros(4, 4))
