"""What the device error word does to other calls: an index out of range is skipped and reported, and
changes nothing else.
"""
import pytest
import torch

from test_gpu_fused import _inputs as _fused_inputs
from test_gpu_loss import _inputs as _loss_inputs
import sru_testlib as tl
from synthetic import SRUConfig, generate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sru():
    import parallelizable_recurrence_b200 as m
    m.load_library()
    assert m.sru_sync_status() in (m.SRU_OK, m.SRU_ERR_INVALID, m.SRU_ERR_TIMEOUT)  # whatever came before is cleared
    return m


def _bad_target(sru):
    """A loss with a target behind the vocabulary; nothing reads the status."""
    H, W, t, _ = _loss_inputs(40, 300, 64, ignored=0.0)
    t[3] = 300
    sru.sru_softmax_loss(H, W, t, torch.empty(40, device="cuda"), torch.empty(40, device="cuda"))


@pytest.mark.parametrize("L,B,d,nd", [(257, 16, 64, 2), (1024, 16, 512, 1)])
def test_fused_forward_after_a_bad_target_has_the_same_bits(sru, L, B, d, nd):
    """The state passes between time tiles on different CTAs: a pending index error must
    not end the waits for it."""
    cfg, inp = _fused_inputs(L, B, d, nd, 14, False, True, hole=False)
    X, W = tl.to_dev_bf16(inp["X"]), tl.to_dev_bf16(inp["W"])
    x, v, b, c0 = (tl.to_dev_f32(inp[k]) for k in ("x", "v", "bias", "c0"))
    h = torch.empty(L, B, nd, d, device="cuda")
    cT = torch.empty(B, nd, d, device="cuda")
    ws = sru.alloc_workspace(L, B, d, nd == 2)

    def run():
        h.fill_(float("nan"))
        cT.fill_(float("nan"))
        sru.sru_forward_fused(X, W, x, v, b, h, cT, ws, c0=c0, bidirectional=nd == 2)

    run()
    assert sru.sru_sync_status() == sru.SRU_OK
    want = h.clone(), cT.clone()
    assert torch.isfinite(want[0]).all()
    _bad_target(sru)
    for _ in range(5):
        run()
        assert torch.equal(h, want[0]) and torch.equal(cT, want[1])
    assert sru.sru_sync_status() == sru.SRU_ERR_INVALID
    assert sru.sru_sync_status() == sru.SRU_OK


def _withheld_carry(sru):
    """A scan whose first carry is never published: its bounded waits run out (about 2 s)."""
    inp = generate(SRUConfig(name="fail", L=256, B=1, d=64, seed=31, proj_dtype="bf16", bias="normal0.1", c0="normal",
                             v_zero=True), u_direct=True, with_grad=False)
    L, B, d = inp["x"].shape
    flags = sru.SRU_FLAG_V_ZERO | sru.SRU_FLAG_FORCE_SCAN
    sru.sru_forward(tl.dev_U(inp), tl.to_dev_f32(inp["x"]), tl.to_dev_f32(inp["v"]), tl.to_dev_f32(inp["bias"]),
                    torch.empty(L, B, 1, d, device="cuda"), torch.empty(B, 1, d, device="cuda"),
                    c0=tl.to_dev_f32(inp["c0"]), workspace=sru.alloc_workspace(L, B, d, False, flags),
                    flags=flags | sru.SRU_FLAG_TEST_WITHHOLD_CARRY)


@pytest.mark.parametrize("order", ["index first", "timeout first"])
def test_a_wait_that_ran_out_is_reported_beside_a_bad_index(sru, order):
    """A bad index is skipped, a wait that ran out leaves outputs that cannot be used: of the two the status
    names the wait."""
    calls = [_bad_target, _withheld_carry]
    for call in calls if order == "index first" else calls[::-1]:
        call(sru)
    assert sru.sru_sync_status() == sru.SRU_ERR_TIMEOUT
    assert sru.sru_sync_status() == sru.SRU_OK
    _bad_target(sru)
    assert sru.sru_sync_status() == sru.SRU_ERR_INVALID
    assert sru.sru_sync_status() == sru.SRU_OK
