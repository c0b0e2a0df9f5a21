"""NaN in a query or in a key or value that counts: out and lse of what reads it are NaN, everything
else keeps its bits.  (-inf in lse means that a request has no keys.)
"""
import math

import pytest
import torch

from test_gpu_cache import _decode_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sru():
    import parallelizable_recurrence_b200 as m
    m.load_library()
    return m


def _attend(sru, q, kc, vc, table, lengths, window=0):
    out = torch.full(q.shape, 7.0, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sru.sru_attention_decode(q, kc, vc, table, lengths, out, lse=lse, window=window)
    assert sru.sru_sync_status() == 0
    return out, lse


# the last: one request in pieces over many CTAs, one within one, one without keys
LENGTHS = [[5], [33, 0, 200], [40000, 20, 0]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (4, 2, 128), (3, 1, 136), (4, 2, 512)])
def test_a_query_of_nan_is_nan_in_out_and_lse(sru, lengths, Hq, Hkv, D):
    q, kc, vc, table, n, _, _ = _decode_inputs(len(lengths), Hq, Hkv, D, lengths, 16, seed=D)
    out, lse = _attend(sru, q, kc, vc, table, n)
    q[0, 1, D - 1] = float("nan")
    got, got_lse = _attend(sru, q, kc, vc, table, n)
    assert got[0, 1].isnan().all() and got_lse[0, 1].isnan()
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    rest[0, 1] = False
    assert torch.equal(got[rest], out[rest]) and torch.equal(got_lse[rest], lse[rest])
    for b, m in enumerate(lengths):
        assert torch.isfinite(lse[b]).all() if m else (lse[b] == -math.inf).all() and (out[b] == 0).all()


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (4, 2, 128), (3, 1, 136), (4, 2, 512)])
def test_a_key_of_nan_is_nan_for_the_heads_that_read_it(sru, lengths, Hq, Hkv, D):
    q, kc, vc, table, n, _, _ = _decode_inputs(len(lengths), Hq, Hkv, D, lengths, 16, seed=D + 1)
    out, lse = _attend(sru, q, kc, vc, table, n)
    at = lengths[0] // 2
    page, row, G = int(table[0, at // 16]), at % 16, Hq // Hkv
    kc[page, 0, row, 3] = float("nan")
    got, got_lse = _attend(sru, q, kc, vc, table, n)
    assert got[0, :G].isnan().all() and got_lse[0, :G].isnan().all()
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    rest[0, :G] = False
    assert torch.equal(got[rest], out[rest]) and torch.equal(got_lse[rest], lse[rest])
    # behind the window it is not read
    if lengths[0] > 10:
        got, got_lse = _attend(sru, q, kc, vc, table, n, window=lengths[0] // 3)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got_lse[0]).all()


@pytest.mark.parametrize("lengths", LENGTHS)
def test_a_value_of_nan_is_nan_in_its_feature_alone(sru, lengths):
    q, kc, vc, table, n, _, _ = _decode_inputs(len(lengths), 4, 2, 128, lengths, 16, seed=3)
    out, lse = _attend(sru, q, kc, vc, table, n)
    at = lengths[0] // 2
    vc[int(table[0, at // 16]), 1, at % 16, 70] = float("nan")
    got, got_lse = _attend(sru, q, kc, vc, table, n)
    assert got[0, 2:, 70].isnan().all() and torch.equal(got_lse, lse)
    got[0, 2:, 70] = out[0, 2:, 70]
    assert torch.equal(got, out)


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 1, 136)])
def test_scores_that_are_all_minus_infinity_weigh_nothing(sru, lengths, Hq, Hkv, D):
    q, kc, vc, table, n, _, _ = _decode_inputs(len(lengths), Hq, Hkv, D, lengths, 16, seed=D + 2)
    out, lse = _attend(sru, q, kc, vc, table, n)
    q[0] = 0
    q[0, :, 5] = 1
    for t in range(lengths[0] // 16 + 1):
        if t * 16 < lengths[0]:
            kc[int(table[0, t]), :, :, 5] = -math.inf
    got, got_lse = _attend(sru, q, kc, vc, table, n)
    assert (got[0] == 0).all() and (got_lse[0] == -math.inf).all()
    assert torch.equal(got[1:], out[1:]) and torch.equal(got_lse[1:], lse[1:])
