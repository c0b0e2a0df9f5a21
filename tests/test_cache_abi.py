"""Host-side argument checks of the paged cache and its attention (nothing is launched)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import parallelizable_recurrence_b200 as m
    from parallelizable_recurrence_b200 import build
    return m.load_library(build.build())


FAKE, HALF, BYTE = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1001)


def _extend(lib, **kw):
    a = dict(lengths=FAKE, new=FAKE, table=FAKE, free=FAKE, count=FAKE, B=4, maxp=8, pages=32, ps=16, T=10,
             lengths_out=FAKE, count_out=FAKE, offsets=FAKE, slots=FAKE, refused=None, st=None)
    a.update(kw)
    return lib.sru_cache_extend(*a.values())


def _append(lib, **kw):
    a = dict(K=FAKE, k_ld=256, V=FAKE, v_ld=256, t=1, slots=FAKE, kc=FAKE, vc=FAKE, T=5, H=2, D=128, ps=16, pages=8,
             st=None)
    a.update(kw)
    return lib.sru_cache_append(*a.values())


def _decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lengths=FAKE, out=FAKE, out_t=1, lse=None, B=4, Hq=8, Hkv=2, D=128,
             ps=16, pages=64, maxp=8, window=0, scale=0.1, ws=FAKE, wsb=1 << 40, st=None)
    a.update(kw)
    return lib.sru_attention_decode(*a.values())


def test_extend_refusals(lib):
    for name in ("lengths", "new", "table", "free", "count", "lengths_out", "count_out", "offsets", "slots"):
        assert _extend(lib, **{name: None}) == 1, name
        assert _extend(lib, **{name: BYTE}) == 1, name
    assert _extend(lib, refused=BYTE) == 1
    for name in ("B", "maxp", "pages", "T"):
        assert _extend(lib, **{name: -1}) == 1, name
    assert _extend(lib, ps=0) == 1
    assert _extend(lib, B=(1 << 20) + 1) == 4
    assert _extend(lib, T=1 << 31) == 4
    assert _extend(lib, pages=1 << 27, ps=16) == 4
    assert _extend(lib, maxp=1 << 27, ps=16) == 4


def test_append_refusals(lib):
    for name in ("K", "V", "slots", "kc", "vc"):
        assert _append(lib, **{name: None}) == 1, name
        assert _append(lib, **{name: BYTE}) == 1, name
    assert _append(lib, K=HALF) == 1 and _append(lib, vc=HALF) == 1
    assert _append(lib, t=2) == 1
    assert _append(lib, T=-1) == 1 and _append(lib, H=0) == 1 and _append(lib, ps=0) == 1
    assert _append(lib, D=12) == 4
    assert _append(lib, k_ld=255) == 1                 # rows overlap
    assert _append(lib, v_ld=257) == 4                 # not a multiple of 16 bytes
    assert _append(lib, t=0, k_ld=258) == 4
    assert _append(lib, pages=1 << 27, ps=16) == 4
    assert _append(lib, T=0) == 0


def test_decode_refusals(lib):
    for name in ("q", "kc", "vc", "table", "lengths", "out", "ws"):
        assert _decode(lib, **{name: None}) == 1, name
        assert _decode(lib, **{name: BYTE}) == 1, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert _decode(lib, **{name: HALF}) == 1, name
    assert _decode(lib, lse=BYTE) == 1
    assert _decode(lib, out_t=3) == 1
    assert _decode(lib, Hq=9) == 1                     # not a multiple of Hkv
    assert _decode(lib, B=-1) == 1 and _decode(lib, Hkv=0) == 1 and _decode(lib, window=-1) == 1
    assert _decode(lib, D=100) == 4 and _decode(lib, D=1032) == 4
    assert _decode(lib, pages=1 << 27, ps=16) == 4 and _decode(lib, maxp=1 << 27, ps=16) == 4
    need = lib.sru_attention_decode_workspace_bytes(4, 8, 2, 128)
    assert need > 0 and _decode(lib, wsb=need - 1) == 1
    assert lib.sru_attention_decode_workspace_bytes(4, 9, 2, 128) == 0
    assert lib.sru_attention_decode_workspace_bytes(4, 8, 2, 2048) == 0
    assert _decode(lib, B=0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import parallelizable_recurrence_b200 as sru
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sru.sru_attention_decode(q, kc, kc, i(3, 2), i(3), q.clone())
    with pytest.raises(ValueError):
        sru.sru_attention_decode(q, kc, kc, i(2, 2), i(3), q.clone())
    with pytest.raises(ValueError):
        sru.sru_cache_append(torch.zeros(5, 2, 64), torch.zeros(5, 2, 64), i(5), kc, kc)
    with pytest.raises(ValueError):
        sru.sru_cache_append(torch.zeros(5, 1, 64), torch.zeros(5, 1, 64), i(5), kc, kc)
    with pytest.raises(ValueError):
        sru.sru_cache_extend(i(3), i(3), i(3, 4), i(9), i(1), 16, i(3), i(1), i(4), i(5))
    with pytest.raises(ValueError):
        sru.sru_cache_extend(i(3), i(3), i(3, 4), i(9), i(1), 16, i(3), i(1), i(3), i(5))
