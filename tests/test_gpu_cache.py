"""GPU parity of the paged cache and of the one-token attention over it.

The bookkeeping and the append are exact: compared value by value with plain
Python loops.  The attention is compared with its formula in 64 bits on the same
bf16 inputs.  Tolerance: a score is an fp32 sum, off by at most
e = 1e-5 (max_j |scale| sum_k |q_k k_jk| + 1) (the bound of the library's fp32
products); p is off by a factor exp(+-2e) and rounded to 16 bits (2^-17, counted
as 2^-16 with the sum's own rounding); so o is off by at most
(3e + 2^-16) sum_j p_j |v_j| / l, and as bf16 by 2^-8 of its value on top.
Slots that no token holds contain NaN throughout.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sru():
    import parallelizable_recurrence_b200 as m
    m.load_library()
    return m


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ bookkeeping
def _extend_reference(lengths, new, table, free, n_free, ps, T):
    """One step by the definition, a request at a time."""
    table, free = [list(r) for r in table], list(free)
    B, maxp = len(lengths), len(table[0]) if table else 0
    for b in range(B):
        if new[b] < 0:
            for i in range(math.ceil(lengths[b] / ps)):
                free[n_free] = table[b][i]
                n_free += 1
    height, wanted, row, refused = n_free, 0, 0, 0
    out, offsets, slots = [], [0], [-1] * T
    for b in range(B):
        n, add = lengths[b], max(new[b], 0)
        held = math.ceil(n / ps)
        row += add
        offsets.append(row)
        if new[b] < 0:
            out.append(0)
            continue
        ok = add > 0 and n + add <= maxp * ps and row <= T
        if ok:
            need = math.ceil((n + add) / ps) - held
            wanted += need
            ok = need == 0 or wanted <= height
            if ok:
                for i in range(need):
                    n_free -= 1
                    table[b][held + i] = free[height - 1 - (wanted - need) - i]
                for j in range(add):
                    slots[row - add + j] = table[b][(n + j) // ps] * ps + (n + j) % ps
        refused += add > 0 and not ok
        out.append(n + add if ok else n)
    return table, free, out, n_free, offsets, slots, refused


def _pool(rng, B, maxp, ps, lengths, pages):
    order = rng.permutation(pages)
    table, at = np.full((B, maxp), -1, np.int64), 0
    for b in range(B):
        held = math.ceil(lengths[b] / ps)
        table[b, :held] = order[at:at + held]
        at += held
    free = np.full(pages, -1, np.int64)
    free[:pages - at] = order[at:]
    return table, free, pages - at


def _extend(sru, lengths, new, table, free, n_free, ps, T, in_place):
    d = dict(lengths=_i32(lengths), new=_i32(new), table=_i32(table).view(len(lengths), -1), free=_i32(free),
             n=_i32([n_free]))
    out = d["lengths"] if in_place else torch.full_like(d["lengths"], -7)
    n_out = d["n"] if in_place else torch.full_like(d["n"], -7)
    offsets = torch.full((len(lengths) + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    refused = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    for _ in range(1 if in_place else 2):  # apart from its inputs, a second call gives the same
        sru.sru_cache_extend(d["lengths"], d["new"], d["table"], d["free"], d["n"], ps, out, n_out, offsets, slots,
                             refused=refused)
    assert sru.sru_sync_status() == 0
    return (d["table"].tolist(), d["free"].tolist(), out.tolist(), int(n_out), offsets.tolist(), slots.tolist(),
            int(refused))


def _check_extend(sru, lengths, new, table, free, n_free, ps, T):
    want = _extend_reference(lengths, new, table, free, n_free, ps, T)
    for in_place in (False, True):
        got = _extend(sru, lengths, new, table, free, n_free, ps, T, in_place)
        for name, a, b in zip(("table", "free", "lengths", "count", "offsets", "slots", "refused"), got, want):
            assert a == b, (name, in_place)


@pytest.mark.parametrize("B,maxp,ps,spare,T,prompts", [
    (1, 4, 16, 0, 8, False),
    (1, 1, 1, 0, 3, False),
    (7, 5, 3, 0, 40, True),
    (200, 9, 16, 0, 300, False),
    (200, 9, 16, -700, 5000, True),      # a short stack: some requests are refused
    (1500, 6, 8, 0, 2000, False),        # more than one chunk of requests
    (1500, 6, 8, -3000, 30000, True),    # the same on the cluster, short of pages
    (64, 300, 24, 0, 100000, True),      # long prompts, shared out in segments
    (64, 300, 24, 0, 30000, True),       # the step's rows run out
    (2100, 40, 64, -20000, 900000, True),
])
def test_extend_matches_the_definition(sru, B, maxp, ps, spare, T, prompts):
    rng = np.random.default_rng(B + maxp + ps + T)
    lengths = rng.integers(0, maxp * ps + 1, B)
    new = rng.integers(0, 3, B)
    if prompts:
        fresh = rng.random(B) < 0.5
        lengths[fresh] = 0
        new[fresh] = rng.integers(1, maxp * ps + 2, int(fresh.sum()))  # some beyond the table's width
    new[rng.random(B) < 0.15] = -1
    pages = B * maxp + spare
    held = sum(math.ceil(n / ps) for n in lengths)
    pages = max(pages, held)
    table, free, n_free = _pool(rng, B, maxp, ps, lengths.tolist(), pages)
    _check_extend(sru, lengths.tolist(), new.tolist(), table.tolist(), free.tolist(), n_free, ps, T)


def test_extend_refuses_and_goes_on(sru):
    """An empty stack, a stack that the released pages alone fill, and a request that needs no page behind refused ones."""
    ps, table = 4, [[0, 1, -1], [2, -1, -1], [3, -1, -1], [4, -1, -1]]
    _check_extend(sru, [8, 4, 3, 4], [1, 1, 1, 1], table, [-1] * 5, 0, ps, 8)
    _check_extend(sru, [8, 4, 3, 4], [-1, 5, 1, 1], table, [-1] * 5, 0, ps, 8)
    _check_extend(sru, [8, 4, 3, 4], [0, 0, 0, 0], table, [-1] * 5, 0, ps, 8)
    _check_extend(sru, [8, 4, 3, 4], [-1, -1, -1, -1], table, [-1] * 5, 0, ps, 8)


def test_extend_of_no_requests_and_of_no_rows(sru):
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    n, offsets = _i32([3]), _i32([-7])
    slots = _i32([5, 5])
    sru.sru_cache_extend(z, z, torch.empty(0, 4, dtype=torch.int32, device="cuda"), _i32([1, 0, 2]), n, 16, z, n,
                         offsets, slots)
    assert sru.sru_sync_status() == 0
    assert n.tolist() == [3] and offsets.tolist() == [0] and slots.tolist() == [-1, -1]
    _check_extend(sru, [3, 3], [0, -1], [[0], [1]], [-1, -1], 0, 4, 0)


@pytest.mark.parametrize("T", [600, 5000])
def test_extend_with_too_many_tokens_stays_inside_its_arrays(sru, T):
    """Tokens from 2^31 on wrap the offsets: what the step grants is unspecified, what lies around its arrays untouched."""
    big, ps, B, maxp = 2**31 - 1, 8, 6, 700
    whole = {n: torch.full((64 + size + 64,), -7, dtype=torch.int32, device="cuda")
             for n, size in (("table", B * maxp), ("slots", T), ("offsets", B + 1), ("free", B * maxp), ("out", B))}
    part = {n: w[64:-64] for n, w in whole.items()}
    for new in ([big, 10, big, 300, 10, 5], [5, big, 300, 2, big, 300], [big] * B, [-1, big, big, 300, -1, 90]):
        part["free"].copy_(torch.arange(B * maxp))
        n = _i32([B * maxp])
        sru.sru_cache_extend(_i32([0] * B), _i32(new), part["table"].view(B, maxp), part["free"], n, ps, part["out"], n,
                             part["offsets"], part["slots"])
        assert sru.sru_sync_status() == 0
        assert int(part["slots"].max()) < B * maxp * ps and 0 <= int(n) <= B * maxp
        for name, w in whole.items():
            assert (w[:64] == -7).all() and (w[-64:] == -7).all(), name
    _check_extend(sru, [3, 3], [0, -1], [[0], [1]], [-1, -1], 0, 4, 0)


# ----------------------------------------------------------------------- append
@pytest.mark.parametrize("T,H,D,ps", [(1, 1, 8, 1), (5, 3, 72, 7), (300, 8, 128, 16), (70, 1, 1024, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("halves", [False, True])
def test_append_places_every_row(sru, T, H, D, ps, dtype, halves):
    rng = np.random.default_rng(T + D)
    pages = T // ps + 3
    slots = rng.permutation(pages * ps)[:T]
    slots[rng.random(T) < 0.2] = -1
    KV = torch.randn(T, 2 * H * D + 8, device="cuda").to(dtype)
    K, V = KV[:, : H * D].unflatten(1, (H, D)), KV[:, H * D:2 * H * D].unflatten(1, (H, D))
    if not halves:
        K, V = K.contiguous(), V.contiguous()
    kc = torch.full((pages, H, ps, D), 9.0, device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    want_k, want_v = kc.clone(), vc.clone()
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // ps, :, s % ps] = K[r].bfloat16()
            want_v[s // ps, :, s % ps] = V[r].bfloat16()
    sru.sru_cache_append(K, V, _i32(slots), kc, vc)
    assert sru.sru_sync_status() == 0
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_append_skips_and_reports_a_slot_behind_the_cache(sru):
    K = torch.randn(3, 1, 64, device="cuda").bfloat16()
    kc = torch.zeros(2, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    sru.sru_cache_append(K, K, _i32([8, 7, 2**31 - 1]), kc, vc)
    assert sru.sru_sync_status() == sru.SRU_ERR_INVALID
    assert sru.sru_sync_status() == sru.SRU_OK
    want = torch.zeros_like(kc)
    want[1, 0, 3] = K[1, 0]
    assert torch.equal(kc, want) and torch.equal(vc, want)


# -------------------------------------------------------------------- attention
def _decode_inputs(B, Hq, Hkv, D, lengths, ps, seed=0):
    """Random q, K, V; the cache's other slots NaN, the table's unused entries out of range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    held = [math.ceil(n / ps) for n in lengths]
    maxp = max(1, max(held))
    pages = sum(held) + 3
    order = rng.permutation(pages)
    table, at = np.full((B, maxp), 2**31 - 1, np.int64), 0
    kc = torch.full((pages, Hkv, ps, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    K, V = [], []
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        n = lengths[b]
        k = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
        v = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
        pos = torch.arange(n, device="cuda")
        page = torch.as_tensor(table[b], device="cuda")[pos // ps]
        kc[page, :, pos % ps] = k
        vc[page, :, pos % ps] = v
        K.append(k)
        V.append(v)
    q = torch.randn(B, Hq, D, generator=g, device="cuda").bfloat16()
    return q, kc, vc, _i32(table), _i32(lengths), K, V


def _check_decode(out, lse, q, K, V, scale, window):
    B, Hq, D = q.shape
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    assert torch.isfinite(out).all()
    for b in range(B):
        n, Hkv = K[b].shape[:2]
        lo = max(0, n - window) if window else 0
        if n == 0:
            assert (out[b] == 0).all() and (lse is None or (lse[b] == -math.inf).all())
            continue
        G = Hq // Hkv
        k, v = K[b][lo:].double().transpose(0, 1), V[b][lo:].double().transpose(0, 1)  # (Hkv, n, D)
        qq = q[b].double().view(Hkv, G, D)
        z = qq @ k.transpose(1, 2) * scale
        # (|scale|: an error bound is the size of the terms, whatever the sign of the scale)
        e = 1e-5 * ((qq.abs() @ k.abs().transpose(1, 2) * abs(scale)).amax(2, keepdim=True) + 1)
        ref_lse = torch.logsumexp(z, 2, keepdim=True)
        p = torch.exp(z - ref_lse)
        o = p @ v
        tol = (3 * e + 2.0 ** -16) * (p @ v.abs()) + half * o.abs()
        over = ((out[b].double().view(Hkv, G, D) - o).abs() - tol).amax()
        assert over <= 0, f"request {b}: beyond the tolerance by {float(over):.3e}"
        if lse is not None:
            assert ((lse[b].double().view(Hkv, G, 1) - ref_lse).abs() <= 2 * e + 1e-6 * ref_lse.abs()).all()


def _decode(sru, inputs, dtype, scale=None, window=0, with_lse=True):
    q, kc, vc, table, lengths, K, V = inputs
    out = torch.full(q.shape, float("nan"), device="cuda", dtype=dtype)
    lse = torch.full(q.shape[:2], float("nan"), device="cuda") if with_lse else None
    sru.sru_attention_decode(q, kc, vc, table, lengths, out, scale=scale, window=window, lse=lse)
    assert sru.sru_sync_status() == 0
    _check_decode(out, lse, q, K, V, q.shape[2] ** -0.5 if scale is None else scale, window)
    return out


EDGES = [0, 1, 15, 16, 17, 31, 33, 0, 100]


@pytest.mark.parametrize("Hq,Hkv,D,ps", [
    (1, 1, 8, 16), (1, 1, 64, 16), (2, 2, 72, 1), (8, 1, 128, 32), (9, 3, 128, 24), (6, 2, 136, 7), (9, 1, 64, 100),
    (1, 1, 256, 16), (16, 1, 192, 16), (40, 2, 96, 8), (1, 1, 384, 64), (3, 1, 512, 16), (5, 1, 640, 48), (1, 1, 320, 16), (4, 2, 896, 16),
    (2, 1, 768, 16), (2, 2, 904, 5), (1, 1, 1024, 16), (17, 1, 1024, 32),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_of_short_and_empty_requests(sru, Hq, Hkv, D, ps, dtype):
    _decode(sru, _decode_inputs(len(EDGES), Hq, Hkv, D, EDGES, ps, seed=D + Hq), dtype)


@pytest.mark.parametrize("lengths,Hq,Hkv,D,ps,window", [
    ([100003], 1, 1, 64, 64, 0),          # one request over every team
    ([20000], 8, 1, 128, 16, 0),
    ([9001], 1, 1, 1024, 48, 0),
    ([5000, 1, 3000, 0, 40, 2999] * 5, 4, 2, 128, 24, 0),
    ([5000, 1, 3000, 0, 40, 2999] * 5, 1, 1, 512, 32, 2560),
    ([777, 1000, 16, 17], 2, 1, 768, 16, 1),
    ([777, 1000, 16, 17], 12, 1, 256, 16, 100),
    (list(range(0, 400)), 1, 1, 64, 16, 0),
    ([33] * 3000, 1, 1, 128, 16, 0),
])
def test_attention_of_ragged_batches(sru, lengths, Hq, Hkv, D, ps, window):
    _decode(sru, _decode_inputs(len(lengths), Hq, Hkv, D, lengths, ps, seed=len(lengths)), torch.bfloat16,
            window=window)


def test_attention_of_sharp_and_equal_scores(sru):
    inp = list(_decode_inputs(3, 2, 1, 128, [500, 500, 40], 16, seed=9))
    _decode(sru, inp, torch.float32, scale=6.0)
    _decode(sru, inp, torch.float32, scale=0.0)
    _decode(sru, inp, torch.float32, scale=-1.0, with_lse=False)


def test_attention_far_into_a_large_cache(sru):
    """Pages whose elements lie beyond 2^31."""
    D, ps, pages = 1024, 64, 36000
    inp = _decode_inputs(2, 1, 1, D, [200, 90], ps, seed=3)
    q, kc, vc, table, lengths, K, V = inp
    big_k = torch.empty(pages, 1, ps, D, device="cuda", dtype=torch.bfloat16)
    big_v = torch.empty_like(big_k)
    assert (pages - kc.shape[0]) * ps * D > 2 ** 31
    big_k[-kc.shape[0]:] = kc
    big_v[-vc.shape[0]:] = vc
    moved = torch.where(table < kc.shape[0], table + pages - kc.shape[0], table)
    _decode(sru, (q, big_k, big_v, moved, lengths, K, V), torch.bfloat16)


def test_bad_pages_and_lengths_are_left_out_and_reported(sru):
    q, kc, vc, table, lengths, K, V = _decode_inputs(2, 1, 1, 128, [100, 64], 16, seed=4)
    table[0, 2] = kc.shape[0]          # keys 32..47
    table[0, 5] = -1                   # keys 80..95
    lengths[1] = 10 ** 9               # the table is 7 pages wide; its entries behind page 3 are out of range
    out = torch.empty(2, 1, 128, device="cuda")
    sru.sru_attention_decode(q, kc, vc, table, lengths, out)
    assert sru.sru_sync_status() == sru.SRU_ERR_INVALID
    assert sru.sru_sync_status() == sru.SRU_OK
    keep = torch.tensor([j for j in range(100) if not 32 <= j < 48 and not 80 <= j < 96], device="cuda")
    _check_decode(out, None, q, [K[0][keep], K[1]], [V[0][keep], V[1]], 128 ** -0.5, 0)


def test_the_same_bits_every_run_and_alone_or_in_a_batch_shape(sru):
    inp = _decode_inputs(40, 4, 2, 256, [(i * 397) % 3000 for i in range(40)], 16, seed=6)
    first = _decode(sru, inp, torch.float32)
    for _ in range(3):
        assert torch.equal(_decode(sru, inp, torch.float32), first)


def test_one_workspace_for_calls_of_any_shape_and_two_graphs(sru):
    """A workspace with anything in it, used by calls of other shapes in turn, and by two
    captured graphs that are replayed in turn."""
    shapes = [([20000], 8, 1, 128, 16), ([3000, 0, 700], 2, 1, 512, 32), ([40] * 50, 4, 4, 64, 16),
              ([9000, 8000], 1, 1, 1024, 64), ([5000] * 3, 16, 2, 96, 24)]
    inputs = [_decode_inputs(len(l), hq, hkv, d, l, ps, seed=i) for i, (l, hq, hkv, d, ps) in enumerate(shapes)]
    need = max(sru.sru_attention_decode_workspace_bytes(len(l), hq, hkv, d) for l, hq, hkv, d, _ in shapes)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    outs = [torch.empty(i[0].shape, device="cuda") for i in inputs]

    def call(k):
        q, kc, vc, table, lengths, K, V = inputs[k]
        sru.sru_attention_decode(q, kc, vc, table, lengths, outs[k], workspace=ws)

    for k in (0, 1, 2, 3, 4, 3, 1, 0):
        outs[k].fill_(float("nan"))
        call(k)
        assert sru.sru_sync_status() == 0
        _check_decode(outs[k], None, inputs[k][0], inputs[k][5], inputs[k][6], inputs[k][0].shape[2] ** -0.5, 0)
    graphs = []
    for k in (0, 3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(k)
        graphs.append((k, g))
    for _ in range(3):
        for k, g in graphs:
            outs[k].fill_(float("nan"))
            g.replay()
    assert sru.sru_sync_status() == 0
    for k in (0, 3):
        _check_decode(outs[k], None, inputs[k][0], inputs[k][5], inputs[k][6], inputs[k][0].shape[2] ** -0.5, 0)


def test_captured_between_copies_and_joined_streams(sru):
    """Captured calls whose predecessors are a copy, a fill, another stream's kernel and a
    kernel of the library, replayed on new data."""
    q, kc, vc, table, lengths, K, V = _decode_inputs(3, 2, 1, 256, [400, 77, 0], 16, seed=5)
    T, ps = 5, 16
    src, rows = torch.randn(3, 2, 256, device="cuda").bfloat16(), torch.randn(T, 1, 256, device="cuda").bfloat16()
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    out, out2, out3 = (torch.empty(3, 2, 256, device="cuda") for _ in range(3))
    qq = torch.zeros_like(q)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        qq.copy_(src)                                                    # a copy
        sru.sru_attention_decode(qq, kc, vc, table, lengths, out)
        out2.zero_()                                                     # a fill
        sru.sru_attention_decode(qq, kc, vc, table, lengths, out2)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            sru.sru_cache_append(rows, rows, slots, kc, vc)              # another stream, joined
        main.wait_stream(side)
        sru.sru_attention_decode(qq, kc, vc, table, lengths, out3)
        qq.add_(1)                                                       # a kernel that writes what was read

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        src.copy_(torch.randn(src.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        for o in (out, out2, out3):
            o.fill_(float("nan"))
        graph.replay()
        assert sru.sru_sync_status() == 0
        for o in (out, out2, out3):
            _check_decode(o, None, src, K, V, 1 / 16, 0)


def test_calls_one_after_another_without_a_wait(sru):
    """Forty calls in a row on one stream, each reading what the one before it wrote."""
    q, kc, vc, table, lengths, K, V = _decode_inputs(4, 2, 1, 128, [700, 300, 5, 64], 16, seed=8)
    x, y = q.clone(), torch.empty_like(q)
    want = q.clone()
    for _ in range(20):
        sru.sru_attention_decode(x, kc, vc, table, lengths, y)
        sru.sru_attention_decode(y, kc, vc, table, lengths, x)
    for _ in range(40):
        got = torch.empty_like(q)
        sru.sru_attention_decode(want, kc, vc, table, lengths, got)
        assert sru.sru_sync_status() == 0
        want = got
    assert torch.equal(x, want)


def _serve(sru, on_stream):
    """A few serving steps as a program runs them: extend, append, attend, with
    requests that come, grow and leave; then the same steps replayed from a graph."""
    B, Hq, Hkv, D, ps, maxp = 6, 4, 2, 128, 8, 12
    pages, T = 40, 64
    rng = np.random.default_rng(12)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(lengths)
    table = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
    free, count = _i32(rng.permutation(pages)), _i32([pages])
    offsets = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int32, device="cuda")
    kc = torch.full((pages, Hkv, ps, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    KV = torch.zeros(T, 2 * Hkv * D, device="cuda", dtype=torch.bfloat16)
    K, V = KV[:, : Hkv * D].unflatten(1, (Hkv, D)), KV[:, Hkv * D:].unflatten(1, (Hkv, D))
    q = torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(sru.sru_attention_decode_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def step():
        sru.sru_cache_extend(lengths, new, table, free, count, ps, lengths, count, offsets, slots)
        sru.sru_cache_append(K, V, slots, kc, vc)
        sru.sru_attention_decode(q, kc, vc, table, lengths, out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held_k, held_v = [torch.zeros(0, Hkv, D) for _ in range(B)], [torch.zeros(0, Hkv, D) for _ in range(B)]
    plan = [[9, 1, 0, 17, 3, 8], [1, 1, 30, 1, 1, 1], [1, -1, 1, 1, 1, 1], [1, 5, 1, -1, 1, 1], [1, 1, 1, 2, -1, 1],
            [1] * 6, [-1] * 6, [8, 16, 1, 9, 7, 2]]
    for i, adds in enumerate(plan):
        g = torch.Generator(device="cuda").manual_seed(i)
        KV.copy_(torch.randn(KV.shape, generator=g, device="cuda"))
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        new.copy_(_i32(adds))
        at = 0
        for b, n in enumerate(adds):
            if n < 0:
                held_k[b], held_v[b] = held_k[b][:0], held_v[b][:0]
                continue
            held_k[b] = torch.cat([held_k[b].cpu(), K[at:at + n].cpu()])
            held_v[b] = torch.cat([held_v[b].cpu(), V[at:at + n].cpu()])
            at += n
        if on_stream:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
        assert sru.sru_sync_status() == 0
        assert lengths.tolist() == [len(k) for k in held_k]
        assert int(count) == pages - sum(math.ceil(len(k) / ps) for k in held_k)
        live = [table[b, :math.ceil(len(held_k[b]) / ps)].tolist() for b in range(B)]
        taken = sum(live, []) + free[:int(count)].tolist()
        assert sorted(taken) == list(range(pages))  # every page is held once or free
        _check_decode(out, None, q, [k.cuda() for k in held_k], [v.cuda() for v in held_v], D ** -0.5, 0)


@pytest.mark.parametrize("on_stream", [False, True])
def test_serving_steps_with_pages_that_come_and_go(sru, on_stream):
    _serve(sru, on_stream)


def test_attention_agrees_with_the_attention_producer(sru):
    """The last token of SRU++'s causal attention producer, computed as serving does:
    the same Q, K, V (bf16) appended to the cache, then one token's attention,
    U = Wo (q + alpha a).  Both are within the library's bf16-projection class."""
    L, B, d, dp, alpha = 72, 3, 128, 64, 0.7
    g = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(L * B, d, generator=g, device="cuda").bfloat16()
    Wq = (torch.randn(dp, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    Wkv = (torch.randn(2 * dp, dp, generator=g, device="cuda") * dp ** -0.5).bfloat16()
    Wo = (torch.randn(3 * d, dp, generator=g, device="cuda") * dp ** -0.5).bfloat16()
    U = torch.empty(L * B, 3 * d, device="cuda")
    sru.sru_attention_project(X, Wq, Wkv, Wo, U, L, B, alpha)
    Q, KV = torch.empty(L * B, dp, device="cuda").bfloat16(), torch.empty(L * B, 2 * dp, device="cuda").bfloat16()
    sru.sru_project(X, Wq, Q)
    sru.sru_project(Q, Wkv, KV)
    ps, maxp = 16, 5
    table = _i32(np.random.default_rng(1).permutation(B * maxp).reshape(B, maxp))
    t, b = torch.arange(L * B, device="cuda") // B, torch.arange(L * B, device="cuda") % B
    slots = (table[b, t // ps] * ps + t % ps).int()
    kc = torch.empty(B * maxp, 1, ps, dp, device="cuda", dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    sru.sru_cache_append(KV[:, :dp].unflatten(1, (1, dp)), KV[:, dp:].unflatten(1, (1, dp)), slots, kc, vc)
    a = torch.empty(B, 1, dp, device="cuda")
    q = Q.view(L, B, 1, dp)[-1].contiguous()
    sru.sru_attention_decode(q, kc, vc, table, _i32([L] * B), a)
    assert sru.sru_sync_status() == 0
    U1 = (q.float() + alpha * a).view(B, dp) @ Wo.float().T
    want = U.view(L, B, -1)[-1]
    assert ((U1 - want).abs() <= 2e-2 * (1 + want.abs())).all()
