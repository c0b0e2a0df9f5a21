"""Calls of the paged cache and of the vocabulary loss among other calls: one after another without a
wait, each reading what the one before it wrote, and two at once on two streams.  Every result
must have the bits that the same call gives when each call is waited for.
"""
import numpy as np
import pytest
import torch

from test_gpu_cache import _decode_inputs, _extend_reference, _i32
from test_gpu_loss import _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sru():
    import parallelizable_recurrence_b200 as m
    m.load_library()
    return m


# B requests, rows per step; the second has the rows kernel behind the bookkeeping and long runs of slots
@pytest.mark.parametrize("B,maxp,T,most", [(24, 8, 64, 3), (40, 30, 2500, 60)])
def test_serving_calls_in_a_row_read_what_was_just_written(sru, B, maxp, T, most):
    """Extend, append and attend on the same buffers, whose contents change at every step."""
    Hq, Hkv, D, ps, steps = 4, 2, 128, 8, 24
    pages = B * maxp
    rng = np.random.default_rng(B)
    adds = rng.integers(0, most + 1, (steps, B))
    adds[rng.random((steps, B)) < 0.05] = -1
    order = rng.permutation(pages)
    g = torch.Generator(device="cuda").manual_seed(B)
    new = _i32(adds)
    KV = torch.randn(steps, T, 2, Hkv, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(steps, B, Hq, D, generator=g, device="cuda").bfloat16()
    ws = torch.empty(sru.sru_attention_decode_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def serve(wait):
        lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
        table = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
        free, count = _i32(order), _i32([pages])
        offsets, slots = torch.zeros_like(_i32(range(B + 1))), torch.zeros(T, dtype=torch.int32, device="cuda")
        kc = torch.zeros(pages, Hkv, ps, D, device="cuda", dtype=torch.bfloat16)
        vc = torch.zeros_like(kc)
        out = torch.zeros(steps, B, Hq, D, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        for i in range(steps):
            sru.sru_cache_extend(lengths, new[i], table, free, count, ps, lengths, count, offsets, slots)
            if wait:
                torch.cuda.synchronize()
            sru.sru_cache_append(KV[i, :, 0], KV[i, :, 1], slots, kc, vc)
            if wait:
                torch.cuda.synchronize()
            sru.sru_attention_decode(q[i], kc, vc, table, lengths, out[i], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        assert sru.sru_sync_status() == 0
        return lengths, table, free, count, offsets, slots, kc, vc, out

    want = serve(True)
    for _ in range(3):
        for got, ref in zip(serve(False), want):
            assert torch.equal(got, ref)
    # the bookkeeping and the caches by the definition, too
    n, table, free, count = [0] * B, [[-1] * maxp for _ in range(B)], order.tolist(), pages
    kc = torch.zeros(pages, Hkv, ps, D, device="cuda", dtype=torch.bfloat16)
    for i in range(steps):
        table, free, n, count, offsets, slots, _ = _extend_reference(n, adds[i].tolist(), table, free, count, ps, T)
        at = torch.tensor(slots, device="cuda")
        there = at >= 0
        kc[at[there] // ps, :, at[there] % ps] = KV[i, there, 0]
    assert want[0].tolist() == n and int(want[3]) == count and want[5].tolist() == slots
    assert torch.equal(want[6], kc)


def test_losses_in_a_row_read_what_was_just_written(sru):
    """Losses and gradients of several batches through the same buffers, the workspace
    shared, each gradient the rows of the next loss."""
    M, V, K = 1100, 2000, 128
    H, W, t, w = _inputs(M, V, K, seed=6)
    ws = torch.empty(sru.sru_softmax_loss_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")

    def steps(wait):
        rows = [H.clone(), torch.empty_like(H)]
        loss, lse = torch.zeros(6, M, device="cuda"), torch.zeros(6, M, device="cuda")
        dW = torch.zeros(6, V, K, device="cuda")
        torch.cuda.synchronize()
        for i in range(6):
            sru.sru_softmax_loss(rows[i % 2], W, t, loss[i], lse[i], workspace=ws)
            if wait:
                torch.cuda.synchronize()
            sru.sru_softmax_loss_backward(rows[i % 2], W, t, lse[i], w, rows[(i + 1) % 2], dW[i], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        assert sru.sru_sync_status() == 0
        return loss, lse, dW, rows[0]

    want = steps(True)
    for _ in range(3):
        for got, ref in zip(steps(False), want):
            assert torch.equal(got, ref)


def _at_once(sru, first, second):
    """first on the current stream, then second on another one while it runs; and the other way round."""
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for a, b in ((first, second), (second, first)):
        for _ in range(3):
            side.wait_stream(torch.cuda.current_stream())
            a(stream=None)
            b(stream=side)
            a(stream=None)
            b(stream=side)
            torch.cuda.current_stream().wait_stream(side)
    assert sru.sru_sync_status() == 0


def test_losses_without_a_workspace_on_two_streams_at_once(sru):
    sizes = [(2048, 20000, 512), (2048, 19000, 512)]
    calls, got, want = [], [], []
    for i, (M, V, K) in enumerate(sizes):
        H, W, t, w = _inputs(M, V, K, seed=i)
        out = [torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, device="cuda"),
               torch.empty(V, K, device="cuda")]

        def call(stream, H=H, W=W, t=t, w=w, out=out):
            sru.sru_softmax_loss(H, W, t, out[0], out[1], stream=stream)
            sru.sru_softmax_loss_backward(H, W, t, out[1], w, out[2], out[3], stream=stream)

        call(None)
        torch.cuda.synchronize()
        want.append([x.clone() for x in out])
        calls.append(call)
        got.append(out)
    _at_once(sru, *calls)
    for a, b in zip(sum(got, []), sum(want, [])):
        assert torch.equal(a, b)


def test_attention_without_a_workspace_on_two_streams_at_once(sru):
    # (long, and every request in pieces that cross the CTAs' borders)
    calls, got, want = [], [], []
    for i, lengths in enumerate(([7001] * 21, [6500] * 23)):
        q, kc, vc, table, lengths, _, _ = _decode_inputs(len(lengths), 1, 1, 1024, lengths, 16, seed=i)
        out = torch.empty(q.shape, device="cuda")

        def call(stream, q=q, kc=kc, vc=vc, table=table, lengths=lengths, out=out):
            sru.sru_attention_decode(q, kc, vc, table, lengths, out, stream=stream)

        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
        calls.append(call)
        got.append(out)
    _at_once(sru, *calls)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_decode_steps_without_a_workspace_on_two_streams_at_once(sru):
    """(8 rows: the product runs in the workspace that the call allocates)"""
    d, B = 2048, 8
    calls, got, want = [], [], []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(i)
        X = torch.randn(B, d, generator=g, device="cuda").bfloat16()
        W = (torch.randn(3 * d, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
        x, c0 = X.float(), torch.randn(B, d, generator=g, device="cuda")
        v, b = torch.randn(2, d, generator=g, device="cuda"), torch.randn(2, d, generator=g, device="cuda")
        c, h = c0.clone(), torch.empty(B, d, device="cuda")

        def call(stream, X=X, W=W, x=x, v=v, b=b, c=c, h=h):
            sru.sru_decode_step(X, W, x, v, b, c, h, stream=stream)

        for _ in range(12):  # as often as both streams take it below: the state runs on
            call(None)
        torch.cuda.synchronize()
        want.append([c.clone(), h.clone()])
        c.copy_(c0)
        calls.append(call)
        got.append([c, h])
    _at_once(sru, *calls)
    for a, b in zip(sum(got, []), sum(want, [])):
        assert torch.equal(a, b)


def test_captured_on_a_forked_stream_without_a_workspace(sru):
    """A graph whose calls allocate their own workspaces, on the capturing stream and on one forked from
    it, replayed on new inputs."""
    M, V, K = 300, 2000, 64
    H, W, t, w = _inputs(M, V, K)
    q, kc, vc, table, lengths, _, _ = _decode_inputs(3, 2, 1, 512, [9000, 40, 2000], 16, seed=2)
    loss, lse, dH = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, device="cuda")
    out, out2 = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        sru.sru_attention_decode(q, kc, vc, table, lengths, out)
        sru.sru_softmax_loss(H, W, t, loss, lse, stream=side)
        sru.sru_softmax_loss_backward(H, W, t, lse, w, dH, stream=side)
        sru.sru_attention_decode(q, kc, vc, table, lengths, out2, stream=side)
        main.wait_stream(side)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        H.copy_(_inputs(M, V, K, seed=seed)[0])
        q.copy_(torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        step()
        assert sru.sru_sync_status() == 0
        torch.cuda.synchronize()
        want = [x.clone() for x in (loss, lse, dH, out, out2)]
        assert torch.equal(out, out2)
        for x in (loss, lse, dH, out, out2):
            x.fill_(float("nan"))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert sru.sru_sync_status() == 0
        for x, y in zip((loss, lse, dH, out, out2), want):
            assert torch.equal(x, y)
