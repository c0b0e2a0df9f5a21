"""GPU parity of the vocabulary loss and its gradients against the formulas in
64 bits (torch float64 on the same bf16 inputs):
  z = H W^T, lse = logsumexp(z), loss = lse - z_t,
  dz = g (softmax(z) - onehot), dH = dz W, dW = dz^T H.

Tolerances.  A logit is an fp32 sum of products: off by at most 1e-5 S with
S = sum_k |h_k w_k| (the bound that every fp32 product of this library is held
to).  lse moves by at most the largest logit error of its row, plus fp32
rounding of values of its size: 1e-5 (max_v S + 1 + |lse|) =: e.  The loss adds
the target's logit: twice that.  dz = g (p - [v = t]) has p off by a factor
exp(+-2e), and is rounded to bf16 (half a step: 2^-8 of the value): each dz is
off by at most 3 e g p + 2^-8 |dz| =: d, hence dH by sum_v d |W| plus the fp32
sum (1e-5 sum |dz W|) plus, as bf16, 2^-8 |dH|; dW the same with H.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sru():
    import parallelizable_recurrence_b200 as m
    m.load_library()
    return m


def _inputs(M, V, K, std=2.0, ignored=0.1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + M + V + K)
    H = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, K, generator=g, device="cuda") * std * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[torch.rand(M, generator=g, device="cuda") < ignored] = -100
    w = torch.rand(M, generator=g, device="cuda") + 0.5
    return H, W, t, w


def _reference(H, W, t, w):
    """Values and error bounds of (loss, lse, dH, dW) before the output's own rounding, in pieces of rows."""
    Wd, Wa = W.double(), W.double().abs()
    V, K = W.shape
    out = {k: [] for k in ("loss", "lse", "e", "dH", "bH")}
    dW = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    bW = torch.zeros_like(dW)
    step = max(1, (1 << 27) // V)
    for i in range(0, H.shape[0], step):
        h, ti, wi = H[i:i + step].double(), t[i:i + step], w[i:i + step].double()
        z, S = h @ Wd.T, h.abs() @ Wa.T
        lse = torch.logsumexp(z, 1)
        e = 1e-5 * (S.amax(1) + 1 + lse.abs())
        there = ti >= 0
        zt = z.gather(1, ti.clamp(min=0)[:, None])[:, 0]
        p = torch.exp(z - lse[:, None])
        g = torch.where(there, wi, 0.0)
        dz = p * g[:, None]
        err = 3 * e[:, None] * dz
        dz[there, ti[there]] -= g[there]
        err += 2.0 ** -8 * dz.abs()
        err += 1e-5 * dz.abs()
        out["loss"].append(torch.where(there, lse - zt, 0.0))
        out["lse"].append(lse)
        out["e"].append(e)
        out["dH"].append(dz @ Wd)
        out["bH"].append(err @ Wa)
        dW += dz.T @ h
        bW += err.T @ h.abs()
    r = {k: torch.cat(v) for k, v in out.items()}
    r.update(dW=dW, bW=bW)
    return r


def _within(name, got, ref, tol):
    got = got.double()
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - tol
    assert over.max() <= 0, f"{name}: beyond the tolerance by {over.max():.3e} at {int(over.argmax())}"


def _run(sru, H, W, t, w, dtype):
    M, K = H.shape
    loss, lse = torch.full((M,), float("nan"), device="cuda"), torch.full((M,), float("nan"), device="cuda")
    dH = torch.full((M, K), float("nan"), device="cuda", dtype=dtype)
    dW = torch.full((W.shape[0], K), float("nan"), device="cuda", dtype=dtype)
    sru.sru_softmax_loss(H, W, t, loss, lse)
    sru.sru_softmax_loss_backward(H, W, t, lse, w, dH, dW)
    assert sru.sru_sync_status() == 0
    return loss, lse, dH, dW


def _check(sru, H, W, t, w, dtype):
    loss, lse, dH, dW = _run(sru, H, W, t, w, dtype)
    r = _reference(H, W, t, w)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    _within("lse", lse, r["lse"], r["e"])
    _within("loss", loss, r["loss"], 2 * r["e"])
    # (1e-30: gradients of rows whose every probability underflows)
    _within("dH", dH, r["dH"], r["bH"] + half * (r["dH"].abs() + r["bH"]) + 1e-30)
    _within("dW", dW, r["dW"], r["bW"] + half * (r["dW"].abs() + r["bW"]) + 1e-30)
    assert (loss[t < 0] == 0).all() and (dH[t < 0] == 0).all()


@pytest.mark.parametrize("M,V,K", [
    (1, 1, 8),          # one row, one class: loss 0
    (1, 1000, 64),
    (3, 2, 16),
    (255, 257, 72),     # one column behind a tile
    (257, 4099, 520),   # one row behind a tile, odd vocabulary, ragged k-blocks
    (129, 255, 64),
    (1000, 513, 1024),
    (300, 20011, 64),   # few row tiles: dH split along the vocabulary
    (16500, 300, 136),  # few vocabulary tiles: dW split along the rows
    (2048, 32000, 512),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_loss_and_gradients_match_the_formulas(sru, M, V, K, dtype):
    _check(sru, *_inputs(M, V, K), dtype)


@pytest.mark.parametrize("M,V,K", [
    (300000, 2100, 16),  # three pieces of the vocabulary, the last one short
    (5000, 60000, 64),   # two pieces, dH split along the vocabulary in both
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_pieces_of_the_vocabulary(sru, M, V, K, dtype):
    _check(sru, *_inputs(M, V, K), dtype)


def test_sharp_and_flat_rows(sru):
    """Logits of +-300 (all but one probability underflow) and all-equal logits."""
    H, W, t, w = _inputs(200, 3001, 64, std=40.0)
    H[100:] = 0
    _check(sru, H, W, t, w, torch.float32)


@pytest.mark.parametrize("M,V,K", [
    (2304, 3000, 256),   # whole rounds of dH tiles and a partial one, dW interleaved
    (18944, 500, 256),   # 74 dH tiles: one whole round on 148 SMs
    (700, 19000, 1024),
])
def test_the_gradients_share_a_launch(sru, M, V, K):
    _check(sru, *_inputs(M, V, K, seed=2), torch.bfloat16)


def test_weights_of_any_size(sru):
    """dz is held over the largest weight: weights over 30 powers of ten, zeros among
    them, and NaN and infinity on rows that do not count."""
    H, W, t, w = _inputs(400, 1200, 64, seed=3)
    w = torch.logspace(-25, 5, 400, device="cuda")[torch.randperm(400, device="cuda")]
    w[::7] = 0.0
    want = w.clone()
    w[t < 0] = float("nan")
    w[(t < 0).nonzero()[0]] = float("inf")
    loss, lse, dH, dW = _run(sru, H, W, t, w, torch.float32)
    r = _reference(H, W, t, want)
    # (a weight far below the largest is held over it: smaller than 2^-126 of it, it may vanish)
    tiny = float(want.max()) * 2.0 ** -126 * W.double().abs().sum(0).max()
    _within("dH", dH, r["dH"], r["bH"] + 2.0 ** -24 * r["dH"].abs() + tiny)
    _within("dW", dW, r["dW"], r["bW"] + 2.0 ** -24 * r["dW"].abs() + tiny)
    assert (dH[want == 0] == 0).all()
    w = torch.zeros_like(w)
    _, _, dH, dW = _run(sru, H, W, t, w, torch.float32)
    assert (dH == 0).all() and (dW == 0).all()


def test_equal_weights_do_not_share_a_rounding_error(sru):
    """1 / 1001 is 2.7e-3 off in bf16.  The gradients' norm is not off by that: every
    row's p - 1 is rounded on its own, so the sum over 64 x 1001 of them is within a
    fifth of half a step."""
    H, W, t, _ = _inputs(1001, 5000, 64, ignored=0.0, seed=4)
    w = torch.full((1001,), 1.0 / 1001, device="cuda")
    _, _, dH, dW = _run(sru, H, W, t, w, torch.float32)
    r = _reference(H, W, t, w)
    for got, ref in ((dH, r["dH"]), (dW, r["dW"])):
        along = float((got.double() * ref).sum() / (ref * ref).sum())
        assert abs(along - 1) < 0.2 * 2.0 ** -8


def test_no_row_counts(sru):
    H, W, t, w = _inputs(70, 500, 64)
    t.fill_(-1)
    w[::2] = float("nan")  # weights of rows that do not count are not used
    loss, lse, dH, dW = _run(sru, H, W, t, w, torch.float32)
    assert (loss == 0).all() and (dH == 0).all() and (dW == 0).all() and torch.isfinite(lse).all()


def test_a_row_of_nan_stays_in_its_row(sru):
    H, W, t, w = _inputs(300, 700, 64, ignored=0.0)
    clean = _run(sru, H, W, t, w, torch.float32)
    H[7] = float("nan")
    loss, lse, dH, _ = _run(sru, H, W, t, w, torch.float32)
    rows = torch.arange(300, device="cuda") != 7
    assert loss[7].isnan() and lse[7].isnan() and dH[7].isnan().all()
    for a, b in ((loss, clean[0]), (lse, clean[1]), (dH, clean[2])):
        assert torch.equal(a[rows], b[rows])


def test_no_rows(sru):
    W = torch.randn(300, 64, device="cuda").bfloat16()
    H, t = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, device="cuda", dtype=torch.int64)
    f = torch.empty(0, device="cuda")
    dW = torch.full((300, 64), float("nan"), device="cuda")
    sru.sru_softmax_loss(H, W, t, f, f)
    sru.sru_softmax_loss_backward(H, W, t, f, f, torch.empty(0, 64, device="cuda"), dW)
    assert sru.sru_sync_status() == 0 and (dW == 0).all()


def test_either_gradient_alone_has_the_same_bits(sru):
    H, W, t, w = _inputs(700, 5003, 200)
    _, lse, dH, dW = _run(sru, H, W, t, w, torch.float32)
    a, b = torch.empty_like(dH), torch.empty_like(dW)
    sru.sru_softmax_loss_backward(H, W, t, lse, w, dH=a)
    sru.sru_softmax_loss_backward(H, W, t, lse, w, dW=b)
    assert sru.sru_sync_status() == 0
    assert torch.equal(a, dH) and torch.equal(b, dW)


def test_a_target_behind_the_vocabulary_is_reported(sru):
    H, W, t, w = _inputs(40, 300, 64, ignored=0.0)
    t[3], t[9] = 300, 1 << 40
    M, K = H.shape
    loss, lse, dH = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, device="cuda")
    sru.sru_softmax_loss(H, W, t, loss, lse)
    assert sru.sru_sync_status() == sru.SRU_ERR_INVALID
    assert sru.sru_sync_status() == sru.SRU_OK
    sru.sru_softmax_loss_backward(H, W, t, lse, w, dH)
    assert sru.sru_sync_status() == sru.SRU_OK
    t[3] = t[9] = -1
    r = _reference(H, W, t, w)
    _within("loss", loss, r["loss"], 2 * r["e"])
    _within("dH", dH, r["dH"], r["bH"] + 2.0 ** -24 * r["dH"].abs())


def test_captured_on_another_stream_and_replayed_on_new_inputs(sru):
    H, W, t, w = _inputs(500, 3001, 128)
    M, V, K = 500, 3001, 128
    ws = torch.empty(sru.sru_softmax_loss_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dH, dW = torch.empty(M, K, device="cuda"), torch.empty(V, K, device="cuda")

    def step():
        sru.sru_softmax_loss(H, W, t, loss, lse, workspace=ws)
        sru.sru_softmax_loss_backward(H, W, t, lse, w, dH, dW, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    H2, W2, t2, w2 = _inputs(500, 3001, 128, seed=1)
    for a, b in ((H, H2), (W, W2), (t, t2), (w, w2)):
        a.copy_(b)
    ws.fill_(0xff)
    graph.replay()
    assert sru.sru_sync_status() == 0
    want = _run(sru, H2, W2, t2, w2, torch.float32)
    for a, b in zip((loss, lse, dH, dW), want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    sru.sru_softmax_loss(H, W, t, loss, lse, stream=side)
    assert sru.sru_sync_status(side) == 0
    assert torch.equal(loss, want[0])


def test_gradients_against_differences(sru):
    """Central differences of the GPU's own loss along random +-1 directions.  H and W
    hold multiples of 2^-4 and 2^-6 that stay exact in bf16 when moved by one step.
    The logits move by a = step (w . s) of standard deviation 2^-4 x 1/2 along rows
    of H; the difference quotient is off by at most max|w . s|^3 step^2 / 6 <=
    (0.5 x 6)^3 2^-8 / 6 < 0.02, and the loss's rounding (1e-5 (1 + 6 + S)) / step
    < 0.01; dH itself is within the tolerances of the tests above."""
    M, V, K = 64, 301, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    H = (torch.randint(-16, 17, (M, K), generator=g, device="cuda") / 16).bfloat16()
    W = (torch.randint(-6, 7, (V, K), generator=g, device="cuda") / 64).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    w = torch.ones(M, device="cuda")
    _, _, dH, dW = _run(sru, H, W, t, w, torch.float32)

    def total(H, W):
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        sru.sru_softmax_loss(H, W, t, loss, lse)
        return loss.double()

    s = torch.randint(0, 2, (M, K), generator=g, device="cuda").double() * 2 - 1
    step = 2.0 ** -4
    quotient = (total((H.double() + step * s).bfloat16(), W) - total((H.double() - step * s).bfloat16(), W)) / (2 * step)
    assert ((dH.double() * s).sum(1) - quotient).abs().max() < 0.05
    # one row of W at a time, by 2^-6: the loss of every row moves by a = 2^-6 (h . s)
    s = torch.randint(0, 2, (K,), generator=g, device="cuda").double() * 2 - 1
    step = 2.0 ** -6
    for v in (int(t[0]), 0, V - 1):
        up, down = W.double().clone(), W.double().clone()
        up[v] += step * s
        down[v] -= step * s
        quotient = (total(H, up.bfloat16()).sum() - total(H, down.bfloat16()).sum()) / (2 * step)
        # off by M (max|h . s|^3 step^2) / 6 x p (p about 1/V) < 0.04, plus M losses' rounding, each
        # 1e-5 (S + 1 + lse) < 1e-4, over the step: < 0.41
        assert abs(float((dW[v].double() * s).sum() - quotient)) < 0.45
