"""Workloads of the paged-cache attention and of the vocabulary loss.

Each case is one pass through one of these operators, as a program calls it:

  extend   sru_cache_extend: block table, slot map and lengths of one serving
           step, from the requests' lengths and new tokens
  append   sru_cache_append: the step's K and V rows into the paged cache
  decode   sru_attention_decode: attention of one new token per request over
           the paged cache
  loss     sru_softmax_loss: softmax cross entropy over the vocabulary
  train    sru_softmax_loss and sru_softmax_loss_backward: the loss and its
           gradients with respect to the rows and the output matrix

With ``own`` false, run() computes the same in elementary torch operations
(fp32, rounded once at the end).
"""
import math

import numpy as np
import torch

own = False


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one step of a small serving batch: a token per request, a few requests finish
        {"name": "extend_step_b48", "op": "extend", "B": 48, "max_len": 2560, "page": 16, "mode": "step"},
        # admission of a wave of prompts next to running requests, large pages
        {"name": "extend_prefill_b1024", "op": "extend", "B": 1024, "max_len": 4096, "page": 64, "mode": "prefill"},
        # one step's K and V rows, eight shared heads
        {"name": "append_step_t64_h8_d128", "op": "append", "T": 64, "H": 8, "D": 128, "page": 16, "src": "bf16"},
        # prompts of 16384 tokens in all through one SRU++ head of the training layer's d' = 512
        {"name": "append_prefill_t16384_d512", "op": "append", "T": 16384, "H": 1, "D": 512, "page": 64,
         "src": "bf16"},
        # batch-1 interactive decoding early in a text: latency
        {"name": "decode_b1_len200_d512", "op": "decode", "B": 1, "Hq": 1, "Hkv": 1, "D": 512, "max_len": 200,
         "page": 16, "window": 0},
        # SRU++ serving batch at the test context of 2560 tokens, ragged lengths, context bounded by a window
        {"name": "decode_b64_len5000_d512_w2560", "op": "decode", "B": 64, "Hq": 1, "Hkv": 1, "D": 512,
         "max_len": 5000, "page": 32, "window": 2560},
        # many query heads over shared key heads, odd page size
        {"name": "decode_b24_len6007_h32_8_d128", "op": "decode", "B": 24, "Hq": 32, "Hkv": 8, "D": 128,
         "max_len": 6007, "page": 24, "window": 0},
        # a large batch of long contexts through wide heads: the cache read at full rate
        {"name": "decode_b96_len8192_d1024", "op": "decode", "B": 96, "Hq": 1, "Hkv": 1, "D": 1024, "max_len": 8192,
         "page": 64, "window": 0},
        # scoring a short text, odd vocabulary
        {"name": "loss_m250_v10007_k512", "op": "loss", "M": 250, "V": 10007, "K": 512, "ignored": 0.0},
        # evaluation of the training layer's batch of rows
        {"name": "loss_m16384_v32000_k1024", "op": "loss", "M": 16384, "V": 32000, "K": 1024, "ignored": 0.05},
        # a small training step, ragged rows and vocabulary
        {"name": "train_m1001_v20011_k520", "op": "train", "M": 1001, "V": 20011, "K": 520, "ignored": 0.1},
        # the training layer's step: L1024 B16 rows of d2048 over a vocabulary of 32000
        {"name": "train_m16384_v32000_k2048", "op": "train", "M": 16384, "V": 32000, "K": 2048, "ignored": 0.05},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "append", "decode", "decode", "loss", "train"])
    while True:
        if op == "extend":
            c = {"op": op, "B": _log_int(rng, 1, 1024), "max_len": _log_int(rng, 64, 4096),
                 "page": rng.choice([8, 16, 24, 32, 64, 100]), "mode": rng.choice(["step", "prefill"])}
        elif op == "append":
            c = {"op": op, "T": _log_int(rng, 1, 16384), "H": rng.choice([1, 1, 2, 4, 8]),
                 "D": rng.choice([64, 72, 128, 192, 256, 512, 768, 1024]), "page": rng.choice([8, 16, 24, 32, 64]),
                 "src": rng.choice(["bf16", "fp32"])}
        elif op == "decode":
            hkv, g = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 1, 2, 3, 4, 8, 16])
            max_len = _log_int(rng, 16, 8192)
            c = {"op": op, "B": _log_int(rng, 1, 128), "Hq": hkv * g, "Hkv": hkv,
                 "D": rng.choice([64, 72, 96, 128, 192, 256, 384, 512, 768, 1024]), "max_len": max_len,
                 "page": rng.choice([8, 16, 24, 32, 64, 128]),
                 "window": rng.choice([0, 0, 0, max(1, max_len // rng.choice([2, 3]))])}
        else:
            c = {"op": op, "M": _log_int(rng, 1, 16384), "V": _log_int(rng, 1000, 50000),
                 "K": 8 * _log_int(rng, 8, 256), "ignored": rng.choice([0.0, 0.1, 0.5])}
        most = {x["op"]: x for x in listed()}[op]  # the last listed case of each operator is its largest
        w, m = work(c), work(most)
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"]:
            return c


# ---------------------------------------------------------------- the inputs
def _lengths(case, seed):
    """Tokens held by each request: spread over [1, max_len], the longest at max_len."""
    r = np.random.default_rng([seed, 1])
    n = r.integers(max(1, case["max_len"] // 8), case["max_len"] + 1, case["B"])
    n[r.integers(case["B"])] = case["max_len"]
    return n


def _sizes(case):
    """(table width, pages of the cache) of a serving case."""
    maxp = -(-case["max_len"] // case["page"])
    return maxp, case["B"] * maxp


def _page_order(case, seed):
    return np.random.default_rng([seed, 2]).permutation(_sizes(case)[1])


def _extend_inputs(case, seed):
    """Lengths, new tokens, block table, free stack and its height, on the host."""
    r = np.random.default_rng([seed, 3])
    B, ps = case["B"], case["page"]
    maxp, pages = _sizes(case)
    lengths = r.integers(0, case["max_len"], B)
    new = np.ones(B, np.int64)
    if case["mode"] == "prefill":  # a quarter of the requests bring a prompt, the rest take a step
        prompt = r.random(B) < 0.25
        lengths[prompt] = 0
        new[prompt] = r.integers(1, case["max_len"] + 1, int(prompt.sum()))
    new[r.random(B) < 0.08] = -1
    held = -(-lengths // ps)
    order = _page_order(case, seed)
    table = np.full((B, maxp), -1, np.int64)
    table[np.arange(maxp)[None, :] < held[:, None]] = order[: held.sum()]
    free = np.full(pages, -1, np.int64)
    n_free = pages - int(held.sum())
    free[:n_free] = order[held.sum():]
    # rows of K and V that the step has room for: more than it has tokens (a padded batch)
    rows = B + 5 if case["mode"] == "step" else case["max_len"] + B * case["max_len"] // 7
    return lengths, new, table, free, n_free, rows


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)


def _normal(shape, seed, dev, dtype, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    op = case["op"]
    s = {"case": dict(case)}
    if op == "extend":
        lengths, new, table, free, n_free, rows = _extend_inputs(case, seed)
        s.update(lengths=_i32(lengths, dev), new=_i32(new, dev), table=_i32(table, dev), free=_i32(free, dev),
                 n_free=_i32([n_free], dev), lengths_out=torch.empty(case["B"], dtype=torch.int32, device=dev),
                 n_free_out=torch.empty(1, dtype=torch.int32, device=dev),
                 offsets=torch.empty(case["B"] + 1, dtype=torch.int32, device=dev),
                 slots=torch.empty(rows, dtype=torch.int32, device=dev),
                 refused=torch.empty(1, dtype=torch.int32, device=dev))
    elif op == "append":
        T, H, D, ps = case["T"], case["H"], case["D"], case["page"]
        r = np.random.default_rng([seed, 4])
        pages = -(-T // ps) + 8
        slots = r.permutation(pages)[np.arange(T) // ps] * ps + np.arange(T) % ps
        slots[r.random(T) < 0.02] = -1  # rows of a padded batch
        src = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        KV = _normal((T, 2 * H * D), seed, dev, src)  # [K | V], as one product writes them
        s.update(K=KV[:, : H * D].unflatten(1, (H, D)), V=KV[:, H * D:].unflatten(1, (H, D)), slots=_i32(slots, dev),
                 k_cache=torch.zeros(pages, H, ps, D, dtype=torch.bfloat16, device=dev),
                 v_cache=torch.zeros(pages, H, ps, D, dtype=torch.bfloat16, device=dev))
    elif op == "decode":
        B, D = case["B"], case["D"]
        maxp, pages = _sizes(case)
        lengths = _lengths(case, seed)
        table = _page_order(case, seed).reshape(B, maxp).copy()
        table[np.arange(maxp)[None, :] >= (-(-lengths // case["page"]))[:, None]] = -1
        shape = (pages, case["Hkv"], case["page"], D)
        s.update(q=_normal((B, case["Hq"], D), seed, dev, torch.bfloat16), table=_i32(table, dev),
                 k_cache=_normal(shape, seed + 1, dev, torch.bfloat16),
                 v_cache=_normal(shape, seed + 2, dev, torch.bfloat16), lengths=_i32(lengths, dev),
                 out=torch.empty(B, case["Hq"], D, dtype=torch.bfloat16, device=dev))
        if own:
            import parallelizable_recurrence_b200 as sru
            n = sru.sru_attention_decode_workspace_bytes(B, case["Hq"], case["Hkv"], D)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        M, V, K = case["M"], case["V"], case["K"]
        r = np.random.default_rng([seed, 5])
        targets = r.integers(0, V, M)
        targets[r.random(M) < case["ignored"]] = -100
        # logits of standard deviation 2, a weight per row as a mean over the counted rows gives
        s.update(H=_normal((M, K), seed, dev, torch.bfloat16),
                 W=_normal((V, K), seed + 1, dev, torch.bfloat16, 2.0 * K ** -0.5),
                 targets=torch.from_numpy(targets).to(dev), loss=torch.empty(M, device=dev),
                 lse=torch.empty(M, device=dev),
                 dloss=torch.full((M,), 1.0 / max(1, int((targets >= 0).sum())), device=dev))
        if op == "train":
            s.update(dH=torch.empty(M, K, dtype=torch.bfloat16, device=dev),
                     dW=torch.empty(V, K, dtype=torch.bfloat16, device=dev))
        if own:
            import parallelizable_recurrence_b200 as sru
            n = sru.sru_softmax_loss_workspace_bytes(M, V, K, op == "train")
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return {"extend": _extend, "append": _append, "decode": _decode, "loss": _loss, "train": _train}[op](state)


def _extend(s):
    ps = s["case"]["page"]
    if own:
        import parallelizable_recurrence_b200 as sru
        sru.sru_cache_extend(s["lengths"], s["new"], s["table"], s["free"], s["n_free"], ps, s["lengths_out"],
                             s["n_free_out"], s["offsets"], s["slots"], refused=s["refused"])
    else:
        B, maxp = s["table"].shape
        T, pages = s["slots"].numel(), s["free"].numel()
        dev = s["table"].device
        lengths, new, table = s["lengths"].long(), s["new"].long(), s["table"].long()
        col = torch.arange(maxp, device=dev)[None, :]
        held = (lengths + ps - 1) // ps
        grow = new.clamp(min=0)
        last = grow.cumsum(0)
        first = last - grow
        # the released requests' pages go onto the stack in request order
        gone = torch.where(new < 0, held, 0)
        base = s["n_free"].long() + gone.cumsum(0) - gone
        avail = s["n_free"].long() + gone.sum()
        put = torch.where(col < gone[:, None], base[:, None] + col, pages)
        stack = torch.cat([s["free"].long(), s["free"].new_zeros(1).long()])
        stack = stack.scatter(0, put.flatten(), table.flatten())
        # pages are granted in request order while the stack lasts
        end = lengths + grow
        fits = (grow > 0) & (end <= maxp * ps) & (last <= T)
        need = torch.where(fits, (end + ps - 1) // ps - held, 0)
        total = need.cumsum(0)
        ok = fits & ((need == 0) | (total <= avail))
        take = torch.where(ok, need, 0)
        rank = (total - need)[:, None] + col - held[:, None]
        mine = (col >= held[:, None]) & (col < (held + take)[:, None])
        table = torch.where(mine, stack[(avail - 1 - rank).clamp(0, pages)], table)
        # a slot for every new token, -1 behind the last
        row = torch.arange(T, device=dev)
        b = torch.searchsorted(last, row, right=True)
        there = b < B
        b = b.clamp(max=B - 1)
        pos = lengths[b] + row - first[b]
        slot = table[b, (pos // ps).clamp(0, maxp - 1)] * ps + pos % ps
        s["slots"].copy_(torch.where(there & ok[b], slot, -1))
        s["table"].copy_(table)
        s["free"].copy_(stack[:pages])
        s["lengths_out"].copy_(torch.where(new < 0, 0, torch.where(ok, end, lengths)))
        s["n_free_out"].copy_(avail - take.sum())
        s["offsets"].copy_(torch.cat([first[:1], last]))
        s["refused"].copy_(((grow > 0) & ~ok).sum())
    return [s[k] for k in ("table", "free", "lengths_out", "n_free_out", "offsets", "slots", "refused")]


def _append(s):
    if own:
        import parallelizable_recurrence_b200 as sru
        sru.sru_cache_append(s["K"], s["V"], s["slots"], s["k_cache"], s["v_cache"])
    else:
        ps, slots = s["case"]["page"], s["slots"].long()
        keep = slots >= 0
        slots = slots[keep]
        s["k_cache"][slots // ps, :, slots % ps] = s["K"][keep].to(torch.bfloat16)
        s["v_cache"][slots // ps, :, slots % ps] = s["V"][keep].to(torch.bfloat16)
    return [s["k_cache"], s["v_cache"]]


def _decode(s):
    c = s["case"]
    scale = c["D"] ** -0.5
    if own:
        import parallelizable_recurrence_b200 as sru
        sru.sru_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"], scale=scale,
                                 window=c["window"], workspace=s["ws"])
    else:
        B, Hkv, D = c["B"], c["Hkv"], c["D"]
        pages = s["table"].long().clamp(min=0)
        q = s["q"].float().view(B, Hkv, c["Hq"] // Hkv, D)
        # (B, pages, Hkv, page, D) -> (B, Hkv, keys, D)
        k = s["k_cache"][pages].transpose(1, 2).reshape(B, Hkv, -1, D).float()
        v = s["v_cache"][pages].transpose(1, 2).reshape(B, Hkv, -1, D).float()
        pos = torch.arange(k.shape[2], device=q.device)[None, :]
        n = s["lengths"].long()[:, None]
        seen = pos < n
        if c["window"]:
            seen = seen & (pos >= n - c["window"])
        z = (q @ k.transpose(2, 3) * scale).masked_fill(~seen[:, None, None, :], -math.inf)
        p = (z - z.amax(-1, keepdim=True)).exp()
        s["out"].copy_(((p @ v) / p.sum(-1, keepdim=True)).view(B, c["Hq"], D))
    return s["out"]


def _loss(s):
    if own:
        import parallelizable_recurrence_b200 as sru
        sru.sru_softmax_loss(s["H"], s["W"], s["targets"], s["loss"], s["lse"], workspace=s["ws"])
    else:
        z = s["H"].float() @ s["W"].float().T
        _plain_loss(s, z)
    return [s["loss"], s["lse"]]


def _plain_loss(s, z):
    t = s["targets"]
    top = z.amax(1)
    s["lse"].copy_(top + (z - top[:, None]).exp().sum(1).log())
    zt = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    s["loss"].copy_(torch.where(t >= 0, s["lse"] - zt, 0.0))


def _train(s):
    if own:
        import parallelizable_recurrence_b200 as sru
        sru.sru_softmax_loss(s["H"], s["W"], s["targets"], s["loss"], s["lse"], workspace=s["ws"])
        sru.sru_softmax_loss_backward(s["H"], s["W"], s["targets"], s["lse"], s["dloss"], s["dH"], s["dW"],
                                      workspace=s["ws"])
    else:
        H, W, t = s["H"].float(), s["W"].float(), s["targets"]
        z = H @ W.T
        _plain_loss(s, z)
        g = torch.where(t >= 0, s["dloss"], 0.0)
        dz = (z - s["lse"][:, None]).exp() * g[:, None]
        dz.scatter_add_(1, t.clamp(min=0)[:, None], -g[:, None])
        s["dH"].copy_(dz @ W)
        s["dW"].copy_(dz.T @ H)
    return [s["loss"], s["lse"], s["dH"], s["dW"]]


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op == "extend":
        _, new, table, _, _, rows = _extend_inputs(case, 0)
        grow = np.maximum(new, 0)
        # lengths and new tokens read, lengths and offsets written, a slot a row, a page id read and written a page
        pages = grow.sum() / case["page"] + case["B"] * 0.08 * table.shape[1] / 2
        return {"bytes": int(16 * case["B"] + 4 * rows + 8 * pages + 16), "flops": 0}
    if op == "append":
        rows = 2 * case["T"] * case["H"] * case["D"]
        return {"bytes": rows * (2 + (2 if case["src"] == "bf16" else 4)) + 4 * case["T"], "flops": 0}
    if op == "decode":
        n = _lengths(case, 0)
        keys = int((np.minimum(n, case["window"]) if case["window"] else n).sum())
        return {"bytes": 4 * keys * case["Hkv"] * case["D"] + 4 * case["B"] * case["Hq"] * case["D"]
                + 4 * keys // case["page"] + 4 * case["B"],
                "flops": 4 * keys * case["Hq"] * case["D"]}
    M, V, K = case["M"], case["V"], case["K"]
    if op == "loss":
        return {"bytes": 2 * (M + V) * K + 16 * M, "flops": 2 * M * V * K}
    return {"bytes": 4 * (M + V) * K + 20 * M, "flops": 6 * M * V * K}


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "extend":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "append":
        ps, k, v = case["page"], s["k_cache"].double(), s["v_cache"].double()
        slots = s["slots"].tolist()
        rows = [i for i, x in enumerate(slots) if x >= 0]
        at = torch.tensor([slots[i] for i in rows], dtype=torch.long, device=k.device)
        rows = torch.tensor(rows, dtype=torch.long, device=k.device)
        k[at.div(ps, rounding_mode="floor"), :, at.remainder(ps)] = s["K"][rows].double()
        v[at.div(ps, rounding_mode="floor"), :, at.remainder(ps)] = s["V"][rows].double()
        return [k, v]
    if op == "decode":
        B, Hkv, D, ps = case["B"], case["Hkv"], case["D"], case["page"]
        G = case["Hq"] // Hkv
        out = torch.empty(B, case["Hq"], D, dtype=torch.float64, device=s["q"].device)
        lengths, table = s["lengths"].tolist(), s["table"].tolist()
        for b in range(B):
            n = lengths[b]
            lo = max(0, n - case["window"]) if case["window"] else 0
            at = torch.tensor([table[b][t // ps] * ps + t % ps for t in range(lo, n)], device=out.device)
            for h in range(Hkv):
                k = s["k_cache"][at // ps, h, at % ps].double()
                v = s["v_cache"][at // ps, h, at % ps].double()
                z = s["q"][b, h * G:(h + 1) * G].double().mm(k.T) / math.sqrt(D)
                out[b, h * G:(h + 1) * G] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)).mm(v)
        return out
    W, n = s["W"].double(), 1024
    loss, lse, dH, dW = [], [], [], torch.zeros_like(W) if op == "train" else None
    for i in range(0, case["M"], n):
        h, t = s["H"][i:i + n].double(), s["targets"][i:i + n]
        z = h.mm(W.T)
        e = torch.logsumexp(z, 1)
        there = t >= 0
        loss.append(torch.where(there, e - z[torch.arange(len(t), device=z.device), t.clamp(min=0)], 0.0))
        lse.append(e)
        if op == "train":
            z = torch.exp(z - e[:, None])
            z[torch.nonzero(there)[:, 0], t[there]] -= 1.0
            z *= torch.where(there, s["dloss"][i:i + n].double(), 0.0)[:, None]
            dH.append(z.mm(W))
            dW += z.T.mm(h)
    done = [torch.cat(loss), torch.cat(lse)]
    return done + [torch.cat(dH), dW] if op == "train" else done
