"""Cases and plain forms of the state pool and beam selection operators.

A state pool holds the recurrent states of many sequences, [layers, slots] pages of Hv states each, as the
serving side of the gated delta rule keeps them: value-major one-byte codes [Hv, Dv, Dk] with one FP32 scale per
block_v value rows (E4M3 or INT8), or FP32 states with the format off. The operators are the recurrent step on
such pages, the exchange of FP32 states with them (before and after a chunk prefill), copies and reorderings of
pages, and the selection over beams and vocabulary.

`run` computes each operator with elementary torch operations, or, with `own` set, by the calls of this
repository's package.
"""
import math

import torch

own = False

OFF, E4M3, INT8 = 0, 1, 2
QMAX = {E4M3: 448.0, INT8: 127.0}
TINY = 2.0 ** -126


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one conversation, one token: the call is all latency
        dict(name="step_e4m3_b1_gqa4x16_d128", op="step", fmt=E4M3, io="bf16", B=1, T=1, Hqk=4, Hv=16, Dk=128,
             Dv=128, bv=64, fork=False, ragged=False, after=False, holes=0),
        # beams: every sequence reads its parent's page and writes its own; a few places of the batch are empty
        dict(name="step_e4m3_b192_gqa4x16_fork", op="step", fmt=E4M3, io="bf16", B=192, T=1, Hqk=4, Hv=16,
             Dk=128, Dv=128, bv=64, fork=True, ragged=False, after=False, holes=5),
        # the largest batch, wide values, output read from the state as written
        dict(name="step_e4m3_b1024_h32_dv256_fork", op="step", fmt=E4M3, io="bf16", B=1024, T=1, Hqk=32, Hv=32,
             Dk=128, Dv=256, bv=64, fork=True, ragged=False, after=True, holes=0),
        # FP32 states and inputs, up to five tokens a sequence (a padded batch of drafts)
        dict(name="step_f32_b90_t5_ragged_d64", op="step", fmt=OFF, io="f32", B=90, T=5, Hqk=2, Hv=6, Dk=64,
             Dv=64, bv=64, fork=False, ragged=True, after=False, holes=3),
        # hand-over of a prefill batch: old states out, new states in
        dict(name="exchange_e4m3_n64_h16_d128", op="exchange", fmt=E4M3, N=64, Hv=16, Dk=128, Dv=128, bv=64),
        dict(name="exchange_int8_n7_h5_dk64_dv256_bv16", op="exchange", fmt=INT8, N=7, Hv=5, Dk=64, Dv=256,
             bv=16),
        # a prompt's page forked to every sample of its requests, all layers
        dict(name="copy_fork_l12_m60_h16", op="copy", fmt=E4M3, L=12, slots=96, moves=60, sources=6, clears=0,
             Hv=16, Dk=128, Dv=128, bv=64),
        # compaction after some requests ended: a few moves, a few pages cleared
        dict(name="copy_compact_l2_m7_h4", op="copy", fmt=INT8, L=2, slots=24, moves=7, sources=7, clears=3,
             Hv=4, Dk=128, Dv=64, bv=32),
        # beams change places in every layer
        dict(name="reorder_l12_g16_w4_h16", op="reorder", fmt=E4M3, L=12, G=16, W=4, Hv=16, Dk=128, Dv=128,
             bv=64),
        dict(name="reorder_f32_l1_g1_w5_h4_d64", op="reorder", fmt=OFF, L=1, G=1, W=5, Hv=4, Dk=64, Dv=64,
             bv=64),
        # one request with four beams; many requests with eight
        dict(name="select_bf16_b1_w4_v131072", op="select", io="bf16", B=1, W=4, V=131072, K=8, masked=False,
             done=0),
        dict(name="select_bf16_b64_w8_v100003", op="select", io="bf16", B=64, W=8, V=100003, K=16, masked=True,
             done=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    hv = _log(rng, 1, 32)
    hqk = rng.choice([d for d in range(1, hv + 1) if hv % d == 0])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128, 256])
    return hqk, hv, dk, dv, rng.choice([b for b in (16, 32, 64, 128, 256) if dv % b == 0])


def draw(rng):
    op = rng.choice(["step", "step", "exchange", "copy", "reorder", "select"])
    if op == "select":
        io, W = rng.choice(["bf16", "bf16", "f32"]), _log(rng, 1, 12)
        B, V = _log(rng, 1, 64), _log(rng, 300, 160000)
        V = min(V, max(300, 40_000_000 // (B * W)))
        return dict(op=op, io=io, B=B, W=W, V=V, K=rng.choice([W, 2 * W]), masked=rng.random() < 0.5,
                    done=rng.randint(0, B * W // 3))
    hqk, hv, dk, dv, bv = _heads(rng)
    page = hv * dk * dv
    fmt = rng.choice([E4M3, E4M3, INT8, OFF])
    if op == "step":
        fmt = rng.choice([E4M3, E4M3, OFF])
        io = "bf16" if fmt else rng.choice(["bf16", "f32"])
        # several tokens a call: E4M3 on few states, FP32 on more
        T = 1 if rng.random() < 0.6 else _log(rng, 2, 40 if fmt else 12)
        most = 2 ** 30 // (page * (1 if fmt else 4))
        B = _log(rng, 1, max(1, min(1024, most // T)))
        if fmt and T > 1:
            B = max(1, min(B, 200 * bv // (hv * dv * T)))
        return dict(op=op, fmt=fmt, io=io, B=B, T=T, Hqk=hqk, Hv=hv, Dk=dk, Dv=dv, bv=bv,
                    fork=bool(fmt) or rng.random() < 0.5, ragged=T > 1 and rng.random() < 0.5,
                    after=T == 1 and rng.random() < 0.5, holes=rng.randint(0, B // 4))
    if op == "exchange":
        return dict(op=op, fmt=fmt, N=_log(rng, 1, max(1, min(256, 2 ** 25 // page))), Hv=hv, Dk=dk, Dv=dv, bv=bv)
    L = _log(rng, 1, 12)
    most = max(1, 2 ** 27 // (page * L * (1 if fmt else 4)))
    if op == "copy":
        moves = _log(rng, 1, min(128, most))
        return dict(op=op, fmt=fmt, L=L, slots=3 * moves + 2, moves=moves, sources=rng.randint(1, moves),
                    clears=rng.randint(0, moves), Hv=hv, Dk=dk, Dv=dv, bv=bv)
    W = _log(rng, 2, 12)
    return dict(op=op, fmt=fmt, L=L, G=_log(rng, 1, max(1, min(64, most // W))), W=W, Hv=hv, Dk=dk, Dv=dv, bv=bv)


# ---------------------------------------------------------------------------------------------- inputs
def _quantize(s, fmt, bv):
    """Value-major FP32 states [..., Dv, Dk] -> (codes, scales [..., Dv / bv]): one scale per bv rows,
    d = max(fl(amax / qmax), 2^-126), codes RNE(fl(x * fl(1 / d)))."""
    if fmt == OFF:
        return s, None
    t = s.reshape(*s.shape[:-2], s.shape[-2] // bv, bv * s.shape[-1])
    d = (t.abs().amax(-1) / QMAX[fmt]).clamp_min(TINY)
    y = t * (1.0 / d).unsqueeze(-1)
    c = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn) if fmt == E4M3 else y.round().clamp(-127, 127).to(torch.int8)
    return c.reshape(s.shape), d


def _values(codes, scales, bv):
    """Codes [..., Dv, Dk] and scales [..., Dv / bv] -> FP32 states."""
    if scales is None:
        return codes
    return codes.float() * scales.repeat_interleave(bv, -1).unsqueeze(-1)


def _pool(gen, dev, fmt, layers, slots, Hv, Dk, Dv, bv):
    """Pages as a running server has them: quantized states with spread-out magnitudes."""
    data, scales = [], []
    for _ in range(layers):
        s = torch.randn(slots, Hv, Dv, Dk, generator=gen, device=dev) * 0.1
        s *= torch.exp(torch.randn(slots, Hv, 1, 1, generator=gen, device=dev))
        c, d = _quantize(s, fmt, bv)
        data.append(c)
        scales.append(d)
    if fmt == OFF:
        return torch.stack(data), None
    return torch.stack([c.view(torch.uint8) for c in data]).view(data[0].dtype), torch.stack(scales)


def _bytes(t):
    """One-byte codes as bytes (to move them); FP32 states as they are."""
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _handle(s, fmt, bv):
    """The pool handle that a serving program keeps."""
    if own:
        from gateddeltanet_chunked_recurrence_amd import SCALE_RECIPROCAL, StatePool
        # _quantize divides the amax by a number, which PyTorch does on the GPU as a product with its reciprocal
        s["pool"] = StatePool.from_tensors(s["data"], s["scales"], state_fmt=fmt, block_v=bv, scale_rule=SCALE_RECIPROCAL)
    return s


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _perm(cg, n):
    return torch.randperm(n, generator=cg).tolist()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cg = torch.Generator()
    cg.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "select":
        B, W, V = case["B"], case["W"], case["V"]
        # a trained model's logits: most tokens unlikely, a few dozen that compete
        x = torch.randn(B, W, V, generator=gen, device=dev) * 2.0
        hot = torch.randint(0, V, (B, W, 40), generator=gen, device=dev)
        x.scatter_add_(2, hot, 6.0 * torch.rand(B, W, 40, generator=gen, device=dev))
        if case["masked"]:  # a grammar leaves some rows few tokens, one of them a single one
            keep = torch.rand(B, 1, V, generator=gen, device=dev) < 0.02
            keep[:, :, 7 % V] = True
            rows = torch.rand(B, W, 1, generator=gen, device=dev) < 0.2
            x.masked_fill_(rows & ~keep, -math.inf)
            x[0, 0] = -math.inf
            x[0, 0, V // 3] = 1.5
        s["logits"] = x.to(torch.bfloat16 if case["io"] == "bf16" else torch.float32)
        s["scores"] = -12.0 - 2.5 * torch.rand(B, W, generator=gen, device=dev)
        done = torch.zeros(B * W, dtype=torch.bool)
        done[_perm(cg, B * W)[: case["done"]]] = True
        s["done"] = done.reshape(B, W).to(dev) if case["done"] else None
        return s
    fmt, Hv, Dk, Dv, bv = case["fmt"], case["Hv"], case["Dk"], case["Dv"], case["bv"]
    if op == "step":
        B, T, Hqk = case["B"], case["T"], case["Hqk"]
        n = (2 if case["fork"] else 1) * B + 1
        s["data"], s["scales"] = _pool(gen, dev, fmt, 1, n, Hv, Dk, Dv, bv)
        order = _perm(cg, n)
        slots, out = order[:B], order[B: 2 * B] if case["fork"] else None
        if out:  # some parents have several children
            slots = [slots[i] for i in torch.randint(0, B, (B,), generator=cg).tolist()]
        for i in _perm(cg, B)[: case["holes"]]:
            slots[i] = -1
        s["slots"], s["out"] = _ints(slots, dev), None if out is None else _ints(out, dev)
        io = torch.bfloat16 if case["io"] == "bf16" else torch.float32
        q, k = (torch.nn.functional.normalize(torch.randn(B, T, Hqk, Dk, generator=gen, device=dev), dim=-1)
                for _ in range(2))
        s["q"], s["k"] = q.to(io), k.to(io)
        s["v"] = torch.randn(B, T, Hv, Dv, generator=gen, device=dev).to(io)
        s["beta"] = torch.sigmoid(torch.randn(B, T, Hv, generator=gen, device=dev))
        s["g"] = -torch.nn.functional.softplus(torch.randn(B, T, Hv, generator=gen, device=dev) + 2.0)
        s["lens"] = torch.randint(0, T + 1, (B,), generator=cg, dtype=torch.int32).to(dev) if case["ragged"] else None
        s["o"] = torch.zeros(B, T, Hv, Dv, device=dev, dtype=io)
        return _handle(s, fmt, bv)
    if op == "exchange":
        N = case["N"]
        s["data"], s["scales"] = _pool(gen, dev, fmt, 1, N + 3, Hv, Dk, Dv, bv)
        s["slots"] = _ints(_perm(cg, N + 3)[:N], dev)
        x = torch.randn(N, Hv, Dk, Dv, generator=gen, device=dev) * 0.2
        s["new"] = x * torch.exp(torch.randn(N, Hv, 1, 1, generator=gen, device=dev))
        return _handle(s, fmt, bv)
    if op == "copy":
        s["data"], s["scales"] = _pool(gen, dev, fmt, case["L"], case["slots"], Hv, Dk, Dv, bv)
        order, k = _perm(cg, case["slots"]), case["sources"]
        dst = order[k: k + case["moves"] + case["clears"]]
        src = [order[i % k] for i in range(case["moves"])] + [-1] * case["clears"]
        s["src"], s["dst"] = _ints(src, dev), _ints(dst, dev)
        return _handle(s, fmt, bv)
    G, W = case["G"], case["W"]
    s["data"], s["scales"] = _pool(gen, dev, fmt, case["L"], G * W + 2, Hv, Dk, Dv, bv)
    s["slots"] = _ints(_perm(cg, G * W + 2)[: G * W], dev).reshape(G, W)
    s["parents"] = torch.randint(0, W, (G, W), generator=cg, dtype=torch.int32).to(dev)
    return _handle(s, fmt, bv)


# ----------------------------------------------------------------------------------------- plain forms
def _step_plain(s, c):
    fmt, bv, T = c["fmt"], c["bv"], c["T"]
    here = s["slots"] >= 0
    src = s["slots"].clamp_min(0).long()
    dst = src if s["out"] is None else s["out"].long()
    rows = torch.nonzero(here).flatten()
    src, dst = src[rows], dst[rows]
    rep = c["Hv"] // c["Hqk"]
    q, k = (s[n][rows].float().repeat_interleave(rep, 2) for n in ("q", "k"))
    v, g, beta = s["v"][rows].float(), s["g"][rows], s["beta"][rows]
    last = torch.full((len(rows),), T, device=rows.device) if s["lens"] is None else s["lens"][rows].clamp(0, T).long()
    data, scales = _bytes(s["data"][0]), None if s["scales"] is None else s["scales"][0]
    codes, ds = data[src], None if scales is None else scales[src]
    S = _values(codes.view(s["data"].dtype), ds, bv)
    scale = c["Dk"] ** -0.5
    for t in range(T):
        on = (t < last)
        S1 = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S1 * k[:, t, :, None, :]).sum(-1))
        S1 = S1 + u.unsqueeze(-1) * k[:, t, :, None, :]
        o = (S1 * q[:, t, :, None, :]).sum(-1)
        c1, d1 = _quantize(S1, fmt, bv)
        if fmt:
            S1 = _values(c1, d1, bv)
            if c["after"]:
                o = (S1 * q[:, t, :, None, :]).sum(-1)
        s["o"][rows, t] = torch.where(on[:, None, None], (o * scale).to(s["o"].dtype), s["o"][rows, t])
        if T == 1 and s["lens"] is None:
            codes, ds = c1, d1
        else:
            m = on[:, None, None, None]
            S = torch.where(m, S1, S)
            codes = torch.where(m, _bytes(c1), codes)
            ds = torch.where(on[:, None, None], d1, ds) if fmt else None
    data[dst] = _bytes(codes)
    if fmt:
        scales[dst] = ds


def _select_plain(s, c):
    B, W, V, K = c["B"], c["W"], c["V"], c["K"]
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.exp(x - m).sum(-1, keepdim=True).log()
    total = s["scores"].double().unsqueeze(-1) + (x - lse)
    if s["done"] is not None:
        total = total.masked_fill(s["done"].unsqueeze(-1), -math.inf)
        total[..., 0] = torch.where(s["done"], s["scores"].double(), total[..., 0])
    total = total.reshape(B, W * V)
    least = torch.topk(total, min(K, W * V), dim=1).values[:, -1:]
    row, col = torch.nonzero((total >= least) & (total > -math.inf), as_tuple=True)
    val = total[row, col]
    order = torch.argsort(val, descending=True, stable=True)      # equal ones stay in the order of their places
    order = order[torch.argsort(row[order], stable=True)]
    row, col, val = row[order], col[order], val[order]
    place = torch.arange(len(row), device=row.device) - torch.searchsorted(row, row)
    row, col, val, place = (t[place < K] for t in (row, col, val, place))
    scores = torch.full((B, K), -math.inf, device=x.device)
    parents, tokens = (torch.full((B, K), -1, dtype=torch.int32, device=x.device) for _ in range(2))
    scores[row, place] = val.float()
    parents[row, place] = (col // V).int()
    tokens[row, place] = (col % V).int()
    return scores, parents, tokens


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "select":
        if own:
            from gateddeltanet_chunked_recurrence_amd import gdn_beam_select
            scores, parents, tokens = gdn_beam_select(s["logits"], s["scores"], c["K"], finished=s["done"], pad_token=0)
        else:
            scores, parents, tokens = _select_plain(s, c)
        return {"scores": scores, "parents": parents, "tokens": tokens}
    if own:
        import gateddeltanet_chunked_recurrence_amd as G
    out = {"codes": s["data"]}
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    if op == "step":
        if own:
            G.gdn_pool_step(s["pool"], 0, s["slots"], s["q"], s["k"], s["v"], s["g"], s["beta"], slots_out=s["out"],
                            lens=s["lens"], out=s["o"],
                            readout=G.READOUT_AFTER_WRITE if c["after"] else G.READOUT_BEFORE_WRITE)
        else:
            _step_plain(s, c)
        out["o"] = s["o"]
    elif op == "exchange":
        if own:
            out["old"] = G.gdn_pool_read(s["pool"], 0, s["slots"])
            G.gdn_pool_write(s["pool"], 0, s["slots"], s["new"])
        else:
            at = s["slots"].long()
            codes, scales = _bytes(s["data"][0]), None if s["scales"] is None else s["scales"][0]
            old = _values(codes[at].view(s["data"].dtype), None if scales is None else scales[at], c["bv"])
            out["old"] = old.transpose(-1, -2).contiguous()
            new, d = _quantize(s["new"].transpose(-1, -2).contiguous(), c["fmt"], c["bv"])
            codes[at] = _bytes(new)
            if scales is not None:
                scales[at] = d
    elif op == "copy":
        if own:
            G.gdn_pool_copy(s["pool"], s["src"], s["dst"])
        else:
            codes, at, keep = _bytes(s["data"]), s["src"].clamp_min(0).long(), s["src"] >= 0
            codes[:, s["dst"].long()] = torch.where(keep[None, :, None, None, None], codes[:, at], 0)
            if s["scales"] is not None:
                s["scales"][:, s["dst"].long()] = torch.where(keep[None, :, None, None], s["scales"][:, at], TINY)
    else:
        if own:
            G.gdn_pool_reorder(s["pool"], s["slots"], s["parents"])
        else:
            src = torch.gather(s["slots"], 1, s["parents"].long()).flatten().long()
            codes, dst = _bytes(s["data"]), s["slots"].flatten().long()
            codes[:, dst] = codes[:, src]
            if s["scales"] is not None:
                s["scales"][:, dst] = s["scales"][:, src]
    return out


# -------------------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    if op == "select":
        rows = case["B"] * case["W"] - case["done"]
        n = rows * case["V"]
        return {"bytes": n * (2 if case["io"] == "bf16" else 4) + case["B"] * (case["W"] * 5 + case["K"] * 12),
                "flops": 4 * n}
    Hv, Dk, Dv = case["Hv"], case["Dk"], case["Dv"]
    page = Hv * Dk * Dv * (1 if case["fmt"] else 4) + (Hv * (Dv // case["bv"]) * 4 if case["fmt"] else 0)
    if op == "step":
        n = case["B"] - case["holes"]
        es = 2 if case["io"] == "bf16" else 4
        tokens = n * case["T"] * (0.5 if case["ragged"] else 1)
        # with children, a parent's page is read once
        read = n if not case["fork"] else case["B"] * (1 - (1 - 1 / case["B"]) ** n) if case["B"] > 1 else n
        return {"bytes": (read + n) * page + tokens * (2 * case["Hqk"] * Dk * es + 2 * Hv * Dv * es + 8 * Hv),
                "flops": 6 * tokens * Hv * Dk * Dv}
    if op == "exchange":
        return {"bytes": 2 * case["N"] * (page + Hv * Dk * Dv * 4), "flops": 4 * case["N"] * Hv * Dk * Dv}
    if op == "copy":
        return {"bytes": case["L"] * page * (case["sources"] + case["moves"] + case["clears"]), "flops": 0}
    W = case["W"]
    moved = case["G"] * W * (1 - 1 / W)                      # beams that change; their distinct sources
    sources = case["G"] * W * (1 - (1 - 1 / W) ** (W - 1))
    return {"bytes": max(1, case["L"] * page * (moved + sources)), "flops": 0}


# ------------------------------------------------------------------------------------ 64-bit definition
def _grid_e4m3(y):
    """Nearest E4M3 value (ties to even): steps of 2^(e-3) in the binade e >= -6, at most 448."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _codes64(s, fmt, bv):
    """Codes and scales of FP64 states with value rows second to last."""
    shape = s.shape
    s = s.unflatten(-2, (shape[-2] // bv, bv))
    d = s.abs().amax((-1, -2)).div(QMAX[fmt]).clamp_min(TINY)
    y = s / d[..., None, None]
    c = _grid_e4m3(y) if fmt == E4M3 else torch.round(y).clamp(-127, 127)
    return c.reshape(shape), d


def exact(case, seed):
    op = case["op"]
    if op in ("copy", "reorder"):
        return None                                          # pages are moved, not computed
    s = prepare(case, seed)
    if op == "select":
        B, W, V, K = case["B"], case["W"], case["V"], case["K"]
        total = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double()[..., None]
        if s["done"] is not None:
            only = torch.full_like(total, -math.inf)
            only[..., 0] = s["scores"].double()
            total = torch.where(s["done"][..., None], only, total)
        best = total.reshape(B, -1).sort(1, descending=True).values[:, :K] if total.numel() < 2e7 else \
            total.reshape(B, -1).topk(K, 1).values
        if best.shape[1] < K:
            best = torch.nn.functional.pad(best, (0, K - best.shape[1]), value=-math.inf)
        return {"scores": best, "parents": None, "tokens": None}
    fmt, bv, Dk = case["fmt"], case["bv"], case["Dk"]
    codes = s["data"][0].double()
    scales = None if fmt == OFF else s["scales"][0].double()
    if op == "exchange":
        at = s["slots"].tolist()
        old, new = [], s["new"].double().mT
        for n, slot in enumerate(at):
            x = codes[slot] if fmt == OFF else \
                (codes[slot].unflatten(-2, (-1, bv)) * scales[slot][..., None, None]).flatten(-3, -2)
            old.append(x.mT)
            if fmt == OFF:
                codes[slot] = new[n]
            else:
                codes[slot], scales[slot] = _codes64(new[n], fmt, bv)
        out = {"codes": codes[None] if fmt != INT8 else None, "old": torch.stack(old)}
        if fmt:
            out["scales"] = scales[None]
        return out
    B, T, rep = case["B"], case["T"], case["Hv"] // case["Hqk"]
    if T * B > 2000:
        return None
    o = s["o"].double()
    slots = s["slots"].tolist()
    to = slots if s["out"] is None else s["out"].tolist()
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    first, first_scales = codes.clone(), None if fmt == OFF else scales.clone()
    for n in range(B):
        if slots[n] < 0:
            continue
        c, d = first[slots[n]], None if fmt == OFF else first_scales[slots[n]]
        for t in range(lens[n]):
            S = c if fmt == OFF else (c.unflatten(-2, (-1, bv)) * d[..., None, None]).flatten(-3, -2)
            q, k = (s[i][n, t].double().repeat_interleave(rep, 0).unsqueeze(-1) for i in ("q", "k"))    # [Hv, Dk, 1]
            S = S * s["g"][n, t].double().exp()[:, None, None]
            u = s["beta"][n, t].double()[:, None, None] * (s["v"][n, t].double().unsqueeze(-1) - S @ k)
            S = S + u * k.mT
            read = S
            c = S
            if fmt != OFF:
                c, d = _codes64(S, fmt, bv)
                if case["after"]:
                    read = (c.unflatten(-2, (-1, bv)) * d[..., None, None]).flatten(-3, -2)
            o[n, t] = (read @ q).squeeze(-1) * Dk ** -0.5
        codes[to[n]] = c
        if fmt:
            scales[to[n]] = d
    out = {"codes": codes[None], "o": o}
    if fmt:
        out["scales"] = scales[None]
    return out
