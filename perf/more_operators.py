"""Cases and plain forms of linear attention with a decay per head, and of the rules on logits before a choice.

Linear attention keeps, like the gated delta rule, one state S [Dk, Dv] per value head, but writes to it without
reading it first:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

with a log-decay g per token and head (or one per head). Its operators are the chunked forward over prompts, the
gradients of that, and the step of single tokens on the pages of a state pool. The rules on logits (penalties of
repeated tokens, biases, grammar masks) stand in front of the selection over beams and vocabulary.

`run` computes each operator with elementary torch operations, or, with `own` set, by the calls of this
repository's package.
"""
import math

import torch

own = False

OFF, E4M3 = 0, 1
TINY = 2.0 ** -126
CHUNK = 64


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a short question to a small layer: the call is all latency
        dict(name="fwd_b1_t150_h4_d64", op="fwd", io="bf16", B=1, T=150, lens="", Hqk=2, Hv=4, Dk=64, Dv=64,
             gate="token", h0=False, view=False),
        # a batch of prompts
        dict(name="fwd_b4_t4096_h16_d128", op="fwd", io="bf16", B=4, T=4096, lens="", Hqk=16, Hv=16, Dk=128, Dv=128,
             gate="token", h0=False, view=False),
        # prompts of different lengths packed into one row, from kept states; q, k, v are views of one projection
        dict(name="fwd_packed_gqa4x16_d128", op="fwd", io="bf16", B=1, T=5996, lens="257,1000,3,4096,640", Hqk=4, Hv=16,
             Dk=128, Dv=128, gate="head", h0=True, view=True),
        # one long document, wide values
        dict(name="fwd_t65536_h32_dk128_dv256", op="fwd", io="bf16", B=1, T=65536, lens="", Hqk=32, Hv=32, Dk=128,
             Dv=256, gate="retention", h0=False, view=False),
        # training in FP32, as small models and checks do it
        dict(name="bwd_f32_b2_t515_h6_d64", op="bwd", io="f32", B=2, T=515, lens="", Hqk=2, Hv=6, Dk=64, Dv=64,
             gate="token", h0=False, view=False),
        # a training batch, states handed from segment to segment
        dict(name="bwd_b2_t8192_h16_d128", op="bwd", io="bf16", B=2, T=8192, lens="", Hqk=16, Hv=16, Dk=128, Dv=128,
             gate="token", h0=True, view=False),
        # packed documents, shared query and key heads, a decay per head
        dict(name="bwd_packed_gqa4x16_d128", op="bwd", io="bf16", B=1, T=5996, lens="257,1000,3,4096,640", Hqk=4, Hv=16,
             Dk=128, Dv=128, gate="head", h0=True, view=True),
        # one conversation, one token: the call is all latency
        dict(name="step_f32_b1_gqa4x16_d128", op="step", fmt=OFF, io="bf16", B=1, T=1, Hqk=4, Hv=16, Dk=128, Dv=128,
             bv=64, gate="token", fork=False, ragged=False, after=False, holes=0),
        # a serving batch, states in FP32; a few places of the batch are empty
        dict(name="step_f32_b301_h32_dv256", op="step", fmt=OFF, io="bf16", B=301, T=1, Hqk=32, Hv=32, Dk=128, Dv=256,
             bv=64, gate="token", fork=False, ragged=False, after=False, holes=4),
        # beams on states in 8 bits: each reads its parent's page and writes its own
        dict(name="step_e4m3_b192_gqa4x16_fork", op="step", fmt=E4M3, io="bf16", B=192, T=1, Hqk=4, Hv=16, Dk=128,
             Dv=128, bv=64, gate="head", fork=True, ragged=False, after=False, holes=5),
        # one request of four beams with a short history
        dict(name="rules_bf16_b1_w4_v131072", op="rules", io="bf16", B=1, W=4, V=131072, L=640, NB=12, penalties=True,
             masked=False),
        # many requests of eight beams, long histories, a grammar over each beam
        dict(name="rules_bf16_b64_w8_v100003", op="rules", io="bf16", B=64, W=8, V=100003, L=4096, NB=300, penalties=True,
             masked=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "rules"])
    if op == "rules":
        B, W, V = _log(rng, 1, 64), _log(rng, 1, 12), _log(rng, 300, 160000)
        V = min(V, max(300, 40_000_000 // (B * W)))
        return dict(op=op, io=rng.choice(["bf16", "bf16", "f32"]), B=B, W=W, V=V, L=_log(rng, 1, 4096),
                    NB=rng.choice([0, _log(rng, 1, 300)]), penalties=rng.random() < 0.8, masked=rng.random() < 0.5)
    hv = _log(rng, 1, 32)
    hqk = rng.choice([d for d in range(1, hv + 1) if hv % d == 0])
    dk, dv, io = rng.choice([64, 128]), rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    gate = rng.choice(["token", "retention", "head"])
    if op == "step":
        fmt = rng.choice([OFF, OFF, E4M3])
        bv = rng.choice([b for b in (16, 32, 64, 128, 256) if dv % b == 0])
        T = 1 if fmt or rng.random() < 0.6 else _log(rng, 2, 12)
        B = _log(rng, 1, max(1, min(1024, 2 ** 30 // (hv * dk * dv * (1 if fmt else 4) * T))))
        return dict(op=op, fmt=fmt, io=io, B=B, T=T, Hqk=hqk, Hv=hv, Dk=dk, Dv=dv, bv=bv, gate=gate,
                    fork=rng.random() < 0.5, ragged=T > 1 and rng.random() < 0.5, after=T == 1 and rng.random() < 0.5,
                    holes=rng.randint(0, B // 4))
    # tokens in all, so that a pass moves at most a few hundred MB
    most = 2 ** (27 if op == "fwd" else 26) // (hv * (dk + dv) * (1 if io == "bf16" else 2))
    most = min(most, 2 ** 31 // (hv * dk * dv * 4) * CHUNK, 32768)
    if rng.random() < 0.4:
        lens = [_log(rng, 1, 8192) for _ in range(rng.randint(1, 12))]
        while sum(lens) > most and len(lens) > 1:
            lens.pop()
        lens[0] = min(lens[0], most)
        B, T, lens = 1, sum(lens), ",".join(map(str, lens))
    else:
        T = _log(rng, 1, max(1, min(16384, most)))
        B, lens = _log(rng, 1, max(1, min(32, most // max(T, CHUNK)))), ""
    return dict(op=op, io=io, B=B, T=T, lens=lens, Hqk=hqk, Hv=hv, Dk=dk, Dv=dv, gate=gate, h0=rng.random() < 0.5,
                view=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------- inputs
def _quantize(s, bv):
    """Value-major FP32 states [..., Dv, Dk] -> (E4M3 codes, scales [..., Dv / bv]): one scale per bv rows,
    d = max(fl(amax / 448), 2^-126), codes RNE(fl(x * fl(1 / d)))."""
    t = s.reshape(*s.shape[:-2], s.shape[-2] // bv, bv * s.shape[-1])
    d = (t.abs().amax(-1) / 448.0).clamp_min(TINY)
    c = (t * (1.0 / d).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return c.reshape(s.shape), d


def _values(codes, scales, bv):
    """Codes [..., Dv, Dk] and scales [..., Dv / bv] -> FP32 states."""
    if scales is None:
        return codes
    return codes.float() * scales.repeat_interleave(bv, -1).unsqueeze(-1)


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _perm(cg, n):
    return torch.randperm(n, generator=cg).tolist()


def _gate(gen, dev, kind, B, T, Hv):
    """Log-decays: one per head, slowly forgetting ones, or such as a gate of the token gives."""
    if kind == "head":
        return torch.log(0.9 + 0.099 * torch.rand(Hv, generator=gen, device=dev))
    if kind == "retention":
        return torch.log(0.9 + 0.099 * torch.rand(B, T, Hv, generator=gen, device=dev))
    return -torch.nn.functional.softplus(torch.randn(B, T, Hv, generator=gen, device=dev))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cg = torch.Generator()
    cg.manual_seed(seed)
    op, s = case["op"], {"case": case}
    io = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    if op == "rules":
        B, W, V, L, NB = (case[n] for n in ("B", "W", "V", "L", "NB"))
        # a trained model's logits: most tokens unlikely, a few dozen that compete
        x = torch.randn(B, W, V, generator=gen, device=dev) * 2.0
        hot = torch.randint(0, V, (B, W, 40), generator=gen, device=dev)
        x.scatter_add_(2, hot, 6.0 * torch.rand(B, W, 40, generator=gen, device=dev))
        s["logits"] = x.to(io)
        # histories repeat themselves: most tokens come from a few hundred, and beams share their prompt
        few = torch.randint(0, V, (B, 300), generator=gen, device=dev)
        pick = torch.randint(0, 300, (B, W, L), generator=gen, device=dev)
        h = torch.gather(few, 1, pick.reshape(B, W * L)).reshape(B, W, L)
        rare = torch.rand(B, W, L, generator=gen, device=dev) < 0.3
        h = torch.where(rare, torch.randint(0, V, (B, W, L), generator=gen, device=dev), h)
        prompt = torch.randint(0, L // 2 + 1, (B,), generator=gen, device=dev)
        first = torch.arange(L, device=dev) < prompt[:, None, None]
        s["tokens"] = torch.where(first, h[:, :1], h).int().contiguous()
        s["lens"] = torch.randint(L // 2, L + 1, (B, W), generator=gen, device=dev).int()
        s["prompt"] = prompt.int()
        s["rep"] = 1.0 + 0.3 * torch.rand(B, generator=gen, device=dev)
        s["pres"], s["freq"] = (torch.rand(B, generator=gen, device=dev) for _ in range(2))
        if NB:
            s["ids"] = torch.randint(0, V, (B, NB), generator=gen, device=dev).int()
            s["ids"][:, NB // 2:: 7] = -1                         # requests with fewer entries
            s["vals"] = 4.0 * torch.randn(B, NB, generator=gen, device=dev)
        if case["masked"]:
            # the states of a grammar: some allow nearly everything, some a few tokens; one in nine beams is free
            words, M = (V + 31) // 32, 2 * B + 3
            bits = torch.rand(M, words, 32, generator=gen, device=dev) < torch.rand(M, 1, 1, generator=gen, device=dev) ** 4
            bits[:, 0, 1] = True
            m = (bits.long() << torch.arange(32, device=dev)).sum(-1)
            s["mask"] = torch.where(m >= 2 ** 31, m - 2 ** 32, m).int()
            rows = torch.randint(0, M, (B, W), generator=gen, device=dev)
            s["rows"] = torch.where(torch.rand(B, W, generator=gen, device=dev) < 0.11, -1, rows).int()
        return s
    B, T, Hqk, Hv, Dk, Dv = (case[n] for n in ("B", "T", "Hqk", "Hv", "Dk", "Dv"))
    q, k = (torch.nn.functional.normalize(torch.randn(B, T, Hqk, Dk, generator=gen, device=dev), dim=-1) for _ in range(2))
    v = torch.randn(B, T, Hv, Dv, generator=gen, device=dev)
    s["g"] = _gate(gen, dev, case["gate"], B, T, Hv)
    if op == "step":
        fmt, bv, n = case["fmt"], case["bv"], (2 if case["fork"] else 1) * B + 1
        # pages as a running server has them, with spread-out magnitudes
        x = torch.randn(1, n, Hv, Dv, Dk, generator=gen, device=dev) * 0.1
        x *= torch.exp(torch.randn(1, n, Hv, 1, 1, generator=gen, device=dev))
        s["data"], s["scales"] = _quantize(x, bv) if fmt else (x, None)
        order = _perm(cg, n)
        slots, to = order[:B], order[B: 2 * B] if case["fork"] else None
        if to:  # some parents have several children
            slots = [slots[i] for i in torch.randint(0, B, (B,), generator=cg).tolist()]
        for i in _perm(cg, B)[: case["holes"]]:
            slots[i] = -1
        s["slots"], s["out"] = _ints(slots, dev), None if to is None else _ints(to, dev)
        s["q"], s["k"], s["v"] = q.to(io), k.to(io), v.to(io)
        s["lens"] = torch.randint(0, T + 1, (B,), generator=cg, dtype=torch.int32).to(dev) if case["ragged"] else None
        s["o"] = torch.zeros(B, T, Hv, Dv, device=dev, dtype=io)
        if own:
            from gateddeltanet_chunked_recurrence_amd import SCALE_RECIPROCAL, StatePool
            # _quantize divides the amax by a number, which PyTorch does on the GPU as a product with its reciprocal
            s["pool"] = StatePool.from_tensors(s["data"], s["scales"], state_fmt=fmt, block_v=bv,
                                               scale_rule=SCALE_RECIPROCAL)
        return s
    if case["view"]:
        x = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], 2).to(io)
        q, k, v = x.split([Hqk * Dk, Hqk * Dk, Hv * Dv], 2)
        s["q"], s["k"], s["v"] = q.unflatten(2, (Hqk, Dk)), k.unflatten(2, (Hqk, Dk)), v.unflatten(2, (Hv, Dv))
    else:
        s["q"], s["k"], s["v"] = q.to(io), k.to(io), v.to(io)
    lens = [int(x) for x in case["lens"].split(",")] if case["lens"] else [T] * B
    offsets = [0]
    for x in lens:
        offsets.append(offsets[-1] + x)
    s["cu"] = _ints(offsets, dev) if case["lens"] else None
    s["seqs"] = lens
    N = len(lens)
    s["h0"] = torch.randn(N, Hv, Dk, Dv, generator=gen, device=dev) * 0.1 if case["h0"] else None
    if op == "bwd":
        s["do"] = torch.randn(B, T, Hv, Dv, generator=gen, device=dev).to(io)
        s["dht"] = torch.randn(N, Hv, Dk, Dv, generator=gen, device=dev) * 0.1 if case["h0"] else None
    return s


# ----------------------------------------------------------------------------------------- plain forms
class _Chunks:
    """The chunks of all sequences side by side: [chunks, heads, 64, ...], short ones padded with zeros."""

    def __init__(self, s):
        dev, c = s["q"].device, s["case"]
        count = torch.tensor([-(-n // CHUNK) for n in s["seqs"]], device=dev)
        lens = torch.tensor(s["seqs"], device=dev)
        self.seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), count)
        self.first = torch.cumsum(count, 0) - count
        at = (torch.arange(len(self.seq), device=dev) - self.first[self.seq]) * CHUNK
        at = at[:, None] + torch.arange(CHUNK, device=dev)
        self.here = at < lens[self.seq, None]
        self.token = ((torch.cumsum(lens, 0) - lens)[self.seq, None] + at).clamp_max(max(1, c["B"] * c["T"]) - 1)
        g = s["g"].double()
        g = g.reshape(-1, g.shape[-1])[self.token] if g.dim() == 3 else g.expand(*self.token.shape, -1)
        gam = torch.cumsum(g * self.here[..., None], 1).transpose(1, 2)            # [C, H, 64]
        self.gam, total = gam, gam[..., -1]
        after = torch.cumsum(total, 0)
        before = after - total                                                     # [C, H]
        same = (self.seq[:, None] == self.seq[None]) & (torch.arange(len(self.seq), device=dev)[:, None] >
                                                        torch.arange(len(self.seq), device=dev)[None])
        # how much of what chunk c' adds reaches the start of chunk c
        self.reach = torch.exp((before.T[:, :, None] - after.T[:, None, :]).masked_fill(~same, -math.inf)).float()
        self.from_start = torch.exp(before - before[self.first[self.seq]]).float()           # [C, H]
        self.last = self.first + count - 1
        self.to_end = torch.exp(after[self.last[self.seq]] - after).float()
        self.decay = torch.exp(total).float()
        self.inner = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(
            torch.triu(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev), 1), -math.inf)).float()

    def take(self, x, heads):
        """[B, T, h, D] -> FP32 [C, heads, 64, D]; a head is repeated for the value heads that share it."""
        x = x.flatten(0, 1)[self.token].float() * self.here[..., None, None]
        return x.repeat_interleave(heads // x.shape[2], 2).transpose(1, 2).contiguous()

    def give(self, x, like):
        """[C, H, 64, D] -> [B, T, H, D], rounded to the type of `like`."""
        out = torch.zeros(like.shape[0] * like.shape[1], x.shape[1], x.shape[3], dtype=like.dtype, device=x.device)
        out[self.token[self.here]] = x.transpose(1, 2)[self.here].to(like.dtype)
        return out.reshape(*like.shape[:2], *out.shape[1:])

    def states(self, k, v, h0):
        """The state before each chunk, and after each sequence."""
        add = (k * torch.exp(self.gam[..., -1:] - self.gam).float()[..., None]).mT.contiguous() @ v
        C, H, Dk, Dv = add.shape
        S = (self.reach @ add.transpose(0, 1).reshape(H, C, Dk * Dv)).reshape(H, C, Dk, Dv).transpose(0, 1)
        if h0 is not None:
            S = S + self.from_start[..., None, None] * h0[self.seq]
        return S, self.decay[self.last][..., None, None] * S[self.last] + add[self.last]


def _fwd_plain(s, c):
    f, scale = _Chunks(s), c["Dk"] ** -0.5
    q, k, v = (f.take(s[n], c["Hv"]) for n in ("q", "k", "v"))
    S, ht = f.states(k, v, s["h0"])
    o = torch.exp(f.gam).float()[..., None] * (q @ S) + (q @ k.mT.contiguous() * f.inner) @ v
    return {"o": f.give(scale * o, s["q"]), "ht": ht}


def _bwd_plain(s, c):
    f, scale, (N, H) = _Chunks(s), c["Dk"] ** -0.5, (len(s["seqs"]), c["Hv"])
    q, k, v, do = (f.take(s[n], H) for n in ("q", "k", "v", "do"))
    S, ht = f.states(k, v, s["h0"])
    grow, left = torch.exp(f.gam).float()[..., None], torch.exp(f.gam[..., -1:] - f.gam).float()[..., None]
    # the gradient of the state after each chunk
    add = scale * (q * grow).mT.contiguous() @ do
    C, _, Dk, Dv = add.shape
    dS = (f.reach.mT.contiguous() @ add.transpose(0, 1).reshape(H, C, Dk * Dv)).reshape(H, C, Dk, Dv).transpose(0, 1)
    if s["dht"] is not None:
        dS = dS + f.to_end[..., None, None] * s["dht"][f.seq]
    P, dP = q @ k.mT.contiguous() * f.inner * scale, do @ v.mT.contiguous() * f.inner * scale
    dq = scale * grow * (do @ S.mT.contiguous()) + dP @ k
    dk = dP.mT.contiguous() @ q + left * (v @ dS.mT.contiguous())
    dv = P.mT.contiguous() @ do + left * (k @ dS)
    # dg_t: what the state after the chunk passes on, and all pairs and reads of this chunk that reach over t
    own_ = (q.double() * dq.double()).sum(-1) - (k.double() * dk.double()).sum(-1)
    after = f.decay[..., None, None] * S + (k * left).mT.contiguous() @ v
    dg = own_.flip(-1).cumsum(-1).flip(-1) + (dS.double() * after.double()).sum((-1, -2))[..., None]
    dg = f.give(dg.float()[..., None], s["g"].new_empty(c["B"], c["T"], 1)).squeeze(-1)
    first = f.first
    dh0 = f.decay[first][..., None, None] * dS[first] + add[first] if s["h0"] is not None else None
    G = H // c["Hqk"]
    out = {n: f.give(x.unflatten(1, (c["Hqk"], G)).sum(2), s["q"]) for n, x in (("dq", dq), ("dk", dk))}
    out |= {"dv": f.give(dv, s["v"]), "dg": dg.double().sum((0, 1)).float() if s["g"].dim() == 1 else dg}
    return out | ({} if dh0 is None else {"dh0": dh0})


def _step_plain(s, c):
    fmt, bv, T = c["fmt"], c["bv"], c["T"]
    dst_all = s["slots"] if s["out"] is None else s["out"]
    rows = torch.nonzero(s["slots"] >= 0).flatten()
    src, dst = s["slots"][rows].long(), dst_all[rows].long()
    rep = c["Hv"] // c["Hqk"]
    q, k = (s[n][rows].float().repeat_interleave(rep, 2).transpose(1, 2) for n in ("q", "k"))   # [n, H, T, Dk]
    v = s["v"][rows].float().transpose(1, 2)
    g = s["g"].expand(c["B"], T, -1)[rows].double().transpose(1, 2)                             # [n, H, T]
    n = torch.full((len(rows),), T, device=rows.device) if s["lens"] is None else s["lens"][rows].long()
    on = (torch.arange(T, device=rows.device) < n[:, None])[:, None]
    gam = torch.cumsum(g * on, -1)
    S = _values(s["data"][0].view(torch.uint8)[src].view(s["data"].dtype) if fmt else s["data"][0][src],
                None if s["scales"] is None else s["scales"][0][src], bv)                       # [n, H, Dv, Dk]
    inner = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(
        torch.triu(torch.ones(T, T, dtype=torch.bool, device=rows.device), 1), -math.inf)).float()
    o = torch.exp(gam).float()[..., None] * (q @ S.mT.contiguous()) + (q @ k.mT.contiguous() * inner) @ v
    left = torch.exp(gam[..., -1:] - gam).float() * on
    S = torch.exp(gam[..., -1]).float()[..., None, None] * S + v.mT.contiguous() @ (k * left[..., None])
    if fmt:
        codes, d = _quantize(S, bv)
        if c["after"]:
            o = q @ _values(codes, d, bv).mT.contiguous()
        s["data"][0].view(torch.uint8)[dst] = codes.view(torch.uint8)
        s["scales"][0][dst] = d
    else:
        s["data"][0][dst] = S
    o = (o * c["Dk"] ** -0.5).transpose(1, 2).to(s["o"].dtype)
    s["o"][rows] = torch.where(on.transpose(1, 2)[..., None], o, s["o"][rows])


def _rules_plain(s, c):
    V = c["V"]
    x = s["logits"].float()
    if c["penalties"]:
        at = torch.arange(c["L"], device=x.device)
        said = at < s["lens"][..., None]
        new = said & (at >= s["prompt"][:, None, None])
        tok = s["tokens"].long()
        zero = torch.zeros_like(x)
        count = zero.scatter_add(2, tok, new.float())
        seen = zero.scatter_add(2, tok, said.float()) > 0
        rep, pres, freq = (s[n][:, None, None] for n in ("rep", "pres", "freq"))
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - freq * count - pres * (count > 0)
    if c["NB"]:
        add = torch.zeros(c["B"], V + 1, device=x.device)
        ids = torch.where(s["ids"] < 0, V, s["ids"].long())
        x = x + add.scatter_add(1, ids, s["vals"])[:, None, :V]
    if c["masked"]:
        v = torch.arange(V, device=x.device)
        allowed = (s["mask"][s["rows"].clamp_min(0).long()][..., v // 32] >> (v % 32).int()) & 1
        x = x.masked_fill((allowed == 0) & (s["rows"] >= 0)[..., None], -math.inf)
    return x.to(s["logits"].dtype)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import gateddeltanet_chunked_recurrence_amd as G
    if op == "fwd":
        if own:
            o, ht = G.gdn_linear_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"])
            return {"o": o, "ht": ht}
        return _fwd_plain(s, c)
    if op == "bwd":
        if own:
            return G.gdn_linear_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], dht=s["dht"], h0=s["h0"], cu_seqlens=s["cu"])
        return _bwd_plain(s, c)
    if op == "step":
        if own:
            G.gdn_pool_linear_step(s["pool"], 0, s["slots"], s["q"], s["k"], s["v"], s["g"], slots_out=s["out"],
                                   lens=s["lens"], out=s["o"],
                                   readout=G.READOUT_AFTER_WRITE if c["after"] else G.READOUT_BEFORE_WRITE)
        else:
            _step_plain(s, c)
        return {"o": s["o"], "states": s["data"]} | ({} if s["scales"] is None else {"scales": s["scales"]})
    # the logits as they come from the model are kept, so that each pass starts from the same ones
    if own:
        rules = dict(bias=(s["ids"], s["vals"])) if c["NB"] else {}
        if c["penalties"]:
            rules |= dict(tokens=s["tokens"], lens=s["lens"], prompt_lens=s["prompt"], repetition=s["rep"],
                          presence=s["pres"], frequency=s["freq"])
        if c["masked"]:
            rules |= dict(mask=s["mask"], mask_rows=s["rows"])
        return {"logits": G.gdn_logits_adjust(s["logits"], **rules)}
    return {"logits": _rules_plain(s, c)}


# -------------------------------------------------------------------------------------------- the work
def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "rules":
        rows = case["B"] * case["W"]
        return {"bytes": rows * case["V"] * 2 * es + (rows * case["L"] * 3 if case["penalties"] else 0) +
                case["B"] * case["NB"] * 8 + (0.89 * rows * case["V"] / 8 if case["masked"] else 0),
                "flops": rows * case["V"]}
    B, T, Hqk, Hv, Dk, Dv = (case[n] for n in ("B", "T", "Hqk", "Hv", "Dk", "Dv"))
    gates = Hv * 4 if case["gate"] == "head" else B * T * Hv * 4
    if case["op"] == "step":
        n = B - case["holes"]
        tokens = n * T * (0.5 if case["ragged"] else 1)
        page = Hv * Dk * Dv * (1 if case["fmt"] else 4) + (Hv * (Dv // case["bv"]) * 4 if case["fmt"] else 0)
        # with children, a parent's page is read once
        read = n if not case["fork"] or B < 2 else B * (1 - (1 - 1 / B) ** n)
        return {"bytes": (read + n) * page + tokens * (2 * Hqk * Dk + 2 * Hv * Dv) * es + gates,
                "flops": 4 * tokens * Hv * Dk * Dv}
    tokens, N = B * T, len(case["lens"].split(",")) if case["lens"] else B
    state = N * Hv * Dk * Dv * 4
    qkv = tokens * (2 * Hqk * Dk + Hv * Dv) * es
    if case["op"] == "fwd":
        return {"bytes": qkv + gates + tokens * Hv * Dv * es + state * (2 if case["h0"] else 1),
                "flops": 4 * tokens * Hv * Dk * Dv}
    return {"bytes": 2 * qkv + 2 * gates + tokens * Hv * Dv * es + state * (3 if case["h0"] else 0),
            "flops": 12 * tokens * Hv * Dk * Dv}


# ------------------------------------------------------------------------------------ 64-bit definition
def _span(s, c):
    """First and last token of each sequence, over all rows."""
    out, at = [], 0
    for n in s["seqs"]:
        out.append((at, at + n))
        at += n
    return out


def _attend(q, k, v, g, h0, scale, lo, hi):
    """Outputs of tokens lo .. hi - 1 of one sequence and head, as one product over all earlier tokens."""
    G = torch.cumsum(g, 0)
    w = G[lo:hi, None] - G[None, :hi]
    late = torch.arange(hi, device=g.device)[None] > torch.arange(lo, hi, device=g.device)[:, None]
    w = torch.exp(w.masked_fill(late, -math.inf))
    o = (w * torch.matmul(q[lo:hi], k[:hi].T.contiguous())) @ v[:hi]
    if h0 is not None:
        o = o + torch.exp(G[lo:hi])[:, None] * (q[lo:hi] @ h0)
    return scale * o


def _final(k, v, g, h0):
    G = torch.cumsum(g, 0)
    S = (torch.exp(G[-1] - G)[:, None] * k).T.contiguous() @ v
    return S if h0 is None else S + torch.exp(G[-1]) * h0


def _e4m3(y):
    """Nearest E4M3 value (ties to even): steps of 2^(e-3) in the binade e >= -6, at most 448."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    op, c = case["op"], case
    s = prepare(case, seed)
    if op == "rules":
        if c["B"] * c["W"] > 1500:
            return None
        x = s["logits"].double()
        for b in range(c["B"]):
            extra = torch.zeros(c["V"], dtype=torch.float64, device=x.device)
            if c["NB"]:
                keep = s["ids"][b] >= 0
                extra.index_put_((s["ids"][b][keep].long(),), s["vals"][b][keep].double(), accumulate=True)
            for w in range(c["W"]):
                y = x[b, w]
                if c["penalties"]:
                    said = s["tokens"][b, w, : int(s["lens"][b, w])].long()
                    hit = torch.bincount(said, minlength=c["V"]) > 0
                    times = torch.bincount(said[int(s["prompt"][b]):], minlength=c["V"]).double()
                    rho = s["rep"][b].double()
                    y = torch.where(hit & (y > 0), y / rho, torch.where(hit, y * rho, y))
                    y = y - s["freq"][b].double() * times - s["pres"][b].double() * times.clamp_max(1)
                y = y + extra
                if c["masked"] and int(s["rows"][b, w]) >= 0:
                    word = s["mask"][int(s["rows"][b, w])].long() & 0xFFFFFFFF
                    bits = (word[:, None] >> torch.arange(32, device=x.device)) & 1
                    y[bits.flatten()[: c["V"]] == 0] = -math.inf
                x[b, w] = y
        return {"logits": x}
    Hqk, Hv, Dk, Dv = c["Hqk"], c["Hv"], c["Dk"], c["Dv"]
    rep, scale = Hv // Hqk, Dk ** -0.5
    if op == "step":
        if c["B"] * c["T"] > 2000:
            return None
        data = s["data"][0].double()
        scales = None if s["scales"] is None else s["scales"][0].double()
        was, was_scales = data.clone(), None if scales is None else scales.clone()
        o = s["o"].double()
        for n, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            to = slot if s["out"] is None else int(s["out"][n])
            S, d = was[slot], None
            if c["fmt"]:
                d = was_scales[slot]
                S = (S.unflatten(-2, (-1, c["bv"])) * d[..., None, None]).flatten(-3, -2)
            raw = was[slot]
            for t in range(c["T"] if s["lens"] is None else int(s["lens"][n])):
                q, k = (s[i][n, t].double().repeat_interleave(rep, 0) for i in ("q", "k"))
                g = (s["g"] if s["g"].dim() == 1 else s["g"][n, t]).double()
                S = S * g.exp()[:, None, None] + s["v"][n, t].double()[:, :, None] * k[:, None]
                read = raw = S
                if c["fmt"]:
                    x = S.unflatten(-2, (-1, c["bv"]))
                    d = x.abs().amax((-1, -2)).div(448.0).clamp_min(TINY)
                    code = _e4m3(x / d[..., None, None])
                    raw = code.flatten(-3, -2)
                    if c["after"]:
                        read = (code * d[..., None, None]).flatten(-3, -2)
                o[n, t] = (read * q[:, None]).sum(-1) * scale
            data[to] = raw
            if c["fmt"]:
                scales[to] = d
        return {"o": o, "states": data[None]} | ({} if scales is None else {"scales": scales[None]})
    spans, dev = _span(s, c), s["q"].device
    flat = lambda n: s[n].flatten(0, 1)                                                    # noqa: E731
    if op == "fwd":
        o = torch.zeros(c["B"] * c["T"], Hv, Dv, dtype=torch.float64, device=dev)
        ht = torch.zeros(len(spans), Hv, Dk, Dv, dtype=torch.float64, device=dev)
    else:
        if max(s["seqs"]) > 16384:
            return None
        zeros = lambda *n: torch.zeros(*n, dtype=torch.float64, device=dev)                # noqa: E731
        dq, dk = zeros(c["B"] * c["T"], Hqk, Dk), zeros(c["B"] * c["T"], Hqk, Dk)
        dv, dg, dh0 = zeros(c["B"] * c["T"], Hv, Dv), zeros(c["B"] * c["T"], Hv), zeros(len(spans), Hv, Dk, Dv)
    for n, (a, b) in enumerate(spans):
        for h in range(Hv):
            q, k, v = flat("q")[a:b, h // rep].double(), flat("k")[a:b, h // rep].double(), flat("v")[a:b, h].double()
            g = (flat("g")[a:b, h] if s["g"].dim() == 3 else s["g"][h].expand(b - a)).double()
            h0 = None if s["h0"] is None else s["h0"][n, h].double()
            if op == "fwd":
                for lo in range(0, b - a, 2048):
                    hi = min(lo + 2048, b - a)
                    o[a + lo: a + hi, h] = _attend(q, k, v, g, h0, scale, lo, hi)
                ht[n, h] = _final(k, v, g, h0)
                continue
            wrt = [x.clone().requires_grad_() for x in (q, k, v, g)] + ([] if h0 is None else [h0.clone().requires_grad_()])
            last = wrt[4] if h0 is not None else None
            ends = (_attend(*wrt[:4], last, scale, 0, b - a), _final(*wrt[1:4], last))
            dht = torch.zeros_like(ends[1]) if s["dht"] is None else s["dht"][n, h].double()
            got = torch.autograd.grad(ends, wrt, (flat("do")[a:b, h].double(), dht))
            dq[a:b, h // rep] += got[0]
            dk[a:b, h // rep] += got[1]
            dv[a:b, h], dg[a:b, h] = got[2], got[3]
            if h0 is not None:
                dh0[n, h] = got[4]
    shape = lambda x: x.unflatten(0, (c["B"], c["T"]))                                     # noqa: E731
    if op == "fwd":
        return {"o": shape(o), "ht": ht}
    out = {"dq": shape(dq), "dk": shape(dk), "dv": shape(dv), "dg": dg.sum(0) if s["g"].dim() == 1 else shape(dg)}
    return out | ({} if s["h0"] is None else {"dh0": dh0})
