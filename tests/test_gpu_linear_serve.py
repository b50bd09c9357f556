"""Linear attention on a state pool: the step of single tokens, the prefill into
pages, and a run of all serving operators together, against float64.

Bounds of a step. o before the write: FP32 sums on the pages' own values (with
codes: factors in bf16 parts of 24 bits together), 2^-14 of the sum of absolute
values, and half a step of the output's type (2^-8 bf16, 2^-24 FP32). The state:
2^-20 of its absolute terms in FP32; with codes half a step of the code on top, E4M3
2^-4 of the value or 2^-10 of the tile's scale below its normal range, INT8 half the
scale, and the scale's own 2^-20."""
import pytest
import torch

import gateddeltanet_chunked_recurrence_amd as G
from gateddeltanet_chunked_recurrence_amd import binding
from oracle.linear import linear_fwd
from parity_util import rel, say

pytestmark = pytest.mark.gpu
QMAX = {G.QDQ_E4M3: 448.0, G.QDQ_INT8: 127.0}


def fill(pool, gen):
    states = torch.randn(pool.slots, pool.Hv, pool.Dk, pool.Dv, generator=gen) * torch.exp(
        torch.randn(pool.slots, pool.Hv, 1, 1, generator=gen))
    slots = torch.arange(pool.slots, dtype=torch.int32, device='cuda')
    for layer in range(pool.layers):
        G.gdn_pool_write(pool, layer, slots, states.cuda())


def values(pool, layer):
    slots = torch.arange(pool.slots, dtype=torch.int32, device='cuda')
    return G.gdn_pool_read(pool, layer, slots).double().cpu()


def inputs(gen, io, B, T, Hqk, Hv, Dk, Dv, gate):
    dt = torch.bfloat16 if io == 'bf16' else torch.float32
    x = torch.randn(B, T, 2 * Hqk * Dk + Hv * Dv, generator=gen).to(dt).cuda()       # one projection's output
    q, k, v = x.split([Hqk * Dk, Hqk * Dk, Hv * Dv], 2)
    g = -torch.nn.functional.softplus(torch.randn(Hv if gate == 'head' else B * T * Hv, generator=gen))
    return (q.unflatten(2, (Hqk, Dk)), k.unflatten(2, (Hqk, Dk)), v.unflatten(2, (Hv, Dv)),
            (g if gate == 'head' else g.reshape(B, T, Hv)).cuda())


def reference(q, k, v, g, S, scale):
    """(o, final S, and both over absolute values) of [T, ...] tokens of one sequence."""
    rep = v.shape[1] // q.shape[1]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    A, out, tops = S.abs(), [], []
    for t in range(q.shape[0]):
        a = torch.exp(g[t])[:, None, None]
        S = a * S + k[t][:, :, None] * v[t][:, None, :]
        A = a * A + (k[t][:, :, None] * v[t][:, None, :]).abs()
        out.append(scale * (S * q[t][:, :, None]).sum(1))
        tops.append(scale * (A * q[t][:, :, None].abs()).sum(1))
    return torch.stack(out), S, torch.stack(tops), A


def code_step(fmt, want, bv):
    """Half a step of the code of each value of [Hv, Dk, Dv]."""
    if fmt == G.QDQ_OFF:
        return torch.zeros_like(want)
    tile = want.abs().unflatten(-1, (-1, bv)).amax((1, 3)) / QMAX[fmt]
    d = tile.repeat_interleave(bv, -1)[:, None, :]
    half = d / 2 if fmt == G.QDQ_INT8 else torch.maximum(want.abs() * 2.0 ** -4, d * 2.0 ** -10)
    return half * 1.001 + d * 2.0 ** -12


@pytest.mark.parametrize('fmt,io,B,Hqk,Hv,Dk,Dv,bv,gate', [
    (G.QDQ_OFF, 'bf16', 1, 1, 1, 64, 64, 64, 'token'), (G.QDQ_OFF, 'bf16', 5, 2, 4, 128, 256, 64, 'head'),
    (G.QDQ_OFF, 'f32', 33, 1, 3, 64, 128, 64, 'token'), (G.QDQ_OFF, 'f32', 2, 4, 4, 128, 64, 64, 'head'),
    (G.QDQ_E4M3, 'bf16', 7, 2, 4, 128, 128, 64, 'token'), (G.QDQ_E4M3, 'f32', 3, 1, 2, 64, 256, 256, 'head'),
    (G.QDQ_E4M3, 'bf16', 3, 1, 2, 64, 64, 16, 'head'), (G.QDQ_INT8, 'bf16', 4, 2, 2, 128, 128, 32, 'token'),
    (G.QDQ_INT8, 'f32', 2, 1, 3, 64, 128, 128, 'head')])
@pytest.mark.parametrize('after', [False, True])
def test_step_of_one_token(fmt, io, B, Hqk, Hv, Dk, Dv, bv, gate, after):
    say(f'linear step fmt {fmt} {io} B {B} heads {Hqk}/{Hv} {Dk} x {Dv} bv {bv} gate {gate} after {after}')
    gen = torch.Generator().manual_seed(B + Dk)
    pool = G.StatePool(2, 2 * B + 1, Hv, Dk, Dv, fmt, bv)
    fill(pool, gen)
    before = [values(pool, 0), values(pool, 1)]
    q, k, v, g = inputs(gen, io, B, 1, Hqk, Hv, Dk, Dv, gate)
    order = torch.randperm(2 * B + 1, generator=gen)
    src, dst = order[:B].tolist(), order[B: 2 * B].tolist()
    src[-1] = src[0]                                                     # two children of one parent
    if B > 2:
        src[1] = -1                                                      # an empty place
    out = torch.full((B, 1, Hv, Dv), 7.0, dtype=q.dtype, device='cuda')
    G.gdn_pool_linear_step(pool, 1, torch.tensor(src, dtype=torch.int32, device='cuda'), q, k, v, g,
                           slots_out=torch.tensor(dst, dtype=torch.int32, device='cuda'), out=out,
                           readout=G.READOUT_AFTER_WRITE if after else G.READOUT_BEFORE_WRITE)
    torch.cuda.synchronize()
    now = values(pool, 1)
    assert torch.equal(values(pool, 0), before[0])
    half = 2.0 ** -8 if io == 'bf16' else 2.0 ** -24
    cpu = [x.double().cpu() for x in (q, k, v, g)]
    for n in range(B):
        if src[n] < 0:
            assert (out[n] == 7.0).all() and torch.equal(now[dst[n]], before[1][dst[n]])
            continue
        gn = cpu[3].expand(1, Hv) if gate == 'head' else cpu[3][n]
        o, S, ao, A = reference(cpu[0][n], cpu[1][n], cpu[2][n], gn, before[1][src[n]], Dk ** -0.5)
        off = (now[dst[n]] - S).abs()
        assert (off <= A * 2.0 ** -20 + code_step(fmt, S, bv)).all(), float(off.max())
        if after and fmt:
            rep = Hv // Hqk
            o = Dk ** -0.5 * (now[dst[n]] * cpu[0][n, 0].repeat_interleave(rep, 0)[:, :, None]).sum(1)[None]
        err = (out[n].double().cpu() - o).abs()
        assert (err <= ao * 2.0 ** -14 + o.abs() * half).all(), float(err.max())
    untouched = [i for i in range(2 * B + 1) if i not in dst]
    assert torch.equal(now[untouched], before[1][untouched])


@pytest.mark.parametrize('fmt,io', [(G.QDQ_OFF, 'bf16'), (G.QDQ_OFF, 'f32'), (G.QDQ_E4M3, 'bf16'), (G.QDQ_INT8, 'f32')])
def test_steps_of_ragged_batches(fmt, io):
    say(f'linear steps of ragged batches fmt {fmt} {io}')
    gen = torch.Generator().manual_seed(3)
    B, T, Hqk, Hv, Dk, Dv, bv = 6, 4, 1, 2, 64, 128, 32
    pool, twin = (G.StatePool(1, B, Hv, Dk, Dv, fmt, bv) for _ in range(2))
    for p in (pool, twin):
        fill(p, torch.Generator().manual_seed(4))
    q, k, v, g = inputs(gen, io, B, T, Hqk, Hv, Dk, Dv, 'token')
    lens = [4, 0, 1, 3, 9, -1]                                           # cut to [0, T]
    slots = torch.arange(B, dtype=torch.int32, device='cuda')
    out = torch.full((B, T, Hv, Dv), 7.0, dtype=q.dtype, device='cuda')
    start = values(pool, 0)
    G.gdn_pool_linear_step(pool, 0, slots, q, k, v, g, lens=torch.tensor(lens, dtype=torch.int32, device='cuda'), out=out)
    one = torch.full_like(out, 7.0)
    for t in range(T):                                                   # the same, token by token
        at = torch.tensor([i if t < n else -1 for i, n in enumerate(lens)], dtype=torch.int32, device='cuda')
        one[:, t: t + 1] = G.gdn_pool_linear_step(twin, 0, at, *(x[:, t: t + 1].contiguous() for x in (q, k, v, g)),
                                                  out=one[:, t: t + 1].contiguous())
    torch.cuda.synchronize()
    a, b, (x, y) = out.double().cpu(), one.double().cpu(), (values(pool, 0), values(twin, 0))
    for n, m in enumerate(lens):
        m = max(0, min(T, m))
        assert (a[n, m:] == 7.0).all()
        if m == 0:
            assert torch.equal(x[n], start[n])
        if fmt == G.QDQ_OFF:
            o, S, ao, A = reference(*(z[n, :m].double().cpu() for z in (q, k, v, g)), start[n], Dk ** -0.5) if m else (None,) * 4
            if m:
                assert ((a[n, :m] - o).abs() <= ao * 2.0 ** -14 + o.abs() * (2.0 ** -8 if io == 'bf16' else 2.0 ** -24)).all()
                assert ((x[n] - S).abs() <= A * 2.0 ** -19).all()
    # codes: a value next to a border may fall on either side, so states are compared as a whole
    assert rel(x, y) <= (2.0 ** -19 if fmt == G.QDQ_OFF else 2.0 ** -9)
    assert rel(a, b) <= (2.0 ** -19 if fmt == G.QDQ_OFF and io == 'f32' else 2.0 ** -7)


def test_pages_named_twice_or_outside_the_pool():
    gen = torch.Generator().manual_seed(6)
    pool = G.StatePool(1, 4, 2, 64, 64)
    fill(pool, gen)
    before = values(pool, 0)
    q, k, v, g = inputs(gen, 'bf16', 4, 1, 1, 2, 64, 64, 'head')
    assert G.device_errors() == 0
    out = G.gdn_pool_linear_step(pool, 0, torch.tensor([0, 0, 4, 2], dtype=torch.int32, device='cuda'), q, k, v, g)
    now = values(pool, 0)
    assert torch.isnan(out[:3]).all() and torch.isfinite(out[3]).all()
    assert torch.equal(now[[0, 1, 3]], before[[0, 1, 3]]) and not torch.equal(now[2], before[2])
    assert G.device_errors() == binding.DEVERR_POOL_SLOT


@pytest.mark.parametrize('fmt', [G.QDQ_OFF, G.QDQ_E4M3])
def test_prompts_then_beams_together(fmt):
    """Prefill into pages, forks, steps, rules on logits, beams that change places: the pages hold
    what float64 makes of each beam's own tokens (codes: compared as a whole, one rounding a write of 2^-4 at most)."""
    say(f'serving run, fmt {fmt}')
    gen = torch.Generator().manual_seed(7)
    B, W, Hqk, Hv, Dk, Dv, V, steps = 2, 3, 1, 2, 64, 64, 900, 4
    pool = G.StatePool(1, B * W + B, Hv, Dk, Dv, fmt, 64)
    lens = [70, 41]
    cu = torch.tensor([0, 70, 111], dtype=torch.int32, device='cuda')
    dt = torch.bfloat16
    q, k = (torch.nn.functional.normalize(torch.randn(1, 111, Hqk, Dk, generator=gen), dim=-1).to(dt) for _ in range(2))
    v, g = torch.randn(1, 111, Hv, Dv, generator=gen).to(dt), torch.log(0.8 + 0.19 * torch.rand(Hv, generator=gen))
    home = torch.tensor([B * W, B * W + 1], dtype=torch.int32, device='cuda')
    G.gdn_pool_linear_prefill(pool, 0, home, q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu_seqlens=cu, resume=False)
    slots = torch.randperm(B * W, generator=gen).int().reshape(B, W)
    G.gdn_pool_copy(pool, home[:, None].expand(B, W).flatten().contiguous(), slots.flatten().cuda())
    own = [[[(q[:, a:b], k[:, a:b], v[:, a:b])] for _ in range(W)] for a, b in ((0, 70), (70, 111))]
    hist = torch.full((B, W, 64), -1, dtype=torch.int32)
    said = [[[1 + b] for _ in range(W)] for b in range(B)]
    scores = torch.zeros(B, W).masked_fill(torch.arange(W) > 0, -1.0).cuda()
    rep = torch.tensor([1.3, 1.0])
    bias = (torch.tensor([[5, -1], [8, 9]]).int(), torch.tensor([[2.0, 0.0], [-torch.inf, 1.0]]))
    mask = torch.full((2, (V + 31) // 32), -1, dtype=torch.int32)
    mask[1, ::2] = 0
    for step in range(steps):
        tq, tk = (torch.nn.functional.normalize(torch.randn(B * W, 1, Hqk, Dk, generator=gen), dim=-1).to(dt) for _ in range(2))
        tv = torch.randn(B * W, 1, Hv, Dv, generator=gen).to(dt)
        out = G.gdn_pool_linear_step(pool, 0, slots.flatten().cuda(), tq.cuda(), tk.cuda(), tv.cuda(), g.cuda())
        for b in range(B):
            for w in range(W):
                i = b * W + w
                own[b][w] = own[b][w] + [(tq[i: i + 1], tk[i: i + 1], tv[i: i + 1])]
                hist[b, w, : len(said[b][w])] = torch.tensor(said[b][w], dtype=torch.int32)
                n = [torch.cat([x[j] for x in own[b][w]], 1).double() for j in range(3)]
                o, ht = linear_fwd(*n, g.double(), Dk ** -0.5)
                tol = 2.0 ** -7 if fmt == G.QDQ_OFF else (step + 2) * 2.0 ** -5
                assert rel(out[i, 0], o[0, -1]) <= tol, (step, b, w, rel(out[i, 0], o[0, -1]))
        logits = (torch.randn(B, W, V, generator=gen) * 3).to(dt).cuda()
        rules = dict(tokens=hist.cuda(), lens=torch.tensor([[len(s) for s in r] for r in said], dtype=torch.int32).cuda(),
                     prompt_lens=torch.tensor([1, 1], dtype=torch.int32).cuda(), repetition=rep.cuda(),
                     frequency=torch.tensor([0.5, 0.0]).cuda(), bias=tuple(t.cuda() for t in bias), mask=mask.cuda(),
                     mask_rows=torch.tensor([[0, -1, 1], [1, 1, 0]], dtype=torch.int32).cuda())
        keep = logits.clone()
        adjusted = G.gdn_logits_adjust(logits, **rules)
        want = G.gdn_beam_select(adjusted, scores)
        got = G.gdn_beam_advance(pool, slots.cuda(), logits, scores, rules=rules)
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(logits, keep)
        scores, parents, tokens = got[0], got[1].cpu(), got[2].cpu()
        own = [[list(own[b][parents[b, w]]) for w in range(W)] for b in range(B)]
        said = [[said[b][parents[b, w]] + [int(tokens[b, w])] for w in range(W)] for b in range(B)]
    now = values(pool, 0)
    for b in range(B):
        for w in range(W):
            n = [torch.cat([x[j] for x in own[b][w]], 1).double() for j in range(3)]
            S = linear_fwd(*n, g.double(), 1.0)[1][0]
            assert rel(now[int(slots[b, w])], S) <= (2.0 ** -13 if fmt == G.QDQ_OFF else (steps + 1) * 2.0 ** -5)
    assert G.device_errors() == 0
