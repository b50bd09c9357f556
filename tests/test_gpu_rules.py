"""Rules on logits (penalties, biases, grammar masks) on the GPU against a float64
loop over the rows.

Bounds: repetition, frequency, presence and bias are one FP32 operation each, at
most six roundings of 2^-24 of the largest intermediate value, and the result is
rounded once to the logits' type (half a step: 2^-8 bf16, 2^-24 FP32). Tokens that no
rule names, and masked ones, are exact."""
import math

import pytest
import torch

import gateddeltanet_chunked_recurrence_amd as G
from gateddeltanet_chunked_recurrence_amd import binding
from parity_util import say

pytestmark = pytest.mark.gpu


def reference(x, tokens=None, lens=None, prompt_lens=None, repetition=None, presence=None, frequency=None, bias=None,
              mask=None, mask_rows=None):
    """(result float64, largest value on the way, touched) of [B, W, V] logits on the CPU."""
    B, W, V = x.shape
    out, top = x.double().clone(), x.double().abs().nan_to_num(0, 0, 0)
    touched = torch.zeros(B, W, V, dtype=torch.bool)
    for b in range(B):
        for w in range(W):
            hist = [] if tokens is None else tokens[b, w, : max(0, min(tokens.shape[2], int(lens[b, w]) if lens is not None else 10 ** 9))].tolist()
            prompt = 0 if prompt_lens is None else int(prompt_lens[b])
            said, times = set(), {}
            for i, t in enumerate(hist):
                if 0 <= t < V:
                    said.add(t)
                    if i >= prompt:
                        times[t] = times.get(t, 0) + 1
            add = {}
            if bias is not None:
                for t, v in zip(bias[0][b].tolist(), bias[1][b].tolist()):
                    if 0 <= t < V:
                        add[t] = add.get(t, 0.0) + v
            rho = 1.0 if repetition is None else float(repetition[b])
            for t in said | set(add):
                v = float(out[b, w, t])
                if t in said:
                    v = v / rho if v > 0 else v * rho
                n = times.get(t, 0)
                if n:
                    v -= (0.0 if frequency is None else float(frequency[b])) * n
                    v -= 0.0 if presence is None else float(presence[b])
                if t in add:
                    v = -math.inf if add[t] == -math.inf else v + add[t]
                extra = (abs(float(frequency[b])) * n if frequency is not None else 0) + abs(add.get(t, 0.0) if math.isfinite(add.get(t, 0.0)) else 0) + \
                    (abs(float(presence[b])) if presence is not None else 0)
                top[b, w, t] = top[b, w, t] * max(rho, 1 / rho) + extra + (
                    sum(abs(v2) for t2, v2 in zip(bias[0][b].tolist(), bias[1][b].tolist()) if t2 == t and math.isfinite(v2)) if t in add else 0)
                out[b, w, t] = v
                touched[b, w, t] = True
            if mask is not None:
                row = b * W + w if mask_rows is None else int(mask_rows[b, w])
                if row >= 0:
                    bits = (mask[row].long()[torch.arange(V) // 32] >> (torch.arange(V) % 32)) & 1
                    out[b, w, bits == 0] = -math.inf
    # beyond the logits' type by half a step or more: infinite in it
    beyond = out.abs() >= torch.finfo(x.dtype).max * (1 + torch.finfo(x.dtype).eps / 4)
    return torch.where(beyond, torch.sign(out) * math.inf, out), top, touched


def check(x, rules, out=None, **kw):
    cuda = {n: tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda() for n, v in rules.items()}
    keep = x.clone()
    got = G.gdn_logits_adjust(x, out=out, **cuda)
    torch.cuda.synchronize()
    want, top, touched = reference(keep.cpu(), **rules)
    g, half = got.double().cpu(), 2.0 ** -8 if x.dtype is torch.bfloat16 else 2.0 ** -24
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(g), torch.isnan(want)) and torch.equal(g[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)])
    off = (g - want).abs()[fin]
    bound = (6 * 2.0 ** -24 * top + half * want.abs() + 2.0 ** -133)[fin]
    assert (off <= bound).all(), float((off / bound).max())
    plain = ~touched & fin
    same = got.cpu()[plain].view(torch.int16 if x.dtype is torch.bfloat16 else torch.int32)
    assert torch.equal(same, keep.cpu()[plain].view(same.dtype))
    return got


def make(gen, B, W, V, L, NB, masks, dtype, odd=True):
    x = torch.randn(B, W, V, generator=gen) * 4
    tokens = torch.randint(-2 if odd else 0, V + (3 if odd else 0), (B, W, L), generator=gen).int()
    if L > 4:
        tokens[:, :, L // 2:: 2] = tokens[:, :, : 1]                    # the same token again and again
    r = dict(tokens=tokens, lens=torch.randint(0, L + 1, (B, W), generator=gen).int(),
             prompt_lens=torch.randint(0, L + 1, (B,), generator=gen).int(), repetition=0.8 + torch.rand(B, generator=gen),
             presence=torch.randn(B, generator=gen), frequency=torch.randn(B, generator=gen))
    if NB:
        ids = torch.randint(-1, V + 1, (B, NB), generator=gen).int()
        ids[:, NB // 2] = ids[:, 0]                                     # an id given twice is added twice
        r['bias'] = (ids, torch.randn(B, NB, generator=gen) * 3)
    if masks:
        r['mask'] = torch.randint(-2 ** 31, 2 ** 31, (masks, (V + 31) // 32), generator=gen).int()
        r['mask_rows'] = torch.randint(-1, masks, (B, W), generator=gen).int()
    return x.to(dtype).cuda(), r


@pytest.mark.parametrize('dtype', [torch.bfloat16, torch.float32], ids=['bf16', 'f32'])
@pytest.mark.parametrize('B,W,V,L,NB,masks', [
    (1, 1, 1, 1, 1, 1), (1, 1, 7, 3, 2, 0), (2, 3, 31, 0, 5, 2), (3, 2, 1000, 64, 0, 3), (1, 4, 1025, 700, 12, 0),
    (2, 1, 8191, 33, 1024, 1), (1, 2, 40003, 2500, 300, 4), (40, 13, 131, 20, 3, 5), (2, 270, 16385, 9, 2, 2)])
def test_rules(B, W, V, L, NB, masks, dtype):
    say(f'rules {B} x {W} x {V}, {L} tokens, {NB} biases, {masks} masks, {dtype}')
    x, r = make(torch.Generator().manual_seed(V), B, W, V, L, NB, masks, dtype)
    check(x, r)


@pytest.mark.parametrize('dtype', [torch.bfloat16, torch.float32], ids=['bf16', 'f32'])
def test_rows_at_any_element_in_place_and_strided(dtype):
    say(f'rules on strided rows {dtype}')
    gen = torch.Generator().manual_seed(5)
    x, r = make(gen, 3, 2, 997, 50, 7, 4, dtype)
    big = torch.full((3, 2, 3, 1003), 7.0, dtype=dtype, device='cuda')
    for off in range(3):
        view = big[:, :, 2, off: off + 997]
        view.copy_(x)
        got = check(view, r, out=view)                                  # the last position, in place
        assert got.data_ptr() == view.data_ptr()
        rest = big.clone()
        rest[:, :, 2, off: off + 997] = 7.0
        assert (rest == 7.0).all()                                      # nothing beside the rows is written
        big.fill_(7.0)
        check(x, r, out=big[:, :, 1, off: off + 997])                   # from one alignment to another
        big.fill_(7.0)


def test_each_rule_alone_and_none():
    gen = torch.Generator().manual_seed(6)
    x, r = make(gen, 2, 2, 500, 40, 9, 3, torch.bfloat16)
    t = {n: r[n] for n in ('tokens', 'lens')}
    for rules in ({}, t, t | {'repetition': r['repetition']}, t | {'presence': r['presence']},
                  t | {'frequency': r['frequency'], 'prompt_lens': r['prompt_lens']}, {'bias': r['bias']},
                  {'mask': r['mask'], 'mask_rows': r['mask_rows']}, {'tokens': r['tokens'], 'repetition': r['repetition']},
                  {'mask': torch.cat([r['mask'], r['mask']])}):
        say('rules alone', sorted(rules))
        check(x, rules)


def test_infinities_nan_bans_and_empty_masks():
    x = torch.tensor([[[1.0, -1.0, math.inf, -math.inf, math.nan, 0.0, -0.0, 3e38]]], device='cuda')
    ids = torch.tensor([[0, 1, 2, 3, 4, 2, 7]]).int()
    vals = torch.tensor([[-math.inf, 5.0, -math.inf, 9.0, -math.inf, 1.0, 3e38]])
    say('rules on infinities')
    got = check(x, dict(tokens=torch.tensor([[[5, 6, 4, 3, 2]]]).int(), repetition=torch.tensor([2.0]), bias=(ids, vals)))
    assert got[0, 0, 0] == -math.inf and got[0, 0, 2] == -math.inf and got[0, 0, 4] == -math.inf   # bans
    assert got[0, 0, 7] == math.inf
    none = check(x, dict(mask=torch.zeros(1, 1).int()))
    assert (none == -math.inf).all()                                    # a mask that leaves nothing, NaN too


def test_mask_rows_outside_the_table_say_so():
    x = torch.randn(1, 3, 300, device='cuda')
    mask = torch.full((2, 10), -1, dtype=torch.int32, device='cuda')
    assert G.device_errors() == 0
    got = G.gdn_logits_adjust(x, mask=mask, mask_rows=torch.tensor([[1, 2, -2]], dtype=torch.int32, device='cuda'))
    assert torch.equal(got[0, 0], x[0, 0]) and torch.isnan(got[0, 1:]).all()
    assert G.device_errors() == binding.DEVERR_RULE_ROW


def test_streams_graphs_and_repeats():
    gen = torch.Generator().manual_seed(8)
    x, r = make(gen, 4, 3, 20000, 300, 20, 3, torch.bfloat16)
    cuda = {n: tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda() for n, v in r.items()}
    want = check(x, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = G.gdn_logits_adjust(x, **cuda)
    side.synchronize()
    bits = lambda t: t.view(torch.int16)                                # noqa: E731
    assert torch.equal(bits(other), bits(want))
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gdn_logits_adjust(x, out=out, **cuda)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(x.dtype))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(G.gdn_logits_adjust(x, **cuda)))
