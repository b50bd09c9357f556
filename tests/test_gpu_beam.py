"""Beam selection on the GPU against a plain FP64 selection: order by total,
ties to the lower beam and then the lower token.

Tolerances: the sum of exponentials is FP32 within a part (at most 64 terms
per lane, then a tree of 8 steps; each exponential off by 2^-22 relative for
|x - m| log2(e) < 4, and by |x - m| 2^-23 for smaller ones, which weigh less),
so a log-sum is off by less than 80 2^-24 = 5e-6 in the worst order and a total
by that; the returned FP32 adds half a step, 2^-24 relative. Two candidates
may change places only where their FP64 totals are within twice 5e-6."""
import math

import pytest
import torch

from gateddeltanet_chunked_recurrence_amd import binding as B
from parity_util import say

pytestmark = pytest.mark.gpu

EPS = 5e-6


def _totals(logits, scores, finished, pad):
    x = logits.double().nan_to_num(nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf).cpu()
    m = x.amax(-1, keepdim=True)
    safe = torch.where(m.isfinite(), m, 0.0)
    s = torch.exp(x - safe).sum(-1, keepdim=True)
    total = torch.where(s > 0, (x - safe) - s.log(), -math.inf) + scores.double().cpu().unsqueeze(-1)
    total = torch.where(total.isnan(), -math.inf, total)
    if finished is not None:
        f = finished.cpu() != 0
        total[f] = -math.inf
        total[..., pad][f] = scores.double().cpu()[f]
    return total


def _check(logits, scores, K, finished=None, pad=0, exact_ids=False):
    Bn, W, V = logits.shape
    got_s, got_p, got_t = (t.cpu() for t in B.gdn_beam_select(logits, scores, K, finished, pad))
    total = _totals(logits, scores, finished, pad)
    for b in range(Bn):
        flat = total[b].reshape(-1)
        order = torch.argsort(flat, descending=True, stable=True)[:K]
        order = order[flat[order] > -math.inf]
        n = len(order)
        want = flat[order]
        assert bool((got_p[b, n:] == -1).all() and (got_t[b, n:] == -1).all() and (got_s[b, n:] == -math.inf).all())
        assert bool((got_p[b, :n] >= 0).all() and (got_p[b, :n] < W).all())
        assert bool((got_t[b, :n] >= 0).all() and (got_t[b, :n] < V).all())
        mine = flat[got_p[b, :n].long() * V + got_t[b, :n].long()]
        bound = EPS + 2.0 ** -24 * want.abs()
        assert bool(((got_s[b, :n].double() - want).abs() <= bound).all()), (b, float((got_s[b, :n] - want).abs().max()))
        assert bool(((mine - want).abs() <= 2 * EPS).all()), b
        ids = got_p[b, :n].long() * V + got_t[b, :n].long()
        assert len(set(ids.tolist())) == n
        # places whose total is not within the bound of a neighbour's are the reference's own
        gap = torch.full((n + 1,), math.inf, dtype=torch.float64)
        gap[1:n] = want[:-1] - want[1:]
        rest = torch.argsort(flat, descending=True, stable=True)[K:K + 1]
        if n == K and len(rest):
            gap[n] = want[-1] - flat[rest[0]]
        # an exact tie within a beam has its order fixed by the tokens
        clear = torch.minimum(gap[:-1], gap[1:]) > 2 * EPS
        if exact_ids:
            clear[:] = True
        assert bool((ids == order)[clear].all()), b
        assert int(clear.sum()) or n == 0 or not exact_ids


def _logits(Bn, W, V, dt, seed, spread=2.0):
    gen = torch.Generator(device='cuda').manual_seed(seed)
    x = torch.randn(Bn, W, V, generator=gen, device='cuda') * spread
    s = -20.0 * torch.rand(Bn, W, generator=gen, device='cuda')
    return x.to(dt), s


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Bn,W,V,K", [(1, 1, 1, 1), (1, 1, 3, 5), (2, 3, 7, 4), (3, 4, 255, 8), (2, 5, 2048, 10),
                                      (1, 4, 4099, 4), (2, 32, 1001, 64), (5, 7, 9973, 14), (1, 4, 131072, 8),
                                      (40, 8, 16385, 16), (200, 6, 33000, 12)])
def test_select_against_fp64(dt, Bn, W, V, K):
    say(f"beam select {dt} B={Bn} W={W} V={V} K={K}")
    x, s = _logits(Bn, W, V, dt, seed=V + K)
    s = s * 0.05                                          # beams close enough to compete
    _check(x, s, K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_of_a_padded_vocabulary(dt):
    """Rows evenly spaced in a wider tensor, starting off 16-byte boundaries."""
    for V, pad in ((1000, 3), (999, 0), (77, 50), (20001, 7)):
        x, s = _logits(3, 4, V + pad, dt, seed=V)
        x[..., V:] = 99.0                                 # never to be read as part of a row
        _check(x[..., :V], s * 0.1, 9)
    x, s = _logits(6, 1, 500, dt, seed=1)                 # one beam per request, every other row of a tensor
    _check(x.view(3, 2, 500)[:, :1], s[::2].contiguous(), 3)


@pytest.mark.parametrize("dt,Bn,W,V,K", [(torch.bfloat16, 3, 32, 40000, 64), (torch.float32, 1, 32, 280001, 64)])
def test_many_candidates_per_request(dt, Bn, W, V, K):
    """More candidates than a workgroup's registers hold; in the second case
    more parts than its LDS does."""
    say(f"beam select {dt} B={Bn} W={W} V={V} K={K}")
    x, s = _logits(Bn, W, V, dt, seed=V)
    _check(x, s * 0.05, K)
    x[0].fill_(-3.0)                                      # all equal: the lowest tokens of the best beams
    s = torch.zeros_like(s)
    got = [t.cpu() for t in B.gdn_beam_select(x, s, K)]
    assert got[1][0].tolist() == [0] * K and got[2][0].tolist() == list(range(K))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 9, 1003, 8191])
def test_the_last_position_of_a_longer_block(dt, V):
    """A view whose first row starts off a 16-byte boundary."""
    T = 4 if V % 2 else 6
    x, s = _logits(6, T, V, dt, seed=V)
    x[:, :-1] = 99.0
    last = x[:, -1].unflatten(0, (2, 3))
    assert last.data_ptr() % 16 or V == 2
    _check(last, s[:, 0].reshape(2, 3) * 0.1, 5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_masked_and_strange_logits(dt):
    V = 5000
    x, s = _logits(4, 3, V, dt, seed=2)
    s = s * 0.1
    x[0, 0] = -math.inf                                   # nothing left
    x[0, 1, 1:] = -math.inf                               # one token left
    x[0, 2] = -math.inf
    x[0, 2, [4999, 7, 2500]] = torch.tensor([1.0, 2.0, 1.0], dtype=dt, device='cuda')
    x[1] = -math.inf                                      # a request without any candidate
    x[2, 0, ::2] = float('nan')                           # NaN counts as masked
    x[2, 1] = float('nan')
    x[2, 2, :] = torch.finfo(dt).min                      # masks of the type's lowest value: an even spread
    x[3, 0, 17] = math.inf                                # all the probability on one token
    x[3, 1, [4000, 30]] = math.inf                        # on two
    for K in (2, 6, 40):
        _check(x, s, K)
    s[3, 2] = -math.inf                                   # a dead beam
    s[0, 1] = -math.inf
    _check(x, s, 6)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,V,K", [(1, 3000, 5), (4, 40000, 16), (32, 9000, 64), (8, 2, 64)])
def test_equal_totals_go_to_the_lowest_places(dt, W, V, K):
    """Constant rows: every total is equal, so the choice is the first K
    tokens of the first beam (then of the next), whatever overflows a list."""
    for value in (0.0, -3.5, -0.0):
        x = torch.full((2, W, V), value, dtype=dt, device='cuda')
        x[1, 0, : V // 2] = x[1, 0, : V // 2] - 1.0
        x[0, :, 1::2] = 0.0 if value == 0 else value      # both zeros are one value
        got_s, got_p, got_t = (t.cpu() for t in B.gdn_beam_select(x, torch.zeros(2, W, device='cuda'), K))
        n = min(K, W * V)
        assert got_p[0, :n].tolist() == [i // V for i in range(n)]
        assert got_t[0, :n].tolist() == [i % V for i in range(n)]
        assert bool(((got_s[0, :n] + math.log(V)).abs() <= EPS + 2.0 ** -24 * math.log(V)).all())
        assert bool((got_t[0, n:] == -1).all())
        # the lowered half of one beam makes its other half the best of all
        top = V - V // 2
        assert got_p[1, : min(K, top)].tolist() == [0] * min(K, top)
        assert got_t[1, : min(K, top)].tolist() == list(range(V // 2, V // 2 + min(K, top)))


def test_ties_of_a_coarse_grid():
    """bf16 logits on a grid of 8 values: hundreds of exact ties inside a
    beam, on both sides of the K-th place."""
    gen = torch.Generator(device='cuda').manual_seed(3)
    x = torch.randint(0, 8, (3, 2, 30000), generator=gen, device='cuda').to(torch.bfloat16)
    s = torch.tensor([[0.0, -0.5]] * 3, device='cuda')
    _check(x, s, 64, exact_ids=True)


def test_ascending_rows():
    """Each next token better than the last: every part's best are its last."""
    x = torch.arange(50000, device='cuda', dtype=torch.float32).expand(1, 2, 50000).contiguous() * 1e-3
    _check(x, torch.tensor([[0.0, -0.0123]], device='cuda'), 20)


@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_finished_beams_offer_one_token(kind):
    x, s = _logits(3, 4, 3001, torch.bfloat16, seed=4)
    s = s * 0.2
    done = torch.tensor([[0, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 1]], device='cuda').to(kind)
    x[0, 1] = float('nan')                                # a finished beam's logits are not read
    x2 = x.clone()
    x2[0, 1] = 0.0
    got = B.gdn_beam_select(x, s, 8, done, 17)
    for a, b in zip(got, B.gdn_beam_select(x2, s, 8, done, 17)):
        assert torch.equal(a, b)
    _check(x2, s, 8, done, 17)
    scores, parents, tokens = (t.cpu() for t in got)
    assert sorted(parents[1, :4].tolist()) == [0, 1, 2, 3] and tokens[1].tolist() == [17] * 4 + [-1] * 4
    # a score of -inf: such a beam offers nothing
    s[1, 2] = -math.inf
    _check(x2, s, 8, done, 17)


def test_calls_on_two_streams_at_once():
    """Each call has its own workspace, so two streams do not disturb each other."""
    xs = [_logits(8, 4, 60000, torch.bfloat16, seed=5 + i) for i in range(2)]
    want = [B.gdn_beam_select(x, s, 8) for x, s in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(B.gdn_beam_select(*xs[i], 8))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("V", [1021, 60001])
def test_rows_shifted_by_a_constant(V):
    """Each beam's logits shifted by another constant, up to 10,000: over several
    waves and parts of a row the log-sum's error is that of the differences, so
    the bound at the top holds at every shift."""
    x, s = _logits(3, 6, V, torch.float32, seed=V)
    shift = torch.tensor([0.0, 101.3, -1000.7, 3001.9, 10000.1, 20.6], device='cuda')
    _check((x + shift[:, None]).contiguous(), s * 0.05, 12)
    _check((x - 7.0 * shift[:, None]).contiguous(), s * 0.05, 12)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [900, 70001])
def test_rows_of_large_finite_logits(dt, V):
    """Rows masked throughout with a large finite number, rows whose logits
    are that large, and rows around the size where the kernel's form changes."""
    for base in (-1e9, -1e10, 1e10, -1e12, 3e15, -1e30, 2.0 ** 99, -2.0 ** 101):
        x, s = _logits(2, 4, V, dt, seed=V)
        s = s * 0.05
        x[0, 0] = base                                    # nothing but the mask
        x[0, 1] = base
        x[0, 1, V // 2] = base * (1 - 2.0 ** -7)          # one logit apart from the rest
        x[0, 2, 11:] = -abs(base)                         # all masked but a few
        x[1, 1, 1::2] = -abs(base)
        x[1, 2, : V // 2] = base                          # whole waves of the mask
        _check(x, s, 7)
    edge = 2.0 ** torch.arange(18, 34, device='cuda', dtype=torch.float32)
    rows = edge.repeat_interleave(2) * torch.tensor([1.0, -1.0], device='cuda').repeat(16)
    step = torch.linspace(-3.0, 3.0, V, device='cuda')
    x = (rows[:, None] + step).to(dt).view(4, 8, V)       # waves on both sides of a power of two
    _check(x, -0.05 * torch.rand(4, 8, device='cuda'), 9)


def test_one_request_of_a_larger_batch():
    """Contiguous slices of scores and finished off 16-byte boundaries."""
    x, s = _logits(5, 3, 777, torch.bfloat16, seed=6)
    done = torch.rand(5, 3, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    for b in range(5):
        assert b != 1 or (s[b:b + 1].data_ptr() % 16 and done[b:b + 1].data_ptr() % 16)
        got = B.gdn_beam_select(x[b:b + 1], s[b:b + 1], 4, done[b:b + 1], 5)
        want = B.gdn_beam_select(x[b:b + 1].clone(), s[b:b + 1].clone(), 4, done[b:b + 1].clone(), 5)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
