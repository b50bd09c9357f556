"""Linear attention with a decay per head on the GPU against the float64 oracle.

Bounds. U = 2^-8 is half a bf16 step. Each value of o is a sum of products; the
kernel rounds the weighted products of pairs and the state it is read from to bf16 at
most once each and the result once, so |error| <= U A + U |o|, with A the same sum over the
absolute values of every factor (which the oracle computes from |q|, |k|, |v|,
|h0|); FP32 sums and exponentials add less than 2^-14 A at these lengths (under
900 sums of 2^-24 each, exponents to 2^-21). dq, dk, dv: the same form. States and
dh0: factors in two bf16 parts, U^2 = 2^-16 A, and the FP32 part. With FP32 inputs
there is the FP32 part alone. dg: its sums run over q . dq and k . dk of one segment
(under 900 tokens here), each with 2^-15 of its absolute value at most (two split factors),
so 2^-15 times the suffix sum of their absolute values, plus the same share of dg's own."""
import math

import pytest
import torch

import gateddeltanet_chunked_recurrence_amd as G
from oracle.linear import linear_bwd, linear_fwd
from parity_util import rel, say

pytestmark = pytest.mark.gpu

U, FP32 = 2.0 ** -8, 2.0 ** -14


def make(io, B, T, lens, Hqk, Hv, Dk, Dv, gate='token', h0=True, view=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)                      # noqa: E731
    dt = torch.bfloat16 if io == 'bf16' else torch.float32
    cu = None
    if lens is not None:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        B, T = 1, max(T, cu[-1])
    q, k, v, do = rnd(B, T, Hqk, Dk), rnd(B, T, Hqk, Dk), rnd(B, T, Hv, Dv), rnd(B, T, Hv, Dv)
    if gate == 'head':
        g = torch.log(0.8 + 0.199 * torch.rand(Hv, generator=gen))
    else:
        g = -torch.nn.functional.softplus(rnd(B, T, Hv) - 1.0)
        if gate == 'reset':                                             # resets, and gates that keep all or nothing
            pick = torch.rand(B, T, Hv, generator=gen)
            g = torch.where(pick < 0.05, -math.inf, torch.where(pick < 0.1, -95.0, torch.where(pick < 0.2, 0.0, g)))
    N = len(lens) if lens is not None else B
    x = dict(q=q.to(dt), k=k.to(dt), v=v.to(dt), g=g, do=do.to(dt),
             h0=rnd(N, Hv, Dk, Dv) if h0 else None, dht=rnd(N, Hv, Dk, Dv) if h0 else None)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    if view:                                                            # one projection's output
        y = torch.cat([x['q'].flatten(2), x['k'].flatten(2), x['v'].flatten(2), x['v'].flatten(2)[..., :64]], 2).cuda()
        s = [Hqk * Dk, Hqk * Dk, Hv * Dv, 64]
        a, b, c, _ = y.split(s, 2)
        d['q'], d['k'], d['v'] = a.unflatten(2, (Hqk, Dk)), b.unflatten(2, (Hqk, Dk)), c.unflatten(2, (Hv, Dv))
    d['cu'] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device='cuda')
    return {n: None if t is None else t.double() for n, t in x.items()}, d, cu


def within(name, got, want, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    off = (got - want).abs()
    worst = float((off / bound.clamp_min(1e-300)).max()) if off.numel() else 0.0
    say(f'  {name}: rel {rel(got, want):.2e}, {worst:.3f} of its bound')
    assert (off <= bound).all(), (name, worst)


def positive(x):
    return {n: None if t is None else t if n == 'g' else t.abs() for n, t in x.items()}


def check_fwd(x, d, cu, io, out=None):
    scale = x['q'].shape[-1] ** -0.5
    o, ht = G.gdn_linear_fwd(d['q'], d['k'], d['v'], d['g'], h0=d['h0'], cu_seqlens=d['cu'], out=out)
    torch.cuda.synchronize()
    p = positive(x)
    wo, wh = linear_fwd(x['q'], x['k'], x['v'], x['g'], scale, x['h0'], cu)
    ao, ah = linear_fwd(p['q'], p['k'], p['v'], x['g'], scale, p['h0'], cu)
    b = io == 'bf16'
    used = slice(None) if cu is None else slice(0, cu[-1])
    within('o', o[:, used], wo[:, used], (ao * (U * b + FP32) + wo.abs() * U * b)[:, used])
    within('ht', ht, wh, ah * (U * U * b + FP32))
    return o


def check_bwd(x, d, cu, io, out=None):
    scale = x['q'].shape[-1] ** -0.5
    got = G.gdn_linear_bwd(d['q'], d['k'], d['v'], d['g'], d['do'], dht=d['dht'], h0=d['h0'], cu_seqlens=d['cu'], out=out)
    torch.cuda.synchronize()
    p = positive(x)
    want = linear_bwd(x['q'], x['k'], x['v'], x['g'], scale, x['do'], x['dht'], x['h0'], cu)
    top = linear_bwd(p['q'], p['k'], p['v'], x['g'], scale, p['do'], p['dht'], p['h0'], cu)
    b = io == 'bf16'
    used = slice(None) if cu is None else slice(0, cu[-1])
    for n in ('dq', 'dk', 'dv'):
        within(n, got[n][:, used], want[n][:, used], (top[n] * (U * b + FP32) + want[n].abs() * U * b)[:, used])
    if x['h0'] is not None:
        within('dh0', got['dh0'], want['dh0'], top['dh0'] * (U * U * b + FP32))
    Hv = x['v'].shape[2]
    rep = Hv // x['q'].shape[2]
    # a head's share of q . dq is at most its group's
    dots = sum((p[a] * top['d' + a]).sum(-1) for a in ('q', 'k')).repeat_interleave(rep, 2)
    sums = torch.zeros_like(dots).flatten(0, 1)
    flat = dots.flatten(0, 1)
    for lo, hi in zip(cu[:-1], cu[1:]) if cu else [(i * x['q'].shape[1], (i + 1) * x['q'].shape[1]) for i in range(x['q'].shape[0])]:
        sums[lo:hi] = flat[lo:hi].flip(0).cumsum(0).flip(0)
    sums = sums.reshape(dots.shape)
    if x['g'].dim() == 1:
        sums = sums.sum((0, 1))
        within('dg', got['dg'], want['dg'], (sums + top['dg']) * 2.0 ** -15 + 1e-30)
    else:
        within('dg', got['dg'][:, used], want['dg'][:, used], ((sums + top['dg']) * 2.0 ** -15 + 1e-30)[:, used])
    if x['q'].shape[1]:
        assert rel(got['dg'] if x['g'].dim() == 1 else got['dg'][:, used], want['dg'] if x['g'].dim() == 1 else want['dg'][:, used]) < 2.0 ** -13
    return got


CASES = [
    # io, B, T, lens, Hqk, Hv, Dk, Dv, gate, h0, view
    ('bf16', 1, 1, None, 1, 1, 64, 64, 'token', True, False),
    ('bf16', 2, 64, None, 1, 2, 64, 64, 'token', False, False),
    ('bf16', 1, 65, None, 2, 2, 128, 128, 'token', True, False),
    ('bf16', 2, 150, None, 1, 3, 128, 64, 'head', True, True),
    ('bf16', 1, 203, None, 1, 1, 64, 256, 'token', True, False),
    ('bf16', 1, 700, None, 1, 2, 128, 256, 'token', True, False),
    ('bf16', 1, 515, None, 1, 1, 64, 128, 'reset', True, False),
    ('bf16', 1, 0, [1, 63, 0, 130, 300, 2], 2, 4, 128, 128, 'token', True, True),
    ('bf16', 1, 900, [257, 64, 500], 1, 1, 64, 64, 'head', False, False),
    ('f32', 1, 1, None, 1, 1, 64, 64, 'token', True, False),
    ('f32', 2, 33, None, 1, 2, 128, 64, 'token', False, True),
    ('f32', 1, 300, None, 1, 2, 64, 128, 'reset', True, False),
    ('f32', 1, 300, None, 1, 1, 128, 256, 'head', True, False),
    ('f32', 1, 0, [0, 31, 130, 1, 200], 1, 3, 128, 128, 'token', True, False),
]


@pytest.mark.parametrize('case', CASES, ids=lambda c: '-'.join(map(str, c)).replace(' ', ''))
def test_forward(case):
    say(f'linear forward {case}')
    check_fwd(*make(*case, seed=1), case[0])


@pytest.mark.parametrize('case', CASES, ids=lambda c: '-'.join(map(str, c)).replace(' ', ''))
def test_backward(case):
    say(f'linear backward {case}')
    check_bwd(*make(*case, seed=2), case[0])


def test_gradient_of_dg_against_differences():
    """FP32, a few gates moved by 2^-9: (loss(g + h) - loss(g - h)) / 2h of the GPU forward, whose own FP32
    error of 2^-22 of a loss of this size is divided by 2h; the curvature's part is h^2 / 6 of the third derivative."""
    x, d, cu = make('f32', 1, 130, None, 1, 2, 64, 64, seed=4)
    got = G.gdn_linear_bwd(d['q'], d['k'], d['v'], d['g'], d['do'], dht=d['dht'], h0=d['h0'])
    h = 2.0 ** -9

    def loss(g):
        o, ht = G.gdn_linear_fwd(d['q'], d['k'], d['v'], g, h0=d['h0'])
        a, b = o.double() * d['do'].double(), ht.double() * d['dht'].double()
        return float(a.sum() + b.sum()), float(a.abs().sum() + b.abs().sum())

    for t, hd in ((0, 0), (31, 1), (32, 0), (100, 1), (129, 0)):
        gp, gm = d['g'].clone(), d['g'].clone()
        gp[0, t, hd] += h
        gm[0, t, hd] -= h
        (lp, size), (lm, _) = loss(gp), loss(gm)
        slope = (lp - lm) / float(gp[0, t, hd].double() - gm[0, t, hd].double())
        say(f'  t {t}: {slope:.6f} and {float(got["dg"][0, t, hd]):.6f}')
        assert abs(slope - float(got['dg'][0, t, hd])) <= size * (2.0 ** -22 / h + h * h)


def test_views_write_to_given_memory_and_leave_other_tokens():
    x, d, cu = make('bf16', 1, 400, [100, 0, 150], 2, 4, 64, 128, seed=5)                # 150 tokens behind the last
    out = torch.full_like(d['v'].contiguous(), 7.0)
    check_fwd(x, d, cu, 'bf16', out=out)
    assert (out[:, 250:] == 7.0).all()
    grads = dict(dq=torch.full_like(d['q'], 7.0), dk=torch.full_like(d['k'], 7.0), dv=torch.full_like(d['v'], 7.0),
                 dg=torch.full_like(d['g'], 7.0))
    got = check_bwd(x, d, cu, 'bf16', out=grads)
    for n in grads:
        assert got[n].data_ptr() == grads[n].data_ptr() and (got[n][:, 250:] == 7.0).all(), n


def test_offsets_beyond_the_buffer_are_cut():
    x, d, _ = make('bf16', 1, 300, None, 1, 2, 64, 64, h0=False, seed=6)
    for bad, good in (([0, 50, 400], [0, 50, 300]), ([-5, 120, 2 ** 30], [0, 120, 300])):
        for cu in (bad, good):
            d['cu'] = torch.tensor(cu, dtype=torch.int32, device='cuda')
            o = torch.zeros_like(d['v'])
            _, ht = G.gdn_linear_fwd(d['q'], d['k'], d['v'], d['g'], cu_seqlens=d['cu'], out=o)
            g = G.gdn_linear_bwd(d['q'], d['k'], d['v'], d['g'], d['do'], cu_seqlens=d['cu'])
            if cu is bad:
                first = o, ht, g
        torch.cuda.synchronize()
        assert torch.equal(first[0], o) and torch.equal(first[1], ht)
        assert all(torch.equal(first[2][n], g[n]) for n in g)


def test_offsets_past_32_bits():
    stride, T = 2 ** 24 - 8, 150
    say(f'linear attention, tokens {stride} elements apart')
    x, d, cu = make('bf16', 1, T, None, 1, 1, 64, 64, seed=7)
    wide = torch.empty((T - 1) * stride + 64, dtype=torch.bfloat16, device='cuda')
    for n in ('q', 'k', 'v'):
        view = wide.as_strided((1, T, 1, 64), (T * stride, stride, 64, 1))
        view.copy_(d[n])
        d[n] = view
        if n == 'k':                                                    # one at a time is enough: 5 GB
            check_fwd(x, d, cu, 'bf16')
            check_bwd(x, d, cu, 'bf16')
        d[n] = x[n].to(torch.bfloat16).cuda()


def _bits(t):
    return t.view(torch.int16 if t.dtype is torch.bfloat16 else torch.int32)


def test_empty_calls():
    q, v = torch.zeros(2, 0, 1, 64, device='cuda'), torch.zeros(2, 0, 2, 64, device='cuda')
    h0 = torch.randn(2, 2, 64, 64, device='cuda')
    for g in (torch.zeros(2, 0, 2, device='cuda'), torch.zeros(2, device='cuda')):
        o, ht = G.gdn_linear_fwd(q, q, v, g, h0=h0)
        assert o.shape == v.shape and torch.equal(ht, h0)
        got = G.gdn_linear_bwd(q, q, v, g, v, dht=2 * h0, h0=h0)
        assert torch.equal(got['dh0'], 2 * h0) and (got['dg'] == 0).all() and got['dg'].shape == g.shape
        none = G.gdn_linear_bwd(q[:0], q[:0], v[:0], g[:0] if g.dim() == 3 else g, v[:0])
        assert (none['dg'] == 0).all()


@pytest.mark.parametrize('gate', ['token', 'head'])
def test_streams_graphs_and_repeats(gate):
    """Another stream, and a graph that is replayed, give the bits of a plain call, with eager work between the replays."""
    x, d, cu = make('bf16', 1, 0, [700, 90, 3, 400], 1, 2, 128, 64, gate=gate, seed=8)
    args = (d['q'], d['k'], d['v'], d['g'])

    def both():
        o, ht = G.gdn_linear_fwd(*args, h0=d['h0'], cu_seqlens=d['cu'])
        g = G.gdn_linear_bwd(*args, d['do'], dht=d['dht'], h0=d['h0'], cu_seqlens=d['cu'])
        return [o, ht] + [g[n] for n in ('dq', 'dk', 'dv', 'dg', 'dh0')]

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(3):
        new = make('bf16', 1, 0, [700, 90, 3, 400], 1, 2, 128, 64, gate=gate, seed=20 + i)[1]
        for n in ('q', 'k', 'v', 'g', 'do', 'h0', 'dht'):
            d[n].copy_(new[n])
        want = both()
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(want, held))


def test_states_handed_on_equal_one_run():
    """A prompt in two calls, the second from the first one's state; both within the bounds of one."""
    x, d, _ = make('bf16', 2, 333, None, 1, 2, 128, 128, seed=9)
    cut, scale = 190, 128 ** -0.5
    part = lambda n, s: d[n][:, s].contiguous()                         # noqa: E731
    o1, h1 = G.gdn_linear_fwd(*(part(n, slice(0, cut)) for n in 'qkvg'), h0=d['h0'])
    o2, h2 = G.gdn_linear_fwd(*(part(n, slice(cut, None)) for n in 'qkvg'), h0=h1)
    torch.cuda.synchronize()
    p = positive(x)
    wo, wh = linear_fwd(x['q'], x['k'], x['v'], x['g'], scale, x['h0'])
    ao, ah = linear_fwd(p['q'], p['k'], p['v'], x['g'], scale, p['h0'])
    within('o', torch.cat([o1, o2], 1), wo, ao * (U + FP32) + wo.abs() * U)
    within('ht', h2, wh, ah * (2 * U * U + FP32))


def test_growing_gates_and_long_decays():
    """Gates above 0 grow the state; a state that decays over many chunks keeps its units."""
    for level, T in ((0.04, 300), (-0.9, 600), (-3.0, 300)):
        x, d, cu = make('bf16', 1, T, None, 1, 1, 64, 64, seed=10)
        x['g'] = torch.full_like(x['g'], level)
        d['g'] = x['g'].float().cuda()
        x['g'] = d['g'].double().cpu()
        say(f'gates of {level}')
        check_fwd(x, d, cu, 'bf16')
        check_bwd(x, d, cu, 'bf16')


@pytest.mark.parametrize('bad', [math.nan, math.inf])
def test_what_is_not_finite_stays_in_its_sequence_and_heads(bad):
    _, d, cu = make('bf16', 1, 0, [37, 300, 1, 64], 2, 4, 64, 128)
    run = lambda: (G.gdn_linear_fwd(d['q'], d['k'], d['v'], d['g'], h0=d['h0'], cu_seqlens=d['cu']),     # noqa: E731
                   G.gdn_linear_bwd(d['q'], d['k'], d['v'], d['g'], d['do'], d['dht'], h0=d['h0'], cu_seqlens=d['cu']))
    (o, ht), grads = run()
    for name in ('q', 'k', 'v', 'do'):
        d[name][:, cu[1]:cu[2], 0] = bad                                # sequence 1, first head
    d['h0'][1, 0] = d['dht'][1, 0] = bad
    (o1, ht1), grads1 = run()
    here = torch.zeros(cu[-1], 4, dtype=torch.bool)
    here[cu[1]:cu[2], :2] = True                                        # the value heads of its group
    rest = ~here.cuda()
    assert torch.equal(_bits(o[0][rest]), _bits(o1[0][rest])) and torch.isnan(o1[0, cu[1]:cu[2], 0]).any()
    for n in ('dv', 'dg'):
        assert torch.equal(_bits(grads[n][0][rest]), _bits(grads1[n][0][rest])), n
    for n in ('dq', 'dk'):
        assert torch.equal(_bits(grads[n][0][rest[:, ::2]]), _bits(grads1[n][0][rest[:, ::2]])), n
    keep = torch.ones(4, 4, dtype=torch.bool, device='cuda')
    keep[1, :2] = False
    for a, b in ((ht, ht1), (grads['dh0'], grads1['dh0'])):
        assert torch.equal(a[keep], b[keep])


def test_outputs_in_the_inputs_memory_are_refused():
    _, d, _ = make('bf16', 1, 70, None, 2, 2, 64, 64)
    for name in ('q', 'v'):
        with pytest.raises(G.GdnError, match='o overlaps ' + name):
            G.gdn_linear_fwd(d['q'], d['k'], d['v'], d['g'], out=d[name])
    out = dict(dq=torch.empty_like(d['q']), dk=torch.empty_like(d['k']), dv=d['do'], dg=torch.empty_like(d['g']))
    with pytest.raises(G.GdnError, match='dv overlaps do'):
        G.gdn_linear_bwd(d['q'], d['k'], d['v'], d['g'], d['do'], out=out)


@pytest.mark.parametrize('gate', ['slow', 'reset', 'head'])
@pytest.mark.parametrize('T', [1024, 1025, 2208])
def test_dg_of_long_segments(gate, T):
    """32, 33 and 69 chunks in one segment: 256 equal heads fill the device, so sequences
    stay whole. Bound: a product passes fewer than 2,300 sums of 2^-24 each, 2^-12.8, and
    two split factors, 2^-15: under 2^-12 of the suffix sum of the absolute dots."""
    H = 256
    x, d, _ = make('bf16', 1, T, None, 1, 1, 64, 64, gate if gate != 'slow' else 'token', seed=11)
    if gate == 'slow':
        x['g'] = x['g'].float().mul(2.0 ** -8).double()
    else:
        x['g'] = x['g'].float().double()
    g = x['g'].float().cuda()
    wide = {n: d[n].repeat_interleave(H, 1 if n in ('h0', 'dht') else 2) for n in ('q', 'k', 'v', 'do', 'h0', 'dht')}
    g = g.repeat_interleave(H, g.dim() - 1)
    got = G.gdn_linear_bwd(wide['q'], wide['k'], wide['v'], g, wide['do'], wide['dht'], h0=wide['h0'])['dg']
    scale = 64 ** -0.5
    want = linear_bwd(x['q'], x['k'], x['v'], x['g'], scale, x['do'], x['dht'], x['h0'])['dg']
    mag = positive(x)
    top = linear_bwd(mag['q'], mag['k'], mag['v'], mag['g'], scale, mag['do'], mag['dht'], mag['h0'])
    dots = sum((mag[n] * top['d' + n]).sum(-1) for n in ('q', 'k'))
    sums = dots.flip(1).cumsum(1).flip(1)
    bound = (sums.sum((0, 1)) if gate == 'head' else sums + top['dg'].abs()) * 2.0 ** -12 + 1e-30
    assert torch.equal(got, got[..., :1].expand_as(got))                # equal heads, equal bits
    within('dg', got[..., -1:], want, bound)
