"""State pool on the GPU: pages in and out, copies, reordering, the recurrent
step and a generation with beams, through the binding, against 64-bit
references (the quantizer's reference is oracle/qdq.py).

Tolerances, from the arithmetic: pages in and out are bit-exact to the FP32
quantizer, copies and reorderings move bytes. The step is FP32: a sum over Dk
keys of terms t_i is off by at most (Dk + 4) 2^-24 sum |t_i| (any order, one
rounding per product, sum and scale), so every output and state element is
bounded by that many roundings of the sums of absolute values, which the
reference carries along; a bf16 output adds half a step, 2^-8 relative. A code
may differ from the reference's only where the FP32 value is that close to
the border between two codes; scales are amax / q_max and carry the state's
bound."""
import math

import numpy as np
import pytest
import torch

from gateddeltanet_chunked_recurrence_amd import binding as B
from oracle.decode import prefill_decode_fwd
from oracle.qdq import qdq32
from parity_util import code_bytes, rel, say

pytestmark = pytest.mark.gpu

OFF, E4M3, INT8 = B.QDQ_OFF, B.QDQ_E4M3, B.QDQ_INT8
BEFORE, AFTER = B.READOUT_BEFORE_WRITE, B.READOUT_AFTER_WRITE
U = 2.0 ** -24


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device='cuda')


def _bits(t):
    return t.contiguous().view(torch.uint8) if t.element_size() == 1 else t.contiguous().view(torch.int32)


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


def _snapshot(pool):
    return pool.data.clone(), None if pool.scales is None else pool.scales.clone()


def _pool_same(pool, snap, slots=None):
    """Whether the pages (of `slots`, or all) are those of the snapshot."""
    at = slice(None) if slots is None else torch.tensor(slots, dtype=torch.long, device='cuda')
    ok = torch.equal(_bits(pool.data)[:, at], _bits(snap[0])[:, at])
    return ok and (pool.scales is None or torch.equal(pool.scales[:, at], snap[1][:, at]))


def _random_pool(fmt, L, S, Hv, Dk, Dv, bv, seed=0):
    gen = torch.Generator(device='cuda').manual_seed(seed)
    pool = B.StatePool(L, S, Hv, Dk, Dv, fmt, bv)
    for layer in range(L):
        x = torch.randn(S, Hv, Dk, Dv, generator=gen, device='cuda')
        x *= 0.1 * torch.exp(torch.randn(S, Hv, 1, 1, generator=gen, device='cuda'))
        B.gdn_pool_write(pool, layer, _ints(list(range(S))), x)
    torch.cuda.synchronize()
    return pool


def _values(pool):
    """FP64 states [layers, slots, Hv, Dk, Dv] of the pages, on the CPU."""
    x = pool.data.double().cpu()
    if pool.scales is not None:
        x = x * pool.scales.double().cpu().repeat_interleave(pool.block_v, -1).unsqueeze(-1)
    return x.transpose(-1, -2)


# ------------------------------------------------------------- pages in and out
PAGES = [(E4M3, 128, 128, 64), (INT8, 128, 128, 64), (E4M3, 64, 64, 16), (INT8, 64, 256, 32),
         (E4M3, 128, 256, 128), (INT8, 64, 256, 256), (E4M3, 128, 256, 16), (E4M3, 64, 128, 32),
         (INT8, 128, 64, 16), (OFF, 64, 64, 64), (OFF, 128, 256, 64), (OFF, 128, 64, 64)]


@pytest.mark.parametrize("fmt,Dk,Dv,bv", PAGES)
def test_write_and_read_are_exact(fmt, Dk, Dv, bv):
    say(f"pool write/read fmt={fmt} Dk={Dk} Dv={Dv} block_v={bv}")
    rng = np.random.default_rng(Dk + 3 * Dv + bv + fmt)
    n, Hv, S = 9, 3, 13
    x = rng.standard_normal((n, Hv, Dk, Dv)).astype(np.float32)
    x[0] = 0.0                                            # zero tiles
    x[1] = -0.0
    x[2] *= np.float32(1e-39)                             # subnormal values
    x[3] = x[3] ** 3 * np.float32(1e4)
    # exact ties on the code grid: amax = q_max 8, so that d = 8
    top = 448.0 if fmt == E4M3 else 127.0
    mids = np.array([2.0 ** -10, 3 * 2.0 ** -10, 0.5625, 1.0625, 14.5, 232.0, 432.0], np.float32) \
        if fmt == E4M3 else np.array([0.5, 1.5, 2.5, 100.5, 126.5], np.float32)
    x[4] = np.resize(mids, (Hv, Dk, Dv)) * 8 * np.where(rng.random((Hv, Dk, Dv)) < 0.5, -1, 1)
    x[4, :, 0, :] = top * 8
    pool = _random_pool(fmt, 2, S, Hv, Dk, Dv, bv)
    snap = _snapshot(pool)
    slots = [4, 0, 12, 7, 3, -1, 9, 1, 5]
    B.gdn_pool_write(pool, 1, _ints(slots), torch.from_numpy(x).cuda())
    got = B.gdn_pool_read(pool, 1, _ints(slots)).cpu().numpy()
    torch.cuda.synchronize()
    assert B.device_errors() == 0
    untouched = [s for s in range(S) if s not in slots]
    assert _pool_same(pool, snap, untouched) and torch.equal(_bits(pool.data)[0], _bits(snap[0])[0])
    if fmt == OFF:
        want = x.copy()
    else:
        want, c, d = qdq32(x.reshape(n, Hv, Dk, Dv // bv, bv), fmt, (2, 4))
        want = want.reshape(x.shape)
        if fmt == INT8:
            want = want + np.float32(0)                   # an integer code has one zero: -0 is read as +0
        codes = code_bytes(c.reshape(x.shape), fmt)
    want[5] = 0.0                                         # the absent slot reads as the zero state
    np.testing.assert_array_equal(got.view(np.uint32), want.view(np.uint32))
    if fmt != OFF:
        page = pool.data.view(torch.uint8)[1].cpu().numpy()
        sc = pool.scales[1].cpu().numpy()
        for i, s in enumerate(slots):
            if s >= 0:
                np.testing.assert_array_equal(page[s], codes[i].transpose(0, 2, 1))
                np.testing.assert_array_equal(sc[s], d[i].reshape(Hv, Dv // bv))


def test_write_equals_the_standalone_quantizer():
    x = torch.randn(5, 4, 128, 128, device='cuda') * 3
    pool = B.StatePool(1, 5, 4, 128, 128, E4M3, 32)
    B.gdn_pool_write(pool, 0, _ints([0, 1, 2, 3, 4]), x)
    y, scales, codes = B.gdn_qdq_state(x.view(20, 128, 128), E4M3, 32, return_codes=True)
    assert torch.equal(pool.data.view(torch.uint8)[0], codes.view(5, 4, 128, 128).mT)
    assert torch.equal(pool.scales[0], scales.view(5, 4, 4))
    assert torch.equal(B.gdn_pool_read(pool, 0, _ints([0, 1, 2, 3, 4])), y.view(5, 4, 128, 128))


@pytest.mark.parametrize("fmt,qmax", [(E4M3, 448.0), (INT8, 127.0)])
def test_reciprocal_scales_are_those_of_pytorch(fmt, qmax):
    """SCALE_RECIPROCAL: the bits of a state quantized in PyTorch on the GPU,
    whose division of a tensor by a number is a product with its reciprocal."""
    x = torch.randn(40, 3, 64, 128, device='cuda') * torch.rand(40, 3, 1, 1, device='cuda')
    pool = B.StatePool(1, 40, 3, 64, 128, fmt, 16, scale_rule=B.SCALE_RECIPROCAL)
    B.gdn_pool_write(pool, 0, _ints(list(range(40))), x)
    t = x.mT.reshape(40, 3, 8, 16 * 64)
    amax = t.abs().amax(-1)
    d = amax * torch.tensor(1.0 / qmax, device='cuda')
    assert torch.equal(pool.scales[0], d) and torch.equal(d, amax / qmax)
    y = t * (1.0 / d).unsqueeze(-1)
    c = y.clamp(-448, 448).to(torch.float8_e4m3fn) if fmt == E4M3 else y.round().clamp(-127, 127).to(torch.int8)
    assert _same(pool.data[0], c.view(40, 3, 128, 64))
    other = B.StatePool(1, 40, 3, 64, 128, fmt, 16)
    B.gdn_pool_write(other, 0, _ints(list(range(40))), x)
    assert float(((other.scales - pool.scales).abs() / other.scales).max()) <= 2.0 ** -22
    # the step writes by the same rule: scales of the two pools differ by at most the rounding
    z = _draw(40, 1, 1, 3, 64, 128, torch.bfloat16, seed=40)
    again = B.StatePool.from_tensors(pool.data.clone(), pool.scales.clone(), fmt, 16)
    B.gdn_pool_step(pool, 0, _ints(list(range(40))), **z)
    B.gdn_pool_step(again, 0, _ints(list(range(40))), **z)
    off = (again.scales - pool.scales).abs() / again.scales
    assert 0 < float(off.max()) <= 2.0 ** -22


@pytest.mark.parametrize("fmt", [E4M3, OFF])
def test_write_refuses_bad_slots(fmt):
    pool = _random_pool(fmt, 1, 6, 2, 64, 64, 64)
    snap = _snapshot(pool)
    x = torch.randn(6, 2, 64, 64, device='cuda')
    B.gdn_pool_write(pool, 0, _ints([3, 1, 3, 6, -2, 4]), x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert _pool_same(pool, snap, [0, 2, 3, 5])
    want = B.StatePool(1, 6, 2, 64, 64, fmt, 64)
    B.gdn_pool_write(want, 0, _ints([-1, 1, -1, -1, -1, 4]), x)
    assert _pool_same(pool, (want.data, want.scales), [1, 4])
    got = B.gdn_pool_read(pool, 0, _ints([6, 0, -1]))
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert bool(got[0].isnan().all()) and bool((got[2] == 0).all())
    assert torch.equal(got[1].double().cpu(), _values(pool)[0, 0].float().double())


# ------------------------------------------------------------------- the step
def _draw(Bn, T, Hqk, Hv, Dk, Dv, dt, seed):
    gen = torch.Generator(device='cuda').manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device='cuda')  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(Bn, T, Hqk, Dk), dim=-1).to(dt) for _ in range(2))
    return dict(q=q, k=k, v=r(Bn, T, Hv, Dv).to(dt), g=-torch.nn.functional.softplus(r(Bn, T, Hv)),
                beta=torch.sigmoid(r(Bn, T, Hv)))


def _reference(pool, S, x, n, scale):
    """One token of sequence n in FP64 from states S [Hv, Dk, Dv]: the updated
    state and output before the write, and bounds of their FP32 errors."""
    q, k, v, g, beta = (x[i][n, 0].double().cpu() for i in ('q', 'k', 'v', 'g', 'beta'))
    G = pool.Hv // q.shape[0]
    q, k = q.repeat_interleave(G, 0), k.repeat_interleave(G, 0)
    c = (pool.Dk + 4) * U
    A = torch.exp(g)[:, None, None] * S
    aA = A.abs()
    p = (A * k.unsqueeze(-1)).sum(1)
    ap = (aA * k.abs().unsqueeze(-1)).sum(1)
    u = beta.unsqueeze(-1) * (v - p)
    eu = beta.unsqueeze(-1) * (c * ap + 3 * U * (v.abs() + p.abs()))
    S1 = A + k.unsqueeze(-1) * u.unsqueeze(1)
    eS = 6 * U * aA + k.abs().unsqueeze(-1) * (eu + 3 * U * u.abs()).unsqueeze(1)
    o = scale * (S1 * q.unsqueeze(-1)).sum(1)
    aq = (aA * q.abs().unsqueeze(-1)).sum(1)
    kq = (k * q).abs().sum(1, keepdim=True)
    eo = scale * (c * aq + kq * (eu + c * u.abs()) + 6 * U * (aq + kq * u.abs()))
    return S1, eS, o, eo, q


STEPS = [(E4M3, torch.bfloat16, 128, 128, 64, 2, 4, BEFORE), (E4M3, torch.bfloat16, 128, 128, 64, 4, 4, AFTER),
         (INT8, torch.bfloat16, 128, 256, 128, 1, 3, AFTER), (INT8, torch.float32, 64, 64, 16, 2, 2, BEFORE),
         (E4M3, torch.float32, 64, 256, 256, 1, 2, AFTER), (E4M3, torch.bfloat16, 64, 128, 32, 1, 5, BEFORE),
         (E4M3, torch.bfloat16, 128, 256, 256, 3, 3, BEFORE), (INT8, torch.bfloat16, 128, 64, 16, 1, 1, AFTER),
         (OFF, torch.float32, 64, 64, 64, 1, 3, BEFORE), (OFF, torch.bfloat16, 128, 256, 64, 2, 4, AFTER),
         (OFF, torch.float32, 128, 128, 64, 1, 1, AFTER)]


def _check_step(pool, before, after_codes, after_scales, x, o, n, to, scale, readout):
    """Sequence n's page and output after one token, from the state `before`."""
    S1, eS, o_ref, eo, q = _reference(pool, before, x, n, scale)
    if pool.state_fmt == OFF:
        err = (after_codes.double().cpu().transpose(-1, -2) - S1).abs()
        assert bool((err <= eS + U * S1.abs() + 1e-40).all()), float((err / (eS + 1e-40)).max())
        kept = S1
    else:
        fmt, bv, Hv = pool.state_fmt, pool.block_v, pool.Hv
        qmax = 448.0 if fmt == E4M3 else 127.0
        T1 = S1.float().numpy().reshape(Hv, pool.Dk, pool.Dv // bv, bv)
        _, c, d = qdq32(T1, fmt, (1, 3))
        c = torch.from_numpy(c.reshape(S1.shape)).double()
        d = torch.from_numpy(d.reshape(Hv, -1)).double()
        got_d = after_scales.double().cpu()
        ed = eS.reshape(Hv, pool.Dk, -1, bv).amax((1, 3)) / qmax + 2 * U * d
        assert bool(((got_d - d).abs() <= ed).all())
        got_c = after_codes.double().cpu().transpose(-1, -2)
        # a differing code: the value lies within the bound of the border between the two
        dd = d.repeat_interleave(bv, -1).unsqueeze(1)
        edd = ed.repeat_interleave(bv, -1).unsqueeze(1)
        y = S1 / dd
        ey = eS / dd + y.abs() * (edd / dd + 4 * U)
        off = got_c != c
        border = (got_c + c) / 2
        assert bool(((y - border).abs() <= ey)[off].all())
        say(f"  seq {n}: {int(off.sum())} of {off.numel()} codes on the other side of a border")
        kept = got_c * got_d.repeat_interleave(bv, -1).unsqueeze(1)
    if readout == AFTER and pool.state_fmt != OFF:
        o_ref = scale * (kept * q.unsqueeze(-1)).sum(1)
        eo = scale * (pool.Dk + 6) * U * (kept.abs() * q.abs().unsqueeze(-1)).sum(1)
    elif readout == AFTER:
        eo = eo + scale * ((eS * q.abs().unsqueeze(-1)).sum(1) + (pool.Dk + 6) * U * (S1.abs() * q.abs().unsqueeze(-1)).sum(1))
    half = 2.0 ** -8 if o.dtype == torch.bfloat16 else U
    err = (o.double().cpu() - o_ref).abs()
    assert bool((err <= (1 + half) * eo + half * o_ref.abs() + 1e-38).all()), float(err.max())


@pytest.mark.parametrize("fmt,dt,Dk,Dv,bv,Hqk,Hv,readout", STEPS)
def test_one_token_against_fp64(fmt, dt, Dk, Dv, bv, Hqk, Hv, readout):
    say(f"pool step fmt={fmt} {dt} Dk={Dk} Dv={Dv} block_v={bv} heads {Hqk}x{Hv} readout {readout}")
    Bn = 4
    pool = _random_pool(fmt, 2, 7, Hv, Dk, Dv, bv, seed=3)
    snap = _snapshot(pool)
    S = _values(pool)[1]
    x = _draw(Bn, 1, Hqk, Hv, Dk, Dv, dt, seed=Dk + Dv + bv)
    x['g'][3] = -120.0                                   # a gate that forgets everything
    slots, scale = [5, 0, -1, 2], 0.37
    out = torch.full((Bn, 1, Hv, Dv), 7.0, dtype=dt, device='cuda')
    o = B.gdn_pool_step(pool, 1, _ints(slots), scale=scale, readout=readout, out=out, **x)
    assert B.device_errors() == 0 and o is out
    assert bool((o[2] == 7.0).all())
    assert _pool_same(pool, snap, [1, 3, 4, 6]) and torch.equal(_bits(pool.data)[0], _bits(snap[0])[0])
    for n, s in enumerate(slots):
        if s >= 0:
            _check_step(pool, S[s], pool.data[1, s], None if fmt == OFF else pool.scales[1, s], x, o[n, 0], n, s,
                        scale, readout)


@pytest.mark.parametrize("fmt,dt,Dk,Dv,bv", [(E4M3, torch.bfloat16, 128, 128, 64), (INT8, torch.bfloat16, 64, 256, 256),
                                             (E4M3, torch.bfloat16, 128, 256, 128), (OFF, torch.float32, 64, 128, 64),
                                             (INT8, torch.float32, 64, 64, 16)])
@pytest.mark.parametrize("readout", [BEFORE, AFTER])
def test_many_tokens_equal_single_ones(fmt, dt, Dk, Dv, bv, readout):
    """T tokens in one call are the same bits as T calls; sequences end at
    their own length, and rows past it keep what they held."""
    Bn, T, Hqk, Hv = 5, 9, 2, 4
    many = _random_pool(fmt, 1, 6, Hv, Dk, Dv, bv, seed=4)
    one = _random_pool(fmt, 1, 6, Hv, Dk, Dv, bv, seed=4)
    x = _draw(Bn, T, Hqk, Hv, Dk, Dv, dt, seed=5)
    slots, lens = [3, 0, 5, -1, 1], [9, 4, 0, 6, 13]      # 13 is cut to T
    out = torch.full((Bn, T, Hv, Dv), 7.0, dtype=dt, device='cuda')
    B.gdn_pool_step(many, 0, _ints(slots), lens=_ints(lens), readout=readout, out=out, **x)
    for t in range(T):
        live = [s if t < n else -1 for s, n in zip(slots, lens)]
        got = torch.full((Bn, 1, Hv, Dv), 7.0, dtype=dt, device='cuda')
        B.gdn_pool_step(one, 0, _ints(live), readout=readout, out=got,
                        **{k: v[:, t:t + 1].contiguous() for k, v in x.items()})
        assert torch.equal(out[:, t], got[:, 0]), t
    assert _pool_same(many, _snapshot(one)) and B.device_errors() == 0


@pytest.mark.parametrize("fmt", [E4M3, INT8, OFF])
def test_children_read_their_parents(fmt):
    """slots_out: the same results as a copy of the parent's page followed by
    a step in place; parents stay, -1 keeps nothing, length 0 only copies."""
    Bn, T, Hv, Dk, Dv = 6, 2, 3, 128, 128
    fork = _random_pool(fmt, 2, 12, Hv, Dk, Dv, 64, seed=6)
    flat = _random_pool(fmt, 2, 12, Hv, Dk, Dv, 64, seed=6)
    snap = _snapshot(fork)
    x = _draw(Bn, T, 1, Hv, Dk, Dv, torch.bfloat16, seed=7)
    src, dst, lens = [4, 4, 0, 2, -1, 7], [9, 1, 3, -1, 11, 10], [2, 1, 2, 2, 2, 0]
    o = B.gdn_pool_step(fork, 1, _ints(src), slots_out=_ints(dst), lens=_ints(lens), **x)
    B.gdn_pool_copy(flat, _ints([4, 4, 0, 7]), _ints([9, 1, 3, 10]))
    flat.data[0].view(torch.uint8).copy_(snap[0][0].view(torch.uint8))
    if fmt != OFF:
        flat.scales[0].copy_(snap[1][0])
    o2 = B.gdn_pool_step(flat, 1, _ints([9, 1, 3, -1, -1, 10]), lens=_ints(lens), **x)
    peek = B.gdn_pool_step(flat, 1, _ints([-1, -1, -1, 2, -1, -1]), slots_out=_ints([-1] * 6), **x)
    assert B.device_errors() == 0
    assert torch.equal(o[[0, 1, 2, 5]], o2[[0, 1, 2, 5]]) and torch.equal(o[3], peek[3])
    assert bool((o[4] == 0).all()) and _pool_same(fork, _snapshot(flat))


def test_token_views_of_a_wider_projection():
    Bn, T, Hqk, Hv, D = 3, 4, 2, 4, 64
    x = _draw(Bn, T, Hqk, Hv, D, D, torch.bfloat16, seed=8)
    wide = torch.full((Bn, T, 2 * Hqk * D + Hv * D + 24), float('nan'), dtype=torch.bfloat16, device='cuda')
    nq = Hqk * D
    wide[..., :nq] = x['q'].flatten(2)
    wide[..., nq:2 * nq] = x['k'].flatten(2)
    wide[..., 2 * nq:2 * nq + Hv * D] = x['v'].flatten(2)
    view = dict(q=wide[..., :nq].unflatten(2, (Hqk, D)), k=wide[..., nq:2 * nq].unflatten(2, (Hqk, D)),
                v=wide[..., 2 * nq:2 * nq + Hv * D].unflatten(2, (Hv, D)), g=x['g'], beta=x['beta'])
    a, b = (_random_pool(E4M3, 1, 3, Hv, D, D, 32, seed=9) for _ in range(2))
    o1 = B.gdn_pool_step(a, 0, _ints([0, 1, 2]), **x)
    o2 = B.gdn_pool_step(b, 0, _ints([0, 1, 2]), **view)
    assert torch.equal(o1, o2) and _pool_same(a, _snapshot(b))
    last = {k: v[:, 3:4] if k in 'qkv' else v[:, 3:4].contiguous() for k, v in view.items()}
    o3 = B.gdn_pool_step(a, 0, _ints([0, 1, 2]), **{k: v.contiguous() for k, v in last.items()})
    assert torch.equal(o3, B.gdn_pool_step(b, 0, _ints([0, 1, 2]), **last))


@pytest.mark.parametrize("fmt,bv", [(E4M3, 64), (INT8, 16), (E4M3, 128), (OFF, 64)])
def test_step_refuses_bad_slots(fmt, bv):
    Bn, Hv, D = 9, 2, 128
    pool, want = (_random_pool(fmt, 1, 8, Hv, D, D, bv, seed=10) for _ in range(2))
    snap = _snapshot(pool)
    x = _draw(Bn, 1, 1, Hv, D, D, torch.bfloat16, seed=11)
    # 2 twice, 8 and -5 outside the pool, the others fine
    slots = [2, 0, 2, 8, 5, -5, -1, 7, 6]
    o = B.gdn_pool_step(pool, 0, _ints(slots), **x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert bool(o[[0, 2, 3, 5]].isnan().all()) and bool((o[6] == 0).all())
    good = [-1, 0, -1, -1, 5, -1, -1, 7, 6]
    o2 = B.gdn_pool_step(want, 0, _ints(good), **x)
    assert torch.equal(o[[1, 4, 7, 8]], o2[[1, 4, 7, 8]]) and _pool_same(pool, _snapshot(want))
    assert _pool_same(pool, snap, [1, 2, 3, 4])
    # a page written while another sequence reads it; two children on one page; a child outside the pool
    snap = _snapshot(pool)
    src, dst = [0, 1, 2, 3, 4, 5, -1, -1, -1], [1, 7, 6, 6, 8, -1, 6, 6, 7]
    o = B.gdn_pool_step(pool, 0, _ints(src), slots_out=_ints(dst), **x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert bool(o[[0, 2, 3, 4]].isnan().all()) and bool(o[[1, 5]].isfinite().all())
    assert _pool_same(pool, snap, [0, 1, 2, 3, 4, 5, 6])
    # the same answer where the entries are many (another wave finds the conflict)
    n = 300
    big = _random_pool(fmt, 1, n, 1, 64, 64, 16, seed=12)
    snap = _snapshot(big)
    x = _draw(n, 1, 1, 1, 64, 64, torch.bfloat16, seed=13)
    slots = list(range(n))
    slots[299] = 1
    o = B.gdn_pool_step(big, 0, _ints(slots), **x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert bool(o[[1, 299]].isnan().all()) and not bool(o[2:299].isnan().any())
    assert _pool_same(big, snap, [1, 299]) and not _pool_same(big, snap, [0])


@pytest.mark.parametrize("fmt,bv,lens", [(E4M3, 64, False), (INT8, 128, True), (OFF, 64, False)])
def test_step_refuses_to_write_a_page_that_another_only_reads(fmt, bv, lens):
    """slots_out -1 keeps no state, but its page is read all the same."""
    Hv, D = 2, 128
    pool, want = (_random_pool(fmt, 1, 8, Hv, D, D, bv, seed=14) for _ in range(2))
    snap = _snapshot(pool)
    x = _draw(5, 1, 1, Hv, D, D, torch.bfloat16, seed=15)
    n = dict(lens=_ints([1] * 5)) if lens else {}
    # 1 is read by entry 1 and would be written by entry 0; 3 is read by entries 2 and 4, not written
    o = B.gdn_pool_step(pool, 0, _ints([0, 1, 3, 5, 3]), slots_out=_ints([1, -1, -1, 5, -1]), **n, **x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    o2 = B.gdn_pool_step(want, 0, _ints([-1, 1, 3, 5, 3]), slots_out=_ints([-1, -1, -1, 5, -1]), **n, **x)
    assert B.device_errors() == 0
    assert bool(o[0].isnan().all()) and torch.equal(o[1:], o2[1:])
    assert _pool_same(pool, _snapshot(want)) and _pool_same(pool, snap, [0, 1, 2, 3, 4, 6, 7])


# ------------------------------------------------------------- page moves
MOVES = [(E4M3, 3, 4, 128, 128, 64), (INT8, 2, 3, 64, 64, 16), (OFF, 1, 1, 64, 64, 64), (E4M3, 1, 5, 128, 256, 256),
         (OFF, 2, 2, 128, 64, 64), (E4M3, 1, 1, 64, 64, 64)]


@pytest.mark.parametrize("fmt,L,Hv,Dk,Dv,bv", MOVES)
def test_copies(fmt, L, Hv, Dk, Dv, bv):
    pool = _random_pool(fmt, L, 12, Hv, Dk, Dv, bv, seed=14)
    data, scales = _snapshot(pool)
    B.gdn_pool_copy(pool, _ints([3, 3, 0, -1, 5, 8, 9]), _ints([1, 7, 2, 4, -1, 8, 11]))
    assert B.device_errors() == 0
    want = {1: 3, 7: 3, 2: 0, 11: 9}
    for s in range(12):
        if s == 4:
            assert bool((pool.data[:, 4].float() == 0).all())
            assert pool.scales is None or bool((pool.scales[:, 4] == 2.0 ** -126).all())
            continue
        assert _same(pool.data[:, s], data[:, want.get(s, s)]), s
        assert scales is None or torch.equal(pool.scales[:, s], scales[:, want.get(s, s)]), s


def test_copy_refuses_bad_slots():
    pool = _random_pool(E4M3, 2, 10, 2, 64, 64, 64, seed=15)
    snap = _snapshot(pool)
    # 1 twice; 4 is another entry's source; 10, -2 and -3 are no slots; the move to 8 is fine
    B.gdn_pool_copy(pool, _ints([0, 2, 3, 4, 10, 5, -2, 6]), _ints([1, 1, 4, 5, 7, 10, 9, 8]))
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert _pool_same(pool, snap, [0, 1, 2, 3, 4, 6, 7, 9])
    assert _same(pool.data[:, 8], snap[0][:, 6]) and not _same(pool.data[:, 8], snap[0][:, 8])


@pytest.mark.parametrize("fmt,L,Hv,Dk,Dv,bv", MOVES)
@pytest.mark.parametrize("G,W", [(1, 2), (3, 4), (5, 3), (2, 8), (1, 11), (2, 16), (1, 32), (2, 19), (4, 1)])
def test_reorder_is_simultaneous(fmt, L, Hv, Dk, Dv, bv, G, W):
    gen = torch.Generator().manual_seed(G * 100 + W)
    n = G * W + 2
    pool = _random_pool(fmt, L, n, Hv, Dk, Dv, bv, seed=16)
    data, scales = _snapshot(pool)
    slots = torch.randperm(n, generator=gen)[:G * W].view(G, W)
    parents = torch.randint(0, W, (G, W), generator=gen)
    parents[0] = torch.arange(W).roll(1)                  # one cycle through every beam
    if W > 2:
        parents[-1, 1], slots[-1, 2] = -1, -1             # a beam that stays, one that is not there
        parents[-1][parents[-1] == 2] = 0
    B.gdn_pool_reorder(pool, slots.int().cuda(), parents.int().cuda())
    assert B.device_errors() == 0
    want = list(range(n))
    for g in range(G):
        for w in range(W):
            if slots[g, w] >= 0 and parents[g, w] >= 0:
                want[slots[g, w]] = int(slots[g, parents[g, w]])
    assert _same(pool.data, data[:, want].contiguous() if fmt == OFF else
                 data.view(torch.uint8)[:, want].view(data.dtype))
    assert scales is None or torch.equal(pool.scales, scales[:, want])


def test_reorder_refuses_bad_entries():
    pool = _random_pool(INT8, 1, 12, 2, 64, 64, 64, seed=17)
    snap = _snapshot(pool)
    slots = [[0, 1, 2, 3], [4, 5, 1, 6], [7, -1, 12, 8]]
    parents = [[1, 0, 2, 4], [1, 0, 3, 2], [1, 0, 0, 2]]
    # group 0: 0 <- 1 fine, 1 is named twice, 3 has parent 4; group 1: 4 <-> 5, 1 again, 6 <- 1 fine;
    # group 2: 7 takes an absent beam, 12 is no slot, 8 takes slot 12
    B.gdn_pool_reorder(pool, _ints(slots), _ints(parents))
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    want = {0: 1, 4: 5, 5: 4, 6: 1}
    for s in range(12):
        assert _same(pool.data[:, s], snap[0][:, want.get(s, s)]), s


def test_pages_beyond_32_bit_offsets():
    """Slots and layers whose bytes start past 2^32 (and 2^33 with FP32)."""
    for fmt, slots in ((E4M3, 9000), (OFF, 4500)):
        Hv, D = 32, 128                                    # pages of 512 KB and 2 MB
        pool = B.StatePool(1, slots, Hv, D, D, fmt, 64)
        assert pool.data.numel() * pool.data.element_size() > 2 ** 32
        last = slots - 1
        x = torch.randn(2, Hv, D, D, device='cuda')
        B.gdn_pool_write(pool, 0, _ints([last, 0]), x)
        small = B.StatePool(1, 4, Hv, D, D, fmt, 64)
        B.gdn_pool_write(small, 0, _ints([3, 0]), x)
        t = _draw(2, 1, 4, Hv, D, D, torch.bfloat16, seed=18)
        a = B.gdn_pool_step(pool, 0, _ints([last, 0]), slots_out=_ints([last - 1, 1]), **t)
        b = B.gdn_pool_step(small, 0, _ints([3, 0]), slots_out=_ints([2, 1]), **t)
        assert torch.equal(a, b)
        B.gdn_pool_copy(pool, _ints([last - 1]), _ints([2]))
        B.gdn_pool_reorder(pool, _ints([[last, 0]]), _ints([[1, 0]]))
        B.gdn_pool_reorder(small, _ints([[3, 0]]), _ints([[1, 0]]))
        for s, w in ((last, 3), (last - 1, 2), (0, 0), (1, 1), (2, 2)):
            assert _same(pool.data[0, s], small.data[0, w]), (fmt, s)
        got = B.gdn_pool_read(pool, 0, _ints([last, 0, last - 1]))
        assert torch.equal(got, B.gdn_pool_read(small, 0, _ints([3, 0, 2])))
        assert B.device_errors() == 0
        del pool
        torch.cuda.empty_cache()


# ------------------------------------------------------------- used together
def test_prefill_then_steps_follow_the_decode_path():
    """gdn_pool_prefill and single-token steps against the decode continuation
    (gdn_prefill_decode_fwd and its FP64 oracle): the same written states up
    to codes next to a border. Bars as for that path: rel-L2 1e-2 with the
    quantizer on, and 1e-5 on the states (3e-3 on bf16 outputs) with it off."""
    for fmt, bv in ((E4M3, 64), (INT8, 32), (OFF, 64)):
        N, T, P, Hqk, Hv, D = 2, 76, 70, 1, 2, 128
        x = _draw(N, T, Hqk, Hv, D, D, torch.bfloat16, seed=19)
        pool = B.StatePool(2, 6, Hv, D, D, fmt, bv)
        slots, scale = _ints([4, 1]), D ** -0.5
        head = {k: v[:, :P].contiguous() for k, v in x.items()}
        o = [B.gdn_pool_prefill(pool, 1, slots, head['q'], head['k'], head['v'], head['g'], head['beta'])]
        for t in range(P, T):
            o.append(B.gdn_pool_step(pool, 1, slots, **{k: v[:, t:t + 1].contiguous() for k, v in x.items()}))
        o = torch.cat(o, 1)
        cpu = [x[k].double().cpu() for k in ('q', 'k', 'v', 'g', 'beta')]
        o_ref, ht_ref = prefill_decode_fwd(*cpu, scale, P, None, None, state_fmt=fmt, w_fmt=OFF, block_v=bv,
                                           readout=BEFORE)[:2]
        o_dec, ht_dec, _ = B.gdn_prefill_decode_fwd(x['q'], x['k'], x['v'], x['g'], x['beta'], P, state_fmt=fmt,
                                                    block_v=bv)
        ht = B.gdn_pool_read(pool, 1, slots)
        r = rel(o, o_ref), rel(ht, ht_ref), rel(o, o_dec), rel(ht, ht_dec)
        say(f"  fmt {fmt}: rel-L2 vs FP64 o {r[0]:.2e} state {r[1]:.2e}; vs the decode path {r[2]:.2e} {r[3]:.2e}")
        assert r[0] <= (3e-3 if fmt == OFF else 1e-2) and r[1] <= (1e-5 if fmt == OFF else 1e-2)
        assert r[2] <= (3e-3 if fmt == OFF else 1e-2) and r[3] <= (1e-5 if fmt == OFF else 1e-2)
        # resumed from its pages, a second prefill is the chunk forward from those states
        again = B.gdn_pool_prefill(pool, 1, slots, head['q'], head['k'], head['v'], head['g'], head['beta'])
        want, want_ht, _ = B.gdn_chunk_fwd(head['q'], head['k'], head['v'], head['g'], head['beta'], h0=ht,
                                           state_fmt=fmt, block_v=bv)
        assert torch.equal(again, want) and B.device_errors() == 0


def _generate(pool, slots, table, x, steps, W):
    """A beam search as a serving loop makes it: token embeddings from `table`,
    a step per layer, logits from the last layer's output."""
    Bn = slots.shape[0]
    flat = slots.reshape(-1)
    tokens = torch.zeros(Bn, W, dtype=torch.int32, device='cuda')
    scores = torch.tensor([[0.0] + [-math.inf] * (W - 1)] * Bn, device='cuda')
    trace = []
    for t in range(steps):
        h = table[tokens.reshape(-1).long()]                                  # [Bn * W, Hv * Dv]
        for layer in range(pool.layers):
            v = h.to(torch.bfloat16).view(Bn * W, 1, pool.Hv, pool.Dv)
            step = {k: x[layer][k][t].expand(Bn * W, *x[layer][k][t].shape).contiguous().unsqueeze(1)
                    for k in ('q', 'k', 'g', 'beta')}
            o = B.gdn_pool_step(pool, layer, flat, v=v, scale=1.0, **step)
            h = h + o.reshape(Bn * W, -1).float()
        logits = (h @ table.T).view(Bn, W, -1)
        scores, parents, tokens = B.gdn_beam_advance(pool, slots, logits, scores)
        trace.append((scores, parents, tokens, logits))
        tokens = tokens.clamp_min(0)
    return trace


def _generation_inputs(Hv, D, V, steps, layers):
    gen = torch.Generator(device='cuda').manual_seed(20)
    table = torch.randn(V, Hv * D, generator=gen, device='cuda') * 0.3
    x = []
    for _ in range(layers):
        d = _draw(1, steps, 1, Hv, D, D, torch.bfloat16, seed=21)
        x.append({k: d[k][0] for k in ('q', 'k', 'g', 'beta')})
    return table, x


def test_beam_search_moves_states_with_their_beams():
    """Every step of a search over two layers, replayed beam by beam: a pool
    in which each beam's whole history is run again from the start, without
    any reordering, holds the same pages, bit for bit."""
    Bn, W, Hv, D, V, steps = 2, 4, 2, 64, 97, 6
    table, x = _generation_inputs(Hv, D, V, steps, 2)
    pool = B.StatePool(2, Bn * W + 1, Hv, D, D, E4M3, 32)
    slots = _ints([[3, 0, 7, 2], [8, 1, 5, 4]])
    trace = _generate(pool, slots, table, x, steps, W)
    assert B.device_errors() == 0
    # the tokens that each final beam consumed, from the parents
    scores, _, _, _ = trace[-1]
    assert bool(scores.isfinite().all())
    for b in range(Bn):
        for w in range(W):
            beam, taken = w, []
            for t in range(steps - 1, -1, -1):
                parent = int(trace[t][1][b, beam])
                taken.append(int(trace[t - 1][2][b, parent]) if t else 0)     # the token that step t consumed
                beam = parent
            taken.reverse()
            alone = B.StatePool(2, 1, Hv, D, D, E4M3, 32)
            for t, tok in enumerate(taken):
                h = table[tok][None]
                for layer in range(2):
                    v = h.to(torch.bfloat16).view(1, 1, Hv, D)
                    step = {k: x[layer][k][t][None, None].clone() for k in ('q', 'k', 'g', 'beta')}
                    o = B.gdn_pool_step(alone, layer, _ints([0]), v=v, scale=1.0, **step)
                    h = h + o.reshape(1, -1).float()
            assert _same(alone.data[:, 0], pool.data[:, int(slots[b, w])]), (b, w)
            assert torch.equal(alone.scales[:, 0], pool.scales[:, int(slots[b, w])])


def test_captured_steps_replay():
    """A captured step, beam choice and reordering, replayed with the
    program's own work between the replays, equals the eager loop."""
    Bn, W, Hv, D, V = 2, 3, 2, 128, 1000
    eager, graphed = (_random_pool(E4M3, 1, Bn * W, Hv, D, D, 64, seed=22) for _ in range(2))
    slots = _ints([[0, 4, 2], [1, 3, 5]])
    flat = slots.reshape(-1)
    x = _draw(Bn * W, 1, 1, Hv, D, D, torch.bfloat16, seed=23)
    proj = torch.randn(Hv * D, V, device='cuda')
    logits = torch.zeros(Bn, W, V, device='cuda')
    scores = torch.zeros(Bn, W, device='cuda')

    def step(pool, scores_in):
        o = B.gdn_pool_step(pool, 0, flat, out=out, **x)
        return (o,) + B.gdn_beam_advance(pool, slots, logits, scores_in)

    out = torch.zeros(Bn * W, 1, Hv, D, dtype=torch.bfloat16, device='cuda')
    keep = _snapshot(graphed)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(graphed, scores)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(graphed, scores)
    graphed.data.view(torch.uint8).copy_(keep[0].view(torch.uint8))
    graphed.scales.copy_(keep[1])
    for r in range(4):
        gen = torch.Generator(device='cuda').manual_seed(30 + r)
        x['v'].copy_(torch.randn(x['v'].shape, generator=gen, device='cuda'))
        logits.copy_((x['v'].reshape(Bn * W, -1).float() @ proj).view(Bn, W, V))
        scores.copy_(-torch.rand(Bn, W, generator=gen, device='cuda'))
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in got]
        want = step(eager, scores)
        for a, b in zip(after, want):
            assert torch.equal(a, b), r
        assert _pool_same(graphed, _snapshot(eager)), r
    assert B.device_errors() == 0


def test_calls_run_on_the_current_stream():
    """Pages written and stepped on a side stream, ordered by events alone."""
    pool, want = (_random_pool(E4M3, 1, 4, 2, 128, 128, 64, seed=24) for _ in range(2))
    x = _draw(4, 1, 1, 2, 128, 128, torch.bfloat16, seed=25)
    new = torch.randn(1, 2, 128, 128, device='cuda')
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            o = B.gdn_pool_step(pool, 0, _ints([0, 1, 2, 3]), **x)
        B.gdn_pool_write(pool, 0, _ints([2]), new)
        B.gdn_pool_reorder(pool, _ints([[0, 1, 2, 3]]), _ints([[3, 2, 1, 0]]))
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        o2 = B.gdn_pool_step(want, 0, _ints([0, 1, 2, 3]), **x)
    B.gdn_pool_write(want, 0, _ints([2]), new)
    B.gdn_pool_reorder(want, _ints([[0, 1, 2, 3]]), _ints([[3, 2, 1, 0]]))
    assert torch.equal(o, o2) and _pool_same(pool, _snapshot(want)) and B.device_errors() == 0


# ------------------------------------------------------------- large batches
# One token of so many heads that a group of waves walks over the tiles of a
# head and over two heads (256 CUs hold 256 to 3,072 groups, by the tile).
LARGE = [(E4M3, torch.bfloat16, 128, 128, 64, 1, 31, 51, True, BEFORE),      # two tiles a head, odd number of heads
         (E4M3, torch.bfloat16, 128, 128, 64, 2, 32, 64, False, AFTER),
         (E4M3, torch.bfloat16, 128, 128, 64, 1, 31, 37, True, AFTER),       # one tile, two elements
         (INT8, torch.bfloat16, 128, 256, 64, 4, 32, 65, False, BEFORE),
         (INT8, torch.bfloat16, 128, 256, 64, 1, 13, 77, True, AFTER),
         (INT8, torch.float32, 128, 256, 256, 1, 9, 39, True, BEFORE),       # one tile a head, of 16 waves
         (INT8, torch.float32, 64, 128, 128, 1, 32, 67, False, AFTER),
         (E4M3, torch.float32, 64, 256, 32, 1, 31, 103, False, BEFORE),      # independent waves, eight tiles
         (E4M3, torch.float32, 128, 256, 128, 1, 11, 71, True, AFTER),
         (E4M3, torch.bfloat16, 64, 64, 16, 1, 31, 101, True, BEFORE),
         (OFF, torch.float32, 64, 128, 64, 2, 32, 64, True, BEFORE)]


@pytest.mark.parametrize("fmt,dt,Dk,Dv,bv,Hqk,Hv,Bn,fork,readout", LARGE)
def test_large_batches_equal_small_ones(fmt, dt, Dk, Dv, bv, Hqk, Hv, Bn, fork, readout):
    """Absent and refused entries next to others, first, last and in a row: the
    same bits as the other entries stepped four at a time, and FP64 for some."""
    say(f"pool step of {Bn} x {Hv} heads fmt={fmt} {dt} Dk={Dk} Dv={Dv} block_v={bv} fork={fork}")
    n = 2 * Bn + 2
    big, small = (_random_pool(fmt, 1, n, Hv, Dk, Dv, bv, seed=40) for _ in range(2))
    snap = _snapshot(big)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(Bn)).tolist()
    slots, out = order[:Bn], order[Bn: 2 * Bn]
    absent, refused = [1, 7, 8, Bn // 2], [0, 2, 9, Bn // 2 + 1, Bn - 1]
    if fork:
        slots = [slots[i // 3] for i in range(Bn)]        # three children each
        out[0] = out[2]                                   # one page for two children
        out[9], out[Bn // 2 + 1], out[Bn - 1] = n, -2, n + 5
    else:
        slots[0] = slots[2]
        slots[9], slots[Bn // 2 + 1], slots[Bn - 1] = n, -2, n + 5
        out = None
    for i in absent:
        slots[i] = -1
    x = _draw(Bn, 1, Hqk, Hv, Dk, Dv, dt, seed=41)
    o = torch.full((Bn, 1, Hv, Dv), 7.0, dtype=dt, device='cuda')
    B.gdn_pool_step(big, 0, _ints(slots), slots_out=None if out is None else _ints(out), readout=readout, out=o, **x)
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    want = torch.full_like(o, 7.0)
    for i in range(0, Bn, 4):
        rows = range(i, min(i + 4, Bn))
        part = [-1 if j in refused else slots[j] for j in rows]
        to = None if out is None else _ints([-1 if j in refused else out[j] for j in rows])
        got = torch.full((len(part), 1, Hv, Dv), 7.0, dtype=dt, device='cuda')
        B.gdn_pool_step(small, 0, _ints(part), slots_out=to, readout=readout, out=got,
                        **{k: v[i: i + 4].contiguous() for k, v in x.items()})
        want[i: i + 4] = got
    assert B.device_errors() == 0
    want[refused] = float('nan')
    assert bool(o[refused].isnan().all()) and bool((o[absent] == 7.0).all())
    assert torch.equal(o.nan_to_num(nan=-5.0), want.nan_to_num(nan=-5.0))
    assert _pool_same(big, _snapshot(small))
    values = B.StatePool.from_tensors(snap[0][:, [slots[j] for j in (3, 10, Bn - 2)]].contiguous() if fmt == OFF else
                                      snap[0].view(torch.uint8)[:, [slots[j] for j in (3, 10, Bn - 2)]].view(snap[0].dtype),
                                      None if fmt == OFF else snap[1][:, [slots[j] for j in (3, 10, Bn - 2)]], fmt, bv)
    before = _values(values)[0]
    for i, j in enumerate((3, 10, Bn - 2)):
        to = slots[j] if out is None else out[j]
        _check_step(big, before[i], big.data[0, to], None if fmt == OFF else big.scales[0, to], x, o[j, 0], j, to,
                    Dk ** -0.5, readout)


# ------------------------------------------------------------- tiles of zeros
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("fmt,dt,Dk,bv", [(E4M3, torch.bfloat16, 128, 64), (INT8, torch.bfloat16, 128, 64),
                                          (INT8, torch.float32, 64, 128), (E4M3, torch.float32, 64, 16)])
def test_a_tile_that_becomes_zero_or_tiny(fmt, dt, Dk, bv, T):
    """A zero tile under a large scale, a state that one token erases, and an
    update far below the tile's scale: codes 0 (or those of the tiny values)
    under the smallest scale, 2^-126."""
    Hv, Dv = 2, 128
    pool = B.StatePool(1, 4, Hv, Dk, Dv, fmt, bv)
    pool.scales.fill_(8.0)
    codes = torch.zeros(4, Hv, Dv, Dk, device='cuda')
    codes[1, :, :, 5] = torch.arange(Dv, device='cuda') % 13 - 6.0         # states along one key
    pool.data[0] = codes.to(pool.data.dtype)
    x = _draw(4, T, 1, Hv, Dk, Dv, dt, seed=50)
    x['k'].zero_()
    x['k'][:, :, :, 5] = 1.0
    x['v'].zero_()
    x['g'].zero_()
    x['beta'].fill_(1.0)
    tiny = fmt != OFF and dt is torch.float32
    if tiny:                                              # 2^-122 is code 16 under 2^-126
        x['v'][2] = 2.0 ** -122
    for readout in (BEFORE, AFTER):
        p = B.StatePool.from_tensors(pool.data.clone(), pool.scales.clone(), fmt, bv)
        o = B.gdn_pool_step(p, 0, _ints([0, 1, 2, -1]), readout=readout, **x)
        assert B.device_errors() == 0
        assert bool(p.data[0, :2].float().eq(0).all()) and bool((p.scales[0, :3] == 2.0 ** -126).all())
        # |states| <= 48 with four roundings each in k . q, S^T q and their sum; the half step of o is within
        assert bool((o[:2].float().abs() <= 48 * 4 * U).all()) and bool(o.isfinite().all())
        want = torch.zeros(Hv, Dv, Dk, device='cuda')
        if tiny:
            want[:, :, 5] = 16.0
        assert torch.equal(p.data[0, 2].float(), want)
        # what follows is a step from the zero state
        y = _draw(4, 1, 1, Hv, Dk, Dv, dt, seed=51)
        fresh = B.StatePool(1, 4, Hv, Dk, Dv, fmt, bv)
        a = B.gdn_pool_step(p, 0, _ints([0, 1, -1, -1]), readout=readout, **y)
        b = B.gdn_pool_step(fresh, 0, _ints([0, 1, -1, -1]), readout=readout, **y)
        assert torch.equal(a, b) and _pool_same(p, _snapshot(fresh), [0, 1])


# ------------------------------------------------ entries that claim no page
@pytest.mark.parametrize("fmt", [E4M3, INT8, OFF])
def test_entries_that_do_nothing_claim_no_page(fmt):
    """Padding rows of length 0 may name a live page, and an entry refused for
    a slot outside the pool does not keep another from its pages."""
    Hv, D, bad = 2, 128, B.DEVERR_POOL_SLOT
    pool, want = (_random_pool(fmt, 1, 9, Hv, D, D, 64, seed=60) for _ in range(2))
    x = _draw(6, 2, 1, Hv, D, D, torch.bfloat16, seed=61)
    # 3 is stepped by entry 0; entries 1 and 4 name it with nothing to do; entry 3 names 5, which entry 2 steps
    slots, lens = [3, 3, 5, 5, 3, 7], [2, 0, 1, -4, 0, 2]
    o = B.gdn_pool_step(pool, 0, _ints(slots), lens=_ints(lens), **x)
    assert B.device_errors() == 0
    o2 = B.gdn_pool_step(want, 0, _ints([3, -1, 5, -1, -1, 7]), lens=_ints(lens), **x)
    assert torch.equal(o, o2) and _pool_same(pool, _snapshot(want))
    # with slots_out: length 0 to the own page or to none does nothing, length 0 to another page is a copy
    out = [4, -1, 5, 5, 3, 2]
    o = B.gdn_pool_step(pool, 0, _ints([3, 4, 5, 5, 3, 7]), slots_out=_ints(out), lens=_ints([2, 0, 1, 0, 0, 0]), **x)
    assert B.device_errors() == 0
    o2 = B.gdn_pool_step(want, 0, _ints([3, -1, 5, -1, -1, 7]), slots_out=_ints(out), lens=_ints([2, 0, 1, 0, 0, 0]), **x)
    assert torch.equal(o, o2) and _pool_same(pool, _snapshot(want))
    # a length of 0 whose copy reads the page still claims it
    snap = _snapshot(pool)
    o = B.gdn_pool_step(pool, 0, _ints([3, 3, -1, -1, -1, -1]), slots_out=_ints([3, 8, 0, 0, 0, 0]),
                        lens=_ints([2, 0, 0, 0, 0, 0]), **x)
    assert B.device_errors() == bad and bool(o[0].isnan().all()) and _pool_same(pool, snap, [3])
    assert _pool_same(pool, (pool.data[:, [3] * 9].contiguous() if fmt == OFF else
                             pool.data.view(torch.uint8)[:, [3] * 9].view(pool.data.dtype),
                             None if fmt == OFF else pool.scales[:, [3] * 9]), [8])
    # one token: entries refused for their own slots
    want.data.view(torch.uint8).copy_(pool.data.view(torch.uint8))
    if fmt != OFF:
        want.scales.copy_(pool.scales)
    y = {k: v[:, :1].contiguous() for k, v in x.items()}
    o = B.gdn_pool_step(pool, 0, _ints([1, 2, 9, 0, -1, -1]), slots_out=_ints([1, 9, 2, 2, 1, -1]), **y)
    assert B.device_errors() == bad and bool(o[[1, 2]].isnan().all())
    o2 = B.gdn_pool_step(want, 0, _ints([1, -1, -1, 0, -1, -1]), slots_out=_ints([1, 9, 2, 2, 1, -1]), **y)
    assert torch.equal(o[[0, 3, 4, 5]], o2[[0, 3, 4, 5]]) and _pool_same(pool, _snapshot(want))
    # no token at all: only copies to another page touch one
    none = {k: v[:, :0] for k, v in x.items()}
    B.gdn_pool_step(pool, 0, _ints([3, 4, 8, 5, 4, -1]), slots_out=_ints([3, 8, 8, -1, 5, -1]), **none)
    assert B.device_errors() == 0
    B.gdn_pool_copy(want, _ints([4, 4]), _ints([8, 5]))
    assert _pool_same(pool, _snapshot(want))
    # pages in
    z = torch.randn(3, Hv, D, D, device='cuda')
    B.gdn_pool_write(pool, 0, _ints([4, 9, -3]), z)
    B.gdn_pool_write(want, 0, _ints([4, -1, -1]), z)
    assert B.device_errors() == bad and _pool_same(pool, _snapshot(want))


def test_moves_that_do_nothing_claim_no_page():
    pool = _random_pool(E4M3, 2, 10, 2, 64, 64, 64, seed=62)
    snap = _snapshot(pool)
    # 3 <- 3 does nothing, so 3 may be written; 6 <- 3 reads it and so may not stand beside
    B.gdn_pool_copy(pool, _ints([3, 0, 5, 5]), _ints([3, 3, 1, 5]))
    assert B.device_errors() == 0
    for s, w in ((3, 0), (1, 5), (5, 5), (0, 0)):
        assert _same(pool.data[:, s], snap[0][:, w]), s
    snap = _snapshot(pool)
    # 4 -> 10 and 11 -> 6 are refused for their own slots; the copies to 4 and 6 are done
    B.gdn_pool_copy(pool, _ints([4, 2, 11, 2, 7, 8]), _ints([10, 4, 6, 6, 9, 7]))
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    for s, w in ((4, 2), (6, 2), (9, 7), (7, 7), (2, 2)):  # 7 is read by another entry
        assert _same(pool.data[:, s], snap[0][:, w]), s


def test_reorder_takes_a_page_only_where_no_other_beam_names_it():
    """Every beam of the call counts, also one that keeps its page."""
    pool = _random_pool(E4M3, 1, 8, 2, 64, 64, 64, seed=63)
    snap = _snapshot(pool)
    B.gdn_pool_reorder(pool, _ints([[0, 1], [2, 0]]), _ints([[1, 0], [-1, -1]]))
    assert B.device_errors() == B.DEVERR_POOL_SLOT
    assert _same(pool.data[:, 0], snap[0][:, 0]) and _same(pool.data[:, 1], snap[0][:, 0])


# ------------------------------------------------------------- unaligned views
def test_tokens_out_of_a_longer_block():
    """One sequence's gates at any token: contiguous slices whose address is a
    multiple of 4 bytes only."""
    Hv, D = 3, 64
    for fmt in (E4M3, OFF):
        a, b = (_random_pool(fmt, 1, 1, Hv, D, D, 32, seed=66) for _ in range(2))
        x = _draw(1, 5, 1, Hv, D, D, torch.bfloat16, seed=67)
        for t in range(5):
            view = {k: v[:, t:t + 1] for k, v in x.items()}
            assert t != 1 or view['g'].data_ptr() % 16
            o1 = B.gdn_pool_step(a, 0, _ints([0]), **view)
            o2 = B.gdn_pool_step(b, 0, _ints([0]), **{k: v.clone() for k, v in view.items()})
            assert torch.equal(o1, o2)
        view = {k: v[:, 1:4] for k, v in x.items()}       # three tokens of it
        lens = _ints([9, 2, 9])[1:2]
        o1 = B.gdn_pool_step(a, 0, _ints([0]), lens=lens, **view)
        o2 = B.gdn_pool_step(b, 0, _ints([0]), lens=lens.clone(), **{k: v.clone() for k, v in view.items()})
        assert torch.equal(o1, o2) and _pool_same(a, _snapshot(b)) and B.device_errors() == 0


# ------------------------------------------------------------- NaN and infinities
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("fmt,dt,bv", [(INT8, torch.bfloat16, 64), (INT8, torch.float32, 16), (INT8, torch.bfloat16, 128),
                                       (E4M3, torch.bfloat16, 64), (OFF, torch.float32, 64)])
def test_a_nan_stays_in_the_page(fmt, dt, bv, T):
    """A token whose inputs are not finite leaves NaN in the states that it
    reaches, with every format, and the next tokens show it; other tiles and
    sequences keep their bits."""
    Hv, D, Bn = 2, 128, 7
    pool, clean = (_random_pool(fmt, 1, Bn, Hv, D, D, bv, seed=68) for _ in range(2))
    x = _draw(Bn, T, 1, Hv, D, D, dt, seed=69)
    y = _draw(Bn, 1, 1, Hv, D, D, dt, seed=70)
    lens = {} if T == 1 else dict(lens=_ints([T] * Bn))
    slots = _ints(list(range(Bn)))
    B.gdn_pool_step(clean, 0, slots, **lens, **x)
    bad = {k: v.clone() for k, v in x.items()}
    nan, inf = float('nan'), math.inf
    bad['g'][1, 0, 0] = nan                               # head 0 of sequence 1
    bad['beta'][2, 0, 1] = nan
    bad['k'][3, 0, 0, 9] = nan                            # both heads
    bad['v'][4, 0, 1, 70] = nan                           # one value row
    bad['v'][5, 0, 0, 3] = inf
    o = B.gdn_pool_step(pool, 0, slots, **lens, **bad)
    rows = bv if fmt == INT8 else 1
    hit = torch.zeros(Bn, Hv, D, dtype=torch.bool, device='cuda')
    hit[1, 0] = hit[2, 1] = hit[3] = True
    hit[4, 1, 70 // rows * rows: 70 // rows * rows + rows] = True
    hit[5, 0, 3 // rows * rows: 3 // rows * rows + rows] = True
    states = B.gdn_pool_read(pool, 0, slots)              # [Bn, Hv, Dk, Dv]
    assert bool((~states.isfinite()).any(2)[hit].all())
    if fmt == INT8:
        assert bool(states.isnan().all(2)[hit].all())
    tiles = hit.unflatten(-1, (-1, bv)).any(-1).repeat_interleave(bv, -1)
    want = B.gdn_pool_read(clean, 0, slots)
    assert torch.equal(states.mT[~tiles], want.mT[~tiles])
    o2, o3 = (B.gdn_pool_step(p, 0, slots, **y) for p in (pool, clean))
    assert not bool(o2[:, 0][hit].isfinite().any())
    assert torch.equal(o2[:, 0][~tiles], o3[:, 0][~tiles])
    assert not bool(B.gdn_pool_read(pool, 0, slots).isfinite().all(2)[hit].any())
    assert B.device_errors() == 0


@pytest.mark.parametrize("fmt,Dk,Dv,bv", [(INT8, 128, 128, 64), (INT8, 64, 256, 16), (INT8, 128, 256, 256),
                                          (E4M3, 128, 128, 64)])
def test_a_nan_state_is_written_as_one(fmt, Dk, Dv, bv):
    x = torch.randn(5, 2, Dk, Dv, device='cuda')
    pool, clean = (B.StatePool(1, 5, 2, Dk, Dv, fmt, bv) for _ in range(2))
    slots = _ints([0, 1, 2, 3, 4])
    B.gdn_pool_write(clean, 0, slots, x)
    hit = torch.zeros(5, 2, Dv // bv, dtype=torch.bool, device='cuda')
    for n, h, i, j, val in ((0, 1, 0, 0, math.nan), (1, 0, Dk - 1, Dv - 1, math.nan), (3, 1, 37, 21, math.inf),
                            (3, 0, 50, bv - 1, -math.nan)):
        x[n, h, i, j] = val
        hit[n, h, j // bv] = True
    B.gdn_pool_write(pool, 0, slots, x)
    got, want = (B.gdn_pool_read(p, 0, slots).unflatten(-1, (-1, bv)) for p in (pool, clean))
    bad = ~got.isfinite()
    assert torch.equal(bad.any(-1).any(2), hit)
    if fmt == INT8:
        assert bool(bad.all(-1).all(2)[hit].all())
    assert torch.equal(got.permute(0, 1, 3, 2, 4)[~hit], want.permute(0, 1, 3, 2, 4)[~hit])


# ------------------------------------------------------------- slots outside
@pytest.mark.parametrize("fmt", [E4M3, OFF])
def test_slots_outside_the_pool_are_always_reported(fmt):
    """Also where the entry would have done nothing."""
    pool = _random_pool(fmt, 1, 6, 2, 64, 64, 64, seed=64)
    snap = _snapshot(pool)
    x = _draw(2, 2, 1, 2, 64, 64, torch.bfloat16, seed=65)
    calls = [lambda: B.gdn_pool_copy(pool, _ints([6, 0]), _ints([6, -1])),
             lambda: B.gdn_pool_copy(pool, _ints([-2, 0]), _ints([-2, -1])),
             lambda: B.gdn_pool_step(pool, 0, _ints([6, -1]), lens=_ints([0, 0]), **x),
             lambda: B.gdn_pool_step(pool, 0, _ints([-1, -2]), lens=_ints([0, 0]), **x),
             lambda: B.gdn_pool_step(pool, 0, _ints([7, -1]), slots_out=_ints([7, -1]), lens=_ints([0, 1]), **x),
             lambda: B.gdn_pool_step(pool, 0, _ints([6, -1]), slots_out=_ints([-1, -1]), lens=_ints([0, 1]), **x),
             lambda: B.gdn_pool_reorder(pool, _ints([[0, 6]]), _ints([[0, 1]])),
             lambda: B.gdn_pool_reorder(pool, _ints([[0, -2]]), _ints([[-1, -1]]))]
    for i, call in enumerate(calls):
        call()
        assert B.device_errors() == B.DEVERR_POOL_SLOT, i
        assert _pool_same(pool, snap), i
    B.gdn_pool_copy(pool, _ints([-1, -1, 0]), _ints([-1, -1, 0]))
    B.gdn_pool_step(pool, 0, _ints([-1, 2]), lens=_ints([0, 0]), **x)
    B.gdn_pool_reorder(pool, _ints([[0, -1, 2]]), _ints([[0, 1, -1]]))
    assert B.device_errors() == 0 and _pool_same(pool, snap)


# ------------------------------------------------------------- scale rules
@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_prefill_into_a_reciprocal_pool(fmt):
    """The chunk forward divides; its final state is written by the pool's rule."""
    N, T, Hv, D = 2, 70, 2, 128
    x = _draw(N, T, 1, Hv, D, D, torch.bfloat16, seed=71)
    pool, want = (B.StatePool(1, 3, Hv, D, D, fmt, 32, scale_rule=B.SCALE_RECIPROCAL) for _ in range(2))
    slots = _ints([2, 0])
    o = B.gdn_pool_prefill(pool, 0, slots, **x)
    o2, ht, _ = B.gdn_chunk_fwd(x['q'], x['k'], x['v'], x['g'], x['beta'], h0=torch.zeros(N, Hv, D, D, device='cuda'),
                                state_fmt=fmt, block_v=32)
    B.gdn_pool_write(want, 0, slots, ht)
    assert torch.equal(o, o2) and _pool_same(pool, _snapshot(want)) and B.device_errors() == 0
