"""Rules on logits and linear attention: what is refused, on the host, before any
launch (status and message of the C entry points, ValueError of the binding)."""
import ctypes

import pytest
import torch

from gateddeltanet_chunked_recurrence_amd import binding as B

FAKE = 0x10000                                   # aligned, never dereferenced on these paths


def _call(name, a):
    lib = B.load_library()
    return getattr(lib, name)(ctypes.byref(a), None), lib.gdn_last_error().decode()


def _logits(**kw):
    a = B.LogitsArgs(B=2, W=3, V=100, io_dtype=B.GDN_BF16, L=10, num_bias=4, num_masks=6, logits=FAKE, out=FAKE * 64,
                     tokens=FAKE, bias_ids=FAKE, bias_vals=FAKE, mask=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize('kw,status,msg', [
    (dict(B=-1), B.GDN_E_INVALID, 'sizes'), (dict(B=65536), B.GDN_E_INVALID, 'sizes'), (dict(W=0), B.GDN_E_INVALID, 'sizes'),
    (dict(V=0), B.GDN_E_INVALID, 'sizes'), (dict(V=2 ** 30 + 1), B.GDN_E_UNSUPPORTED, 'large'),
    (dict(L=-1), B.GDN_E_INVALID, 'sizes'), (dict(L=1 << 20), B.GDN_E_UNSUPPORTED, '2^20'),
    (dict(num_bias=-1), B.GDN_E_UNSUPPORTED, 'num_bias'), (dict(num_bias=1025), B.GDN_E_UNSUPPORTED, 'num_bias'),
    (dict(io_dtype=2), B.GDN_E_INVALID, 'io_dtype'), (dict(row_stride=99), B.GDN_E_INVALID, 'row_stride'),
    (dict(out_stride=-1), B.GDN_E_INVALID, 'out_stride'), (dict(token_stride=9), B.GDN_E_INVALID, 'token_stride'),
    (dict(logits=None), B.GDN_E_INVALID, 'logits is NULL'), (dict(out=None), B.GDN_E_INVALID, 'out is NULL'),
    (dict(out=FAKE * 64 + 1), B.GDN_E_INVALID, 'out is not'), (dict(tokens=FAKE + 2), B.GDN_E_INVALID, 'tokens is not'),
    (dict(bias_ids=None), B.GDN_E_INVALID, 'bias_ids is NULL'), (dict(bias_vals=FAKE + 2), B.GDN_E_INVALID, 'bias_vals is not'),
    (dict(num_masks=5), B.GDN_E_INVALID, 'num_masks'), (dict(mask=None, mask_rows=FAKE), B.GDN_E_INVALID, 'mask is NULL'),
    (dict(out=FAKE + 2), B.GDN_E_INVALID, 'overlaps'), (dict(out=FAKE, out_stride=128), B.GDN_E_INVALID, 'overlaps'),
    (dict(out=FAKE + 1198), B.GDN_E_INVALID, 'overlaps'), (dict(out=FAKE - 1198), B.GDN_E_INVALID, 'overlaps'),
])
def test_logits_adjust_checks_its_arguments(kw, status, msg):
    got, text = _call('gdn_logits_adjust', _logits(**kw))
    assert got == status and msg in text and (msg == 'io_dtype' or 'gdn_logits_adjust' in text), (got, text)


def test_logits_adjust_with_nothing_to_do():
    assert _call('gdn_logits_adjust', _logits(B=0, logits=None, out=None))[0] == B.GDN_OK


def _linear(**kw):
    a = B.LinearArgs(B=2, T=100, Hqk=2, Hv=4, Dk=128, Dv=256, num_seqs=2, io_dtype=B.GDN_BF16, scale=0.1)
    for name in ('q', 'k', 'v', 'g', 'o'):
        setattr(a, name, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


LINEAR = [
    (dict(B=-1), B.GDN_E_INVALID, 'sizes'), (dict(T=-1), B.GDN_E_INVALID, 'sizes'), (dict(Hqk=0), B.GDN_E_INVALID, 'sizes'),
    (dict(Hqk=3), B.GDN_E_INVALID, 'multiple'), (dict(Hv=65536), B.GDN_E_UNSUPPORTED, 'Hv'),
    (dict(Dk=96), B.GDN_E_UNSUPPORTED, 'Dk'), (dict(Dv=512), B.GDN_E_UNSUPPORTED, 'Dv'),
    (dict(io_dtype=2), B.GDN_E_INVALID, 'io_dtype'), (dict(g_per_head=2), B.GDN_E_INVALID, 'g_per_head'),
    (dict(scale=float('nan')), B.GDN_E_INVALID, 'scale'), (dict(num_seqs=3), B.GDN_E_INVALID, 'num_seqs'),
    (dict(cu_seqlens=FAKE), B.GDN_E_INVALID, 'cu_seqlens'), (dict(B=1, cu_seqlens=FAKE, num_seqs=0), B.GDN_E_INVALID, 'num_seqs'),
    (dict(B=70000, num_seqs=70000, T=1), B.GDN_E_UNSUPPORTED, 'num_seqs'),
    (dict(B=2, T=1 << 30), B.GDN_E_UNSUPPORTED, 'tokens'),
    (dict(T=1 << 29, Hv=64), B.GDN_E_UNSUPPORTED, 'too large'),
    (dict(q_stride=255), B.GDN_E_INVALID, 'q_stride'), (dict(k_stride=260), B.GDN_E_INVALID, 'k_stride'),
    (dict(v_stride=1 << 24), B.GDN_E_INVALID, 'v_stride'),
    (dict(q=None), B.GDN_E_INVALID, 'q is NULL'), (dict(g=None), B.GDN_E_INVALID, 'g is NULL'),
    (dict(k=FAKE + 8), B.GDN_E_INVALID, 'k is not'), (dict(g=FAKE + 2), B.GDN_E_INVALID, 'g is not'),
    (dict(h0=FAKE + 4), B.GDN_E_INVALID, 'h0 is not'),
]


@pytest.mark.parametrize('kw,status,msg', LINEAR + [
    (dict(o=None), B.GDN_E_INVALID, 'o is NULL'), (dict(ht=FAKE + 8), B.GDN_E_INVALID, 'ht is not'),
    (dict(T=65536), B.GDN_E_WORKSPACE, 'workspace'), (dict(T=65536, workspace=FAKE, workspace_bytes=100), B.GDN_E_WORKSPACE, 'needed')])
def test_linear_forward_checks_its_arguments(kw, status, msg):
    got, text = _call('gdn_linear_fwd', _linear(**kw))
    assert got == status and msg in text, (got, text)


@pytest.mark.parametrize('kw,status,msg', LINEAR + [
    (dict(do_=None), B.GDN_E_INVALID, 'do is NULL'), (dict(dg=None), B.GDN_E_INVALID, 'dg is NULL'),
    (dict(dv=FAKE + 8), B.GDN_E_INVALID, 'dv is not'), (dict(dh0=FAKE + 4), B.GDN_E_INVALID, 'dh0 is not'),
    (dict(), B.GDN_E_WORKSPACE, 'workspace')])
def test_linear_backward_checks_its_arguments(kw, status, msg):
    own = {k: v for k, v in kw.items() if k in ('do_', 'dht', 'dq', 'dk', 'dv', 'dg', 'dh0')}
    b = B.LinearBwdArgs(fwd=_linear(**{k: v for k, v in kw.items() if k not in own}))
    for name in ('do_', 'dq', 'dk', 'dv', 'dg'):
        setattr(b, name, FAKE)
    for k, v in own.items():
        setattr(b, k, v)
    got, text = _call('gdn_linear_bwd', b)
    assert got == status and msg in text, (got, text)


# the last byte of one and the first of another, in a call whose tensors lie apart otherwise
def _apart(names, at):
    return {n: 0x100000000 + (i << 32) for i, n in enumerate(names)} | at


QB, VB, SB = 2 * 100 * 2 * 128 * 2, 2 * 100 * 4 * 256 * 2, 2 * 4 * 128 * 256 * 4


@pytest.mark.parametrize('out,of,off', [
    ('o', 'v', 0), ('o', 'q', QB - 16), ('o', 'k', 16 - VB), ('o', 'g', 0), ('ht', 'h0', 0), ('ht', 'o', VB - 16),
    ('o', 'q', 'strided')])
def test_linear_forward_refuses_outputs_in_other_memory(out, of, off):
    kw = _apart(('q', 'k', 'v', 'g', 'h0', 'o', 'ht'), {})
    if off == 'strided':
        kw['q_stride'] = 1024
        off = 199 * 1024 * 2
    kw[out] = kw[of] + off
    got, text = _call('gdn_linear_fwd', _linear(**kw))
    assert got == B.GDN_E_INVALID and f'{out} overlaps {of}' in text, (got, text)


@pytest.mark.parametrize('out,of,off', [
    ('dq', 'q', 0), ('dk', 'dq', QB - 16), ('dv', 'do_', 0), ('dv', 'v', 16 - VB), ('dg', 'g', 0), ('dh0', 'dht', SB - 16)])
def test_linear_backward_refuses_outputs_in_other_memory(out, of, off):
    kw = _apart(('q', 'k', 'v', 'g', 'h0', 'do_', 'dht', 'dq', 'dk', 'dv', 'dg', 'dh0', 'workspace'), {})
    kw[out] = kw[of] + off
    own = {k: kw.pop(k) for k in ('do_', 'dht', 'dq', 'dk', 'dv', 'dg', 'dh0', 'workspace')}
    b = B.LinearBwdArgs(fwd=_linear(**kw), workspace_bytes=1 << 31, **own)
    got, text = _call('gdn_linear_bwd', b)
    assert got == B.GDN_E_INVALID and f'{out} overlaps {of.rstrip("_")}' in text, (got, text)


@pytest.mark.parametrize('kw', [
    dict(B=65535, num_seqs=65535, T=1, Hv=512, Hqk=512, Dk=64, Dv=64),          # workgroups of the walks
    dict(B=1, num_seqs=65535, T=1 << 20, Hv=256, Hqk=128, cu_seqlens=FAKE)])
def test_linear_refuses_grids_past_32_bits(kw):
    got, text = _call('gdn_linear_fwd', _linear(**kw))
    assert got == B.GDN_E_UNSUPPORTED and 'too large' in text, (got, text)
    assert B.load_library().gdn_linear_fwd_workspace_bytes(ctypes.byref(_linear(**kw))) == 0


def test_linear_backward_refuses_a_sum_over_heads_past_32_bits():
    b = B.LinearBwdArgs(fwd=_linear(B=1, num_seqs=1, T=1 << 20, Hqk=128, Hv=256, Dv=64))
    for name in ('do_', 'dq', 'dk', 'dv', 'dg'):
        setattr(b, name, FAKE)
    got, text = _call('gdn_linear_bwd', b)
    assert got == B.GDN_E_UNSUPPORTED and 'Hqk * Dk is too large' in text, (got, text)


def test_logits_adjust_refuses_grids_past_32_bits():
    got, text = _call('gdn_logits_adjust', _logits(B=65535, W=300, V=10, out=FAKE, mask=None))
    assert got == B.GDN_E_UNSUPPORTED and 'too large' in text, (got, text)


def test_linear_with_nothing_to_do():
    for kw in (dict(B=0, num_seqs=0), dict(T=0)):
        assert _call('gdn_linear_fwd', _linear(**kw))[0] == B.GDN_OK
        assert B.load_library().gdn_linear_fwd_workspace_bytes(ctypes.byref(_linear(**kw))) == 0


def test_linear_workspace_grows_with_the_segments():
    lib = B.load_library()
    one = lib.gdn_linear_fwd_workspace_bytes(ctypes.byref(_linear(B=64, num_seqs=64, T=128, Hv=16)))
    many = lib.gdn_linear_fwd_workspace_bytes(ctypes.byref(_linear(B=1, num_seqs=1, T=65536, Hv=4)))
    assert one == 0                                             # enough heads: one segment each
    assert many > 4 * 128 * 256 * 4 and many % 4 == 0


@pytest.mark.parametrize('kw,status,msg', [
    (dict(g_per_head=2), B.GDN_E_INVALID, 'g_per_head'), (dict(T=-1), B.GDN_E_INVALID, 'sizes'),
    (dict(Hqk=3), B.GDN_E_INVALID, 'multiple'), (dict(layer=2), B.GDN_E_INVALID, 'layer'),
    (dict(v=None), B.GDN_E_INVALID, 'v is NULL'), (dict(g=None), B.GDN_E_INVALID, 'g is NULL'),
    (dict(slots_out=FAKE + 4), B.GDN_E_INVALID, 'slots_out is not')])
def test_linear_step_checks_its_arguments(kw, status, msg):
    pool = B.PoolStruct(2, 5, 4, 128, 128, B.QDQ_OFF, 64, B.SCALE_DIVIDE, FAKE, None)
    a = B.PoolLinearStepArgs(B.PoolStepArgs(B=3, T=2, Hqk=2, io_dtype=B.GDN_BF16, scale=0.1), 0)
    for name in ('slots', 'q', 'k', 'v', 'g', 'o'):
        setattr(a.step, name, FAKE)
    for k, v in kw.items():
        setattr(a if k == 'g_per_head' else a.step, k, v)
    lib = B.load_library()
    got = lib.gdn_pool_linear_step(ctypes.byref(pool), ctypes.byref(a), None)
    text = lib.gdn_last_error().decode()
    assert got == status and msg in text and 'gdn_pool_linear_step' in text, (got, text)
    assert lib.gdn_pool_linear_step(ctypes.byref(pool), None, None) == B.GDN_E_INVALID


def test_binding_refuses_tensors_of_another_kind():
    x = torch.zeros(2, 3, 50)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)                 # noqa: E731
    bad = [
        (x[0], {}), (x.half(), {}), (x.expand(4, 2, 3, 50)[:, 0], {}), (x[..., ::2], {}), (x, dict(tokens=i32(2, 3))),
        (x, dict(tokens=torch.zeros(2, 3, 4, dtype=torch.int64))), (x, dict(tokens=i32(2, 3, 4), lens=i32(2))),
        (x, dict(tokens=i32(2, 3, 4), repetition=torch.zeros(3))), (x, dict(repetition=torch.zeros(2))),
        (x, dict(lens=i32(2, 3))), (x, dict(bias=(i32(2, 4), torch.zeros(2, 5)))), (x, dict(mask=i32(6, 3))),
        (x, dict(mask_rows=i32(2, 3))), (x, dict(mask=i32(6, 2), mask_rows=i32(3, 2))), (x, dict(out=x[:, :2])),
        (x, dict(out=x.bfloat16())), (x, dict(out=torch.zeros(2, 3, 100)[..., ::2])),
    ]
    for t, kw in bad:
        with pytest.raises(ValueError):
            B.gdn_logits_adjust(t, **kw)
    with pytest.raises(ValueError, match='GPU'):
        B.gdn_logits_adjust(x)
    q, k, v, g = torch.zeros(1, 5, 2, 64), torch.zeros(1, 5, 2, 64), torch.zeros(1, 5, 4, 64), torch.zeros(1, 5, 4)
    for args, kw in [((q[0], k, v, g), {}), ((q, k.bfloat16(), v, g), {}), ((q.half(), k.half(), v.half(), g), {}),
                     ((q, k[:, :4], v, g), {}), ((q, k, v, g[..., :2]), {}), ((q, k, v, g[0, 0, :2]), {}),
                     ((q, k, v, g.double()), {}), ((q.transpose(1, 2), k, v, g), {}),
                     ((q, k, v, g), dict(h0=torch.zeros(1, 4, 64, 32))), ((q, k, v, g), dict(cu_seqlens=torch.zeros(2))),
                     ((q, k, v, g), dict(cu_seqlens=i32(1))), ((q, k, v, g), dict(out=torch.zeros(1, 5, 4, 32)))]:
        with pytest.raises(ValueError):
            B.gdn_linear_fwd(*args, **kw)
    for kw in (dict(do=v[:, :4]), dict(do=v.bfloat16()), dict(do=v, dht=torch.zeros(1, 4, 64)),
               dict(do=v, out=dict(dq=q, dk=k, dv=q, dg=g))):
        with pytest.raises(ValueError):
            B.gdn_linear_bwd(q, k, v, g, **kw)
    with pytest.raises(ValueError, match='GPU'):
        B.gdn_linear_fwd(q, k, v, g)
