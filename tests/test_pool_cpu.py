"""State pool and beam selection: what is refused, on the host, before any
launch. The C entry points return the documented status and message; the
binding raises ValueError for tensors of another type, shape, layout or
device. No call here reaches a kernel."""
import ctypes

import pytest
import torch

from gateddeltanet_chunked_recurrence_amd import binding as B

FAKE = 0x10000                                   # aligned, never dereferenced on these paths


def _pool(**kw):
    p = B.PoolStruct(2, 5, 4, 128, 128, B.QDQ_E4M3, 64, B.SCALE_DIVIDE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _call(name, *args):
    lib = B.load_library()
    status = getattr(lib, name)(*args)
    return status, lib.gdn_last_error().decode()


BAD_POOL = [
    (dict(state_fmt=3), B.GDN_E_UNSUPPORTED, 'format'),
    (dict(layers=0), B.GDN_E_INVALID, 'sizes'),
    (dict(slots=0), B.GDN_E_INVALID, 'sizes'),
    (dict(Hv=0), B.GDN_E_INVALID, 'sizes'),
    (dict(Dk=96), B.GDN_E_UNSUPPORTED, 'Dk'),
    (dict(Dv=512), B.GDN_E_UNSUPPORTED, 'Dv'),
    (dict(block_v=48), B.GDN_E_UNSUPPORTED, 'block_v'),
    (dict(block_v=256), B.GDN_E_INVALID, 'divide'),
    (dict(scale_rule=2), B.GDN_E_INVALID, 'scale_rule'),
    (dict(scales=None), B.GDN_E_INVALID, 'scales is NULL'),
    (dict(scales=FAKE + 4), B.GDN_E_INVALID, 'scales is not'),
    (dict(data=None), B.GDN_E_INVALID, 'data is NULL'),
    (dict(data=FAKE + 8), B.GDN_E_INVALID, 'data is not'),
]


@pytest.mark.parametrize("kw,status,msg", BAD_POOL)
def test_every_pool_call_checks_the_pool(kw, status, msg):
    p = ctypes.byref(_pool(**kw))
    step, beam = B.PoolStepArgs(), None
    for name, args in (('gdn_pool_write', (p, 0, FAKE, 1, FAKE, None)),
                       ('gdn_pool_read', (p, 0, FAKE, 1, FAKE, None)),
                       ('gdn_pool_copy', (p, FAKE, FAKE, 1, None)),
                       ('gdn_pool_reorder', (p, FAKE, FAKE, 1, 4, None)),
                       ('gdn_pool_step', (p, ctypes.byref(step), None))):
        got, text = _call(name, *args)
        assert got == status and msg in text and name in text, (name, got, text)


@pytest.mark.parametrize("name,args,status,msg", [
    ('gdn_pool_write', (2, FAKE, 1, FAKE), B.GDN_E_INVALID, 'layer'),
    ('gdn_pool_write', (-1, FAKE, 1, FAKE), B.GDN_E_INVALID, 'layer'),
    ('gdn_pool_write', (0, FAKE, -1, FAKE), B.GDN_E_INVALID, 'entries'),
    ('gdn_pool_write', (0, FAKE, 70000, FAKE), B.GDN_E_UNSUPPORTED, 'entries'),
    ('gdn_pool_write', (0, None, 1, FAKE), B.GDN_E_INVALID, 'slots is NULL'),
    ('gdn_pool_write', (0, FAKE, 1, None), B.GDN_E_INVALID, 'states is NULL'),
    ('gdn_pool_read', (0, FAKE + 4, 1, FAKE), B.GDN_E_INVALID, 'slots is not'),
    ('gdn_pool_read', (0, FAKE, 1, FAKE + 4), B.GDN_E_INVALID, 'states is not'),
    ('gdn_pool_copy', (None, FAKE, 1), B.GDN_E_INVALID, 'src is NULL'),
    ('gdn_pool_copy', (FAKE, FAKE + 2, 1), B.GDN_E_INVALID, 'dst is not'),
    ('gdn_pool_copy', (FAKE, FAKE, 65536), B.GDN_E_UNSUPPORTED, 'entries'),
    ('gdn_pool_reorder', (FAKE, FAKE, 1, 0), B.GDN_E_UNSUPPORTED, 'width'),
    ('gdn_pool_reorder', (FAKE, FAKE, 1, 33), B.GDN_E_UNSUPPORTED, 'width'),
    ('gdn_pool_reorder', (FAKE, FAKE, -1, 4), B.GDN_E_INVALID, 'groups'),
    ('gdn_pool_reorder', (FAKE, FAKE, 1 << 28, 32), B.GDN_E_UNSUPPORTED, 'groups'),
    ('gdn_pool_reorder', (FAKE, None, 1, 4), B.GDN_E_INVALID, 'parents is NULL'),
])
def test_pool_calls_check_their_arguments(name, args, status, msg):
    got, text = _call(name, ctypes.byref(_pool()), *args, None)
    assert got == status and msg in text, (got, text)


def _step(**kw):
    a = B.PoolStepArgs(B=3, T=2, Hqk=2, io_dtype=B.GDN_BF16, scale=0.1)
    for name in ('slots', 'q', 'k', 'v', 'g', 'beta', 'o'):
        setattr(a, name, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=-1), B.GDN_E_INVALID, 'sizes'),
    (dict(B=-1), B.GDN_E_INVALID, 'entries'),
    (dict(B=65536), B.GDN_E_UNSUPPORTED, 'entries'),
    (dict(Hqk=3), B.GDN_E_INVALID, 'multiple'),
    (dict(Hqk=0), B.GDN_E_INVALID, 'sizes'),
    (dict(io_dtype=2), B.GDN_E_INVALID, 'io_dtype'),
    (dict(layer=2), B.GDN_E_INVALID, 'layer'),
    (dict(readout=2), B.GDN_E_INVALID, 'readout'),
    (dict(scale=float('inf')), B.GDN_E_INVALID, 'scale'),
    (dict(q=None), B.GDN_E_INVALID, 'q is NULL'),
    (dict(beta=None), B.GDN_E_INVALID, 'beta is NULL'),
    (dict(o=FAKE + 2), B.GDN_E_INVALID, 'o is not'),
    (dict(slots=None), B.GDN_E_INVALID, 'slots is NULL'),
    (dict(slots_out=FAKE + 4), B.GDN_E_INVALID, 'slots_out is not'),
    (dict(lens=FAKE + 4), B.GDN_E_INVALID, 'lens is not'),
    (dict(q_stride=255), B.GDN_E_INVALID, 'q_stride'),
    (dict(k_stride=-256), B.GDN_E_INVALID, 'k_stride'),
    (dict(v_stride=516), B.GDN_E_INVALID, 'v_stride'),
])
def test_step_checks_its_arguments(kw, status, msg):
    got, text = _call('gdn_pool_step', ctypes.byref(_pool()), ctypes.byref(_step(**kw)), None)
    assert got == status and msg in text, (got, text)


def test_calls_without_entries_do_nothing():
    p = ctypes.byref(_pool())
    assert _call('gdn_pool_write', p, 0, None, 0, None, None)[0] == B.GDN_OK
    assert _call('gdn_pool_read', p, 0, None, 0, None, None)[0] == B.GDN_OK
    assert _call('gdn_pool_copy', p, None, None, 0, None)[0] == B.GDN_OK
    assert _call('gdn_pool_reorder', p, None, None, 0, 4, None)[0] == B.GDN_OK
    assert _call('gdn_pool_step', p, ctypes.byref(_step(B=0, slots=None, q=None)), None)[0] == B.GDN_OK


def _beam(**kw):
    a = B.BeamArgs(B=2, W=4, V=1000, K=8, io_dtype=B.GDN_BF16, logits=FAKE, scores=FAKE, out_scores=FAKE,
                   parents=FAKE, tokens=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,msg", [
    (dict(V=0), B.GDN_E_INVALID, 'sizes'),
    (dict(B=-1), B.GDN_E_INVALID, 'sizes'),
    (dict(W=0), B.GDN_E_UNSUPPORTED, 'beams'),
    (dict(W=33), B.GDN_E_UNSUPPORTED, 'beams'),
    (dict(K=0), B.GDN_E_UNSUPPORTED, 'K 0'),
    (dict(K=65), B.GDN_E_UNSUPPORTED, 'K 65'),
    (dict(V=(1 << 30) + 1), B.GDN_E_UNSUPPORTED, '2^30'),
    (dict(B=65535, W=32, V=1 << 30), B.GDN_E_UNSUPPORTED, 'too large'),
    (dict(io_dtype=5), B.GDN_E_INVALID, 'io_dtype'),
    (dict(row_stride=999), B.GDN_E_INVALID, 'row_stride'),
    (dict(logits=None), B.GDN_E_INVALID, 'logits is NULL'),
    (dict(logits=FAKE + 1), B.GDN_E_INVALID, 'logits is not 2'),
    (dict(logits=FAKE + 2, io_dtype=B.GDN_F32), B.GDN_E_INVALID, 'logits is not 4'),
    (dict(scores=FAKE + 4), B.GDN_E_INVALID, 'scores is not'),
    (dict(finished=FAKE + 1), B.GDN_E_INVALID, 'finished is not'),
    (dict(tokens=None), B.GDN_E_INVALID, 'tokens is NULL'),
    (dict(workspace=None), B.GDN_E_WORKSPACE, 'workspace'),
    (dict(workspace_bytes=16), B.GDN_E_WORKSPACE, 'needed'),
])
def test_beam_select_checks_its_arguments(kw, status, msg):
    got, text = _call('gdn_beam_select', ctypes.byref(_beam(**kw)), None)
    assert got == status and msg in text, (got, text)


def test_beam_workspace_covers_every_part():
    """8 bytes and K keys of 8 bytes per (row, split), rounded up; 0 for
    arguments that the call refuses."""
    lib = B.load_library()
    a = _beam(B=1, W=4, V=131072, K=8)
    n = lib.gdn_beam_workspace_bytes(ctypes.byref(a))
    assert n > 0 and n % 8 == 0
    more = lib.gdn_beam_workspace_bytes(ctypes.byref(_beam(B=2, W=4, V=131072, K=8)))
    assert n < more <= 2 * n + 48
    assert lib.gdn_beam_workspace_bytes(ctypes.byref(_beam(K=65))) == 0


# ------------------------------------------------------------- the binding
def _cpu_pool(fmt=B.QDQ_E4M3):
    return B.StatePool(2, 5, 4, 64, 64, fmt, 32, device='cpu')


def test_new_pool_holds_zero_states():
    p = _cpu_pool()
    assert p.data.shape == (2, 5, 4, 64, 64) and p.data.dtype is torch.float8_e4m3fn
    assert p.scales.shape == (2, 5, 4, 2) and bool((p.scales == 2.0 ** -126).all())
    assert bool((p.data.float() == 0).all())
    assert B.StatePool(1, 2, 1, 64, 64, B.QDQ_OFF, device='cpu').scales is None


@pytest.mark.parametrize("data,scales,fmt,bv", [
    (torch.zeros(1, 2, 3, 64, 64), None, B.QDQ_E4M3, 64),                       # another type
    (torch.zeros(1, 2, 3, 64, 64, dtype=torch.int8), None, B.QDQ_INT8, 64),    # no scales
    (torch.zeros(1, 2, 3, 64, 64, dtype=torch.int8), torch.ones(1, 2, 3, 2), B.QDQ_INT8, 64),
    (torch.zeros(1, 2, 3, 64, 64, dtype=torch.int8), torch.ones(1, 2, 3, 1).double(), B.QDQ_INT8, 64),
    (torch.zeros(1, 2, 3, 64, 64), torch.ones(1, 2, 3, 1), B.QDQ_OFF, 64),
    (torch.zeros(2, 3, 64, 64), None, B.QDQ_OFF, 64),
    (torch.zeros(1, 2, 3, 64, 64).transpose(3, 4), None, B.QDQ_OFF, 64),
    (torch.zeros(1, 2, 3, 64, 64, dtype=torch.int8), torch.ones(1, 2, 3, 1), B.QDQ_INT8, 48),
])
def test_pool_refuses_other_tensors(data, scales, fmt, bv):
    with pytest.raises(ValueError):
        B.StatePool.from_tensors(data, scales, fmt, bv)


def _ints(n):
    return torch.zeros(n, dtype=torch.int32)


def _inputs(Bn=2, T=3, dt=torch.bfloat16):
    return dict(q=torch.zeros(Bn, T, 2, 64, dtype=dt), k=torch.zeros(Bn, T, 2, 64, dtype=dt),
                v=torch.zeros(Bn, T, 4, 64, dtype=dt), g=torch.zeros(Bn, T, 4),
                beta=torch.zeros(Bn, T, 4), slots=_ints(Bn))


@pytest.mark.parametrize("change,msg", [
    (dict(q=torch.zeros(2, 3, 2, 64, dtype=torch.float16)), 'bfloat16 or float32'),
    (dict(q=torch.zeros(2, 3, 128, dtype=torch.bfloat16)), 'q: '),
    (dict(k=torch.zeros(2, 3, 2, 64)), 'k: '),
    (dict(v=torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)), 'v: '),
    (dict(k=torch.zeros(2, 3, 64, 2, dtype=torch.bfloat16).transpose(2, 3)), 'contiguous'),
    (dict(k=torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16).transpose(0, 1)), 'evenly'),
    (dict(q=torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16).expand(2, 3, 2, 64)), 'evenly'),
    (dict(v=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16).expand(2, 3, 4, 64)), 'evenly'),
    (dict(g=torch.zeros(2, 3, 4).double()), 'g: '),
    (dict(g=torch.zeros(2, 4, 3).transpose(1, 2)), 'not contiguous'),
    (dict(beta=torch.zeros(2, 3, 2)), 'beta: '),
    (dict(slots=torch.zeros(2, dtype=torch.int64)), 'slots: '),
    (dict(slots_out=_ints(3)), 'slots_out: '),
    (dict(lens=torch.zeros(2)), 'lens: '),
    (dict(out=torch.zeros(2, 3, 4, 64)), 'out: '),
    ({}, 'GPU'),                                       # everything fits, but lives on the CPU
])
def test_step_refuses_other_tensors(change, msg):
    x = {**_inputs(), **change}
    with pytest.raises(ValueError, match=msg):
        B.gdn_pool_step(_cpu_pool(), 0, x.pop('slots'), **x)


def test_page_calls_refuse_other_tensors():
    p = _cpu_pool()
    for call in (lambda: B.gdn_pool_write(p, 0, _ints(2), torch.zeros(2, 4, 64, 128)),
                 lambda: B.gdn_pool_write(p, 0, _ints(2).long(), torch.zeros(2, 4, 64, 64)),
                 lambda: B.gdn_pool_write(p, 0, _ints(2), torch.zeros(2, 4, 64, 64).mT),
                 lambda: B.gdn_pool_read(p, 0, _ints(2), out=torch.zeros(1, 4, 64, 64)),
                 lambda: B.gdn_pool_copy(p, _ints(2), _ints(3)),
                 lambda: B.gdn_pool_copy(p, _ints(4)[::2], _ints(2)),
                 lambda: B.gdn_pool_reorder(p, _ints(4), _ints(4)),
                 lambda: B.gdn_pool_reorder(p, _ints(4).view(2, 2), _ints(4)),
                 lambda: B.gdn_pool_copy(p, _ints(2), _ints(2))):
        with pytest.raises(ValueError):
            call()


def test_beam_select_refuses_other_tensors():
    x, s = torch.zeros(2, 3, 50), torch.zeros(2, 3)
    for call in (lambda: B.gdn_beam_select(x.half(), s), lambda: B.gdn_beam_select(x[0], s),
                 lambda: B.gdn_beam_select(x, s.double()), lambda: B.gdn_beam_select(x, s[:1]),
                 lambda: B.gdn_beam_select(x.transpose(0, 1), s.T),
                 lambda: B.gdn_beam_select(torch.zeros(2, 50, 3).mT, s),
                 lambda: B.gdn_beam_select(torch.zeros(2, 1, 50).expand(2, 3, 50), s),
                 lambda: B.gdn_beam_select(x, s, finished=torch.zeros(2, 3)),
                 lambda: B.gdn_beam_select(x, s),
                 lambda: B.gdn_beam_advance(_cpu_pool(), _ints(6), x, s)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.GdnError, match='K 65'):
        B.gdn_beam_select(x, s, 65)


@pytest.mark.parametrize("name", ['g', 'beta'])
def test_gates_are_aligned_to_an_element(name):
    got, text = _call('gdn_pool_step', ctypes.byref(_pool()), ctypes.byref(_step(**{name: FAKE + 2})), None)
    assert got == B.GDN_E_INVALID and f'{name} is not 4-byte' in text, (got, text)
    # at 4 bytes the next check speaks, not this one
    got, text = _call('gdn_pool_step', ctypes.byref(_pool()), ctypes.byref(_step(**{name: FAKE + 4}, q_stride=255)), None)
    assert got == B.GDN_E_INVALID and 'q_stride' in text, (got, text)
