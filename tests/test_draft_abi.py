"""Host-side argument checks of the draft-model calls: every refusal happens
before any GPU work (so no GPU is needed for these calls)."""
import ctypes
import os

import pytest
import torch

import draft_token_verification_vocab_amd as sv

# fake device addresses that host-side validation must reject
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device pointers: host-only validation test")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sv.lib_path()):
        from draft_token_verification_vocab_amd import build
        build.build()
    return sv.load()


@host_only
def test_row_topk_validates_on_host(L):
    P = ctypes.c_void_p
    a = P(16)

    def call(logits=a, rows=4, V=1024, S=1024, dt=1, T=1.0, k=8, values=a, ids=a):
        return L.spec_row_topk(logits, rows, V, S, dt, T, k, values, ids, None, None)
    assert call(rows=0, logits=None, values=None, ids=None) == 0
    for kw in (dict(rows=-1), dict(k=0), dict(V=1), dict(S=1000), dict(S=1028), dict(dt=7),
               dict(T=0.0), dict(T=float("nan")), dict(logits=P(8)), dict(logits=None),
               dict(values=None), dict(ids=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(k=129), dict(V=(1 << 20) + 8, S=(1 << 20) + 8), dict(rows=1 << 31)):
        assert call(**kw) == -2, kw


@host_only
def test_distill_validates_on_host(L):
    P = ctypes.c_void_p
    a = P(16)

    def params(**kw):
        base = dict(rows=4, vocab=1024, dtype=1, row_stride=1024, k=8, temperature=1.0, reserved=0)
        base.update(kw)
        return ctypes.byref(sv._DistillParams(**base))

    def loss(student=a, ids=a, logits=a, p=None, out=a, state=a, **kw):
        return L.spec_distill_loss(student, ids, logits, None, None, p or params(**kw), out, state,
                                   None)

    def grad(student=a, ids=a, logits=a, state=a, out=a, **kw):
        return L.spec_distill_grad(student, ids, logits, state, None, params(**kw), out, None)

    def step(student=a, ids=a, logits=a, out=a, g=a, **kw):
        return L.spec_distill_step(student, ids, logits, None, None, None, params(**kw), out, g,
                                   None)
    for call in (loss, grad, step):
        for kw in (dict(rows=-1), dict(k=0), dict(vocab=1), dict(row_stride=1000),
                   dict(row_stride=1028), dict(dtype=7), dict(temperature=0.0),
                   dict(temperature=float("nan")), dict(reserved=1), dict(student=None),
                   dict(student=P(8)), dict(ids=None), dict(logits=None), dict(out=None)):
            assert call(**kw) == -1, kw
        for kw in (dict(k=129), dict(vocab=(1 << 20) + 8, row_stride=(1 << 20) + 8),
                   dict(rows=1 << 40), dict(row_stride=1 << 31)):
            assert call(**kw) == -2, kw
        assert call(rows=0, student=None, ids=None, logits=None, out=None) == 0
    assert L.spec_distill_loss(a, a, a, None, None, None, a, a, None) == -1
    assert loss(state=P(8)) == -1
    assert grad(state=None) == -1 and grad(state=P(8)) == -1 and grad(out=P(8)) == -1
    assert step(g=None) == -1 and step(g=P(8)) == -1
    # the gradient replaces the logits exactly or not at all (4 rows of 2048 bytes)
    base = P(1 << 20)
    for g in ((1 << 20) + 16, (1 << 20) - 16, (1 << 20) + 8176):
        assert step(student=base, g=P(g)) == -1 and grad(student=base, out=P(g)) == -1
    assert L.spec_distill_state_bytes(7) == 7 * 48 and L.spec_distill_state_bytes(0) == 0
    assert L.spec_distill_state_bytes(-1) == 0


@host_only
def test_distill_refuses_row_counts_whose_products_pass_64_bits(L):
    a = ctypes.c_void_p(16)
    for rows, stride in (((1 << 62) + 1, 16384), ((1 << 63) - 1, 1 << 20), (1 << 61, 1 << 20),
                         ((1 << 32) + 5, 1024)):
        p = sv._DistillParams(rows=rows, vocab=1024, dtype=1, row_stride=stride, k=8,
                              temperature=1.0, reserved=0)
        p = ctypes.byref(p)
        assert L.spec_distill_loss(a, a, a, None, None, p, a, a, None) == -2, rows
        assert L.spec_distill_grad(a, a, a, a, None, p, a, None) == -2, rows
        assert L.spec_distill_step(a, a, a, None, None, None, p, a, a, None) == -2, rows


@host_only
def test_distill_takes_the_batches_that_its_launches_hold(L):
    # without a GPU a call that passes every check ends in a failed launch (-4)
    s, g, x = (ctypes.c_void_p(1 << n) for n in (40, 44, 46))

    def calls(rows, vocab, stride, dtype):
        p = ctypes.byref(sv._DistillParams(rows=rows, vocab=vocab, dtype=dtype, row_stride=stride,
                                           k=8, temperature=1.0, reserved=0))
        return (L.spec_distill_loss(s, x, x, None, None, p, x, x, None),
                L.spec_distill_step(s, x, x, None, None, None, p, x, g, None),
                L.spec_distill_grad(s, x, x, x, None, p, g, None))
    for case in ((131072, 152064, 152064, 1), (1 << 21, 4100, 4104, 1), ((1 << 22) - 1, 8, 8, 0)):
        assert calls(*case) == (-4, -4, -4), case
    assert calls(1 << 22, 8, 8, 0) == (-2, -2, -2)
    # rows of 512 KiB are eight parts for the gradient alone
    assert calls((1 << 21) - 1, 131072, 131072, 0) == (-4, -4, -4)
    assert calls(1 << 21, 131072, 131072, 0) == (-4, -4, -2)


@host_only
def test_beam_select_validates_on_host(L):
    P = ctypes.c_void_p
    a, big = P(16), 1 << 30

    def call(logits=a, S=1024, scores=a, B=4, W=4, V=1024, dt=1, T=1.0, n=8, out=a, par=a, tok=a,
             ws=a, size=big):
        return L.spec_beam_select(logits, S, scores, None, B, W, V, dt, T, n, 2, out, par, tok,
                                  None, ws, size, None)
    assert call(B=0, logits=None, scores=None, out=None, ws=None) == 0
    for kw in (dict(B=-1), dict(W=0), dict(n=0), dict(V=1), dict(S=1000), dict(S=1028),
               dict(dt=7), dict(T=0.0), dict(T=float("inf")), dict(logits=None),
               dict(logits=P(8)), dict(scores=None), dict(out=None), dict(par=None),
               dict(tok=None), dict(ws=P(8))):
        assert call(**kw) == -1, kw
    for kw in (dict(W=33), dict(n=65), dict(W=32, n=17), dict(V=(1 << 20) + 8, S=(1 << 20) + 8),
               dict(B=1 << 30, W=32)):
        assert call(**kw) == -2, kw
    need = L.spec_beam_workspace_bytes(4, 4, 1024, 1, 8)
    assert need > 0
    assert call(ws=None) == -3 and call(size=need - 1) == -3
    assert L.spec_beam_workspace_bytes(4, 33, 1024, 1, 8) == 0
    assert L.spec_beam_workspace_bytes(0, 4, 1024, 1, 8) == 0


@host_only
def test_beam_reorder_validates_on_host(L):
    P = ctypes.c_void_p
    a = P(16)

    def call(B=2, W=4, n=4, par=a, count=1, states=True, **kw):
        base = dict(src=1 << 20, dst=1 << 30, position_bytes=16, segments=2, positions=8)
        base.update(kw)
        st = (sv._BeamState * 1)(sv._BeamState(**base))
        return L.spec_beam_reorder(par, None, B, W, n, st if states else None, count, None)
    assert call(B=0, par=None) == 0 and call(count=0, par=None, states=False) == 0
    for kw in (dict(B=-1), dict(W=0), dict(n=0), dict(count=-1), dict(par=None),
               dict(states=False), dict(src=None), dict(dst=None), dict(position_bytes=0),
               dict(segments=0), dict(positions=-1),
               dict(dst=1 << 20, n=3),                     # in place means beam for beam
               dict(dst=(1 << 20) + 16),                   # other overlaps
               dict(src=(1 << 30) + 2 * 4 * 256 - 16)):
        assert call(**kw) == -1, kw
    # two states: a dst twice, or one state's dst in the other's src
    def two(a, b):
        st = (sv._BeamState * 2)(*[sv._BeamState(s, d, 16, 2, 8) for s, d in (a, b)])
        return L.spec_beam_reorder(P(16), None, 2, 4, 4, st, 2, None)
    x, y, z = 1 << 20, 1 << 21, 1 << 22
    for pair in (((x, x), (x, x)), ((x, y), (z, y)), ((x, y), (y, z)), ((y, z), (x, y)),
                 ((x, y), (z, y + 2032)), ((x, x), (x + 16, z))):
        assert two(*pair) == -1, pair
    for kw in (dict(W=33), dict(n=65), dict(position_bytes=1 << 31),
               dict(position_bytes=1 << 30, positions=1 << 30, segments=1 << 10),
               dict(B=1 << 30, dst=1 << 60)):
        assert call(**kw) == -2, kw


@host_only
def test_beam_reorder_takes_each_state_by_its_own_size(L):
    # without a GPU a call that passes every check ends in a failed launch (-4)
    def call(*states, B=1):
        st = (sv._BeamState * len(states))(*[sv._BeamState(*s) for s in states])
        return L.spec_beam_reorder(ctypes.c_void_p(16), None, B, 4, 4, st, len(states), None)
    cache = (1 << 40, 1 << 44, 256, 2, 1 << 24)          # 8 GiB a beam, in 16-byte units
    flags = (1 << 46, 1 << 47, 1, 1, 37)                 # 37 single bytes
    assert call(cache) == -4 and call(flags) == -4
    assert call(cache, flags) == -4 and call(flags, cache) == -4
    # more workgroups in all than one launch holds, fewer in each state
    many = [((1 << 40) + (i << 34), (1 << 45) + (i << 34), 20, 1, (1 << 31) // 20)
            for i in range(16)]
    assert call(*many) == -4
    # a state that one launch cannot hold: 64 GiB, 16 GiB and 4 GiB a beam
    for unit, positions, segments in ((16, 1 << 28, 16), (4, 1 << 28, 16), (1, 1 << 28, 16)):
        over = (1 << 50, 1 << 54, unit, segments, positions)
        under = (1 << 50, 1 << 54, unit, segments - 1, positions)
        assert call(over) == -2 and call(cache, over) == -2, unit
        assert call(under) == -4, unit


def test_binding_refuses_host_tensors_and_wrong_shapes():
    f, i = torch.zeros(2, 3, 8), torch.zeros(2, 3, 4, dtype=torch.int32)
    for call in (lambda: sv.row_topk(f, 2), lambda: sv.distill_loss(f, i, i.float()),
                 lambda: sv.distill_step(f, i, i.float()),
                 lambda: sv.distill_grad(f, i, i.float(), torch.zeros(240, dtype=torch.uint8)),
                 lambda: sv.beam_select(f, torch.zeros(2, 3), 2),
                 lambda: sv.beam_reorder(torch.zeros(2, 3, dtype=torch.int32), [f])):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_long_runs_are_cut_into_positions_that_keep_their_unit():
    for nbytes, unit in ((2 ** 31, 16), (2 ** 31 + 16, 16), (2 ** 33 + 48, 16), (2 ** 31 + 1, 1),
                         (5 * 10 ** 9 + 4, 4), (2 ** 32 + 2, 1), (3 * 2 ** 34, 16)):
        n = sv._positions(nbytes)
        assert nbytes % n == 0 and nbytes // n <= 2 ** 31 - 1 and nbytes // n % unit == 0, nbytes
    assert sv._positions(2147483659) == 1            # a prime past 2^31: refused by the library
