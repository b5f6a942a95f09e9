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
    a, big = P(16), 1 << 30

    def call(logits=a, rows=4, V=1024, S=1024, dt=1, T=1.0, k=8, values=a, ids=a, ws=a, n=big):
        return L.spec_row_topk(logits, rows, V, S, dt, T, k, values, ids, None, ws, n, None)
    assert call(rows=0, logits=None, values=None, ids=None, ws=None) == 0
    for kw in (dict(rows=-1), dict(k=0), dict(V=1), dict(S=1000), dict(S=1028), dict(dt=7),
               dict(T=0.0), dict(T=float("nan")), dict(logits=P(8)), dict(logits=None),
               dict(values=None), dict(ids=None), dict(V=40000, S=40000, ws=P(8))):
        assert call(**kw) == -1, kw
    for kw in (dict(k=129), dict(V=(1 << 20) + 8, S=(1 << 20) + 8), dict(rows=1 << 31)):
        assert call(**kw) == -2, kw
    # four long rows are cut into segments, whose lists need the workspace
    need = L.spec_row_topk_workspace_bytes(4, 40000, 1, 8)
    assert need > 0 and need % 256 == 0
    assert call(V=40000, S=40000, ws=None) == -3
    assert call(V=40000, S=40000, n=need - 1) == -3
    assert L.spec_row_topk_workspace_bytes(300, 40000, 1, 8) == 0   # a workgroup per row
    assert L.spec_row_topk_workspace_bytes(4, 40000, 1, 129) == 0


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
    assert L.spec_distill_state_bytes(7) == 280 and L.spec_distill_state_bytes(0) == 0
    assert L.spec_distill_state_bytes(-1) == 0
