"""Refusals of the rotating epilogue: every one comes before anything is queued."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def call(**kw):
    a = dict(ql=1 << 20, ql_t=512 * 16, ql_h=512, qp=2 << 20, qp_t=64 * 16, qp_h=64, kc=3 << 20,
             kc_t=512, kp=4 << 20, kp_t=64, pos=5 << 20, cs=6 << 20, max_pos=100, inter=1,
             slots=7 << 20, T=4, H=16, q_out=8 << 20, cache=9 << 20, pages=10, ps=16, dtype=0,
             scale=None, early=0, status=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.lib().mla_decode_rope_epilogue(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(ql=None), dict(qp=None), dict(kc=None), dict(kp=None), dict(pos=None), dict(cs=None),
    dict(slots=None), dict(q_out=None), dict(cache=None), dict(T=-1), dict(H=0), dict(H=129),
    dict(pages=0), dict(ps=0), dict(dtype=2), dict(dtype=1), dict(inter=2), dict(early=2),
    dict(max_pos=0), dict(ql_t=-8), dict(ql_h=4), dict(qp_t=12), dict(qp_h=-64), dict(kc_t=2),
    dict(kp_t=-512), dict(ql=(1 << 20) + 8), dict(qp=(2 << 20) + 2), dict(kc=(3 << 20) + 4),
    dict(kp=(4 << 20) + 8), dict(cs=(6 << 20) + 4), dict(pos=(5 << 20) + 4), dict(slots=(7 << 20) + 4),
    dict(q_out=(8 << 20) + 8), dict(cache=(9 << 20) + 8), dict(dtype=1, scale=(1 << 20) + 2),
    dict(status=(1 << 20) + 1)])
def test_refuses(kw):
    assert call(**kw) == mla.ERR_INVALID_ARG


def test_too_many_rows():
    assert call(T=1 << 25, H=128, ql_t=8, qp_t=8) == mla.ERR_UNSUPPORTED


def test_no_tokens_queue_nothing():
    assert call(T=0) == mla.OK


def test_binding_refuses_host_tensors():
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(mla.MLADecodeError) as e:
        mla.rope_epilogue(z(2, 4, 512), z(2, 4, 64), z(2, 512), z(2, 64), torch.zeros(2, dtype=torch.int64),
                          torch.zeros(10, 64), torch.zeros(2, dtype=torch.int64), z(2, 4, 576), z(3, 16, 576))
    assert e.value.status == mla.ERR_INVALID_ARG
