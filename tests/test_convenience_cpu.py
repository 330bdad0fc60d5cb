"""decode and decode_prefix, which allocate for the caller, with a stream given: everything that
they allocate and copy belongs to that stream.  Nothing is launched: the calls that would are
recorded instead."""
import contextlib

import numpy as np
import pytest

import paged_mla_decode_latent_gb300 as mla


class Stream:
    cuda_stream = 4096


class Lens:
    """seq_lens whose copy to the host is recorded."""
    shape = (2,)

    def __init__(self, note):
        self.note = note

    def cpu(self):
        self.note("cpu")
        return np.array([300, 290], np.int32)


@pytest.fixture
def recorded(monkeypatch):
    import torch
    mla.build()
    log, active, kept = [], [None], []
    note = lambda what: log.append((what, active[0]))  # noqa: E731

    @contextlib.contextmanager
    def on(s):
        before, active[0] = active[0], s
        yield
        active[0] = before

    empty, plan, prefix_plan = torch.empty, mla.plan, mla.prefix_plan
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[0] or "current")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a, **k: ("external", h))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (note("empty"), empty(*a, **k))[1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((tuple(t.shape), s)))
    for name in ("fwd", "combine", "prefix_fwd"):
        monkeypatch.setattr(mla, name, lambda *a, _n=name, **k: note(_n))
    # The host plans ask no GPU for its SMs here.
    monkeypatch.setattr(mla, "plan", lambda *a, **k: plan(*a, num_sms=152, **k))
    monkeypatch.setattr(mla, "prefix_plan", lambda *a, **k: prefix_plan(*a, num_sms=152, **k))
    return log, kept, note


def call(which, note, **kw):
    import torch
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16)
    cache = torch.zeros(40, 16, 576, dtype=torch.bfloat16)
    bt = torch.zeros(2, 19, dtype=torch.int32)
    if which == "decode":
        return mla.decode(q, cache, bt, Lens(note), **kw)
    return mla.decode_prefix(q, cache, bt[0], bt, Lens(note), 256, **kw)


@pytest.mark.parametrize("which", ["decode", "decode_prefix"])
@pytest.mark.parametrize("stream,on", [(Stream(), None), (4096, ("external", 4096)), (0, "default"), (1, "default")])
def test_a_given_stream_owns_what_is_allocated(recorded, which, stream, on):
    log, kept, note = recorded
    out, lse = call(which, note, stream=stream)
    on = on or stream
    assert {w for w, _ in log} >= {"cpu", "empty"} | ({"fwd", "combine"} if which == "decode" else {"prefix_fwd"})
    assert [w for w, _ in log].count("empty") == 3  # out, lse, workspace
    assert all(s == on for _, s in log), log
    # The caller goes on using the results on the current stream.
    assert kept == [(tuple(out.shape), "current"), (tuple(lse.shape), "current")]


@pytest.mark.parametrize("which", ["decode", "decode_prefix"])
def test_without_a_stream_the_current_one_does(recorded, which):
    log, kept, note = recorded
    call(which, note)
    assert all(s is None for _, s in log) and kept == []


@pytest.mark.parametrize("plan_causal", [False, True])
def test_a_plan_for_something_else_is_refused(recorded, plan_causal):
    """The plan's prefix length and mask are the call's: arguments that contradict it raise."""
    log, _, note = recorded
    p = mla.prefix_plan([300, 290], 256, 16, 1, 16, mla.KV_BF16, plan_causal)
    call("decode_prefix", note, p=p)
    call("decode_prefix", note, p=p, causal=plan_causal)
    with pytest.raises(mla.MLADecodeError) as e:
        call("decode_prefix", note, p=p, causal=not plan_causal)
    assert e.value.status == mla.ERR_INVALID_ARG
    with pytest.raises(mla.MLADecodeError) as e:
        call("decode_prefix", note, p=mla.prefix_plan([300, 290], 255, 16, 1, 16, mla.KV_BF16, plan_causal))
    assert e.value.status == mla.ERR_INVALID_ARG
    assert [w for w, _ in log].count("prefix_fwd") == 2
