"""decode and decode_prefix on a stream of the caller's, while the current stream goes on allocating
and writing: nothing that the call allocated is handed out under it."""
import numpy as np
import pytest

from parity import assert_close
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["decode", "decode_prefix"])
@pytest.mark.parametrize("handle", [False, True])
def test_allocations_follow_the_stream(which, handle):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(8, 1, 64, [2000 + 7 * i for i in range(8)], 1984, 16, seed=2)
    t = p.to_device()
    full = t["bt"].clone()
    full[:, :124] = t["pt"]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        stream = s.cuda_stream if handle else s
        if which == "decode":
            got.append(mla.decode(t["q"], t["cache"], full, t["lens"], softmax_scale=p.scale, stream=stream))
        else:
            got.append(mla.decode_prefix(t["q"], t["cache"], t["pt"], full, t["lens"], 1984, softmax_scale=p.scale,
                                         stream=stream))
        # Blocks of the sizes just freed, on the current stream, full of what no step leaves behind.
        for n in (1 << 10, 1 << 20, 8 << 20, 32 << 20):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.current_stream().wait_stream(s)
    ref = p.reference()
    for out, lse in got:
        assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, which)


def test_results_outlive_their_stream():
    """Results read on the current stream and dropped: the next call on the stream does not write there first."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(4, 1, 128, [600 + i for i in range(4)], 590, 16, seed=3)
    t = p.to_device()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for _ in range(8):
        out, lse = mla.decode_prefix(t["q"], t["cache"], t["pt"], t["bt"], t["lens"], 590, seq_lens_host=p.lens,
                                     softmax_scale=p.scale, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(2_000_000)  # the reader is late
        kept.append((out * 1, lse * 1))
        del out, lse
    torch.cuda.synchronize()
    first = kept[0]
    assert np.isfinite(first[1].cpu().numpy()).all()
    for out, lse in kept[1:]:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
