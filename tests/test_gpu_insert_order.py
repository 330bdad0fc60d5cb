"""The insert without rotation right behind the kernel that writes its slots."""
import numpy as np
import pytest

from pages_book import Book, Gpu

pytestmark = pytest.mark.gpu


def bf(rng, *shape):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def test_slots_from_the_kernel_before():
    """The slots are what the kernel before writes last: it lets this one start early, and copies them, as the bits of
    its query rows, while this one already runs.  What lay there before were slots too."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    T, H, n, pages, page = 512, 128, 128, 40, 16
    rng = np.random.default_rng(1)
    ql, qp, kc, kp = bf(rng, T, H, 512), bf(rng, T, H, 64), bf(rng, T, 512), bf(rng, T, 64)
    q = torch.empty(T, H, 576, dtype=torch.bfloat16, device="cuda")
    slots = q[T - 1, H - 1, :512].view(torch.int64)
    positions, nowhere = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.full((T,), -1, device="cuda")
    cos_sin = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()
    cache = torch.zeros(pages, page, 576, dtype=torch.bfloat16, device="cuda")
    a = [bf(rng, n, 8, 512), bf(rng, n, 8, 64), bf(rng, n, 512), bf(rng, n, 64)]
    rows, q2 = torch.cat(a[2:], 1), torch.empty(n, 8, 576, dtype=torch.bfloat16, device="cuda")
    for k in range(20):
        now, old = (torch.from_numpy(rng.permutation(pages * page)[:n]).cuda() for _ in range(2))
        ql[T - 1, H - 1] = now.view(torch.bfloat16)
        slots.copy_(old)
        cache.zero_()
        want = torch.zeros(pages * page, 576, dtype=torch.bfloat16, device="cuda")
        want[now] = rows
        torch.cuda.synchronize()
        mla.rope_epilogue(ql, qp, kc, kp, positions, cos_sin, nowhere, q, cache)
        mla.epilogue(*a, slots, q2, cache)
        assert torch.equal(slots, now)
        assert torch.equal(cache.view(-1, 576), want), k


@pytest.mark.parametrize("pages,page,width", [(200, 16, 20), (33000, 2, 160)])  # one launch a call, a kernel a step
def test_insert_right_behind_a_resize(pages, page, width):
    """Rows grow, shrink and end; each call's tokens go where that call says, eager and in a graph."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    B, tokens, heads = 5, 3, 4
    rng = np.random.default_rng(4)
    b = Book(pages, page, B, width, 1, 1152, 3)
    b.scatter(2, 0.2)
    g = Gpu(b)
    lens = [[30, 0, 7, 64, 1], [33, 3, 0, 67, 4], [5, 6, 100, 70, 7], [8, 0, 103, 73, 10], [0, 40, 106, 76, 13]]
    new = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in lens]
    ins = [[bf(rng, B * tokens, heads, 512), bf(rng, B * tokens, heads, 64), bf(rng, B * tokens, 512), bf(rng, B * tokens, 64)]
           for _ in lens]
    slots = torch.empty(B, tokens, dtype=torch.int64, device="cuda")
    q = torch.empty(B * tokens, heads, 576, dtype=torch.bfloat16, device="cuda")
    cache = g.cache[0].view(torch.bfloat16)

    def steps():
        for n, x in zip(new, ins):
            mla.pages_resize(g.refs, g.table, g.lens, n, page, g.ws, slots, g.status)
            mla.epilogue(*x, slots.view(-1), q, cache, status=g.status)

    start = [x.clone() for x in (g.refs, g.table, g.lens, g.cache)]
    for x, n in zip(ins, lens):
        row = torch.cat(x[2:], 1).contiguous().view(torch.uint8).cpu().numpy()
        for at, one in zip(b.resize(n, tokens)[0].ravel(), row):
            if at >= 0:
                b.cache[0, at // page, at % page] = one
    steps()
    g.same_as(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(10):
        for x, y in zip((g.refs, g.table, g.lens, g.cache), start):
            x.copy_(y)
        graph.replay()
        g.same_as(b)
    assert g.flags() == 0
