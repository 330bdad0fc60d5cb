"""The page calls on the GPU against the plain book: whole numbers and bytes, equal everywhere."""
import numpy as np
import pytest

import fp4_rows as f4
from pages_book import Book, Gpu
from parity import assert_close

pytestmark = pytest.mark.gpu


def started(pages, page, rows, width, layers=1, row=16, seed=0, keep=0.3, fill=0.7):
    """A book with scattered holes and rows of random lengths, and its twin on the GPU."""
    rng = np.random.default_rng(seed)
    b = Book(pages, page, rows, width, layers, row, seed)
    b.scatter(seed, keep)
    room = int(len(b.free()) * fill)
    lens = np.zeros(rows, np.int64)
    for r in rng.permutation(rows):
        h = int(rng.integers(0, min(width, max(1, room)) + 1)) if room else 0
        room -= h
        lens[r] = max(0, h * page - int(rng.integers(0, page)))
    b.resize(lens)
    return b, Gpu(b, extra=int(rng.integers(0, 5)))


SIZES = [(1, 1, 1, 1), (9, 7, 3, 4), (100, 16, 5, 40), (4096, 1, 33, 300), (4097, 3, 8, 600), (8192, 64, 64, 100),
         (20001, 16, 70, 2500), (513, 4096, 4, 3),
         (40001, 2, 50, 900), (300, 16, 600, 500)]  # these two: a kernel a step


@pytest.mark.parametrize("pages,page,rows,width", SIZES)
@pytest.mark.parametrize("tokens", [0, 1, 5])
def test_resize(pages, page, rows, width, tokens):
    b, g = started(pages, page, rows, width, row=16, seed=pages + tokens)
    rng = np.random.default_rng(tokens)
    for step in range(4):
        most = width * page
        new = np.array([rng.choice([0, n, n + 1, n + tokens, n // 2, int(rng.integers(0, most + 1))]) for n in b.lens])
        new = np.clip(new, 0, most)
        slots, out = b.resize(new, tokens)
        got = g.resize(new, tokens)
        g.same_as(b, step)
        if tokens:
            assert np.array_equal(got.cpu().numpy(), slots), step
        assert (g.flags() & g.mla.DEVFLAG_NO_PAGES != 0) == out


@pytest.mark.parametrize("pages,page,rows,width", SIZES)
@pytest.mark.parametrize("layers,row", [(1, 16), (3, 48)])
def test_fork(pages, page, rows, width, layers, row):
    b, g = started(pages, page, rows, width, layers, row, seed=pages, fill=0.5)
    rng = np.random.default_rng(layers)
    for step, n in enumerate([rows, 2 * rows, max(1, rows // 2), rows]):
        parents = rng.integers(-1, len(b.lens), n)
        table = np.full((n, width + step), -3, np.int32)
        out = b.fork(parents, table.copy())
        g.fork(parents, table)
        g.same_as(b, step)
        assert g.flags() == (g.mla.DEVFLAG_NO_PAGES if out else 0)


@pytest.mark.parametrize("pages,page,rows,width", SIZES)
@pytest.mark.parametrize("layers,row", [(1, 16), (2, 416)])
def test_compact(pages, page, rows, width, layers, row):
    if pages * page * layers * row > 1 << 28:
        row = 16
    b, g = started(pages, page, rows, width, layers, row, seed=pages + row)
    for step in range(3):
        where, n = b.compact()
        got, m = g.compact()
        g.same_as(b, step)
        assert np.array_equal(got.cpu().numpy(), where) and int(m) == n and g.flags() == 0
        new = [int(x) // (step + 2) for x in b.lens]
        b.resize(new)
        g.resize(new)


@pytest.mark.parametrize("live", ["none", "all", "first half", "second half"])
@pytest.mark.parametrize("pages", [4096, 8192, 5000, 8, 40000])
def test_compact_at_the_ends(live, pages):
    b = Book(pages, 2, 1, 1, seed=2)
    held = {"none": slice(0), "all": slice(None), "first half": slice(pages // 2), "second half": slice(pages // 2, None)}[live]
    b.refs[held] = 3
    g = Gpu(b)
    where, n = b.compact()
    got, m = g.compact()
    g.same_as(b)
    assert np.array_equal(got.cpu().numpy(), where) and int(m) == n


def test_compact_without_a_table():
    b = Book(300, 4, 1, 1, layers=2, row=32, seed=3)
    b.scatter(3)
    g = Gpu(b)
    where, n = b.compact()
    got, m = g.torch.empty_like(g.refs), g.torch.empty(1, dtype=g.torch.int32, device="cuda")
    g.mla.pages_compact(g.refs, None, None, g.cache, got, m, g.ws)
    g.same_as(b)
    assert np.array_equal(got.cpu().numpy(), where) and int(m) == n


def test_many_rows():
    b, g = started(3000, 2, 1500, 4, row=16, seed=8)
    parents = np.random.default_rng(1).integers(-1, 1500, 2000)
    table = np.zeros((2000, 4), np.int32)
    out = b.fork(parents, table.copy())
    g.fork(parents, table)
    g.same_as(b)
    assert g.flags() == (g.mla.DEVFLAG_NO_PAGES if out else 0)
    new = np.random.default_rng(2).integers(0, 9, 2000)
    slots, _ = b.resize(new, 3)
    assert np.array_equal(g.resize(new, 3).cpu().numpy(), slots)
    g.same_as(b)


def test_one_row_asks_for_more_than_there_is():
    b = Book(50, 4, 3, 4000, seed=1)
    g = Gpu(b)
    b.resize([40, 16000, 8])
    g.resize([40, 16000, 8])
    g.same_as(b)
    assert list(b.lens) == [40, 0, 0] and g.flags() == g.mla.DEVFLAG_NO_PAGES
    b.resize([0, 100, 100])  # pages given back in a call serve it
    g.resize([0, 100, 100])
    g.same_as(b)


@pytest.mark.parametrize("seed", range(4))
def test_a_long_mixed_history(seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([1, 3, 16]))
    b, g = started(700, page, 9, 60, 2, 32, seed=seed)
    for step in range(25):
        kind = rng.integers(0, 4)
        if kind == 0:
            parents = rng.integers(-1, len(b.lens), int(rng.integers(1, 14)))
            table = rng.integers(0, 9, (len(parents), 60)).astype(np.int32)
            b.fork(parents, table.copy())
            g.fork(parents, table)
        elif kind == 1:
            b.compact()
            g.compact()
        else:
            # as a caller may: a row grows in its last page only where nobody else holds it
            new = []
            for r, n in enumerate(map(int, b.lens)):
                m = int(np.clip(rng.choice([0, n - 2, n + 1, n + 40]), 0, 60 * page))
                if m > n and n % page and b.refs[b.table[r, n // page]] > 1:
                    m = n
                new.append(m)
            slots, _ = b.resize(new, 2)
            assert np.array_equal(g.resize(new, 2).cpu().numpy(), slots)
        g.same_as(b, (step, kind))
        assert g.flags() & ~g.mla.DEVFLAG_NO_PAGES == 0


def test_flags():
    m = Gpu(Book(4, 4, 1, 1)).mla

    def fresh():
        b = Book(40, 4, 3, 8, row=16, seed=4)
        b.resize([10, 7, 0])
        return b, Gpu(b)

    b, g = fresh()
    g.fork([0, 3, -2], np.zeros((3, 8), np.int32))
    assert g.flags() == m.DEVFLAG_BAD_ROW and g.lens.tolist() == [10, 0, 0]
    b, g = fresh()
    g.resize([33, -1, 5])  # 32 is what the table holds
    assert g.flags() == m.DEVFLAG_CTX_RANGE and g.lens.tolist() == [32, 0, 5]
    for bad in (40, -1, 1 << 30):
        b, g = fresh()
        g.table[0, 1] = bad
        g.resize([0, 7, 0])
        assert g.flags() == m.DEVFLAG_BAD_PAGE and int(g.refs.sum()) == 3  # of row 1 two, and the one that row 0 does not name
        b, g = fresh()
        g.table[0, 2] = bad
        before = g.cache.clone()
        g.fork([0, 0, 1], np.zeros((3, 8), np.int32))  # a copy from a page that does not exist is none
        assert g.flags() == m.DEVFLAG_BAD_PAGE and g.torch.equal(g.cache, before)
        b, g = fresh()
        g.table[0, 1] = bad
        g.compact()
        assert g.flags() == m.DEVFLAG_BAD_PAGE and int(g.table[0, 1]) == bad
    b, g = fresh()
    g.refs[int(g.table[0, 0])] = 0
    g.resize([0, 7, 0])
    assert g.flags() & m.DEVFLAG_REFS
    b, g = fresh()
    g.refs[int(g.table[1, 1])] = 0
    g.compact()
    assert g.flags() == m.DEVFLAG_REFS
    b, g = fresh()
    g.refs[int(g.table[0, 2])] += 1  # the page that row 0 grows in
    g.resize([11, 7, 0])
    assert g.flags() == m.DEVFLAG_SHARED
    g.resize([11, 8, 0])
    assert g.flags() == 0


def test_captured_calls_follow_the_state():
    import torch
    b = Book(600, 4, 6, 40, 2, 32, seed=5)
    g = Gpu(b)
    new, parents = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda")
    slots, table, lens = torch.zeros(6, 2, dtype=torch.int64, device="cuda"), torch.zeros_like(g.table), torch.zeros_like(g.lens)
    where, n = torch.zeros_like(g.refs), torch.zeros(1, dtype=torch.int32, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        g.mla.pages_resize(g.refs, g.table, g.lens, new, 4, g.ws, slots, g.status)
        g.mla.pages_fork(g.refs, g.table, g.lens, parents, table, lens, g.cache, g.ws, g.status)
        g.table.copy_(table)
        g.lens.copy_(lens)
        g.mla.pages_compact(g.refs, g.table, g.lens, g.cache, where, n, g.ws, g.status)
    g.same_as(b)  # nothing ran yet
    rng = np.random.default_rng(0)
    for step in range(6):
        want = rng.integers(0, 100, 6)
        who = rng.integers(-1, 6, 6)
        new.copy_(torch.tensor(want))
        parents.copy_(torch.tensor(who))
        graph.replay()
        torch.cuda.synchronize()
        # rows that would grow in a page that they share are part of the comparison too: counts only
        ref_slots, _ = b.resize(want, 2)
        assert np.array_equal(slots.cpu().numpy(), ref_slots)
        b.fork(who, np.zeros((6, 40), np.int32))
        b.compact()
        g.same_as(b, step)


def test_two_streams_two_workspaces():
    import torch
    pairs = [started(3000, 16, 20, 60, 2, 416, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for step in range(5):
        for (b, g), s in zip(pairs, streams):
            parents = np.random.default_rng(step).integers(-1, 20, 20)
            with torch.cuda.stream(s):
                g.fork(parents, np.zeros((20, 60), np.int32))
                g.compact(stream=s)
    torch.cuda.synchronize()
    for b, g in pairs:
        for step in range(5):
            b.fork(np.random.default_rng(step).integers(-1, 20, 20), np.zeros((20, 60), np.int32))
            b.compact()
        g.same_as(b)


def test_pages_beyond_four_gigabytes():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    pages, page, row = 240000, 16, 1152  # 4.4 GB
    cache = torch.zeros(pages, page, row // 2, dtype=torch.bfloat16, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    held = torch.tensor([239999, 239000, 235001], device="cuda")
    refs[held] = 1
    table, lens = held.to(torch.int32).view(1, 3).contiguous(), torch.tensor([40], dtype=torch.int32, device="cuda")
    x = torch.randn(3, page, row // 2, device="cuda").to(torch.bfloat16)
    cache[held] = x
    refs[:200000] = 1  # the lowest free page lies beyond 2^31 bytes
    ws, out, lens_out = mla.pages_workspace(pages, 2), torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    mla.pages_fork(refs, table, lens, torch.zeros(2, dtype=torch.int32, device="cuda"), out, lens_out, cache, ws)
    assert out.tolist() == [[239999, 239000, 235001], [239999, 239000, 200000]]
    assert torch.equal(cache[200000, :8], x[2, :8]) and not cache[200000, 8:].any()
    refs[:200000] = 0
    where, n = torch.zeros_like(refs), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.pages_compact(refs, out, lens_out, cache, where, n, ws)
    # held in order: 200000, 235001, 239000, 239999
    assert int(n) == 4 and out.tolist() == [[3, 2, 1], [3, 2, 0]] and lens_out.tolist() == [40, 40]
    assert torch.equal(cache[3], x[0]) and torch.equal(cache[2], x[1]) and torch.equal(cache[1], x[2])


def test_bindings_refuse():
    import torch
    b, g = started(100, 16, 5, 40, 2, 48, seed=1)
    m = g.mla
    new, par, out, lo = g.lens.clone(), g.lens.clone(), torch.zeros_like(g.table), torch.zeros_like(g.lens)
    where, n = torch.zeros_like(g.refs), torch.zeros(1, dtype=torch.int32, device="cuda")
    i64, host = lambda t: t.to(torch.int64), lambda t: t.cpu()
    slots = torch.zeros(5, 2, dtype=torch.int64, device="cuda")
    bad = [lambda: m.pages_resize(i64(g.refs), g.table, g.lens, new, 16, g.ws),
           lambda: m.pages_resize(g.refs, g.table, g.lens[:4], new, 16, g.ws),
           lambda: m.pages_resize(g.refs, g.table, g.lens, host(new), 16, g.ws),
           lambda: m.pages_resize(g.refs, g.table.t(), g.lens, new, 16, g.ws),
           lambda: m.pages_resize(g.refs, g.table, g.lens, g.lens, 16, g.ws),
           lambda: m.pages_resize(g.refs, g.table, g.lens, new, 0, g.ws),
           lambda: m.pages_resize(g.refs, g.table, g.lens, new, 16, g.ws, slots[:4]),
           lambda: m.pages_resize(g.refs, g.table, g.lens, new, 16, g.ws, slots.to(torch.int32)),
           lambda: m.pages_resize(g.refs, g.table, g.lens, new, 16, g.ws[:256]),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, g.table, lo, g.cache, g.ws),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, out, g.lens, g.cache, g.ws),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, out[:, :39], lo, g.cache, g.ws),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, out, lo, g.cache[:, :50], g.ws),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, out, lo, g.cache[..., :32], g.ws),
           lambda: m.pages_fork(g.refs, g.table, g.lens, par, out, lo, g.cache[0, 0], g.ws),
           lambda: m.pages_compact(g.refs, g.table, None, g.cache, where, n, g.ws),
           lambda: m.pages_compact(g.refs, g.table, g.lens, g.cache, where[:50], n, g.ws),
           lambda: m.pages_compact(g.refs, g.table, g.lens, g.cache, i64(where), n, g.ws)]
    for k, f in enumerate(bad):
        with pytest.raises(m.MLADecodeError):
            f()
    g.same_as(b)
    m.pages_fork(g.refs, g.table, g.lens, par.fill_(-1), out, lo, g.cache[:1], g.ws)  # one layer of several


def test_a_generation_with_beams_over_a_4_bit_cache():
    """Prompts come in, beams fork, tokens are appended and attended to, chats end, the cache is compacted: each
    step's attention is that over the tokens that the beam has seen."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    H, page, pages, W, B = 16, 4, 120, 24, 6
    rng = np.random.default_rng(3)
    dev = dict(device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, **dev)  # noqa: E731
    cache = torch.full((pages, page, 416), 0x7F, dtype=torch.uint8, **dev)  # what nobody wrote is NaN
    refs, table, lens = torch.zeros(pages, dtype=torch.int32, **dev), torch.zeros(B, W, dtype=torch.int32, **dev), i32([0] * B)
    scale, status, ws = torch.tensor([0.01], **dev), i32([0]), mla.pages_workspace(pages, B)
    cos_sin = torch.cat([torch.ones(200, 32), torch.zeros(200, 32)], 1).cuda()
    d = mla.dplan_info(B, H, 1, page, mla.KV_FP4_E2M1, False, W * page)
    dws = mla.workspace_for(d)
    seen = [np.zeros((0, 576)) for _ in range(B)]

    def append(new, tokens):
        slots = torch.empty(B, tokens, dtype=torch.int64, **dev)
        old = [len(s) for s in seen]
        mla.pages_resize(refs, table, lens, i32(new), page, ws, slots, status)
        bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
        T = B * tokens
        ql, qp, kc, kp, q = bf(T, H, 512), bf(T, H, 64), bf(T, 512), bf(T, 64), torch.empty(T, H, 576, dtype=torch.bfloat16, **dev)
        mla.rope_epilogue(ql, qp, kc, kp, torch.zeros(T, dtype=torch.int64, **dev), cos_sin, slots.view(-1), q, cache, scale)
        x = f4.decode_rows(f4.encode(kc.double().cpu().numpy(), kp.double().cpu().numpy(), 0.01)) * np.float64(np.float32(0.01))
        for b, n in enumerate(new):
            add = max(0, n - old[b])
            rows = x[b * tokens:(b + 1) * tokens]
            seen[b] = np.concatenate([seen[b][:n], rows[tokens - add:]])
        return q.view(B, tokens, H, 576)[:, -1:].contiguous()

    def attend(q):
        out, lse = torch.empty(B, 1, H, 512, dtype=torch.bfloat16, **dev), torch.empty(B, 1, H, **dev)
        mla.plan_device(d, lens, dws)
        mla.fwd_dplan(d, q, cache, scale, table, 1 / 192 ** .5, out, lse, dws)
        mla.combine_dplan(d, out, lse, dws)
        assert mla.dplan_check(d, dws) == 0
        ref, ref_l = np.zeros((B, 1, H, 512)), np.full((B, 1, H), -np.inf)
        qn = q.double().cpu().numpy()
        for b in range(B):
            if len(seen[b]):
                z = qn[b, 0] @ seen[b].T / 192 ** .5
                ref_l[b, 0] = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
                ref[b, 0] = np.exp(z - ref_l[b, 0][:, None]) @ seen[b][:, :512]
        assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, ref_l, "beams")

    attend(append([10, 0, 7, 0, 0, 12], 12))
    for parents in ([0, 0, 0, 2, 2, 5], [1, 1, 3, 3, 4, 0], [5, 4, 3, 2, 1, 0], [0, 0, 0, 0, 0, -1], [2, 2, 1, 1, 0, 0]):
        t2, l2 = torch.zeros_like(table), torch.zeros_like(lens)
        mla.pages_fork(refs, table, lens, i32(parents), t2, l2, cache, ws, status)
        table, lens = t2, l2
        seen = [seen[p].copy() if p >= 0 else np.zeros((0, 576)) for p in parents]
        attend(append([len(s) + 1 if len(s) else 0 for s in seen], 1))
        where, n = torch.empty_like(refs), i32([0])
        mla.pages_compact(refs, table, lens, cache, where, n, ws, status)
        cache[int(n):] = 0x7F
        attend(append([len(s) + (3 if b % 2 else 2) if len(s) else 0 for b, s in enumerate(seen)], 3))
    append([0] * B, 1)
    assert int(status) == 0 and not refs.any()


@pytest.mark.parametrize("pages,page,W", [(200, 16, 20), (33000, 2, 160)])  # one launch a call, a kernel a step
def test_a_decode_right_behind_sees_the_new_lengths(pages, page, W):
    """Rows shrink and grow and the decode follows with nothing between, one call after another and in a graph: the
    lengths, tables and copied rows that it reads are those of the call before it."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    H, B = 16, 5
    rng = np.random.default_rng(2)
    b = Book(pages, page, B, W, 1, 416, 3)
    b.cache = f4.encode(rng.standard_normal((pages * page, 512)), rng.standard_normal((pages * page, 64)), 0.01).reshape(1, pages, page, 416)
    b.resize([300, 17, 0, 64, 200])
    g = Gpu(b)
    q = torch.from_numpy(rng.standard_normal((B, 1, H, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    scale = torch.tensor([0.01], device="cuda")
    plan = mla.plan([W * page] * B, H, 1, page, mla.KV_FP4_E2M1)
    ws = mla.workspace_for(plan)
    new = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in
           ([1, 0, 33, 320, 7], [310, 5, 0, 2, 7], [16, 290, 100, 0, 15], [0, 1, 320, 48, 49], [300, 17, 0, 64, 200])]
    parents = torch.tensor([4, 0, 0, 3, 1], dtype=torch.int32, device="cuda")
    table2, lens2 = torch.zeros(B, W, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = [(torch.empty(B, 1, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, H, device="cuda")) for _ in range(len(new) + 1)]

    def attend(table, lens, out, lse):
        mla.fwd(plan, q, g.cache[0], scale, table, lens, 0.05, out, lse, ws)
        mla.combine(plan, lens, out, lse, ws)

    def steps():
        for n, o in zip(new, outs):
            mla.pages_resize(g.refs, g.table, g.lens, n, page, g.ws, None, g.status)
            attend(g.table, g.lens, *o)
        mla.pages_fork(g.refs, g.table, g.lens, parents, table2, lens2, g.cache, g.ws, g.status)
        attend(table2, lens2, *outs[-1])

    start = [x.clone() for x in (g.refs, g.table, g.lens, g.cache)]

    def again():
        for x, y in zip((g.refs, g.table, g.lens, g.cache), start):
            x.copy_(y)

    def expected(table, lens):
        rows = f4.decode_rows(g.cache[0].cpu().numpy()) * 0.01
        ref, lse, qq = np.zeros((B, 1, H, 512)), np.full((B, 1, H), -np.inf), q.double().cpu().numpy()
        for i, n in enumerate(lens):
            if n == 0:
                continue
            j = np.arange(n)
            keys = rows[table[i, j // page], j % page]
            z = qq[i, 0] @ keys.T * 0.05
            w = np.exp(z - z.max(1, keepdims=True))
            lse[i, 0], ref[i, 0] = z.max(1) + np.log(w.sum(1)), w / w.sum(1, keepdims=True) @ keys[:, :512]
        return ref, lse

    plain = []
    for n in new:
        b.resize(n.cpu().numpy())
        plain.append((b.table.copy(), b.lens.copy()))
    steps()
    want = [expected(*s) for s in plain] + [expected(table2.cpu().numpy(), lens2.cpu().numpy())]
    first = [o.clone() for o, _ in outs]
    for k, (o, (ref, lse)) in enumerate(zip(outs, want)):
        assert_close(o[0].double().cpu().numpy(), o[1].double().cpu().numpy(), ref, lse, f"step {k}")
    again()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(20):
        again()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, f) for (o, _), f in zip(outs, first))
