"""rb_pages_*: page management of the paged cache against the one-page-at-a-time oracle, bit for
bit, with every page that is not written checked to be left as it was."""
import numpy as np
import pytest
import torch

import oracle.pages as ref

pytestmark = pytest.mark.gpu


class State:
    """A random pool: rows of pages, some shared, and the oracle's copy of it."""

    def __init__(self, rb, seed, rows=12, max_blocks=9, B=16, nkv=2, hd=64, r=1, null=0,
                 spare=20, max_tokens=None):
        rng = np.random.default_rng(seed)
        pt = B * r
        self.cached = rng.integers(0, (max_tokens or max_blocks * pt) + 1, rows).astype(np.int32)
        self.cached[rng.random(rows) < 0.2] = 0
        need = [-(-int(c) // pt) for c in self.cached]
        E = 1 + sum(need) + spare
        ids = [int(i) for i in rng.permutation(E) if i != null // r]
        self.table, at = [], 0
        for i, n in enumerate(need):
            row = ids[at:at + n]
            at += n
            if i and rng.random() < 0.4:
                common = min(len(row), len(self.table[i - 1]))
                row[:common] = self.table[i - 1][:common]
            self.table.append(row)
        self.null = null // r
        self.dims = rb.Dims(block_size=B, num_q_heads=nkv, num_kv_heads=nkv, head_dim=hd,
                            max_num_reqs=rows, max_model_len=max_blocks * pt,
                            max_blocks_per_req=max_blocks, num_blocks=E * r, null_block=null,
                            kernel_blocks_per_manager_block=r)
        self.E, self.pt, self.MB, self.rows = E, pt, max_blocks, rows
        bt = np.full((rows, max_blocks), -7, np.int32)   # past a row's count: not state
        for i, row in enumerate(self.table):
            bt[i, :len(row)] = row
        self.bt0 = bt.copy()
        cuda = lambda a: torch.as_tensor(np.ascontiguousarray(a)).cuda()
        self.bt = cuda(bt)
        self.nb = cuda(np.array([len(x) for x in self.table], np.int32))
        self.ref = ref.count(self.table, E)
        g = torch.Generator().manual_seed(seed)
        self.host = [torch.randint(-30000, 30000, (E, pt, nkv * hd), dtype=torch.int16,
                                   generator=g) for _ in range(2)]
        dev = [c.cuda().view(torch.bfloat16).view(E * pt, nkv, hd) for c in self.host]
        self.k, self.v = dev
        self.pool = rb.PagePool(self.dims, self.k, self.v, self.bt, self.nb)
        assert self.pool.ref_count.cpu().tolist() == self.ref

    def i32(self, xs):
        return torch.as_tensor(np.asarray(xs, np.int32)).cuda()

    def check(self, bits=0):
        torch.cuda.synchronize()
        assert int(self.pool.error_word.item()) == bits
        assert self.nb.cpu().tolist() == [len(x) for x in self.table]
        bt = self.bt.cpu().numpy()
        for i, row in enumerate(self.table):
            assert bt[i, :len(row)].tolist() == row
        assert self.pool.ref_count.cpu().tolist() == self.ref
        for got, want in zip((self.k, self.v), self.host):
            assert torch.equal(got.view(torch.int16).cpu().view(want.shape), want)


GEOMETRY = [dict(), dict(nkv=8, hd=128), dict(nkv=1, hd=8), dict(r=2, null=2), dict(null=5),
            dict(B=1, max_blocks=40), dict(nkv=3, hd=128, r=4, null=8), dict(B=7, nkv=1, hd=24)]


@pytest.mark.parametrize("geo", GEOMETRY)
@pytest.mark.parametrize("seed", range(3))
def test_fork_free_compact_in_turn(rb, geo, seed):
    s = State(rb, seed, **geo)
    rng = np.random.default_rng(seed + 50)
    for turn in range(4):
        full = [i for i in range(s.rows) if s.table[i]]
        gone = rng.choice(s.rows, size=int(rng.integers(0, s.rows)), replace=False).tolist()
        freed = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        s.pool.free(s.i32(gone + gone[:2]), num_freed=freed)   # the second time frees nothing
        for r in gone:
            s.bt0[r, :len(s.table[r])] = -1
        want = ref.free(s.table, s.ref, gone)
        s.check()
        assert int(freed.item()) == want
        for r in gone:
            s.cached[r] = 0
            assert (s.bt[r].cpu().numpy() == s.bt0[r]).all()
        full = [i for i in range(s.rows) if i not in gone]
        empty = [i for i in range(s.rows) if not s.table[i]]
        if full and empty:
            dst = rng.permutation(empty)[:max(1, len(empty) - 1)].tolist()
            src = rng.choice([f for f in full if f not in dst] or full, size=len(dst)).tolist()
            keep = [(a, b) for a, b in zip(src, dst) if a != b]
            src, dst = [a for a, _ in keep], [b for _, b in keep]
            tails = sum(int(s.cached[a]) % s.pt != 0 for a in src)
            if tails <= sum(n == 0 for i, n in enumerate(s.ref) if i != s.null):
                s.pool.fork(s.i32(src), s.i32(dst), s.i32(s.cached))
                ref.fork(s.table, s.ref, src, dst, s.cached, s.pt, s.null, s.host)
                s.check()
                for a, b in zip(src, dst):
                    s.cached[b] = s.cached[a]
                    s.bt0[b, :len(s.table[b])] = s.table[b]
        page_map, live = s.i32(np.full(s.E, -9)), s.i32([-9])
        s.pool.compact(page_map=page_map, num_live=live)
        new, n = ref.compact(s.table, s.ref, s.null, s.host)
        for i, row in enumerate(s.table):
            s.bt0[i, :len(row)] = row
        s.check()
        assert page_map.cpu().tolist() == new and int(live.item()) == n
        assert (s.bt.cpu().numpy() == s.bt0).all()


@pytest.mark.parametrize("E,live", [(5000, 3000), (2049, 2048), (2048, 1), (4097, 4096), (10, 0)])
def test_compact_over_chunk_borders(rb, E, live):
    """Pools larger than one scan chunk, packed or nearly empty, the null page anywhere."""
    rng = np.random.default_rng(E + live)
    for null in (0, E - 1, live if live < E else 0, E // 2):
        ids = [int(i) for i in rng.permutation(E) if i != null][:live]
        dims = rb.Dims(block_size=1, num_q_heads=1, num_kv_heads=1, head_dim=8, max_num_reqs=3,
                       max_model_len=E, max_blocks_per_req=E, num_blocks=E, null_block=null)
        table = [ids[:live // 3], [], ids[live // 3:]]
        bt = np.full((3, E), -1, np.int32)
        for i, row in enumerate(table):
            bt[i, :len(row)] = row
        host = [torch.randint(-9999, 9999, (E, 1, 8), dtype=torch.int16) for _ in range(2)]
        k, v = (h.cuda().view(torch.bfloat16) for h in host)
        nb = torch.tensor([len(x) for x in table], dtype=torch.int32).cuda()
        pool = rb.PagePool(dims, k, v, torch.as_tensor(bt).cuda(), nb)
        count = ref.count(table, E)
        pool.compact()
        ref.compact(table, count, null, host)
        assert int(pool.error_word.item()) == 0
        assert pool.ref_count.cpu().tolist() == count
        got = pool.block_table.cpu().numpy()
        for i, row in enumerate(table):
            assert got[i, :len(row)].tolist() == row
        assert torch.equal(k.view(torch.int16).cpu(), host[0])
        assert torch.equal(v.view(torch.int16).cpu(), host[1])


@pytest.mark.parametrize("geo", GEOMETRY)
def test_copy(rb, geo):
    s = State(rb, 3, **geo)
    rng = np.random.default_rng(1)
    pages = [int(i) for i in rng.permutation(s.E) if i != s.null]
    for n in (1, 2, len(pages) // 2):
        src, dst = pages[:n], pages[len(pages) - n:]
        src = src[:n // 2] + [src[0]] * (n - n // 2)       # one page copied to many
        src[n // 3], dst[n // 4] = (-1, dst[n // 4]) if n > 4 else (src[n // 3], dst[n // 4])
        s.pool.copy(s.i32(src), s.i32(dst))
        ref.copy(src, dst, s.host)
        s.check()
    s.pool.copy(s.i32([]), s.i32([]))
    s.check()


def test_copy_flags_bad_pairs(rb):
    s = State(rb, 4)
    bits_of = lambda t: t.view(torch.int16)   # compared as bits: some are NaN patterns
    before = [bits_of(s.k).clone(), bits_of(s.v).clone()]
    a, b, c = [i for i in range(s.E) if i != s.null][:3]
    for src, dst, bit in (([a], [s.null], rb.EBIT_BLOCK_ID), ([s.null], [a], rb.EBIT_BLOCK_ID),
                          ([s.E], [a], rb.EBIT_BLOCK_ID), ([a], [s.E + 5], rb.EBIT_BLOCK_ID)):
        s.pool.error_word.zero_()
        s.pool.copy(s.i32(src), s.i32(dst))
        assert int(s.pool.error_word.item()) == bit
        assert torch.equal(bits_of(s.k), before[0]) and torch.equal(bits_of(s.v), before[1])
    for src, dst in (([a, b], [c, c]), ([a, b], [b, c]), ([a], [a])):
        s.pool.error_word.zero_()
        s.pool.copy(s.i32(src), s.i32(dst))
        assert int(s.pool.error_word.item()) == rb.EBIT_PAGE_PAIR
        others = [i for i in range(s.E) if i not in (a, b, c)]
        for t, t0 in ((s.k, before[0]), (s.v, before[1])):
            t, t0 = bits_of(t).view(s.E, -1), t0.view(s.E, -1)
            assert torch.equal(t[others], t0[others])
        bits_of(s.k).copy_(before[0]), bits_of(s.v).copy_(before[1])


def test_refused_forks_change_nothing(rb):
    s = State(rb, 6, rows=6, spare=1, max_blocks=4)
    s.cached[:] = [17, 5, 0, 0, 0, 33]
    for r, c in enumerate(s.cached):
        s.table[r] = []
    pages = iter(i for i in range(s.E) if i != s.null)
    s.table = [[next(pages) for _ in range(-(-int(c) // 16))] for c in s.cached]
    s.bt.fill_(-1)
    for r, row in enumerate(s.table):
        s.bt[r, :len(row)] = s.i32(row)
    s.nb.copy_(s.i32([len(x) for x in s.table]))
    s.ref = ref.count(s.table, s.E)
    s.pool.count()
    s.check()
    cases = [([0], [0]), ([0], [1]), ([0, 1], [2, 2]), ([6], [2]), ([0], [-1]), ([0], [6])]
    cached = s.i32(s.cached)
    for src, dst in cases:
        s.pool.error_word.zero_()
        s.pool.fork(s.i32(src), s.i32(dst), cached)
        s.check(bits=rb.EBIT_ROW)
    for bad in (-1, 65, 1 << 30):     # more cached tokens than the row has pages for
        s.pool.error_word.zero_()
        s.pool.fork(s.i32([0]), s.i32([2]), s.i32([bad, 5, 0, 0, 0, 33]))
        s.check(bits=rb.EBIT_ROW)
    # too few pages: hold all free ones but one, then fork two partial pages
    holes = [i for i, n in enumerate(s.ref) if n == 0 and i != s.null]
    for i in holes[1:]:
        s.pool.ref_count[i] = 1
        s.ref[i] = 1
    s.pool.error_word.zero_()
    s.pool.fork(s.i32([0, 1]), s.i32([2, 3]), cached)
    s.check(bits=rb.EBIT_NO_PAGE)
    s.pool.error_word.zero_()
    s.pool.fork(s.i32([0]), s.i32([2]), cached)     # one fits
    ref.fork(s.table, s.ref, [0], [2], s.cached, 16, s.null, s.host)
    s.check()


def test_free_flags_what_it_skips(rb):
    s = State(rb, 8)
    r = next(i for i in range(s.rows) if len(s.table[i]) > 1 and
             all(s.ref[p] == 1 for p in s.table[i]))
    s.pool.ref_count[s.table[r][0]] = 0
    s.ref[s.table[r][0]] = 0
    s.pool.free(s.i32([r, s.rows, -1]))
    for p in s.table[r][1:]:
        s.ref[p] -= 1
    s.table[r] = []
    s.check(bits=rb.EBIT_ROW | rb.EBIT_PAGE_REF)


def test_counts_of_a_bad_table(rb):
    s = State(rb, 9)
    r = next(i for i in range(s.rows) if len(s.table[i]) > 1)
    q = next(i for i in range(s.rows) if i != r and s.table[i])
    s.bt[r, 0] = s.E + 3
    s.nb[q] = s.MB + 1
    s.pool.count()
    table = [[] if i == q else row[1:] if i == r else row for i, row in enumerate(s.table)]
    assert int(s.pool.error_word.item()) == rb.EBIT_BLOCK_ID | rb.EBIT_ROW
    assert s.pool.ref_count.cpu().tolist() == ref.count(table, s.E)
    before = s.bt.clone()
    s.pool.error_word.zero_()
    s.pool.compact()          # an entry outside the pool and a bad row stay as they are
    assert int(s.pool.error_word.item()) == rb.EBIT_BLOCK_ID | rb.EBIT_ROW
    assert int(s.bt[r, 0]) == s.E + 3 and torch.equal(s.bt[q], before[q])


def test_a_captured_turn_replays(rb):
    """Fork, free and compact captured once; every replay does the turn on the tables of then."""
    a, b = State(rb, 12, rows=9, spare=40), State(rb, 12, rows=9, spare=40)
    src = [i for i in range(9) if a.table[i]][:3]
    gone = [i for i in range(9) if a.table[i] and i not in src][:2]
    for s in (a, b):
        s.pool.free(s.i32([i for i in range(9) if i not in src + gone]))
        ref.free(s.table, s.ref, [i for i in range(9) if i not in src + gone])
    empty = [i for i in range(9) if not a.table[i]][:len(src)]
    src = src[:len(empty)]
    args = [(s.i32(src), s.i32(empty), s.i32(s.cached)) for s in (a, b)]
    tensors = [(s.bt.clone(), s.nb.clone(), s.pool.ref_count.clone()) for s in (a, b)]
    gone_t = [s.i32(gone) for s in (a, b)]

    def turn(s, i):
        s.pool.fork(*args[i])
        s.pool.free(gone_t[i])
        s.pool.compact()

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        turn(a, 0)
    for _ in range(2):
        for s, saved in zip((a, b), tensors):
            s.bt.copy_(saved[0]), s.nb.copy_(saved[1]), s.pool.ref_count.copy_(saved[2])
        graph.replay()
        turn(b, 1)
        torch.cuda.synchronize()
        assert torch.equal(a.bt, b.bt) and torch.equal(a.nb, b.nb)
        assert torch.equal(a.pool.ref_count, b.pool.ref_count)
        assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16))
        assert int(a.pool.error_word.item()) == 0


def test_pool_of_a_persistent_batch(rb):
    """The pool follows a PersistentBatch's live rows: requests enter through the scheduler's
    delta, one is forked into a row the scheduler added without pages, freed and compacted."""
    from types import SimpleNamespace as NS

    batch = rb.PersistentBatch(8, 128, 8)
    new = [NS(req_id=7, num_computed=33, num_prompt=40, tokens=list(range(40)),
              blocks=[9, 4, 6]),
           NS(req_id=8, num_computed=5, num_prompt=9, tokens=list(range(9)), blocks=[11]),
           NS(req_id=9, num_computed=33, num_prompt=40, tokens=list(range(40)), blocks=[])]
    batch.apply(NS(scheduled={7: 7, 8: 4, 9: 7}, new=new, cached=[]))
    dims = rb.Dims(block_size=16, num_q_heads=2, num_kv_heads=2, head_dim=64, max_num_reqs=8,
                   max_model_len=128, max_blocks_per_req=8, num_blocks=16)
    k = torch.randn(256, 2, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn(256, 2, 64, device="cuda").to(torch.bfloat16)
    pool = rb.PagePool(dims, k, v, batch=batch)
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32, device="cuda")
    pool.fork(i32([0]), i32([2]), batch.num_computed)
    snap = batch.snapshot()
    assert snap["blocks"][2].tolist() == [9, 4, 1]
    assert torch.equal(k[16:17], k[96:97]) and torch.equal(v[16:17], v[96:97])
    assert pool.ref_count.cpu().tolist() == [0, 1, 0, 0, 2, 0, 1, 0, 0, 2, 0, 1, 0, 0, 0, 0]
    pool.free(i32([0]))
    pool.compact()
    snap = batch.snapshot()
    assert [b.tolist() for b in snap["blocks"]] == [[], [3], [2, 4, 1]]
    assert int(pool.error_word.item()) == 0 and int(batch.error_word.item()) == 0


@pytest.mark.parametrize("geo", [dict(), dict(r=2, null=2), dict(nkv=8, hd=128)])
def test_a_second_layer_follows_with_copies(rb, geo):
    """Fork and compact through one layer's pool; a second layer's caches follow by copies, and
    every row reads the same tokens in both layers as before."""
    s = State(rb, 31, rows=10, spare=30, **geo)
    k2, v2 = s.k.flip(0).contiguous(), s.v.flip(0).contiguous()
    layer = rb.PagePool(s.dims, k2, v2)
    cached = s.cached.copy()
    gone = [i for i in range(s.rows) if i % 3 == 0 and s.table[i]]
    s.pool.free(s.i32(gone))
    ref.free(s.table, s.ref, gone)
    cached[gone] = 0
    empty = [i for i in range(s.rows) if not s.table[i]][:3]
    src = [i for i in range(s.rows) if s.table[i]][:len(empty)]
    empty = empty[:len(src)]

    def tokens(kv, row, n):
        bt = s.bt[row].long().cpu()
        slots = torch.cat([bt[j] * s.pt + torch.arange(s.pt) for j in range(-(-n // s.pt))])[:n]
        return kv.view(torch.int16).cpu()[slots]

    want = {d: [tokens(c, r, int(cached[r])) for c in (s.k, s.v, k2, v2)]
            for r, d in zip(src, empty)}
    want.update({r: want[d] for r, d in zip(src, empty)})

    full = cached[src] // s.pt
    s.pool.fork(s.i32(src), s.i32(empty), s.i32(cached))
    at = torch.as_tensor(np.minimum(full, s.MB - 1)).long().cuda()
    skip = s.i32(cached[src] % s.pt) == 0
    entry = lambda rows: s.bt[torch.as_tensor(rows).cuda(), at].masked_fill(skip, -1)
    layer.copy(entry(src).contiguous(), entry(empty).contiguous())
    page_map = torch.empty(s.E, dtype=torch.int32, device="cuda")
    s.pool.compact(page_map=page_map)
    ids = torch.arange(s.E, dtype=torch.int32, device="cuda")
    layer.copy(ids.masked_fill((page_map == ids) | (page_map < 0), -1), page_map)
    torch.cuda.synchronize()
    assert int(s.pool.error_word.item()) == 0 and int(layer.error_word.item()) == 0
    assert any(int(cached[r]) % s.pt for r in src)
    for row, parts in want.items():
        for c, part in zip((s.k, s.v, k2, v2), parts):
            assert torch.equal(tokens(c, row, len(part)), part)


def test_captured_behind_a_join_of_two_streams(rb):
    """Calls that may start beside the kernel before them, captured where two branches of the
    graph meet, behind a memcpy and behind a memset: all of what comes before is waited for."""
    s = State(rb, 33, rows=8, spare=40)
    free = [i for i, c in enumerate(s.ref) if c == 0 and i != s.null]
    live = [i for i, c in enumerate(s.ref) if c > 0]
    n = min(len(free), len(live), 12)
    src, dst = s.i32([-1] * n), s.i32([-1] * n)
    src_now, dst_now = s.i32(live[:n]), s.i32(free[:n])
    scratch = torch.zeros(1 << 24, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(4):
                scratch.add_(1.0)      # the longer branch
            src.copy_(src_now)
        dst.add_(dst_now + 1)          # -1 + id + 1
        main.wait_stream(side)
        s.pool.copy(src, dst)          # two branches, one of them a memcpy
        s.pool.count()                 # a memset and a kernel
        s.pool.compact()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(live[:n], free[:n]):
        for h in s.host:
            h[b] = h[a]
    ref.compact(s.table, s.ref, s.null, s.host)
    s.check()


def test_a_pool_made_on_a_busy_device(rb):
    """A pool built for another stream while the current one is busy: what it fills and counts
    belongs to that stream, and a fork there reads finished counts."""
    s = State(rb, 21, rows=8, spare=12)
    src = next(i for i in range(s.rows) if s.table[i] and s.cached[i] % s.pt)
    dst = next(i for i in range(s.rows) if i != src)
    s.pool.free(s.i32([dst]))
    ref.free(s.table, s.ref, [dst])
    s.cached[dst] = 0
    s.check()
    args = s.i32([src]), s.i32([dst]), s.i32(s.cached)
    scratch = torch.zeros(1 << 26, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(1000):              # some 80 ms of work on the current stream
        scratch.add_(1.0)
    pool = rb.PagePool(s.dims, s.k, s.v, s.bt, s.nb, stream=side)
    pool.fork(*args, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()      # it was busy all along
    ref.fork(s.table, s.ref, [src], [dst], s.cached, s.pt, s.null, s.host)
    s.pool = pool
    s.check()


@pytest.mark.parametrize("bad", ["over", -1, 2 ** 31 - 1, -2 ** 31])
def test_free_leaves_a_row_with_a_bad_count_alone(rb, bad):
    """A count outside [0, max_blocks_per_req]: the row keeps it, its entries and its pages'
    counts; the other rows named are freed, one of them twice."""
    s = State(rb, 10)
    full = [i for i in range(s.rows) if s.table[i]]
    r, other = full[0], full[1]
    bad = s.MB + 1 if bad == "over" else bad
    s.nb[r] = bad
    before = s.bt.clone()
    freed = s.i32([-9])
    s.pool.free(s.i32([other, r, other, r]), num_freed=freed)
    want = ref.free(s.table, s.ref, [other])
    torch.cuda.synchronize()
    assert int(s.pool.error_word.item()) == rb.EBIT_ROW
    assert int(s.nb[r]) == bad and int(freed.item()) == want
    assert torch.equal(s.bt[r], before[r])
    s.nb[r] = len(s.table[r])
    s.check(bits=rb.EBIT_ROW)
