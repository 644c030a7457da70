"""Two decoder layers as a serving step uses the operators, one over a cache in 16 bits and one over a
cache in 4: the residual's addition and norm, a fused projection, its queries and keys rotated and
its keys and values appended, attention, and at the end the sampled rows' log probabilities.
Prompts, decodes, padding, forked samples, a compacted pool and a captured step.  Each operator is
held against its 64-bit oracle on what it was given, the attention on each request's own history.
"""
from types import SimpleNamespace as NS

import numpy as np
import pytest
import torch

from oracle import kv4 as ref
from oracle import norm as ref_norm
from oracle.logprobs import token_logprobs as oracle_logprobs
from oracle.scores import paged_attention_scored as oracle_attention
from test_gpu_norm import _check16, _check8
from test_gpu_scored_attention import _compare

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NH, NKV, HD, VOCAB, PAGES, EPS = 8, 2, 64, 1003, 40, 1e-5
HIDDEN, KV, POSITIONS = NH * HD, NKV * HD, 256
K_SCALE, V_SCALE = 0.5, 3.0


def f64(t):
    return t.double().cpu().numpy()


class Model:
    def __init__(self, rb, seed):
        self.rb = rb
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = rb.Dims(block_size=16, num_q_heads=NH, num_kv_heads=NKV, head_dim=HD,
                            max_num_reqs=8, max_model_len=POSITIONS, max_blocks_per_req=16,
                            num_blocks=PAGES)
        w = lambda *shape: (torch.randn(*shape, generator=self.gen, device="cuda") /
                            shape[0] ** 0.5).to(BF)
        self.qkv = [w(HIDDEN, HIDDEN + 2 * KV) for _ in range(2)]
        self.proj = [w(HIDDEN, HIDDEN) for _ in range(2)]
        self.norms = [(1 + 0.2 * torch.randn(HIDDEN, generator=self.gen, device="cuda")).to(BF)
                      for _ in range(3)]
        self.embed, self.head = w(VOCAB, HIDDEN) * 8, w(HIDDEN, VOCAB)
        self.rotation = [rb.Rotation(rb.rotary_table(POSITIONS, HD)),
                         rb.Rotation(rb.rotary_table(POSITIONS, HD // 2, 5000.0), True)]
        self.k, self.v = (torch.zeros(PAGES * 16, NKV, HD, dtype=BF, device="cuda") for _ in "kv")
        self.k4, self.v4 = rb.kv4_cache(self.dims)
        self.batch = rb.PersistentBatch(8, POSITIONS, 16)
        self.pool = rb.PagePool(self.dims, self.k, self.v, batch=self.batch)
        # the 4-bit layer's pages follow the table's
        view = lambda c: rb.kv4_pages(c).view(PAGES, NKV, 9 * HD // 2)
        self.pool4 = rb.PagePool(rb.kv4_page_dims(self.dims), view(self.k4), view(self.v4))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.history = {}  # request id -> per layer (keys, values) that its cache stands for
        self.cached = {}

    def rows(self, ids):
        return torch.tensor([self.row[i] for i in ids], dtype=torch.int32, device="cuda")

    def apply(self, scheduled, new=(), cached=()):
        self.batch.apply(NS(scheduled=scheduled, new=list(new), cached=list(cached)))
        self.scheduled = scheduled
        self.row = dict(zip(scheduled, self.batch.row_of_sched[:len(scheduled)].tolist()))

    def prepare(self, pad=3):
        b, R = self.batch, self.batch.num_reqs
        N = sum(self.scheduled.values())
        return R, N, self.rb.prepare_inputs(self.dims, R, R, N, N + pad, b.token_table,
                                            b.num_computed, b.num_scheduled, b.block_table)

    def forward(self, R, N, meta, seen, workspace=None):
        """The step; what each operator was given and gave is listed in ``seen``."""
        rb = self.rb
        hidden = self.embed[meta["input_ids"].long().clamp(0, VOCAB - 1)]
        delta = torch.zeros_like(hidden)
        for layer in range(2):
            given = (delta, hidden.clone())
            x = rb.add_rms_norm(delta, self.norms[layer], EPS, residual=hidden)
            n = x.shape[0]
            q, k, v = (x @ self.qkv[layer]).split([HIDDEN, KV, KV], 1)
            q, k, v = q.view(n, NH, HD), k.view(n, NKV, HD), v.view(n, NKV, HD)
            common = dict(positions=meta["positions"], rotation=self.rotation[layer],
                          error_word=self.err)
            tables = (self.batch.block_table, meta["query_start_loc"], meta["seq_lens"])
            if layer == 0:
                turned = rb.kv_append(self.dims, q, k, v, meta["slot_mapping"], self.k, self.v,
                                      **common)
                o = rb.paged_attention(self.dims, R, N, turned, self.k, self.v, *tables,
                                       error_word=self.err, workspace=workspace)
            else:
                turned = rb.kv4_append(self.dims, q, k, v, meta["slot_mapping"], self.k4, self.v4,
                                       k_scale=K_SCALE, v_scale=V_SCALE, **common)
                o = rb.paged_attention_kv4(self.dims, R, N, turned, self.k4, self.v4, *tables,
                                           k_scale=K_SCALE, v_scale=V_SCALE, workspace=workspace,
                                           error_word=self.err)
            seen.append((given, hidden.clone(), x, q, k, v, turned, o))
            delta = o.view(n, HIDDEN) @ self.proj[layer]
        codes, scales = rb.add_rms_norm_fp8(delta, self.norms[2], EPS, residual=hidden, group=64)
        last = rb.gather_rows((codes.view(n, -1, 64).float() * scales[..., None]).to(BF).view(n, -1),
                              meta["logits_indices"])
        seen.append((hidden, codes, scales))
        return last @ self.head

    def check(self, R, N, meta, seen):
        by_row = sorted(self.scheduled, key=self.row.get)
        loc, lens = meta["query_start_loc"].tolist(), meta["seq_lens"].tolist()
        pos = meta["positions"][:N].cpu().numpy()
        for layer in range(2):
            (delta, before), hidden, x, q, k, v, turned, o = seen[layer]
            assert torch.equal(hidden, (delta.float() + before.float()).to(BF))
            _check16(ref_norm.rms_norm(f64(hidden), f64(self.norms[layer]), EPS), x, "bf16", 0)
            rot = self.rotation[layer]
            angle = rot.table.cpu().numpy()[pos]
            turn = lambda t: torch.from_numpy(ref.rotate(t[:N].float().cpu().numpy(), angle,
                                                         rot.interleaved)).to(BF)
            assert torch.equal(turned[:N].cpu(), turn(q))
            new = [f64(turn(k)), f64(v[:N])]
            if layer == 1:
                new = [ref.decode(*ref.encode(t, s), s) for t, s in zip(new, (K_SCALE, V_SCALE))]
            for i, a, e in zip(by_row, loc, loc[1:]):
                old = self.history.setdefault(i, {}).get(layer, [t[:0] for t in new])
                self.history[i][layer] = [np.concatenate([h, t[a:e]]) for h, t in zip(old, new)]
            keys, values = ([self.history[i][layer][j] for i in by_row] for j in (0, 1))
            want, weight = oracle_attention(f64(turned), keys, values, loc, lens)
            if layer == 0:
                _compare(o, want, weight, N)
            else:  # P in fp16, the output in bf16, scores in fp32 (test_gpu_kv4_attention.py)
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -10) * weight + 1e-6
                assert (np.abs(f64(o) - want) <= tol).all() and bool((o[N:] == 0).all())
        hidden, codes, scales = seen[2]
        _check8(ref_norm.rms_norm(f64(hidden), f64(self.norms[2]), EPS), codes, scales, 64)

    def step(self):
        R, N, meta = self.prepare()
        seen = []
        logits = self.forward(R, N, meta, seen)
        tokens = logits.float().argmax(1).to(torch.int32)
        lp = self.rb.token_logprobs(logits, tokens, 3, error_word=self.err)
        torch.cuda.synchronize()
        assert [int(e.item()) for e in (self.err, meta["scalars"][3], self.pool.error_word,
                                        self.pool4.error_word, self.batch.error_word)] == [0] * 5
        self.check(R, N, meta, seen)
        want = oracle_logprobs(f64(logits), tokens.tolist(), 3)
        assert np.abs(f64(lp.logprobs) - want[0]).max() < 1e-4
        assert lp.ranks.tolist() == want[1].tolist()
        for i in self.scheduled:
            self.cached[i] += self.scheduled[i]
        by_row = sorted(self.scheduled, key=self.row.get)
        self.next = dict(zip(by_row, tokens.tolist()))
        return R, N, meta, seen

    def grow(self, i):
        return NS(req_id=i, num_computed=self.cached[i], new_tokens=[self.next[i]], new_blocks=[],
                  replace_blocks=False)


def test_layers_of_both_caches(rb):
    m = Model(rb, 5)
    prompts = {10: (90, list(range(1, 8))), 11: (37, [20, 9, 31]), 12: (5, [39])}
    m.cached = {i: 0 for i in prompts}
    m.apply({i: n for i, (n, _) in prompts.items()},
            new=[NS(req_id=i, num_computed=0, num_prompt=n,
                    tokens=[(i * j) % VOCAB for j in range(n)], blocks=p)
                 for i, (n, p) in prompts.items()])
    m.pool.count()
    m.step()
    # two samples of request 10 and one of 12: the table and layer 0 are forked, layer 1 follows
    samples = {20: 10, 21: 10, 22: 12}
    for s, i in samples.items():
        m.cached[s], m.next[s] = m.cached[i], m.next[i]
        m.history[s] = {layer: list(kv) for layer, kv in m.history[i].items()}
    new = [NS(req_id=s, num_computed=m.cached[i], num_prompt=m.cached[i],
              tokens=list(range(m.cached[i])) + [m.next[i]], blocks=[])
           for s, i in samples.items()]
    everyone = list(prompts) + list(samples)
    m.apply({i: 1 for i in everyone}, new=new, cached=[m.grow(i) for i in prompts])
    m.pool.fork(m.rows(samples.values()), m.rows(samples), m.batch.num_computed)
    at = [m.cached[i] // 16 if m.cached[i] % 16 else -1 for i in samples.values()]
    entry = lambda ids: torch.stack([m.batch.block_table[m.row[i], a] if a >= 0 else
                                     torch.tensor(-1, dtype=torch.int32, device="cuda")
                                     for i, a in zip(ids, at)])
    m.pool4.copy(entry(samples.values()), entry(samples))
    m.step()
    for _ in range(2):
        m.apply({i: 1 for i in everyone}, cached=[m.grow(i) for i in everyone])
        m.step()
    # two finish, the pool is compacted and the 4-bit layer's pages go the same way
    m.pool.free(m.rows([10, 22]))
    left = [i for i in everyone if i not in (10, 22)]
    m.apply({i: 1 for i in left}, cached=[m.grow(i) for i in left])
    R, N, meta, seen = m.step()
    page_map = torch.empty(PAGES, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.pool.compact(page_map=page_map, num_live=live)
    old = torch.arange(PAGES, dtype=torch.int32, device="cuda")
    m.pool4.copy(old, torch.where(page_map == old, -1, page_map))
    m.apply({i: 1 for i in left}, cached=[m.grow(i) for i in left])
    m.step()
    # one more step, captured: the same bits as its calls one by one, on every replay
    m.apply({i: 1 for i in left}, cached=[m.grow(i) for i in left])
    caches = (m.k, m.v, m.k4, m.v4)
    before = [c.clone() for c in caches]
    R, N, meta, seen = m.step()
    after = [c.clone() for c in caches]
    want = [seen[0][7], seen[1][7], *seen[2]]
    workspace = torch.empty(rb.workspace_size(m.dims, R, N), dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    again = []
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        m.forward(R, N, meta, again, workspace)
    for _ in range(3):
        for c, old in zip(caches, before):
            c.copy_(old)
        graph.replay()
        torch.cuda.synchronize()
        got = [again[0][7], again[1][7], *again[2]]
        assert all(torch.equal(g[:N].view(torch.uint8), w[:N].view(torch.uint8))
                   for g, w in zip(got, want))
        # (padding tokens share the reserved page's slots)
        assert all(torch.equal(c[c.shape[0] // PAGES:], w[c.shape[0] // PAGES:])
                   for c, w in zip(caches, after))
    assert int(m.err.item()) == 0


def test_forks_where_every_layer_is_in_four_bits(rb):
    """The table's own pool is then a stand-in of 16 bytes a token."""
    d = rb.Dims(16, 4, 2, 64, max_num_reqs=4, max_model_len=64, max_blocks_per_req=4,
                num_blocks=20)
    k, v = (torch.randint(0, 256, (20, 2, 576), dtype=torch.uint8, device="cuda") for _ in "kv")
    k0, v0 = k.clone(), v.clone()
    table = torch.tensor([[7, 3, 4, -1], [-1] * 4, [-1] * 4], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 0, 0], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    stand_in = [torch.zeros(320, 1, 8, dtype=BF, device="cuda") for _ in "kv"]
    pool = rb.PagePool(rb.Dims(16, 1, 1, 8, 4, 64, 4, 20), *stand_in, table, count)
    view = lambda c: rb.kv4_pages(c).view(20, 2, 288)
    layer = rb.PagePool(rb.kv4_page_dims(d), view(k), view(v))
    pool.fork(i32(0, 0), i32(1, 2), i32(37, 0, 0))  # 37 tokens: two whole pages and five rows
    layer.copy(table[[0, 0], [2, 2]], table[[1, 2], [2, 2]])
    rows = table.tolist()
    assert rows[1][:2] == rows[2][:2] == [7, 3] and len({rows[r][2] for r in range(3)}) == 3
    for r in (1, 2):
        assert torch.equal(k[rows[r][2]], k0[4]) and torch.equal(v[rows[r][2]], v0[4])
    assert int(pool.error_word.item()) == 0 and int(layer.error_word.item()) == 0
