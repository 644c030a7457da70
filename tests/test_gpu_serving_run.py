"""A serving run through the operators together: prompts enter the persistent batch, attention
with score rules runs over the paged cache, requests are forked into samples, finished ones
freed and the pool compacted, and the next tokens' log probabilities are taken from the gathered
rows, every step against the float64 oracles on each request's own contiguous history."""
from types import SimpleNamespace as NS

import numpy as np
import pytest
import torch

from oracle.logprobs import token_logprobs as oracle_logprobs
from oracle.scores import paged_attention_scored as oracle_scored
from test_gpu_scored_attention import _alibi, _compare

pytestmark = pytest.mark.gpu

NH, NKV, HD, VOCAB, WINDOW = 8, 2, 64, 1003, 70


class Run:
    def __init__(self, rb, seed):
        self.rb = rb
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = rb.Dims(block_size=16, num_q_heads=NH, num_kv_heads=NKV, head_dim=HD,
                            max_num_reqs=8, max_model_len=256, max_blocks_per_req=16,
                            num_blocks=40)
        self.batch = rb.PersistentBatch(8, 256, 16)
        self.k = self.randn(640, NKV, HD)
        self.v = self.randn(640, NKV, HD)
        self.pool = rb.PagePool(self.dims, self.k, self.v, batch=self.batch)
        self.head = self.randn(NH * HD, VOCAB)
        self.kv = {}                  # request id -> (keys, values) so far, contiguous
        self.cached = {}              # request id -> cached tokens
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def rows(self, ids):
        return torch.tensor([self.row[i] for i in ids], dtype=torch.int32, device="cuda")

    def apply(self, scheduled, new=(), cached=()):
        self.batch.apply(NS(scheduled=scheduled, new=list(new), cached=list(cached)))
        self.scheduled = scheduled
        got = self.batch.row_of_sched[:len(scheduled)].tolist()
        self.row = dict(zip(scheduled, got))

    def step(self, rules_of):
        """Prepare, write, attend, gather and score the scheduled tokens; checks all of it."""
        rb, b, R = self.rb, self.batch, self.batch.num_reqs
        by_row = sorted(self.scheduled, key=self.row.get)
        q_lens = [self.scheduled[i] for i in by_row]
        N, pad = sum(q_lens), 3
        q, k, v = (self.randn(N + pad, h, HD) for h in (NH, NKV, NKV))
        meta = rb.prepare_inputs(self.dims, R, R, N, N + pad, b.token_table, b.num_computed,
                                 b.num_scheduled, b.block_table)
        rb.kv_write(self.dims, k, v, meta["slot_mapping"], self.k, self.v, error_word=self.err)
        at, starts, prefix = 0, [], []
        for i, n in zip(by_row, q_lens):
            old = self.kv.get(i, (k[:0], v[:0]))
            self.kv[i] = (torch.cat([old[0], k[at:at + n]]), torch.cat([old[1], v[at:at + n]]))
            p = self.cached[i] + np.arange(n)
            starts += list(np.maximum(0, p - WINDOW + 1) if rules_of(i) == "window" else 0 * p)
            prefix.append(20 if rules_of(i) == "prefix" else 0)
            self.cached[i] += n
            at += n
        i32 = lambda xs: torch.as_tensor(np.asarray(xs, np.int32)).cuda()
        slopes = torch.tensor(_alibi(NH), device="cuda")
        rules = rb.ScoreRules(softcap=25.0, head_slopes=slopes, key_start=i32(starts),
                              prefix_lens=i32(prefix))
        args = (self.dims, R, N, q, self.k, self.v, b.block_table, meta["query_start_loc"],
                meta["seq_lens"], rules)
        out = rb.paged_attention_scored(*args, error_word=self.err)
        rows = rb.gather_rows(out.view(N + pad, NH * HD), meta["logits_indices"])
        logits = rows @ self.head
        tokens = torch.randint(VOCAB, (R,), generator=self.gen, device="cuda").to(torch.int32)
        lp = rb.token_logprobs(logits, tokens, 4, error_word=self.err)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0 and int(meta["scalars"][3].item()) == 0
        assert int(self.pool.error_word.item()) == 0 and int(b.error_word.item()) == 0
        f64 = lambda t: t.double().cpu().numpy()
        want, weight = oracle_scored(f64(q), [f64(self.kv[i][0]) for i in by_row],
                                     [f64(self.kv[i][1]) for i in by_row],
                                     meta["query_start_loc"].tolist(), meta["seq_lens"].tolist(),
                                     softcap=25.0, slopes=_alibi(NH), key_start=starts,
                                     prefix_lens=prefix)
        _compare(out, want, weight, N)
        w = oracle_logprobs(f64(logits), tokens.tolist(), 4)
        assert np.abs(f64(lp.logprobs) - w[0]).max() < 1e-4
        assert lp.ranks.tolist() == w[1].tolist() and lp.top_ids.tolist() == w[3].tolist()
        assert np.abs(f64(lp.entropy) - w[2]).max() < 1e-4
        return args, out


def test_serving_run(rb):
    run = Run(rb, 4)
    rules_of = lambda i: {0: "window", 1: "prefix", 2: "causal"}[i % 3]
    prompts = {10: (90, list(range(1, 8))), 11: (37, [20, 9, 31]), 12: (5, [39])}
    run.cached = {i: 0 for i in prompts}
    run.apply({i: n for i, (n, _) in prompts.items()},
              new=[NS(req_id=i, num_computed=0, num_prompt=n, tokens=list(range(n)), blocks=p)
                   for i, (n, p) in prompts.items()])
    run.pool.count()
    run.step(rules_of)
    # two samples of request 10 and one of 12: rows without pages, then forked on the device
    samples = {20: 10, 21: 10, 22: 12}
    for s, i in samples.items():
        run.cached[s] = run.cached[i]
        run.kv[s] = run.kv[i]
    everyone = list(prompts) + list(samples)
    grow = lambda i: NS(req_id=i, num_computed=run.cached[i], new_tokens=[7], new_blocks=[],
                        replace_blocks=False)
    new = [NS(req_id=s, num_computed=run.cached[i], num_prompt=run.cached[i],
              tokens=list(range(run.cached[i])) + [7], blocks=[]) for s, i in samples.items()]
    run.apply({i: 1 for i in everyone}, new=new, cached=[grow(i) for i in prompts])
    run.pool.fork(run.rows(samples.values()), run.rows(samples), run.batch.num_computed)
    counts = run.pool.ref_count.tolist()
    assert sorted(counts)[-5:] == [3, 3, 3, 3, 3]     # request 10's five full pages, three holders
    run.step(rules_of)
    for _ in range(2):                                # decode on: the copies diverge
        run.apply({i: 1 for i in everyone}, cached=[grow(i) for i in everyone])
        run.step(rules_of)
    # requests 10 and 22 finish: free their rows, then the scheduler drops them
    freed = torch.zeros(1, dtype=torch.int32, device="cuda")
    run.pool.free(run.rows([10, 22]), num_freed=freed)
    assert int(freed.item()) == 3                     # 10's tail and spare page, 22's one page
    left = [i for i in everyone if i not in (10, 22)]
    run.apply({i: 1 for i in left}, cached=[grow(i) for i in left])
    run.step(rules_of)
    run.apply({i: 1 for i in left}, cached=[grow(i) for i in left])
    args, before = run.step(rules_of)
    page_map = torch.empty(40, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    run.pool.compact(page_map=page_map, num_live=live)
    n = int(live.item())
    assert sorted(x for x in page_map.tolist() if x >= 0) == list(range(n + 1))
    assert torch.equal(rb.paged_attention_scored(*args), before)   # the same step, pages moved
    run.apply({i: 1 for i in left}, cached=[grow(i) for i in left])
    run.step(rules_of)
    reference = run.pool.ref_count.clone()
    run.pool.count()
    assert torch.equal(run.pool.ref_count, reference)
