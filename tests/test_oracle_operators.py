"""Pins of the operators' oracles: special cases, closed forms and hand-written small cases."""
import math

import numpy as np
import pytest

import oracle
import oracle.logprobs
import oracle.pages as pages
from oracle.scores import paged_attention_scored


def _batch(seed, qc, nh=4, nkv=2, hd=8):
    rng = np.random.default_rng(seed)
    qsl = np.concatenate([[0], np.cumsum([q for q, _ in qc])])
    lens = [q + c for q, c in qc]
    q = rng.normal(size=(qsl[-1], nh, hd))
    keys = [rng.normal(size=(n, nkv, hd)) for n in lens]
    values = [rng.normal(size=(n, nkv, hd)) for n in lens]
    return q, keys, values, qsl, lens


def test_without_rules_it_is_the_attention_oracle():
    qc = [(3, 5), (1, 9), (7, 0)]
    q, keys, values, qsl, lens = _batch(0, qc)
    got, weight = paged_attention_scored(q, keys, values, qsl, lens)
    new = lambda x: np.concatenate([x[i][c:] for i, (_, c) in enumerate(qc)])
    want = oracle.paged_attention(q, [k[:c] for k, (_, c) in zip(keys, qc)],
                                  [v[:c] for v, (_, c) in zip(values, qc)], new(keys),
                                  new(values), qsl, lens, 3)
    assert np.abs(got - want).max() < 1e-12
    assert (weight >= np.abs(got) - 1e-12).all()


def test_score_rules_in_closed_form():
    q, keys, values, qsl, lens = _batch(1, [(4, 3)])
    # a cap of nearly nothing leaves the mean of the visible values
    got, _ = paged_attention_scored(q, keys, values, qsl, lens, softcap=1e-12)
    for j in range(4):
        assert np.abs(got[j, 0] - values[0][:4 + j, 0].mean(0)).max() < 1e-9
    # an enormous cap does nothing; a very steep bias leaves the query's own key, a very steep
    # rising one the farthest
    none, _ = paged_attention_scored(q, keys, values, qsl, lens)
    cap, _ = paged_attention_scored(q, keys, values, qsl, lens, softcap=1e9)
    assert np.abs(none - cap).max() < 1e-12
    near, _ = paged_attention_scored(q, keys, values, qsl, lens, slopes=[1e6] * 4)
    far, _ = paged_attention_scored(q, keys, values, qsl, lens, slopes=[-1e6] * 4)
    for j in range(4):
        assert np.abs(near[j, 3] - values[0][3 + j, 1]).max() < 1e-12
        assert np.abs(far[j, 3] - values[0][0, 1]).max() < 1e-12
    # one visible key, no visible key, a prefix over everything
    one, _ = paged_attention_scored(q, keys, values, qsl, lens, key_start=[3, 4, 99, 6])
    assert np.abs(one[0, 2] - values[0][3, 1]).max() < 1e-12
    assert not one[2].any()
    both, _ = paged_attention_scored(q, keys, values, qsl, lens, prefix_lens=[99])
    s = q[0, 0] @ keys[0][:, 0].T / math.sqrt(8)
    p = np.exp(s) / np.exp(s).sum()
    assert np.abs(both[0, 0] - p @ values[0][:, 0]).max() < 1e-12


def test_unseen_values_do_not_count():
    q, keys, values, qsl, lens = _batch(2, [(3, 4)])
    clean, _ = paged_attention_scored(q, keys, values, qsl, lens, key_start=[2, 2, 5])
    values[0][1] = np.nan
    values[0][6, 0, 0] = np.inf       # the last token's own key
    keys[0][0] = np.nan
    got, _ = paged_attention_scored(q, keys, values, qsl, lens, key_start=[2, 2, 5])
    assert np.abs(got[:2] - clean[:2]).max() < 1e-12    # (sums of fewer terms: another order)
    assert np.isinf(got[2, 0, 0]) and np.abs(got[2, 2:] - clean[2, 2:]).max() < 1e-12


def test_logprobs_closed_forms():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [math.log(1), math.log(2), math.log(5), -np.inf],
                  [-np.inf] * 4, [0, np.nan, 1, 2], [1.0, 3.0, 3.0, 2.0]])
    lp, rank, ent, ids, best = oracle.logprobs.token_logprobs(x, [2, 1, 0, 0, -1], 3)
    assert lp[0] == pytest.approx(-math.log(4)) and ent[0] == pytest.approx(math.log(4))
    assert rank[0] == 1 and ids[0].tolist() == [0, 1, 2]
    assert lp[1] == pytest.approx(math.log(2 / 8)) and rank[1] == 2
    assert ids[1].tolist() == [2, 1, 0] and best[1, 0] == pytest.approx(math.log(5 / 8))
    assert lp[2] == -np.inf and ent[2] == 0 and rank[2] == 1
    assert np.isnan(lp[3]) and rank[3] == 0 and ids[3].tolist() == [-1, -1, -1]
    assert lp[4] == 0 and rank[4] == 0 and ids[4].tolist() == [1, 2, 3]


def test_pages_by_hand():
    k = np.arange(8)[:, None] * np.ones((8, 4), int)
    table = [[3, 6], [6, 2, 7], []]
    ref = pages.count(table, 8)
    assert ref == [0, 0, 1, 1, 0, 0, 2, 1]
    pages.fork(table, ref, [0], [2], [5, 9, 0], 4, 0, [k])   # 5 tokens: one full page, one row
    assert table[2] == [3, 1] and ref == [0, 1, 1, 2, 0, 0, 2, 1]
    assert k[1].tolist() == [6, 1, 1, 1]
    assert pages.free(table, ref, [1]) == 2 and table[1] == []
    assert ref == [0, 1, 0, 2, 0, 0, 1, 0]
    new, live = pages.compact(table, ref, 0, [k])
    assert live == 3 and new == [0, 1, -1, 3, -1, -1, 2, -1]
    assert table == [[3, 2], [], [3, 1]] and ref == [0, 1, 1, 2, 0, 0, 0, 0]
    assert k[2].tolist() == [6] * 4
    pages.copy([1, -1, 1], [4, 5, 6], [k])
    assert k[4].tolist() == k[6].tolist() == [6, 1, 1, 1] and k[5].tolist() == [5] * 4
