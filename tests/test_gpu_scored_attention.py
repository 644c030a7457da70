"""rb_paged_attention_scored against the float64 oracle.

Tolerance of one output value o = sum p_k v_k, with w = sum p_k |v_k|: P is rounded to bf16
before the product (2^-8 of each term: 2^-8 w) and o once at the end (2^-8 |o|).  The scores'
own errors stay far below: fp32 accumulation of hd exact products (hd 2^-24 sum |q_i k_i| scale
<= 128 * 2^-24 * 100 * 0.09 < 2^-13), roundings in log2 units of scores up to 2^7
that matter (a term 2^-40 below the maximum adds nothing) at 2^-24 each (a few 2^-17), and 2^-22 of
ex2; their relative effect on a p is under 2^-11, twice (numerator and sum): 2^-10 w.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from gpu_cases import dims_of, i32, jump_tensors, oracle_meta, to64
from oracle.scores import paged_attention_scored as oracle_scored

pytestmark = pytest.mark.gpu


def _full(spec, tens):
    """Each request's keys and values, history then this step's rows, in float64."""
    qsl = np.concatenate([[0], np.cumsum(spec.num_scheduled)])
    cat = lambda hist, new, i: np.concatenate([to64(hist[i]), to64(new)[qsl[i]:qsl[i + 1]]])
    R = spec.num_reqs
    return ([cat(tens.hist_k, tens.k, i) for i in range(R)],
            [cat(tens.hist_v, tens.v, i) for i in range(R)])


def _setup(rb, spec, tens=None):
    tens = wl.make_tensors(spec, device="cuda") if tens is None else tens
    meta = oracle_meta(spec)
    rb.kv_write(dims_of(spec), tens.k, tens.v, i32(meta["slot_mapping"]), tens.k_cache,
                tens.v_cache)
    return tens, meta


def _rules(rb, softcap=0.0, slopes=None, key_start=None, prefix_lens=None):
    f = lambda a: None if a is None else torch.as_tensor(np.asarray(a, np.float32)).cuda()
    g = lambda a: None if a is None else i32(a)
    return rb.ScoreRules(softcap=softcap, head_slopes=f(slopes), key_start=g(key_start),
                         prefix_lens=g(prefix_lens))


def _compare(got, out, weight, N):
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(out))
    with np.errstate(invalid="ignore"):
        inf = np.isinf(out)
        assert np.array_equal(g[inf], out[inf])
        fine = np.isfinite(out)
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -10) * weight + 1e-30
        diff = np.abs(g - out)
        worst = np.where(fine, diff / tol, 0.0)
    assert worst.max(initial=0.0) <= 1.0, f"{worst.max()} of the tolerance"
    assert np.all(g[N:] == 0.0), "padding rows must be zero"


def _check(rb, spec, tens=None, table=None, **rules):
    tens, meta = _setup(rb, spec, tens)
    R, N = spec.num_reqs, spec.num_tokens
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dims_of(spec), R, N, tens.q, tens.k_cache, tens.v_cache,
            i32(spec.block_table if table is None else table),
            i32(meta["query_start_loc"][:R + 1]), i32(meta["seq_lens"][:R]))
    r = _rules(rb, **rules)
    got = rb.paged_attention_scored(*args, r, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    keys, values = _full(spec, tens)
    out, weight = oracle_scored(to64(tens.q), keys, values, meta["query_start_loc"][:R + 1],
                                meta["seq_lens"][:R], **rules)
    _compare(got, out, weight, N)
    return got, args, r, tens


def _positions(spec):
    return np.concatenate([np.arange(c, c + q) for c, q in
                           zip(spec.num_computed, spec.num_scheduled)] or [np.zeros(0)])


def _documents(spec, rng, mean):
    """First position of the document of each new token, documents packed from position 0."""
    starts = []
    for c, q in zip(spec.num_computed, spec.num_scheduled):
        bounds = [0]
        while bounds[-1] < c + q:
            bounds.append(bounds[-1] + int(rng.integers(1, 2 * mean)))
        starts += [bounds[np.searchsorted(bounds, p, side="right") - 1] for p in range(c, c + q)]
    return np.array(starts, np.int64)


def _alibi(nh):
    return [2.0 ** (-8.0 * (h + 1) / nh) for h in range(nh)]


HEADS = [(4, 4), (4, 2), (8, 2), (16, 2), (32, 8), (16, 1), (6, 2), (12, 2), (28, 4), (10, 1),
         (14, 2), (15, 1)]


@pytest.mark.parametrize("seed", range(48))
def test_fuzzed_mixes_and_rules(rb, seed):
    nh, nkv = HEADS[seed % 12]
    hd = 64 if seed % 2 else 128
    spec = wl.random_batch(seed, num_q_heads=nh, num_kv_heads=nkv, head_dim=hd, max_reqs=7,
                           max_q=150, max_c=400, pad_tokens=seed % 4, decode_frac=0.5)
    rng = np.random.default_rng(seed)
    pos = _positions(spec)
    lens = np.asarray(spec.num_computed) + np.asarray(spec.num_scheduled)
    rules = {}
    if rng.random() < 0.5:
        rules["softcap"] = float(rng.choice([2.0, 20.0, 50.0]))
    if rng.random() < 0.5:
        rules["slopes"] = _alibi(nh)
    kind = int(rng.integers(0, 5))
    if kind == 1:
        rules["key_start"] = pos - int(rng.integers(1, 200)) + 1            # a window
    elif kind == 2:
        rules["key_start"] = _documents(spec, rng, int(rng.choice([3, 40, 200])))
    elif kind == 3:
        rules["key_start"] = rng.integers(-5, int(lens.max()) + 20, size=len(pos))  # any
    if rng.random() < 0.4:
        rules["prefix_lens"] = rng.integers(-3, int(lens.max()) + 30, size=spec.num_reqs)
    _check(rb, spec, **rules)


@pytest.mark.parametrize("q,c", [(1, 0), (1, 1), (1, 15), (1, 16), (1, 127), (2, 30), (8, 0),
                                 (9, 40), (63, 1), (64, 0), (65, 64), (127, 1), (128, 0),
                                 (129, 127), (200, 0), (1, 1000)])
def test_edge_lengths(rb, q, c):
    for nh, nkv in ((8, 1), (4, 2), (8, 8), (7, 1)):
        spec = wl.batch_from_lists([c, 3], [q, 1], num_q_heads=nh, num_kv_heads=nkv,
                                   head_dim=128, seed=q * 1000 + c)
        L = c + q
        for start in (0, 1, L // 2, L - 1, L):
            _check(rb, spec, softcap=30.0, slopes=_alibi(nh),
                   key_start=[start] * q + [0], prefix_lens=[L // 3, 2])
        _check(rb, spec, prefix_lens=[L, 10])


def test_rows_that_see_nothing_are_zero(rb):
    spec = wl.batch_from_lists([300, 20, 0, 700], [1, 3, 150, 200], num_q_heads=8,
                               num_kv_heads=2, head_dim=64, seed=3)
    start = np.zeros(spec.num_tokens, np.int64)
    start[0] = 301                       # a whole decode
    start[2] = 1000                      # one of three tokens
    start[4:154] = 1 << 30               # a whole prompt
    start[160:330:7] = 2000              # some rows of a chunk
    got, _, _, _ = _check(rb, spec, key_start=start, slopes=_alibi(8))
    assert not got[0].any() and not got[2].any() and not got[4:154].any()
    assert got[1].any() and got[155].any()


@pytest.mark.parametrize("slopes", [0.9, 3.0, -0.5, 1e-4])
def test_steep_rising_and_flat_biases(rb, slopes):
    """Scores that change by hundreds between key tiles, either way."""
    spec = wl.batch_from_lists([900, 0, 700, 1500], [200, 500, 1, 1], num_q_heads=8,
                               num_kv_heads=2, head_dim=128, seed=7)
    s = [slopes * (1 + h / 8) for h in range(8)]
    _check(rb, spec, slopes=s)
    _check(rb, spec, slopes=s, prefix_lens=[600, 300, 100, 1501], softcap=10.0)


@pytest.mark.parametrize("nh,nkv,hd", [(32, 8, 128), (8, 1, 128), (12, 2, 64)])
def test_score_jumps_across_key_tiles(rb, nh, nkv, hd):
    spec = wl.batch_from_lists([600, 0, 700], [300, 400, 1], num_q_heads=nh, num_kv_heads=nkv,
                               head_dim=hd, seed=nh * 100 + hd)
    scale = 128 / hd
    for hot in ({(300, 340): 2.0 * scale, (560, 570): 4.0 * scale},
                {(0, 20): 6.0 * scale, (330, 340): 3.0 * scale}):
        tens = jump_tensors(spec, hot)
        _check(rb, spec, tens=tens)
        _check(rb, spec, tens=tens, softcap=40.0, slopes=_alibi(nh))


@pytest.mark.parametrize("softcap", [0.05, 1.0, 15.0, 3e4, 1e8])
def test_soft_caps_of_any_size(rb, softcap):
    """Far below the scores (all near +-cap) to far above (no effect: tanh u = u)."""
    spec = wl.batch_from_lists([100, 0, 333], [60, 130, 1], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=11)
    _check(rb, spec, softcap=softcap)


def test_prefix_rows_that_do_not_see_their_own_key(rb):
    """A prefix ahead of the query and a first key past it: with a steep bias every visible score
    lies far below the soft cap's range (by hundreds of log2 units)."""
    spec = wl.batch_from_lists([0, 100, 5], [300, 150, 1], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=12)
    start = np.concatenate([np.full(300, 280), np.full(150, 240), [0]])
    for softcap in (30.0, 60.0, 0.0):
        _check(rb, spec, softcap=softcap, slopes=[1.0 + h for h in range(8)], key_start=start,
               prefix_lens=[300, 250, 6])


def test_capped_scores_at_both_ends_and_large_values(rb):
    """Scores that go from -cap to cap along a row, with V up to 1e12."""
    spec = wl.batch_from_lists([600, 0, 700], [300, 400, 1], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=14)
    tens = jump_tensors(spec, {(0, 256): 3.0, (300, 340): -20.0, (560, 700): 20.0})
    for v in [tens.v] + tens.hist_v:
        v.mul_(2.0 ** 40)
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    for softcap in (20.0, 50.0, 70.0):
        _check(rb, spec, tens=tens, softcap=softcap)
        _check(rb, spec, tens=tens, softcap=softcap, slopes=_alibi(8))


def test_long_decodes_are_split(rb):
    spec = wl.batch_from_lists([20000, 9000, 100], [1, 1, 2], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=2)
    _check(rb, spec, softcap=25.0, slopes=_alibi(8))
    _check(rb, spec, key_start=[12345, 8990, 7, 8])
    _check(rb, spec, key_start=[19000, 100, 0, 0], slopes=_alibi(8))


@pytest.mark.parametrize("ratio", [1, 2])
def test_pages_nobody_sees_may_be_gone(rb, ratio):
    """A window's old pages: their entries are -1 and their rows hold NaN; the rows of the first
    visible page before the window hold NaN too."""
    spec = wl.batch_from_lists([500, 333, 1000], [1, 90, 5], num_q_heads=8, num_kv_heads=2,
                               head_dim=64, seed=5, manager_ratio=ratio)
    tens = wl.make_tensors(spec, device="cuda")
    pos = _positions(spec)
    start = np.maximum(0, pos - 100)
    table = np.array(spec.block_table)
    qsl = np.concatenate([[0], np.cumsum(spec.num_scheduled)])
    pt = 16 * ratio
    for i in range(spec.num_reqs):
        first = int(start[qsl[i]])
        tens.hist_k[i][:first] = float("nan")
        tens.hist_v[i][:first] = float("inf")
        table[i, :first // pt] = -1
    wl.place_history(spec, tens.hist_k, tens.k_cache)
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    _check(rb, spec, tens=tens, table=table, key_start=start)


def test_what_lies_past_a_sequence_does_not_matter(rb):
    spec = wl.batch_from_lists([500, 0, 30], [1, 90, 2], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=6)
    tens = wl.make_tensors(spec, device="cuda")
    tens.k_cache.fill_(float("nan"))
    tens.v_cache.fill_(float("nan"))
    wl.place_history(spec, tens.hist_k, tens.k_cache)
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    _check(rb, spec, tens=tens, softcap=30.0, prefix_lens=[10, 500, 500])


def test_without_rules_it_is_paged_attention(rb):
    spec = wl.config2()
    tens, meta = _setup(rb, spec)
    R, N = spec.num_reqs, spec.num_tokens
    args = (dims_of(spec), R, N, tens.q, tens.k_cache, tens.v_cache, i32(spec.block_table),
            i32(meta["query_start_loc"][:R + 1]), i32(meta["seq_lens"][:R]))
    a = rb.paged_attention(*args).float()
    b = rb.paged_attention_scored(*args, rb.ScoreRules()).float()
    assert (a - b).abs().max().item() <= 2e-2 and (a - b).abs().mean().item() <= 2e-3


def test_runs_agree_bit_for_bit(rb):
    spec = wl.batch_from_lists([3000, 0, 700, 40], [1, 400, 1, 3], num_q_heads=8,
                               num_kv_heads=2, head_dim=128, seed=8)
    got, args, r, _ = _check(rb, spec, softcap=30.0, slopes=_alibi(8), prefix_lens=[5, 90, 0, 43])
    for _ in range(5):
        assert torch.equal(rb.paged_attention_scored(*args, r), got)


def test_captured_and_replayed_on_another_stream(rb):
    spec = wl.batch_from_lists([300, 0, 700], [1, 200, 1], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=9)
    start = np.maximum(0, _positions(spec) - 50)
    got, args, r, tens = _check(rb, spec, key_start=start, softcap=20.0)
    out = torch.empty_like(tens.q)
    ws = torch.empty(rb.workspace_size(args[0], args[1], args[2]), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rb.paged_attention_scored(*args, r, out=out, workspace=ws)
    for k in range(3):   # the rules' arrays are read at the replay
        r.key_start.copy_(i32(np.maximum(0, _positions(spec) - 50 * k)))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rb.paged_attention_scored(*args, r))


def test_two_calls_at_once(rb):
    """Two streams, each with its own workspace."""
    calls = []
    for seed in (1, 2):
        spec = wl.batch_from_lists([3000, 100, 700], [1, 300, 1], num_q_heads=8, num_kv_heads=2,
                                   head_dim=128, seed=seed)
        calls.append(_check(rb, spec, slopes=_alibi(8)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [rb.paged_attention_scored(*args, r, stream=s)
                for (_, args, r, _), s in zip(calls, streams)]
        torch.cuda.synchronize()
        for o, (got, _, _, _) in zip(outs, calls):
            assert torch.equal(o, got)


def test_bad_pages_and_metadata_are_flagged(rb):
    spec = wl.batch_from_lists([5, 0], [1, 20], num_q_heads=4, num_kv_heads=2, head_dim=64)
    tens, meta = _setup(rb, spec)
    dims = dims_of(spec)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rules = rb.ScoreRules(softcap=30.0)

    def call(bt, sl):
        err.zero_()
        rb.paged_attention_scored(dims, 2, 21, tens.q, tens.k_cache, tens.v_cache, i32(bt),
                                  i32(meta["query_start_loc"][:3]), i32(sl), rules,
                                  error_word=err)
        return int(err.item())

    sl = meta["seq_lens"][:2]
    assert call(spec.block_table, [6, 3]) & rb.EBIT_ATTN_META
    for row in (0, 1):
        bt = spec.block_table.copy()
        bt[row, 0] = spec.dims.num_blocks + 5
        assert call(bt, sl) == rb.EBIT_BLOCK_ID
        bt[row, 0] = 0                                        # the null page
        assert call(bt, sl) == rb.EBIT_BLOCK_ID
    assert call(spec.block_table, sl) == 0


@pytest.mark.parametrize("nh,nkv,hd", [(8, 2, 128), (4, 4, 64), (12, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("kind", ["documents", "window", "prefix", "causal"])
def test_infinities_and_nan_stay_with_the_rows_that_see_them(rb, nh, nkv, hd, kind):
    """K and V of some keys are infinite or NaN: rows that do not see those keys are as without
    them, rows that do get infinities and NaN (the oracle leaves unseen keys out of its sums)."""
    spec = wl.batch_from_lists([300, 0, 40, 17, 500], [200, 390, 2, 1, 3], num_q_heads=nh,
                               num_kv_heads=nkv, head_dim=hd, seed=nh + hd)
    tens = wl.make_tensors(spec, device="cuda")
    rng = np.random.default_rng(3)
    pos = _positions(spec)
    qsl = np.concatenate([[0], np.cumsum(spec.num_scheduled)])
    rules = {"documents": lambda: dict(key_start=_documents(spec, rng, 60)),
             "window": lambda: dict(key_start=pos - 20, softcap=30.0),
             "prefix": lambda: dict(prefix_lens=[350, 33, 41, 5, 499], slopes=_alibi(nh)),
             "causal": lambda: dict()}[kind]()
    bad = [float("inf"), float("-inf"), float("nan")]
    for i in range(spec.num_reqs):
        c, q = int(spec.num_computed[i]), int(spec.num_scheduled[i])
        for n, p in enumerate(rng.choice(c + q, size=5, replace=False).tolist() + [c + q - 1]):
            hist = p < c
            kv = (tens.hist_v[i] if hist else tens.v)
            row = p if hist else int(qsl[i]) + p - c
            kv[row, int(rng.integers(nkv)), int(rng.integers(hd))] = bad[n % 3]
            if n == 2:   # a key that is NaN makes its readers' rows NaN, and only theirs
                (tens.hist_k[i] if hist else tens.k)[row, :, 5] = float("nan")
    wl.place_history(spec, tens.hist_k, tens.k_cache)
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    got, _, _, _ = _check(rb, spec, tens=tens, **rules)
    finite = torch.isfinite(got.float()).flatten(1).all(1)
    assert not bool(finite.all())
    if kind != "prefix":      # (there every row may see a NaN key)
        assert bool(finite.any())


def test_a_step_without_requests_writes_padding_only(rb):
    spec = wl.batch_from_lists([5], [3], num_q_heads=4, num_kv_heads=2, head_dim=128, seed=1)
    tens, _ = _setup(rb, spec)
    q = torch.randn(24, 4, 128, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.empty(rb.workspace_size(dims_of(spec), 1, 8), dtype=torch.uint8, device="cuda")
    r = _rules(rb, softcap=20.0, slopes=_alibi(4), key_start=[0], prefix_lens=[0])
    rb.paged_attention_scored(dims_of(spec), 0, 0, q, tens.k_cache, tens.v_cache,
                              i32(spec.block_table), i32([0]), i32([0]), r, out=out,
                              workspace=work, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not out.any()


@pytest.mark.parametrize("nh,nkv,hd", [(8, 1, 128), (8, 2, 64), (6, 3, 128), (16, 1, 64)])
def test_merges_of_many_splits(rb, nh, nkv, hd):
    """Splits of one to some hundred per request, next to each other; infinities in the last."""
    spec = wl.batch_from_lists([33000, 12345, 4100, 130, 15, 1], [1, 1, 1, 1, 1, 1],
                               num_q_heads=nh, num_kv_heads=nkv, head_dim=hd, seed=nh)
    tens = wl.make_tensors(spec, device="cuda")
    tens.hist_v[0][-1, :, 3] = float("inf")
    tens.hist_v[1][5, :, 4] = float("-inf")
    for hist, cache in ((tens.hist_k, tens.k_cache), (tens.hist_v, tens.v_cache)):
        wl.place_history(spec, hist, cache)
    _check(rb, spec, tens=tens)
    _check(rb, spec, slopes=_alibi(nh), key_start=[1000, 0, 4090, 5, 16, 0])


def _check_with_pages_gone(rb, c, q, start, gone, nh, nkv, ratio=1):
    """One request of q tokens behind c cached ones, its pages `gone` out of the table, their
    rows NaN and infinite."""
    spec = wl.batch_from_lists([c], [q], num_q_heads=nh, num_kv_heads=nkv, head_dim=64, seed=c,
                               manager_ratio=ratio)
    tens = wl.make_tensors(spec, device="cuda")
    table = np.array(spec.block_table)
    for page in gone:
        table[0, page] = -1
        keys = slice(page * 16 * ratio, min(c, (page + 1) * 16 * ratio))
        tens.hist_k[0][keys] = float("nan")
        tens.hist_v[0][keys] = float("inf")
    wl.place_history(spec, tens.hist_k, tens.k_cache)
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    for rules in ({}, dict(softcap=20.0, slopes=_alibi(nh))):
        _check(rb, spec, tens=tens, table=table, key_start=start, **rules)


@pytest.mark.parametrize("ratio", [1, 2])
def test_pages_before_rows_that_see_nothing_may_be_gone(rb, ratio):
    """Tokens with a window of no keys do not make the pages of their empty window read: a
    prompt (rows that see something start later), a decode of several tokens, and requests none
    of whose tokens sees a key."""
    old = lambda key: range(key // (16 * ratio))
    # a chunk: positions 333 .. 422; the first ten see nothing, the others their own and 2 before
    pos = np.arange(333, 423)
    start = np.where(pos < 343, pos + 1, pos - 2)
    _check_with_pages_gone(rb, 333, 90, start, old(341), 8, 2, ratio)
    # decode of 8 tokens of one head: positions 505 .. 512, only the last sees a key, its own
    start = np.append(np.arange(505, 512) + 1, 512)
    _check_with_pages_gone(rb, 505, 8, start, old(512), 1, 1, ratio)
    # nobody sees a key: no page is needed, the last one neither
    for c, q, nh, nkv in ((500, 1, 8, 2), (500, 2, 4, 2), (300, 60, 8, 2), (31, 1, 2, 2)):
        pos = np.arange(c, c + q)
        pages = range(-(-(c + q) // (16 * ratio)))
        _check_with_pages_gone(rb, c, q, pos + 1, pages, nh, nkv, ratio)
        _check_with_pages_gone(rb, c, q, np.full(q, 1 << 30), pages, nh, nkv, ratio)



def test_splits_of_a_decode_whose_first_tokens_see_nothing(rb):
    """Several splits per request; a token that sees nothing beside tokens that see infinities."""
    spec = wl.batch_from_lists([5000, 3000], [4, 2], num_q_heads=4, num_kv_heads=2, head_dim=128,
                               seed=15)
    tens = wl.make_tensors(spec, device="cuda")
    tens.hist_v[0][4321, :, 3] = float("inf")
    tens.hist_v[1][17, :, 4] = float("nan")
    wl.place_history(spec, tens.hist_v, tens.v_cache)
    start = [5001, 1000, 1 << 30, 4400, 3001, 0]
    got, _, _, _ = _check(rb, spec, tens=tens, key_start=start, slopes=_alibi(4))
    assert not got[0].any() and not got[2].any() and not got[4].any()


@pytest.mark.parametrize("q", [1, 150])
@pytest.mark.parametrize("softcap", [50.0, 66.0, 70.0, 100.0, 300.0, 1000.0, 4000.0, 16000.0])
def test_soft_cap_keeps_its_precision(rb, softcap, q):
    """Scores about 0.3 and 0.7 of the cap, the two sides of each worth +v and -v: an error of
    the cap that differs from side to side moves the sum.

    Tolerance: the raw scores are exact here (multiples of 2^-6 below 2^14, in every order of
    summation).  With c = cap log2(e), a capped score in log2 units is off by 2^-11 at most from
    its tanh as the polynomial has it; by 2 c r (E r 2^-22 + 2^-24 + 2^-23) with E = e^2u and
    r = 1 / (1 + E) where the exponential form has it (ex2, the sum, the reciprocal), which is
    below 2^-22 c for u >= 0.3; and by two roundings of its size, 2 x 2^-24 c.  Each probability
    then moves by ln 2 of that, relatively, and o = sum p v / sum p by that times
    sum p |v - o| <= w + |o|; P and the output are rounded to bf16 (2^-8 each) as everywhere."""
    c = softcap * 1.4426950408889634
    for u in (0.3162, 0.7071):
        spec = wl.batch_from_lists([700 - q], [q], num_q_heads=4, num_kv_heads=2, head_dim=128,
                                   seed=int(softcap))
        tens = wl.make_tensors(spec, device="cuda")
        g = torch.Generator().manual_seed(int(softcap))
        L = 700
        border = int(u * softcap)
        fine = torch.randint(-96, 97, (L, 2), generator=g).float() / 64       # within 1.5
        fine = torch.round((fine + u * softcap - border) * 64) / 64
        keys = torch.zeros(L, 2, 128)
        keys[:, :, 0] = border // 64            # (bf16 holds whole numbers up to 256)
        keys[:, :, 1] = border % 64
        keys[:, :, 2] = fine
        values = torch.rand(L, 2, 128, generator=g) + 0.5
        side = fine > u * softcap - border
        values = torch.where(side[..., None], -values, values)
        keys, values = keys.to(torch.bfloat16), values.to(torch.bfloat16)
        tens.q.zero_()
        tens.q[:, :, 0], tens.q[:, :, 1], tens.q[:, :, 2] = 64.0, 1.0, 1.0
        tens.hist_k[0].copy_(keys[:700 - q])
        tens.hist_v[0].copy_(values[:700 - q])
        tens.k[:q], tens.v[:q] = keys[700 - q:].cuda(), values[700 - q:].cuda()
        wl.place_history(spec, tens.hist_k, tens.k_cache)
        wl.place_history(spec, tens.hist_v, tens.v_cache)
        tens, meta = _setup(rb, spec, tens)
        got = rb.paged_attention_scored(
            dims_of(spec), 1, q, tens.q, tens.k_cache, tens.v_cache, i32(spec.block_table),
            i32(meta["query_start_loc"][:2]), i32(meta["seq_lens"][:1]),
            rb.ScoreRules(softcap=softcap), softmax_scale=1.0)
        ks, vs = _full(spec, tens)
        out, weight = oracle_scored(to64(tens.q), ks, vs, meta["query_start_loc"][:2],
                                    meta["seq_lens"][:1], scale=1.0, softcap=softcap)
        off = np.log(2.0) * (2.0 ** -11 + (2.0 ** -22 + 2.0 ** -23) * c)
        tol = ((2.0 ** -8 + off) * (np.abs(out) + weight)) + 1e-30
        worst = (np.abs(got.double().cpu().numpy() - out) / tol).max()
        assert worst <= 1.0, (u, worst)


@pytest.mark.parametrize("softcap", [3.0, 12.0, 20.0, 50.0, 51.0])
def test_capped_scores_at_either_end_with_values_of_any_size(rb, softcap):
    """Rows whose scores are all at +cap, all at -cap, and that go from one to the other either
    way, with V about 2^80 and 2^-60."""
    spec = wl.batch_from_lists([600, 0, 700, 900], [300, 400, 1, 150], num_q_heads=8,
                               num_kv_heads=2, head_dim=128, seed=16)
    everywhere = 40.0
    for hot in ({(0, 2000): everywhere}, {(0, 2000): -everywhere},
                {(0, 300): everywhere, (300, 2000): -everywhere},
                {(0, 300): -everywhere, (300, 2000): everywhere}):
        for size in (2.0 ** 80, 2.0 ** -60):
            tens = jump_tensors(spec, hot)
            for v in [tens.v] + tens.hist_v:
                v.mul_(size)
            wl.place_history(spec, tens.hist_v, tens.v_cache)
            _check(rb, spec, tens=tens, softcap=softcap)
            _check(rb, spec, tens=tens, softcap=softcap, slopes=_alibi(8))
            _check(rb, spec, tens=tens, softcap=softcap, slopes=_alibi(8),
                   prefix_lens=[700, 256, 701, 1050])
