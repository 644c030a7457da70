"""rb_paged_attention_kv4 against the float64 attention oracle over the values that the cache's bytes
stand for.

Tolerance of one output value o = sum p_k v_k, with w = sum p_k |v_k|: P is rounded to fp16 before
the product (2^-11 of each term) and o once to bf16 (2^-8 |o|).  K and V are exact; so is Q (fp16 of
bf16 over a power of two, but for values below 2^-14 of the row's largest: 2^-25 of it).  fp32
scores: hd roundings of a sum whose terms are together below S = max sum |q_i k_i| scale, 2^-24 hd S
<= 2^-17 S, with S below 50 in these cases: 2^-11; the roundings in log2 units (2^7 at most: 2^-17)
and ex2 (2^-22) less; twice (numerator and sum): 2^-10 w.  Weights below 2^-31 of a row's reference
vanish: 2^-30 times keys times max |v| covers them.
"""
import dataclasses

import numpy as np
import pytest
import torch

import workloads as wl
from gpu_cases import dims_of, i32, oracle_meta, to64
from oracle import kv4 as ref
from oracle.scores import paged_attention_scored as oracle_attention

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _bytes(rng, pages, nkv, hd, values, sb=(44, 64)):
    """Random codes with scales of 0.375 to 2, as bytes, and the values they stand for."""
    code = rng.integers(0, 16, (pages, 16, nkv, hd)).astype(np.uint8)
    s = rng.integers(*sb, (pages, 16, nkv, hd // 16)).astype(np.uint8)
    return ref.pack(code, s, values), ref.decode(code, s).reshape(pages * 16, nkv, hd)


class Batch:
    def __init__(self, spec, seed=0, q_scale=1.0, k_scale=1.0, v_scale=1.0, sb=(44, 64)):
        self.spec, self.d = spec, dims_of(spec)
        d, rng = self.d, np.random.default_rng(seed)
        self.k_scale, self.v_scale = k_scale, v_scale
        meta = oracle_meta(spec)
        self.R, self.N = spec.num_reqs, spec.num_tokens
        self.qsl, self.lens = meta["query_start_loc"][:self.R + 1], meta["seq_lens"][:self.R]
        self.k, kv = _bytes(rng, d.num_blocks, d.num_kv_heads, d.head_dim, False, sb)
        self.v, vv = _bytes(rng, d.num_blocks, d.num_kv_heads, d.head_dim, True, sb)
        r = max(1, d.kernel_blocks_per_manager_block)
        used = np.zeros(d.num_blocks * 16, bool)
        self.keys, self.values = [], []
        for i in range(self.R):
            p = np.arange(self.lens[i])
            page = spec.block_table[i, p // (16 * r)] * r + p // 16 % r
            slot = page * 16 + p % 16
            used[slot] = True
            self.keys.append(kv[slot] * k_scale)
            self.values.append(vv[slot] * v_scale)
        # what no request owns holds any bytes
        for cache, values in ((self.k, False), (self.v, True)):
            code, s = (x.copy() for x in ref.unpack(cache, d.head_dim, values))
            code, s = code.reshape(-1, *code.shape[2:]), s.reshape(-1, *s.shape[2:])
            code[~used] = rng.integers(0, 16, code[~used].shape)
            s[~used] = rng.integers(0, 256, s[~used].shape)
            shape = (d.num_blocks, 16, d.num_kv_heads, -1)
            cache[:] = ref.pack(code.reshape(shape), s.reshape(shape), values)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = (q_scale / k_scale * torch.randn(spec.num_tokens_padded, d.num_q_heads,
                                                  d.head_dim, generator=g, device="cuda")).to(BF)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, table=None):
        c = lambda x: torch.from_numpy(x).cuda()
        return (self.d, self.R, self.N, self.q, c(self.k), c(self.v),
                i32(self.spec.block_table if table is None else table), i32(self.qsl),
                i32(self.lens))

    def run(self, rb, **kw):
        out = rb.paged_attention_kv4(*self.args(), k_scale=self.k_scale, v_scale=self.v_scale,
                                     error_word=self.err, **kw)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        return out

    def check(self, got, softmax_scale=None):
        out, weight = oracle_attention(to64(self.q), self.keys, self.values, self.qsl, self.lens,
                                       scale=softmax_scale)
        g = got.double().cpu().numpy()
        top = max((np.abs(v).max() for v in self.values if v.size), default=0.0)
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -10) * weight + \
            2.0 ** -30 * max(self.lens, default=0) * top + 1e-30
        worst = (np.abs(g - out) / tol).max(initial=0.0)
        assert worst <= 1.0, f"{worst} of the tolerance"
        assert np.all(g[self.N:] == 0.0), "padding rows must be zero"


HEADS = [(4, 4), (4, 2), (8, 2), (16, 2), (32, 8), (16, 1), (6, 2), (12, 2), (28, 4), (10, 1),
         (14, 2), (15, 1)]


@pytest.mark.parametrize("q,c", [(1, 0), (1, 1), (1, 15), (1, 16), (1, 17), (1, 31), (1, 48),
                                 (1, 127), (1, 700)])
@pytest.mark.parametrize("nh,nkv,hd", [(4, 2, 128), (8, 1, 64), (3, 3, 128), (7, 1, 64)])
def test_decodes(rb, q, c, nh, nkv, hd):
    spec = wl.batch_from_lists([c, 3], [q, 1], num_q_heads=nh, num_kv_heads=nkv, head_dim=hd,
                               seed=c)
    b = Batch(spec, seed=c)
    b.check(b.run(rb))


@pytest.mark.parametrize("q,c", [(2, 30), (8, 0), (9, 40), (63, 1), (64, 0), (65, 64), (127, 1),
                                 (128, 0), (129, 127), (200, 0), (1, 3000), (300, 500)])
@pytest.mark.parametrize("nh,nkv,hd", [(8, 1, 128), (4, 2, 64), (8, 8, 128), (7, 1, 128)])
def test_prompts(rb, q, c, nh, nkv, hd):
    spec = wl.batch_from_lists([c, 3], [q, 1], num_q_heads=nh, num_kv_heads=nkv, head_dim=hd,
                               seed=q * 1000 + c)
    b = Batch(spec, seed=q)
    b.check(b.run(rb))


@pytest.mark.parametrize("seed", range(36))
def test_fuzzed_mixes(rb, seed):
    nh, nkv = HEADS[seed % 12]
    spec = wl.random_batch(seed, num_q_heads=nh, num_kv_heads=nkv, head_dim=64 if seed % 2 else 128,
                           max_reqs=9, max_q=170, max_c=500, pad_tokens=seed % 4, decode_frac=0.5)
    b = Batch(spec, seed, k_scale=[1.0, 0.25, 3.7][seed % 3], v_scale=[1.0, 9.0][seed % 2])
    b.check(b.run(rb))


def test_queries_of_any_size(rb):
    """Rows of Q from 1e-30 to 1e30 (with layer scales to match) keep their bits."""
    spec = wl.batch_from_lists([40, 5, 70], [1, 70, 2], num_q_heads=4, num_kv_heads=2, head_dim=64,
                               seed=5)
    for size in (1e-30, 1e-6, 1e6, 1e30):
        b = Batch(spec, 3)
        g = torch.Generator(device="cuda").manual_seed(1)
        b.q = (size * torch.randn(b.q.shape, generator=g, device="cuda")).to(BF)
        scale = 0.125 / size
        b.check(b.run(rb, softmax_scale=scale), scale)


@pytest.mark.parametrize("sb,size", [((0, 8), 300.0), ((0, 20), 60.0), ((120, 128), 0.002)])
@pytest.mark.parametrize("hd", [64, 128])
def test_smallest_and_largest_scales(rb, hd, sb, size):
    """Subnormal scales (2^-9 and up) and the largest ones (480), decodes and prompts."""
    spec = wl.batch_from_lists([200, 77, 30], [1, 150, 2], num_q_heads=4, num_kv_heads=2,
                               head_dim=hd, seed=9)
    b = Batch(spec, 6, q_scale=size, sb=sb)
    b.check(b.run(rb))


def test_a_key_far_above_the_others_first_and_last(rb):
    """One key's score exceeds the others' by 2^5 to 2^20 in weight, at either end of a long
    sequence: the vanishing share of the many others is still theirs."""
    for place in (0, 1999):
        for gap in (4.0, 12.0):
            spec = wl.batch_from_lists([1999, 1870], [1, 130], num_q_heads=2, num_kv_heads=1,
                                       head_dim=64, seed=1)
            b = Batch(spec, 2, sb=(40, 48))
            # every key but one is 0 (score 0), the one aligned with the queries
            d = b.d
            code, s = (x.copy() for x in ref.unpack(b.k, 64, False))
            for i in range(2):
                p = np.arange(b.lens[i])
                page, off = spec.block_table[i, p // 16], p % 16
                code[page, off] = 0
                code[page[place], off[place]] = 2
                s[page[place], off[place]] = 56
                b.keys[i][:] = 0
                b.keys[i][place] = 1
            b.k = ref.pack(code, s, False)
            b.q = torch.full_like(b.q, gap / 8)  # score gap / 8 * 64 / 8 = gap
            b.check(b.run(rb))


def test_rising_scores_move_the_reference(rb):
    """Scores that climb by 40 (log2 units) over a sequence: references move, sums stay right."""
    spec = wl.batch_from_lists([1500, 900], [1, 600], num_q_heads=4, num_kv_heads=2, head_dim=128,
                               seed=2)
    b = Batch(spec, 4, sb=(40, 48))
    code, s = (x.copy() for x in ref.unpack(b.k, 128, False))
    for i in range(2):
        p = np.arange(b.lens[i])
        page, off = spec.block_table[i, p // 16], p % 16
        code[page, off] = 2
        s[page, off] = (p * 80 // b.lens[i] + 8)[:, None, None]   # 2^-6 up to 2^3 and more
        b.keys[i][:] = ref.decode(code[page, off], s[page, off])
    b.k = ref.pack(code, s, False)
    b.q = torch.full_like(b.q, 0.125)
    b.check(b.run(rb))


def _scaled_check(b, got, rows=None):
    """As ``Batch.check``, in units of the values' layer scale."""
    v = [x / b.v_scale for x in b.values]
    out, weight = oracle_attention(to64(b.q), b.keys, v, b.qsl, b.lens)
    g = got.double().cpu().numpy() / b.v_scale
    top = max(np.abs(x).max() for x in v)
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -10) * weight + \
        2.0 ** -30 * max(b.lens) * top
    near = np.abs(g - out) <= tol
    assert (near if rows is None else near[rows]).all()


@pytest.mark.parametrize("k_scale", [2.0 ** -100, 2.0 ** -40, 1e-9])
@pytest.mark.parametrize("nh,nkv,hd", [(4, 2, 64), (8, 1, 128), (6, 2, 128)])
def test_rows_of_zeros_over_a_small_layer_scale(rb, k_scale, nh, nkv, hd):
    """Their scores are 0 and the result is V's mean, whatever the scale; tiny rows are next to it.
    Pages partly filled and odd counts of them, in one piece and in many; prompts."""
    spec = wl.batch_from_lists([40, 5, 70, 1500, 0, 333], [1, 70, 2, 1, 130, 1], num_q_heads=nh,
                               num_kv_heads=nkv, head_dim=hd, seed=5)
    b = Batch(spec, 3, k_scale=k_scale)
    b.q[::2] = 0
    b.q[1::6] = (1e-38 * torch.randn(b.q[1::6].shape, device="cuda")).to(BF)
    b.q[:, 0] = 0
    _scaled_check(b, b.run(rb))
    b.q.zero_()
    _scaled_check(b, b.run(rb))


@pytest.mark.parametrize("q_size,k_scale", [(1e5, 1.0), (3e7, 1.0), (1e12, 1.0), (1e30, 1.0),
                                            (1.0, 1e30), (1e30, 2.0 ** 100), (1e35, 2.0 ** 100)])
@pytest.mark.parametrize("nh,nkv,hd", [(4, 2, 64), (8, 1, 128)])
def test_scores_of_any_size(rb, q_size, k_scale, nh, nkv, hd):
    """Scores from 1e6 to 1e66: a row is the value of its largest score, exactly, and rows of zeros
    among them are V's mean.  Sums of fp32 (hd roundings of terms together below S: 2^-24 hd S) tell the
    two largest scores of a row apart in the rows that are compared."""
    spec = wl.batch_from_lists([40, 5, 70, 1500, 0, 333], [1, 70, 2, 1, 130, 1], num_q_heads=nh,
                               num_kv_heads=nkv, head_dim=hd, seed=5)
    b = Batch(spec, 3, k_scale=k_scale, v_scale=4.0)
    b.q = (q_size * torch.randn(b.q.shape, generator=torch.Generator(device="cuda").manual_seed(2),
                                device="cuda")).to(BF)
    b.q[3::7] = 0
    got = b.run(rb)
    assert bool(torch.isfinite(got).all())
    rows = np.zeros(b.q.shape[:2], bool)
    q = to64(b.q)
    for i in range(b.R):
        for t in range(b.qsl[i], b.qsl[i + 1]):
            n = b.lens[i] - (b.qsl[i + 1] - 1 - t)
            for h in range(nh):
                k = b.keys[i][:n, h // (nh // nkv)]
                s = np.sort(k @ q[t, h]) * hd ** -0.5
                size = (np.abs(k) @ np.abs(q[t, h])).max() * hd ** -0.5
                gap = s[-1] - s[-2] if n > 1 else np.inf
                rows[t, h] = size == 0 or gap > max(100.0, 2.0 ** -22 * hd * size)
    assert rows[:b.N].mean() > 0.9
    _scaled_check(b, got, rows)


def test_equal_scores_of_any_size(rb):
    """Keys that are all the same have the same weight, however large their scores are."""
    spec = wl.batch_from_lists([40, 70, 1500, 0], [1, 2, 1, 200], num_q_heads=4, num_kv_heads=2,
                               head_dim=64, seed=5)
    for size, k_scale in ((1e6, 1.0), (3e8, 1.0), (1e30, 1.0), (1e30, 2.0 ** 100)):
        for sign in (1, -1):
            b = Batch(spec, 3, k_scale=k_scale)
            code, s = (x.copy() for x in ref.unpack(b.k, 64, False))
            code[:], s[:] = 5, 57
            b.k = ref.pack(code, s, False)
            for k in b.keys:
                k[:] = 3 * 1.125 * k_scale
            b.q = torch.full_like(b.q, sign * size)
            b.q[::5] = 0
            _scaled_check(b, b.run(rb))


def test_rising_scores_beyond_24_bits(rb):
    """Scores that climb from 1e2 past 1e9 and fall again: a row is the value of the largest one."""
    spec = wl.batch_from_lists([1500, 900], [1, 600], num_q_heads=4, num_kv_heads=2, head_dim=128,
                               seed=2)
    for top in (1e4, 1e6, 1e9):
        for sign in (1.0, -1.0):
            b = Batch(spec, 4, sb=(40, 48))
            code, s = (x.copy() for x in ref.unpack(b.k, 128, False))
            for i in range(2):
                p = np.arange(b.lens[i])
                page, off = spec.block_table[i, p // 16], p % 16
                code[page, off] = 2
                s[page, off] = (8 + 8 * (p // 16 * 7 % 12) + p % 8)[:, None, None]
                b.keys[i][:] = ref.decode(code[page, off], s[page, off])
            b.k = ref.pack(code, s, False)
            b.q = torch.full_like(b.q, sign * top / 128)
            _scaled_check(b, b.run(rb))


@pytest.mark.parametrize("c", [3000, 250000])
@pytest.mark.parametrize("v_scale", [2.0 ** 100, 2.0 ** -100])
def test_values_of_the_largest_size_in_many_pieces(rb, c, v_scale):
    """V's largest value everywhere and a layer scale at the end of its range: the sums of a piece do
    not fit fp32 with the scale in them, the result does and is exact."""
    spec = wl.batch_from_lists([c, 700], [1, 40], num_q_heads=2, num_kv_heads=1, head_dim=64, seed=1)
    b = Batch(spec, 9, sb=(40, 48), v_scale=v_scale)
    code, s = (x.copy() for x in ref.unpack(b.v, 64, True))
    code[:], s[:] = 7, 126
    b.v = ref.pack(code, s, True)
    b.q.zero_()
    got = b.run(rb).double().cpu().numpy()
    assert (got == 6 * 448 * v_scale).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("top", [3e4, 1e7, 1e12])
def test_references_that_move_in_every_part_of_a_tile(rb, hd, top):
    """Scores that rise every few keys by far more than a reference bears: O and P of a tile's earlier
    columns are moved several times a tile, and a row is the mean of its last keys."""
    spec = wl.batch_from_lists([1500, 900], [1, 600], num_q_heads=4, num_kv_heads=2, head_dim=hd,
                               seed=2)
    b = Batch(spec, 4, sb=(40, 48))
    code, s = (x.copy() for x in ref.unpack(b.k, hd, False))
    for i in range(2):
        p = np.arange(b.lens[i])
        page, off = spec.block_table[i, p // 16], p % 16
        code[page, off] = 2
        s[page, off] = (p * 80 // b.lens[i] + 8)[:, None, None]
        b.keys[i][:] = ref.decode(code[page, off], s[page, off])
    b.k = ref.pack(code, s, False)
    b.q = torch.full_like(b.q, top / hd)
    want = b.run(rb)
    _scaled_check(b, want)
    for _ in range(10):
        assert torch.equal(b.run(rb), want)


def test_more_requests_than_planner_threads(rb):
    """1300 requests, most of one token, some of many and some of none."""
    rng = np.random.default_rng(0)
    new = np.where(rng.random(1300) < 0.1, rng.integers(3, 40, 1300), 1)
    spec = wl.batch_from_lists(rng.integers(0, 60, 1300).tolist(), new.tolist(), num_q_heads=4,
                               num_kv_heads=1, head_dim=64, seed=3)
    b = Batch(spec)
    b.check(b.run(rb))


@pytest.mark.parametrize("ratio", [2, 4])
@pytest.mark.parametrize("seed", range(4))
def test_manager_blocks(rb, seed, ratio):
    spec = wl.random_batch(seed, num_q_heads=8, num_kv_heads=2, head_dim=64, max_reqs=6, max_q=100,
                           max_c=300, decode_frac=0.5, manager_ratio=ratio)
    b = Batch(spec, 1)
    b.check(b.run(rb))


def test_invalid_pages_are_reported(rb):
    spec = wl.batch_from_lists([100, 60], [1, 40], num_q_heads=4, num_kv_heads=2, head_dim=64,
                               seed=1)
    b = Batch(spec)
    for row, col, bad in ((0, 3, -1), (1, 0, spec.dims.num_blocks), (1, 2, spec.dims.null_block)):
        table = spec.block_table.copy()
        table[row, col] = bad
        b.err.zero_()
        rb.paged_attention_kv4(*b.args(table), error_word=b.err)
        torch.cuda.synchronize()
        assert int(b.err.item()) == rb.EBIT_BLOCK_ID
    for name, bad in (("qsl", np.array([0, 1, 40], np.int32)),
                      ("lens", np.array([101, 39], np.int32))):
        b = Batch(spec)
        setattr(b, name, bad)
        rb.paged_attention_kv4(*b.args(), error_word=b.err)
        torch.cuda.synchronize()
        assert int(b.err.item()) & rb.EBIT_ATTN_META


def test_rows_claimed_again_and_again_are_reported(rb):
    """Every second request claims all rows, more of them than the list of tiles is made for; and a
    length whose pages do not fit 32 bits."""
    d = rb.Dims(16, 16, 1, 64, max_num_reqs=64, max_model_len=256, max_blocks_per_req=16,
                num_blocks=20)
    k, v = rb.kv4_cache(d)
    q = torch.ones(256, 16, 64, dtype=BF, device="cuda")
    table = torch.ones(64, 16, dtype=torch.int32, device="cuda")
    loc = torch.tensor([0, 256] * 32 + [0], dtype=torch.int32, device="cuda")
    lens = torch.full((64,), 256, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rb.paged_attention_kv4(d, 64, 256, q, k, v, table, loc, lens, error_word=err)
    assert int(err.item()) == rb.EBIT_ATTN_META
    for new in (1, 40):
        err.zero_()
        loc = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        lens = torch.full((1,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        rb.paged_attention_kv4(d, 1, new, q[:new], k, v, table, loc, lens, error_word=err)
        assert int(err.item()) == rb.EBIT_ATTN_META


def test_no_list_of_rows_claimed_again_and_again(rb):
    """32 requests that claim all 256 rows are 512 pairs of tiles, the list holds 81: nothing is
    written behind it, and no row of the output."""
    d = rb.Dims(16, 16, 1, 64, max_num_reqs=64, max_model_len=256, max_blocks_per_req=16,
                num_blocks=20)
    k, v = rb.kv4_cache(d)
    q = torch.ones(256, 16, 64, dtype=BF, device="cuda")
    table = torch.ones(64, 16, dtype=torch.int32, device="cuda")
    loc = torch.tensor([0, 256] * 32 + [0], dtype=torch.int32, device="cuda")
    lens = torch.full((64,), 256, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = torch.full((rb.workspace_size(d, 64, 256),), 0x5a, dtype=torch.uint8, device="cuda")
    rb.paged_attention_kv4(d, 64, 256, q, k, v, table, loc, lens, out=out, workspace=ws,
                           error_word=err)
    assert int(err.item()) == rb.EBIT_ATTN_META
    # header, two lists of offsets (65 words each), 64 counters, the list itself, in 256-byte pieces
    start = 256 + 2 * 512 + 256 + 512
    assert bool((ws[start:] == 0x5a).all()) and bool((out == 7).all())


def test_empty_batches(rb):
    d = rb.Dims(16, 4, 2, 64, max_num_reqs=3, max_model_len=64, max_blocks_per_req=4, num_blocks=8)
    k, v = rb.kv4_cache(d)
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    q = torch.ones(5, 4, 64, dtype=BF, device="cuda")
    for reqs in (0, 3):
        err = z(1)
        out = rb.paged_attention_kv4(d, reqs, 0, q, k, v, z((3, 4)), z(4), z(3), error_word=err)
        assert int(err.item()) == 0 and bool((out == 0).all())
    # a request without new tokens among others
    lens = torch.tensor([7, 20, 9], dtype=torch.int32, device="cuda")
    loc = torch.tensor([0, 2, 2, 3], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1, 0, 0, 0], [2, 3, 0, 0], [4, 0, 0, 0]], dtype=torch.int32,
                         device="cuda")
    out = rb.paged_attention_kv4(d, 3, 3, q, k, v, table, loc, lens)
    assert bool((out == 0).all())  # all values are 0


@pytest.mark.parametrize("reqs", [0, 1, 3])
@pytest.mark.parametrize("pad", [1, 700])
def test_padding_rows_are_cleared(rb, reqs, pad):
    new = [1, 40, 3][:reqs]
    spec = wl.batch_from_lists([20, 5, 9][:reqs] or [0], new or [0], num_q_heads=6, num_kv_heads=2,
                               head_dim=64, seed=1, num_tokens_padded=sum(new) + pad)
    b = Batch(spec)
    b.R = b.R if reqs else 0
    out = torch.full_like(b.q, float("nan"))
    args = list(b.args())
    args[1] = b.R
    rb.paged_attention_kv4(*args, out=out, error_word=b.err)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    assert bool((out[sum(new):] == 0).all()) and bool(torch.isfinite(out).all())


def test_not_finite_queries_stay_in_their_rows(rb):
    spec = wl.batch_from_lists([100, 60], [2, 90], num_q_heads=4, num_kv_heads=1, head_dim=64,
                               seed=1)
    b = Batch(spec)
    b.q[1, 2, 5] = float("nan")
    b.q[50, 0, 63] = float("inf")
    got = b.run(rb)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1, 2] = bad[50, 0] = True
    assert bool(torch.isnan(got[bad]).all())
    clean = Batch(spec)
    want = clean.run(rb)
    assert torch.equal(got[~bad], want[~bad])


def test_a_row_of_nothing_but_minus_infinity_is_nan(rb):
    """As softmax of such a row is: its weights are 0 / 0.  The other rows are right."""
    spec = wl.batch_from_lists([100, 1500, 60], [2, 1, 90], num_q_heads=4, num_kv_heads=1,
                               head_dim=64, seed=1)
    b = Batch(spec)
    code, s = (x.copy() for x in ref.unpack(b.k, 64, False))
    for i in range(b.R):
        p = np.arange(b.lens[i])
        page, off = spec.block_table[i, p // 16], p % 16
        code[page, off, :, 5] = 3
        b.keys[i][:] = ref.decode(code[page, off], s[page, off])
    b.k = ref.pack(code, s, False)
    rows = np.ones(b.q.shape[:2], bool)
    for t, h in ((1, 2), (2, 0), (50, 0), (70, 3)):
        b.q[t, h, 5] = -float("inf")
        rows[t, h] = False
    got = b.run(rb)
    assert bool(torch.isnan(got[torch.from_numpy(~rows).cuda()]).all())
    with np.errstate(invalid="ignore"):
        _scaled_check(b, got, rows)


def test_captured_with_a_workspace_of_its_own_and_replayed(rb):
    spec = wl.batch_from_lists([300, 60, 9], [1, 90, 1], num_q_heads=8, num_kv_heads=2,
                               head_dim=128, seed=1)
    b = Batch(spec)
    a = list(b.args())
    s = torch.cuda.Stream()
    out = torch.empty_like(b.q)
    ws = torch.empty(rb.workspace_size(b.d, b.R, b.N), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rb.paged_attention_kv4(*a, out=out, workspace=ws)
    for seed in (1, 2):
        n = Batch(spec, seed)
        b.q.copy_(n.q)
        a[4].copy_(torch.from_numpy(n.k))
        a[5].copy_(torch.from_numpy(n.v))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n.check(out)
        assert torch.equal(out, n.run(rb, stream=s))  # the same bits


def test_pages_behind_32_bit_offsets_and_shared_ones(rb):
    """Requests that share pages at the end of a cache whose byte offsets pass 2^31."""
    spec = wl.batch_from_lists([300, 300, 40], [1, 90, 1], num_q_heads=16, num_kv_heads=8,
                               head_dim=128, seed=4)
    b = Batch(spec, 8)
    d, shift, shared = b.d, 262144 - b.d.num_blocks, 17
    b.keys[1][:shared * 16] = b.keys[0][:shared * 16]
    b.values[1][:shared * 16] = b.values[0][:shared * 16]
    table = np.where(spec.block_table >= 0, spec.block_table + shift, spec.block_table)
    table[1, :shared] = table[0, :shared]
    far = dataclasses.replace(d, num_blocks=262144)
    a = list(b.args(table.astype(np.int32)))
    caches = []
    for c in a[4:6]:
        big = torch.full((262144, *c.shape[1:]), 0x55, dtype=torch.uint8, device="cuda")
        big[shift:] = c
        caches.append(big)
    out = rb.paged_attention_kv4(far, *a[1:4], *caches, *a[6:], error_word=b.err)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    b.check(out)


@pytest.mark.parametrize("c,q", [(250000, 1), (120000, 70), (65537, 2)])
def test_long_sequences(rb, c, q):
    spec = wl.batch_from_lists([c], [q], num_q_heads=2, num_kv_heads=1, head_dim=64, seed=1)
    b = Batch(spec, 9, sb=(40, 48))
    b.check(b.run(rb))


def test_calls_on_two_streams_at_once(rb):
    specs = [wl.random_batch(s, num_q_heads=8, num_kv_heads=2, head_dim=128, max_reqs=8, max_q=300,
                             max_c=2000, decode_frac=0.5) for s in (1, 2)]
    batches = [Batch(spec, i) for i, spec in enumerate(specs)]
    want = [b.run(rb) for b in batches]
    args = [b.args() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, b in enumerate(batches):
            got[i].append(rb.paged_attention_kv4(*args[i], error_word=b.err, stream=streams[i]))
    torch.cuda.synchronize()
    for b, w, outs in zip(batches, want, got):
        assert int(b.err.item()) == 0
        b.check(w)
        assert all(torch.equal(o, w) for o in outs)


@pytest.mark.parametrize("hd", [64, 128])
def test_tiles_written_again_and_again(rb, hd):
    """Prompts of many key tiles, whose two stages of K and V and whose Q are rewritten hundreds of
    times a call: the right values, and the same bits every time."""
    spec = wl.batch_from_lists([2900, 1500, 0], [700, 260, 900], num_q_heads=8, num_kv_heads=4,
                               head_dim=hd, seed=6)
    b = Batch(spec, 5)
    args = b.args()
    want = rb.paged_attention_kv4(*args, error_word=b.err)
    b.check(want)
    for _ in range(50):
        assert torch.equal(rb.paged_attention_kv4(*args, error_word=b.err), want)
    assert int(b.err.item()) == 0


def test_it_is_the_attention_over_the_same_values(rb):
    """The 16-bit cache's attention over the rows that kv4_read gives."""
    spec = wl.random_batch(7, num_q_heads=8, num_kv_heads=2, head_dim=128, max_reqs=6, max_q=100,
                           max_c=600, decode_frac=0.5)
    b = Batch(spec, 7)
    a = b.args()
    slots = torch.arange(b.d.num_blocks * 16, dtype=torch.int32, device="cuda")
    k, v = rb.kv4_read(b.d, slots, a[4], a[5])
    want = rb.paged_attention(*a[:4], k, v, *a[6:])
    got = b.run(rb)
    w = oracle_attention(to64(b.q), b.keys, b.values, b.qsl, b.lens)[1]
    diff = (got.double() - want.double()).abs().cpu().numpy()
    size = np.abs(to64(want))
    assert (diff <= 2.0 ** -7 * size + (2.0 ** -8 + 2.0 ** -9) * w + 1e-6).all()


def test_a_wait_that_runs_out(rb):
    """The bounded waits give up when a unit is never handed over, and the next call is right."""
    # more units than all CTAs take ahead, so that CTA 0 has one to withhold
    b = Batch(wl.batch_from_lists([60], [6000], num_q_heads=32, num_kv_heads=8, head_dim=64,
                                  seed=1))
    lib = rb.lib
    assert lib.rb_debug_attention_wait_limit(2_000_000, 1) == 0
    try:
        rb.paged_attention_kv4(*b.args(), error_word=b.err)
        torch.cuda.synchronize()
        assert int(b.err.item()) == rb.EBIT_TIMEOUT
    finally:
        assert lib.rb_debug_attention_wait_limit(0, 0) == 0
    b = Batch(wl.batch_from_lists([60], [200], num_q_heads=8, num_kv_heads=2, head_dim=64, seed=1))
    b.check(b.run(rb))


def test_refusals(rb):
    spec = wl.batch_from_lists([60], [3], num_q_heads=4, num_kv_heads=2, head_dim=64, seed=1)
    b = Batch(spec)
    a = list(b.args())

    def call(i=None, x=None, **kw):
        args = list(a)
        if i is not None:
            args[i] = x
        return rb.paged_attention_kv4(*args, **kw)

    for i, x in ((3, a[3].float()), (3, a[3][:, :3]), (3, a[3].cpu()), (4, a[4][:-1]),
                 (5, a[5].to(torch.int32)), (6, a[6].flatten()[:1]), (7, a[7][:1]),
                 (8, a[8].long()), (7, a[7].cpu())):
        with pytest.raises(ValueError):
            call(i, x)
    for kw in (dict(out=a[3][:1].clone()), dict(workspace=torch.empty(9, device="cuda")),
               dict(error_word=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(softmax_scale=0.0), dict(softmax_scale=-1.0), dict(k_scale=0.0),
               dict(v_scale=float("nan")), dict(softmax_scale=float("inf")),
               dict(k_scale=1e30, softmax_scale=1e30),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(rb.RbError):
            call(**kw)
