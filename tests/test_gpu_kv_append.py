"""rb_kv_append, rb_kv4_append and rb_kv4_read against the oracle, bit for bit: the rotation's
products and sums and the 4-bit format's quotients are rounded one by one in fp32 on both sides.
Rotated rows are also within half a bf16 step of the float64 rotation (and 3 fp32 roundings of terms
no larger than |x| + |y|)."""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _dims(rb, nh=4, nkv=2, hd=64, pages=12, **kw):
    return rb.Dims(block_size=kw.pop("block_size", 16), num_q_heads=nh, num_kv_heads=nkv,
                   head_dim=hd, max_num_reqs=1, max_model_len=16, max_blocks_per_req=1,
                   num_blocks=pages, **kw)


class Case:
    def __init__(self, rb, d, tokens, seed=0, fused=False, positions=3000, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: (scale * torch.randn(*s, generator=g, device="cuda")).to(BF)
        nh, nkv, hd = d.num_q_heads, d.num_kv_heads, d.head_dim
        if fused:
            self.q, self.k, self.v = randn(tokens, nh + 2 * nkv, hd).split([nh, nkv, nkv], 1)
        else:
            self.q, self.k, self.v = randn(tokens, nh, hd), randn(tokens, nkv, hd), \
                randn(tokens, nkv, hd)
        rng = np.random.default_rng(seed)
        self.pos = rng.integers(0, positions, tokens).astype(np.int32)
        total = d.num_blocks * d.block_size
        self.slots = rng.permutation(np.arange(d.block_size, total))[:tokens].astype(np.int32)
        assert len(self.slots) == tokens
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_position = positions

    def args(self):
        i32 = lambda a: torch.from_numpy(a).cuda()
        return dict(slot_mapping=i32(self.slots), positions=i32(self.pos), error_word=self.err)


def _f(t):
    return t.float().cpu().numpy()


def _rotated(x, c, table, inter):
    """bf16 rows after the rotation, bit for bit; checked against float64 on the way."""
    if table is None:
        return x.clone()
    rows = table.cpu().numpy()[c.pos]
    y = torch.from_numpy(ref.rotate(_f(x), rows, inter)).to(BF)
    z = ref.rotate(_f(x), rows, inter, exact=True)
    size = np.abs(_f(x)).max()
    assert (np.abs(_f(y) - z) <= np.abs(z) * 2.0 ** -8 + 3 * 2.0 ** -24 * 2 * size).all()
    return y.cuda()


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


SHAPES = [  # nh, nkv, hd, rotary, interleaved
    (4, 2, 64, 64, False), (4, 2, 64, 64, True), (32, 8, 128, 128, False),
    (12, 3, 128, 64, True), (7, 1, 128, 32, False), (5, 5, 64, 16, False), (16, 1, 64, 48, False),
]


@pytest.mark.parametrize("tokens", [1, 3, 65])
@pytest.mark.parametrize("nh,nkv,hd,rot,inter", SHAPES + [(3, 3, 96, 96, False),
                                                          (2, 1, 256, 64, True),
                                                          (9, 1, 16, 16, False),
                                                          (1, 1, 2048, 2048, False)])
def test_append(rb, nh, nkv, hd, rot, inter, tokens):
    d = _dims(rb, nh, nkv, hd)
    c = Case(rb, d, tokens, seed=tokens, fused=tokens == 65)
    table = rb.rotary_table(3000, rot)
    assert np.abs(table.cpu().numpy() - ref.rotary_table(3000, rot)).max() <= 2.0 ** -24
    kc, vc = (torch.randn(d.num_blocks * 16, nkv, hd, device="cuda").to(BF) for _ in range(2))
    want_k, want_v = kc.clone(), vc.clone()
    if tokens > 2:
        c.slots[1] = -1
    at = torch.from_numpy(c.slots[c.slots >= 0].astype(np.int64)).cuda()
    here = torch.from_numpy(c.slots >= 0).cuda()
    want_k[at] = _rotated(c.k, c, table, inter)[here]
    want_v[at] = c.v[here]
    q = rb.kv_append(d, c.q, c.k, c.v, k_cache=kc, v_cache=vc,
                     rotation=rb.Rotation(table, inter), **c.args())
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert np.array_equal(_bits(q), _bits(_rotated(c.q, c, table, inter)))
    assert np.array_equal(_bits(kc), _bits(want_k))
    assert np.array_equal(_bits(vc), _bits(want_v))


@pytest.mark.parametrize("tokens", [1, 5, 130])
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.3, 7.0)])
@pytest.mark.parametrize("nh,nkv,hd,rot,inter", SHAPES)
def test_append_in_four_bits(rb, nh, nkv, hd, rot, inter, scales, tokens):
    d = _dims(rb, nh, nkv, hd)
    c = Case(rb, d, tokens, seed=tokens, fused=tokens == 5)
    table = rb.rotary_table(3000, rot)
    kc, vc = (torch.randint(0, 256, (d.num_blocks, nkv, 9 * hd), dtype=torch.uint8,
                            device="cuda") for _ in range(2))
    if tokens > 2:
        c.slots[1] = -7
    here = c.slots >= 0
    want = []
    for cache, x, s, values in ((kc, _rotated(c.k, c, table, inter), scales[0], False),
                                (vc, c.v, scales[1], True)):
        code, sb = ref.unpack(cache.cpu().numpy(), hd, values)
        code, sb = code.copy(), sb.copy()
        page, off = c.slots[here] // 16, c.slots[here] % 16
        code[page, off], sb[page, off] = ref.encode(_f(x)[here], s)
        want.append((ref.pack(code, sb, values), code, sb, s))
    q = rb.kv4_append(d, c.q, c.k, c.v, k_cache=kc, v_cache=vc, k_scale=scales[0],
                      v_scale=scales[1], rotation=rb.Rotation(table, inter), **c.args())
    rows = rb.kv4_read(d, torch.from_numpy(c.slots).cuda(), kc, vc, *scales, error_word=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert np.array_equal(_bits(q), _bits(_rotated(c.q, c, table, inter)))
    for got, row, (b, code, sb, s) in zip((kc, vc), rows, want):
        assert np.array_equal(got.cpu().numpy(), b)
        page, off = c.slots // 16, c.slots % 16
        value = ref.decode(code[page, off], sb[page, off]).astype(np.float32) * np.float32(s)
        value = torch.from_numpy(np.where(here[:, None, None], value, 0)).to(BF)
        assert np.array_equal(_f(row), _f(value))


def test_every_code_and_scale_reads_back(rb):
    d = _dims(rb, 1, 1, 64, pages=16)
    sb = np.arange(256, dtype=np.uint8)                       # every scale byte: one a token
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 4))
    grid = lambda a, w: a.reshape(16, 16, 1, w)
    one = np.repeat(sb[:, None], 4, 1)
    kc, vc = (torch.from_numpy(ref.pack(grid(code, 64), grid(one, 4), v)).cuda()
              for v in (False, True))
    slots = torch.arange(256, dtype=torch.int32, device="cuda")
    k, v = rb.kv4_read(d, slots, kc, vc)
    want = ref.decode(code, one)
    assert np.array_equal(_f(k)[:, 0], want) and np.array_equal(_f(v)[:, 0], want)


@pytest.mark.parametrize("four", [False, True])
def test_extreme_values(rb, four):
    """Blocks of zeros, subnormal and huge values, infinities and NaN."""
    d = _dims(rb, 1, 1, 64)
    c = Case(rb, d, 9, positions=1)
    k = torch.zeros(9, 1, 64)
    k[1] = 6 * 2.0 ** -11
    k[2] = 1e-40
    k[3], k[4] = 1e30, -3e38
    k[5, 0, 3], k[5, 0, 40] = float("inf"), -float("inf")
    k[6, 0, 17] = float("nan")
    k[7] = torch.linspace(-2688, 2688, 64)
    k[8] = torch.linspace(-7, 7, 64)
    c.k, c.v = k.to(BF).cuda(), (-k).to(BF).cuda()
    a = c.args()
    if not four:
        kc, vc = (torch.zeros(d.num_blocks * 16, 1, 64, dtype=BF, device="cuda") for _ in "kv")
        rb.kv_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **a)
        at = torch.from_numpy(c.slots.astype(np.int64)).cuda()
        assert np.array_equal(_bits(kc[at]), _bits(c.k)) and np.array_equal(_bits(vc[at]),
                                                                           _bits(c.v))
        assert int(c.err.item()) == 0
        return
    kc, vc = rb.kv4_cache(d)
    assert rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **a) is None
    assert int(c.err.item()) == rb.EBIT_NOT_FINITE
    for cache, x, values in ((kc, c.k, False), (vc, c.v, True)):
        code, sb = ref.unpack(cache.cpu().numpy(), 64, values)
        page, off = c.slots // 16, c.slots % 16
        want = ref.encode(_f(x))
        assert np.array_equal(code[page, off], want[0])
        assert np.array_equal(sb[page, off], want[1])


@pytest.mark.parametrize("k_scale,v_scale", [(0.25, 3.0), (2.0 ** -100, 2.0 ** 100), (1e-20, 7e19)])
def test_extreme_values_over_a_layer_scale(rb, k_scale, v_scale):
    """Infinities and quotients beyond fp32 keep their signs; NaN and 0 are 0."""
    d = _dims(rb, 1, 1, 64)
    c = Case(rb, d, 6, positions=1)
    k = torch.zeros(6, 1, 64)
    k[0, 0, 3], k[0, 0, 4], k[0, 0, 40] = float("inf"), -float("inf"), -float("inf")
    k[1, 0, 17], k[1, 0, 18] = float("nan"), -float("nan")
    k[2], k[3] = -3e38, 3e38
    v = -k
    k[4], v[4] = (torch.linspace(-7, 7, 64) * s for s in (k_scale, v_scale))
    c.k, c.v = k.to(BF).cuda(), v.to(BF).cuda()
    kc, vc = rb.kv4_cache(d)
    rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, k_scale=k_scale, v_scale=v_scale,
                  **c.args())
    assert int(c.err.item()) == rb.EBIT_NOT_FINITE
    for cache, x, scale, values in ((kc, c.k, k_scale, False), (vc, c.v, v_scale, True)):
        code, sb = ref.unpack(cache.cpu().numpy(), 64, values)
        page, off = c.slots // 16, c.slots % 16
        want = ref.encode(_f(x), scale)
        assert np.array_equal(sb[page, off], want[1])
        # (a NaN's code is 0 of either sign)
        nan = np.isnan(_f(x))
        assert np.array_equal(code[page, off][~nan], want[0][~nan])
        assert (code[page, off][nan] % 8 == 0).all()


@pytest.mark.parametrize("bad", [0.0, -1.0, float("inf"), float("nan"), 1e-31, 1e31, 1e-39])
def test_layer_scales_out_of_range(rb, bad):
    d = _dims(rb, 1, 1, 64)
    c = Case(rb, d, 4)
    kc, vc = rb.kv4_cache(d)
    a = c.args()
    for scales in ((bad, 1.0), (1.0, bad)):
        with pytest.raises(rb.RbError):
            rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, k_scale=scales[0],
                          v_scale=scales[1], **a)
        with pytest.raises(rb.RbError):
            rb.kv4_read(d, a["slot_mapping"], kc, vc, *scales)
    torch.cuda.synchronize()
    assert not kc.any() and not vc.any()


def test_padding_tokens_that_are_not_finite_are_not_reported(rb):
    """Tokens on the reserved page pad a batch: what they hold is no error.  Elsewhere it is."""
    for null in (0, 3):
        d = _dims(rb, 2, 1, 64, null_block=null)
        c = Case(rb, d, 6)
        c.slots = np.array([17, 40, 16 * null, 16 * null, 16 * null + 5, -1], np.int32)
        for t in (c.k, c.v):
            t[2], t[3, 0, 5], t[4], t[5] = float("nan"), float("inf"), float("nan"), float("nan")
        kc, vc = rb.kv4_cache(d)
        rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **c.args())
        assert int(c.err.item()) == 0
        c.v[1, 0, 63] = float("nan")
        rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **c.args())
        assert int(c.err.item()) == rb.EBIT_NOT_FINITE


@pytest.mark.parametrize("four", [False, True])
def test_tokens_left_out(rb, four):
    """A position outside the table leaves its token out, a slot outside the pool its K and V."""
    d = _dims(rb, 2, 1, 64, pages=4)
    c = Case(rb, d, 6, positions=40)
    table = rb.rotary_table(40, 64)
    c.pos[1], c.pos[2] = 40, -1
    c.slots[3], c.slots[4] = 64, 2 ** 31 - 1
    kc, vc = rb.kv4_cache(d) if four else [torch.zeros(64, 1, 64, dtype=BF, device="cuda")
                                           for _ in "kv"]
    q_out = torch.full((6, 2, 64), 5.0, dtype=BF, device="cuda")
    fn = rb.kv4_append if four else rb.kv_append
    fn(d, c.q, c.k, c.v, k_cache=kc, v_cache=vc, rotation=rb.Rotation(table), q_out=q_out,
       **c.args())
    assert int(c.err.item()) == rb.EBIT_POSITION | rb.EBIT_SLOT
    assert (_f(q_out)[1:3] == 5).all()
    keep = [0, 3, 4, 5]
    c.pos[1:3] = 0
    assert np.array_equal(_bits(q_out)[keep], _bits(_rotated(c.q, c, table, False))[keep])
    if four:
        code, _ = ref.unpack(vc.cpu().numpy(), 64, True)
        used = (code.reshape(64, 64) != 0).any(1)
    else:
        used = (_f(vc).reshape(64, 64) != 0).any(1)
    assert sorted(np.nonzero(used)[0]) == sorted(c.slots[[0, 5]])
    if four:
        c.err.zero_()
        slots = torch.tensor([-1, 64, 3], dtype=torch.int32, device="cuda")
        k, _ = rb.kv4_read(d, slots, kc, vc, error_word=c.err)
        assert int(c.err.item()) == rb.EBIT_SLOT and (_f(k)[:2] == 0).all()


def test_in_place_on_a_fused_projection(rb):
    d = _dims(rb, 8, 2, 64)
    c = Case(rb, d, 33, fused=True)
    table = rb.rotary_table(3000, 64)
    want = _rotated(c.q, c, table, False)
    v = c.v.clone()
    kc, vc = (torch.zeros(d.num_blocks * 16, 2, 64, dtype=BF, device="cuda") for _ in "kv")
    out = rb.kv_append(d, c.q, c.k, c.v, k_cache=kc, v_cache=vc, rotation=rb.Rotation(table),
                       q_out=c.q, **c.args())
    assert out is c.q
    assert np.array_equal(_bits(c.q), _bits(want)) and np.array_equal(_bits(c.v), _bits(v))


def test_without_rotation_it_is_the_write(rb):
    d = _dims(rb, 2, 2, 128)
    c = Case(rb, d, 40)
    caches = [torch.zeros(d.num_blocks * 16, 2, 128, dtype=BF, device="cuda") for _ in range(4)]
    q = rb.kv_append(d, c.q, c.k, c.v, k_cache=caches[0], v_cache=caches[1], **c.args())
    rb.kv_write(d, c.k, c.v, torch.from_numpy(c.slots).cuda(), caches[2], caches[3])
    assert torch.equal(q, c.q)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_long_caches_pass_32_bit_offsets(rb):
    """Slots whose byte offsets pass 2^31 (4-bit) and whose value offsets do (16-bit)."""
    d = _dims(rb, 8, 8, 128, pages=262144)
    c = Case(rb, _dims(rb, 8, 8, 128), 4)
    c.slots = np.array([16, 2097153, 3000000, 4194303], np.int32)
    at = torch.from_numpy(c.slots.astype(np.int64)).cuda()
    kc, vc = (torch.empty(d.num_blocks, 8, 1152, dtype=torch.uint8, device="cuda") for _ in "kv")
    rb.kv4_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **c.args())
    for cache, x, values in ((kc, c.k, False), (vc, c.v, True)):
        code, sb = ref.unpack(cache[at // 16].cpu().numpy(), 128, values)
        want = ref.encode(_f(x))
        for i, s in enumerate(c.slots):
            assert np.array_equal(code[i, s % 16], want[0][i])
            assert np.array_equal(sb[i, s % 16], want[1][i])
    del kc, vc
    kc, vc = (torch.empty(d.num_blocks * 16, 8, 128, dtype=BF, device="cuda") for _ in "kv")
    rb.kv_append(d, None, c.k, c.v, k_cache=kc, v_cache=vc, **c.args())
    assert torch.equal(kc[at], c.k) and torch.equal(vc[at], c.v)
    assert int(c.err.item()) == 0


def test_pages_of_a_four_bit_cache_move(rb):
    """PagePool copies and compacts a 4-bit cache's pages whole."""
    d = rb.Dims(16, 4, 2, 64, max_num_reqs=3, max_model_len=64, max_blocks_per_req=4,
                num_blocks=20)
    k, v = (torch.randint(0, 256, (20, 2, 576), dtype=torch.uint8, device="cuda") for _ in "kv")
    k0, v0 = k.clone(), v.clone()
    table = torch.tensor([[17, 3, -1, -1], [-1] * 4, [9, 19, 2, -1]], dtype=torch.int32,
                         device="cuda")
    count = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    pool = rb.PagePool(rb.kv4_page_dims(d), rb.kv4_pages(k).view(20, 2, 288),
                       rb.kv4_pages(v).view(20, 2, 288), table, count)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pool.copy(i32(17, 9), i32(5, 6))
    assert torch.equal(k[[5, 6]], k0[[17, 9]]) and torch.equal(v[[5, 6]], v0[[17, 9]])
    pool.compact()
    assert sorted(table[0, :2].tolist() + table[2, :3].tolist()) == [1, 2, 3, 4, 5]
    old = [17, 3, 9, 19, 2]
    new = table[0, :2].tolist() + table[2, :3].tolist()
    assert torch.equal(k[new], k0[old]) and torch.equal(v[new], v0[old])
    assert int(pool.error_word.item()) == 0


def test_captured_and_replayed_on_another_stream(rb):
    d = _dims(rb, 4, 2, 64)
    c = Case(rb, d, 20)
    rotation = rb.Rotation(rb.rotary_table(3000, 64))
    a = c.args()
    kc, vc = rb.kv4_cache(d)
    q_out = torch.empty_like(c.q)
    rows = tuple(torch.empty(20, 2, 64, dtype=BF, device="cuda") for _ in "kv")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rb.kv4_append(d, c.q, c.k, c.v, k_cache=kc, v_cache=vc, rotation=rotation, q_out=q_out,
                      **a)
        rb.kv4_read(d, a["slot_mapping"], kc, vc, out=rows)
    for seed in (1, 2):
        n = Case(rb, d, 20, seed=seed)
        for name in ("q", "k", "v"):
            getattr(c, name).copy_(getattr(n, name))
        a["positions"].copy_(torch.from_numpy(n.pos))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        k2, v2 = rb.kv4_cache(d)
        q2 = rb.kv4_append(d, n.q, n.k, n.v, torch.from_numpy(c.slots).cuda(), k2, v2,
                           torch.from_numpy(n.pos).cuda(), rotation, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(q2, q_out) and torch.equal(kc, k2) and torch.equal(vc, v2)
        want = rb.kv4_read(d, a["slot_mapping"], k2, v2)
        assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1])


def test_refusals(rb):
    d = _dims(rb, 4, 2, 64)
    c = Case(rb, d, 5)
    a = c.args()
    table = rb.rotary_table(3000, 64)
    rot = rb.Rotation(table)
    kc, vc = (torch.zeros(d.num_blocks * 16, 2, 64, dtype=BF, device="cuda") for _ in "kv")

    def call(q=c.q, k=c.k, v=c.v, kc=kc, vc=vc, rotation=rot, **kw):
        return rb.kv_append(d, q, k, v, k_cache=kc, v_cache=vc, rotation=rotation, **{**a, **kw})

    for bad in (dict(q=c.q[:, :3]), dict(q=c.q[:4]), dict(k=c.k.float()), dict(v=c.v[:4]),
                dict(k=c.k.transpose(1, 2)), dict(kc=kc[:-1]), dict(vc=vc.float()),
                dict(positions=None), dict(positions=a["positions"][:4]),
                dict(slot_mapping=a["slot_mapping"].long()), dict(q_out=c.q[:4]),
                dict(q=None, q_out=c.q), dict(k=c.k.cpu()), dict(kc=kc.cpu()),
                dict(slot_mapping=a["slot_mapping"].cpu()), dict(error_word=c.err.float())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        rb.Rotation(table.double())
    with pytest.raises(ValueError):
        rb.Rotation(table[:, ::2])
    with pytest.raises(rb.RbError):
        call(rotation=rb.Rotation(rb.rotary_table(10, 40)))
    k4, v4 = rb.kv4_cache(d)
    with pytest.raises(ValueError):
        rb.kv4_append(d, c.q, c.k, c.v, k_cache=k4[:-1], v_cache=v4, **a)
    with pytest.raises(rb.RbError):
        rb.kv4_append(d, c.q, c.k, c.v, k_cache=k4, v_cache=v4, k_scale=0.0, **a)
    with pytest.raises(ValueError):
        rb.kv4_read(d, a["slot_mapping"], k4, v4, out=(c.k[:4], c.v))
    call(k=c.k[:0], q=c.q[:0], v=c.v[:0])  # no tokens: nothing to do
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
