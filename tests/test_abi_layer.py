"""Host checks of the append, 4-bit cache and norm entry points: bad arguments are refused before
anything is enqueued (no GPU is touched)."""
import ctypes

import pytest

from test_abi import FAKE, MISALIGNED, _dims, lib  # noqa: F401  (lib is the fixture)


def _rot(lib, **kw):
    r = lib.rb_rotation(128, 0, 4096, 0, FAKE)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _append(lib, four, d, rot, tokens=3, pos=FAKE, q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE,
            vs=1024, slots=FAKE, q_out=FAKE, qos=4096, kc=FAKE, vc=FAKE, scales=(1.0, 1.0)):
    D = None if d is None else ctypes.byref(d)
    R = None if rot is None else ctypes.byref(rot)
    head = (D, tokens, R, pos, q, qs, k, ks, v, vs, slots)
    tail = (q_out, qos, kc, vc, None, None)
    if four:
        return lib.lib.rb_kv4_append(*head, *scales, *tail)
    return lib.lib.rb_kv_append(*head, *tail)


@pytest.mark.parametrize("four", [False, True])
def test_append_host_checks(lib, four):  # noqa: F811
    d, r = _dims(lib), _rot(lib)
    call = lambda d=d, rot=r, **kw: _append(lib, four, d, rot, **kw)
    assert call(tokens=0, k=None, q=None, q_out=None, slots=None) == 0  # nothing to do
    assert call(d=None) == 1 and call(tokens=-1) == 1
    for name in ("block_size", "num_q_heads", "num_kv_heads", "head_dim", "num_blocks"):
        assert call(d=_dims(lib, **{name: 0})) == 1, name
    assert call(d=_dims(lib, head_dim=72)) == 5
    assert call(rot=_rot(lib, reserved=1)) == 1
    assert call(rot=_rot(lib, interleaved=2)) == 1
    assert call(rot=_rot(lib, max_position=0)) == 1
    assert call(rot=_rot(lib, rotary_dim=0)) == 1
    assert call(rot=_rot(lib, rotary_dim=144)) == 1
    assert call(rot=_rot(lib, rotary_dim=24)) == 5
    assert call(rot=_rot(lib, d_cos_sin=None)) == 1
    assert call(rot=_rot(lib, d_cos_sin=MISALIGNED)) == 1
    assert call(pos=None) == 1
    for name in ("k", "v", "slots", "kc", "vc", "q", "q_out"):
        assert call(**{name: None}) == 1, name
    for name in ("k", "v", "kc", "vc", "q", "q_out"):
        assert call(**{name: MISALIGNED}) == 1, name
    for name in ("qs", "qos"):
        assert call(**{name: 4088}) == 1 and call(**{name: 4100}) == 1
    for name in ("ks", "vs"):
        assert call(**{name: 1016}) == 1 and call(**{name: 1028}) == 1
    if four:
        assert call(d=_dims(lib, block_size=32)) == 5
        assert call(d=_dims(lib, head_dim=96), rot=None) == 5
        assert call(d=_dims(lib, num_kv_heads=256, num_q_heads=256), qs=32768, qos=32768,
                    ks=32768, vs=32768) == 5
        assert call(d=_dims(lib, num_blocks=1 << 28)) == 2
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert call(scales=(bad, 1.0)) == 1 and call(scales=(1.0, bad)) == 1


def test_read_host_checks(lib):  # noqa: F811
    def call(d=_dims(lib), rows=3, slots=FAKE, kc=FAKE, vc=FAKE, ks=1.0, vs=1.0, k=FAKE, v=FAKE):
        return lib.lib.rb_kv4_read(None if d is None else ctypes.byref(d), rows, slots, kc, vc,
                                   ks, vs, k, v, None, None)

    assert call(rows=0, slots=None) == 0
    assert call(d=None) == 1 and call(rows=-1) == 1
    assert call(d=_dims(lib, block_size=8)) == 5 and call(d=_dims(lib, head_dim=32)) == 5
    assert call(d=_dims(lib, num_blocks=0)) == 1
    assert call(ks=0.0) == 1 and call(vs=float("nan")) == 1
    for name in ("slots", "kc", "vc", "k", "v"):
        assert call(**{name: None}) == 1, name
    for name in ("kc", "vc", "k", "v"):
        assert call(**{name: MISALIGNED}) == 1, name


def test_attention_host_checks(lib):  # noqa: F811
    def call(d=_dims(lib), reqs=2, tokens=3, padded=4, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE,
             loc=FAKE, lens=FAKE, scale=1.0, ks=1.0, vs=1.0, out=FAKE, ws=FAKE, size=1 << 40):
        return lib.lib.rb_paged_attention_kv4(
            None if d is None else ctypes.byref(d), reqs, tokens, padded, q, kc, vc, table, loc,
            lens, scale, ks, vs, out, ws, size, None, None)

    assert call(d=None) == 1 and call(reqs=-1) == 1 and call(tokens=-1) == 1 and call(padded=2) == 1
    assert call(d=_dims(lib, block_size=32)) == 5 and call(d=_dims(lib, head_dim=96)) == 5
    for name in ("q", "kc", "vc", "table", "loc", "lens", "out", "ws"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert call(**{name: MISALIGNED}) == 1, name
    assert call(size=256) == 2
    for bad in (0.0, -1.0, float("inf"), float("nan"), 1e-31, 1e31):
        assert call(ks=bad) == 1 and call(vs=bad) == 1, bad
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=bad) == 1, bad
    assert call(scale=1e30, ks=1e7) == 1
    many = _dims(lib, max_num_reqs=40000, max_blocks_per_req=4)
    assert call(d=many, reqs=32769, tokens=32769, padded=32769) == 2
    long = _dims(lib, max_num_reqs=2, max_blocks_per_req=1 << 30)
    assert call(d=long) == 2
    # a tile pair holds 2 * 128 / 16 tokens of a group of 16
    wide = _dims(lib, num_q_heads=16, num_kv_heads=1)
    assert call(d=wide, reqs=1, tokens=1 << 20, padded=1 << 20) == 2


def test_attention_refuses_a_product_of_scales_that_loses_bits(lib):  # noqa: F811
    def call(scale, ks):
        return lib.lib.rb_paged_attention_kv4(
            ctypes.byref(_dims(lib)), 2, 3, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, scale, ks, 1.0,
            FAKE, FAKE, 1 << 40, None, None)

    assert call(1e-9, 1e-30) == 1 and call(1e-20, 1e-30) == 1  # subnormal, 0


def test_norm_host_checks(lib):  # noqa: F811
    ODD = ctypes.c_void_p(0x100001)

    def call(rows=3, n=256, dtype=0, x=FAKE, xs=256, res=FAKE, rs=256, ro=FAKE, ros=256, w=FAKE,
             eps=1e-6, out_dtype=0, group=0, out=FAKE, scales=None):
        return lib.lib.rb_add_rms_norm(rows, n, dtype, x, xs, res, rs, ro, ros, w, eps, out_dtype,
                                       group, out, scales, None)

    eight = dict(out_dtype=3, scales=FAKE)
    assert call(rows=0, x=None) == 0
    assert call(rows=-1) == 1 and call(n=0) == 1 and call(n=40000, xs=40000, rs=40000,
                                                          ros=40000) == 5
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == 1
    assert call(dtype=3) == 5 and call(dtype=-1) == 5 and call(out_dtype=1) == 5
    assert call(group=128) == 1                       # groups are the 8-bit output's
    assert call(group=24, **eight) == 5 and call(group=-16, **eight) == 1
    assert call(group=128, n=200, **eight) == 1
    assert call(out_dtype=3) == 1 and call(scales=FAKE) == 1
    assert call(res=None) == 1 and call(ro=None) == 1
    for name in ("xs", "rs", "ros"):
        assert call(**{name: 255}) == 1, name
    for name in ("x", "w", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "w", "out", "res", "ro"):
        assert call(**{name: ODD}) == 1, name
