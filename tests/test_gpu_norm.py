"""rb_add_rms_norm against float64: types, widths, strides, groups, rows without a value.

With u = 2^-24: a thread adds up to 32 squares in turn, a row's threads meet in at most 10 sums, the
division, the sum with eps, rsqrt (2 ulp) and two products follow: a value is within
(42 / 2 + 2 + 2 * 2 + 2) u < 32 u of the exact one, a scale (one more quotient) within 33 u."""
import numpy as np
import pytest
import torch

from oracle import norm as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(rows, n, dtype, gap=0, offset=0, seed=0, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(scale):
        flat = torch.randn(rows * (n + gap) + offset, generator=g, device="cuda") * scale
        return flat.to(TYPES[dtype])[offset:].view(rows, n + gap)[:, :n]

    w = (1 + 0.3 * torch.randn(n + offset, generator=g, device="cuda")).to(TYPES[dtype])[offset:]
    return make(2.0), make(5.0) if residual else None, w


def _check16(y, got, dtype, weight_size):
    info = torch.finfo(TYPES[dtype])
    half = info.eps / 2 + 32 * U
    tiny = info.smallest_normal * info.eps  # half a step below the normal range, and the ends
    assert (np.abs(got.double().cpu().numpy() - y) <= np.abs(y) * half + tiny).all()


def _check8(y, codes, scales, group):
    s = ref.scales_of(y, group)
    got = scales.double().cpu().numpy()
    assert (np.abs(got - s) <= 33 * U * s).all()
    n = y.shape[1]
    each = np.repeat(got, group or n, 1)
    c = codes.float().cpu().numpy().astype(np.float64)
    t = np.divide(y, each, out=np.zeros_like(y), where=each > 0)
    # half a step: 2^-4 of the value, 2^-10 below 2^-6
    assert (np.abs(c - t) <= np.maximum(np.abs(t) * (2.0 ** -4 + 70 * U), 2.0 ** -10 + 1e-7)).all()
    assert (np.abs(c) <= 448).all()


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 100), (64, 128), (9, 1000), (2, 1024), (7, 1025), (4, 2889),
          (130, 4096), (3, 5120), (2, 8200), (2, 16384), (1, 20001), (2, 32768)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("gap,offset", [(0, 0), (8, 0), (3, 1)])
def test_sixteen_bits(rb, rows, n, dtype, gap, offset):
    x, res, w = _inputs(rows, n, dtype, gap, offset)
    r = (x.float() + res.float()).to(x.dtype)
    after = torch.zeros_like(r)
    out = rb.add_rms_norm(x, w, 1e-5, residual=res, residual_out=after)
    torch.cuda.synchronize()
    assert torch.equal(after, r)
    _check16(ref.rms_norm(r.double().cpu().numpy(), w.double().cpu().numpy(), 1e-5), out, dtype, 1)
    plain = rb.add_rms_norm(r, w, 1e-5)      # the sum's norm is the same, bit for bit
    assert torch.equal(plain, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,n,group", [(1, 16, 16), (3, 100, 0), (5, 2889, 0), (64, 128, 128),
                                          (7, 4096, 0), (7, 4096, 128), (33, 5120, 64),
                                          (4, 1024, 256), (4, 1280, 256), (2, 96, 32),
                                          (2, 32768, 128), (130, 256, 16)])
@pytest.mark.parametrize("gap,offset", [(0, 0), (5, 1)])
def test_eight_bits(rb, rows, n, group, dtype, gap, offset):
    x, res, w = _inputs(rows, n, dtype, gap, offset, seed=1)
    r = (x.float() + res.float()).to(x.dtype)
    codes, scales = rb.add_rms_norm_fp8(x, w, 1e-6, residual=res, group=group)
    torch.cuda.synchronize()
    assert torch.equal(res, r)               # the sum went back into the residual
    _check8(ref.rms_norm(r.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6), codes, scales,
            group)


def test_in_place(rb):
    x, res, w = _inputs(6, 512, "bf16")
    r = (x.float() + res.float()).to(x.dtype)
    want = rb.add_rms_norm(r, w)
    y = x.clone()
    rb.add_rms_norm(y, w, residual=res, residual_out=res, out=y)
    assert torch.equal(y, want) and torch.equal(res, r)
    y, z = x.clone(), torch.empty_like(x)
    res = (r.float() - 0).to(x.dtype)
    rb.add_rms_norm(y, w, residual=torch.zeros_like(x), residual_out=y, out=z)
    assert torch.equal(y, x)


@pytest.mark.parametrize("group", [0, 128])
def test_rows_of_zeros_and_extremes(rb, group):
    x = torch.zeros(5, 512, device="cuda", dtype=torch.bfloat16)
    x[1] = 1e-30
    x[2] = 1e15
    x[3, 5] = float("inf")
    x[4, 500] = float("nan")
    w = torch.ones(512, device="cuda", dtype=torch.bfloat16)
    out = rb.add_rms_norm(x, w, 1e-6).float().cpu().numpy()
    assert (out[0] == 0).all() and np.isfinite(out[:3]).all() and np.allclose(out[2], 1, 0.01)
    assert np.isnan(out[3, 5]) and np.isnan(out[4]).all()
    codes, scales = rb.add_rms_norm_fp8(x, w, 1e-6, group=group)
    c, s = codes.float().cpu().numpy(), scales.cpu().numpy()
    assert (c[0] == 0).all() and (s[0] == 0).all() and (c[2] == 448).all()
    assert np.isnan((c[4] * np.repeat(s[4], (group or 512)))).all()
    # eps 0 and zeros: 0 / 0
    assert np.isnan(rb.add_rms_norm(x[:1], w, 0.0).float().cpu().numpy()).all()


def test_streams_and_graphs(rb):
    x, res, w = _inputs(40, 4096, "bf16")
    out, after = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rb.add_rms_norm(x, w, residual=res, residual_out=after, out=out)
    x2, res2, _ = _inputs(40, 4096, "bf16", seed=7)
    x.copy_(x2)
    res.copy_(res2)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    r = res2.clone()
    want = rb.add_rms_norm(x2, w, residual=r, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(after, r)


def test_refusals(rb):
    x, res, w = _inputs(4, 256, "bf16")
    for bad in (dict(weight=w[:255]), dict(weight=w.float()), dict(residual=res[:3]),
                dict(residual=res.float()), dict(residual_out=res), dict(out=x[:, :255]),
                dict(out=torch.empty(4, 512, device="cuda", dtype=x.dtype)[:, ::2]),
                dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            rb.add_rms_norm(x, **{"weight": w, **bad})
    for y in (x[0], x.double(), x.cpu(), x.t()):
        with pytest.raises(ValueError):
            rb.add_rms_norm(y, w)
    with pytest.raises(rb.RbError):
        rb.add_rms_norm_fp8(x, w, group=24)
    with pytest.raises(rb.RbError):
        rb.add_rms_norm_fp8(x, w, eps=-1.0)
    with pytest.raises(ValueError):
        rb.add_rms_norm_fp8(x, w, group=128, scales=torch.empty(4, 1, device="cuda"))
    assert rb.add_rms_norm(x[:0], w).shape == (0, 256)


@pytest.mark.parametrize("group", [0, 64])
def test_a_weight_that_is_nan_stays_in_its_column(rb, group):
    x, _, w = _inputs(5, 256, "bf16", residual=False)
    w[70] = float("nan")
    rest = torch.arange(256, device="cuda") != 70
    out = rb.add_rms_norm(x, w)
    codes, scales = rb.add_rms_norm_fp8(x, w, group=group)
    assert bool(torch.isnan(out[:, 70]).all()) and bool(torch.isnan(codes.float()[:, 70]).all())
    assert not bool(torch.isnan(out[:, rest]).any()) and bool(torch.isfinite(scales).all())
    w[70] = 0
    want, want_scales = rb.add_rms_norm_fp8(x, w, group=group)
    assert torch.equal(codes.float()[:, rest], want.float()[:, rest])
    assert torch.equal(scales, want_scales)


def test_squares_beyond_fp32(rb):
    """Rows whose squares overflow are 0, the others are as ever."""
    x = torch.full((3, 256), 1e25, device="cuda")
    x[1] = 2.0
    w = torch.ones(256, device="cuda")
    out = rb.add_rms_norm(x, w)
    codes, scales = rb.add_rms_norm_fp8(x, w, group=64)
    assert bool((out[[0, 2]] == 0).all()) and bool((codes.float()[[0, 2]] == 0).all())
    assert bool((scales[[0, 2]] == 0).all()) and bool((codes[1].float() == 448).all())
    # 4 + 1e-6 and its root within a few roundings of fp32
    assert (out[1].double() - 2 / (4 + 1e-6) ** 0.5).abs().max().item() <= 8 * U


@pytest.mark.parametrize("dtype,group", [("fp32", 0), ("fp32", 64), ("bf16", 0), ("bf16", 128)])
@pytest.mark.parametrize("gap,offset", [(0, 0), (3, 1)])
def test_vanishing_rows_in_eight_bits(rb, dtype, group, gap, offset):
    """Rows and groups of 1e-37 to 1e-33 among ordinary ones: the scale is theirs (an ordinary number of
    fp32), and the codes fill their range.  Weighted values below 2^-126 are off by 2^-150, which
    is less than 2^-24 of rows of 1e-37."""
    x, _, w = _inputs(12, 512, dtype, gap, offset, residual=False)
    x[:6] *= torch.logspace(-37, -33, 6, device="cuda")[:, None].to(x.dtype)
    x[7, 128:256] = 0
    codes, scales = rb.add_rms_norm_fp8(x, w, 1e-6, group=group)
    assert bool((scales[:6] > 2.0 ** -126).all())
    _check8(ref.rms_norm(x.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6), codes, scales,
            group)
    assert bool((codes[:6].float().abs().amax(1) == 448).all())
