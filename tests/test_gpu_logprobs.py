"""rb_token_logprobs against the float64 oracle: types, vocabulary sizes, strides, ties, masks.

Tolerance of a log probability (fp32, natural units), with u = 2^-24: each term 2^t carries the
rounding of x - ref and of the product with log2(e) (3 u |t| ln 2; weighted by its share of the
sum |t| is at most log2 V + 16, the lag of the reference) and ex2's 2^-22; a thread adds at most
V / 512 / 4 vectors' sums and the tree 40 more (u each); then the logarithm and the two
differences round the result (4 u |log p|).  The entropy's sum carries the same relative error
on terms of size |t| <= ln V + 11.
"""
import numpy as np
import pytest
import torch

import oracle.logprobs as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _tol(vocab):
    lag = np.log2(max(vocab, 2)) + 16
    return 4 * U + 3 * U * lag * 0.7 + (vocab / 2048 + 50) * U


def _check(rb, logits, tokens, top, out=None, stream=None, bits=0):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok = torch.as_tensor(np.asarray(tokens, np.int32)).cuda()
    got = rb.token_logprobs(logits, tok, top, out=out, error_word=err, stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == bits
    vocab = logits.shape[1]
    x = logits.double().cpu().numpy()
    lp, rank, ent, ids, best = ref.token_logprobs(x, tokens, top)
    tol = _tol(vocab)
    close = lambda g, w, extra: np.testing.assert_array_less(
        np.abs(np.where(np.isfinite(w), g - w, 0.0)), tol * extra + 4 * U * np.abs(
            np.where(np.isfinite(w), w, 0.0)) + 1e-30)
    f = lambda t: t.double().cpu().numpy()
    for g, w, extra in ((f(got.logprobs), lp, 1.0), (f(got.top_logprobs), best, 1.0),
                        (f(got.entropy), ent, np.log(max(vocab, 2)) + 12)):
        assert np.array_equal(np.isnan(g), np.isnan(w))
        assert np.array_equal(np.isneginf(g), np.isneginf(w))
        assert np.array_equal(np.isfinite(g), np.isfinite(w))
        with np.errstate(invalid="ignore"):
            close(g, w, extra)
    assert np.array_equal(got.ranks.cpu().numpy(), rank)
    assert np.array_equal(got.top_ids.cpu().numpy(), ids)
    return got


def _rows(rows, vocab, dtype, seed, stride=None, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = stride or vocab
    flat = torch.randn(rows * stride + offset, generator=g, device="cuda") * 3
    x = flat.to(dtype)[offset:].view(rows, stride)[:, :vocab]
    tok = np.random.default_rng(seed).integers(0, vocab, rows)
    tok[::3] = x.float().argmax(1).cpu().numpy()[::3]
    return x, tok


DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 33, 127, 512, 1000, 4097, 32000])
def test_sizes(rb, dtype, vocab):
    for rows, top in ((1, 0), (3, 5), (5, 32)):
        x, tok = _rows(rows, vocab, dtype, vocab + rows)
        _check(rb, x, tok, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,top", [(1, 200001, 20), (40, 100003, 20), (200, 50021, 5),
                                            (700, 9001, 1)])
def test_row_counts_take_every_split(rb, dtype, rows, vocab, top):
    """One CTA or a cluster of 2 to 8 per row."""
    x, tok = _rows(rows, vocab, dtype, rows)
    _check(rb, x, tok, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (0, 64), (7, 1)])
def test_rows_off_any_alignment(rb, dtype, offset, pad):
    x, tok = _rows(9, 5001, dtype, offset, stride=5001 + pad, offset=offset)
    _check(rb, x, tok, 8)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lowest_id(rb, dtype):
    vocab = 20011
    g = torch.Generator(device="cuda").manual_seed(5)
    coarse = torch.randint(0, 4, (6, vocab), generator=g, device="cuda").to(dtype)
    _check(rb, coarse, [0, 5, vocab - 1, 7, 8, 9], 32)
    _check(rb, torch.full((3, vocab), 2.5, device="cuda").to(dtype), [0, 100, vocab - 1], 20)
    signed = torch.zeros(2, 300, device="cuda").to(dtype)
    signed[:, ::2] = -0.0                       # the two zeros are equal
    _check(rb, signed, [1, 2], 5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_logits(rb, dtype):
    """-inf and the type's lowest value in masked places: a few, most, all but three, all."""
    vocab = 30011
    for fill in (-np.inf, torch.finfo(dtype).min):
        x, tok = _rows(6, vocab, dtype, 3)
        x = x.clone()
        x[0, 5:20] = fill
        x[1, 3:] = fill
        x[2, :-2] = fill
        x[3, :] = fill
        x[4, 1::2] = fill
        tok = [7, 0, vocab - 1, 4, 2, 3]
        _check(rb, x, tok, 20)
        _check(rb, x[:, :11].contiguous(), [0, 3, 4, 10, 1, 2], 20)


def test_rows_without_a_distribution(rb):
    for dtype in DTYPES:
        x, _ = _rows(4, 3001, dtype, 11)
        x = x.clone()
        x[0, 17] = float("nan")
        x[2, 2999] = float("inf")
        _check(rb, x, [1, 2, 3, 4], 4, bits=rb.EBIT_LOGITS)


def test_no_token_and_bad_tokens(rb):
    x, _ = _rows(4, 301, torch.bfloat16, 1)
    got = _check(rb, x, [3, -1, -1, 300], 2)
    assert got.ranks[1].item() == 0 and got.logprobs[1].item() == 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok = torch.tensor([301, -2, 0, 1], dtype=torch.int32, device="cuda")
    got = rb.token_logprobs(x, tok, 1, error_word=err)
    assert int(err.item()) == rb.EBIT_TOKEN_ID
    assert got.logprobs[:2].tolist() == [0, 0] and got.ranks[:2].tolist() == [0, 0]


@pytest.mark.parametrize("scale", [1e-3, 1.0, 60.0, 1e4])
def test_wide_and_narrow_rows(rb, scale):
    """Flat rows (entropy ln V) to one-hot ones, and logits far from zero."""
    for shift in (0.0, 500.0, -2e4):
        g = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn(5, 12345, generator=g, device="cuda") * scale + shift
        _check(rb, x, [0, 1, 2, 3, 4], 6)


def test_rising_and_falling_rows(rb):
    """A reference that has to move all the way up, or never."""
    up = torch.linspace(-80, 80, 40000, device="cuda")
    x = torch.stack([up, up.flip(0), up.view(200, 200).t().flatten()])
    for dtype in DTYPES:
        _check(rb, x.to(dtype), [0, 39999, 20000], 32)


def test_more_candidates_than_the_buffer(rb):
    """31 lane groups hold thousands of logits above every other group's: the bound on the
    32nd logit is low and the selection takes its slow way."""
    vocab = 100003
    v = torch.arange(vocab, device="cuda") // 4
    high = ((v % 512) // 4) < 31
    g = torch.Generator(device="cuda").manual_seed(9)
    noise = torch.rand(vocab, generator=g, device="cuda")
    x = torch.where(high, 5 + noise, noise).expand(320, -1).contiguous()
    _check(rb, x, np.arange(320), 32)


def test_captured_and_replayed_with_new_logits_on_another_stream(rb):
    x, tok = _rows(50, 40001, torch.bfloat16, 21)
    x = x.clone()
    t = torch.as_tensor(tok.astype(np.int32)).cuda()
    out = rb.TokenLogprobs.allocate(50, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rb.token_logprobs(x, t, 5, out=out)
    for seed in (1, 2):
        y, _ = _rows(50, 40001, torch.bfloat16, seed)
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = _check(rb, y, tok, 5)
        for name in ("logprobs", "ranks", "entropy", "top_ids", "top_logprobs"):
            assert torch.equal(getattr(out, name), getattr(want, name)), name


def test_no_rows(rb):
    x = torch.empty(0, 100, device="cuda", dtype=torch.bfloat16)
    got = rb.token_logprobs(x, torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert got.top_ids.shape == (0, 3)


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 1000), (torch.bfloat16, 65536),
                                         (torch.bfloat16, 65537), (torch.float16, 5003),
                                         (torch.float32, 32768), (torch.float32, 32769),
                                         (torch.bfloat16, 131072), (torch.bfloat16, 131073),
                                         (torch.float32, 65537)])
@pytest.mark.parametrize("top", [1, 8, 9, 32])
def test_rows_enough_for_every_sm(rb, dtype, vocab, top):
    """One CTA per row, of 128 or 256 threads; logits of few values, so that the bound on the
    top entries is met many times."""
    rows = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    g = torch.Generator(device="cuda").manual_seed(vocab + top)
    x = (torch.randn(rows, vocab, device="cuda", generator=g) * 40).round() / 8
    tok = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    _check(rb, x.to(dtype), tok.tolist(), top)


@pytest.mark.parametrize("rows", [2, 400])
def test_zeros_of_either_sign_are_equal(rb, rows):
    """In one CTA's list and where the lists of a row's CTAs are merged."""
    x = torch.full((rows, 40000), -1.0)
    x[:, 7::97] = 0.0
    x[:, 104::194] = -0.0
    x[::2, 39990] = -0.0
    for top in (3, 20):
        _check(rb, x.to(torch.bfloat16).cuda(), [104] * rows, top)


def test_two_logits_far_above_a_large_sum(rb):
    """A thread's sum of many terms near its reference, then two logits of 1e31: the sum
    vanishes against them, and its weighted part with it."""
    vocab = 24 << 20
    logits = torch.full((1, vocab), 10.9, device="cuda")
    for c in range(8):             # every thread's first batch, where its reference comes from
        logits[0, c * (vocab // 8):c * (vocab // 8) + 4 * 4 * 256] = 0.0
    at = [vocab // 2 - 5, vocab - 9]
    logits[0, at] = 1e31
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = torch.tensor(at[1:], dtype=torch.int32, device="cuda")
    got = rb.token_logprobs(logits, tokens, 2, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert abs(float(got.logprobs) + np.log(2.0)) <= 4 * U
    assert abs(float(got.entropy) - np.log(2.0)) <= 4 * U
    assert int(got.ranks) == 1 and got.top_ids.tolist() == [at]
