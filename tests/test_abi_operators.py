"""Host checks of the scored-attention, page and log-probability entry points: bad arguments are refused before
anything is enqueued (no GPU is touched)."""
import ctypes

import pytest

from test_abi import FAKE, MISALIGNED, _dims, lib  # noqa: F401  (lib is the fixture)


def _tables(lib, rows=8, **kw):
    t = lib.rb_page_tables(rows, 0, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _page_calls(lib, d, t, ws=FAKE, ws_bytes=1 << 30, k=FAKE, v=FAKE, n=2, lists=FAKE):
    """The status of each rb_pages_* call for these arguments."""
    L, D, T = lib.lib, None if d is None else ctypes.byref(d), None if t is None else ctypes.byref(t)
    return dict(
        count=lambda: L.rb_pages_count(D, T, None, None),
        copy=lambda: L.rb_pages_copy(D, n, lists, lists, k, v, ws, ws_bytes, None, None),
        fork=lambda: L.rb_pages_fork(D, T, n, lists, lists, lists, k, v, ws, ws_bytes, None, None),
        free=lambda: L.rb_pages_free(D, T, n, lists, None, None, None),
        compact=lambda: L.rb_pages_compact(D, T, None, None, k, v, ws, ws_bytes, None, None))


def test_pages_host_checks(lib):  # noqa: F811
    d = _dims(lib)
    need = lib.lib.rb_pages_workspace_size(ctypes.byref(d))
    assert need > 4 * 1000
    assert lib.lib.rb_pages_workspace_size(None) == 0
    bad = _dims(lib, null_block=1000)
    assert lib.lib.rb_pages_workspace_size(ctypes.byref(bad)) == 0

    def refused(status, only=None, **kw):
        args = dict(d=d, t=_tables(lib))
        args.update(kw)
        for name, call in _page_calls(lib, **args).items():
            if only is None or name in only:
                assert call() == status, (name, kw)

    refused(1, d=None)
    refused(1, d=bad)
    refused(1, d=_dims(lib, block_size=0))
    refused(5, d=_dims(lib, num_kv_heads=1, num_q_heads=1, head_dim=3))  # 6-byte token rows
    tables = ("count", "fork", "free", "compact")
    refused(1, only=tables, t=None)
    refused(1, only=tables, t=_tables(lib, reserved=1))
    refused(1, only=tables, t=_tables(lib, num_rows=-1))
    refused(2, only=tables, t=_tables(lib, num_rows=9))
    refused(1, only=tables, t=_tables(lib, d_ref_count=None))
    refused(1, only=tables, t=_tables(lib, d_num_blocks=None))
    caches = ("copy", "fork", "compact")
    refused(1, only=caches, k=None)
    refused(1, only=caches, v=MISALIGNED)
    refused(1, only=caches, ws=None)
    refused(1, only=caches, ws=ctypes.c_void_p(0x100010))
    refused(2, only=caches, ws_bytes=need - 1)
    refused(1, only=("copy", "fork", "free"), n=-1)
    refused(1, only=("copy", "fork", "free"), lists=None)
    refused(2, only=("copy",), n=1001)                       # more pairs than pages
    refused(2, only=("fork",), n=9)                          # more forks than rows
    calls = _page_calls(lib, d, _tables(lib), n=0, lists=None)
    assert calls["copy"]() == calls["fork"]() == calls["free"]() == 0


def test_token_logprobs_host_checks(lib):  # noqa: F811
    def call(rows=2, vocab=100, stride=100, dtype=0, logits=FAKE, tokens=FAKE, top=3, lp=FAKE,
             ids=FAKE, best=FAKE):
        return lib.lib.rb_token_logprobs(rows, vocab, stride, dtype, logits, tokens, top, lp,
                                         FAKE, FAKE, ids, best, None, None)

    assert call(rows=-1) == 1
    assert call(vocab=0) == 1
    assert call(stride=99) == 1
    assert call(top=-1) == 1
    assert call(top=33) == 5
    assert call(dtype=3) == 5
    assert call(vocab=(1 << 30) + 1, stride=1 << 31) == 5
    assert call(rows=1 << 28) == 2
    assert call(logits=None) == 1
    assert call(tokens=None) == 1                            # log probabilities of no token
    assert call(ids=None) == 1
    assert call(best=None) == 1
    assert call(logits=ctypes.c_void_p(0x100001)) == 1
    assert call(dtype=2, logits=ctypes.c_void_p(0x100002)) == 1
    assert call(rows=0, logits=None) == 0


def test_scored_attention_host_checks(lib):  # noqa: F811
    def call(d=None, rules="none", R=2, N=4, Np=4, ws=FAKE, ws_bytes=1 << 30, scale=0.1, **kw):
        d = _dims(lib) if d is None else d
        c = lib.rb_score_rules(0.0, 0, None, None, None)
        for k, v in kw.items():
            setattr(c, k, v)
        return lib.lib.rb_paged_attention_scored(
            ctypes.byref(d), R, N, Np, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.c_float(scale),
            ctypes.byref(c) if rules == "none" else None, FAKE, ws, ws_bytes, None, None)

    d = _dims(lib)
    need = lib.lib.rb_paged_attention_workspace_size(ctypes.byref(d), 2, 4)
    assert call(rules=None) == 1
    assert call(reserved=1) == 1
    for cap in (-1.0, float("nan"), float("inf"), 1e-40):
        assert call(softcap=cap) == 1, cap
    assert call(softcap=30.0, scale=float("inf")) == 1
    assert call(scale=0.0) == 1 and call(scale=-0.1) == 1
    assert call(d_key_start=0x100001) == 1
    assert call(d=_dims(lib, head_dim=96)) == 5
    assert call(d=_dims(lib, num_q_heads=64, num_kv_heads=2)) == 5
    assert call(R=9) == 2
    assert call(N=5, Np=4) == 1
    assert call(ws_bytes=need - 1) == 2
    assert call(ws=ctypes.c_void_p(0x100010)) == 1


def test_python_checks_come_first(lib):  # noqa: F811
    """The Python face names the tensor that does not fit before the library is called."""
    import torch

    import ragged_mixed_paged_gb300 as rb

    cpu = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="CUDA"):
        rb.token_logprobs(cpu, torch.zeros(4, dtype=torch.int32))
    dims = rb.Dims(16, 2, 2, 64, 4, 64, 4, 10)
    kv = torch.zeros(160, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache must be"):
        rb.PagePool(dims, kv[:150], kv)
    with pytest.raises(ValueError, match="belong together"):
        rb.PagePool(dims, kv, kv, block_table=torch.zeros(4, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        rb.PagePool(dims, kv, kv)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="key_start must have 4 entries"):
        rb.paged_attention_scored(dims, 1, 4, q, kv, kv, kv, kv, kv,
                                  rb.ScoreRules(key_start=torch.zeros(3, dtype=torch.int32)))
    with pytest.raises(ValueError, match="prefix_lens must have 2 entries"):
        rb.paged_attention_scored(dims, 2, 4, q, kv, kv, kv, kv, kv,
                                  rb.ScoreRules(prefix_lens=torch.zeros(1, dtype=torch.int32)))


@pytest.mark.parametrize("name,short", [
    ("q", (4, 2, 32)), ("q", (4, 3, 64)), ("q", (4 * 2 * 64 + 1,)), ("k_cache", (159, 2, 64)),
    ("v_cache", (160, 1, 64)), ("block_table", (2, 3)), ("query_start_loc", (2,)),
    ("seq_lens", (1,)), ("out", (3, 2, 64))])
def test_scored_attention_refuses_short_tensors(lib, name, short):  # noqa: F811
    """A tensor that the kernel would read or write past its end is named and refused."""
    import torch

    import ragged_mixed_paged_gb300 as rb

    dims = rb.Dims(16, 2, 2, 64, 4, 64, 4, 10)
    bf, i32 = torch.bfloat16, torch.int32
    args = dict(q=torch.zeros(4, 2, 64, dtype=bf), k_cache=torch.zeros(160, 2, 64, dtype=bf),
                v_cache=torch.zeros(160, 2, 64, dtype=bf), block_table=torch.zeros(2, 4, dtype=i32),
                query_start_loc=torch.zeros(3, dtype=i32), seq_lens=torch.zeros(2, dtype=i32),
                out=torch.zeros(4, 2, 64, dtype=bf))
    args[name] = torch.zeros(short, dtype=args[name].dtype)
    with pytest.raises(ValueError, match="^%s " % name):
        rb.paged_attention_scored(dims, 2, 4, rules=rb.ScoreRules(), **args)
