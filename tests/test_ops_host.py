"""Refusals and sizes of the windowed, weight-collecting, chunk and eviction calls, on a host without a
GPU: every bad argument is refused before anything is launched."""
import ctypes

import pytest

import bit_asymmetric_kv_kivi_gb300 as kivi
from bit_asymmetric_kv_kivi_gb300 import _build

P = ctypes.c_void_p
ONE = P(16)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kivi.lib()


def window(lib, cfg, nseq=2, seqs=ONE, kv=ONE, q=ONE, out=ONE, scale=0.1, win=100, sinks=4, mkl=5000, ws=ONE, n=BIG):
    return lib.kivi_decode_window_attn(cfg, nseq, seqs, kv, q, out, scale, win, sinks, mkl, ws, n, ONE, None)


def weights(lib, cfg, nseq=2, seqs=ONE, kv=ONE, q=ONE, out=ONE, w_in=ONE, w_out=ONE, stride=200, decay=1.0, scale=0.1,
            mkl=5000, ws=ONE, n=BIG, sc=ONE, m=BIG):
    return lib.kivi_decode_attn_weights(cfg, nseq, seqs, kv, q, out, w_in, w_out, stride, decay, scale, mkl, ws, n, sc, m,
                                        ONE, None)


def chunk(lib, cfg, nseq=2, seqs=ONE, kv=ONE, k=ONE, v=ONE, n_new=ONE, max_new=7, q=ONE, start=ONE, out=ONE, scale=0.1,
          win=0, sinks=0, mkl=5000, sc=ONE, m=BIG):
    return lib.kivi_chunk_attn(cfg, nseq, seqs, kv, k, v, n_new, max_new, q, start, out, scale, win, sinks, mkl, sc, m, ONE,
                               None)


def evict(lib, cfg, nseq=2, seqs=ONE, kv=ONE, w=ONE, stride=50, keep=8, sink=1, recent=2, sc=ONE, m=BIG, status=ONE):
    return lib.kivi_evict_groups(cfg, nseq, seqs, kv, w, stride, keep, sink, recent, sc, m, status, None)


CALLS = (window, weights, chunk, evict)


@pytest.mark.parametrize("bad", [dict(bits=3), dict(v_bits=1), dict(group=48), dict(residual=100), dict(head_dim=512),
                                 dict(num_q_heads=6, num_kv_heads=4), dict(dtype=7), dict(num_kv_heads=0)])
def test_bad_configs(lib, bad):
    cfg = kivi.Config(**bad)
    for call in CALLS:
        assert call(lib, cfg.c()) == kivi.ERR_ARG
    assert cfg.decode_ext_workspace_bytes(2, 100) == 0
    assert cfg.decode_weights_scratch_bytes(2, 100) == 0
    assert cfg.chunk_scratch_bytes(2, 100) == 0


def test_null_pointers_and_negative_sizes(lib):
    cfg = kivi.Config(num_q_heads=8, num_kv_heads=2).c()
    for call, names in ((window, ("seqs", "kv", "q", "out")), (weights, ("seqs", "kv", "q", "out", "w_out")),
                        (chunk, ("seqs", "kv", "k", "v", "n_new", "q", "start", "out")), (evict, ("seqs", "kv", "w", "status"))):
        for name in names:
            assert call(lib, cfg, **{name: None}) == kivi.ERR_ARG, (call.__name__, name)
        assert call(lib, cfg, nseq=-1) == kivi.ERR_ARG
        assert call(lib, cfg, nseq=65536) == kivi.ERR_ARG
    for call in (window, weights, chunk):
        assert call(lib, cfg, mkl=-1) == kivi.ERR_ARG
        for x in (float("nan"), float("inf")):
            assert call(lib, cfg, scale=x) == kivi.ERR_ARG
    for call in (window, chunk):
        assert call(lib, cfg, win=-1) == kivi.ERR_ARG
        assert call(lib, cfg, sinks=-1) == kivi.ERR_ARG
    assert weights(lib, cfg, stride=-1) == kivi.ERR_ARG
    assert weights(lib, cfg, stride=156) == kivi.ERR_ARG          # 156 groups of 32 are fewer than 5000 tokens
    assert weights(lib, cfg, decay=float("nan")) == kivi.ERR_ARG
    assert chunk(lib, cfg, max_new=-1) == kivi.ERR_ARG
    for kw in (dict(keep=-1), dict(sink=-1), dict(recent=-1), dict(stride=-1), dict(keep=2, sink=2, recent=1),
               dict(keep=2 ** 31 - 1, sink=2 ** 31 - 1, recent=1)):
        assert evict(lib, cfg, **kw) == kivi.ERR_ARG, kw


def test_unsupported(lib):
    other = kivi.Config(head_dim=64, num_q_heads=8, num_kv_heads=2).c()
    for call in (window, weights, chunk):
        assert call(lib, other) == kivi.ERR_UNSUPPORTED
    wide = kivi.Config(num_q_heads=66, num_kv_heads=2).c()         # 33 query heads to a kv head
    assert window(lib, wide) == kivi.ERR_UNSUPPORTED and weights(lib, wide) == kivi.ERR_UNSUPPORTED
    cfg = kivi.Config(num_q_heads=8, num_kv_heads=2).c()
    assert chunk(lib, cfg, max_new=2 ** 30) == kivi.ERR_UNSUPPORTED     # (query, head) rows past 32 bits
    assert chunk(lib, cfg, nseq=65535, max_new=2 ** 28) == kivi.ERR_UNSUPPORTED   # row tiles past 32 bits
    assert chunk(lib, cfg, mkl=2 ** 31 - 1) == kivi.ERR_UNSUPPORTED     # positions past 32 bits
    assert evict(lib, kivi.Config(residual=12800).c()) == kivi.ERR_UNSUPPORTED


def test_workspaces(lib):
    c = kivi.Config(num_q_heads=8, num_kv_heads=2)
    cfg = c.c()
    ws, sc = c.decode_ext_workspace_bytes(2, 5000), c.decode_weights_scratch_bytes(2, 5000)
    assert ws > 0 and sc == 2 * 8 * (157 * 8 + 4)                  # 157 tiles of 32 tokens; a float2 each, and one float a head
    for call in (window, weights):
        assert call(lib, cfg, n=ws - 1) == kivi.ERR_WORKSPACE
        assert call(lib, cfg, ws=None) == kivi.ERR_WORKSPACE
    assert weights(lib, cfg, m=sc - 1) == kivi.ERR_WORKSPACE
    assert weights(lib, cfg, sc=None) == kivi.ERR_WORKSPACE
    n = c.chunk_scratch_bytes(2, 7)
    assert c.chunk_scratch_bytes(2, 33) > n > 0                    # more than 128 rows: two row tiles a record
    assert chunk(lib, cfg, m=n - 1) == kivi.ERR_WORKSPACE and chunk(lib, cfg, sc=None) == kivi.ERR_WORKSPACE
    e = int(lib.kivi_evict_scratch_bytes(2, 50))
    assert e == 2 * 52 * 4
    assert evict(lib, cfg, m=e - 1) == kivi.ERR_WORKSPACE and evict(lib, cfg, sc=None) == kivi.ERR_WORKSPACE
    assert int(lib.kivi_evict_scratch_bytes(-1, 50)) == 0


def test_empty_calls_do_nothing(lib):
    cfg = kivi.Config(num_q_heads=8, num_kv_heads=2).c()
    assert window(lib, cfg, nseq=0, seqs=None, kv=None, q=None, out=None, ws=None, n=0) == kivi.OK
    assert weights(lib, cfg, nseq=0, seqs=None, kv=None, q=None, out=None, w_in=None, w_out=None, ws=None, n=0, sc=None,
                   m=0) == kivi.OK
    assert chunk(lib, cfg, nseq=0, seqs=None, kv=None, q=None, out=None, sc=None, m=0) == kivi.OK
    assert chunk(lib, cfg, max_new=0, seqs=None, kv=None, q=None, out=None, sc=None, m=0) == kivi.OK
    assert evict(lib, cfg, nseq=0, seqs=None, kv=None, w=None, sc=None, m=0, status=None) == kivi.OK
