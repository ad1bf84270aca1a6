"""GPU tests of windowed decode attention (kivi_decode_window_attn) against a 64-bit statement
of the visible tokens, and of the per-group weights of kivi_decode_attn_weights."""
import numpy as np
import pytest
import torch

import bit_asymmetric_kv_kivi_gb300 as kivi
import oracle
import synth
from gpu_util import configs, dev_tensor
from ops_ref import attend, decode_bounds, dense, visible, widen

pytestmark = pytest.mark.gpu

LENGTHS = (0, 1, 31, 33, 95, 128, 160, 161, 300, 1000, 2500)


def build(wl, kb, vb, G, R, cap, paged=False):
    kcfg, ocfg = configs(2, wl.dtype, wl.num_q_heads, wl.num_kv_heads, R=R, G=G, kb=kb, vb=vb)
    cache = kivi.KVCache(kcfg, wl.batch, cap, paged=paged, page_seed=3)
    refs, ks, vs = [], [], []
    for b, L in enumerate(wl.lengths):
        K, V = wl.kv_seq(b, 0, L)
        ks.append(dev_tensor(K, wl.dtype))
        vs.append(dev_tensor(V, wl.dtype))
        r = oracle.SeqCache(ocfg, cap)
        assert r.append(K, V) == oracle.OK
        refs.append(r)
    cache.append(ks, vs)
    return cache, refs


def check(wl, cache, refs, out, window, sinks, weights=None, before=None, decay=1.0):
    q = widen(wl.query(0), refs[0].cfg.dtype)
    out = out.cpu().numpy()
    assert int(cache.status.item()) == 0
    G = refs[0].cfg.group
    for b, r in enumerate(refs):
        if r.L == 0:
            assert np.all(out[b] == 0)
            if weights is not None:
                assert np.all(weights[b] == 0)
            continue
        k, v, km, vm = dense(r)
        want, p = attend(q[b:b + 1], k, v, visible(r.L, 1, window, sinks), wl.softmax_scale)
        tol, rel = decode_bounds(q[b:b + 1], km, vm, p, wl.softmax_scale)
        bad = np.abs(out[b] - want[0]) > tol[0]
        assert not bad.any(), (b, r.L, np.abs(out[b] - want[0]).max(), tol[0].max())
        if weights is not None:
            n = -(-r.L // G)
            pad = np.zeros((p.shape[1], n * G))
            pad[:, :r.L] = p[0]
            per = pad.reshape(p.shape[1], n, G).sum(-1)                   # [Hq][groups]
            w = per.sum(0) + decay * before[b, :n].astype(np.float64)
            lim = (per * rel[0]).sum(0) + 2.0 ** -22 * np.abs(w) + 1e-30
            assert (np.abs(weights[b, :n] - w) <= lim).all(), (b, np.abs(weights[b, :n] - w).max(), lim.max())
            assert np.all(weights[b, n:] == 0)


@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8, 12])
@pytest.mark.parametrize("kb,vb,G,R,dtype", [(2, 2, 32, 128, "bf16"), (4, 2, 64, 64, "f16"), (2, 4, 32, 32, "f16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (256, 33), (700, 200), (5000, 4)])
def test_window_edges(g, kb, vb, G, R, dtype, window, sinks):
    """Windows from one token to more than the sequence, sinks that end inside a tile, overlap the
    window, or reach into the residual tokens; every length at an edge of the packed split."""
    H = 2
    wl = synth.Workload("win", len(LENGTHS), g * H, H, 128, LENGTHS, dtype, seed=60 + g)
    cache, refs = build(wl, kb, vb, G, R, 2560, paged=g % 2 == 1)
    out = cache.decode_window(dev_tensor(wl.query(0), dtype), window, sinks, softmax_scale=wl.softmax_scale)
    check(wl, cache, refs, out, window, sinks)
    assert int(cache._ext_ws.count_nonzero()) == 0


def test_window_long_stream_precision():
    """One long stream over many CTAs, next to short ones: the output keeps its 32 bits."""
    lengths = (30000, 50, 7000)
    wl = synth.Workload("long", 3, 4, 1, 128, lengths, "f16", seed=77)
    cache, refs = build(wl, 2, 2, 32, 128, 30016)
    q = dev_tensor(wl.query(0), "f16")
    for window, sinks in ((0, 0), (20000, 5), (29999, 0)):
        check(wl, cache, refs, cache.decode_window(q, window, sinks, softmax_scale=wl.softmax_scale), window, sinks)


def test_window_whole_cache_equals_decode_closely():
    wl = synth.Workload("same", 3, 8, 2, 128, (700, 161, 5), "bf16", seed=8)
    cache, _ = build(wl, 2, 2, 32, 128, 704)
    q = dev_tensor(wl.query(0), "bf16")
    a, b = cache.decode(q), cache.decode_window(q, 0)
    c = cache.decode_window(q, 100000, 3)
    assert torch.equal(b, c)
    assert float((a - b).abs().max()) <= 1e-4


def test_window_bad_length_gives_nan_and_status():
    wl = synth.Workload("bad", 2, 2, 1, 128, (300, 100), "f16", seed=10)
    cache, refs = build(wl, 2, 2, 32, 128, 256)
    q = dev_tensor(wl.query(0), "f16")
    w = torch.full((2, 7), 2.0, device="cuda")
    out, got = cache.decode_weights(q, w, torch.empty_like(w), max_kv_len=200)
    assert int(cache.status.item()) == kivi.ERR_LENGTH
    assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())
    assert bool((got[0] == 2).all()) and bool((got[1, 4:] == 0).all())


@pytest.mark.parametrize("g", [1, 2, 4, 5, 8, 20])
@pytest.mark.parametrize("kb,vb,G,R,dtype", [(2, 2, 32, 128, "bf16"), (4, 4, 64, 128, "f16")])
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.5])
def test_weights(g, kb, vb, G, R, dtype, decay):
    H = 2
    wl = synth.Workload("wts", len(LENGTHS), g * H, H, 128, LENGTHS, dtype, seed=160 + g)
    cache, refs = build(wl, kb, vb, G, R, 2560, paged=g == 4)
    rng = np.random.default_rng(g)
    before = rng.random((wl.batch, cache.weight_groups()), dtype=np.float32)
    w_in = torch.from_numpy(before).cuda()
    if decay == 0.0:
        w_in.fill_(float("nan"))          # not read
        before = np.zeros_like(before)
    w_out = torch.full_like(w_in, 9.0)
    q = dev_tensor(wl.query(0), dtype)
    out, got = cache.decode_weights(q, w_in, w_out, decay=decay, softmax_scale=wl.softmax_scale)
    assert got is w_out
    check(wl, cache, refs, out, 0, 0, got.cpu().numpy(), before, decay)
    again, got2 = cache.decode_weights(q, w_in, None, decay=decay, softmax_scale=wl.softmax_scale)   # in place
    assert got2 is w_in and torch.equal(got2, got) and torch.equal(again, out)
    assert int(cache._ext_ws.count_nonzero()) == 0
    _, got3 = cache.decode_weights(q, None, softmax_scale=wl.softmax_scale)
    assert got3.shape == (wl.batch, cache.weight_groups())


def test_window_and_weights_captured_and_replayed():
    """Captured calls read the lengths at replay; a call that would have to make its workspace
    during the capture is refused."""
    wl = synth.Workload("graph", 3, 8, 2, 128, (400, 161, 900), "f16", seed=18)
    cache, refs = build(wl, 2, 2, 32, 128, 2048)
    q = dev_tensor(wl.query(0), "f16")
    out = torch.zeros((3, 8, 128), device="cuda")
    w = torch.zeros((3, cache.weight_groups()), device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with pytest.raises(RuntimeError, match="before the capture"):
            with torch.cuda.graph(graph, stream=stream):
                cache.decode_window(q, 256, 4, out=out, max_kv_len=2000)
    torch.cuda.synchronize()
    cache.decode_weights(q, w, decay=0.0, out=out, max_kv_len=2000)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_window(q, 256, 4, out=out, max_kv_len=2000)
        cache.decode_weights(q, w, decay=0.0, max_kv_len=2000)
    for n in (1, 300):
        ks = [dev_tensor(wl.kv_seq(b, refs[b].L, n)[0], "f16") for b in range(3)]
        vs = [dev_tensor(wl.kv_seq(b, refs[b].L, n)[1], "f16") for b in range(3)]
        for b, r in enumerate(refs):
            assert r.append(*wl.kv_seq(b, r.L, n)) == oracle.OK
        cache.append(ks, vs)
        graph.replay()
        torch.cuda.synchronize()
        check(wl, cache, refs, out, 256, 4)
        assert abs(float(w.sum()) - 3 * 8) < 1e-3


def test_captured_window_beside_decode_that_grows_its_workspace():
    """A graph's workspace stays its own when decode and decode_multi make and replace theirs, inside a
    capture and outside, and memory that they gave back is written."""
    wl = synth.Workload("beside", 3, 8, 2, 128, (4000, 161, 2900), "f16", seed=19)
    cache, refs = build(wl, 2, 2, 32, 128, 4096)
    q = dev_tensor(wl.query(0), "f16")
    out = torch.zeros((3, 8, 128), device="cuda")
    cache.decode(q)
    cache._ws = None
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        cache.decode(q)              # its workspace belongs to this graph, filled at replay
    cache.decode_window(q, 256, 4, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_window(q, 256, 4, out=out)
    many = q[:, None].expand(3, 8, 8, 128).contiguous()
    cache._ws = None
    for n in (1, 8):
        cache.decode_multi(many[:, :n].contiguous())
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 22) * 2]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(wl, cache, refs, out, 256, 4)
    assert int(cache._ext_ws.count_nonzero()) == 0 and len(junk) == 8
