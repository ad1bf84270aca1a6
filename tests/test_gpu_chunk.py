"""GPU tests of chunk attention (kivi_chunk_attn): chunks of any lengths over the packed cache against
a 64-bit statement, the cache untouched, and the chunk appended afterwards."""
import numpy as np
import pytest
import torch

import bit_asymmetric_kv_kivi_gb300 as kivi
import oracle
import synth
from gpu_util import configs, dev_tensor
from ops_ref import KEY_STEP, attend, chunk_bounds, dense, visible, widen
from test_gpu_window import build

pytestmark = pytest.mark.gpu

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def chunk_inputs(wl, new, seed=0):
    """Per sequence: queries [n][Hq][D] and the next n keys and values [H][n][D] (bit patterns)."""
    rng = np.random.default_rng(seed)
    q = [synth.to_dtype_bits(rng.standard_normal((n, wl.num_q_heads, 128)), wl.dtype) for n in new]
    kv = [wl.kv_seq(b, wl.lengths[b], n) for b, n in enumerate(new)]
    return q, [x for x, _ in kv], [x for _, x in kv]


def check(wl, refs, q, k, v, outs, window, sinks, key_step=None):
    dt = refs[0].cfg.dtype
    num = den = lim = 0.0
    for b, r in enumerate(refs):
        n = q[b].shape[0]
        if n == 0:
            continue
        qf = widen(q[b], dt)
        kc, vc, km, _ = dense(r)
        kk, vv = np.concatenate([kc, widen(k[b], dt)], 1), np.concatenate([vc, widen(v[b], dt)], 1)
        km = np.concatenate([km, np.abs(widen(k[b], dt))], 1)
        want, p = attend(qf, kk, vv, visible(r.L + n, n, window, sinks), wl.softmax_scale)
        got = outs[b].double().cpu().numpy()
        el, rel = chunk_bounds(qf, kk, vv, p, want, wl.softmax_scale, HALF[wl.dtype], key_step or KEY_STEP[dt], km)
        bad = ~(np.abs(got - want) <= el)
        assert not bad.any(), (b, r.L, n, np.argwhere(bad)[:4], np.abs(got - want).max(), el.max())
        num, den, lim = num + ((got - want) ** 2).sum(), den + (want ** 2).sum(), max(lim, rel)
    assert den == 0 or np.sqrt(num / den) <= lim, (np.sqrt(num / den), lim)


def run(cache, wl, q, k, v, window=0, sinks=0):
    d = lambda xs: [dev_tensor(x, wl.dtype) for x in xs]   # noqa: E731
    outs = cache.chunk(d(q), d(k), d(v), window=window, sinks=sinks, softmax_scale=wl.softmax_scale)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    return outs


@pytest.mark.parametrize("n", [1, 2, 5, 40, 127, 128, 300])
@pytest.mark.parametrize("L", [0, 1, 100, 160, 161, 1000])
def test_one_sequence(n, L):
    wl = synth.Workload("one", 1, 1, 1, 128, (L,), "f16", seed=L + n)
    cache, refs = build(wl, 2, 2, 32, 128, 1024)
    q, k, v = chunk_inputs(wl, [n], n)
    check(wl, refs, q, k, v, run(cache, wl, q, k, v), 0, 0)


@pytest.mark.parametrize("g", [1, 3, 4, 7, 8, 40])
@pytest.mark.parametrize("kb,vb,G,R,dtype,paged", [(2, 2, 32, 128, "bf16", True), (4, 4, 64, 64, "f16", False),
                                                   (2, 4, 32, 32, "f16", True), (4, 2, 64, 128, "bf16", False)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (130, 4), (300, 200), (5000, 4)])
def test_ragged_batch(g, kb, vb, G, R, dtype, paged, window, sinks):
    """Empty and one-token chunks next to long ones, empty caches and every edge of the packed split."""
    lengths, new = (0, 700, 33, 161, 0, 1500, 95), (130, 1, 0, 7, 1, 65, 260)
    H = 2
    wl = synth.Workload("ragged", len(lengths), g * H, H, 128, lengths, dtype, seed=70 + g)
    cache, refs = build(wl, kb, vb, G, R, 1536, paged=paged)
    q, k, v = chunk_inputs(wl, new, g)
    check(wl, refs, q, k, v, run(cache, wl, q, k, v, window, sinks), window, sinks)


@pytest.mark.parametrize("kb,vb,dtype", [(4, 4, "f16"), (4, 4, "bf16"), (2, 2, "f16"), (2, 4, "bf16")])
def test_many_short_sequences(kb, vb, dtype):
    """Hundreds of segments a CTA of every kind behind one another: narrow and wide, one tile and several,
    no packed tokens, one subtile of them, or many. Twice, bit for bit."""
    rng = np.random.default_rng(kb + vb)
    nseq, H, g, R = 700, 2, 4, 32
    lengths = tuple(int(x) for x in rng.choice([0, 5, 64, 70, 96, 130, 200, 300], nseq))
    new = [int(x) for x in rng.choice([0, 1, 2, 3, 33, 40], nseq, p=[0.1, 0.3, 0.2, 0.2, 0.1, 0.1])]
    wl = synth.Workload("short", nseq, g * H, H, 128, lengths, dtype, seed=19)
    cache, refs = build(wl, kb, vb, 32, R, 320, paged=True)
    q, k, v = chunk_inputs(wl, new, 5)
    outs = run(cache, wl, q, k, v)
    check(wl, refs, q, k, v, outs, 0, 0)
    for _ in range(3):
        again = run(cache, wl, q, k, v)
        assert all(torch.equal(a, b) for a, b in zip(outs, again))
    check(wl, refs, q, k, v, run(cache, wl, q, k, v, 60, 10), 60, 10)


@pytest.mark.parametrize("H,g,n", [(1, 4, 3), (2, 1, 1), (1, 8, 64)])
def test_long_cache_split_over_ctas(H, g, n):
    """Few rows over a long cache: every CTA takes a part and the parts are joined."""
    wl = synth.Workload("split", 1, H * g, H, 128, (20000,), "f16", seed=5)
    cache, refs = build(wl, 2, 2, 32, 128, 20000)
    q, k, v = chunk_inputs(wl, [n])
    for window, sinks in ((0, 0), (9000, 5)):
        check(wl, refs, q, k, v, run(cache, wl, q, k, v, window, sinks), window, sinks)


def test_large_scores_and_scales():
    """Scores that leave one token all the weight, queries far from 1, and negative and zero scales."""
    wl = synth.Workload("scores", 2, 4, 1, 128, (300, 20), "bf16", seed=3)
    cache, refs = build(wl, 2, 2, 32, 128, 512)
    q, k, v = chunk_inputs(wl, (150, 9))
    fq = [widen(x, oracle.BF16) for x in q]
    for s in (2.0 ** 12, 2.0 ** -30):
        qs = [synth.to_dtype_bits(x * s, "bf16") for x in fq]
        w = wl
        for scale in (w.softmax_scale / s, -w.softmax_scale / s, 0.0, 3 * w.softmax_scale / s):
            d = lambda xs: [dev_tensor(x, "bf16") for x in xs]   # noqa: E731
            outs = cache.chunk(d(qs), d(k), d(v), softmax_scale=scale)
            for b, r in enumerate(refs):
                qf = widen(qs[b], oracle.BF16)
                kc, vc, km, _ = dense(r)
                kk, vv, km = (np.concatenate([c, f(widen(x[b], oracle.BF16))], 1)
                              for c, x, f in ((kc, k, lambda y: y), (vc, v, lambda y: y), (km, k, np.abs)))
                n = qf.shape[0]
                want, p = attend(qf, kk, vv, visible(r.L + n, n, 0, 0), scale)
                el, _ = chunk_bounds(qf, kk, vv, p, want, abs(scale), HALF["bf16"], KEY_STEP[oracle.BF16], km)
                assert (np.abs(outs[b].double().cpu().numpy() - want) <= el).all()


@pytest.mark.parametrize("kb", [2, 4])
@pytest.mark.parametrize("size,key_step", [(2.0 ** -16, 2.0 ** -11), (2.0 ** -9, None), (200.0, 2.0 ** -11)])
def test_key_magnitudes(kb, size, key_step):
    """fp16 keys of every size: tiny ones (whose scales are subnormal f16 numbers, so the rests are too), small
    ones, and ones past 2^13, which are kept in one f16 number."""
    wl = synth.Workload("mags", 1, 4, 1, 128, (600,), "f16", seed=kb)
    k0, v0 = wl.kv_seq(0, 0, 640)
    k0 = synth.to_dtype_bits(widen(k0, oracle.F16) * size, "f16")
    kcfg, ocfg = configs(2, "f16", 4, 1, kb=kb, vb=2)
    cache, r = kivi.KVCache(kcfg, 1, 640), oracle.SeqCache(ocfg, 640)
    assert r.append(np.ascontiguousarray(k0[:, :600]), np.ascontiguousarray(v0[:, :600])) == oracle.OK
    d = lambda x: dev_tensor(np.ascontiguousarray(x), "f16")   # noqa: E731
    cache.append([d(k0[:, :600])], [d(v0[:, :600])])
    rng = np.random.default_rng(1)
    q = [synth.to_dtype_bits(rng.standard_normal((40, 4, 128)), "f16")]
    k, v = [np.ascontiguousarray(k0[:, 600:])], [np.ascontiguousarray(v0[:, 600:])]
    scale = wl.softmax_scale / size
    outs = cache.chunk([d(q[0])], [d(k[0])], [d(v[0])], softmax_scale=scale)
    assert int(cache.status.item()) == 0
    qf = widen(q[0], oracle.F16)
    kc, vc, km, _ = dense(r)
    kk, vv = np.concatenate([kc, widen(k[0], oracle.F16)], 1), np.concatenate([vc, widen(v[0], oracle.F16)], 1)
    km = np.concatenate([km, np.abs(widen(k[0], oracle.F16))], 1)
    want, p = attend(qf, kk, vv, visible(640, 40, 0, 0), scale)
    el, rel = chunk_bounds(qf, kk, vv, p, want, scale, HALF["f16"], key_step or KEY_STEP[oracle.F16], km)
    # levels below 2^-14 are rounded at 2^-24 of one, whatever their size
    el = el + 2 * scale * 2.0 ** -24 * np.abs(qf).sum(-1, keepdims=True) * np.einsum("nht,htd->nhd", p, np.repeat(np.abs(vv), 4, 0))
    got = outs[0].double().cpu().numpy()
    assert (np.abs(got - want) <= el).all(), (np.abs(got - want) / el).max()


def test_rows_between_sequences_and_bad_lengths():
    """Rows that no sequence owns stay as they were; a bad count writes nothing, a bad length NaN."""
    lengths, new = (300, 50, 200), (5, 3, 4)
    wl = synth.Workload("rows", 3, 8, 2, 128, lengths, "f16", seed=12)
    cache, refs = build(wl, 2, 2, 32, 128, 512)
    q, k, v = chunk_inputs(wl, new)
    start = [20, 2, 10]
    qd = torch.zeros((30, 8, 128), dtype=torch.float16, device="cuda")
    for b in range(3):
        qd[start[b]:start[b] + new[b]] = dev_tensor(q[b], "f16")
    out = torch.full_like(qd, 7.0)
    kd, vd = [dev_tensor(x, "f16") for x in k], [dev_tensor(x, "f16") for x in v]
    i = lambda x, t: torch.tensor(x, dtype=t, device="cuda")   # noqa: E731
    args = (qd, i(start, torch.int32), i([x.data_ptr() for x in kd], torch.int64), i([x.data_ptr() for x in vd], torch.int64))
    cache.chunk_attn(*args, i(new, torch.int32), 5, out=out, softmax_scale=wl.softmax_scale)
    assert int(cache.status.item()) == 0
    check(wl, refs, q, k, v, [out[s:s + n] for s, n in zip(start, new)], 0, 0)
    owned = torch.zeros(30, dtype=torch.bool)
    for s, n in zip(start, new):
        owned[s:s + n] = True
    assert bool((out[~owned.cuda()] == 7).all())
    out.fill_(7.0)
    cache.chunk_attn(*args, i((5, 9, 4), torch.int32), 5, out=out, softmax_scale=wl.softmax_scale, max_kv_len=250)
    assert int(cache.status.item()) == kivi.ERR_LENGTH
    assert bool(out[20:25].isnan().all()) and bool((out[2:10] == 7).all())
    check(wl, refs[2:], q[2:], k[2:], v[2:], [out[10:14]], 0, 0)


def test_cache_untouched_then_appended_in_chunks():
    """A prompt in chunks of odd sizes: attention, then append; the state equals the oracle's and every
    chunk's attention the 64-bit statement on it. Captured calls read the lengths at replay."""
    H, g = 2, 4
    wl = synth.Workload("prefill", 2, g * H, H, 128, (0, 0), "bf16", seed=44)
    cache, refs = build(wl, 2, 2, 32, 64, 1024, paged=True)
    pos = [0, 0]
    for step, n in enumerate(((200, 1), (1, 130), (77, 64), (300, 300))):
        at = synth.Workload("prefill", 2, g * H, H, 128, tuple(pos), "bf16", seed=44)
        q, k, v = chunk_inputs(at, n, step)
        before = [cache.seq_numpy(b) for b in range(2)]
        check(wl, refs, q, k, v, run(cache, wl, q, k, v), 0, 0)
        for b in range(2):
            after = cache.seq_numpy(b)
            assert all(np.array_equal(before[b][x], after[x]) for x in after)
            assert refs[b].append(k[b], v[b]) == oracle.OK
            pos[b] += n[b]
        cache.append([dev_tensor(x, "bf16") for x in k], [dev_tensor(x, "bf16") for x in v])
    from gpu_util import assert_state_equal
    for b in range(2):
        assert_state_equal(cache, b, refs[b])


def test_captured_and_on_another_stream():
    wl = synth.Workload("cap", 2, 8, 2, 128, (500, 90), "f16", seed=21)
    cache, refs = build(wl, 2, 2, 32, 128, 1024)
    q, k, v = chunk_inputs(wl, (33, 20))
    kd, vd = [dev_tensor(x, "f16") for x in k], [dev_tensor(x, "f16") for x in v]
    i = lambda x, t: torch.tensor(x, dtype=t, device="cuda")   # noqa: E731
    qd = torch.cat([dev_tensor(x, "f16") for x in q])
    n = i((33, 20), torch.int32)
    args = (qd, i((0, 33), torch.int32), i([x.data_ptr() for x in kd], torch.int64), i([x.data_ptr() for x in vd], torch.int64), n, 40)
    out = torch.zeros_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.chunk_attn(*args, out=out, softmax_scale=wl.softmax_scale, max_kv_len=900)
    torch.cuda.synchronize()
    check(wl, refs, q, k, v, out.split((33, 20)), 0, 0)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.chunk_attn(*args, out=out, softmax_scale=wl.softmax_scale, max_kv_len=900)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    n.copy_(i((1, 20), torch.int32))          # fewer tokens: same rows, read at replay
    out.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((out[1:33] == 3).all()) and bool((out[:1] != 3).any())
