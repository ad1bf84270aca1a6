"""GPU tests of kivi_evict_groups: which groups stay, and that the buffers, tables, rings and
weights close up exactly as the plain statement says, bit for bit."""
import numpy as np
import pytest
import torch

import bit_asymmetric_kv_kivi_gb300 as kivi
import oracle
import synth
from gpu_util import configs, dev_tensor
from ops_ref import evict
from test_gpu_window import build, check

pytestmark = pytest.mark.gpu

LENGTHS = (0, 1, 128, 160, 161, 400, 1000, 2500, 2559)


def expect(before, cfg, kept, turn):
    """Buffers of one sequence (seq_numpy) after the eviction: packed entries and the whole ring."""
    G, n = cfg.group, len(kept)
    kept = np.array(kept, dtype=np.int64)
    want = {}
    for name in ("k_codes", "v_codes", "v_scale", "v_zero"):
        x = before[name]
        x = x.reshape(x.shape[0], -1, G, x.shape[-1])[:, kept]
        want[name] = x.reshape(x.shape[0], n * G, x.shape[-1])
    for name in ("k_scale", "k_zero"):
        want[name] = before[name][:, kept]
    ring = cfg.residual + G
    rows = (np.arange(ring) + turn) % ring
    for name in ("k_res", "v_res"):
        want[name] = before[name][:, rows]
    want["kv_len"] = before["kv_len"] - turn
    return want


def same(got, want):
    for name, x in want.items():
        if name == "kv_len":
            assert got[name] == x
        else:
            assert np.array_equal(got[name][:, :x.shape[1]], x), name


def weights_for(cache, kind, seed):
    shape = (cache.nseq, cache.weight_groups())
    rng = np.random.default_rng(seed)
    if kind == "ties":
        w = rng.integers(0, 3, shape).astype(np.float32)
        w[w == 0] = -0.0
        w[:, ::5] = 0.0
    elif kind == "equal":
        w = np.full(shape, 0.25, np.float32)
    else:
        w = np.exp(4 * rng.standard_normal(shape)).astype(np.float32)
        w[:, 3::7] *= -1
        w[:, 2] = np.inf
        w[:, 4] = np.nan
        w[:, 6] = -np.inf
        w[:, 9] = 1e-42
    return w


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kb,vb,G,R,dtype", [(2, 2, 32, 128, "bf16"), (4, 2, 64, 64, "f16"), (2, 4, 32, 32, "f16")])
@pytest.mark.parametrize("keep,sink,recent,kind", [(20, 1, 2, "wide"), (7, 0, 0, "ties"), (33, 2, 3, "equal"), (5, 3, 2, "wide"),
                                                   (0, 0, 0, "wide"), (1000, 0, 0, "ties"), (71, 1, 0, "wide")])
def test_evict(paged, kb, vb, G, R, dtype, keep, sink, recent, kind):
    H = 3
    wl = synth.Workload("evict", len(LENGTHS), H, H, 128, LENGTHS, dtype, seed=90)
    cache, _ = build(wl, kb, vb, G, R, 2560, paged=paged)
    w = weights_for(cache, kind, keep)
    before = [cache.seq_numpy(b) for b in range(wl.batch)]
    tables = cache.block_tables.cpu().numpy() if paged else None
    wd = torch.from_numpy(w).cuda()
    cache.evict(wd, keep, sink_groups=sink, recent_groups=recent)
    got_w = wd.cpu().numpy()
    assert int(cache.status.item()) == 0
    for b, L in enumerate(LENGTHS):
        kept, gone, want_w, turn = evict(oracle.Cfg(group=G, residual=R), w[b], L, keep, sink, recent)
        same(cache.seq_numpy(b), expect(before[b], cache.cfg, kept, turn))
        assert np.array_equal(got_w[b], want_w, equal_nan=True), b
        if paged and gone:
            t = cache.block_tables[b].cpu().numpy()
            n = len(kept) + len(gone)
            assert np.array_equal(t, np.concatenate([tables[b][kept], tables[b][gone], tables[b][n:]]))
    assert cache.max_len <= max(keep * G + R + G - 1, 0)


@pytest.mark.parametrize("D,G,R", [(64, 64, 256), (96, 32, 1024), (256, 64, 64), (32, 32, 12768)])
def test_evict_other_head_dims_and_rings(D, G, R):
    """Every head_dim of the codec; rings up to the longest that fits."""
    cfg = kivi.Config(head_dim=D, num_q_heads=2, num_kv_heads=2, residual=R, group=G)
    cap = 40 * G
    cache = kivi.KVCache(cfg, 2, cap)
    gen = torch.Generator(device="cuda").manual_seed(D)
    L = (R + 37 * G + 5, R + 20)
    cache.append([torch.randn((2, n, D), generator=gen, device="cuda").half() for n in L],
                 [torch.randn((2, n, D), generator=gen, device="cuda").half() for n in L])
    before = [cache.seq_numpy(b) for b in range(2)]
    w = weights_for(cache, "wide", D)
    wd = torch.from_numpy(w).cuda()
    cache.evict(wd, 11, 1, 1)
    for b in range(2):
        kept, gone, want_w, turn = evict(oracle.Cfg(group=G, residual=R), w[b], L[b], 11, 1, 1)
        same(cache.seq_numpy(b), expect(before[b], cfg, kept, turn))
        assert np.array_equal(wd[b].cpu().numpy(), want_w, equal_nan=True)


def test_evict_very_long_sequence():
    """More groups than the selection keeps in shared memory."""
    D, G, R, n = 32, 32, 32, 9001
    cfg = kivi.Config(head_dim=D, residual=R, group=G)
    cache = kivi.KVCache(cfg, 1, n * G, paged=True, page_seed=1)
    L = R + n * G + 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache.append(torch.randn((1, 1, L, D), generator=gen, device="cuda").half(),
                 torch.randn((1, 1, L, D), generator=gen, device="cuda").half())
    before, table = cache.seq_numpy(0), cache.block_tables[0].cpu().numpy()
    for keep, kind in ((8800, "wide"), (300, "ties")):
        w = weights_for(cache, kind, keep)
        wd = torch.from_numpy(w).cuda()
        kept, gone, want_w, turn = evict(oracle.Cfg(group=G, residual=R), w[0], before["kv_len"], keep, 3, 5)
        cache.evict(wd, keep, 3, 5)
        same(cache.seq_numpy(0), expect(before, cfg, kept, turn))
        assert np.array_equal(wd[0].cpu().numpy(), want_w, equal_nan=True)
        got = cache.block_tables[0].cpu().numpy()
        assert np.array_equal(got[:keep], table[kept]) and sorted(got) == sorted(table)
        before, table = cache.seq_numpy(0), got
    assert int(cache.status.item()) == 0


def test_cache_over_given_buffers():
    """KVCache.from_buffers reads and writes the caller's tensors; tensors that do not fit are refused."""
    wl = synth.Workload("given", 2, 4, 2, 128, (700, 161), "f16", seed=6)
    cache, refs = build(wl, 2, 2, 32, 128, 704, paged=True)
    buf = {n: getattr(cache, n) for n in kivi.SEQ_FIELDS}
    args = (cache.cfg, buf, cache.kv_len, 704)
    other = kivi.KVCache.from_buffers(*args, block_tables=cache.block_tables, max_len=700)
    q = dev_tensor(wl.query(0), "f16")
    assert torch.equal(other.decode_window(q, 300, 4), cache.decode_window(q, 300, 4))
    w = torch.rand((2, other.weight_groups()), device="cuda")
    other.evict(w, 5)
    assert other.max_len == 5 * 32 + 159 and int(cache.kv_len[0]) == 700 - (17 - 5) * 32
    halves = {n: t.view(torch.float16) if t.dtype == torch.int16 else t for n, t in buf.items()}
    kivi.KVCache.from_buffers(cache.cfg, halves, cache.kv_len, 704, block_tables=cache.block_tables)
    for name in kivi.SEQ_FIELDS:
        for bad in (buf[name][:, :1], buf[name].float(), buf[name].cpu()):
            with pytest.raises(ValueError):
                kivi.KVCache.from_buffers(cache.cfg, {**buf, name: bad}, cache.kv_len, 704, block_tables=cache.block_tables)
    with pytest.raises(ValueError):
        kivi.KVCache.from_buffers(cache.cfg, buf, cache.kv_len, 700, block_tables=cache.block_tables)
    with pytest.raises(ValueError):
        kivi.KVCache.from_buffers(cache.cfg, buf, cache.kv_len, 704, block_tables=cache.block_tables[:, :4])
    with pytest.raises(ValueError):
        other.decode_window(q, 300, out=torch.empty((2, 4, 128), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        other.decode_window(q.bfloat16(), 300)
    with pytest.raises(ValueError):
        other.decode_weights(q, w.double())
    for call in (lambda x: other.decode_window(q, x), lambda x: other.decode_window(q, 5, x), lambda x: other.evict(w, x),
                 lambda x: other.evict(w, 5, x), lambda x: other.decode_window(q, 5, max_kv_len=x)):
        for x in (2 ** 32 + 5, -2 ** 31 - 1):
            with pytest.raises(ValueError):
                call(x)


def test_evict_refusals_leave_the_cache_alone():
    wl = synth.Workload("refuse", 2, 2, 2, 128, (1000, 500), "f16", seed=5)
    cache, _ = build(wl, 2, 2, 32, 128, 1024)
    before = [cache.seq_numpy(b) for b in range(2)]
    w = torch.rand((2, cache.weight_groups()), device="cuda")
    for bad in (dict(keep_groups=-1), dict(keep_groups=3, sink_groups=2, recent_groups=2), dict(keep_groups=3, sink_groups=-1)):
        with pytest.raises(kivi.KiviError):
            cache.evict(w, **bad)
    with pytest.raises(ValueError):
        cache.evict(w[:, :10].contiguous(), 4)
    with pytest.raises(ValueError):
        cache.evict(w.half(), 4)
    # a row too short for one sequence (device check): that one keeps its groups, the other is cut
    cache.max_len = 0
    w2 = torch.rand((2, 20), device="cuda")
    cache.evict(w2, 4)
    assert int(cache.status.item()) == kivi.ERR_LENGTH
    got = cache.seq_numpy(0)
    same(got, {k: v for k, v in before[0].items()})
    assert cache.seq_numpy(1)["kv_len"] < 500


@pytest.mark.parametrize("paged", [False, True])
def test_serving_run(paged):
    """Decode steps that collect weights, an eviction when the budget is passed, more steps: attention
    after each eviction equals the 64-bit attention over exactly the kept tokens, with the oracle
    cache cut the same way (the packed groups that follow go to the freed pages)."""
    H, g, G, R, keep = 2, 4, 32, 64, 6
    lengths = (300, 40, 420)
    wl = synth.Workload("serve", 3, g * H, H, 128, lengths, "bf16", seed=33)
    cache, refs = build(wl, 2, 2, G, R, 512, paged=paged)
    w = torch.zeros((3, cache.weight_groups()), device="cuda")
    pos = list(lengths)
    for step in range(70):
        kn, vn = zip(*(wl.kv_seq(b, pos[b], 1) for b in range(3)))
        for b, r in enumerate(refs):
            assert r.append(kn[b], vn[b]) == oracle.OK
            pos[b] += 1
        cache.append([dev_tensor(x, "bf16") for x in kn], [dev_tensor(x, "bf16") for x in vn])
        before = w.cpu().numpy()
        out, _ = cache.decode_weights(dev_tensor(wl.query(0), "bf16"), w, softmax_scale=wl.softmax_scale)
        check(wl, cache, refs, out, 0, 0, w.cpu().numpy(), before)
        if step % 20 == 10:
            ws = w.cpu().numpy()
            cache.evict(w, keep, sink_groups=1, recent_groups=1)
            for b, r in enumerate(refs):
                kept, _, _, turn = evict(r.cfg, ws[b], r.L, keep, 1, 1)
                buf = {n: getattr(r, n) for n in kivi.SEQ_FIELDS}
                want = expect({**buf, "kv_len": r.L}, cache.cfg, kept, turn)
                for n in kivi.SEQ_FIELDS:
                    getattr(r, n)[:, :want[n].shape[1]] = want[n]
                r.kv_len[0] = want["kv_len"]
                got = cache.seq_numpy(b)
                assert got["kv_len"] == r.L
    assert int(cache.status.item()) == 0
