"""Four operators over the packed KIVI cache: what is timed, and their plain forms.

window   one new token per sequence attends to the newest `window` cached tokens and to the
         first `sinks` ones (KVCache.decode_window)
weights  decode attention that also keeps, for each G-token group, the attention weight that
         all query heads gave to its tokens (KVCache.decode_weights)
evict    drops the packed groups of least weight until `keep` are left (KVCache.evict)
chunk    a chunk of new tokens per sequence attends to the cache and, causally, to itself,
         before it is appended (KVCache.chunk_attn)

A cached token is c * s + z where it is packed (2- or 4-bit codes, fp16 scale and zero; keys
per channel over G tokens, values per token over G channels) and as stored in the ring of
R + G slots where it is not: the first n_packed(L) = G floor(max(L - R, 0) / G) are packed.
"""
import math
import random

import torch

own = False

D = 128
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, nseq, hq, h, kv, dtype="bf16", kb=2, vb=2, G=32, R=128, paged=True, window=0, sinks=0,
          new=(0, 0), keep=0, sink_groups=0, recent_groups=0, decay=1.0, lens=1):
    return {"name": name, "op": op, "nseq": nseq, "hq": hq, "h": h, "kv_lo": kv[0], "kv_hi": kv[1], "dtype": dtype,
            "kb": kb, "vb": vb, "G": G, "R": R, "paged": paged, "window": window, "sinks": sinks, "new_lo": new[0],
            "new_hi": new[1], "keep": keep, "sink_groups": sink_groups, "recent_groups": recent_groups,
            "decay": decay, "lens": lens}


def listed():
    return [
        # one short conversation on a single head: what a call costs when there is hardly any work
        _case("window_tiny", "window", 1, 1, 1, (1024, 1024), "f16", window=256, sinks=4),
        # a full serving batch whose requests run with a bounded window
        _case("window_llama3_64x32k", "window", 64, 32, 8, (32768, 32768), window=4096, sinks=4),
        # ragged long requests, wider keys, 64-token groups, a prompt prefix that ends inside a tile kept visible
        _case("window_varlen_32", "window", 32, 32, 8, (1024, 131072), "f16", kb=4, G=64, R=64, window=8192, sinks=100),
        # a decode step of the serving batch while weights are collected for a later eviction
        _case("weights_llama3_64x32k", "weights", 64, 32, 8, (32768, 32768)),
        # a few short ragged requests, seven query heads to a kv head, weights that fade
        _case("weights_odd_g7", "weights", 3, 28, 4, (1, 9001), "f16", kb=4, G=64, R=64, paged=False, decay=0.875),
        # five draft tokens of one short request
        _case("chunk_tiny", "chunk", 1, 4, 1, (1000, 1000), "f16", new=(5, 5)),
        # four draft tokens of every request of the serving batch, checked before they are appended
        _case("chunk_verify_64x32k", "chunk", 64, 32, 8, (32768, 32768), new=(4, 4)),
        # one 2048-token piece of a long prompt, 32768 tokens in
        _case("chunk_long_2048", "chunk", 1, 32, 8, (32768, 32768), new=(2048, 2048)),
        # continuous batching: pieces of prompts and single tokens side by side, sliding window with sinks
        _case("chunk_ragged_g7", "chunk", 8, 28, 4, (0, 9000), "f16", kb=4, vb=4, G=64, R=64, window=4096, sinks=4,
              new=(1, 700), lens=59),
        # first pieces of two prompts: nothing cached yet, a kv head for each query head
        _case("chunk_first_mha", "chunk", 2, 32, 32, (0, 0), "f16", new=(4096, 4096), paged=False),
        # one short request over its budget
        _case("evict_tiny", "evict", 1, 8, 8, (1024, 1024), "f16", keep=16, sink_groups=1, recent_groups=2),
        # the whole serving batch cut to half
        _case("evict_llama3_64x32k", "evict", 64, 32, 8, (32768, 32768), keep=512, sink_groups=1, recent_groups=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.floor(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["window", "weights", "evict", "chunk", "chunk"])
    h = rng.choice([1, 2, 4, 8, 8, 32])
    g = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
    g = g if h * g <= 64 else max(1, 64 // h)
    G = rng.choice([32, 32, 64])
    R = G * rng.choice([1, 2, 4])
    top = _log_int(rng, 512 if op == "evict" else 1, 65536)
    # at most as many cached (token, kv head) pairs as the largest listed batch holds
    nseq = _log_int(rng, 1, max(1, min(64, 16777216 // (top * h))))
    lo = rng.choice([top, max(1, top // 7), 0 if op == "chunk" else 1])
    c = _case("", op, nseq, h * g, h, (lo, top), rng.choice(["f16", "bf16"]), rng.choice([2, 2, 4]),
              rng.choice([2, 2, 4]), G, R, rng.random() < 0.6, lens=rng.randrange(1 << 30))
    if op == "window" or (op == "chunk" and rng.random() < 0.5):
        c["window"] = _log_int(rng, 1, 16384)
        c["sinks"] = rng.choice([0, 1, 4, 4, 33, 128])
    if op == "weights":
        c["decay"] = rng.choice([0.0, 0.5, 0.99, 1.0])
    if op == "chunk":
        # at most the query-key pairs of the largest listed chunk: n (top + n) of each head
        pairs = 2048 * 33792 * 32 / (nseq * h * g)
        n = _log_int(rng, 1, max(1, min(4096, int((math.sqrt(top * top + 4 * pairs) - top) / 2))))
        c["new_lo"], c["new_hi"] = rng.choice([n, 1]), n
    if op == "evict":
        ng = max(1, top // G)
        c["paged"] = True   # a contiguous cache is cut in place, which cannot be repeated on the same state
        c["sink_groups"], c["recent_groups"] = rng.choice([0, 1, 3]), rng.choice([0, 1, 8])
        c["keep"] = max(c["sink_groups"] + c["recent_groups"], _log_int(rng, 1, ng))
    del c["name"]
    return c


# ---------------------------------------------------------------- sizes
def _lengths(case):
    """Cached tokens and new tokens of each sequence: log-uniform in the case's ranges."""
    r = random.Random(case["lens"])
    kv = [case["kv_hi"] if case["kv_lo"] == case["kv_hi"] else
          int(math.exp(r.uniform(math.log(case["kv_lo"] + 1), math.log(case["kv_hi"] + 1)))) - (case["kv_lo"] == 0)
          for _ in range(case["nseq"])]
    new = [case["new_hi"] if case["new_lo"] == case["new_hi"] else
           int(math.exp(r.uniform(math.log(max(case["new_lo"], 1)), math.log(case["new_hi"] + 1))))
           for _ in range(case["nseq"])]
    return [min(max(x, case["kv_lo"]), case["kv_hi"]) for x in kv], new


def _n_packed(L, R, G):
    return max(L - R, 0) // G * G


def _visible(lo, hi, sinks):
    """Tokens of [0, hi) that are below sinks or at least lo."""
    lo = max(lo, 0)
    return hi - lo + min(sinks, lo)


def work(case):
    kv, new = _lengths(case)
    h, hq, G, R = case["h"], case["hq"], case["G"], case["R"]
    packed = h * (D * (case["kb"] + case["vb"]) / 8 + 8 * D / G)   # bytes of a packed token, all kv heads
    stored = h * D * 2 * 2
    if case["op"] == "evict":
        # the weights and the block table of every sequence that is cut, read and written, and its ring turned
        cut = [L for L in kv if _n_packed(L, R, G) // G > case["keep"]]
        return {"bytes": sum(2 * 8 * -(-L // G) + 2 * stored * (L - _n_packed(L, R, G)) for L in cut) + 8 * len(kv),
                "flops": 0}
    nbytes = flops = 0
    for L, n in zip(kv, new):
        p = _n_packed(L, R, G)
        W, S = case["window"], case["sinks"]
        if case["op"] == "chunk":
            lo = max(0, L - W + 1) if W else 0              # the first query's window
            seen_p, seen = _visible(min(lo, p), p, min(S, p)), _visible(min(lo, L), L, min(S, L))
            nbytes += packed * seen_p + stored * (seen - seen_p) + stored * n + 4 * n * hq * D
            pairs = sum(_visible(i + 1 - W if W else 0, i + 1, S) for i in range(L, L + n))
        else:
            lo = max(0, L - W) if W else 0
            seen_p, seen = _visible(min(lo, p), p, min(S, p)), _visible(lo, L, min(S, L))
            nbytes += packed * seen_p + stored * (seen - seen_p) + (2 + 4) * hq * D
            pairs = seen
            if case["op"] == "weights":
                nbytes += 8 * -(-L // G)
        flops += 4 * D * hq * pairs
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- inputs
def _pack(c, bits):
    """[..., D] integer codes -> [..., D * bits / 8] bytes, lowest bits first."""
    per = 8 // bits
    shift = torch.arange(per, device=c.device, dtype=torch.int32) * bits
    return (c.to(torch.int32).unflatten(-1, (-1, per)) << shift).sum(-1).to(torch.uint8)


def _quantize(x, dim, bits):
    """Codes, scale and zero of x over `dim` (kept, of size one, in scale and zero)."""
    q = (1 << bits) - 1
    mn, mx = x.amin(dim, True), x.amax(dim, True)
    s, z = ((mx - mn) / q).half(), mn.half()
    c = ((x - z.float()) / s.float()).round().clamp(0, q)
    return torch.where(s == 0, torch.zeros_like(c), c), s, z


def prepare(case, seed):
    """A cache in the layout of include/kivi.h (pools of G-token pages and a block table, or one
    run of tokens per sequence and head), the new tokens and the queries of the call.
    Keys are normal with four channels of each head twenty times as large, values normal
    with one token in a hundred ten times as large."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, G, R, h, hq, nseq = TORCH[case["dtype"]], case["G"], case["R"], case["h"], case["hq"], case["nseq"]
    kv, new = _lengths(case)
    ring = R + G
    ngs = [_n_packed(L, R, G) // G for L in kv]
    cap = max(max(ngs), 1) * G + 4 * G                    # packed tokens a sequence has room for
    cg = cap // G

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    out_ch = torch.rand((h, D), generator=gen, device=dev).argsort(-1)[:, :4]
    k_scale_ch = torch.ones((h, D), device=dev).scatter_(1, out_ch, 20.0)

    def keys(*lead):   # [*lead, h, tokens, D] of the storage type
        return (normal(*lead, D) * k_scale_ch[:, None, :]).to(dt)

    def values(*lead):
        burst = torch.rand((*lead, 1), generator=gen, device=dev) < 0.01
        return (normal(*lead, D) * (1 + 9 * burst)).to(dt)

    pages = sum(ngs) + 4 * nseq if case["paged"] else nseq * cg
    k = keys(pages, h, G).float()
    kc, ks, kz = _quantize(k, 2, case["kb"])
    kc = _pack(kc, case["kb"])
    del k
    v = values(pages, h, G).float().unflatten(-1, (D // G, G))
    vc, vs, vz = _quantize(v, -1, case["vb"])
    vc = _pack(vc.flatten(-2), case["vb"])
    del v
    buf = {"k_codes": kc, "k_scale": ks[:, :, 0], "k_zero": kz[:, :, 0], "v_codes": vc, "v_scale": vs[..., 0],
           "v_zero": vz[..., 0]}                          # [pages][h][...]
    if case["paged"]:
        # the pages of each sequence's groups, then four spare ones; entries past its own room name page 0
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        start = torch.tensor([sum(ngs[:b]) + 4 * b for b in range(nseq)], device=dev)
        room = torch.tensor([n + 4 for n in ngs], device=dev)
        j = torch.arange(cg, device=dev)
        table = torch.where(j < room[:, None], order[(start[:, None] + j).clamp(max=pages - 1)], 0)
        buf = {n: t.contiguous() for n, t in buf.items()}
    else:
        table = None
        buf = {n: t.unflatten(0, (nseq, cg)).transpose(1, 2).contiguous() for n, t in buf.items()}  # [nseq][h][cg][..]
        buf = {n: t if n in ("k_scale", "k_zero") else t.flatten(2, 3) for n, t in buf.items()}
    buf = {n: t.view(torch.int16) if t.dtype == torch.float16 else t for n, t in buf.items()}
    buf["k_res"], buf["v_res"] = keys(nseq, h, ring), values(nseq, h, ring)
    s = {"case": dict(case), "buf": buf, "table": table, "cap": cap, "kv": kv, "new": new,
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "chunk":
        n = sum(new)
        # each sequence's new tokens as [h][n][D], one after the other
        s["q"] = normal(n, hq, D).to(dt)
        s["k_new"], s["v_new"] = keys(1, h, n)[0], values(1, h, n)[0]
        at = [sum(new[:b]) for b in range(nseq)]
        kn = [s["k_new"][:, a:a + m].contiguous() for a, m in zip(at, new)]
        vn = [s["v_new"][:, a:a + m].contiguous() for a, m in zip(at, new)]
        s["kn"], s["vn"] = kn, vn
        s["k_ptrs"] = torch.tensor([t.data_ptr() for t in kn], dtype=torch.int64, device=dev)
        s["v_ptrs"] = torch.tensor([t.data_ptr() for t in vn], dtype=torch.int64, device=dev)
        s["n_new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["q_start"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["q"] = normal(nseq, hq, D).to(dt)
        s["out"] = torch.empty((nseq, hq, D), device=dev)
    if case["op"] in ("weights", "evict"):
        # what earlier steps gave: a few groups hold most of it; rounded, so that some are equal
        stride = cg + ring // G + 1
        w = torch.exp(2 * normal(nseq, stride)).bfloat16().float()
        live = torch.tensor([-(-L // G) for L in kv], device=dev)
        s["weights"] = torch.where(torch.arange(stride, device=dev) < live[:, None], w, 0.0)
        s["weights_out"] = torch.empty_like(s["weights"])
    if case["op"] == "evict":
        s["live"] = {"kv_len": s["kv_len"].clone(), "weights": s["weights"].clone(), "table": table.clone(),
                     "k_res": buf["k_res"].clone(), "v_res": buf["v_res"].clone()}
    return s


# ---------------------------------------------------------------- plain forms
def _unpack(rows, bits):
    per = 8 // bits
    shift = torch.arange(per, device=rows.device, dtype=torch.uint8) * bits
    return ((rows[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2).float()


def _tokens(s, pos):
    """Keys and values at positions pos [nseq][P] as [nseq][h][P][D] in 32 bits (any values at
    positions that the sequence does not hold)."""
    c, buf = s["case"], s["buf"]
    G, ring, nseq = c["G"], c["R"] + c["G"], c["nseq"]
    pos = pos.clamp(0, s["cap"] + ring)
    b = torch.arange(nseq, device=pos.device)[:, None]
    pk = pos.clamp(max=s["cap"] - 1)
    half = lambda t: t.view(torch.float16).float()   # noqa: E731
    if c["paged"]:
        page, at = s["table"][b, pk // G].long(), pk % G
        kc, vc = buf["k_codes"][page, :, at], buf["v_codes"][page, :, at]
        ks, kz = half(buf["k_scale"])[page], half(buf["k_zero"])[page]
        vs, vz = half(buf["v_scale"])[page, :, at], half(buf["v_zero"])[page, :, at]
    else:
        kc, vc = buf["k_codes"][b, :, pk], buf["v_codes"][b, :, pk]
        ks, kz = half(buf["k_scale"])[b, :, pk // G], half(buf["k_zero"])[b, :, pk // G]
        vs, vz = half(buf["v_scale"])[b, :, pk], half(buf["v_zero"])[b, :, pk]
    k = _unpack(kc, c["kb"]) * ks + kz                                        # [nseq][P][h][D]
    v = _unpack(vc, c["vb"]).unflatten(-1, (D // G, G)) * vs[..., None] + vz[..., None]
    k, v = k.transpose(1, 2), v.flatten(-2).transpose(1, 2)
    n_packed = ((s["kv_len"] - c["R"]).clamp(min=0) // G * G)[:, None]
    stored = (pos >= n_packed)[:, None, :, None]
    kr, vr = buf["k_res"][b, :, pos % ring], buf["v_res"][b, :, pos % ring]
    return torch.where(stored, kr.float().transpose(1, 2), k), torch.where(stored, vr.float().transpose(1, 2), v)


def _softmax(x):
    m = x.amax(-1, True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, True)
    return e / torch.where(t == 0, 1.0, t)


def _plain_decode(s):
    c = s["case"]
    h, g, L = c["h"], c["hq"] // c["h"], s["kv_len"].long()[:, None]
    top = max(s["kv"])
    if c["op"] == "window" and c["sinks"] + c["window"] < top:
        first = torch.arange(c["sinks"], device=L.device).expand(c["nseq"], -1)
        last = L - c["window"] + torch.arange(c["window"], device=L.device)
        pos = torch.cat([first, last], 1)
        ok = torch.cat([first < L, last >= c["sinks"]], 1)
    else:
        pos = torch.arange(top, device=L.device).expand(c["nseq"], -1)
        ok = pos < L
        if c["op"] == "window":
            ok = ok & ((pos >= L - c["window"]) | (pos < c["sinks"]))
    k, v = _tokens(s, pos)
    q = s["q"].float().unflatten(1, (h, g))
    p = _softmax((q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~ok[:, None, None], -math.inf))
    out = (p @ v).flatten(1, 2)
    if c["op"] == "window":
        return out
    stride, G = s["weights"].shape[1], c["G"]
    w = torch.nn.functional.pad(p.sum((1, 2)), (0, stride * G - top)).unflatten(-1, (stride, G)).sum(-1)
    live = torch.arange(stride, device=L.device) < (L + G - 1) // G
    return out, torch.where(live, c["decay"] * s["weights"] + w, 0.0)


def _plain_chunk(s):
    c = s["case"]
    nseq, h, g = c["nseq"], c["h"], c["hq"] // c["h"]
    L, n = s["kv_len"].long()[:, None], s["n_new"].long()[:, None]
    top, most, dev = max(s["kv"]), max(s["new"]), s["q"].device
    i = torch.arange(most, device=dev).expand(nseq, -1)
    row = (s["q_start"].long()[:, None] + i.minimum(n - 1)).clamp(min=0)     # this query's row of q
    q = s["q"].float()[row].unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [nseq][h][most g][D]
    pos = torch.arange(top, device=dev).expand(nseq, -1)
    k, v = _tokens(s, pos)
    k = torch.cat([k, s["k_new"].float()[:, row].transpose(0, 1)], 2)
    v = torch.cat([v, s["v_new"].float()[:, row].transpose(0, 1)], 2)
    at = torch.cat([pos, L + i], 1)[:, None]                                # position of each key
    held = torch.cat([pos < L, i < n], 1)[:, None]
    own_at = (L + i)[..., None]                                             # and of each query
    ok = held & (at <= own_at)
    if c["window"]:
        ok = ok & ((at > own_at - c["window"]) | (at < c["sinks"]))
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (most, g))
    x.masked_fill_(~ok[:, None, :, None], -math.inf)
    out = (_softmax(x).flatten(2, 3) @ v).unflatten(2, (most, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out[i < n].to(s["q"].dtype)


def _plain_evict(s):
    c = s["case"]
    G, R, ring = c["G"], c["R"], c["R"] + c["G"]
    w, L, dev = s["weights"], s["kv_len"].long(), s["q"].device
    stride, cg = w.shape[1], s["cap"] // G
    ng = (L - R).clamp(min=0) // G
    j = torch.arange(stride, device=dev)
    keep = torch.where(ng > c["keep"], torch.full_like(ng, c["keep"]), ng)[:, None]
    packed = j < ng[:, None]
    held = packed & ((j < c["sink_groups"]) | (j >= ng[:, None] - c["recent_groups"]))
    rank = torch.where(held, math.inf, torch.where(packed, w, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(packed).scatter_(1, order, j < keep) & packed
    gone = packed & ~kept
    # kept groups, then groups that are not packed, then dropped ones, each in their order
    last = torch.where(gone, 1, 0).argsort(dim=1, stable=True)
    m = gone.sum(1)
    weights = torch.where(j < stride - m[:, None], w.gather(1, last), 0.0)
    jt = torch.arange(cg, device=dev)
    kind = torch.where(kept, 0, torch.where(gone, 1, 2))[:, :cg].argsort(dim=1, stable=True)
    table = s["table"].gather(1, kind)
    kv = L - m * G
    slot = (torch.arange(ring, device=dev) + (m * G)[:, None]) % ring        # the slot each ring row comes from
    b = torch.arange(c["nseq"], device=dev)[:, None]
    return {"kv_len": kv.to(torch.int32), "weights": weights, "table": table,
            "k_res": s["buf"]["k_res"][b, :, slot].transpose(1, 2), "v_res": s["buf"]["v_res"][b, :, slot].transpose(1, 2)}


# ---------------------------------------------------------------- the framework's calls
def _cache(s):
    """The handle a serving program keeps: the package's cache over the buffers of the state."""
    if "cache" not in s:
        import bit_asymmetric_kv_kivi_gb300 as kivi
        c = s["case"]
        cfg = kivi.Config(k_bits=c["kb"], v_bits=c["vb"], head_dim=D, num_q_heads=c["hq"], num_kv_heads=c["h"],
                          dtype=kivi.F16 if c["dtype"] == "f16" else kivi.BF16, residual=c["R"], group=c["G"])
        buf, live = dict(s["buf"]), s.get("live")
        if live:
            buf["k_res"], buf["v_res"] = live["k_res"], live["v_res"]
        s["cache"] = kivi.KVCache.from_buffers(cfg, buf, live["kv_len"] if live else s["kv_len"], s["cap"],
                                               block_tables=live["table"] if live else s["table"],
                                               max_len=max(s["kv"]))
    return s["cache"]


def _own(s):
    c, cache = s["case"], _cache(s)
    if c["op"] == "window":
        return cache.decode_window(s["q"], c["window"], c["sinks"], out=s["out"], softmax_scale=s["scale"])
    if c["op"] == "weights":
        return cache.decode_weights(s["q"], s["weights"], s["weights_out"], decay=c["decay"], out=s["out"],
                                    softmax_scale=s["scale"])
    if c["op"] == "chunk":
        return cache.chunk_attn(s["q"], s["q_start"], s["k_ptrs"], s["v_ptrs"], s["n_new"], c["new_hi"],
                                out=s["out"], window=c["window"], sinks=c["sinks"], softmax_scale=s["scale"])
    # eviction changes the cache in place: every pass starts from the state as it was
    live = s["live"]
    live["kv_len"].copy_(s["kv_len"])
    live["weights"].copy_(s["weights"])
    live["table"].copy_(s["table"])
    live["k_res"].copy_(s["buf"]["k_res"])
    live["v_res"].copy_(s["buf"]["v_res"])
    cache.evict(live["weights"], c["keep"], sink_groups=c["sink_groups"], recent_groups=c["recent_groups"])
    return live


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_chunk(state) if op == "chunk" else _plain_evict(state) if op == "evict" else _plain_decode(state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The same outputs in 64 bits, sequence by sequence, from the definitions at the top."""
    s = prepare(case, seed)
    kv, new = _lengths(case)
    G, R, h, g = case["G"], case["R"], case["h"], case["hq"] // case["h"]
    f8, buf, dev = torch.float64, s["buf"], s["q"].device
    pairs = sum((L + n) * max(n, 1) for L, n in zip(kv, new)) * case["hq"]
    if pairs * D * 4 > 3e12:
        return None
    if case["op"] == "evict":
        # every output is moved, none is computed
        return None
    outs, rows, stride = [], [], s["weights"].shape[1] if "weights" in s else 0
    for b, (L, n) in enumerate(zip(kv, new)):
        np_, ng = _n_packed(L, R, G), _n_packed(L, R, G) // G
        part = {}
        for name in ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero"):
            if case["paged"]:
                t = buf[name][s["table"][b, :ng].long()].transpose(0, 1)      # [h][groups][...]
            else:
                t = buf[name][b]
                t = t[:, :ng] if name in ("k_scale", "k_zero") else t[:, :np_].unflatten(1, (ng, G)) if ng else t[:, :0]
            part[name] = (t if t.dtype == torch.uint8 else t.view(torch.float16).to(f8)).reshape(
                (h, ng, D) if name in ("k_scale", "k_zero") else (h, ng * G, -1) if ng else (h, 0, t.shape[-1]))
        code = {}
        for name, bits in (("k_codes", case["kb"]), ("v_codes", case["vb"])):
            byte, ch = part[name].to(torch.int64), torch.arange(D, device=dev)
            code[name] = ((byte[..., ch * bits // 8] >> (ch * bits % 8)) % (1 << bits)).to(f8)
        k = code["k_codes"] * part["k_scale"].repeat_interleave(G, 1) + part["k_zero"].repeat_interleave(G, 1)
        v = (code["v_codes"] * part["v_scale"].repeat_interleave(G, 2) + part["v_zero"].repeat_interleave(G, 2))
        tail = torch.arange(np_, L, device=dev) % (R + G)
        k = torch.cat([k, buf["k_res"][b][:, tail].to(f8)], 1)
        v = torch.cat([v, buf["v_res"][b][:, tail].to(f8)], 1)
        nq = 1
        if case["op"] == "chunk":
            k, v, nq = torch.cat([k, s["kn"][b].to(f8)], 1), torch.cat([v, s["vn"][b].to(f8)], 1), n
            a = sum(new[:b])
            q = s["q"][a:a + n].to(f8)
        else:
            q = s["q"][b:b + 1].to(f8)
        T = k.shape[1]
        t, p = torch.arange(T, device=dev)[None], torch.arange(T - nq, T, device=dev)[:, None]
        see = t <= p
        if case["window"]:
            see &= (p - t < case["window"]) | (t < case["sinks"])
        out = torch.empty((nq, case["hq"], D), dtype=f8, device=dev)
        total = torch.zeros(T, dtype=f8, device=dev)
        for hh in range(h):
            x = torch.einsum("ngd,td->gnt", q[:, hh * g:(hh + 1) * g], k[hh]) / math.sqrt(D)
            x = torch.where(see, x, -math.inf)
            x = torch.exp(x - x.amax(-1, True))
            x /= x.sum(-1, True)
            out[:, hh * g:(hh + 1) * g] = (x @ v[hh]).transpose(0, 1)
            if case["op"] == "weights":
                total += x.sum((0, 1))
        outs.append(out)
        if case["op"] == "weights":
            row = torch.zeros(stride, dtype=f8, device=dev)
            at = torch.arange(T, device=dev) // G
            row.index_add_(0, at, total)
            live = -(-L // G)
            row[:live] += case["decay"] * s["weights"][b, :live].to(f8)
            rows.append(row)
    out = torch.cat(outs)
    return (out, torch.stack(rows)) if case["op"] == "weights" else out
