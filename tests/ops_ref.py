"""Plain 64-bit statements of the operators over the packed cache, on the oracle's sequence
caches (oracle.SeqCache), and the error bounds their tests use."""
import numpy as np

import oracle


def widen(bits: np.ndarray, dtype: int) -> np.ndarray:
    if dtype == oracle.F16:
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def unpack(rows: np.ndarray, bits: int) -> np.ndarray:
    d = np.arange(rows.shape[-1] * 8 // bits)
    return (rows[..., d * bits // 8].astype(np.int64) >> (d * bits % 8)) & ((1 << bits) - 1)


def dense(ref: "oracle.SeqCache"):
    """Keys and values of the cached tokens, [H][L][D] in 64 bits, and the magnitudes |c s| + |z| of
    what the kernels add up to form them (the stored value's own where it is not packed)."""
    c, L = ref.cfg, ref.L
    P, G, ring = oracle.n_packed(c, L), c.group, c.ring
    ks, kz = (np.repeat(widen(x[:, :P // G], oracle.F16), G, 1) for x in (ref.k_scale, ref.k_zero))
    vs, vz = (np.repeat(widen(x[:, :P], oracle.F16), G, 2) for x in (ref.v_scale, ref.v_zero))
    kc, vc = unpack(ref.k_codes[:, :P], c.k_bits) * ks, unpack(ref.v_codes[:, :P], c.v_bits) * vs
    slots = np.arange(P, L) % ring
    kr, vr = widen(ref.k_res[:, slots], c.dtype), widen(ref.v_res[:, slots], c.dtype)
    cat = lambda a, b: np.concatenate([a, b], 1)   # noqa: E731
    return cat(kc + kz, kr), cat(vc + vz, vr), cat(np.abs(kc) + np.abs(kz), np.abs(kr)), cat(np.abs(vc) + np.abs(vz), np.abs(vr))


def attend(q, k, v, see, scale):
    """q [n][Hq][D], k and v [H][T][D], see [n][T] -> out [n][Hq][D], p [n][Hq][T]; zeros where nothing is seen."""
    g = q.shape[1] // k.shape[0]
    kh, vh = np.repeat(k, g, 0), np.repeat(v, g, 0)
    x = np.einsum("nhd,htd->nht", q, kh) * scale
    x = np.where(see[:, None, :], x, -np.inf)
    m = x.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(x - np.where(np.isfinite(m), m, 0))
    t = e.sum(-1, keepdims=True)
    p = e / np.where(t == 0, 1, t)
    return np.einsum("nht,htd->nhd", p, vh), p


def visible(L, n, window, sinks):
    """[n][L + n'] mask: query i at position L - n + i of the L keys sees t <= its position, within window and sinks."""
    t, pos = np.arange(L)[None], np.arange(L - n, L)[:, None]
    see = t <= pos
    if window:
        see &= (t > pos - window) | (t < sinks)
    return see


# Bounds of the fp32 decode kernels. Scores: 128 products of f16 hi + lo operands (2^-22 of each
# product) are added by about twenty truncating tensor-core steps, 2^-23 of the partial sum
# each, so a score is off by at most 2^-18 of A = scale * sum_d |q_d| (|c s| + |z|), and its weight by
# about that much, relative; normalising doubles it. Values: the same operands (2^-21), a few
# truncating steps per tile, and one rounding (2^-24) per tile of a warp's share of the
# stream, under 2^7 here: 2^-17 of sum_t p_t (|c s| + |z|) in all.
def decode_bounds(q, kmag, vmag, p, scale):
    """Bounds for out [n][Hq][D] and, relative, for the weights [n][Hq][1]."""
    g = q.shape[1] // kmag.shape[0]
    a = scale * np.einsum("nhd,htd->nht", np.abs(q), np.repeat(kmag, g, 0)).max(-1, initial=0.0)
    rel = 2 * 2.0 ** -18 * a[..., None] + 2.0 ** -17
    return rel * np.einsum("nht,htd->nhd", p, np.repeat(vmag, g, 0)) + 1e-30, rel


def evict(cfg, weights, L, keep, sink, recent):
    """Kept groups in order, dropped groups in order, the new weights row and the ring turn."""
    P = oracle.n_packed(cfg, L)
    ng = P // cfg.group
    if ng <= keep:
        return list(range(ng)), [], weights.copy(), 0
    held = set(range(sink)) | set(range(ng - recent, ng))
    rank = sorted((j for j in range(ng) if j not in held),
                  key=lambda j: (-weights[j] if weights[j] == weights[j] else np.inf, j))
    kept = sorted(held | set(rank[:keep - len(held)]))
    gone = [j for j in range(ng) if j not in set(kept)]
    out = np.zeros_like(weights)
    rest = weights[ng:]
    out[:keep] = weights[kept]
    out[keep:keep + len(rest)] = rest
    return kept, gone, out, len(gone) * cfg.group


# Bounds of chunk attention. A packed key is rounded by key_step of its group's largest level (one f16
# number with bf16 storage: 2^-11; two f16 parts with fp16 storage: 2^-16, see KEY_STEP), so a score
# is off by at most that of A = scale * sum_d |q_d| (|c s| + |z|) (fp32 steps: 2^-18 of it, as above), its weight by as
# much and the normalised weight by twice that; probabilities and dequantized values add 2^-11 each, the
# fp32 steps 2^-12, and the output is rounded once to its type. Errors of different tokens and
# channels are independent, so in the 2-norm each factor counts by its root mean square: a
# rounding of half step h has rms h / sqrt(3).
KEY_STEP = {oracle.F16: 2.0 ** -16, oracle.BF16: 2.0 ** -11}


def chunk_bounds(q, k, v, p, want, scale, half_step, key_step, kmag):
    """(bound per output element, bound of the relative 2-norm of the whole output); kmag: |c s| + |z| of each key."""
    g = q.shape[1] // k.shape[0]
    kh, vh = np.repeat(kmag, g, 0), np.repeat(v, g, 0)
    h = 2.0 ** -11
    a = scale * np.einsum("nhd,htd->nht", np.abs(q), kh).max(-1, initial=0.0)[..., None]
    el = (2 * (key_step + 2.0 ** -18) * a + 2 * h + 2.0 ** -12) * np.einsum("nht,htd->nhd", p, np.abs(vh)) + half_step * np.abs(want) + 1e-7
    rms = key_step * scale * np.sqrt(np.einsum("nhd,htd->nht", q * q, kh * kh)).max(-1, initial=0.0)
    rel = np.sqrt((2 * (2 * rms.max(initial=0.0) ** 2 + 2 * h * h) + half_step ** 2) / 3) + 2.0 ** -12
    return el, 2 * rel
