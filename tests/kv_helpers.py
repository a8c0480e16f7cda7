"""Plain restatement of the 4-bit key/value cache for the tests: the byte places
of an atom from their formulas, the block quantizer from the oracle's codecs,
and attention in float64."""
import numpy as np
import torch

import oracle

LN2 = float(np.log(2.0))


def places(D):
    """Byte places in an atom: (k_codes [16, D/2], v_codes [16, D/2], k_scales [16, D/16], v_scales [16, D/16])."""
    n, w = D // 64, max(1, D // 128)
    kc, vc = np.zeros((16, D // 2), np.int64), np.zeros((16, D // 2), np.int64)
    ks, vs = np.zeros((16, D // 16), np.int64), np.zeros((16, D // 16), np.int64)
    for t in range(16):
        i, j = 2 * (t // 8) + t % 2, (t // 2) % 4
        for y in range(D // 2):
            b = y // 8
            s, lane = (t // 8) * n + b % n, 4 * (t % 8) + b // n
            kc[t, y] = (s // 2) * 512 + 16 * lane + 8 * (s % 2) + y % 8
            r, x = y // (D // 16), i * (D // 16) + y % (D // 16)
            vc[t, y] = 8 * D + (x // 16) * 512 + 16 * (4 * r + j) + x % 16
        for b in range(D // 16):
            s, lane = (t // 8) * n + b % n, 4 * (t % 8) + b // n
            ks[t, b] = 16 * D + 2 * n * lane + s
            vs[t, b] = 17 * D + 4 * w * (4 * (b // w) + j) + i * w + b % w
    return kc, vc, ks, vs


def quantize(x, g):
    """(packed codes uint8 [..., D/2], scales uint8 [..., D/16]) of float32 x [..., D]; the roundings of the contract."""
    x = np.ascontiguousarray(x, np.float32)
    D = x.shape[-1]
    b = x.reshape(-1, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        amax = np.fmax.reduce(np.abs(b), axis=-1, initial=np.float32(0))
        sf = oracle.e4m3_encode((amax / np.float32(6)) / g)
        step = (oracle.e4m3_decode(sf) * g).astype(np.float32)
        mult = np.where(step == 0, np.float32(0), np.float32(1) / step).astype(np.float32)
        codes = oracle.e2m1_encode((b * mult[:, None]).astype(np.float32).reshape(-1)).reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sf.reshape(*x.shape[:-1], D // 16)


def write(cache, slots, k, v, gk, gv, D, page):
    """Append in numpy: cache uint8 [pages, H, page * D * 9 / 8], k and v float32 [T, H, D]."""
    kc_at, vc_at, ks_at, vs_at = places(D)
    kc, ks = quantize(k, gk)
    vc, vs = quantize(v, gv)
    for n, slot in enumerate(np.asarray(slots)):
        if slot < 0:
            continue
        p, t = divmod(int(slot), page)
        base, t = (t // 16) * 18 * D, t % 16
        for h in range(k.shape[1]):
            row = cache[p, h]
            row[base + kc_at[t]] = kc[n, h]
            row[base + vc_at[t]] = vc[n, h]
            row[base + ks_at[t]] = ks[n, h]
            row[base + vs_at[t]] = vs[n, h]


def decode(cache, D, page):
    """float64 (k, v) [pages, page, H, D] of a cache (torch uint8, any device), without the global scales."""
    dev = cache.device
    pages, H, _ = cache.shape
    atoms = cache.reshape(pages, H, page // 16, 18 * D)
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev)
    e4m3 = torch.from_numpy(oracle.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)).to(dev)
    out = []
    kc, vc, ks, vs = (torch.from_numpy(a).to(dev) for a in places(D))
    for c_at, s_at in ((kc, ks), (vc, vs)):
        c = atoms[..., c_at].long()
        x = torch.stack([e2m1[c & 15], e2m1[c >> 4]], -1).flatten(-2)
        s = e4m3[atoms[..., s_at].long()]
        x = x * s.repeat_interleave(16, -1)
        out.append(x.permute(0, 2, 3, 1, 4).reshape(pages, page, H, D))
    return out


def attention(q, k, v, gk, gv, table, kv_lens, cu, page, scale, window=0, causal=True):
    """float64 (out, lse, bound on |out - exact|, bound on |lse - exact|) of the
    library's contract; q bf16 [T, Hq, D], k and v from `decode`.

    The bounds count the roundings of the contract: the output's to bf16 (half a
    step, 2^-8), the weights' to f16 (2^-11, and 2^-25 below f16's normal
    range, where the largest weight is at least 1), float32 products and sums
    (D steps of 2^-23 in a score, which also covers an accumulation that
    truncates), the scaled score's and its difference's (2^-23 of it each) and the
    exponential's (2^-22); sums over n keys lose n * 2^-23."""
    T, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        c0, c1, n = int(cu[b]), int(cu[b + 1]), int(kv_lens[b])
        if c1 == c0 or n == 0:
            continue
        key = torch.arange(n, device=q.device)
        pages = table[b, : -(-n // page)].long()
        kb = k[pages].reshape(-1, k.shape[2], D)[:n].repeat_interleave(G, 1)  # n, Hq, D
        vb = v[pages].reshape(-1, v.shape[2], D)[:n].repeat_interleave(G, 1)
        qb = q[c0:c1].double()
        pos = torch.arange(n - (c1 - c0), n, device=q.device)[:, None]
        see = torch.ones(c1 - c0, n, dtype=torch.bool, device=q.device)
        if causal:
            see &= key <= pos
        if window:
            see &= key > pos - window
        s = torch.einsum("ihd,jhd->hij", qb, kb) * (scale * gk)
        mag = torch.einsum("ihd,jhd->hij", qb.abs(), kb.abs()) * abs(scale * gk)
        s = s.masked_fill(~see, -float("inf"))
        mag = mag.masked_fill(~see, 0.0).amax(-1)  # h, i
        some = see.any(-1)
        p = torch.where(some[None, :, None], torch.softmax(s, -1), 0.0)
        p = torch.nan_to_num(p, nan=0.0)
        o = torch.einsum("hij,jhd->ihd", p, vb) * gv
        a = torch.einsum("hij,jhd->ihd", p, vb.abs()) * abs(gv)
        worst = torch.where(see, s, 0.0).abs().amax(-1)
        eps = (D * 2.0**-23 * mag + 2 * 2.0**-23 * worst) + 2.0**-22  # relative error of a weight
        few = 2.0**-25 * (see.double() @ vb.abs().transpose(0, 1)).transpose(0, 1) * abs(gv)  # i, h, d
        err = a * (2.0**-11 + 2 * eps + 2 * n * 2.0**-23).T[..., None] + few
        out[c0:c1] = o
        tol[c0:c1] = 2.0**-8 * (o.abs() + err) + err
        lse[c0:c1] = torch.logsumexp(s, -1).T
        tol_lse[c0:c1] = (eps + n * 2.0**-23).T + 2.0**-22 * (1 + torch.nan_to_num(lse[c0:c1], neginf=0.0).abs())
    return out, lse, tol, tol_lse


def plan(cached, new, table, free, head, T, page):
    """nq_kv_plan in plain Python for lengths that fit: (cu, kv_lens, positions, slots, head); fills `table`."""
    cu, pos, slots = [0], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        for i in range(-(-c // page), -(-(c + n) // page)):
            table[b, i] = free[head] if head < len(free) else -1
            head += 1
        for i in range(n):
            p = int(table[b, (c + i) // page])
            pos.append(c + i)
            slots.append(p * page + (c + i) % page if p >= 0 else -1)
        cu.append(cu[-1] + n)
    pos += [-1] * (T - len(pos))
    slots += [-1] * (T - len(slots))
    return (np.array(cu, np.int32), np.array([c + n for c, n in zip(cached, new)], np.int32), np.array(pos, np.int32),
            np.array(slots, np.int64), head)
