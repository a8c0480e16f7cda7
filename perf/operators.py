"""Timed cases of the 4-bit key/value cache: block tables and slots from request lengths, the quantizing append, the
gather that reads tokens back, and attention over the cache.

Every case names its operator in "op".  ``run`` takes a prepared state through the operator's plain form (elementary
torch operations) where ``own`` is false, and through the library's calls where it is true.

Cache layout (see include/nq.h): uint8 [pages, kv heads, page / 16 * 18 * D].  16 tokens of one kv head form an atom of
18 * D bytes: the key codes (8 D), the value codes (8 D), the key scales (D), the value scales (D), each in the order in
which the 32 lanes of a warp take them into a 16 x 8 x 16 matrix product.
"""
import random

import torch

own = False

E2M1_MAX = 6.0
E4M3_MAX = 448.0
# What a serving program sets aside once for attention's partial results, zero-filled.
WORKSPACE_BYTES = 64 << 20


# ------------------------------------------------------------------------------------------------ the cases ----
def listed():
    return [
        # One decode step of a mid-size batch: every request grows by a token, some of them into a new page.
        dict(name="plan_decode", op="plan", requests=64, new=1, cached=8000, page=16, ragged=True),
        # A large scheduler step: thousands of requests, prompt chunks among single tokens.
        dict(name="plan_step", op="plan", requests=2048, new=63, cached=4000, page=64, ragged=True),
        # The keys and values of one decode step, sliced out of the fused projection's output.
        dict(name="append_decode", op="append", tokens=64, kv_heads=8, heads=32, d=128, page=64, pad=0),
        # A prompt batch of odd length with padding tokens behind it.
        dict(name="append_prompt", op="append", tokens=16389, kv_heads=8, heads=32, d=128, page=16, pad=59),
        # A shared prefix read back for a full-precision pass: short, small heads.
        dict(name="gather_prefix", op="gather", tokens=777, kv_heads=4, d=64, page=16),
        # A long document's keys and values read back.
        dict(name="gather_long", op="gather", tokens=65536, kv_heads=8, d=128, page=64),
        # Latency: a single request with a short context.
        dict(name="decode_short", op="attention", requests=1, new=1, kv=512, heads=32, kv_heads=8, d=128, page=16,
             window=0, ragged=False, lse=False),
        # An ordinary serving batch of ragged contexts.
        dict(name="decode_batch", op="attention", requests=128, new=1, kv=8192, heads=32, kv_heads=8, d=128, page=64,
             window=0, ragged=True, lse=False),
        # Two very long contexts: the key axis has to be split over the whole GPU.
        dict(name="decode_long", op="attention", requests=2, new=1, kv=131071, heads=64, kv_heads=8, d=128, page=128,
             window=0, ragged=False, lse=False),
        # Draft verification, a few tokens a request, under a sliding window, log-sum-exp kept.
        dict(name="verify_window", op="attention", requests=48, new=4, kv=6000, heads=64, kv_heads=8, d=64, page=32,
             window=1024, ragged=True, lse=True),
        # A whole prompt at once.
        dict(name="prompt_8k", op="attention", requests=1, new=8192, kv=8192, heads=32, kv_heads=8, d=128, page=64,
             window=0, ragged=False, lse=False),
        # A mixed step: prompt chunks of ragged length behind cached prefixes, wide heads.
        dict(name="chunks_mixed", op="attention", requests=20, new=1000, kv=4100, heads=16, kv_heads=8, d=256, page=32,
             window=0, ragged=True, lse=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op=op, requests=_log(rng, 1, 2048), new=_log(rng, 1, 63), cached=_log(rng, 1, 8000), page=page,
                    ragged=rng.random() < 0.8)
    d = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16000), kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 4, 8]), d=d,
                    page=page, pad=rng.choice([0, 0, 7, 61]))
    if op == "gather":
        return dict(op=op, tokens=_log(rng, 1, 16000), kv_heads=kv_heads, d=d, page=page)
    group = rng.choice([1, 2, 4, 5, 8, 16])
    case = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, d=d, page=page, ragged=rng.random() < 0.7,
                lse=rng.random() < 0.5)
    if rng.random() < 0.5:  # single tokens, or a few of them
        case.update(requests=_log(rng, 1, 128), new=rng.choice([1, 1, 1, 2, 4, 7]))
        case.update(kv=_log(rng, 16, max(16, min(65536, (1 << 29) // (case["requests"] * kv_heads * d)))))
    else:  # prompts, no dearer than the longest listed one
        case.update(requests=_log(rng, 1, 16))
        most = (1 << 37) // (case["requests"] * case["heads"] * d)  # new * kv
        case.update(new=_log(rng, 9, min(3000, int(most ** 0.5) - 1)))
        case.update(kv=case["new"] + _log(rng, 1, min(8000, most // case["new"] - case["new"])))
    case.update(window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    return case


def _lens(case):
    """(new tokens, total length) of each request: a function of the case alone."""
    B, new = case["requests"], case["new"]
    r = random.Random("lens %d %d" % (B, new))
    total = case["cached"] + new if case["op"] == "plan" else max(case["kv"], new)
    n, t = [], []
    for b in range(B):
        if not case["ragged"] or b == 0:  # the first request has the full lengths
            n.append(new)
            t.append(total)
        elif case["op"] == "attention":
            n.append(r.randint(1, new))
            t.append(n[-1] + r.randint(0, total - new))
        else:  # a step's requests: mostly single tokens, some prompts
            n.append(new if new == 1 else r.choice([1, 1, r.randint(0, 2 * new), 2 * new]))
            t.append(n[-1] + r.randint(0, total - new))
    return n, t


def _pairs(case):
    """(row, key) pairs one head computes, and the tokens a kv head reads, over all requests."""
    pairs = tokens = 0
    w = case["window"]
    for n, t in zip(*_lens(case)):
        c = t - n  # keys before the first new token
        if w == 0:
            pairs += n * c + n * (n + 1) // 2
            tokens += t
        else:
            full = max(0, t - max(c, w - 1))  # rows that see a whole window
            part = n - full
            pairs += full * w + part * c + part * (part + 1) // 2
            tokens += t - max(0, c - w + 1)
    return pairs, tokens


def work(case):
    if case["op"] == "plan":
        n, t = _lens(case)
        P = case["page"]
        pages = sum(-(-b // P) - -(-(b - a) // P) for a, b in zip(n, t))
        return {"bytes": 8 * len(n) + 4 + 4 * pages + 4 * (2 * len(n) + 2) + 12 * sum(n) + 4 * pages, "flops": 0}
    if case["op"] in ("append", "gather"):
        x = case["tokens"] * case["kv_heads"] * case["d"]
        # append: bf16 keys and values in, codes and scales out, and the values that they stand for read back
        return {"bytes": (8 + 1.125 if case["op"] == "append" else 4 + 1.125) * x + 8 * case["tokens"], "flops": 0}
    pairs, tokens = _pairs(case)
    rows = sum(_lens(case)[0]) * case["heads"]
    return {"bytes": 1.125 * tokens * case["kv_heads"] * case["d"] + 4 * rows * case["d"] + (4 * rows if case["lse"] else 0),
            "flops": 4 * case["d"] * case["heads"] * pairs}


# ------------------------------------------------------------------------------------- the format, in torch ----
def _encode(x, g):
    """Codes (uint8, one per element) and block scales (uint8 e4m3) of float32 x [..., D] under the global scale g."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1, keepdim=True)
    six = torch.full_like(g, E2M1_MAX)  # a tensor: division by a number would multiply by its rounded reciprocal
    sf = ((amax / six) / g).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    step = sf.float() * g
    t = blocks * torch.where(step == 0, torch.zeros_like(step), 1.0 / step)
    a = t.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(t).to(torch.uint8) * 8
    return code.flatten(-2), sf.squeeze(-1).view(torch.uint8)


def _decode(code, sf):
    """float32 e2m1 * block scale of codes [..., D] (uint8, one per element) and scales [..., D / 16]."""
    mag = (code & 7).to(torch.int32)
    bits = (((mag >> 1) + 126) << 23) | ((mag & 1) << 22)
    v = torch.where(mag < 2, mag * 0.5, bits.view(torch.float32))
    v = torch.where(code >= 8, -v, v)
    return (v.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _pack(kc, ks, vc, vs):
    """Atoms [..., 18 D] of codes [..., 16 tokens, D] and scales [..., 16, D / 16] of the keys and the values."""
    lead, D = kc.shape[:-2], kc.shape[-1]
    n = D // 64
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(-1, 2, 8, 4, n, 8)  # e, r, j, c, byte
    kb = kb.permute(0, 1, 4, 2, 3, 5).reshape(-1, n, 2, 8, 4, 8).permute(0, 1, 3, 4, 2, 5)  # plane, r, j, half, byte
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(-1, 2, 4, 2, 8, D // 16)  # i1, j, i0, r, byte
    vb = vb.permute(0, 4, 2, 1, 3, 5).reshape(-1, 8, 4, n, 16).permute(0, 3, 1, 2, 4)  # plane, r, j, byte
    kp = ks.reshape(-1, 2, 8, 4, n).permute(0, 2, 3, 1, 4)  # r, j, e, c
    w = max(1, D // 128)  # blocks of a lane
    vp = vs.reshape(-1, 2, 4, 2, D // 16 // w, w).permute(0, 4, 2, 1, 3, 5)  # r (or pairs of r), j, i1, i0, block
    return torch.cat([x.reshape(*lead, -1) for x in (kb, vb, kp, vp)], -1)


def _unpack(atoms):
    """The inverse of _pack: (kc, ks, vc, vs)."""
    lead, D = atoms.shape[:-1], atoms.shape[-1] // 18
    n, w = D // 64, max(1, D // 128)
    kb, vb, kp, vp = atoms.split([8 * D, 8 * D, D, D], -1)
    kb = kb.reshape(-1, n, 8, 4, 2, 8).permute(0, 1, 4, 2, 3, 5).reshape(-1, 2, n, 8, 4, 8).permute(0, 1, 3, 4, 2, 5)
    vb = vb.reshape(-1, n, 8, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1, 8, 4, 2, 2, D // 16).permute(0, 3, 2, 4, 1, 5)
    ks = kp.reshape(-1, 8, 4, 2, n).permute(0, 3, 1, 2, 4).reshape(*lead, 16, D // 16)
    vs = vp.reshape(-1, D // 16 // w, 4, 2, 2, w).permute(0, 3, 2, 4, 1, 5).reshape(*lead, 16, D // 16)
    kb, vb = kb.reshape(*lead, 16, D // 2), vb.reshape(*lead, 16, D // 2)
    kc = torch.stack([kb & 15, kb >> 4], -1).flatten(-2)
    vc = torch.stack([vb & 15, vb >> 4], -1).flatten(-2)
    return kc, ks, vc, vs


def _global_scale(x):
    """float32 [1]: the largest value maps to the largest code under the largest block scale."""
    return (x.float().abs().amax() / (E2M1_MAX * E4M3_MAX)).reshape(1)


def _random_cache(gen, pages, kv_heads, d, page, dev):
    """A cache whose every slot holds a token, as a server's does after a while, and its global scales."""
    def values():
        x = torch.randn(pages * (page // 16), kv_heads, 16, d, generator=gen, device=dev, dtype=torch.bfloat16)
        return x
    k, v = values(), values()
    k[..., 3::32] *= 4  # keys have a few large channels
    gk, gv = _global_scale(k), _global_scale(v)
    kc, ks = _encode(k.float(), gk)
    del k
    vc, vs = _encode(v.float(), gv)
    del v
    atoms = _pack(kc, ks, vc, vs)  # pages * page / 16, kv_heads, 18 d
    cache = atoms.reshape(pages, page // 16, kv_heads, 18 * d).transpose(1, 2).reshape(pages, kv_heads, -1)
    return cache.contiguous(), gk, gv


# ------------------------------------------------------------------------------------------------- prepare ----
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    P = case["page"]
    if case["op"] == "plan":
        n, t = _lens(case)
        new = torch.tensor(n, dtype=torch.int32, device=dev)
        cached = torch.tensor(t, dtype=torch.int32, device=dev) - new
        have = (cached + P - 1) // P
        width = max(-(-x // P) for x in t) + 1
        used = int(have.sum())
        total = sum(-(-x // P) for x in t) + 64
        ids = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
        table = torch.full((len(n), width), -1, dtype=torch.int32, device=dev)
        at = torch.arange(width, device=dev)[None, :] < have[:, None]
        table[at] = ids[:used]
        return dict(case=case, tokens=sum(n), new=new, cached=cached, table=table, free=ids[used:].contiguous(),
                    head=torch.tensor([3], dtype=torch.int32, device=dev))
    H, d = case["kv_heads"], case["d"]
    if case["op"] in ("append", "gather"):
        T = case["tokens"]
        pages = -(-T // P) + 3
        cache, gk, gv = _random_cache(gen, pages, H, d, P, dev)
        slots = torch.randperm(pages * P, generator=gen, device=dev)[:T].to(torch.int64)
        if T > 1:  # runs of tokens share a page, as a prompt's do
            at = torch.randperm(pages, generator=gen, device=dev).to(torch.int64)
            slots = (at[:, None] * P + torch.arange(P, device=dev)).reshape(-1)[:T].contiguous()
        state = dict(case=case, cache=cache, slots=slots, gk=gk, gv=gv)
        if case["op"] == "append":
            if case["pad"]:
                slots[max(1, T - case["pad"]):] = -1
            qkv = torch.randn(T, case["heads"] + 2 * H, d, generator=gen, device=dev, dtype=torch.bfloat16)
            state.update(k=qkv[:, -2 * H:-H], v=qkv[:, -H:])
        return state
    n, t = _lens(case)
    B, width = len(n), max(-(-x // P) for x in t)
    need = torch.tensor([-(-x // P) for x in t], device=dev)
    pages = int(need.sum()) + 2
    cache, gk, gv = _random_cache(gen, pages, H, d, P, dev)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = torch.arange(width, device=dev)[None, :] < need[:, None]
    table[at] = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[:pages - 2]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    cu[1:] = torch.tensor(n, device=dev).cumsum(0)
    q = torch.randn(sum(n), case["heads"], d, generator=gen, device=dev, dtype=torch.bfloat16)
    return dict(case=case, q=q, cache=cache, table=table, cu=cu, kv_lens=torch.tensor(t, dtype=torch.int32, device=dev),
                gk=gk, gv=gv, longest=max(n), workspace=torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------------------------------- the plain forms ----
def _plain_plan(s):
    P, T = s["case"]["page"], s["tokens"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    have, need = (cached + P - 1) // P, (cached + new + P - 1) // P
    cu = torch.zeros(new.numel() + 1, dtype=torch.int64, device=new.device)
    cu[1:] = new.cumsum(0)
    first = s["head"].long() + (need - have).cumsum(0) - (need - have)  # the request's first entry in the free list
    col = torch.arange(table.shape[1], device=new.device)
    at = (col >= have[:, None]) & (col < need[:, None])
    table[at] = s["free"][(first[:, None] + col - have[:, None])[at]]
    token = torch.arange(T, device=new.device)
    b = torch.searchsorted(cu, token, right=True) - 1
    pos = cached[b] + token - cu[b]
    slots = table[b, pos // P].long() * P + pos % P
    return dict(cu=cu.int(), kv_lens=(cached + new).int(), positions=pos.int(), slots=slots, table=table,
                head=s["head"] + (need - have).sum().int())


def _atom_of(s, slots):
    """(page, atom, token in the atom) of each slot; a slot below zero takes slot 0's."""
    P = s["case"]["page"]
    slots = slots.clamp(min=0)
    return slots // P, slots % P // 16, slots % 16


def _plain_gather(s):
    c = s["case"]
    atoms = s["cache"].view(s["cache"].shape[0], c["kv_heads"], c["page"] // 16, 18 * c["d"])
    page, atom, t = _atom_of(s, s["slots"])
    kc, ks, vc, vs = _unpack(atoms[page, :, atom])  # tokens, kv heads, 16, d
    row = torch.arange(t.numel(), device=t.device)
    live = (s["slots"] >= 0)[:, None, None]
    k = _decode(kc[row, :, t], ks[row, :, t]) * s["gk"]
    v = _decode(vc[row, :, t], vs[row, :, t]) * s["gv"]
    return dict(k=torch.where(live, k, 0.0).bfloat16(), v=torch.where(live, v, 0.0).bfloat16())


def _plain_append(s):
    c = s["case"]
    atoms = s["cache"].view(s["cache"].shape[0], c["kv_heads"], c["page"] // 16, 18 * c["d"])
    live = s["slots"] >= 0
    page, atom, t = _atom_of(s, s["slots"][live])
    # where each byte of an atom comes from: codes of the atom's own byte numbers, sent through the unpacking
    number = torch.arange(18 * c["d"], device=t.device)
    low, high = (number & 255).to(torch.uint8), (number >> 8).to(torch.uint8)
    k_at, ks_at, v_at, vs_at = _places(low, high)
    kc, ks = _encode(s["k"][live].float(), s["gk"])
    vc, vs = _encode(s["v"][live].float(), s["gv"])
    head = torch.arange(c["kv_heads"], device=t.device)[None, :, None]
    where = (page[:, None, None], head, atom[:, None, None])
    atoms[(*where, k_at[t][:, None])] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    atoms[(*where, v_at[t][:, None])] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    atoms[(*where, ks_at[t][:, None])] = ks
    atoms[(*where, vs_at[t][:, None])] = vs
    return _plain_gather(s)


def _places(low, high):
    """Byte places in an atom, [16 tokens, bytes], of the key codes, key scales, value codes and value scales."""
    def join(x):
        return x[..., 0::2] | (x[..., 1::2] << 4)
    a, b = _unpack(low), _unpack(high)
    whole = [y.long() + (z.long() << 8) for y, z in ((join(a[0]), join(b[0])), (a[1], b[1]), (join(a[2]), join(b[2])), (a[3], b[3]))]
    return whole


def _plain_attention(s):
    c = s["case"]
    B, P, H, d, G = s["table"].shape[0], c["page"], c["kv_heads"], c["d"], c["heads"] // c["kv_heads"]
    dev = s["q"].device
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    width = s["table"].shape[1]
    atoms = s["cache"][s["table"].clamp(min=0).long()].view(B, width, H, P // 16, 18 * d)
    kc, ks, vc, vs = _unpack(atoms)  # B, width, H, P / 16, 16, d
    del atoms
    L = width * P
    key = torch.arange(L, device=dev)
    inside = (key < kv[:, None])[:, None, :, None]
    k = torch.where(inside, _decode(kc, ks).permute(0, 2, 1, 3, 4, 5).reshape(B, H, L, d), 0.0)
    del kc, ks
    v = torch.where(inside, _decode(vc, vs).permute(0, 2, 1, 3, 4, 5).reshape(B, H, L, d), 0.0)
    del vc, vs
    Q = s["longest"]
    row = torch.arange(Q, device=dev)
    live = row < n[:, None]  # B, Q
    token = (cu[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().view(B, Q, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, d)
    sc = (q @ k.transpose(-1, -2)).mul_(s["gk"] * d ** -0.5).view(B, H, G, Q, L)
    pos = (kv - n)[:, None] + row  # B, Q
    see = (key <= pos[..., None]) & (key < kv[:, None, None])
    if c["window"]:
        see &= key > pos[..., None] - c["window"]
    sc.masked_fill_(~see[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, G * Q, L) @ v).view(B, H, G, Q, d) * (s["gv"] / torch.where(total == 0, 1.0, total))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H * G, d)[live].bfloat16()
    if not c["lse"]:
        return dict(out=o)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, Q, H * G)[live]
    return dict(out=o, lse=lse)


# ---------------------------------------------------------------------------------------------------- run ----
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "gather": _plain_gather,
                "attention": _plain_attention}[op](s)
    import fp4_activation_quantization_b200 as nq
    if op == "plan":
        cu, kv_lens, positions, slots, head = nq.nq_kv_plan(s["cached"], s["new"], s["table"], s["free"], s["head"],
                                                            s["tokens"], s["case"]["page"])
        return dict(cu=cu, kv_lens=kv_lens, positions=positions, slots=slots, table=s["table"], head=head)
    if op == "append":
        nq.nq_kv_append_nvfp4(s["k"], s["v"], s["slots"], s["cache"], s["gk"], s["gv"])
    if op in ("append", "gather"):
        k, v = nq.nq_kv_gather_nvfp4(s["cache"], s["slots"], s["gk"], s["gv"], s["case"]["d"])
        return dict(k=k, v=v)
    out, lse = nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"],
                                        window=s["case"]["window"], want_lse=s["case"]["lse"], workspace=s["workspace"])
    return dict(out=out, lse=lse) if s["case"]["lse"] else dict(out=out)


# -------------------------------------------------------------------------------------------------- exact ----
def _exact_token(s, page, head, t):
    """float64 key and value of token t (a long tensor of positions in their pages) of one kv head: the bytes are
    looked up one by one at the places that the layout gives them."""
    D = s["case"]["d"]
    dev = t.device
    flat = s["cache"][:, head].reshape(-1)
    base = (page * s["cache"].shape[2] + (t // 16) * 18 * D)[:, None]
    t = (t % 16)[:, None]
    dim = torch.arange(D, device=dev)[None, :]
    blk, byte, n = dim // 16, dim % 16 // 2, D // 64
    turn = t // 8 * n + blk % n
    lane = t % 8 * 4 + blk // n
    k_at = turn // 2 * 512 + lane * 16 + turn % 2 * 8 + byte
    ks_at = 16 * D + lane * (D // 32) + turn
    i, j, r = t // 8 * 2 + t % 2, t // 2 % 4, dim // (D // 8)
    w = i * (D // 16) + dim % (D // 8) // 2
    v_at = 8 * D + w // 16 * 512 + (4 * r + j) * 16 + w % 16
    per = max(1, D // 128)
    vs_at = 17 * D + (blk // per * 4 + j) * 4 * per + i * per + blk % per
    values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev)
    sf = torch.arange(256, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()

    def value(at, sf_at):
        c = flat[base + at].long()
        return values[torch.where(dim % 2 == 0, c % 16, c // 16)] * sf[flat[base + sf_at].long()]
    return value(k_at, ks_at), value(v_at, vs_at)


def _exact_codes(x, g):
    """float64 values that x stands for once it is held in 4 bits.  The scale's and the multiplier's roundings to
    float32 and e4m3 are part of the format's definition; the nearest code is looked for in 64 bits."""
    b = x.double().unflatten(-1, (-1, 16))
    third = (b.abs().amax(-1, keepdim=True) / 6).float()
    sf = (third.double() / g.double()).float().clamp(max=448).to(torch.float8_e4m3fn).double()
    step = (sf * g.double()).float().double()
    by = torch.where(step > 0, (1 / step).float().double(), 0.0)
    t = (b * by).float().double()
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=x.device) / 2
    off = (t.abs()[..., None] - grid).abs()
    off = off * 2 + torch.tensor([0, 1, 0, 1, 0, 1, 0, 1], device=x.device) * 1e-12  # a tie takes the even code
    return (grid[off.argmin(-1)] * t.sign() * sf).flatten(-2) * g.double()


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        live = (s["slots"] >= 0)[:, None, None]
        return dict(k=_exact_codes(s["k"], s["gk"]) * live, v=_exact_codes(s["v"], s["gv"]) * live)
    H, d, P = case["kv_heads"], case["d"], case["page"]
    if case["op"] == "gather":
        page, t = s["slots"] // P, s["slots"] % P
        kv = [_exact_token(s, page, h, t) for h in range(H)]
        return dict(k=torch.stack([x[0] for x in kv], 1) * s["gk"].double(),
                    v=torch.stack([x[1] for x in kv], 1) * s["gv"].double())
    G = case["heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, t) in enumerate(zip(*_lens(case))):
        key = torch.arange(t, device="cuda")
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        hide = key > pos
        if case["window"]:
            hide |= key <= pos - case["window"]
        for h in range(H):
            k, v = _exact_token(s, s["table"][b].long()[key // P], h, key % P)
            for g in range(h * G, h * G + G):
                x = (s["q"][at:at + n, g].double() @ k.T) * (s["gk"].double() / d ** 0.5)
                x.masked_fill_(hide, float("-inf"))
                lse[at:at + n, g] = x.logsumexp(-1)
                out[at:at + n, g] = x.softmax(-1) @ v * s["gv"].double()
        at += n
    return dict(out=out, lse=lse) if case["lse"] else dict(out=out)
