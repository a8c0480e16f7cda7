"""GPU tests of the 4-bit key/value cache: plans, append and gather (exact), attention (against float64 within the
bounds that its roundings give), and a run of all of them together."""
import numpy as np
import pytest
import torch

import kv_helpers as K
import oracle
from gpu_helpers import SENTINEL, Guarded, host_u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nq():
    import fp4_activation_quantization_b200 as nq
    return nq


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f32(x):
    return torch.tensor([x], dtype=torch.float32, device="cuda")


# ---------------------------------------------------------------------------------------------------- plans ----
@pytest.mark.parametrize("B,most,cached,page,pad", [
    (1, 1, 0, 16, 0), (1, 1, 15, 16, 0), (1, 1, 16, 16, 3), (3, 40, 100, 16, 0), (64, 1, 5000, 16, 0),
    (64, 9, 700, 128, 7), (513, 33, 300, 32, 0), (2049, 5, 90, 64, 11), (4100, 3, 40, 16, 1), (2, 9000, 50, 64, 0),
])
def test_plan(nq, B, most, cached, page, pad):
    rng = np.random.default_rng(B + most)
    new = rng.integers(0, most + 1, B)
    new[0] = most
    old = rng.integers(0, cached + 1, B)
    width = int(max(-(-(o + n) // page) for o, n in zip(old, new))) + 2
    held = -(-old // page)
    ids = rng.permutation(int(held.sum()) + int(new.sum()) + 2 * B + 9).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free, T = ids[at:], int(new.sum()) + pad
    want_table = table.copy()
    want = K.plan(old.tolist(), new.tolist(), want_table, free, 2, T, page)
    wide = torch.full((B, width + 3), -7, dtype=torch.int32, device="cuda")  # a table with a row stride of its own
    wide[:, :width] = i32(table)
    got = nq.nq_kv_plan(i32(old), i32(new), wide[:, :width], i32(free), i32([2]), T, page)
    for g, w in zip(got, want[:4]):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(got[4]) == want[4]
    assert np.array_equal(wide[:, :width].cpu().numpy(), want_table)
    assert bool((wide[:, width:] == -7).all())
    nq.nq_check_device_errors()


def test_plan_without_requests_or_tokens(nq):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    cu, kv, pos, slots, head = nq.nq_kv_plan(none, none, table, none, i32([0]), 5, 16)
    assert cu.tolist() == [0] and kv.numel() == 0 and pos.tolist() == [-1] * 5 and slots.tolist() == [-1] * 5
    assert int(head) == 0
    nq.nq_check_device_errors()


def test_plan_advances_its_list_in_place(nq):
    table, head = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), i32([0])
    free = i32(range(100, 120))
    lens = i32([0, 0])
    for step in range(5):
        out = nq.nq_kv_plan(lens, i32([16, 1]), table, free, head, 17, 16, free_head_out=head)
        lens = out[1]
        assert out[4] is head
    assert lens.tolist() == [80, 5] and int(head) == 6
    assert table[0, :5].tolist() == [100, 102, 103, 104, 105] and int(table[1, 0]) == 101
    nq.nq_check_device_errors()


@pytest.mark.parametrize("case", ["list", "table", "tokens", "negative"])
def test_plan_overruns_are_reported_and_stay_in_bounds(nq, case):
    table = torch.full((3, 6), -7, dtype=torch.int32, device="cuda")
    table[1, 0] = 50
    view = table[:, :4]
    args = dict(old=[0, 5, 0], new=[20, 30, 3], free=list(range(10, 30)), T=53)
    if case == "list":
        args["free"] = [10, 11, 12]
    elif case == "table":
        args["new"] = [20, 100, 3]
        args["T"] = 123
    elif case == "tokens":
        args["T"] = 40
    else:
        args["new"] = [20, -4, 3]
        args["T"] = 23
    cu, kv, pos, slots, _ = nq.nq_kv_plan(i32(args["old"]), i32(args["new"]), view, i32(args["free"]), i32([0]),
                                          args["T"], 16)
    with pytest.raises(nq.NQError, match="bit 3"):
        nq.nq_check_device_errors()
    assert bool((table[:, 4:] == -7).all())
    slots, pos = slots.cpu().numpy(), pos.cpu().numpy()
    if case == "list":  # pages 10, 11 | 50 (held), 12, none | none
        assert slots[:20].tolist() == [*range(160, 180)]
        assert slots[20:47].tolist() == [*range(50 * 16 + 5, 51 * 16), *range(12 * 16, 13 * 16)]
        assert (slots[47:] == -1).all()
        assert table[1, :3].tolist() == [50, 12, -1] and int(table[2, 0]) == -1
    elif case == "table":
        assert kv.tolist() == [20, 64, 3]
        assert (slots[20:20 + 59] >= 0).all() and (slots[79:120] == -1).all() and (slots[120:] >= 0).all()
    elif case == "tokens":
        assert cu.tolist() == [0, 20, 40, 40] and (slots >= 0).all()
    else:
        assert cu.tolist() == [0, 20, 20, 23] and kv.tolist() == [20, 5, 3] and (slots >= 0).all()


# ----------------------------------------------------------------------------------------- append and gather ----
def tokens_like(shape, seed, special=True):
    """bf16 values with blocks of zeros, signed zeros, single large and tiny elements, and infinities."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if special:
        f = x.view(-1, 16)
        n = f.shape[0]
        f[1 % n] = 0.0
        f[2 % n] = -0.0
        f[3 % n] *= 1e30
        f[4 % n] *= 1e-30
        f[5 % n, 3] = 1000.0
        f[6 % n, 7] = float("inf")
        f[7 % n] = torch.arange(16) * 0.25  # on the borders between codes
    return x.bfloat16()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,T,H", [(16, 1, 1), (16, 37, 3), (64, 130, 2), (128, 129, 5), (32, 31, 1)])
def test_append_then_gather(nq, D, page, T, H):
    pages = -(-T // page) + 2
    rng = np.random.default_rng(T * D + H)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[:T // 2] = np.arange(T // 2) + page // 2  # a run, as a prompt's
        slots[T // 2:] = rng.permutation(np.setdiff1d(np.arange(pages * page), slots[:T // 2]))[:T - T // 2]
        slots[[1, T - 1]] = -1
    qkv = tokens_like((T, 2 * H + 1, D), seed=T)
    k, v = qkv[:, 1:H + 1], qkv[:, H + 1:]
    gk, gv = np.float32(0.0123), np.float32(3.0 / 2688)
    cache = rng.integers(0, 256, nq.kv_cache_shape(pages, H, D, page), dtype=np.uint8)
    cache[..., :] = np.where(rng.random(cache.shape) < 0.1, 0x7F, cache)
    dev = torch.from_numpy(cache.copy()).cuda()
    q = qkv.cuda()
    nq.nq_kv_append_nvfp4(q[:, 1:H + 1], q[:, H + 1:], torch.from_numpy(slots).cuda(), dev, f32(gk), f32(gv))
    want = cache.copy()
    K.write(want, slots, k.float().numpy(), v.float().numpy(), gk, gv, D, page)
    assert np.array_equal(host_u8(dev), want)

    # every slot of the cache back (its bytes where nothing was appended may decode to NaN), some twice, some padding
    again = np.concatenate([slots, slots[:3], [-1, pages * page - 1]]).astype(np.int64)
    kk, vv = nq.nq_kv_gather_nvfp4(dev, torch.from_numpy(again).cuda(), f32(gk), f32(gv), D)
    dk, dv = K.decode(torch.from_numpy(want), D, page)
    for got, x, g in ((kk, dk, gk), (vv, dv, gv)):
        x = x.reshape(-1, H, D)[torch.from_numpy(np.maximum(again, 0))].float() * float(g)
        x = torch.where(torch.from_numpy(again >= 0)[:, None, None], x, torch.zeros(())).bfloat16()
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=7e9), torch.nan_to_num(x.float(), nan=7e9))
    nq.nq_check_device_errors()


def test_append_takes_any_strides_and_alignment(nq):
    T, H, D, page = 19, 3, 128, 16
    x = tokens_like((2, T, H, D), seed=3).cuda()
    slots = torch.randperm(48, device="cuda", generator=torch.Generator("cuda").manual_seed(1))[:T]
    want = torch.zeros(nq.kv_cache_shape(3, H, D, page), dtype=torch.uint8, device="cuda")
    nq.nq_kv_append_nvfp4(x[0], x[1], slots, want, f32(0.01), f32(0.02))
    flat = torch.zeros(1 + 2 * T * (H * D + 1), dtype=torch.bfloat16, device="cuda")
    odd = [flat[1 + i * T * (H * D + 1):][:T * (H * D + 1)].view(T, H * D + 1)[:, 1:].view(T, H, D) for i in (0, 1)]
    head_major = [torch.empty((H, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1) for _ in (0, 1)]
    for k, v in (odd, head_major):
        k.copy_(x[0])
        v.copy_(x[1])
        # the pages of three layers side by side, and slot tensors of a stream's own
        layers = torch.zeros((3, 3, *want.shape[1:]), dtype=torch.uint8, device="cuda")
        nq.nq_kv_append_nvfp4(k, v, slots, layers[:, 1], f32(0.01), f32(0.02))
        assert torch.equal(layers[:, 1], want) and not layers[:, 0].any() and not layers[:, 2].any()
    a, b = nq.nq_kv_gather_nvfp4(want, slots, f32(0.01), f32(0.02), D)
    for k, v in (odd, head_major):
        nq.nq_kv_gather_nvfp4(want, slots, f32(0.01), f32(0.02), D, k_out=k, v_out=v)
        assert torch.equal(k, a) and torch.equal(v, b)


def test_slots_past_the_cache_are_skipped(nq):
    T, H, D, page = 5, 2, 64, 16
    x = tokens_like((2, T, H, D), seed=9).cuda()
    raw = torch.full((4, *nq.kv_cache_shape(1, H, D, page)[1:]), SENTINEL, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([3, 32, 1 << 40, -1, 31], device="cuda")
    nq.nq_kv_append_nvfp4(x[0], x[1], slots, raw[1:3], f32(0.01), f32(0.01))
    with pytest.raises(nq.NQError, match="bit 2"):
        nq.nq_check_device_errors()
    assert bool((raw[0] == SENTINEL).all()) and bool((raw[3] == SENTINEL).all())
    k, v = nq.nq_kv_gather_nvfp4(raw[1:3], slots, f32(0.01), f32(0.01), D)
    with pytest.raises(nq.NQError, match="bit 2"):
        nq.nq_check_device_errors()
    assert not k[1:4].any() and not v[1:4].any() and bool(k[0].any()) and bool(v[4].any())


# ------------------------------------------------------------------------------------------------- attention ----
def make(nq, n, t, heads, kv_heads, D, page, seed=0, spread=1.0, tail=0, q_scale=1.0):
    """A ragged batch over a cache whose unused bytes are noise (NaN scales among them)."""
    gen = torch.Generator("cuda").manual_seed(seed)
    B, T = len(n), sum(n) + tail
    need = [-(-x // page) for x in t]
    width, pages = max([*need, 1]) + 1, sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, width), 1 << 30, dtype=torch.int32, device="cuda")  # entries behind a request's pages are not read
    at = 1
    slots, req = [], []
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        tok = torch.arange(t[b], device="cuda")
        slots.append(table[b].long()[tok // page] * page + tok % page)
    slots = torch.cat(slots) if slots else torch.empty(0, dtype=torch.int64, device="cuda")
    cache = torch.randint(0, 256, nq.kv_cache_shape(pages, kv_heads, D, page), generator=gen, device="cuda").to(torch.uint8)
    noise = torch.rand(cache.shape, generator=gen, device="cuda")
    cache[noise < 0.2] = 0x7F
    k = torch.randn((slots.numel(), kv_heads, D), generator=gen, device="cuda").mul_(spread).bfloat16()
    v = torch.randn((slots.numel(), kv_heads, D), generator=gen, device="cuda").bfloat16()
    gk, gv = f32(4.6 * spread / 2688), f32(4.6 / 2688)
    if slots.numel():
        nq.nq_kv_append_nvfp4(k, v, slots, cache, gk, gv)
    q = torch.randn((T, heads, D), generator=gen, device="cuda").mul_(q_scale).bfloat16()
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    return dict(q=q, cache=cache, table=table, kv_lens=i32(t), cu=cu, gk=gk, gv=gv, n=n, t=t, page=page, D=D)


def expect(s, scale=None, window=0, causal=True):
    k, v = K.decode(s["cache"], s["D"], s["page"])  # looked up only where tokens were appended
    return K.attention(s["q"], k, v, float(s["gk"]), float(s["gv"]), s["table"], s["t"], s["cu"].tolist(), s["page"],
                       s["D"] ** -0.5 if scale is None else scale, window, causal)


def check(nq, s, scale=None, window=0, causal=True, workspace=None, **more):
    rows = sum(s["n"])
    out = torch.full_like(s["q"], 123.0)
    lse = torch.full(s["q"].shape[:2], 123.0, device="cuda")
    nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"], scale=scale,
                             window=window, out=out, lse=lse, workspace=workspace,
                             flags=0 if causal else nq.FLAG_NONCAUSAL, **more)
    o, l, tol, tol_lse = expect(s, scale, window, causal)
    assert bool((out[rows:] == 123.0).all()) and bool((lse[rows:] == 123.0).all())
    empty = torch.isneginf(l[:rows])
    assert torch.equal(torch.isneginf(lse[:rows]), empty)
    d = (out[:rows].double() - o[:rows]).abs()
    assert bool((d <= tol[:rows]).all()), float((d / tol[:rows].clamp(min=1e-300)).max())
    assert not out[:rows][empty].any()
    d = torch.where(empty, 0.0, (lse[:rows].double() - l[:rows]).abs())
    assert bool((d <= tol_lse[:rows]).all()), float((d / tol_lse[:rows]).max())
    nq.nq_check_device_errors()
    return out, lse


SHAPES = [(1, 1, 64), (8, 1, 64), (8, 8, 64), (10, 2, 64), (16, 2, 64), (1, 1, 128), (4, 1, 128), (32, 8, 128),
          (20, 4, 128), (16, 1, 128), (2, 2, 256), (8, 4, 256), (16, 1, 256)]


@pytest.mark.parametrize("heads,kv_heads,D", SHAPES)
@pytest.mark.parametrize("page", [16, 128])
def test_single_tokens(nq, heads, kv_heads, D, page):
    check(nq, make(nq, [1] * 7, [1, 2, 15, 16, 17, 300, 1029], heads, kv_heads, D, page, seed=heads + D))


@pytest.mark.parametrize("heads,kv_heads,D", SHAPES)
@pytest.mark.parametrize("window,causal", [(0, True), (33, True), (0, False), (100, False), (1, True)])
def test_few_tokens(nq, heads, kv_heads, D, window, causal):
    # empty requests, requests without keys, more rows than keys (rows whose mask leaves nothing)
    s = make(nq, [3, 0, 5, 2, 4, 1, 7], [3, 40, 2, 0, 517, 130, 64], heads, kv_heads, D, 32, seed=D, tail=3)
    check(nq, s, window=window, causal=causal)


@pytest.mark.parametrize("heads,kv_heads,D", SHAPES)
@pytest.mark.parametrize("window,causal", [(0, True), (190, True), (0, False)])
def test_prompts(nq, heads, kv_heads, D, window, causal):
    s = make(nq, [129, 1, 0, 257, 40], [129, 300, 5, 600, 41], heads, kv_heads, D, 64, seed=D + 1, tail=2)
    check(nq, s, window=window, causal=causal)


@pytest.mark.parametrize("heads,kv_heads,D", [(16, 4, 64), (16, 4, 128), (16, 4, 256)])
def test_many_chunks_from_a_cold_cache(nq, heads, kv_heads, D):
    """More tiles than the GPU holds at once, first with the cache's bytes out of L2 (slow), then in it: the same bits."""
    s = make(nq, [400] * 12, [700 + 60 * i for i in range(12)], heads, kv_heads, D, 64, seed=15)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(4):
        if i % 2 == 0:
            flush.fill_(i)
        outs.append(check(nq, s))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_rows_beyond_the_keys(nq, D):
    check(nq, make(nq, [300, 200], [130, 0], 8, 2, D, 16, seed=4))
    check(nq, make(nq, [300, 200], [130, 0], 8, 2, D, 16, seed=4), window=7)


@pytest.mark.parametrize("D,heads,kv_heads", [(64, 8, 1), (128, 4, 1), (128, 16, 8), (256, 2, 1)])
def test_one_long_request_is_split_over_the_gpu(nq, D, heads, kv_heads):
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    # one workspace for calls that split their keys in different ways, one after another
    for n, t in (([1], [40001]), ([70], [9000]), ([1, 1], [700, 33]), ([1] * 700, [90] * 699 + [9000]), ([1], [40001])):
        check(nq, make(nq, n, t, heads, kv_heads, D, 128, seed=2), workspace=ws)


@pytest.mark.parametrize("n,t", [([1] * 5, [3000] * 5), ([200, 90], [1500, 900])])
@pytest.mark.parametrize("q_scale,spread", [(30.0, 1.0), (1e-3, 1e3), (1e4, 1.0), (1e-6, 1e-6)])
def test_sharp_and_flat_scores(nq, n, t, q_scale, spread):
    s = make(nq, n, t, 8, 2, 128, 64, seed=6, q_scale=q_scale, spread=spread)
    check(nq, s)


@pytest.mark.parametrize("n,t", [([1] * 3, [2000] * 3), ([300], [2000])])
def test_scores_that_keep_rising(nq, n, t):
    """Keys that grow along the axis raise the running maximum again and again."""
    s = make(nq, n, t, 4, 1, 128, 64, seed=7)
    x = torch.linspace(0.01, 1, sum(t), device="cuda") * 4.0
    gen = torch.Generator("cuda").manual_seed(1)
    base = torch.randn((1, 1, 128), generator=gen, device="cuda")
    k = (base * x[:, None, None]).bfloat16()
    slots = torch.cat([s["table"][b].long()[torch.arange(m, device="cuda") // 64] * 64 + torch.arange(m, device="cuda") % 64
                       for b, m in enumerate(t)])
    nq.nq_kv_append_nvfp4(k, k, slots, s["cache"], s["gk"] * 4, s["gv"] * 4)
    s["gk"], s["gv"] = s["gk"] * 4, s["gv"] * 4
    s["q"].copy_((base * torch.rand(s["q"].shape[:2], generator=gen, device="cuda")[..., None] * 3).bfloat16())
    check(nq, s)


@pytest.mark.parametrize("n,t", [([1, 2, 1], [700, 40, 90]), ([150, 20], [150, 300])])
def test_a_nan_row_stays_alone(nq, n, t):
    s = make(nq, n, t, 4, 2, 128, 16, seed=8)
    args = (s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    want, want_lse = nq.nq_attention_nvfp4_kv(s["q"], *args, want_lse=True)
    q = s["q"].clone()
    q[1, 2, 5] = float("nan")
    got, got_lse = nq.nq_attention_nvfp4_kv(q, *args, want_lse=True)
    assert bool(got[1, 2].isnan().all()) and bool(got_lse[1, 2].isnan())
    got[1, 2], got_lse[1, 2] = want[1, 2], want_lse[1, 2]
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


@pytest.mark.parametrize("n,t", [([1] * 9, [5000] * 9), ([130, 260], [700, 1300])])
def test_same_bits_every_time_and_in_any_place(nq, n, t):
    s = make(nq, n, t, 16, 4, 128, 32, seed=9)
    args = (s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    want, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
    for _ in range(3):
        assert torch.equal(nq.nq_attention_nvfp4_kv(s["q"], *args)[0], want)
    T, H, D = s["q"].shape
    raw = torch.full((T * (H * D + 3) + 5,), 9.0, dtype=torch.bfloat16, device="cuda")
    odd = raw[5:].view(T, H * D + 3)[:, :H * D].view(T, H, D)  # rows that start off every alignment
    odd.copy_(s["q"])
    out = Guarded(T, H * D, torch.bfloat16, pad=5)
    nq.nq_attention_nvfp4_kv(odd, *args, out=out.view.view(T, H, D))
    assert torch.equal(out.view.reshape(T, H, D), want) and out.guards_intact()
    head_major = s["q"].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((H, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    nq.nq_attention_nvfp4_kv(head_major, *args, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,t", [([1] * 4, [200, 900, 64, 65]), ([64, 200], [300, 900])])
def test_pages_outside_the_cache_are_skipped(nq, n, t):
    s = make(nq, n, t, 8, 2, 128, 16, seed=10)
    args = [s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"]]
    bad = s["table"].clone()
    bad[1, 2], bad[0, 1] = -1, s["cache"].shape[0]
    args[1] = bad
    out, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
    with pytest.raises(nq.NQError, match="bit 2"):
        nq.nq_check_device_errors()
    # as if the keys of those pages were not there
    k, v = K.decode(s["cache"], 128, 16)
    keep = [torch.ones(x, dtype=torch.bool, device="cuda") for x in t]
    keep[0][16:32] = False
    keep[1][32:48] = False
    at = 0
    for b, x in enumerate(t):
        key = torch.arange(x, device="cuda")
        pages = s["table"][b].long()[key // 16]
        kb, vb = k[pages, key % 16].repeat_interleave(4, 1), v[pages, key % 16].repeat_interleave(4, 1)
        sc = torch.einsum("ihd,jhd->hij", s["q"][at:at + n[b]].double(), kb) * (float(s["gk"]) * 128 ** -0.5)
        see = (key <= torch.arange(x - n[b], x, device="cuda")[:, None]) & keep[b]
        sc = sc.masked_fill(~see, -float("inf"))
        p = torch.nan_to_num(torch.softmax(sc, -1), nan=0.0)
        o = torch.einsum("hij,jhd->ihd", p, vb) * float(s["gv"])
        a = torch.einsum("hij,jhd->ihd", p, vb.abs()) * float(s["gv"])
        # the bf16 step, and 2^-10 of sum p |v| for the weights' f16 step and the scores' float32 errors
        assert bool(((out[at:at + n[b]].double() - o).abs() <= 2.0**-8 * o.abs() + 2.0**-10 * a + 1e-6).all())
        at += n[b]


def test_lengths_beyond_the_tensors_stay_in_bounds(nq):
    """Lengths past the table's width and rows past the query tensor are cut."""
    s = make(nq, [2, 3], [60, 64], 4, 2, 128, 16, seed=11)
    table = s["table"][:, :4].contiguous()
    want, _ = nq.nq_attention_nvfp4_kv(s["q"], s["cache"], table, i32([64, 64]), s["cu"], s["gk"], s["gv"])
    got, _ = nq.nq_attention_nvfp4_kv(s["q"], s["cache"], table, i32([1 << 29, 65]), s["cu"], s["gk"], s["gv"])
    # bit for bit: keys 60 ... 63 of the first request were never written, and its rows may be NaN
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    out = torch.full((8, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    nq.nq_attention_nvfp4_kv(s["q"], s["cache"], table, i32([60, 64]), i32([0, 2, 900]), s["gk"], s["gv"], out=out[:5])
    assert bool((out[5:] == 5.0).all())


def test_offsets_past_32_bits(nq):
    """A cache larger than 4 GB whose request lies at its end."""
    page, H, D = 128, 8, 128
    one = page * H * D * 9 // 8
    pages = (1 << 32) // one + 40
    cache = torch.zeros(nq.kv_cache_shape(pages, H, D, page), dtype=torch.uint8, device="cuda")
    s = make(nq, [1, 3], [1000, 300], 16, H, D, page, seed=12)
    need = s["cache"].shape[0]
    cache[-need:] = s["cache"]
    want, _ = nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    far = torch.where(s["table"] < need, s["table"] + (pages - need), s["table"])
    got, _ = nq.nq_attention_nvfp4_kv(s["q"], cache, far, s["kv_lens"], s["cu"], s["gk"], s["gv"])
    assert torch.equal(got, want)
    slot = torch.tensor([pages * page - 1, (pages - need) * page], device="cuda")
    k = tokens_like((2, H, D), seed=1, special=False).cuda()
    nq.nq_kv_append_nvfp4(k, k, slot, cache, f32(0.002), f32(0.002))
    kk, vv = nq.nq_kv_gather_nvfp4(cache, slot, f32(0.002), f32(0.002), D)
    assert torch.equal(kk, vv)
    # a code is within half its block's widest gap (a sixth of the largest element, and the scale's 2^-4)
    top = k.float().unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True)
    assert bool(((kk.float() - k.float()).unflatten(-1, (-1, 16)).abs() <= top * (1 / 6 + 2.0**-4)).all())
    nq.nq_check_device_errors()


@pytest.mark.parametrize("n,t", [([1] * 6, [900] * 6), ([100, 140], [400, 900])])
def test_captured_and_replayed(nq, n, t):
    s = make(nq, n, t, 8, 2, 128, 32, seed=13)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, other = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    lens = s["kv_lens"].clone()
    args = (s["cache"], s["table"], lens, s["cu"], s["gk"], s["gv"])
    graphs = []
    stream = torch.cuda.Stream()
    for o in (out, other):  # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=stream):
            nq.nq_attention_nvfp4_kv(s["q"], *args, out=o, workspace=ws)
        graphs.append(g)
    for cut in (0, 250, 7):
        lens.copy_(s["kv_lens"] - cut)
        for g in graphs:
            g.replay()
        want, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
        assert torch.equal(out, want) and torch.equal(other, want)


def test_other_stream_and_programmatic_launch(nq):
    s = make(nq, [1] * 6, [900] * 6, 8, 2, 128, 32, seed=14)
    args = (s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    want, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    outs = [torch.empty_like(want) for _ in range(4)]
    for o in outs:  # each call may start while the one before it ends
        nq.nq_attention_nvfp4_kv(s["q"], *args, out=o, workspace=ws, flags=nq.FLAG_PDL, stream=stream)
    stream.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def many(nq, B, heads, kv_heads, D, least, most, seed, rows=1):
    """B requests of `rows` tokens whose pages are the same (a shared prefix), of lengths least ... most."""
    s = make(nq, [rows], [most], heads, kv_heads, D, 16, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    t = torch.randint(least, most + 1, (B,), generator=gen, device="cuda").tolist()
    n = [rows] * B
    s.update(q=torch.randn((B * rows, heads, D), generator=gen, device="cuda").bfloat16(), table=s["table"].repeat(B, 1),
             kv_lens=i32(t), cu=i32(np.arange(B + 1) * rows), n=n, t=t)
    return s


# Lengths from one tile of keys to shares that are long enough to be claimed in small parts (64 x 8 heads x 7500).
@pytest.mark.parametrize("B,heads,kv_heads,D,least,most,rows", [
    (400, 8, 2, 128, 1, 300, 1), (64, 8, 8, 64, 7000, 8000, 1), (200, 16, 4, 64, 5, 2000, 3), (200, 8, 4, 256, 5, 900, 1),
    (150, 16, 4, 128, 4, 1200, 3)])
def test_many_requests_share_out_evenly(nq, B, heads, kv_heads, D, least, most, rows):
    s = many(nq, B, heads, kv_heads, D, least, most, seed=15, rows=rows)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, lse = check(nq, s, workspace=ws)
    for _ in range(3):  # the parts that are claimed differ from run to run, the bits do not
        again, lse_again = check(nq, s, workspace=ws)
        assert torch.equal(again, out) and torch.equal(lse_again, lse)


@pytest.mark.parametrize("heads,kv_heads,D,window", [(16, 4, 64, 0), (16, 4, 128, 150), (8, 4, 256, 0), (12, 4, 128, 0)])
def test_more_tiles_than_multiprocessors(nq, heads, kv_heads, D, window):
    """Prompts and chunks of every length, some of no token, in one call: a CTA takes several tiles of them."""
    rng = np.random.default_rng(D + heads)
    n = [int(x) for x in rng.integers(0, 400, 60)]
    n[3], n[7], n[8], n[59] = 0, 0, 129, 0
    t = [x + int(y) for x, y in zip(n, rng.integers(0, 300, 60))]
    s = make(nq, n, t, heads, kv_heads, D, 16, seed=18, tail=3)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, lse = check(nq, s, window=window, workspace=ws)
    args = (s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    again = torch.empty_like(out)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(2):
            nq.nq_attention_nvfp4_kv(s["q"], *args, window=window, out=again, workspace=ws, flags=nq.FLAG_PDL)
    for _ in range(3):
        again.fill_(123.0)
        graph.replay()
        assert torch.equal(again, out)
    nq.nq_check_device_errors()


def test_many_requests_captured_with_a_shared_workspace(nq):
    s = many(nq, 400, 8, 2, 128, 1, 500, seed=16)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, other = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    lens = s["kv_lens"].clone()
    args = (s["cache"], s["table"], lens, s["cu"], s["gk"], s["gv"])
    graphs = []
    stream = torch.cuda.Stream()
    for o in (out, other):
        g = torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=stream):
            for _ in range(2):  # the second call may start under the first one's end
                nq.nq_attention_nvfp4_kv(s["q"], *args, out=o, workspace=ws, flags=nq.FLAG_PDL)
        graphs.append(g)
    for cut in (0, 100, 499):
        lens.copy_((s["kv_lens"] - cut).clamp_(min=0))
        for g in graphs:
            g.replay()
        want, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
        assert torch.equal(out, want) and torch.equal(other, want)
    nq.nq_check_device_errors()


def test_own_workspace_on_another_stream(nq):
    """Without a workspace the call zeroes one in the order of its stream, whatever the memory held."""
    s = many(nq, 400, 8, 2, 128, 1, 500, seed=17)
    args = (s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"])
    want, _ = nq.nq_attention_nvfp4_kv(s["q"], *args)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for handle in (stream, stream.cuda_stream):
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        nq.nq_attention_nvfp4_kv(s["q"], *args, out=out, stream=handle)
        stream.synchronize()
        assert torch.equal(out, want)


def test_plan_reports_sums_past_32_bits(nq):
    """Four requests of 2^30 tokens: their sum is 0 modulo 2^32."""
    B, width = 4, (1 << 30) // 128
    table = torch.full((B, width + 1), -7, dtype=torch.int32, device="cuda")
    zero = i32([0] * B)
    cu, kv, pos, slots, _ = nq.nq_kv_plan(zero, i32([1 << 30] * B), table[:, :width], i32([5, 6]), i32([0]), 8, 128)
    with pytest.raises(nq.NQError, match="bit 3"):
        nq.nq_check_device_errors()
    assert bool((table[:, width] == -7).all()) and kv.tolist() == [1 << 30] * B


def test_binding_refusals(nq):
    s = make(nq, [1], [20], 4, 2, 128, 16)
    good = dict(q=s["q"], cache=s["cache"], block_table=s["table"], kv_lens=s["kv_lens"], cu_q=s["cu"], k_scale=s["gk"],
                v_scale=s["gv"])
    for name, bad in [("q", s["q"].float()), ("q", s["q"][0]), ("cache", s["cache"].view(torch.int8)),
                      ("cache", s["cache"][..., :-1]), ("block_table", s["table"].long()),
                      ("block_table", s["table"][0]), ("kv_lens", s["kv_lens"].long()), ("cu_q", s["cu"][:1]),
                      ("k_scale", s["gk"].double()), ("v_scale", torch.ones(2, device="cuda")), ("q", s["q"].cpu())]:
        with pytest.raises(ValueError):
            nq.nq_attention_nvfp4_kv(**{**good, name: bad})
    with pytest.raises(ValueError):
        nq.nq_attention_nvfp4_kv(**good, out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        nq.nq_attention_nvfp4_kv(**good, lse=torch.empty(1, 3, device="cuda"))
    with pytest.raises(nq.NQError):
        nq.nq_attention_nvfp4_kv(**good, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    for window in (-1, 1 << 32):
        with pytest.raises(ValueError, match="window"):
            nq.nq_attention_nvfp4_kv(**good, window=window)
    with pytest.raises(ValueError):
        nq.nq_kv_append_nvfp4(s["q"], s["q"], torch.zeros(1, dtype=torch.int64, device="cuda"), s["cache"], s["gk"], s["gv"])
    with pytest.raises(ValueError):
        nq.nq_kv_gather_nvfp4(s["cache"], torch.zeros(1, dtype=torch.int32, device="cuda"), s["gk"], s["gv"], 128)
    with pytest.raises(ValueError):
        nq.nq_kv_plan(s["kv_lens"].long(), s["kv_lens"], s["table"], s["kv_lens"], s["kv_lens"], 1, 16)
    for name in good:  # no tensor at all
        with pytest.raises(ValueError, match=name):
            nq.nq_attention_nvfp4_kv(**{**good, name: None})
    args = [s["kv_lens"], s["kv_lens"], s["table"], s["kv_lens"], s["kv_lens"]]
    for i in range(5):
        for bad in (None, 3, args[i].cpu(), args[i].float(), args[i][..., None]):
            with pytest.raises(ValueError):
                nq.nq_kv_plan(*[bad if i == j else a for j, a in enumerate(args)], 1, 16)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    args = [k, k, torch.zeros(2, dtype=torch.int64, device="cuda"), s["cache"], s["gk"], s["gv"]]
    for i in range(6):
        for bad in (None, args[i].cpu(), args[i].double(), args[i][None]):
            with pytest.raises(ValueError):
                if i >= 4 and bad is not None and bad.dtype == torch.float32 and bad.is_cuda:
                    raise ValueError  # one element in any shape is taken
                nq.nq_kv_append_nvfp4(*[bad if i == j else a for j, a in enumerate(args)])
    with pytest.raises(ValueError):
        nq.nq_kv_append_nvfp4(k.transpose(1, 2), k.transpose(1, 2), *args[2:])


# ----------------------------------------------------------------------------------------- all of it together ----
def test_a_server_s_steps(nq):
    """Prompts, a chunk behind a prefix, then single tokens: plan, append, attention, and the quantized input of the
    output projection, against float64 attention over keys and values that went through the oracle's codecs."""
    H, G, D, page, B = 2, 4, 128, 16, 3
    gen = torch.Generator("cuda").manual_seed(20)
    gk, gv = f32(4.6 / 2688), f32(4.6 / 2688)
    cache = torch.randint(0, 256, nq.kv_cache_shape(40, H, D, page), generator=gen, device="cuda").to(torch.uint8)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(40, generator=gen, device="cuda").to(torch.int32), i32([0])
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    lens = i32([0, 0, 0])
    shadow = np.zeros(nq.kv_cache_shape(40, H, D, page), np.uint8)
    for new in ([37, 0, 90], [1, 50, 1], [1, 1, 1], [1, 1, 1], [4, 1, 0]):
        T = sum(new) + 2
        cu, lens_now, pos, slots, _ = nq.nq_kv_plan(lens, i32(new), table, free, head, T, page, free_head_out=head)
        qkv = torch.randn((T, H * G + 2 * H, D), generator=gen, device="cuda").bfloat16()
        q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        nq.nq_kv_append_nvfp4(k, v, slots, cache, gk, gv)
        out, lse = nq.nq_attention_nvfp4_kv(q, cache, table, lens_now, cu, gk, gv, want_lse=True, workspace=ws)
        q8, s8 = nq.nq_per_token_group_quant_fp8(out[:sum(new)].reshape(-1, H * G * D), 128)
        K.write(shadow, slots.cpu().numpy(), k.float().cpu().numpy(), v.float().cpu().numpy(), float(gk), float(gv), D, page)
        kd, vd = K.decode(torch.from_numpy(shadow).cuda(), D, page)
        o, l, tol, tol_lse = K.attention(q, kd, vd, float(gk), float(gv), table, lens_now.tolist(), cu.tolist(), page,
                                         D ** -0.5)
        n = sum(new)
        assert bool(((out[:n].double() - o[:n]).abs() <= tol[:n]).all())
        assert bool(((lse[:n].double() - l[:n]).abs() <= tol_lse[:n]).all())
        rows = out[:n].reshape(n, -1).view(torch.int16).cpu().numpy().view(np.uint16)
        eq, es = oracle.per_token_group_quant_fp8(rows, 128)
        assert np.array_equal(host_u8(q8), eq) and np.array_equal(s8.cpu().numpy(), es)
        lens = lens_now
    assert lens.tolist() == [44, 53, 93]
    nq.nq_check_device_errors()
