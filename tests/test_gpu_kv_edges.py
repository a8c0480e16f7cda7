"""GPU tests of the 4-bit key/value cache at its edges: rows and requests without keys among others, weights far below
the largest, scales and queries of extreme size, lengths that do not fit, streams, and every form of the kernels."""
import numpy as np
import pytest
import torch

import kv_helpers as K
from gpu_helpers import Guarded
from test_gpu_kv import check, f32, i32, make, nq  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def call(nq, s, **more):
    return nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"], **more)


@pytest.mark.parametrize("heads,kv_heads,D", [(16, 1, 64), (16, 2, 128), (8, 2, 256)])
@pytest.mark.parametrize("seed", range(4))
def test_runs_of_tiles_without_keys(nq, heads, kv_heads, D, seed):
    """Most requests without keys, of every number of rows: a CTA takes several tiles without keys one after another."""
    rng = np.random.default_rng(seed)
    n = [int(x) for x in rng.integers(1, 180, 120)]
    t = [int(x) for x in rng.choice([0, 0, 0, 0, 1, 5, 300], 120)]
    s = make(nq, n, t, heads, kv_heads, D, 16, seed=seed, tail=1)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for causal in (False, True):
        for _ in range(5):
            check(nq, s, causal=causal, workspace=ws)


# Rows and keys of a batch that takes each form of the kernels: one chunk a CTA, a share a warp, 128-row tiles.
FORMS = {"chunks": ([1] * 3, [700, 40, 300]), "walk": ([1] * 300, [100 + 7 * (i % 50) for i in range(300)]),
         "tiles": ([150, 200], [300, 200])}


# ------------------------------------------------------------------------------------------- tiles without keys ----
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pattern", [(300, 0), (200, 0, 0, 130), (0, 0, 90)])
def test_tiles_without_keys_between_others(nq, D, pattern):
    """Several tiles a CTA, those of requests without keys among them: queries of a tile meet its own keys only."""
    B = 60
    s = make(nq, [256] * B, [pattern[i % len(pattern)] for i in range(B)], 8, 8, D, 32, seed=D)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    out, lse = check(nq, s, workspace=ws)
    for _ in range(20):  # which CTA takes which tile differs from run to run
        again, lse_again = call(nq, s, workspace=ws, want_lse=True)
        assert torch.equal(again, out) and torch.equal(lse_again, lse)


# --------------------------------------------------------------------------------- weights far below the largest ----
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,t", [*FORMS.values(), ([1] * 2, [131073, 5000]), ([150, 90], [9000, 4000])])
def test_a_flat_tail_behind_one_early_peak(nq, n, t, D):
    """The first key is e^17.4 = 2^25.1 times as heavy as any other and its value is zero: the output is the tail's."""
    page = 64
    s = make(nq, n, t, 4, 1, D, page, seed=D)
    first = torch.cat([(torch.arange(x, device="cuda") == 0) for x in t])
    k = torch.zeros((sum(t), 1, D), device="cuda")
    k[first, :, 0] = 1.0
    v = torch.ones_like(k)
    v[first] = 0.0
    slots = torch.cat([s["table"][b].long()[torch.arange(x, device="cuda") // page] * page + torch.arange(x, device="cuda") % page
                       for b, x in enumerate(t)])
    nq.nq_kv_append_nvfp4(k.bfloat16(), v.bfloat16(), slots, s["cache"], s["gk"], s["gv"])
    kd, vd = K.decode(s["cache"][s["table"][0, 0]][None], D, page)
    key, value = float(kd[0, 0, 0, 0]) * float(s["gk"]), float(vd[0, 1, 0, 0]) * float(s["gv"])
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    scale = float(np.float32(17.4 / key))
    out, lse = call(nq, s, scale=scale, want_lse=True)
    tail = torch.cat([torch.arange(x - m, x, device="cuda") for m, x in zip(n, t)]).double()  # keys behind the first
    peak = scale * key
    w = np.exp(-peak)
    want = (value * tail * w / (1 + tail * w))[:, None, None]
    # As for any row (a weight's f16 half step and its exponent's float32 errors, the sums' over `tail` keys, the output's
    # bf16 half step); f16's smallest half step, 2^-25, beside a largest weight of 2^7 at least, for each key of the tail.
    eps = D * 2.0**-23 * peak + 2 * 2.0**-23 * peak + 2.0**-22
    err = want * (2.0**-11 + 2 * eps + 2 * (tail[:, None, None] + 1) * 2.0**-23) + 2.0**-32 * value * tail[:, None, None]
    d = (out.double() - want).abs()
    assert bool((d <= 2.0**-8 * (want + err) + err).all()), float((d / want.clamp(min=1e-300)).max())
    want = peak + torch.log1p(tail * w)[:, None]
    assert bool(((lse.double() - want).abs() <= eps + (tail[:, None] + 1) * 2.0**-23 + 2.0**-22 * (1 + want)).all())
    nq.nq_check_device_errors()


# ----------------------------------------------------------------------------------------- plans that do not fit ----
def test_a_plan_of_more_than_32_bits_of_tokens_is_cut(nq):
    B, T, page = 4, 8, 128
    width = (1 << 30) // page
    table = torch.full((B, width), -7, dtype=torch.int32, device="cuda")
    zero, head = i32([0] * B), i32([1])
    out = nq.nq_kv_plan(zero, i32([1 << 30] * B), table, i32([4, 5, 6]), head, T, page, free_head_out=head)
    with pytest.raises(nq.NQError, match="bit 3"):
        nq.nq_check_device_errors()
    cu, kv, pos, slots, _ = (x.tolist() for x in out)
    assert cu == [0, T, T, T, T] and kv == [1 << 30] * B
    assert pos == list(range(T)) and slots == list(range(5 * page, 5 * page + T))
    assert int(head) == 3  # the pages that the list still held
    assert table[0, :3].tolist() == [5, 6, -1] and bool((table[1:] == -1).all())


@pytest.mark.parametrize("in_place", [False, True])
def test_a_plan_takes_the_pages_that_are_left(nq, in_place):
    table = torch.full((3, 4), -7, dtype=torch.int32, device="cuda")
    free, head = i32([10, 11, 12]), i32([1])
    for step, (want, left) in enumerate([([[11, -7], [12, -1], [-1, -7]], 3), ([[11, -1], [12, -1], [-1, -1]], 3)]):
        out = nq.nq_kv_plan(i32([16 * step, 32 * step, 16 * step]), i32([16, 32 if step == 0 else 0, 16]), table, free, head,
                            64 if step == 0 else 32, 16, free_head_out=head if in_place else None)
        with pytest.raises(nq.NQError, match="bit 3"):
            nq.nq_check_device_errors()
        head = out[4]
        assert int(head) == left and table[:, :2].tolist() == want and bool((table[:, 2:] == -7).all())


def test_a_plan_of_more_than_32_bits_of_pages_is_cut(nq):
    """66 requests of 2^26 pages each."""
    B, T, page = 66, 5, 16
    width = (1 << 30) // page
    table = torch.empty((B, width), dtype=torch.int32, device="cuda")
    table[-1] = -7
    out = nq.nq_kv_plan(i32([0] * B), i32([1 << 30] * B), table, i32([4, 5, 6]), i32([0]), T, page)
    with pytest.raises(nq.NQError, match="bit 3"):
        nq.nq_check_device_errors()
    cu, kv, pos, slots, head = (x.tolist() for x in out)
    assert cu == [0] + [T] * B and kv == [1 << 30] * B and head == [3]
    assert pos == list(range(T)) and slots == list(range(4 * page, 4 * page + T))
    assert table[0, :4].tolist() == [4, 5, 6, -1] and bool((table[:31, 3:] == -1).all())
    assert bool((table[-1] == -7).all())  # past the 2^31 - 1 pages that a plan lays out


# -------------------------------------------------------------------------------- scales and queries at their ends ----
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,t", [([1] * 3, [700, 0, 300]), ([1] * 300, [(7 * i) % 350 for i in range(300)]),
                                 ([150, 200], [300, 120]), ([1], [20000]), ([150], [9000])])
def test_a_nan_scale_is_seen(nq, n, t, D):
    s = make(nq, n, t, 8, 2, D, 16, seed=D)
    keys = torch.cat([torch.arange(x - m, x, device="cuda") >= 0 for m, x in zip(n, t)])
    nan = f32(float("nan"))
    for gk, gv in ((nan, s["gv"]), (s["gk"], nan)):
        out, lse = call(nq, {**s, "gk": gk, "gv": gv}, want_lse=True)
        assert bool(out[keys].isnan().all()) and not out[~keys].any()
        assert bool(torch.isneginf(lse[~keys]).all())
        if gk is nan:
            assert bool(lse[keys].isnan().all())
        else:
            assert bool(lse[keys].isfinite().all())
    nq.nq_check_device_errors()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("power", [100, 120, 130])
def test_small_queries_of_large_keys(nq, form, D, power):
    """Queries down to bf16's subnormal numbers under a key scale that is as large: scores of ordinary size."""
    s = make(nq, *FORMS[form], 8, 2, D, 16, seed=power)
    s["q"] = (s["q"].double() * 2.0**-power).bfloat16()
    assert bool((s["q"] != 0).any())
    s["gk"] = (s["gk"].double() * 2.0**power).float()
    check(nq, s)


# ------------------------------------------------------------------------------------------------- other streams ----
def test_a_workspace_of_the_default_stream(nq, monkeypatch):
    """Handle 0 is the default stream: the workspace is zeroed there, in front of the kernel, whatever stream is current."""
    s = make(nq, *FORMS["walk"], 8, 2, 128, 16, seed=19)
    want, want_lse = call(nq, s, want_lse=True)
    torch.cuda.synchronize()
    made, zeros = [], torch.zeros

    def noted(*args, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return zeros(*args, **kw)
    side = torch.cuda.Stream()
    monkeypatch.setattr(torch, "zeros", noted)
    for current in (torch.cuda.default_stream(), side):
        for handle in (0, torch.cuda.default_stream(), side, side.cuda_stream):
            with torch.cuda.stream(current):
                out, lse = call(nq, s, out=torch.empty_like(want), lse=torch.empty_like(want_lse), stream=handle)
            assert made.pop() == (side.cuda_stream if handle in (side, side.cuda_stream) else 0) and not made
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_results_belong_to_the_stream_of_the_call(nq):
    """The current stream still writes to memory that it has given back when a call on another stream makes its results."""
    D, page = 128, 16
    s = make(nq, [1] * 6, [900] * 6, 8, 2, D, page, seed=14)
    table, lens, head = s["table"].clone(), i32([900] * 6), i32([0])
    free = torch.arange(40, dtype=torch.int32, device="cuda")
    slots = torch.arange(2000, device="cuda")

    def results(**on):
        out = call(nq, s, want_lse=True, **on)
        kv = nq.nq_kv_gather_nvfp4(s["cache"], slots, s["gk"], s["gv"], D, **on)
        return *out, *kv, *nq.nq_kv_plan(lens, i32_one, table, free, head, 6, page, **on)
    i32_one = i32([1] * 6)
    want = results()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda._sleep(1 << 28)
        old = [torch.full_like(w, 77) for w in want for _ in range(2)]
        del old  # its memory is the current stream's again, and the fills are still to come
        got = results(stream=handle)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(torch.nan_to_num(g.float(), nan=7e9), torch.nan_to_num(w.float(), nan=7e9))
    nq.nq_check_device_errors()


# -------------------------------------------------------------- every form of the kernel for few rows, many requests ----
# (query heads, kv heads, D, new tokens at most): 4 to 60 rows a request and kv head, and so one to four row tiles of a
# warp, one to three tiles a request
WALKS = [(8, 2, 64, 1), (8, 2, 64, 3), (8, 2, 64, 6), (8, 2, 64, 11), (12, 2, 64, 10), (8, 2, 128, 3), (8, 2, 128, 7),
         (8, 2, 128, 11), (4, 2, 256, 4), (4, 2, 256, 6), (8, 2, 256, 6)]


def ragged(nq, heads, kv_heads, D, most, B=150, least=0, seed=0):
    """B requests of 0 ... `most` new tokens (two thirds of them of `most`) and of lengths from `least` on."""
    rng = np.random.default_rng(seed + D + most)
    n = [most if x else int(rng.integers(0, most + 1)) for x in rng.random(B) < 0.67]
    t = [max(least, int(x)) for x in rng.integers(0, 500, B)]
    t[:4] = [1, 16, 17, 1500]
    return make(nq, n, t, heads, kv_heads, D, 16, seed=seed, tail=3)


@pytest.mark.parametrize("heads,kv_heads,D,most", WALKS)
@pytest.mark.parametrize("window,causal", [(0, True), (90, True), (0, False), (200, False), (1, True)])
def test_many_requests_of_few_rows(nq, heads, kv_heads, D, most, window, causal):
    check(nq, ragged(nq, heads, kv_heads, D, most), window=window, causal=causal)


@pytest.mark.parametrize("heads,kv_heads,D,most", WALKS)
def test_many_requests_at_any_address(nq, heads, kv_heads, D, most):
    s = ragged(nq, heads, kv_heads, D, most, seed=1)
    T, H, rows = s["q"].shape[0], heads, sum(s["n"])
    want, want_lse = call(nq, s, want_lse=True)
    raw = torch.full((T * (H * D + 3) + 5,), 9.0, dtype=torch.bfloat16, device="cuda")
    odd = raw[5:].view(T, H * D + 3)[:, :H * D].view(T, H, D)  # rows that start off every alignment
    odd.copy_(s["q"])
    out = Guarded(T, H * D, torch.bfloat16, pad=5)
    lse = torch.full((T, H + 3), 9.0, device="cuda")
    call(nq, {**s, "q": odd}, out=out.view.view(T, H, D), lse=lse[:, :H])
    assert torch.equal(out.view.reshape(T, H, D)[:rows], want[:rows]) and out.guards_intact()
    assert torch.equal(lse[:rows, :H], want_lse[:rows]) and bool((lse[:, H:] == 9.0).all()) and bool((lse[rows:] == 9.0).all())
    out = torch.empty((H, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    call(nq, {**s, "q": s["q"].transpose(0, 1).contiguous().transpose(0, 1)}, out=out)
    assert torch.equal(out[:rows], want[:rows])


@pytest.mark.parametrize("heads,kv_heads,D,most", WALKS)
def test_many_requests_with_pages_outside_the_cache(nq, heads, kv_heads, D, most):
    """First, middle and last pages without a page in the cache: as if their keys were not there (all keys in sight)."""
    s = ragged(nq, heads, kv_heads, D, most, least=60, seed=2)
    rng = np.random.default_rng(3)
    bad, rest, left = s["table"].clone(), torch.full_like(s["table"], 1 << 30), []
    for b, t in enumerate(s["t"]):
        pages = -(-t // 16)
        gone = {0: [], 1: [0], 2: [pages - 1], 3: sorted({0, pages // 3, pages // 2}), 4: list(range(pages)),
                5: sorted(rng.permutation(pages)[:pages // 2].tolist())}[b % 6]
        keep = [p for p in range(pages) if p not in gone]
        for p in gone:
            bad[b, p] = [-1, s["cache"].shape[0], 1 << 30][p % 3]
        rest[b, :len(keep)] = s["table"][b, keep]
        left.append(t - sum(min(16, t - 16 * p) for p in gone))
    out, lse = call(nq, {**s, "table": bad}, want_lse=True, flags=nq.FLAG_NONCAUSAL)
    with pytest.raises(nq.NQError, match="bit 2"):
        nq.nq_check_device_errors()
    k, v = K.decode(s["cache"], D, 16)
    o, l, tol, tol_lse = K.attention(s["q"], k, v, float(s["gk"]), float(s["gv"]), rest, left, s["cu"].tolist(), 16, D**-0.5,
                                     causal=False)
    rows = sum(s["n"])
    assert bool(((out[:rows].double() - o[:rows]).abs() <= tol[:rows]).all())
    empty = torch.isneginf(l[:rows])
    assert bool(empty.any()) and torch.equal(torch.isneginf(lse[:rows]), empty)
    assert bool((torch.where(empty, 0.0, (lse[:rows].double() - l[:rows]).abs()) <= tol_lse[:rows]).all())


# ------------------------------------------------------------------------------------------ groups and empty requests ----
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,kv_heads", [(3, 2), (7, 1), (33, 1), (129, 1), (1024, 1)])
@pytest.mark.parametrize("B", [3, 40, 300])
def test_groups_of_any_size_among_empty_requests(nq, D, group, kv_heads, B):
    """Three requests that have rows; the others hold keys only, as those of a padded batch (which makes the average of
    rows small, and so sends groups of up to 1024 heads to the kernel for few rows)."""
    n, t = [0] * B, [5 + b % 40 for b in range(B)]
    for b, (m, x) in zip((0, B // 2, B - 1), ((2, 300), (1, 77), (3, 2))):
        n[b], t[b] = m, x
    s = make(nq, n, t, group * kv_heads, kv_heads, D, 16, seed=group, tail=2)
    check(nq, s)
    check(nq, s, window=20)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_before_the_first_request_are_left(nq, form, D):
    s = make(nq, *FORMS[form], 8, 2, D, 16, seed=21)
    want, want_lse = call(nq, s, want_lse=True)
    q = torch.cat([torch.full_like(s["q"][:3], float("nan")), s["q"]])
    out, lse = torch.full_like(q, 123.0), torch.full(q.shape[:2], 123.0, device="cuda")
    call(nq, {**s, "q": q, "cu": s["cu"] + 3}, out=out, lse=lse)
    assert bool((out[:3] == 123.0).all()) and bool((lse[:3] == 123.0).all())
    if form == "chunks":  # the same parts; elsewhere rows and parts fall differently
        assert torch.equal(out[3:], want) and torch.equal(lse[3:], want_lse)
    o, l, tol, tol_lse = K.attention(s["q"], *K.decode(s["cache"], D, 16), float(s["gk"]), float(s["gv"]), s["table"], s["t"],
                                     s["cu"].tolist(), 16, D**-0.5)
    assert bool(((out[3:].double() - o).abs() <= tol).all()) and bool(((lse[3:].double() - l).abs() <= tol_lse).all())
    nq.nq_check_device_errors()


# ---------------------------------------------------------------------------------------------------- the binding ----
def test_scales_of_one_element_in_any_shape(nq):
    s = make(nq, [1, 2], [20, 40], 4, 2, 128, 16, seed=22)
    want, _ = call(nq, s)
    slots = torch.arange(32, device="cuda")
    back = nq.nq_kv_gather_nvfp4(s["cache"], slots, s["gk"], s["gv"], 128)
    cache, again = torch.zeros_like(s["cache"]), torch.zeros_like(s["cache"])
    nq.nq_kv_append_nvfp4(*back, slots, cache, s["gk"], s["gv"])
    for shape in ((), (1, 1), (1, 1, 1)):
        gk, gv = s["gk"].reshape(shape), s["gv"].reshape(shape)
        assert torch.equal(call(nq, {**s, "gk": gk, "gv": gv})[0], want)
        got = nq.nq_kv_gather_nvfp4(s["cache"], slots, gk, gv, 128)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, back))
        nq.nq_kv_append_nvfp4(*back, slots, again.zero_(), gk, gv)
        assert torch.equal(again, cache)


# ------------------------------------------------------------------------------------------- calls beside one another ----
def test_calls_at_the_same_time(nq):
    """Every form of the kernels on four streams at once, a workspace each: the bits that each gives alone."""
    batches = [make(nq, *FORMS[f], 8, 2, D, 16, seed=23) for D in (64, 128, 256) for f in FORMS]
    batches += [make(nq, [400] * 6, [700 + 60 * i for i in range(6)], 16, 4, D, 64, seed=24) for D in (128, 256)]
    want = [call(nq, s, want_lse=True) for s in batches]
    streams = [torch.cuda.Stream() for _ in range(4)]
    spaces = [torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[tuple(torch.empty_like(x) for x in w) for w in want] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(len(batches)):
            for j, stream in enumerate(streams):
                k = (i + 3 * j) % len(batches)
                call(nq, batches[k], out=outs[j][k][0], lse=outs[j][k][1], workspace=spaces[j], stream=stream)
        torch.cuda.synchronize()
        for got in outs:
            for (o, l), (ow, lw) in zip(got, want):
                assert torch.equal(o, ow) and torch.equal(l, lw)
                o.fill_(9.0)
                l.fill_(9.0)
        torch.cuda.synchronize()
    nq.nq_check_device_errors()


@pytest.mark.parametrize("new", [[1] * 40, [3, 0, 90] * 4, [150, 1]])
def test_a_step_whose_launches_overlap(nq, new):
    """Plan, append, attention and gather, each of which may start while the one before ends, captured and replayed."""
    H, G, D, page, B = 2, 4, 128, 16, len(new)
    T = sum(new) + 3
    gen = torch.Generator("cuda").manual_seed(B)
    gk = f32(4.6 / 2688)
    qkv = torch.randn((T, H * G + 2 * H, D), generator=gen, device="cuda").bfloat16()
    q, k, v = qkv.split_with_sizes((H * G, H, H), 1)
    steps, pages = 6, 6 * sum(new) + B
    free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    ws = torch.zeros(nq.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def server():
        return dict(cache=torch.zeros(nq.kv_cache_shape(pages, H, D, page), dtype=torch.uint8, device="cuda"),
                    table=torch.full((B, -(-steps * max(new) // page)), -1, dtype=torch.int32, device="cuda"), head=i32([0]),
                    lens=i32([0] * B))

    def step(s, flags):
        cu, lens, _, slots, _ = nq.nq_kv_plan(s["lens"], i_new, s["table"], free, s["head"], T, page, free_head_out=s["head"],
                                              flags=flags)
        nq.nq_kv_append_nvfp4(k, v, slots, s["cache"], gk, gk, flags=flags)
        out, _ = nq.nq_attention_nvfp4_kv(q, s["cache"], s["table"], lens, cu, gk, gk, workspace=ws, flags=flags,
                                          out=s.setdefault("out", torch.zeros_like(q)))
        back = nq.nq_kv_gather_nvfp4(s["cache"], slots, gk, gk, D, flags=flags)
        s["lens"].copy_(lens)
        return out, *back
    i_new = i32(new)
    plain, graphed = server(), server()
    step({**server()}, nq.FLAG_PDL)  # everything is loaded before the capture
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    graphed["out"] = torch.zeros_like(q)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        got = step(graphed, nq.FLAG_PDL)
    for _ in range(steps):
        graph.replay()
        want = step(plain, 0)
        for name in ("cache", "table", "head", "lens"):
            assert torch.equal(plain[name], graphed[name]), name
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert plain["lens"].tolist() == [steps * n for n in new]
    nq.nq_check_device_errors()
