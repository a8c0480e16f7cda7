"""GPU tests of the 4-bit key/value cache at its edges."""
import numpy as np
import pytest
import torch

import kv_helpers as K
from test_gpu_kv import check, f32, i32, make, nq  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def call(nq, s, **more):
    return nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"], **more)


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
