"""The 4-bit key/value cache without a GPU: refusals of the C ABI, the sizes it
states, and the byte places of an atom."""
import re

import numpy as np
import pytest

import kv_helpers as K
from test_abi import FAKE, HEADER, nq  # noqa: F401  (fixture)


def attend(nq, q=FAKE, heads=8, kv_heads=2, d=128, page=16, T=4, B=2, width=4, ld_table=4, pages=9, stride=None,
           ws=FAKE, ws_bytes=None, scale=0.1, window=0, flags=0, qt=None, qh=None, ld_lse=8, lse=None, cache=FAKE,
           table=FAKE):
    stride = kv_heads * page * d * 9 // 8 if stride is None else stride
    ws_bytes = nq.ATTENTION_WORKSPACE_BYTES if ws_bytes is None else ws_bytes
    return nq.lib.nq_attention_nvfp4_kv(q, heads * d if qt is None else qt, d if qh is None else qh, cache, stride, pages,
                                        table, ld_table, width, FAKE, FAKE, FAKE, FAKE, FAKE, heads * d, d, lse, ld_lse,
                                        ws, ws_bytes, T, B, heads, kv_heads, d, page, scale, window, flags, None)


def test_attention_refusals(nq):
    INV, UNS = nq.NQ_ERR_INVALID_ARGUMENT, nq.NQ_ERR_UNSUPPORTED
    assert attend(nq, d=96) == UNS and b"head dimension" in nq.lib.nq_last_error()
    assert attend(nq, page=8) == UNS and attend(nq, page=24) == UNS and attend(nq, page=256) == UNS
    assert attend(nq, heads=7) == INV and attend(nq, heads=1) == INV
    assert attend(nq, kv_heads=0) == INV
    assert attend(nq, heads=1025, kv_heads=1, ld_lse=1025) == UNS
    assert attend(nq, q=None) == INV and attend(nq, cache=None) == INV and attend(nq, table=None) == INV
    assert attend(nq, ws=None) == INV and attend(nq, ws=FAKE + 8) == INV
    assert attend(nq, ws_bytes=1 << 20) == INV and b"WORKSPACE" in nq.lib.nq_last_error()
    assert attend(nq, scale=float("inf")) == INV and attend(nq, scale=float("nan")) == INV
    assert attend(nq, window=-1) == INV
    assert attend(nq, ld_table=3) == INV
    assert attend(nq, stride=16) == INV and attend(nq, cache=FAKE + 4) == INV
    assert attend(nq, stride=2 * 16 * 128 * 9 // 8 + 8) == INV
    assert attend(nq, flags=nq.FLAG_UE8M0) == INV and attend(nq, flags=1 << 30) == INV
    assert attend(nq, qt=64) == INV and attend(nq, qh=64) == INV
    assert attend(nq, lse=FAKE, ld_lse=7) == INV
    assert attend(nq, T=-1) == INV and attend(nq, B=-1) == INV
    assert attend(nq, T=1 << 31) == UNS
    assert attend(nq, width=1 << 27, ld_table=1 << 27) == UNS
    assert attend(nq, T=0, q=None) == nq.NQ_OK and attend(nq, B=0, q=None) == nq.NQ_OK


def test_noncausal_is_an_attention_flag(nq):
    L = nq.lib
    assert L.nq_per_token_group_quant_fp8(FAKE, 256, FAKE, 256, FAKE, 2, 4, 256, 128, nq.FLAG_NONCAUSAL,
                                          None) == nq.NQ_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", ["nq_kv_append_nvfp4", "nq_kv_gather_nvfp4"])
def test_copy_refusals(nq, name):
    INV, UNS = nq.NQ_ERR_INVALID_ARGUMENT, nq.NQ_ERR_UNSUPPORTED

    def call(k=FAKE, v=FAKE, kt=256, kh=128, slots=FAKE, gk=FAKE, cache=FAKE, stride=2 * 16 * 144, pages=5, T=4, H=2,
             d=128, page=16, flags=0):
        if name == "nq_kv_append_nvfp4":
            return nq.lib.nq_kv_append_nvfp4(k, kt, kh, v, kt, kh, slots, gk, FAKE, cache, stride, pages, T, H, d, page,
                                             flags, None)
        return nq.lib.nq_kv_gather_nvfp4(cache, stride, pages, slots, gk, FAKE, k, kt, kh, v, kt, kh, T, H, d, page,
                                         flags, None)
    assert call(d=80) == UNS and call(page=1) == UNS
    for bad in ("k", "v", "slots", "gk", "cache"):
        assert call(**{bad: None}) == INV, bad
    assert call(T=-1) == INV and call(H=0) == INV and call(pages=-1) == INV
    assert call(kt=128) == INV and call(kh=64) == INV  # rows that overlap
    assert call(cache=FAKE + 1) == INV and call(stride=2 * 16 * 144 - 16) == INV
    assert call(flags=nq.FLAG_SCALE_DIV) == INV
    assert call(T=1 << 31) == UNS
    assert call(T=0, k=None, v=None, slots=None) == nq.NQ_OK


def test_plan_refusals(nq):
    INV, UNS = nq.NQ_ERR_INVALID_ARGUMENT, nq.NQ_ERR_UNSUPPORTED
    A = [0x10000 * (i + 1) for i in range(10)]

    def call(B=4, T=8, page=16, width=4, ld=4, flags=0, n_free=3, **at):
        p = dict(cached=A[0], new=A[1], table=A[2], free=A[3], head=A[4], head_out=A[5], cu=A[6], kv=A[7], pos=A[8],
                 slots=A[9])
        p.update(at)
        return nq.lib.nq_kv_plan(p["cached"], p["new"], p["table"], ld, width, p["free"], n_free, p["head"],
                                 p["head_out"], p["cu"], p["kv"], p["pos"], p["slots"], B, T, page, flags, None)
    for bad in ("cached", "new", "table", "free", "head", "head_out", "cu", "kv", "pos", "slots"):
        assert call(**{bad: None}) == INV, bad
    assert call(page=0) == UNS and call(page=48) == UNS
    assert call(B=nq.NQ_KV_MAX_REQUESTS + 1) == UNS
    assert call(B=-1) == INV and call(T=-1) == INV and call(n_free=-1) == INV
    assert call(ld=3) == INV and call(width=1 << 28, ld=1 << 28) == UNS
    assert call(flags=nq.FLAG_E5M2) == INV
    # other CTAs still read the lengths when the first results are written
    assert call(kv=A[0]) == INV and call(cu=A[0] + 12) == INV and call(kv=A[1] - 12) == INV
    assert b"overlap" in nq.lib.nq_last_error()


def test_constants_match_header(nq):
    text = open(HEADER).read()
    assert re.search(r"#define NQ_KV_MAX_REQUESTS (\d+)", text).group(1) == str(nq.NQ_KV_MAX_REQUESTS)
    m = re.search(r"#define NQ_ATTENTION_WORKSPACE_BYTES \((\d+) << (\d+)\)", text)
    assert int(m.group(1)) << int(m.group(2)) == nq.ATTENTION_WORKSPACE_BYTES
    m = re.search(r"#define NQ_FLAG_NONCAUSAL \(1u << (\d+)\)", text)
    assert 1 << int(m.group(1)) == nq.FLAG_NONCAUSAL
    for H, d, page in ((1, 64, 16), (8, 128, 64), (5, 256, 128)):
        shape = nq.kv_cache_shape(7, H, d, page)
        assert shape == (7, H, page // 16 * 18 * d)
        assert nq.lib.nq_kv_page_bytes(H, d, page) == shape[1] * shape[2]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_atom_places_cover_every_byte_once(D):
    kc, vc, ks, vs = K.places(D)
    assert np.array_equal(np.sort(np.concatenate([a.ravel() for a in (kc, vc, ks, vs)])), np.arange(18 * D))
    assert kc.max() < 8 * D <= vc.min() and vc.max() < 16 * D <= ks.min() and ks.max() < 17 * D <= vs.min()


def test_plan_reference_by_hand():
    table = np.full((3, 3), -1, np.int32)
    table[1, 0] = 9
    cu, kv, pos, slots, head = K.plan([0, 15, 0], [17, 2, 0], table, [4, 5, 6, 7], 1, 21, 16)
    assert cu.tolist() == [0, 17, 19, 19] and kv.tolist() == [17, 17, 0] and head == 4
    assert table.tolist() == [[5, 6, -1], [9, 7, -1], [-1, -1, -1]]
    assert slots.tolist() == [*range(80, 96), 96, 9 * 16 + 15, 7 * 16, -1, -1]
    assert pos.tolist() == [*range(17), 15, 16, -1, -1]
