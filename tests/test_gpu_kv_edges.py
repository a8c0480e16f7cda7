"""GPU tests of the 4-bit key/value cache at its edges."""
import pytest
import torch

from test_gpu_kv import check, make, nq  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def call(nq, s, **more):
    return nq.nq_attention_nvfp4_kv(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"], s["gk"], s["gv"], **more)


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
