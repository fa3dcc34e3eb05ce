"""Calls of attention over latent rows beyond what one call may ask for: refused as a whole."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_units_than_a_call_may_have():
    from out_proj_block_gb300 import build
    build.build()
    from out_proj_block_gb300 import cfa
    B, H, ps, width = 128, 128, 4096, 1 << 18
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros(B, H, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.full((B, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), 5.0, device="cuda")
    pages = torch.zeros(1, ps, 576, dtype=torch.bfloat16, device="cuda")
    tables = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    with cfa.Latent(B, B, H, ps) as plan:
        # 2^30 rows for each of 128 tiles: 2^30 + 256 units
        plan.attend(q, ints(list(range(B + 1))), ints([1 << 30] * B), tables, pages, out, lse=lse)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert torch.all(out == 5.0) and torch.all(lse == 5.0)
        plan.attend(q, ints(list(range(B + 1))), ints([ps] * B), tables, pages, out, lse=lse)  # the next call is as ever
        assert plan.status() == cfa.CFA_OK
        assert not out.any() and torch.all((lse - 8.317766166719343).abs() < 1e-4)  # ln 4096
