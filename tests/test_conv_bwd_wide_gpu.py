"""The convolution's backward over so many channels that its sums take several launches."""
import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner
from _layer_ref import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W", [4, 8])
def test_conv_bwd_wide(W):
    """Channels are apart from each other: some at the ends, and where one launch's columns end, show all."""
    D, b, L = 2 ** 28 // (W + 1) // 64 * 64 + 64, 2, 1   # (more steps of so many channels are refused)
    banner("conv bwd wide %d" % D)
    g = torch.Generator(device="cuda").manual_seed(W)
    x = torch.randn(b, L, D, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(b, L, D, generator=g, device="cuda", dtype=torch.bfloat16)
    w, bias = torch.randn(D, W, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    out = ssm.causal_conv1d_bwd(dy, x, w, bias=bias, silu=True)
    cols = set(range(40)) | set(range(D - 40, D))
    for line in range(2 ** 26, (W + 1) * D, 2 ** 26):
        cols |= {(line + i) % D for i in range(-40, 40)}
    cols = torch.tensor(sorted(cols))
    pick = lambda t: t.index_select(-1, cols.cuda()).cpu()  # noqa: E731
    rows = lambda t: t.index_select(0, cols.cuda()).cpu()  # noqa: E731
    r = ref.conv_bwd(pick(dy), pick(x), rows(w), rows(bias), True)
    check(pick(out["dx"]), r["dx"], r["mag_dx"], ref.rel_conv_bwd(W, r["amax"]), "dx")
    rel = ref.rel_conv_sum(W, r["amax"], L, b)
    check(rows(out["dweight"]), r["dweight"], r["mag_dweight"], rel, "dweight")
    check(rows(out["dbias"]), r["dbias"], r["mag_dbias"], rel, "dbias")
