"""Slot moves of rows so wide that a launch's workgroups do not cover them."""
import pytest
import torch

import selective_state_space_60_amd as ssm
from _gpu import banner

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,row,moves", [(torch.bfloat16, 2 ** 27 - 1, 17), (torch.bfloat16, 2 ** 26 + 3, 1025),
                                             (torch.float32, 2 ** 26 + 1, 1025), (torch.float32, 2 ** 27 - 1, 40)])
def test_move_wide_rows(dtype, row, moves):
    """Two slots change places, a third is cleared; the other moves go nowhere."""
    banner("move wide %s %d %d" % (dtype, row, moves))
    pool = torch.empty(3, row, dtype=dtype, device="cuda")
    index = torch.arange(row, device="cuda", dtype=torch.int32)
    first, second = (index % 127).to(dtype), (-1 - index % 113).to(dtype)
    pool[0], pool[1], pool[2] = first, second, 5
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    ssm.state_move(pool, i32([1, 0, -1] + [0] * (moves - 3)), i32([0, 1, 2] + [-1] * (moves - 3)))
    assert torch.equal(pool[0], second) and torch.equal(pool[1], first) and not bool(pool[2].any())
