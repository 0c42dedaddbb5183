"""The latent page cache's kernels one by one: shapes that select each of them, on data that reaches their rarer paths."""
import numpy as np
import pytest
import torch

from test_gpu_mla import BF16, F32, _append_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kda_delta_rule_gb300 import kda
    kda.kda_device_errors()
    return kda


@pytest.mark.parametrize("through_ctypes", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 1), (1, 1)])
def test_append_rotates_in_place(K, T, H, dtype, through_ctypes):
    """The decode step of one sequence, and single heads: the stride of an axis of one entry has no say."""
    pages, slots, pos, table, fused, qs, w = _append_case(T, H, 128, 64, dtype, T + H, 2, 16)
    page = np.int64(16) if through_ctypes else 16
    args = (page, slots.cuda(), pos.cuda(), table.cuda(), fused.cuda()[:, :128], fused.cuda()[:, 128:])
    q = qs[:, :, 128:].contiguous().cuda()
    a, b = pages.cuda(), pages.cuda()
    out = K.kda_mla_append(a.view(torch.uint8), *args, q_pe=q)
    assert K.kda_mla_append(b.view(torch.uint8), *args, q_pe=q, q_pe_out=q) is q
    assert torch.equal(out, q) and torch.equal(a, b)
    assert K.kda_device_errors() == 0
