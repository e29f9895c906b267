"""A cluster whose CTAs read one another's partial results: once one of them has given up a wait, none writes.  The
self-test ends as the few-tile kernel of the dense layer does, with the same helper; a wait that nothing completes
runs out after 20 ms and is recorded."""

import pytest
import torch

import fp8_transformer_gb300 as te

b = te.binding


def test_arguments():
    f = te.lib().te_selftest_cluster_abort
    for limit, rank, out in ((0, 0, 64), (-1, 0, 64), (1000001, 0, 64), (10, -2, 64), (10, 8, 64), (10, 0, None), (10, 0, 66)):
        assert f(limit, rank, out, None) == b.TE_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [0, 3, 7])
def test_no_cta_writes_once_one_has_given_up(rank):
    torch.cuda.synchronize()
    assert te.get_device_status() == b.TE_OK
    out = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    te.selftest_cluster_abort(out, rank)
    assert te.get_device_status() == b.TE_ERR_TIMEOUT
    assert out.tolist() == [0] * 8
    te.selftest_cluster_abort(out, -1)
    assert te.get_device_status() == b.TE_OK
    assert out.tolist() == [1] * 8
