"""The low-rank adapters without a GPU: what the entry points refuse on the host."""
import ctypes as C
import os

import pytest
import torch

import sharded_gemm_alltosharded_amd as sg

PTR = 0x1000  # never dereferenced: the calls below fail before


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sg.LIB_PATH):
        pytest.skip("library not built")
    return sg.lib()


def err(L):
    return L.sg_last_error().decode()


def test_plan_refuses(L):
    assert L.sg_adapter_plan(PTR, -1, 1, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_adapter_plan(PTR, 1, 0, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_adapter_plan(PTR, 1, 1025, PTR, None) == sg.ERR_UNSUPPORTED and "1024 adapters" in err(L)
    assert L.sg_adapter_plan(PTR, (1 << 25) + 1, 1, PTR, None) == sg.ERR_UNSUPPORTED
    assert L.sg_adapter_plan(None, 1, 1, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_adapter_plan(PTR, 1, 1, None, None) == sg.ERR_INVALID_ARG
    assert L.sg_adapter_plan_ints(-1, 1) == 0 and L.sg_adapter_plan_ints(1, 0) == 0
    assert L.sg_adapter_plan_ints(1, 1025) == 0 and L.sg_adapter_plan_ints((1 << 25) + 1, 1) == 0


@pytest.mark.parametrize("T,n", [(0, 1), (1, 1), (16, 32), (63, 1), (64, 1), (4096, 8), (5000, 1024)])
def test_plan_holds_every_grouping(L, T, n):
    """Offsets, rows and as many tiles as the tokens can make up, however they fall."""
    height = 64 if T >= 32 * (n + 1) else 16
    ints = L.sg_adapter_plan_ints(T, n)
    tiles = (ints - (n + 2 + 2 * T + 3) // 4 * 4) // 4
    groups = min(T, n + 1)
    # the most tiles: every group but one has a single row in its last tile
    assert tiles >= (groups + (T - groups) // height if T else 0)


def test_missing_layers_are_refused(L):
    ad = sg._AdaptersArg(PTR, PTR, None, 2, 8)
    ref = C.byref(ad)
    assert L.sg_adapted_all_to_sharded(None, ref, PTR, PTR, 1, PTR, 1, 0, 1, PTR, 0, None) == sg.ERR_INVALID_ARG
    assert "layer is NULL" in err(L)
    assert L.sg_adapted_sharded_to_all(None, ref, PTR, PTR, 1, PTR, 1, PTR, 0, None) == sg.ERR_INVALID_ARG
    for f in (L.sg_adapted_all_to_sharded_backward, L.sg_adapted_sharded_to_all_backward):
        assert f(None, ref, PTR, PTR, PTR, 1, PTR, 1, PTR, PTR, 1, PTR, 0, None) == sg.ERR_INVALID_ARG
    assert L.sg_adapted_workspace(None, ref, 4) == 0 and L.sg_adapted_backward_workspace(None, ref, 4) == 0


def test_binding_refuses():
    with pytest.raises(sg.ShardGemmError, match="which is None"):
        sg.adapter_plan(None, 2)
    with pytest.raises(sg.ShardGemmError, match="dtype"):
        sg.adapter_plan(torch.zeros(4, dtype=torch.int64), 2)
    with pytest.raises(sg.ShardGemmError, match="shape"):
        sg.adapter_plan(torch.zeros((4, 1), dtype=torch.int32), 2)
