"""Low-rank adapters where calls meet: captures of other threads, the widest tiles."""
import math
import threading

import pytest
import torch

import moe_ref as ref
import sharded_gemm_alltosharded_amd as sg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    sg.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


@pytest.mark.parametrize("i,o", [(72, 104), (96, 80)])  # stored row-major; in fragments that are not the tiles'
def test_first_adapted_call_while_another_thread_captures(i, o):
    g = gen(i)
    T, n, r = 40, 2, 8
    w = normal(g, (o, i), BF, 0.1).cuda()
    keep, first, same = (sg.shard_linear(w, "all-to-sharded", P=2) for _ in range(3))
    ad = sg.Adapters(normal(g, (n, r, i), BF, 0.1).cuda(), normal(g, (n, o, r), BF, 0.1).cuda())
    x, dy = normal(g, (T, i), BF).cuda(), normal(g, (2, T, o // 2), BF).cuda()
    plan = sg.adapter_plan(torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda(), n)

    def both(layer):
        return (sg.adapted_all_to_sharded(layer, x, ad, plan),
                *sg.adapted_all_to_sharded_backward(layer, x, dy, ad, plan))

    want, plain = both(same), sg.all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hold = torch.empty(8, device="cuda")  # keeps 2 MiB of torch's, whose own allocation would end the capture
    torch.cuda.synchronize()
    capturing, errors, got = threading.Event(), [], []

    def call():
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(side):  # (a wait of torch's own would end it, too)
                if capturing.wait(60):
                    got.extend(both(first))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    other = threading.Thread(target=call)
    other.start()
    with torch.cuda.graph(graph):
        capturing.set()
        other.join()
        sg.all_to_sharded(keep, x, out=out)
    side.synchronize()
    assert not errors, errors
    assert len(got) == 4 and all(torch.equal(a, b) for a, b in zip(got, want))
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain)
    del hold


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mode,i,o", [(0, 64, 96), (0, 80, 64), (1, 64, 96), (1, 96, 64)])
def test_first_backward_call_captured(mode, i, o, dtype):
    """A backward call captured before the layer has its transposed copy: the vector units' sums."""
    g = gen(i + o + mode)
    B, P = 20, 2
    w = normal(g, (o, i), dtype, 1 / math.sqrt(o))
    layer = sg.shard_linear(w.cuda(), mode, P=P)
    dys = [normal(g, (P, B, o // P) if mode == 0 else (B, o), dtype).cuda() for _ in range(3)]
    dy, graph = dys[0].clone(), torch.cuda.CUDAGraph()
    back = sg.all_to_sharded_backward if mode == 0 else sg.sharded_to_all_backward
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, _ = back(layer, None, dy, need_dw=False, dx_dtype=F32)
    for k in (1, 2, 0):
        dy.copy_(dys[k])
        graph.replay()
        eager, _ = back(layer, None, dys[k], need_dw=False, dx_dtype=F32)
        torch.cuda.synchronize()
        full = dys[k].double().cpu()
        if mode == 0:
            full = full.transpose(0, 1).flatten(1)
        want, mag = full @ w.double(), full.abs() @ w.double().abs()
        if mode == 1:
            want, mag = (v.view(B, P, i // P).transpose(0, 1) for v in (want, mag))
        for got, name in ((out, "captured"), (eager, "eager")):
            ref.close(got, want, ref.sum_bound(mag, o), name)
