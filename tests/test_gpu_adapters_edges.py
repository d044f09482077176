"""Low-rank adapters where calls meet: captures of other threads, the widest tiles."""
import math
import threading

import pytest
import torch

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
