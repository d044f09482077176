"""What the entry points do on the host, without a GPU: refusals ahead of any device
work, and what becomes of failures of the runtime.  The calls are in host_calls.py."""
import os
import shutil
import subprocess
import sys

import pytest

import sharded_gemm_alltosharded_amd as sg

HERE = os.path.dirname(os.path.abspath(__file__))
ROCM = os.path.dirname(os.path.dirname(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")))


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    if not os.path.exists(sg.LIB_PATH):
        pytest.skip("library not built")
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("no host compiler or no HIP headers")
    to = str(tmp_path_factory.mktemp("stub") / "libstub.so")
    subprocess.check_call([cxx, "-shared", "-fPIC", "-O1", "-std=c++17", "-I", os.path.join(ROCM, "include"),
                           os.path.join(HERE, "host_stub.cpp"), "-o", to])
    return to


def calls(stub, name):
    r = subprocess.run([sys.executable, os.path.join(HERE, "host_calls.py"), stub, sg.LIB_PATH, name],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def test_block_backward_refuses_token_counts(stub):
    calls(stub, "block_backward_tokens")


def test_first_adapted_call_beside_a_capture(stub):
    calls(stub, "first_adapted_call_beside_a_capture")


def test_first_backward_call_beside_a_capture(stub):
    calls(stub, "first_backward_call_beside_a_capture")


def test_no_memory_for_a_copy(stub):
    calls(stub, "no_memory_for_a_copy")


def test_adapted_calls_on_another_device(stub):
    calls(stub, "adapted_calls_on_another_device")


def test_projections_that_cannot_be_launched(stub):
    calls(stub, "projections_that_cannot_be_launched")


def test_workspace_of_decoded_weights(stub):
    calls(stub, "workspace_of_decoded_weights")


def test_weight_gradient_tiles(stub):
    calls(stub, "weight_gradient_tiles")


def test_layers_given_up_beside_a_capture(stub):
    calls(stub, "layers_given_up_beside_a_capture")


def test_input_gradients_beside_a_bias(stub):
    calls(stub, "input_gradients_beside_a_bias")
