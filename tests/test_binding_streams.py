"""The binding's current stream on a torch without the raw-stream query (no GPU)."""
import types

import pytest

import scatter_boundary_tile_gb300 as sbt

torch = pytest.importorskip("torch")


@pytest.fixture
def fresh(monkeypatch):
    """The binding as before its first call, and a torch whose current stream is a stand-in."""
    for name in ("_torch", "_raw_stream", "_device_index", "_CODES"):
        monkeypatch.setattr(sbt, name, None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
        cuda_stream={None: 77, 3: 77}[device]))
    return monkeypatch


def test_without_the_raw_query_the_public_one_answers(fresh):
    fresh.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert sbt._stream(None) == 77


def test_types_are_known_without_it(fresh):
    fresh.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert sbt._dtype_code(torch.zeros(1, dtype=torch.float16), None) == sbt.SBT_F16
    assert sbt._dtype_code(torch.zeros(1), None) == sbt.SBT_F32


def test_with_it_both_name_the_same_stream(fresh):
    fresh.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: {3: 77}[device], raising=False)
    assert sbt._stream(None) == 77


def test_a_stream_that_is_given_is_taken(fresh):
    assert sbt._stream(5) == 5 and sbt._stream(types.SimpleNamespace(cuda_stream=9)) == 9
