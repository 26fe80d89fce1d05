"""The stream that a call without one goes to."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_int4_gb300 import _build
    _build.build()
    from block_quantized_int4_gb300 import qmm as m
    return m


def test_streams_given_by_handle_or_object(qmm):
    assert qmm._stream(77) == 77
    assert qmm._stream(types.SimpleNamespace(cuda_stream=78)) == 78


def test_without_the_private_look_up(qmm, monkeypatch):
    monkeypatch.setattr(qmm, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=79))
    assert qmm._stream(None) == 79


@pytest.mark.gpu
def test_both_look_ups_name_the_current_stream(qmm, monkeypatch):
    s = torch.cuda.Stream()
    assert s.cuda_stream != torch.cuda.current_stream().cuda_stream
    for raw in (qmm._raw_stream, None):
        monkeypatch.setattr(qmm, "_raw_stream", raw)
        assert qmm._stream(None) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(s):
            assert qmm._stream(None) == s.cuda_stream
