"""The stream that a call without one goes to."""
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("private", [True, False])
def test_default_stream_is_torchs_current_one(monkeypatch, private):
    """By torch's private function where it is there, by the stream object where not."""
    if not private:
        monkeypatch.setattr(se, "_raw_stream", None)
    side = torch.cuda.Stream()
    handles = []
    for s in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(s):
            handles.append(se._stream(None))
            assert handles[-1] == torch.cuda.current_stream().cuda_stream == se._stream(s)
    assert handles[0] != handles[1]
