"""How the binding finds the current stream, without a GPU: by torch's quick
raw look-up where this torch has it, else by the public one."""
from types import SimpleNamespace

import torch

from combine_topk_ids_dest_amd import binding as B


def test_the_raw_look_up_is_taken_where_it_exists():
    c = SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 100 + device)
    assert B._raw_stream_lookup(c)(3) == 103


def test_without_it_the_public_stream_is_asked(monkeypatch):
    asked = []

    def current_stream(device):
        asked.append(device)
        return SimpleNamespace(cuda_stream=77)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    assert B._raw_stream_lookup(SimpleNamespace())(2) == 77 and asked == [2]


def test_calls_go_by_the_look_up(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 40 + device)
    assert B._stream(None) == 41
    call = B.PreparedCall("moe_ep_matmul", (), ())
    seen = []
    call.fn = lambda *args: seen.append(args) or B.OK
    call()
    assert seen == [(41,)]
