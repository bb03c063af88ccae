"""The binding's own checks of gnf4_moe_route, gnf4_moe_experts and gnf4_gemv, which come before
the library sees a pointer (no GPU: host tensors pass as device ones up to the library)."""
import pytest
import torch

import grouped_nf4_w4a16_b200 as gnf4
from grouped_nf4_w4a16_b200 import binding


@pytest.fixture
def as_if_on_device(monkeypatch):
    monkeypatch.setattr(binding, "_here", lambda t, where: 0)


def calls(**kw):
    bf = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = torch.zeros((128, 32), dtype=torch.uint8)
    s = torch.zeros((128, 1))
    ids = torch.zeros((2, 1), dtype=torch.int32)
    return [
        lambda: gnf4.gnf4_moe_route(bf, bf, 1, **kw),
        lambda: gnf4.gnf4_moe_experts(bf, ids, torch.zeros((2, 1)), w[None], s[None], w[None, :64],
                                      s[None, :64], **kw),
        lambda: gnf4.gnf4_gemv(bf, w, s, **kw),
    ]


@pytest.mark.parametrize("call", range(3))
def test_workspaces_that_count_more_bytes_than_they_hold(as_if_on_device, call):
    one = torch.zeros(1, dtype=torch.uint8)
    # a byte shown 2^30 times; every other byte of a buffer
    for workspace in (one.expand(1 << 30), torch.zeros(1 << 24, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            calls(workspace=workspace)[call]()
    # an ordinary one gets as far as the library, which knows host memory
    with pytest.raises(gnf4.Gnf4Error, match="HOST_POINTER"):
        calls(workspace=torch.zeros(1 << 24, dtype=torch.uint8))[call]()


class FakeStream:
    def __init__(self, device):
        self.device = torch.device(device)


class Nothing:
    def __init__(self, *args, **kw):
        pass

    def __enter__(self):
        return self

    def __exit__(self, *args):
        return False


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """torch.cuda.stream(s) makes s's device current, so the call would have gone to the tensors'
    device and its current stream."""
    used = []
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "device", Nothing)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s) or Nothing())
    t = type("T", (), dict(device=torch.device("cuda:0")))()
    ran = lambda: "ran"
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        binding._elsewhere(ran, t, FakeStream("cuda:1"), (), {})
    own = FakeStream("cuda:0")
    assert binding._elsewhere(ran, t, own, (), {}) == "ran" and used == [own]


@pytest.mark.parametrize("handle,kind", [(0, "default"), (1, "default"), (2, 2), (0x7f00, 0x7f00)])
def test_stream_handles(monkeypatch, handle, kind):
    """Handles 0 and 1 are the legacy default stream (1 is no address an ExternalStream can hold)."""
    used = []
    monkeypatch.setattr(torch.cuda, "device", Nothing)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s) or Nothing())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: h)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    t = type("T", (), dict(device=torch.device("cuda:0")))()
    binding._elsewhere(lambda: None, t, handle, (), {})
    assert used == [kind]


BEYOND = 1 << 32


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: gnf4.gnf4_moe_route(meta(1, BEYOND + 64), meta(2, BEYOND + 64), 1),
    lambda: gnf4.gnf4_moe_route(meta(1, 64), meta(BEYOND + 4, 64), 1),
    lambda: gnf4.gnf4_moe_route(meta(1, 64), meta(4, 64), BEYOND + 1),
    lambda: gnf4.gnf4_moe_route(meta(1, 64), meta(4, 64), 2 - BEYOND),
    lambda: gnf4.gnf4_moe_experts(
        meta(1, 64), meta(1, BEYOND + 1, dtype=torch.int32), meta(1, BEYOND + 1, dtype=torch.float32),
        meta(2, 128, 32, dtype=torch.uint8), meta(2, 128, 1, dtype=torch.float32),
        meta(2, 64, 32, dtype=torch.uint8), meta(2, 64, 1, dtype=torch.float32)),
    lambda: gnf4.gnf4_moe_experts(
        meta(1, 64), meta(1, 1, dtype=torch.int32), meta(1, 1, dtype=torch.float32),
        meta(BEYOND + 2, 128, 32, dtype=torch.uint8), meta(BEYOND + 2, 128, 1, dtype=torch.float32),
        meta(BEYOND + 2, 64, 32, dtype=torch.uint8), meta(BEYOND + 2, 64, 1, dtype=torch.float32)),
    lambda: gnf4.gnf4_moe_experts(
        meta(1, 64), meta(1, 1, dtype=torch.int32), meta(1, 1, dtype=torch.float32),
        meta(2, 2 * (BEYOND + 64), 32, dtype=torch.uint8), meta(2, 2 * (BEYOND + 64), 1, dtype=torch.float32),
        meta(2, 64, (BEYOND + 64) // 2, dtype=torch.uint8), meta(2, 64, (BEYOND + 64) // 64, dtype=torch.float32)),
    lambda: gnf4.gnf4_gemv(meta(1, 64), meta(BEYOND + 5, 32, dtype=torch.uint8), meta(BEYOND + 5, 1, dtype=torch.float32)),
    lambda: gnf4.gnf4_gemv(meta(1, BEYOND + 64), meta(5, (BEYOND + 64) // 2, dtype=torch.uint8),
                           meta(5, (BEYOND + 64) // 64, dtype=torch.float32)),
    lambda: gnf4.gnf4_gemv(meta(BEYOND + 1, 64), meta(5, 32, dtype=torch.uint8), meta(5, 1, dtype=torch.float32)),
])
def test_sizes_beyond_32_bits_are_refused(as_if_on_device, call):
    """They do not fit the C fields, where their low 32 bits would look like an ordinary size."""
    with pytest.raises(gnf4.Gnf4Error, match="UNSUPPORTED_SHAPE"):
        call()
