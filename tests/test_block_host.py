"""The Python calls of the operators around a mixing layer without a GPU: what they check and hand to
the library, with tensors that say which device they are on and a library that only listens."""
import pytest
import torch

from gated_delta_rule_41_gb300 import block
from gated_delta_rule_41_gb300.block import KdaError

BF16, F32 = torch.bfloat16, torch.float32


class On(torch.Tensor):
    """A tensor in the host's memory that passes for one on CUDA device ``dev``."""
    dev = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.dev


def on(dev, *shape, dtype=BF16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.dev = dev
    return t


class Listening:
    """Every entry succeeds; the calls' arguments by name.  Workspaces grow with the device's number."""

    def __init__(self, host):
        self.host, self.calls = host, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_bytes"):
                return 1000 * (1 + self.host["dev"])
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def host(monkeypatch):
    """Current device and library."""
    h = dict(dev=0)
    h["lib"] = Listening(h)
    monkeypatch.setattr(block, "_get_device", lambda: h["dev"])
    monkeypatch.setattr(block, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(block, "_lib", lambda: h["lib"])

    def fresh(stream, shape, dtype, device):
        return on(h["dev"], shape, dtype=dtype)

    monkeypatch.setattr(block, "_fresh", fresh)
    monkeypatch.setattr(block, "_plans", {})
    return h


def gated_bwd(dev, **kw):
    t = lambda: on(dev, 6, 2, 64)  # noqa: E731
    return block.gated_norm_bwd(t(), t(), on(dev, 64, dtype=F32), t(), **kw)


def add_bwd(dev, **kw):
    t = lambda: on(dev, 6, 64)  # noqa: E731
    return block.add_norm_bwd(t(), on(dev, 64, dtype=F32), t(), t(), **kw)


def scan_bwd(dev, **kw):
    t = lambda: on(dev, 2, 70, 64)  # noqa: E731
    return block.gated_scan_bwd(t(), t(), t(), on(dev, 2, 2, 64, dtype=F32), **kw)


@pytest.mark.parametrize("call", [gated_bwd, add_bwd])
def test_workspaces_are_as_large_as_the_device_asks(host, call):
    """The same call on devices of unequal size, in turn."""
    for dev in (0, 1, 0):
        host["dev"] = dev
        call(dev)
        _, args = host["lib"].calls[-1]
        assert args[-2] == 1000 * (1 + dev)


def grads_of(call, dev):
    """Tensors for a call's results, on this device."""
    if call is scan_bwd:
        return dict(dx=on(dev, 2, 70, 64), dg=on(dev, 2, 70, 64), dh0=on(dev, 2, 64, dtype=F32))
    if call is gated_bwd:
        return dict(dx=on(dev, 6, 2, 64), dgate=on(dev, 6, 2, 64), dw=on(dev, 64, dtype=F32))
    return dict(dres=on(dev, 6, 64), dx=on(dev, 6, 64), dw=on(dev, 64, dtype=F32),
                dalpha=on(dev, 64, dtype=F32))


@pytest.mark.parametrize("call", [scan_bwd, gated_bwd, add_bwd])
def test_grads_on_another_device_are_refused(host, call):
    """As all other tensors are; nothing is launched."""
    kw = dict(x=on(0, 6, 64), alpha=on(0, 64, dtype=F32)) if call is add_bwd else {}
    for name in grads_of(call, 0):
        grads = grads_of(call, 0)
        grads[name].dev = 1
        with pytest.raises(KdaError) as e:
            call(0, grads=grads, **kw)
        assert e.value.status == 1 and not host["lib"].calls
    call(0, grads=dict(grads_of(call, 0), other=on(1, 3)), **kw)      # (what is not asked for is not looked at)
    assert host["lib"].calls


@pytest.mark.parametrize("call", [gated_bwd, add_bwd])
def test_a_workspace_holds_what_it_says(host, call):
    """One whose elements share memory, or lie apart, is refused: the kernels write as many bytes as its
    elements have from its first one on."""
    one = on(0, 1, dtype=torch.uint8)
    wide = one.expand(1 << 20)
    wide.dev = 0
    apart = on(0, 1 << 12, dtype=torch.uint8)[::2]
    apart.dev = 0
    for ws in (wide, apart):
        assert isinstance(ws, On) and not ws.is_contiguous()
        with pytest.raises(KdaError) as e:
            call(0, workspace=ws)
        assert e.value.status == 1 and not host["lib"].calls
    ws = on(0, 4096, dtype=torch.uint8)
    call(0, workspace=ws)
    assert host["lib"].calls[-1][1][-3] == ws.data_ptr()
    call(0, workspace=on(0, 10, dtype=torch.uint8))            # too small: the call makes its own
    assert len(host["lib"].calls) == 2
    none = dict(dx=on(0, 6, 2, 64), dgate=on(0, 6, 2, 64)) if call is gated_bwd else dict(dres=on(0, 6, 64))
    call(0, workspace=apart, grads=none)                       # not used
    assert len(host["lib"].calls) == 3


def test_gradients_that_are_one_tensor(host):
    """Without alpha dx may be the tensor dres, as in what a call returns; with another factor these are
    two results, and one tensor for both is refused."""
    call = lambda **kw: add_bwd(0, **kw)  # noqa: E731
    got = call()
    assert got["dx"] is got["dres"]
    again = call(grads=got)
    assert again is got and got["dx"] is got["dres"]
    name, args = host["lib"].calls[-1]
    assert name == "kda_add_norm_bwd" and args[7] == got["dres"].data_ptr() and args[8] is None
    empty = torch.zeros(0, 64, dtype=BF16).as_subclass(On)
    w = on(0, 64, dtype=F32)
    block.add_norm_bwd(empty, w, empty, alpha=0.5, grads=dict(dres=empty, dx=torch.empty_like(empty), dw=w))
    before = len(host["lib"].calls)
    for kw in (dict(alpha=0.5), dict(alpha=on(0, 64, dtype=F32), x=on(0, 6, 64))):
        with pytest.raises(KdaError) as e:
            call(grads=got, **kw)
        assert e.value.status == 1
    assert len(host["lib"].calls) == before
