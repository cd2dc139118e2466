"""What GradClip asks of its tensors before it uses its table again (host
code: tensors of the CPU, the calls into the library left out)."""
import pytest
import torch

from convolution_video_vae_amd import layer


def changes():
    """(name, a change of a [8, 6] fp32 tensor's data at the same address)."""
    return [("shorter", lambda t: t.data[:3]), ("flat", lambda t: t.data.view(-1)[:7]),
            ("other type of that size", lambda t: t.data.view(torch.int32)),
            ("shorter type", lambda t: t.data.view(torch.bfloat16)),
            ("apart", lambda t: torch.as_strided(t.data, (4, 6), (12, 1))),
            ("turned", lambda t: torch.as_strided(t.data, (8, 6), (1, 8))),
            ("same strides, other shape", lambda t: torch.as_strided(t.data, (6, 8), (6, 1)))]


def make(tensors, monkeypatch, cls):
    """A GradClip over tensors of the host."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: None)
    monkeypatch.setattr(layer, "_layouts_class", cls)
    return layer.GradClip(tensors)


@pytest.mark.parametrize("cls", [layer._Layouts, None], ids=["plain", "default"])
@pytest.mark.parametrize("calls", [0, 1, 2, 5])
@pytest.mark.parametrize("what,change", changes(), ids=lambda v: v if isinstance(v, str) else "")
def test_changes_at_the_same_address_are_seen(what, change, calls, cls, monkeypatch):
    whole = torch.zeros(100)                       # what "apart" spans lies inside
    t = whole[:48].view(8, 6)
    op = make([torch.zeros(5), t], monkeypatch, cls)
    for _ in range(calls):
        assert op._as_built()
    t.data = change(t)
    assert t.data_ptr() == whole.data_ptr() and not op._as_built()


@pytest.mark.parametrize("calls", [0, 1, 2, 5])
def test_a_shortened_tensor_is_looked_up_again(calls, monkeypatch):
    t = torch.zeros(64, 8)
    op = make([t, torch.zeros(3)], monkeypatch, None)
    for _ in range(calls):
        assert op._as_built()
    assert op._table[0].numel == 512
    t.data = t.data[:2]
    assert not op._as_built()
    op._rebuild()
    assert op._as_built() and op._table[0].numel == 16


@pytest.mark.parametrize("calls", [0, 1, 2, 5])
def test_a_storage_cut_short_is_refused(calls, monkeypatch):
    t, other = torch.zeros(4096), torch.zeros(16)
    op = make([other, t], monkeypatch, None)
    for _ in range(calls):
        assert op._as_built()
    t.untyped_storage().resize_(1024)
    assert not op._as_built()
    with pytest.raises(ValueError, match="storage"):
        op._rebuild()


def test_dense_tensors_in_another_order(monkeypatch):
    t = torch.zeros(2, 3, 4).permute(2, 0, 1)
    op = make([t], monkeypatch, None)
    assert op._as_built()
    t.data = torch.as_strided(t.data, (4, 2, 3), (1, 4, 8))
    assert not op._as_built()


def test_both_ways_of_comparing_agree():
    assert layer._tells_apart(layer._Layouts)
    layer._layouts([torch.zeros(3)])
    assert layer._tells_apart(layer._layouts)


def test_addresses():
    ts = [torch.zeros(3), torch.zeros(5, dtype=torch.bfloat16)]
    ptrs = [t.data_ptr() for t in ts]
    for same in (layer._same_addresses, layer._plain_same_addresses):
        assert same(ts, ptrs, [0, 1])
        assert not same([ts[0], torch.zeros(5)], ptrs, [0, 1])
        assert not same([ts[0], torch.zeros(0)], ptrs, [0, 1])
        assert same([torch.zeros(0)], [0], [0])
