"""A W4 whose tensors' storage is swapped under it (t.data = ..., set_, offloading and
reloading): a call takes the addresses that the tensors have then."""
import copy
import pickle

import pytest
import torch

import combine_topk_ids_expert_gb300 as ep


@pytest.fixture
def host_pointers(monkeypatch):
    """Addresses of host tensors, which a call refuses."""
    monkeypatch.setattr(ep, "_ptr", lambda t: None if t is None else t.data_ptr())


def w4():
    return ep.W4(torch.zeros((2, 8, 64), dtype=torch.uint8), torch.ones((2, 8, 2)),
                 torch.zeros((2, 8, 2), dtype=torch.uint8))


def struct(w):
    made = w._struct
    return made() if callable(made) else made


def addresses(w):
    c = struct(w)
    return c.codes, c.scales, c.zeros


@pytest.mark.parametrize("field", ["codes", "scales", "zeros"])
def test_swapped_storage_is_the_one_used(host_pointers, field):
    w = w4()
    assert addresses(w) == (w.codes.data_ptr(), w.scales.data_ptr(), w.zeros.data_ptr())
    t = getattr(w, field)
    held = t.data          # the old storage stays alive, so the new one is elsewhere
    t.data = t.data.clone()
    assert t.data_ptr() != held.data_ptr()
    assert addresses(w) == (w.codes.data_ptr(), w.scales.data_ptr(), w.zeros.data_ptr())


def test_a_tensor_moved_to_the_host_is_refused(monkeypatch):
    w = w4()
    with monkeypatch.context() as m:
        m.setattr(ep, "_ptr", lambda t: None if t is None else t.data_ptr())
        struct(w)           # as if the tensors had been on the device
    with pytest.raises(ValueError, match="CUDA"):
        struct(w)


@pytest.mark.parametrize("field,shape", [("codes", (2, 8, 32)), ("scales", (2, 8, 1)),
                                         ("zeros", (2, 4, 2))])
def test_changed_shapes_are_refused(host_pointers, field, shape):
    w = w4()
    struct(w)
    t = getattr(w, field)
    t.data = t.data.new_zeros(shape)
    with pytest.raises(ValueError, match="changed"):
        struct(w)


def test_copies_after_a_call(host_pointers):
    w = w4()
    struct(w)
    for twin in (copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert (twin.din, twin.rows, twin.group) == (128, 8, 64)
        assert addresses(twin) == (twin.codes.data_ptr(), twin.scales.data_ptr(),
                                   twin.zeros.data_ptr())
        assert twin.codes.data_ptr() != w.codes.data_ptr()
