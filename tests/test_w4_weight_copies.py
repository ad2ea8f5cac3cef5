"""A packed weight's addresses are those of its own tensors: in copies, in restored ones, and for as long as it lives."""
import copy
import io
import pickle

import pytest
import torch

Q = pytest.importorskip("quantized_linear_layers_token_amd")


def weight(zeros):
    return Q.W4Weight(torch.arange(2048, dtype=torch.int32).to(torch.uint8), torch.arange(32, dtype=torch.int16),
                      torch.full((32,), 3, dtype=torch.uint8) if zeros else None, 1, 20, 128, 128)


def check_addresses(w):
    s = Q.QlinW4Weight.from_buffer_copy(w._bytes)
    assert (s.q_w, s.s_w, s.z_w, s.n) == (w.packed.data_ptr(), w.scales.data_ptr(), w.zeros.data_ptr() if w.zeros is not None else None, w.N)


def saved(w):
    buf = io.BytesIO()
    torch.save(w, buf)
    buf.seek(0)
    return torch.load(buf, weights_only=False)      # a file of this test's own


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda w: pickle.loads(pickle.dumps(w)), saved])
def test_copies_read_their_own_tensors(how, zeros):
    w = weight(zeros)
    check_addresses(w)
    c = how(w)
    check_addresses(c)
    assert (c.experts, c.N, c.K, c.group, c.device) == (w.experts, w.N, w.K, w.group, w.device)
    assert torch.equal(c.packed, w.packed) and torch.equal(c.scales, w.scales)
    assert (c.zeros is None) == (w.zeros is None) and (c.zeros is None or torch.equal(c.zeros, w.zeros))


@pytest.mark.parametrize("name", ["packed", "scales", "zeros", "N", "K", "group", "experts", "device"])
def test_its_parts_cannot_be_replaced(name):
    w = weight(True)
    value = getattr(w, name)
    with pytest.raises(AttributeError):
        setattr(w, name, value.clone() if isinstance(value, torch.Tensor) else value)
    check_addresses(w)
