"""Handles that hold device addresses (sampling settings, LM heads): what they were made from
cannot be taken away under a later call."""
import copy

import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd


def test_sampling_params_are_fixed():
    """The descriptor that calls read holds the tensors' addresses: another tensor in an
    attribute would leave it pointing at freed memory, another n would read past the arrays."""
    p = sd.SamplingParams([0.5, 0.9], [3, 4], [0.7, 0.8], 0.1, device="cpu")
    was = bytes(p._desc)
    for name in ("temperature", "top_k", "top_p", "min_p", "n", "device"):
        old = getattr(p, name)
        with pytest.raises(AttributeError):
            setattr(p, name, None if name == "device" else 4 if name == "n" else torch.ones(2))
        with pytest.raises(AttributeError):
            delattr(p, name)
        assert getattr(p, name) is old
    with pytest.raises(AttributeError):
        p.min_q = 0.1                               # a slip of the pen is not kept either
    q = copy.copy(p)
    with pytest.raises(AttributeError):
        q.top_p = None
    assert bytes(p._desc) == was == bytes(q._desc)
    assert [p._desc.temperature, p._desc.top_k, p._desc.top_p, p._desc.min_p] == [
        t.data_ptr() for t in (p.temperature, p.top_k, p.top_p, p.min_p)]
    p.top_p.fill_(0.25)                             # writing into them is how settings change
    assert p.top_p.tolist() == [0.25] * 2


def test_w12_descriptor_follows_its_tensors():
    """A W12 LM head whose tensors are replaced (moved, say) is read where they are now."""
    w = sd.W12Weights.from_bf16(np.full((4, 256), 0x3f80, dtype=np.uint16), device="cpu")
    for name in ("codes", "corr"):
        setattr(w, name, torch.cat([getattr(w, name)]))
    d = w.descriptor()._obj
    assert (d.codes, d.corr) == (w.codes.data_ptr(), w.corr.data_ptr())
    assert (d.cap, d.b2) == (w.cap, w.b2)


@pytest.mark.gpu
def test_mxfp4_weights_are_fixed():
    """The product reads V ids of d columns from buf: a shorter buffer, or larger sizes, would be
    read past the end."""
    head = sd.Mxfp4Weights.from_tensor(torch.ones((70, 256), dtype=torch.bfloat16, device="cuda"))
    for name in ("buf", "V", "d", "shape", "nbytes", "device"):
        old = getattr(head, name)
        with pytest.raises(AttributeError):
            setattr(head, name, old[:1] if name == "buf" else 1 << 20)
        assert getattr(head, name) is old
    h = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    assert bool((sd.sd_mxfp4_logits(h, copy.copy(head)) == 256).all())
