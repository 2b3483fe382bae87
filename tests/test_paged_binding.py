"""CPU checks of what the binding of the cache operators hands to native code."""
import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn

COPIES = {
    "copy": copy.copy,
    "deepcopy": copy.deepcopy,
    "pickle": lambda x: pickle.loads(pickle.dumps(x)),
    "replace": dataclasses.replace,
}


def _fields(c):
    return [getattr(c, name) for name, _ in c._fields_]


@pytest.mark.parametrize("how", sorted(COPIES))
@pytest.mark.parametrize("used", [False, True])
def test_copied_dims_have_a_struct_of_their_own(how, used):
    """Copies of dims that were used before point to their own struct, with the same geometry, also
    when the original and its struct are gone."""
    d = gdn.KVDims(12, 3, 128, page_size=32, dtype=torch.float32, cache="e4m3", window=77)
    if used:
        d.address()
    want = _fields(gdn.KVDims(**{f.name: getattr(d, f.name) for f in dataclasses.fields(d)}).c())
    e = COPIES[how](d)
    assert e == d and e.address() == ctypes.addressof(e.c())
    if how != "copy":
        assert e.address() != d.address()
    del d
    noise = [gdn.KVDims(1, 1, 64, page_size=16) for _ in range(64)]
    assert all(n.address() != e.address() for n in noise)
    assert _fields(gdn._KVDims.from_address(e.address())) == want
