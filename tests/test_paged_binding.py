"""CPU checks of what the binding of the cache operators hands to native code."""
import copy
import ctypes
import dataclasses
import pickle
import sysconfig

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from gated_deltanet_linear_mixer_gb300 import _build

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


# --------------------------------------------------- tensors of several devices
D = gdn.KVDims(4, 2, 64, page_size=16, rope_dim=16)


def _calls(fake):
    """name -> (call, its tensor arguments); tensors without memory on a device of that name."""
    def t(*shape, dtype=torch.float32):
        return fake(shape, dtype)

    i32, bf = torch.int32, torch.bfloat16
    host = torch.tensor([0, 3], dtype=i32)
    cache = {"cache.k": t(5, 2, 16, 64, dtype=torch.int8), "cache.v": t(5, 2, 16, 64, dtype=torch.int8),
             "cache.k_scale": t(5, 2), "cache.v_scale": t(5, 2)}
    batch = {"cu_seqlens": t(2, dtype=i32), "lens": t(1, dtype=i32), "block_table": t(1, 4, dtype=i32)}
    rows = {"k": t(3, 2, 64, dtype=bf), "v": t(3, 2, 64, dtype=bf), "q": t(3, 4, 64, dtype=bf)}

    def held(a):
        c = object.__new__(gdn.KVCache)
        c.k, c.v, c.k_scale, c.v_scale = (a[f"cache.{x}"] for x in ("k", "v", "k_scale", "v_scale"))
        return c

    append = dict(**cache, **batch, **rows, rope=t(20, 16), positions=t(3, dtype=i32), q_out=t(3, 4, 64, dtype=bf))
    read = dict(**cache, **batch, k_out=t(3, 2, 64, dtype=bf), v_out=t(3, 2, 64, dtype=bf))
    attend = dict(**cache, **batch, q=rows["q"], out=t(3, 4, 64, dtype=bf), workspace=t(1 << 20, dtype=torch.uint8))
    accept = dict(drafts=t(2, 3, dtype=i32), target=t(2, 4, 10), draft=t(2, 3, 10), uniforms=t(2, 3), noise=t(2, 10),
                  temperature=t(2), accepted=t(2, dtype=i32), tokens=t(2, 4, dtype=i32))
    return {
        "append": (lambda a: gdn.kv_append(D, held(a), (a["cu_seqlens"], host), a["lens"], a["block_table"], a["k"],
                                           a["v"], q=a["q"], rope=a["rope"], positions=a["positions"],
                                           q_out=a["q_out"]), append),
        "read": (lambda a: gdn.kv_read(D, held(a), (a["cu_seqlens"], host), a["lens"], a["block_table"],
                                       k_out=a["k_out"], v_out=a["v_out"]), read),
        "attention": (lambda a: gdn.kv_attention(D, held(a), (a["cu_seqlens"], host), a["lens"], a["block_table"],
                                                 a["q"], max_kv_len=10, out=a["out"], workspace=a["workspace"]), attend),
        "accept": (lambda a: gdn.accept_drafts(a["drafts"], a["target"], a["draft"], a["uniforms"], a["noise"],
                                               form="logits", temperature=a["temperature"], accepted=a["accepted"],
                                               tokens=a["tokens"]), accept),
    }


@pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU: nothing can be launched")
@pytest.mark.parametrize("name", ["append", "read", "attention", "accept"])
@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_of_two_devices_are_refused(name):
    """Each tensor in turn on another device than the rest."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    _build.build()
    mode = FakeTensorMode(allow_non_fake_inputs=True)

    def on(device):
        def make(shape, dtype):
            with mode:
                return torch.empty(shape, dtype=dtype, device=device)
        return make

    call, args = _calls(on("cuda:0"))[name]
    _, others = _calls(on("cuda:1"))[name]
    for moved in args:
        with pytest.raises(ValueError, match="device"):
            call({**args, moved: others[moved]})


# ------------------------------------------------------------ the C entry points
@pytest.mark.parametrize("vocab,fits", [(2 ** 31 - 1, False), (2 ** 31 - 4096, False), (2 ** 31 - 4097, True),
                                        (2 ** 30, True)])
def test_vocabularies_whose_indexes_leave_32_bits_are_refused(monkeypatch, vocab, fits):
    """The kernel steps up to 2048 past a row's end in 32 bits.  No call gets past the checks: those
    that are accepted end in the injected failure."""
    _build.build()
    lib, at = gdn.load(), 0x10000
    monkeypatch.setenv("GDN_FAULT", "accept")
    got = lib.gdn_accept_drafts(1, 1, vocab, 0, 0, at, at, vocab, at, vocab, None, at, at, vocab, at, at, None)
    assert got == (gdn.GDN_ERR_INJECTED if fits else 2)
    assert ("vocab" in lib.gdn_last_error().decode()) == (not fits)


# ------------------------------------------------------------------- the build
@pytest.mark.parametrize("what", ["torch", "python"])
def test_a_binding_built_for_another_pytorch_is_rebuilt(monkeypatch, what):
    """The binding's module is tied to the PyTorch and the Python that it was built with."""
    _build.build()
    assert _build.up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "2.9.0+other")
    else:
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda name, old=sysconfig.get_config_var: ".other.so" if name == "EXT_SUFFIX" else old(name))
    assert not _build.up_to_date()
