"""The short way's module (binding/calls.cpp) and the library that it is bound to, on the host."""
import ctypes

import pytest

import gated_deltanet_state_delta_amd._lib as L
from gated_deltanet_state_delta_amd import build as B

ENTRIES = ("attn_decode", "attn_decode_workspace_size", "kv_append", "kv_read", "rope")


def _address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


def test_the_library_tells_its_header():
    assert L.load().gdn_header_digest().decode() == B.header_digest()


@pytest.mark.parametrize("digest", [b"0123456789abcdef", b"", None])
def test_a_library_of_another_header_is_refused(digest):
    """Its structs may be laid out otherwise: nothing may be called through them."""
    lib, module = L.load(), L.calls()
    text = None if digest is None else ctypes.create_string_buffer(digest)
    other = ctypes.CFUNCTYPE(ctypes.c_void_p)(lambda: text and ctypes.addressof(text))
    entries = [_address(getattr(lib, "gdn_" + name)) for name in ENTRIES]
    with pytest.raises(RuntimeError, match="different headers"):
        module.bind(_address(other), *entries)
    module.bind(_address(lib.gdn_header_digest), *entries)
    with pytest.raises(TypeError):
        module.bind(*entries)
