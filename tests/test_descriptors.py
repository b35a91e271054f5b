"""The packed descriptors that the binding sends are the ctypes structures of the header, in
size and in where every field lies."""
import ctypes

import pytest

from test_sequence_layers_gb300 import abi


@pytest.mark.parametrize("packed,struct", [(abi._ROPE_DESC, abi.RopeDesc), (abi._NORM_DESC, abi.BlockNormDesc),
                                           (abi._NORM_PAR, abi.BlockNormVectors), (abi._RECUR_DESC, abi.RecurrenceDesc)])
def test_same_bytes(packed, struct):
    assert packed.size == ctypes.sizeof(struct)
    n = len(packed.unpack(bytes(packed.size)))
    read = struct.from_buffer_copy(packed.pack(*range(1, n + 1)))
    fields = []
    for name, _ in struct._fields_:
        v = getattr(read, name)
        fields += list(v) if isinstance(v, ctypes.Array) else [v]
    assert [int(v) for v in fields] == list(range(1, n + 1))
