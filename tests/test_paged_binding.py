"""Pointers and streams that the binding takes (no GPU needed)."""
import enum

import pytest

import masked_block_diffusion_denoise_b200 as dlm


class Handle(int):
    pass


class Name(enum.IntEnum):
    LEGACY = 1


class Tensor:
    def data_ptr(self):
        return 0x40


class Stream:
    cuda_stream = 0x80


@pytest.mark.parametrize("x,address", [(None, None), (0, 0), (0x10, 0x10), (Handle(0x20), 0x20),
                                       (Name.LEGACY, 1), (True, 1), (Tensor(), 0x40)])
def test_pointers(x, address):
    assert dlm._ptr(x) == address


@pytest.mark.parametrize("x,handle", [(None, None), (0, 0), (0x10, 0x10), (Handle(0x20), 0x20),
                                      (Name.LEGACY, 1), (Stream(), 0x80)])
def test_streams(x, handle):
    assert dlm._stream(x) == handle


def test_a_call_with_an_address_of_a_subclass():
    """Refused for its sizes by the library, not by the binding."""
    with pytest.raises(dlm.DlmError):
        dlm.dlm_paged_resize(Handle(64), Handle(64), Handle(64), 0, Handle(64), 1, 8, Handle(64), 1,
                             Handle(64), Handle(64), Handle(64), None, 0, stream=Name.LEGACY)


@pytest.mark.parametrize("dtype,stride", [(dlm.DLM_BF16, 2 ** 39), (dlm.DLM_BF16, 2 ** 40),
                                          (dlm.DLM_F32, 2 ** 38), (dlm.DLM_BF16, 2 ** 62)])
def test_strides_beyond_a_tensor_map_are_refused(dtype, stride):
    """As bad arguments, before anything is asked of the device."""
    a = 0x10000

    class Work:
        def numel(self):
            return 1 << 30

        def element_size(self):
            return 1

        def data_ptr(self):
            return a

    c = dlm.dlm_paged_cache(a, a, 16, 16, 2, 128, dtype)
    for fn, args, kw in ((dlm.dlm_paged_kv_write, (c, a, a, a, 4), ("k_stride", "v_stride")),
                         (dlm.dlm_paged_attention, (c, a, a, a, a, a, 8, 1, 4, 4, 1, Work()),
                          ("q_stride", "o_stride"))):
        for name in kw:
            with pytest.raises(dlm.DlmError) as e:
                fn(*args, **{name: stride})
            assert e.value.code == dlm.DLM_EINVAL, name
