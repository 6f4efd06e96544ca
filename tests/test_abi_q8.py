"""CPU checks of the 8-bit cache's and the rotary calls' boundary: struct layouts, sizing, refusals that need no GPU."""

import ctypes

import pytest

from quantised_kv_cache_gb300 import tq


@pytest.fixture(scope="module", autouse=True)
def _built():
    from quantised_kv_cache_gb300 import build
    build.build()


def test_the_packed_attention_arguments_are_the_struct():
    """The binding packs tq_q8_attn with struct; every field lands where the C struct has it."""
    fields = tq.tq_q8_attn._fields_
    values, want = [], {}
    for k, (name, ftype) in enumerate(fields):
        n = 3 if name.endswith("strides") else 1
        got = [100 + k + i for i in range(n)]
        values += got
        want[name] = got
    raw = tq._pack_attn.pack(*values)
    assert len(raw) == ctypes.sizeof(tq.tq_q8_attn)
    a = tq.tq_q8_attn.from_buffer_copy(raw)
    for name, got in want.items():
        v = getattr(a, name)
        assert (list(v) if len(got) == 3 else [v]) == got, name


def test_host_refusals():
    L = tq.lib()
    h = ctypes.c_void_p()
    assert L.tq_init(128, 4, tq.TQ_SCHEME_Q8, ctypes.c_uint64(1), ctypes.byref(h)) == tq.TQ_ERR_ARG
    assert L.tq_init(64, 8, tq.TQ_SCHEME_Q8, ctypes.c_uint64(1), ctypes.byref(h)) == tq.TQ_ERR_UNSUPPORTED
    assert L.tq_init(128, 8, tq.TQ_SCHEME_KQV, ctypes.c_uint64(1), ctypes.byref(h)) == tq.TQ_ERR_ARG
    assert L.tq_set_rope(None, None) == tq.TQ_ERR_ARG
    none = tq._strides3()
    assert L.tq_rotary(None, None, none, None, none, 0, 1, 1, 1, None, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_append(None, None, None, none, None, none, 0, 1, 1, 1, None, None, 0, None, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_attention(None, None, None, None, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_attention_workspace(None, 1, 1, 1, 1, 1, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_evict(None, None, None, 1, 1, None, None, 1, 0, 0, None, None, None, None, None, None) == tq.TQ_ERR_ARG
    assert tq.tq_status_str(tq.TQ_ERR_NONFINITE).startswith("an infinity")
