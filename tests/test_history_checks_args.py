"""Arguments of the 4-bit history and selected-block calls: what is accepted, and
which error a wrong one gives (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import sparse_state_reuse_b200 as dt

A = 4096     # an aligned address that no call here reaches


class Address(int):
    pass


def test_an_address_may_be_any_int():
    kv = dt.kv4(4, 2, 64, Address(A))
    assert kv.data == A
    for T, status in ((-1, 1), (3, 1)):
        with pytest.raises(dt.DitangoError) as e:      # refused for T, then for the strides
            dt.ditango_kv4_write(kv, T, Address(A), Address(2 * A), (128, 60), (128, 64), Address(3 * A), stream=0)
        assert e.value.status == status
    dt.ditango_kv4_write(kv, 0, Address(A), Address(2 * A), (128, 64), (128, 64), Address(3 * A), stream=0)


def test_attention_of_no_rows_does_nothing():
    a = dict(R=2, H=4, T=0, max_q=0, max_blocks=4, Q=None, q_strides=(256, 64), q_off=A, kv_len=A, block_table=A,
             out=None, out_is_fp32=1, workspace=None, workspace_bytes=0)
    dt.ditango_kv4_attn(dt.kv4(4, 2, 64, A), stream=0, **a)
    for kw in (dict(max_q=-1), dict(T=1)):
        with pytest.raises(dt.DitangoError) as e:
            dt.ditango_kv4_attn(dt.kv4(4, 2, 64, A), stream=0, **{**a, **kw})
        assert e.value.status == 1
