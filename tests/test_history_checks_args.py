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


def on_the_host(cls, **attrs):
    """An object whose buffers would be on the CPU: the checks run, and a launch fails the test."""
    def launch(*a):
        raise AssertionError("reached the library")

    o = cls.__new__(cls)
    o.__dict__.update(dict(device=torch.device("cpu"), _run=launch), **attrs)
    return o


BAD_LISTS = [([[1, 2]], TypeError), (torch.tensor(3), TypeError), (torch.zeros((2, 2, 3)), TypeError),
             (torch.zeros((2, 2, 0), dtype=torch.int32), ValueError),
             (torch.zeros((2, 3, 3), dtype=torch.int32), ValueError), (5, TypeError)]


@pytest.mark.parametrize("sel,error", BAD_LISTS)
def test_lists_that_are_no_lists_are_refused(sel, error):
    c = on_the_host(dt.KV4Cache, H=4, Hkv=2, d=64, _batch={"requests": 2})
    Q, count = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(error, match="sel"):
        c.attend(Q, torch.zeros_like(Q), sel=sel, sel_count=count)
    b = on_the_host(dt.BlockSparseAttention, B=2, H=4, Hkv=2, Nq=100, Nk=70, d=64, n_q=1)
    Q, K = (torch.zeros((2, h, n, 64), dtype=torch.bfloat16) for h, n in ((4, 100), (2, 70)))
    if isinstance(sel, torch.Tensor) and sel.dim() == 3:
        sel = sel[:, :, None]
    with pytest.raises(error, match="sel"):
        b.attend(Q, K, K, torch.zeros_like(Q), sel=sel, sel_count=count[..., None])


def test_block_attention_refuses_strides_of_lse_that_lie_on_one_another():
    s = (64 * 640, 640, 64)
    a = dict(B=1, H=2, Hkv=1, Nq=10, Nk=10, d=64, Q=A, K=2 * A, V=3 * A, q_strides=s, k_strides=s, v_strides=s,
             sel=A, sel_count=A, max_sel=2, out=8 * A, out_is_fp32=0, out_lse=9 * A)
    for strides in ((20, 0, 1), (20, 10, 0), (20, -10, 1)):
        with pytest.raises(dt.DitangoError) as e:
            dt.ditango_block_attn(lse_strides=strides, stream=0, **a)
        assert e.value.status == 1
    b = on_the_host(dt.BlockSparseAttention, B=2, H=4, Hkv=2, Nq=100, Nk=70, d=64, n_q=1, status=None)
    Q, K = (torch.zeros((2, h, n, 64), dtype=torch.bfloat16) for h, n in ((4, 100), (2, 70)))
    for lse, error in ((torch.zeros((2, 4, 100), dtype=torch.bfloat16), TypeError), (7, TypeError),
                       (torch.zeros((2, 4, 99)), ValueError)):
        with pytest.raises(error, match="out_lse"):
            b.attend(Q, K, K, torch.zeros_like(Q), lse)


def test_a_cache_borrows_from_one_of_its_sizes_only():
    like = on_the_host(dt.KV4Cache, n_pages=9, H=4, Hkv=2, d=64, max_requests=3, max_blocks=5, max_tokens=7,
                       block_table=None, _batch={"requests": 2})
    ok = dict(n_pages=9, Hkv=2, d=64, max_requests=3, max_blocks=5, max_tokens=7, H=4, like=like)
    for kw, error in ((dict(n_pages=8), ValueError), (dict(H=2), ValueError), (dict(d=96), ValueError),
                      (dict(max_tokens=8), ValueError), (dict(max_blocks=4), ValueError), (dict(like=3), TypeError),
                      (dict(block_table=torch.zeros((3, 5), dtype=torch.int32)), ValueError)):
        with pytest.raises(error):
            dt.KV4Cache(**{**ok, **kw})
    like.n_requests = 1
    assert like.n_requests == 1
