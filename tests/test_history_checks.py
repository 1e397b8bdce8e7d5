"""Refusals of the 4-bit history and selected-block calls (no GPU needed), and
the oracle's own pins."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_state_reuse_b200 as dt
from oracle import history as OH

A = 4096     # an aligned address that no call here reaches


def refused(fn, *a, status=1, **kw):
    with pytest.raises(dt.DitangoError) as e:
        fn(*a, stream=0, **kw)
    assert e.value.status == status, e.value


def tables(**kw):
    a = dict(R=2, max_blocks=4, max_tokens=8, n_pages=9, ctx_len=A, new_len=2 * A, free_pages=3 * A, n_free=5,
             block_table=4 * A, kv_len=5 * A, q_off=6 * A, slot_map=7 * A, pages_used=8 * A)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), 1), (dict(R=4097), 2), (dict(max_blocks=0), 1), (dict(max_blocks=2 ** 26), 2),
    (dict(max_tokens=0), 1), (dict(n_pages=0), 1), (dict(n_free=-1), 1), (dict(free_pages=None), 1),
    (dict(ctx_len=None), 1), (dict(slot_map=None), 1), (dict(pages_used=None), 1),
    (dict(kv_len=A), 1),                       # the new lengths over the old ones
    (dict(kv_len=2 * A - 4), 1), (dict(q_off=5 * A + 4), 1), (dict(block_table=3 * A - 8), 1),
])
def test_tables_refuse(kw, status):
    refused(dt.ditango_block_tables, status=status, **tables(**kw))


@pytest.mark.parametrize("kv,kw,status", [
    ((4, 2, 80, A), {}, 2), ((0, 2, 64, A), {}, 1), ((4, 0, 64, A), {}, 1), ((4, 2, 64, A + 8), {}, 1),
    ((4, 2, 64, None), {}, 1), ((4, 2, 64, A), dict(T=-1), 1), ((4, 2, 64, A), dict(K=None), 1),
    ((4, 2, 64, A), dict(V=A + 2), 1), ((4, 2, 64, A), dict(k_strides=(128, 60)), 1),
    ((4, 2, 64, A), dict(v_strides=(0, 64)), 1), ((4, 2, 64, A), dict(k_strides=None), 1),
    ((4, 2, 64, A), dict(slot_map=None), 1), ((4, 70000, 64, A), {}, 2),
])
@pytest.mark.parametrize("call", [dt.ditango_kv4_write, dt.ditango_kv4_read])
def test_rows_refuse(call, kv, kw, status):
    a = dict(T=3, K=A, V=A, k_strides=(128, 64), v_strides=(128, 64), slot_map=A)
    a.update(kw)
    refused(call, dt.kv4(*kv), status=status, **a)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), 1), (dict(R=5000), 2), (dict(H=3), 1), (dict(H=0), 1), (dict(T=-1), 1), (dict(max_q=0), 1),
    (dict(max_blocks=0), 1), (dict(Q=None), 1), (dict(Q=A + 4), 1), (dict(out=3 * A), 1),   # out is Q
    (dict(q_strides=(256, 60)), 1), (dict(q_off=None), 1), (dict(kv_len=None), 1), (dict(block_table=None), 1),
    (dict(sel=A), 1), (dict(sel=A, sel_count=A), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(out=None), 1), (dict(out=5 * A + 8), 1), (dict(out_strides=(256, 2)), 1),
    (dict(workspace=None), 1), (dict(workspace=A + 8), 1), (dict(workspace_bytes=100), 1),
    (dict(lse_strides=(0, 1)), 1),
])
def test_history_attention_refuses(kw, status):
    a = dict(R=2, H=4, T=5, max_q=3, max_blocks=4, Q=3 * A, q_strides=(256, 64), q_off=A, kv_len=A, block_table=A,
             out=5 * A, out_is_fp32=1, workspace=A, workspace_bytes=dt.ditango_kv4_attn_workspace_size(64))
    a.update(kw)
    refused(dt.ditango_kv4_attn, dt.kv4(4, 2, 64, A), status=status, **a)


def test_summary_select_and_attention_refuse():
    s = (64 * 640, 640, 64)
    ok = dict(B=1, H=2, N=10, d=64, block=64, x=A, strides=(1280, 640, 64), codes=A, scale=A)
    for kw, st in ((dict(block=32), 1), (dict(d=72), 2), (dict(B=0), 1), (dict(x=A + 2), 1), (dict(B=70000), 2),
                   (dict(strides=(1280, 640, 60)), 1), (dict(codes=None), 1), (dict(strides=None), 1)):
        refused(dt.ditango_block_summary, status=st, **{**ok, **kw})
    ok = dict(B=1, H=4, Hkv=2, n_q=3, n_k=7, d=64, k=3, band=1, sink=1, own_blocks=2, max_sel=5, q_codes=A,
              q_scale=A, k_codes=A, k_scale=A, sel=A, sel_count=A)
    for kw, st in ((dict(H=3), 1), (dict(n_k=0), 1), (dict(k=-1), 1), (dict(band=-2), 1), (dict(sink=-1), 1),
                   (dict(max_sel=4), 1), (dict(k=6), 1), (dict(n_k=60000), 2), (dict(d=32), 2),
                   (dict(q_codes=A + 4), 1), (dict(block_table=A, n_pages=0), 1), (dict(sel_count=None), 1),
                   (dict(own_blocks=-1), 1)):
        refused(dt.ditango_block_select, status=st, **{**ok, **kw})
    ok = dict(B=1, H=4, Hkv=2, Nq=10, Nk=10, d=64, Q=A, q_strides=s, K=2 * A, k_strides=s, q_codes=A, q_scale=A,
              k_codes=A, k_scale=A)
    for kw, st in ((dict(H=3), 1), (dict(d=72), 2), (dict(Nk=0), 1), (dict(Q=A + 2), 1), (dict(K=None), 1),
                   (dict(k_strides=(1280, 640, 60)), 1), (dict(k_scale=None), 1), (dict(H=65534), 2),
                   (dict(H=2 ** 31 - 2), 2), (dict(B=70000), 2)):
        refused(dt.ditango_block_summaries, status=st, **{**ok, **kw})
    ok = dict(R=2, H=4, max_blocks=7, k=3, band=1, sink=1, max_sel=4, Q=A, q_strides=(256, 64), sum_codes=A,
              sum_scale=A, block_table=A, kv_len=A, q_codes=A, q_scale=A, sel=A, sel_count=A)
    for kw, st in ((dict(R=0), 1), (dict(R=5000), 2), (dict(H=3), 1), (dict(max_blocks=0), 1), (dict(k=-1), 1),
                   (dict(max_sel=3), 1), (dict(band=-2), 1), (dict(max_blocks=60000), 2), (dict(Q=A + 8), 1),
                   (dict(q_strides=(256, 60)), 1), (dict(q_strides=None), 1), (dict(kv_len=None), 1),
                   (dict(sum_codes=A + 4), 1), (dict(q_codes=None), 1), (dict(band=2 ** 25, max_sel=8), 2)):
        refused(dt.ditango_kv4_select, dt.kv4(4, 2, 64, A), status=st, **{**ok, **kw})
    refused(dt.ditango_kv4_select, dt.kv4(4, 2, 80, A), status=2, **ok)
    ok = dict(B=1, H=2, Hkv=1, Nq=10, Nk=10, d=64, Q=A, K=2 * A, V=3 * A, q_strides=s, k_strides=s, v_strides=s,
              sel=A, sel_count=A, max_sel=2, out=8 * A, out_is_fp32=0)
    for kw, st in ((dict(H=3, Hkv=2), 1), (dict(d=80), 2), (dict(Nq=0), 1), (dict(max_sel=0), 1),
                   (dict(Q=A + 2), 1), (dict(out=A), 1), (dict(out=2 * A), 1), (dict(out=8 * A + 8), 1),
                   (dict(k_strides=(64, 64, 63)), 1), (dict(out_strides=(1280, 640, 60)), 1),
                   (dict(scale=-0.5), 1), (dict(sel=None), 1), (dict(H=70000, Hkv=1), 2)):
        refused(dt.ditango_block_attn, status=st, **{**ok, **kw})
    assert dt.ditango_kv4_attn_workspace_size(100) == 0 < dt.ditango_kv4_attn_workspace_size(96)


def test_objects_refuse_bad_shapes_before_any_allocation():
    for kw in (dict(d=100), dict(H=3), dict(n_pages=0), dict(device="cpu"), dict(max_tokens=0)):
        a = dict(n_pages=4, Hkv=2, d=64, max_requests=2, max_blocks=3, max_tokens=8)
        a.update(kw)
        with pytest.raises(ValueError):
            dt.KV4Cache(**a)
    with pytest.raises(ValueError, match="CUDA"):
        dt.KV4Cache(4, 2, 64, 2, 3, 8, data=torch.zeros((4, 2, 64 * 72), dtype=torch.uint8))
    for kw in (dict(d=32), dict(Hkv=3), dict(k=-1), dict(band=-2), dict(Nk=0), dict(device="cpu")):
        a = dict(B=1, H=4, Nq=10, Nk=10, d=64, k=2)
        a.update(kw)
        with pytest.raises(ValueError):
            dt.BlockSparseAttention(**a)


# ---------------------------------------------------------------- the oracle's pins
def test_quantiser_reaches_every_value_within_half_a_step():
    rng = np.random.default_rng(0)
    for _ in range(200):
        x = (rng.standard_normal(64) * 10.0 ** rng.integers(-6, 6) + rng.standard_normal()).astype(np.float32)
        x = ((x.view(np.uint32) >> 16) << 16).view(np.float32).astype(np.float64)
        c, s, lo = OH.quantize_row(x)
        assert c.min() == 0 and c.max() <= 15 and OH.bf16_value(OH.bf16_bits(s)) == s
        assert np.abs(OH.row_values(c, s, lo) - x).max() <= s / 2
        assert s <= (x.max() - x.min()) / 15 * (1 + 2.0 ** -7)


def test_least_bf16_not_below():
    assert OH.least_bf16_not_below(1.0) == 1.0
    assert OH.least_bf16_not_below(1.0 + 1e-12) == 1.0 + 2.0 ** -7
    assert OH.least_bf16_not_below(0.0) == 0.0


def test_choose_and_scores_by_hand():
    assert OH.choose(np.array([1.0, 3, 3, 2]), {0}, 2) == [0, 1]
    assert OH.choose(np.array([1.0, 1, 1]), set(), 2) == [0, 1]
    assert OH.choose(np.array([1.0, 2]), {0, 1, 9, -1}, 1) == [0, 1]
    s = OH.scores(np.array([[1, -2]], np.int8), [0.5], np.array([[3, 4], [0, -1]], np.int8),
                  np.array([2.0, 1.0]))
    assert s.tolist() == [-5.0, 1.0]


def test_tables_by_hand():
    t, kv, off, slots, used, bad = OH.tables([63, 0], [2, 1], [7, 8, 9], [[4, 0], [0, 0]], 4)
    assert t.tolist() == [[4, 7], [8, 0]] and kv.tolist() == [65, 1] and off.tolist() == [0, 2, 3]
    assert slots.tolist() == [4 * 64 + 63, 7 * 64, 8 * 64, -1] and used == 2 and not bad
