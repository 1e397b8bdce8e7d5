"""Block summaries, selection and attention over selected key blocks on the
GPU against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_state_reuse_b200 as dt
from oracle import history as OH

import history_common as HC

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

PAGE, QB = dt.PAGE, dt.QBLOCK


def ints(x):
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def strided(x, how):
    """The bf16 tensor of x [B, H, N, d]: packed, or a view of a wider one."""
    t = HC.up(x)
    if how == "packed":
        return t
    B, H, N, d = t.shape
    wide = torch.full((B, N + 3, H, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, 1:N + 1, :, 8:].transpose(1, 2)
    view.copy_(t)
    return view


def block_lists(sel, count):
    return [[[sel[b, g, i, :count[b, g, i]].tolist() for i in range(sel.shape[2])]
             for g in range(sel.shape[1])] for b in range(sel.shape[0])]


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,k,band,sink,k_len", [
    (1, 1, 1, 1, 1, 1, 0, 0, None),
    (1, 2, 2, 300, 1000, 4, 1, 1, None),
    (2, 6, 2, 1000, 640, 3, -1, 0, [640, 130]),
    (2, 2, 1, 129, 2500, 50, 2, 3, [0, 2499]),
    (1, 3, 3, 2600, 70, 0, 0, 0, None),
])
def test_selection_matches_the_oracle(d, B, H, Hkv, Nq, Nk, k, band, sink, k_len):
    rng = np.random.default_rng(d + Nq + Nk)
    q = HC.bf16_round(rng.standard_normal((B, H, Nq, d)))
    kk = HC.bf16_round(rng.standard_normal((B, Hkv, Nk, d)))
    kk[:, :, :PAGE] = 0                        # a block of zeros: codes 0, scale 0, ties with nothing
    if k_len is not None:
        for b in range(B):
            kk[b, :, k_len[b]:] = np.nan       # behind the valid keys: anything
    op = dt.BlockSparseAttention(B, H, Nq, Nk, d, k, band, sink, Hkv=Hkv)
    sel, count = op.select(strided(q, "view"), strided(kk, "packed"),
                           None if k_len is None else ints(k_len))
    torch.cuda.synchronize()
    assert op.status.item() == 0
    sel, count = sel.cpu().numpy(), count.cpu().numpy()
    for b in range(B):
        n_keys = Nk if k_len is None else k_len[b]
        nk = -(-n_keys // PAGE)
        for g in range(Hkv):
            ks = [OH.summary(kk[b, g, j * PAGE:min(n_keys, (j + 1) * PAGE)].astype(np.float64))
                  for j in range(nk)]
            for j in range(nk):
                assert (op.k_codes[b, g, j].cpu().numpy() == ks[j][0]).all()
                assert op.k_scale[b, g, j].item() == ks[j][1]
                np.testing.assert_allclose(op.k_mean[b, g, j].cpu().numpy(), ks[j][2], rtol=2 ** -23, atol=1e-30)
            for i in range(op.n_q):
                rows = [q[b, h, i * QB:(i + 1) * QB].astype(np.float64)
                        for h in range(g * (H // Hkv), (g + 1) * (H // Hkv))]
                qs = [OH.summary(r) for r in rows]
                sc = OH.scores([x[0] for x in qs], [x[1] for x in qs],
                               np.array([x[0] for x in ks]).reshape(nk, d), np.array([x[1] for x in ks], np.float32))
                forced = set(range(sink))
                if band >= 0:
                    forced |= set(range(2 * i - band, 2 * i + 2 + band))
                want = OH.choose(sc, forced, k)
                assert count[b, g, i] == len(want), (b, g, i)
                assert sel[b, g, i, :len(want)].tolist() == want, (b, g, i)
                assert (sel[b, g, i, len(want):] == -1).all()


def test_ties_go_to_the_lower_block():
    """Equal key blocks: all scores tie, the first k are taken; a pattern of
    two values takes every larger one first."""
    d, nk, k = 64, 300, 37
    rng = np.random.default_rng(0)
    row = HC.bf16_round(rng.standard_normal(d))
    q = np.broadcast_to(row, (1, 1, QB, d))
    for pattern in (np.ones(nk), 1.0 + (np.arange(nk) % 7 == 3), -1.0 - (np.arange(nk) % 2)):
        kk = np.repeat(pattern, PAGE)[None, None, :, None] * row
        op = dt.BlockSparseAttention(1, 1, QB, nk * PAGE, d, k, -1, 0)
        sel, count = op.select(HC.up(q), HC.up(kk))
        torch.cuda.synchronize()
        want = sorted(np.argsort(-pattern, kind="stable")[:k].tolist())
        assert count.item() == k and sel[0, 0, 0].tolist() == want


def test_many_key_blocks_leave_fewer_rows_a_block():
    """More key blocks than 16 rows of scores fit: 8, 4, 2 and 1 rows."""
    rng = np.random.default_rng(3)
    for nk in (1700, 3400, 7000, 26000, 51200):
        d, n_q, k = 64, 5, 9
        kc = rng.integers(-127, 128, (nk, d)).astype(np.int8)
        qc = rng.integers(-127, 128, (n_q, d)).astype(np.int8)
        ks, qs = rng.random(nk).astype(np.float32), rng.random(n_q).astype(np.float32)
        dev = [torch.from_numpy(x).cuda() for x in (qc, qs, kc, ks)]
        sel = torch.zeros((n_q, k), dtype=torch.int32, device="cuda")
        count = torch.zeros(n_q, dtype=torch.int32, device="cuda")
        dt.ditango_block_select(1, 1, 1, n_q, nk, d, k, -1, 0, 2, k, *dev, sel, count)
        torch.cuda.synchronize()
        for i in range(n_q):
            want = OH.choose(OH.scores([qc[i]], [qs[i]], kc, ks), set(), k)
            assert sel[i].tolist() == want, (nk, i)


def check_attend(q, kk, v, sel, count, out, lse, n_keys, scale=None):
    B, H, Nq, d = q.shape
    G = H // kk.shape[1]
    scale = d ** -0.5 if scale is None else scale
    got_o, got_l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        for h in range(H):
            for i in range(sel.shape[2]):
                blocks = [j for j in sel[b, h // G, i, :count[b, h // G, i]]]
                at = np.concatenate([np.arange(j * PAGE, max(j * PAGE, min(n_keys[b], (j + 1) * PAGE)))
                                     for j in blocks] or [np.zeros(0)]).astype(int)
                rows = slice(i * QB, min(Nq, (i + 1) * QB))
                qr = q[b, h, rows].astype(np.float64)
                k_, v_ = kk[b, h // G, at].astype(np.float64), v[b, h // G, at].astype(np.float64)
                o, e, P = OH.attend_rows(qr, k_, v_, scale)
                HC.check(got_o[b, h, rows], got_l[b, h, rows], o, e, P, v_, v_,
                         HC.logit_bound(qr, np.abs(k_), scale, d), out.dtype == torch.bfloat16, (b, h, i))


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,most,k_len,how,dtype", [
    (1, 1, 1, 1, 1, 1, None, "packed", torch.float32),
    (1, 2, 2, 127, 64, 1, None, "packed", torch.bfloat16),
    (2, 4, 2, 1000, 1333, 9, None, "view", torch.bfloat16),
    (2, 2, 1, 257, 700, 11, [130, 0], "view", torch.float32),
    (1, 3, 3, 128, 4097, 65, [4097], "packed", torch.float32),
    (3, 1, 1, 300, 500, 8, [500, 1, 449], "packed", torch.bfloat16),
])
def test_attention_over_listed_blocks_matches_the_oracle(d, B, H, Hkv, Nq, Nk, most, k_len, how, dtype):
    rng = np.random.default_rng(d + Nq + Nk)
    q = HC.bf16_round(1.5 * rng.standard_normal((B, H, Nq, d)))
    kk = HC.bf16_round(rng.standard_normal((B, Hkv, Nk, d)))
    v = HC.bf16_round(rng.standard_normal((B, Hkv, Nk, d)))
    n_q, nk = -(-Nq // QB), -(-Nk // PAGE)
    n_keys = [Nk] * B if k_len is None else k_len
    for b in range(B):                       # behind the valid keys: NaN and infinities
        kk[b, :, n_keys[b]:] = np.nan
        v[b, :, n_keys[b]:] = np.inf
    sel = np.full((B, Hkv, n_q, most + 1), 10 ** 6)      # behind the count: anything
    count = np.zeros((B, Hkv, n_q), int)
    for b in range(B):
        for g in range(Hkv):
            for i in range(n_q):
                n = min(most, nk) if rng.random() < 0.5 else int(rng.integers(0, min(most, nk) + 1))
                sel[b, g, i, :n] = rng.permutation(nk)[:n]     # any order
                count[b, g, i] = n
    op = dt.BlockSparseAttention(B, H, Nq, Nk, d, most, Hkv=Hkv)
    wide = torch.full((B, Nq + 2, H, d + 8), 5.0, dtype=dtype, device="cuda")
    out = wide[:, 1:Nq + 1, :, :d].transpose(1, 2)
    lse = torch.full((B, H, Nq), 5.0, device="cuda")
    op.attend(strided(q, how), strided(kk, how), strided(v, how), out, lse, ints(sel), ints(count),
              None if k_len is None else ints(k_len))
    torch.cuda.synchronize()
    assert op.status.item() == 0
    check_attend(q, kk, v, sel, count, out, lse, n_keys)
    assert (wide[:, 0] == 5).all() and (wide[:, -1] == 5).all() and (wide[..., d:] == 5).all()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,most,k_len,how,dtype", [
    (1, 100, 50, 60, 900, 14, None, "packed", torch.bfloat16),            # two parts
    (1, 60, 30, 60, 700, 10, None, "packed", torch.float32),              # four
    (2, 2, 1, 200, 3000, 40, [3000, 70], "view", torch.bfloat16),         # eight, most of them empty in one entry
    (1, 1, 1, 129, 1500, 23, None, "packed", torch.float32),
])
def test_lists_cut_into_parts(d, B, H, Hkv, Nq, Nk, most, k_len, how, dtype):
    """Few query blocks: their lists are shared out over blocks of threads; lists of
    any length, some without a tile for every part."""
    test_attention_over_listed_blocks_matches_the_oracle(d, B, H, Hkv, Nq, Nk, most, k_len, how, dtype)


def test_parts_of_a_list_give_the_same_bits_and_replay():
    op = dt.BlockSparseAttention(1, 2, 200, 5000, 64, 40)
    g = torch.Generator(device="cuda").manual_seed(1)
    Q, K, V = (torch.randn((1, 2, n, 64), generator=g, device="cuda").bfloat16() for n in (200, 5000, 5000))
    out, lse = torch.empty((1, 2, 200, 64), device="cuda"), torch.empty((1, 2, 200), device="cuda")
    op.step(Q, K, V, out, lse)
    torch.cuda.synchronize()
    ref = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.step(Q, K, V, out, lse)
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    assert op.status.item() == 0


def test_entries_and_counts_out_of_range_are_empty_and_recorded():
    rng = np.random.default_rng(2)
    d, Nq, Nk = 128, 200, 320
    q, kk, v = (HC.bf16_round(rng.standard_normal((1, 1, n, d))) for n in (Nq, Nk, Nk))
    op = dt.BlockSparseAttention(1, 1, Nq, Nk, d, 4)
    out, lse = torch.empty((1, 1, Nq, d), device="cuda"), torch.empty((1, 1, Nq), device="cuda")
    for bad in (5, -1, 2 ** 30):
        op.status.zero_()
        sel = np.array([[[[bad, 2, 0, 4], [3, bad, bad, 1]]]])
        op.attend(HC.up(q), HC.up(kk), HC.up(v), out, lse, ints(sel), ints([[[4, 3]]]))
        torch.cuda.synchronize()
        assert op.status.item() == 5
        check_attend(q, kk, v, np.array([[[[2, 0, 4], [3, 0, 0]]]]), np.array([[[3, 1]]]), out, lse, [Nk])
    op.status.zero_()
    sel = np.array([[[[0, 1, 2, 3], [0, 1, 2, 3]]]])
    op.attend(HC.up(q), HC.up(kk), HC.up(v), out, lse, ints(sel), ints([[[9, -3]]]))
    torch.cuda.synchronize()
    assert op.status.item() == 5
    check_attend(q, kk, v, sel, np.array([[[4, 0]]]), out, lse, [Nk])


def test_a_nan_key_block_reaches_only_those_that_list_it():
    rng = np.random.default_rng(8)
    d, Nq, Nk = 64, 256, 256
    q, kk, v = (HC.bf16_round(rng.standard_normal((1, 1, n, d))) for n in (Nq, Nk, Nk))
    v[0, 0, 70] = np.inf
    kk[0, 0, 200, 3] = np.nan
    op = dt.BlockSparseAttention(1, 1, Nq, Nk, d, 4)
    out, lse = torch.empty((1, 1, Nq, d), device="cuda"), torch.empty((1, 1, Nq), device="cuda")
    sel = np.array([[[[0, 2, 0, 0], [1, 3, 2, 0]]]])
    op.attend(HC.up(q), HC.up(kk), HC.up(v), out, lse, ints(sel), ints([[[2, 3]]]))
    torch.cuda.synchronize()
    check_attend(q[:, :, :QB], kk, v, sel[:, :, :1], np.array([[[2]]]), out[:, :, :QB], lse[:, :, :QB], [Nk])
    assert torch.isnan(out[0, 0, QB:]).all() and torch.isnan(lse[0, 0, QB:]).all()


def test_every_block_listed_is_dense_attention_and_the_step_replays():
    """With all blocks listed the operator gives the partitions' attention;
    a captured step gives the eager step's bits."""
    rng = np.random.default_rng(6)
    B, H, N, d = 1, 3, 1111, 96
    q, kk, v = (HC.up(HC.bf16_round(rng.standard_normal((B, H, N, d)))) for _ in range(3))
    nk = -(-N // PAGE)
    op = dt.BlockSparseAttention(B, H, N, N, d, nk)
    out, lse = torch.empty((B, H, N, d), device="cuda"), torch.empty((B, H, N), device="cuda")
    op.step(q, kk, v, out, lse)
    pa = dt.PartitionedAttention(B, H, N, d, [0, N])
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    pa.step(q, kk, v, ref, ref_lse, anchor=True)
    torch.cuda.synchronize()
    assert (op.sel_count == nk).all()
    # both round the probabilities once: twice 2^-8 of sum P |v| <= max |v|
    assert (out - ref).abs().max().item() <= 2 * HC.EPS * v.float().abs().max().item()
    assert (lse - ref_lse).abs().max().item() <= 1e-4
    op = dt.BlockSparseAttention(B, H, N, N, d, 5, band=1, sink=1)
    op.step(q, kk, v, out, lse)
    torch.cuda.synchronize()
    ref = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        op.step(q, kk, v, out, lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (out == ref).all()
    sel, count = op.sel.cpu().numpy(), op.sel_count.cpu().numpy()
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    check_attend(f(q), f(kk), f(v), sel, count, out, lse, [N])
