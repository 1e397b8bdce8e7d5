"""The paged 4-bit history on the GPU against the fp64 oracle: tables, writing
and reading back, page summaries, attention of few and of many rows, and a run
of them together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_state_reuse_b200 as dt
from oracle import history as OH

import history_common as HC

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

PAGE = dt.PAGE


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x).tolist(), dtype=dtype, device="cuda")


# ---------------------------------------------------------------- tables
def run_tables(ctx, new, n_pages, width, max_tokens, free, table):
    R = len(ctx)
    c = dt.KV4Cache(n_pages, 1, 64, R, width, max_tokens, block_table=ints(table))
    c.tables(ints(ctx), ints(new), ints(free))
    torch.cuda.synchronize()
    return c


def check_tables(c, want):
    table, kv, off, slots, used, bad = want
    assert (c.block_table.cpu().numpy() == table).all()
    assert (c.kv_len.cpu().numpy() == kv).all()
    assert (c.q_off.cpu().numpy() == off).all()
    assert (c.slot_map.cpu().numpy() == slots).all()
    assert c.pages_used.item() == used
    assert c.status.item() == (5 if bad else 0)


@pytest.mark.parametrize("R,hi,new_hi,seed", [(1, 1, 1, 0), (1, 0, 300, 1), (7, 200, 3, 2), (64, 500, 1, 3),
                                              (300, 130, 70, 4), (1025, 70, 9, 5)])
def test_tables_match_the_definition(R, hi, new_hi, seed):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, hi + 1, R), rng.integers(0, new_hi + 1, R)
    width = int(max(-(-(ctx + new) // PAGE))) + 2
    n_pages = int(sum(-(-(ctx + new) // PAGE))) + 5
    perm = rng.permutation(n_pages)
    table, at = rng.integers(-5, 10 ** 9, (R, width)), 0    # entries behind the last page: anything
    for r in range(R):
        n = -(-int(ctx[r]) // PAGE)
        table[r, :n] = perm[at:at + n]
        at += n
    T = max(1, int(new.sum()) + 3)
    free = perm[at:]
    check_tables(run_tables(ctx, new, n_pages, width, T, free, table),
                 OH.tables(ctx, new, free, table, T))


@pytest.mark.parametrize("what", ["free list", "width", "negative context", "negative new", "slot map",
                                  "no free pages"])
def test_requests_that_do_not_fit_take_nothing(what):
    ctx, new = np.array([10, 100, 64, 0, 5]), np.array([3, 200, 1, 70, 2])
    width, T, n_pages = 6, 400, 40
    table = np.arange(30).reshape(5, 6)
    free = np.arange(30, 40)
    if what == "free list":
        free = free[:3]
    elif what == "no free pages":
        free = free[:0]
    elif what == "width":
        width, table = 4, table[:, :4]
    elif what == "negative context":
        ctx[2] = -7
    elif what == "negative new":
        new[1] = -1
    else:
        T = 250
    want = OH.tables(ctx, new, free, table, T)
    assert want[-1]
    check_tables(run_tables(ctx, new, n_pages, width, T, free, table), want)


def test_a_request_that_needs_nothing_fits_behind_one_that_does_not():
    """No free page left for the first request, too many tokens for the second:
    the third (room on its last page, if there are token places) and the fourth
    (idle) go on."""
    ctx, new, table = [64, 10, 70, 20], [1, 500, 3, 0], np.arange(12).reshape(4, 3)
    for T, fits in ((64, [False, False, False, True]), (1000, [False, False, True, True])):
        want = OH.tables(ctx, new, [], table, T)
        assert [k == c + n for k, c, n in zip(want[1], ctx, new)] == fits and want[-1]
        check_tables(run_tables(ctx, new, 12, 3, T, [], table), want)


def test_a_page_number_out_of_range_gives_no_slot():
    table = np.array([[3, 99, 0]])
    c = run_tables([100], [60], 8, 3, 64, [5], table)
    slots = c.slot_map.cpu().numpy()
    assert (slots[:28] == -1).all()                    # positions 100..127 lie in page 99 of 8
    assert (slots[28:60] == 5 * PAGE + np.arange(32)).all() and (slots[60:] == -1).all()
    assert c.status.item() == 5


# ---------------------------------------------------------------- write, read
def special_rows(d):
    """Rows where the quantiser can go wrong."""
    rng = np.random.default_rng(7)
    rows = [np.zeros(d), np.full(d, -0.0), np.full(d, 3.25), np.full(d, -1e30),
            np.where(np.arange(d) == 5, 1.0, 0.0), np.arange(d) % 16 * 1.0, np.arange(d) % 31 * 0.5,
            rng.standard_normal(d) * 1e-38, rng.standard_normal(d) * 1e-30, rng.standard_normal(d) * 1e37,
            np.where(np.arange(d) % 2 == 0, 3.3e38, -3.3e38), 100 + rng.standard_normal(d) * 0.5,
            np.where(np.arange(d) == 1, -100.0, rng.standard_normal(d) * 1e-6), rng.standard_normal(d)]
    for bad in (np.nan, np.inf, -np.inf):
        r = rng.standard_normal(d)
        r[d // 2] = bad
        rows.append(r)
    # ties: (x - least) / scale halfway between two codes
    tie = (np.arange(d) % 30) * 0.25
    tie[0], tie[1] = 0.0, 7.5
    rows.append(tie)
    return np.stack([HC.bf16_round(r) for r in rows])


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (18, 1), (67, 3), (700, 2)])
def test_write_is_exact_and_read_gives_the_values(d, T, Hkv):
    rng = np.random.default_rng(T * d + Hkv)
    K, V = HC.keys_values(rng, T, Hkv, d)
    if T == 18:
        K[:, 0] = special_rows(d)[:18]
        V[:, 0] = special_rows(d)[17::-1]
    n_pages = -(-T // PAGE) + 2
    slots = rng.permutation(n_pages * PAGE)[:T]
    slots[T // 2] = -1 if T > 1 else slots[0]
    want = HC.HostPages(n_pages, Hkv, d, fill=0xab)
    for t in range(T):
        for h in range(Hkv):
            if slots[t] >= 0:
                want.put(slots[t] // PAGE, slots[t] % PAGE, h, 0, K[t, h])
                want.put(slots[t] // PAGE, slots[t] % PAGE, h, 1, V[t, h])
    data = torch.full((n_pages, Hkv, PAGE * (d + 8)), 0xab, dtype=torch.uint8, device="cuda")
    c = dt.KV4Cache(n_pages, Hkv, d, 1, n_pages, T, data=data)
    # strided views: tokens of a wider tensor, heads of an interleaved one
    wide = torch.zeros((T, 2, Hkv, d + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, 0, :, :d] = HC.up(K)
    wide[:, 1, :, 8:] = HC.up(V)
    c.write(wide[:, 0, :, :d], wide[:, 1, :, 8:], ints(slots, torch.int64))
    torch.cuda.synchronize()
    got = data.cpu().numpy()
    bad = np.argwhere(got != want.data)
    # -0 and 0 are the same least value
    half = PAGE * d
    for p, h, b in bad:
        assert b >= half and got[p, h, b] % 128 == want.data[p, h, b] % 128 == 0, (p, h, b)
    Kr = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    Vr = Kr.clone()
    c.read(ints(slots, torch.int64), Kr, Vr)
    torch.cuda.synchronize()
    for t in range(T):
        for h in range(Hkv):
            for which, (x, r) in enumerate(((K, Kr), (V, Vr))):
                g = r[t, h].float().cpu().numpy().astype(np.float64)
                if slots[t] < 0:
                    assert (g == 7.0).all()
                    continue
                e = OH.row_values(*OH.quantize_row(x[t, h]))
                assert (np.isnan(g) == np.isnan(e)).all()
                if not np.isnan(e).any():
                    step = OH.quantize_row(x[t, h])[1]
                    tiny = 2.0 ** -133                       # half the least bf16 number
                    big = np.abs(e) * (2.0 ** -8 + 2.0 ** -23) + tiny
                    fin = np.isfinite(g)                     # 15 steps can pass the largest bf16
                    assert (np.abs(g - e)[fin] <= big[fin]).all()
                    assert (np.abs(e)[~fin] > 3.38e38).all()
                    assert (np.abs(e - x[t, h]) <= 0.5 * step * (1 + 1e-9)).all()
    assert c.status.item() == 0


def test_slots_out_of_range_are_left_out_and_recorded():
    c = dt.KV4Cache(3, 2, 64, 1, 1, 8)
    c.data.fill_(9)
    K, V = (HC.up(x) for x in HC.keys_values(np.random.default_rng(1), 4, 2, 64))
    c.write(K, V, ints([3 * PAGE, -1, 10 ** 15, -5], torch.int64))
    torch.cuda.synchronize()
    assert (c.data == 9).all() and c.status.item() == 5
    c.status.zero_()
    Kr, Vr = torch.full_like(K, 2.0), torch.full_like(V, 2.0)
    c.read(ints([3 * PAGE, -1, 10 ** 15, -5], torch.int64), Kr, Vr)
    torch.cuda.synchronize()
    assert (Kr == 2).all() and (Vr == 2).all() and c.status.item() == 5
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    c.write(e, e, torch.zeros(0, dtype=torch.int64, device="cuda"))     # no tokens: nothing to do


# ---------------------------------------------------------------- a filled cache
def filled(rng, kv, Hkv, d, H, T, fill=0xff, width=None):
    """A cache whose requests hold kv[r] tokens on random pages; every place
    without a token holds `fill` (0xff: scales that are NaN)."""
    need = [-(-n // PAGE) for n in kv]
    width = max(max(need), 1) if width is None else width
    n_pages = sum(need) + 2
    host = HC.HostPages(n_pages, Hkv, d, fill)
    perm = rng.permutation(n_pages)
    table = rng.integers(-3, n_pages + 3, (len(kv), width))
    at = 0
    for r, n in enumerate(kv):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
        K, V = HC.keys_values(rng, n, Hkv, d)
        for t in range(n):
            for h in range(Hkv):
                host.put(table[r, t // PAGE], t % PAGE, h, 0, K[t, h])
                host.put(table[r, t // PAGE], t % PAGE, h, 1, V[t, h])
    c = dt.KV4Cache(n_pages, Hkv, d, len(kv), width, max(T, 1), H=H,
                    data=torch.from_numpy(host.data.copy()).cuda(), block_table=ints(table))
    c.kv_len.copy_(ints(kv))
    return c, host, table


def check_attend(c, host, table, kv, q_lens, Q, out, lse, causal, lists=None, scale=None, what=""):
    d, H, Hkv = c.d, c.H, c.Hkv
    G = H // Hkv
    scale = d ** -0.5 if scale is None else scale
    got_o, got_l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    q = Q.float().cpu().numpy().astype(np.float64)
    at = 0
    for r, n in enumerate(q_lens):
        for h in range(Hkv):
            blocks = list(range(-(-kv[r] // PAGE))) if lists is None else lists[r][h]
            parts = [host.get(table[r, b], h) for b in blocks]
            pos = np.concatenate([b * PAGE + np.arange(PAGE) for b in blocks]) if blocks else np.zeros(0)
            k, v, y, x = (np.concatenate([p[i] for p in parts]) if parts else np.zeros((0, d))
                          for i in range(4))
            for t in range(n):
                seen = pos < (kv[r] - (n - 1 - t) if causal else kv[r])
                rows = q[at + t, h * G:(h + 1) * G]
                o, e, P = OH.attend_rows(rows, k[seen], v[seen], scale)
                dS = HC.logit_bound(rows, y[seen], scale, d)
                HC.check(got_o[at + t, h * G:(h + 1) * G], got_l[at + t, h * G:(h + 1) * G], o, e, P,
                         x[seen], v[seen], dS, out.dtype == torch.bfloat16, (what, r, h, t))
        at += n


def attend(c, q_lens, Q, out, lse, **kw):
    c.q_off.copy_(ints(np.concatenate([[0], np.cumsum(q_lens)])))
    c.attend(Q, out, lse, **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,kv,q_lens,causal", [
    (1, 1, [1], [1], False),
    (2, 2, [0, 1, 63, 64, 65, 200], [1, 1, 1, 1, 1, 1], True),
    (5, 1, [129, 0, 700], [1, 2, 0], True),
    (8, 2, [300, 5], [4, 9], True),          # 9 new tokens on 5 places: rows that see nothing
    (6, 2, [257], [37], True),
    (3, 3, [130, 64], [20, 1], False),
    (16, 1, [190], [1], False),
    (4, 2, [333, 90], [70, 90], True),
    (2, 1, [700, 0, 65], [129, 20, 1], True),     # many rows, none of them and few in one batch
    (3, 1, [1000], [300], False),
])
def test_attend_matches_the_oracle(d, H, Hkv, kv, q_lens, causal):
    rng = np.random.default_rng(d + H * 7 + sum(kv))
    T = sum(q_lens)
    c, host, table = filled(rng, kv, Hkv, d, H, T)
    Q = HC.up(HC.bf16_round(1.5 * rng.standard_normal((T, H, d))))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((T, H, d), 5.0, dtype=dtype, device="cuda")
        lse = torch.full((T, H), 5.0, device="cuda")
        attend(c, q_lens, Q, out, lse, max_q=max(q_lens), causal=causal)
        assert c.status.item() == 0
        check_attend(c, host, table, kv, q_lens, Q, out, lse, causal, what=str(dtype))


def with_ballast(rng, kv, Hkv, d, H, q_lens):
    """filled(), and one more request of so much work (600 queries over 20000
    tokens, all on one page) that the batch's many rows go to their own kernel."""
    n, pages = 600, -(-20000 // PAGE)
    c, host, table = filled(rng, list(kv) + [0], Hkv, d, H, sum(q_lens) + n, fill=0x11, width=pages)
    c.block_table[-1] = c.n_pages - 1
    c.kv_len[-1] = 20000
    return c, host, table, list(q_lens) + [n]


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,kv,q_lens,causal", [
    (5, 1, [129, 0, 700], [1, 2, 0], True),
    (8, 2, [300, 5], [4, 9], True),          # 9 new tokens on 5 places: rows that see nothing
    (6, 2, [257], [37], True),
    (3, 3, [130, 64], [20, 1], False),
    (4, 2, [333, 90], [70, 90], True),
    (2, 1, [700, 0, 65], [129, 20, 1], True),     # many rows, none of them and few in one batch
    (3, 1, [1000], [300], False),
])
def test_attend_in_a_batch_of_much_work_matches_the_oracle(d, H, Hkv, kv, q_lens, causal):
    rng = np.random.default_rng(d + H * 5 + sum(kv))
    T = sum(q_lens)
    c, host, table, all_q = with_ballast(rng, kv, Hkv, d, H, q_lens)
    Q = HC.up(HC.bf16_round(1.5 * rng.standard_normal((T + all_q[-1], H, d))))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full(Q.shape, 5.0, dtype=dtype, device="cuda")
        lse = torch.full(Q.shape[:2], 5.0, device="cuda")
        attend(c, all_q, Q, out, lse, max_q=max(all_q), causal=causal)
        assert c.status.item() == 0
        check_attend(c, host, table, kv, q_lens, Q[:T], out[:T], lse[:T], causal, what=str(dtype))


@pytest.mark.parametrize("d", [64, 96, 128])
def test_values_of_any_kind_in_a_batch_of_much_work(d):
    """What test_values_that_are_not_finite_stay_in_their_rows and
    test_scales_of_any_size do, in the kernel of many rows."""
    rng = np.random.default_rng(d)
    Hkv, H, n, q = 1, 2, 200, 30
    c, host, table, all_q = with_ballast(rng, [n, n], Hkv, d, H, [q, q])
    K, V = HC.keys_values(rng, n, Hkv, d)
    V[190] = 3e38                    # the last tokens: seen by the later rows only
    V[195, :, 3] = np.inf
    c.kv_len[:2] = n
    slots = ints([int(table[1, t // PAGE]) * PAGE + t % PAGE for t in range(n)], torch.int64)
    c.write(HC.up(K), HC.up(V), slots)
    Q = HC.up(HC.bf16_round(rng.standard_normal((2 * q + all_q[-1], H, d))))
    out, lse = torch.zeros(Q.shape, device="cuda"), torch.zeros(Q.shape[:2], device="cuda")
    attend(c, all_q, Q, out, lse, max_q=max(all_q), causal=True)
    assert c.status.item() == 0
    check_attend(c, host, table, [n, n], [q], Q[:q], out[:q], lse[:q], True)    # the request before: untouched
    got = out[q:2 * q].cpu().numpy()
    sees = np.arange(q) + n - (q - 1)                 # keys that row t sees
    assert np.isfinite(got[sees <= 195]).all() and np.isnan(got[sees > 195]).all()
    assert torch.isfinite(lse[q:2 * q]).all()


def test_attend_takes_strided_rows_and_leaves_the_others():
    rng = np.random.default_rng(5)
    d, H, Hkv, kv, q_lens, T = 96, 4, 2, [150, 70], [3, 2], 9     # four rows behind the last token
    c, host, table = filled(rng, kv, Hkv, d, H, T)
    q = HC.up(HC.bf16_round(rng.standard_normal((T, H, d))))
    wide = torch.zeros((T, H + 1, d + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:, :d] = q
    out = torch.full((H, T + 2, d), 5.0, device="cuda")             # head-major, as a state buffer
    lse = torch.full((H, T + 2), 5.0, device="cuda")
    attend(c, q_lens, wide[:, 1:, :d], out[:, :T].transpose(0, 1), lse[:, :T].transpose(0, 1),
           scale=0.25, max_q=1)     # a bound that is too small: only slower
    check_attend(c, host, table, kv, q_lens, q[:5], out[:, :5].transpose(0, 1), lse[:, :5].transpose(0, 1),
                 False, scale=0.25)
    assert (out[:, 5:] == 5).all() and (lse[:, 5:] == 5).all()


@pytest.mark.parametrize("H,Hkv,q", [(2, 2, 1), (10, 2, 1), (16, 1, 1), (4, 1, 40), (2, 2, 200)])
def test_one_long_request_is_split_and_joined_alike_every_time(H, Hkv, q):
    """More pages than blocks of the launch: every item is cut, and the joined
    result is the same bits run after run."""
    rng = np.random.default_rng(q)
    d, kv = 64, 64 * 700 + 13
    need = -(-kv // PAGE)
    host = HC.HostPages(need, Hkv, d)
    codes = rng.integers(0, 256, (need, Hkv, 64 * d), dtype=np.uint8)
    host.data[:, :, :64 * d] = codes
    s = HC.bf16_round(0.2 + 0.1 * rng.random((need, Hkv, 2, PAGE, 1)))
    lo = HC.bf16_round(-7.5 * s + 0.1 * rng.standard_normal(s.shape))
    meta = OH.bf16_bits(np.concatenate([s, lo], -1))
    host.data[:, :, 64 * d:] = meta.reshape(need, Hkv, -1).view(np.uint8).reshape(need, Hkv, -1)
    table = rng.permutation(need)[None]
    c = dt.KV4Cache(need, Hkv, d, 1, need, q, H=H, data=torch.from_numpy(host.data).cuda(),
                    block_table=ints(table))
    c.kv_len.copy_(ints([kv]))
    Q = HC.up(HC.bf16_round(rng.standard_normal((q, H, d))))
    out, lse = torch.empty((q, H, d), device="cuda"), torch.empty((q, H), device="cuda")
    attend(c, [q], Q, out, lse, causal=True)
    ref = out.clone(), lse.clone()
    rows = [0, q - 1]
    for t in sorted(set(rows)):
        k, v, y, x = (np.concatenate([host.get(p, 0)[i] for p in table[0]]) for i in range(4))
        n = kv - (q - 1 - t)
        qr = Q[t, :H // Hkv].float().cpu().numpy().astype(np.float64)
        o, e, P = OH.attend_rows(qr, k[:n], v[:n], d ** -0.5)
        HC.check(out[t, :H // Hkv].cpu().numpy().astype(np.float64),
                 lse[t, :H // Hkv].cpu().numpy().astype(np.float64), o, e, P, x[:n], v[:n],
                 HC.logit_bound(qr, y[:n], d ** -0.5, d), False, t)
    for _ in range(3):
        out.fill_(0)
        attend(c, [q], Q, out, lse, causal=True)
        assert (out == ref[0]).all() and (lse == ref[1]).all()


def test_listed_blocks_only():
    rng = np.random.default_rng(9)
    d, H, Hkv, kv, q_lens = 128, 6, 2, [400, 64, 1000], [1, 1, 5]
    c, host, table = filled(rng, kv, Hkv, d, H, 7)
    Q = HC.up(HC.bf16_round(rng.standard_normal((7, H, d))))
    lists = [[[0, 3, 6], [5]], [[0], []], [[15, 2, 7, 9], list(range(16))]]
    room = 17
    sel = np.full((3, Hkv, room), 123456)          # behind the count: anything
    count = np.zeros((3, Hkv))
    for r in range(3):
        for h in range(Hkv):
            sel[r, h, :len(lists[r][h])] = lists[r][h]
            count[r, h] = len(lists[r][h])
    out, lse = torch.empty((7, H, d), device="cuda"), torch.empty((7, H), device="cuda")
    attend(c, q_lens, Q, out, lse, sel=ints(sel), sel_count=ints(count.astype(int)), causal=True)
    assert c.status.item() == 0
    check_attend(c, host, table, kv, q_lens, Q, out, lse, True, lists)


def test_bad_pages_lists_and_offsets_are_recorded_and_not_followed():
    rng = np.random.default_rng(3)
    d, H, kv = 64, 2, [200, 100]
    Q = HC.up(HC.bf16_round(rng.standard_normal((2, H, d))))
    out, lse = torch.empty((2, H, d), device="cuda"), torch.empty((2, H), device="cuda")
    c, host, table = filled(rng, kv, H, d, H, 2)
    for bad in (c.n_pages, -1, 2 ** 30):
        c.block_table[0, 1] = bad
        c.status.zero_()
        attend(c, [1, 1], Q, out, lse)
        assert c.status.item() == 5
        check_attend(c, host, table, kv, [1, 1], Q, out, lse, False, [[[0, 2, 3]] * H, [[0, 1]] * H])
    c.block_table[0, 1] = int(table[0, 1])
    sel = ints([[[0, 2 ** 30, 2]] * H, [[-1, 1, 0]] * H])
    c.status.zero_()
    attend(c, [1, 1], Q, out, lse, sel=sel, sel_count=ints([[3] * H, [2] * H]))
    assert c.status.item() == 5
    check_attend(c, host, table, kv, [1, 1], Q, out, lse, False, [[[0, 2]] * H, [[1]] * H])
    # offsets past the rows, lengths past the table: clipped, and recorded
    c.status.zero_()
    out.fill_(5)
    c.q_off.copy_(ints([0, 1, 99]))
    c.attend(Q, out, lse, max_q=1)
    torch.cuda.synchronize()
    assert c.status.item() == 5 and (out[1] == 5).all() and (out[0] != 5).any()


def test_values_that_are_not_finite_stay_in_their_rows():
    """A NaN key reaches the rows that see it, and no others."""
    rng = np.random.default_rng(4)
    d, H, kv = 96, 2, [70, 70]
    c, host, table = filled(rng, kv, H, d, H, 4, fill=0)
    K, V = (HC.up(HC.bf16_round(rng.standard_normal((1, H, d)))) for _ in range(2))
    K[0, 1, 3] = float("nan")
    V[0, 0, 0] = float("inf")
    slot = int(table[0, 1]) * PAGE + 5                     # token 69 of request 0
    c.write(K, V, ints([slot], torch.int64))
    Q = HC.up(HC.bf16_round(rng.standard_normal((4, H, d))))
    out, lse = torch.empty((4, H, d), device="cuda"), torch.empty((4, H), device="cuda")
    attend(c, [2, 2], Q, out, lse, causal=True)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()     # row 0 does not see it
    assert torch.isnan(out[1]).all()
    assert torch.isnan(lse[1, 1]) and torch.isfinite(lse[1, 0])
    n = 40                                                  # the same with many rows
    c, host, table = filled(rng, kv, H, d, H, 2 * n, fill=0xff)
    slot = int(table[0, 1]) * PAGE + 3                      # token 67: seen by the last 3 rows of 40
    c.write(K, V, ints([slot], torch.int64))
    Q = HC.up(HC.bf16_round(rng.standard_normal((2 * n, H, d))))
    out, lse = torch.empty((2 * n, H, d), device="cuda"), torch.empty((2 * n, H), device="cuda")
    attend(c, [n, n], Q, out, lse, causal=True, max_q=n)
    assert torch.isfinite(out[:n - 3]).all() and torch.isfinite(out[n:]).all()
    assert torch.isnan(out[n - 3:n]).all()
    assert torch.isnan(lse[n - 3:n, 1]).all() and torch.isfinite(lse[n - 3:n, 0]).all()


@pytest.mark.parametrize("q", [1, 60])
def test_scales_of_any_size(q):
    """V rows from 2^-60 to 2^60 of each other, and Q rows as far apart: what
    is small beside what it is added to may be lost, nothing overflows."""
    rng = np.random.default_rng(q)
    d, H, n = 64, 2, 400
    c, host, table = filled(rng, [n], H, d, H, q)
    K, V = HC.keys_values(rng, n, H, d)
    V = HC.bf16_round(V * 2.0 ** np.linspace(-60, 60, n).round()[:, None, None])
    for t in range(n):
        for h in range(H):
            host.put(table[0, t // PAGE], t % PAGE, h, 1, V[t, h])
    c.data.copy_(torch.from_numpy(host.data))
    Q = HC.bf16_round(rng.standard_normal((q, H, d)))
    Q[0, 1] = HC.bf16_round(Q[0, 1] * 2.0 ** 40)       # one key takes all
    if q > 1:
        Q[1] = HC.bf16_round(Q[1] * 2.0 ** -100)       # all keys alike
        Q[2] = 0
    Q = HC.up(Q)
    out, lse = torch.empty((q, H, d), device="cuda"), torch.empty((q, H), device="cuda")
    attend(c, [q], Q, out, lse, max_q=q)
    # against the largest V at all: fp16 keeps 2^-25 of it
    got = out.cpu().numpy().astype(np.float64)
    qf = Q.float().cpu().numpy().astype(np.float64)
    for t in range(q):
        for h in range(H):
            parts = [host.get(p, h) for p in table[0]]
            k, v, y, x = (np.concatenate([p[i] for p in parts])[:n] for i in range(4))
            o, e, P = OH.attend_rows(qf[t, h:h + 1], k, v, d ** -0.5)
            dS = HC.logit_bound(qf[t, h:h + 1], y, d ** -0.5, d)
            if dS > 0.1:
                continue                                   # the logits themselves are not known to a unit
            tol = HC.EPS * (P @ np.abs(v)) + 2 * dS * (P @ np.abs(v)) + 2.0 ** -22 * np.abs(v).max()
            assert (np.abs(got[t, h] - o[0]) <= tol[0]).all(), (t, h)
            assert abs(lse[t, h].item() - e[0]) <= dS + 2.0 ** -18 * (1 + abs(e[0]))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


# ---------------------------------------------------------------- summaries, selection
@pytest.mark.parametrize("d", [64, 96, 128])
def test_page_summaries_and_selection_match_the_oracle(d):
    rng = np.random.default_rng(d)
    kv, Hkv, H = [1, 64, 500, 0, 1290], 2, 6
    c, host, table = filled(rng, kv, Hkv, d, H, 5)
    c.sum_codes.fill_(77)
    c.summarize(ints([0, 0, 0, 0, 0]))
    torch.cuda.synchronize()
    codes, scale = c.sum_codes.cpu().numpy(), c.sum_scale.cpu().numpy()
    for r, n in enumerate(kv):
        for b in range(-(-n // PAGE)):
            for h in range(Hkv):
                k = host.get(table[r, b], h)[0][:min(PAGE, n - b * PAGE)]
                wc, ws, _ = OH.summary(k)
                assert (codes[table[r, b], h] == wc).all() and scale[table[r, b], h] == ws
    # a summary does not depend on how the page was filled
    c.summarize(ints([0, 63, 499, 0, 1289]))
    torch.cuda.synchronize()
    assert (c.sum_codes.cpu().numpy() == codes).all() and (c.sum_scale.cpu().numpy() == scale).all()
    Q = HC.up(HC.bf16_round(rng.standard_normal((5, H, d))))
    q = Q.float().cpu().numpy().astype(np.float64)
    for k, band, sink in ((1, -1, 0), (4, 0, 1), (100, 1, 2), (0, 2, 0)):
        sel, count = c.select(Q, k, band, sink)
        torch.cuda.synchronize()
        assert c.status.item() == 0
        sel, count = sel.cpu().numpy(), count.cpu().numpy()
        for r, n in enumerate(kv):
            nb = -(-n // PAGE)
            for h in range(Hkv):
                qs = [OH.summary(q[r, g:g + 1]) for g in range(h * 3, h * 3 + 3)]
                sc = OH.scores([x[0] for x in qs], [x[1] for x in qs], codes[table[r, :nb], h],
                               scale[table[r, :nb], h])
                forced = set(range(sink)) | (set(range(nb - 1 - band, nb + band)) if band >= 0 else set())
                want = OH.choose(sc, forced, k)
                assert count[r, h] == len(want) and sel[r, h, :len(want)].tolist() == want
                assert (sel[r, h, len(want):] == -1).all()


def test_selection_over_a_long_table_and_with_fewer_requests():
    """More places than the scores of all heads fit beside one another; then a
    batch of fewer requests with the same widths."""
    rng = np.random.default_rng(17)
    kv, Hkv, H, d, k = [900, 64, 3000], 1, 16, 64, 7
    c, host, table = filled(rng, kv, Hkv, d, H, 3)
    long_ = dt.KV4Cache(c.n_pages, Hkv, d, 3, 6000, 3, H=H, data=c.data)
    long_.block_table[:, :table.shape[1]] = c.block_table
    long_.kv_len.copy_(c.kv_len)
    Q = HC.up(HC.bf16_round(rng.standard_normal((3, H, d))))
    got = []
    for x in (c, long_):
        x.summarize(ints([0, 0, 0]))
        sel, count = x.select(Q, k, band=0, sink=1)
        torch.cuda.synchronize()
        assert x.status.item() == 0
        got.append((sel.cpu(), count.cpu()))
        x.n_requests = 2
        sel2, count2 = x.select(Q[:2], k, band=0, sink=1)
        torch.cuda.synchronize()
        x.n_requests = 3
        assert torch.equal(sel2.cpu(), got[-1][0][:2]) and torch.equal(count2.cpu(), got[-1][1][:2])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][1].tolist() == [[7], [1], [7]]


@pytest.mark.parametrize("d", [64, 96, 128])
def test_single_queries_of_any_size_and_equal_scores(d):
    """Both ways to a single query's list (its codes formed by the selection, or
    before it) and the oracle agree on rows of huge, tiny, zero and not finite
    values, and on pages that are all alike (ties)."""
    rng = np.random.default_rng(d)
    kv, Hkv, H = [1500] * 6, 2, 4
    c, host, table = filled(rng, kv, Hkv, d, H, 6)
    q = HC.bf16_round(rng.standard_normal((6, H, d)))
    q[0] *= 2.0 ** 126 / 2
    q[1] = HC.bf16_round(q[1] * 2.0 ** -128)
    q[2] = 0
    q[3, 1, 5] = np.inf
    q[4] = HC.bf16_round(np.sign(q[4]) * 2.0 ** 127 * 1.9)
    Q = HC.up(q)
    q = Q.float().cpu().numpy().astype(np.float64)
    long_ = dt.KV4Cache(c.n_pages, Hkv, d, 6, 14000, 6, H=H, data=c.data)
    long_.block_table[:, :table.shape[1]] = c.block_table
    long_.kv_len.copy_(c.kv_len)
    for alike in (False, True):
        for x in (c, long_):
            x.summarize(ints([0] * 6))
            if alike:
                x.sum_codes.fill_(3)
                x.sum_scale.fill_(0.25)
        codes, scale = c.sum_codes.cpu().numpy(), c.sum_scale.cpu().numpy()
        for k, band, sink in ((5, 0, 1), (24, -1, 0), (1, -1, 0)):
            got = [[t.cpu() for t in x.select(Q, k, band, sink)] for x in (c, long_)]
            assert all(torch.equal(a, b) for a, b in zip(*got))
            for r in range(6):
                for h in range(Hkv):
                    qs = [OH.summary(q[r, g:g + 1]) for g in range(2 * h, 2 * h + 2)]
                    with np.errstate(all="ignore"):
                        sc = OH.scores([x[0] for x in qs], [x[1] for x in qs], codes[table[r, :24], h],
                                       scale[table[r, :24], h])
                    forced = set(range(sink)) | ({23} if band == 0 else set())
                    want = OH.choose(sc, forced, k)
                    assert got[0][0][r, h, :len(want)].tolist() == want and got[0][1][r, h] == len(want)


def test_pages_past_four_gib():
    """The same tokens on the first pages of a small cache and on the last ones of
    a cache of more than 2^32 bytes: every result is the same."""
    rng = np.random.default_rng(23)
    Hkv, H, d, n, many = 8, 16, 128, 700, 62000
    assert many * Hkv * PAGE * (d + 8) > 2 ** 32
    need = -(-n // PAGE)
    K, V = (HC.up(x) for x in HC.keys_values(rng, n, Hkv, d))
    Q1, Q2 = (HC.up(HC.bf16_round(rng.standard_normal((t, H, d)))) for t in (1, 40))
    got = []
    for pages, first in ((need, 0), (many, many - need)):
        c = dt.KV4Cache(pages, Hkv, d, 1, need, n, H=H)
        c.tables(ints([0]), ints([n]), torch.arange(first, first + need, dtype=torch.int32, device="cuda"))
        c.write(K, V)
        c.summarize(ints([0]))
        back = torch.zeros((2, n, Hkv, d), dtype=torch.bfloat16, device="cuda")
        c.read(c.slot_map, back[0], back[1])
        sel, count = c.select(Q1, 5, band=0, sink=1)
        res = [back, sel, count]
        for Q in (Q1, Q2):
            out = torch.zeros((len(Q), H, d), device="cuda")
            lse = torch.zeros((len(Q), H), device="cuda")
            attend(c, [len(Q)], Q, out, lse, causal=True)
            res += [out, lse]
        assert c.status.item() == 0
        got.append([x.cpu() for x in res])
        del c
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------- together
def test_a_batch_of_steps_together_and_in_a_graph():
    """Tables, write, summaries, selection and attention of a growing batch;
    the last step again as a captured and replayed graph."""
    rng = np.random.default_rng(11)
    R, Hkv, H, d, n_pages, width = 3, 2, 4, 128, 40, 9
    c = dt.KV4Cache(n_pages, Hkv, d, R, width, 256, H=H)
    host = HC.HostPages(n_pages, Hkv, d)
    free = rng.permutation(n_pages)
    ctx, used = np.zeros(R, int), 0
    table = np.zeros((R, width), int)
    ctx_t = torch.zeros(R, dtype=torch.int32, device="cuda")
    for new in ([100, 3, 0], [64, 60, 64], [1, 1, 1], [1, 1, 1]):
        new = np.array(new)
        T = int(new.sum())
        K, V = HC.keys_values(rng, T, Hkv, d)
        Q = HC.up(HC.bf16_round(rng.standard_normal((T, H, d))))
        want = OH.tables(ctx, new, free[used:], table, 256)
        c.tables(ctx_t, ints(new), ints(free[used:]))
        c.write(HC.up(K), HC.up(V))
        c.summarize(ctx_t)
        out, lse = torch.empty((T, H, d), device="cuda"), torch.empty((T, H), device="cuda")
        c.attend(Q, out, lse, max_q=int(new.max()), causal=True)
        torch.cuda.synchronize()
        table, kv, off, slots, n_used, bad = want
        assert not bad and c.status.item() == 0 and c.pages_used.item() == n_used
        for t in range(T):
            for h in range(Hkv):
                host.put(slots[t] // PAGE, slots[t] % PAGE, h, 0, K[t, h])
                host.put(slots[t] // PAGE, slots[t] % PAGE, h, 1, V[t, h])
        check_attend(c, host, table, kv, new, Q, out, lse, True)
        ctx, used = kv, used + n_used
        ctx_t.copy_(c.kv_len)
    # single tokens over selected pages, eager and as a graph on another stream
    before = ints(ctx - 1)
    one, fr = ints([1, 1, 1]), ints(free[used:])
    Kt, Vt = HC.up(K), HC.up(V)

    def step():
        c.tables(before, one, fr)
        c.write(Kt, Vt)
        c.summarize(before)
        sel, count = c.select(Q, 2, band=0, sink=1)
        c.attend(Q, out, lse, max_q=1, sel=sel, sel_count=count)
        return sel, count

    sel, count = step()
    torch.cuda.synchronize()
    lists = [[sel[r, h, :count[r, h]].tolist() for h in range(Hkv)] for r in range(R)]
    assert all(len(x) == min(2, -(-int(ctx[r]) // PAGE)) for r in range(R) for x in lists[r])
    check_attend(c, host, table, ctx, [1, 1, 1], Q, out, lse, False, lists)
    ref = out.clone(), lse.clone(), sel.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (out == ref[0]).all() and (lse == ref[1]).all() and (sel == ref[2]).all()
    assert c.status.item() == 0


def test_objects_on_two_streams_do_not_touch_each_other():
    rng = np.random.default_rng(21)
    d, H, kv = 128, 8, [3000, 900]
    runs = []
    for _ in range(2):
        c, host, table = filled(rng, kv, 1, d, H, 2)
        Q = HC.up(HC.bf16_round(rng.standard_normal((2, H, d))))
        c.q_off.copy_(ints([0, 1, 2]))
        runs.append((c, host, table, Q, torch.empty((2, H, d), device="cuda"),
                     torch.empty((2, H), device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, _, _, Q, out, lse, s in runs:
            c.attend(Q, out, lse, max_q=1, stream=s)
    torch.cuda.synchronize()
    for c, host, table, Q, out, lse, _ in runs:
        check_attend(c, host, table, kv, [1, 1], Q, out, lse, False)


def test_history_state_merges_with_the_partitions_states():
    """A chunk of new tokens as partition 1 after a history held in 4 bits
    (partition 0): the history's state is written into its slot of the state
    buffer, the chunk's own is fresh, and the merge joins them."""
    rng = np.random.default_rng(31)
    H, d, n0, n1 = 2, 128, 320, 200
    c, host, table = filled(rng, [n0], H, d, H, n1)
    pa = dt.PartitionedAttention(1, H, n0 + n1, d, [0, n0, n0 + n1])
    qkv = [HC.bf16_round(rng.standard_normal((H, n0 + n1, d))) for _ in range(3)]
    Q, K, V = (HC.up(x)[None] for x in qkv)
    pa.plan.copy_(torch.tensor([0, 0, 2, 1], dtype=torch.int8))      # (1, 0) reused, (1, 1) fresh
    pa.fresh_list[0] = 3
    pa.counts.copy_(ints([1, 1]))
    slot = dt.ditango_slot_table(pa.geom)[1]
    pa.partial(Q, K, V)
    rows = Q[0, :, n0:].transpose(0, 1)                                # [n1, H, d], strided
    c.q_off.copy_(ints([0, n1]))
    c.attend(rows, pa.state_O[slot[0], :, :n1].transpose(0, 1), pa.state_lse[slot[0], :, :n1].t(),
             max_q=n1)
    out = torch.empty((1, H, n0 + n1, d), device="cuda")
    out_lse = torch.empty((1, H, n0 + n1), device="cuda")
    pa.merge(out, out_lse)
    torch.cuda.synchronize()
    assert pa.status.item() == 0 and c.status.item() == 0
    for h in range(H):
        parts = [host.get(p, h) for p in table[0]]
        k = np.concatenate([p[0] for p in parts] + [qkv[1][h, n0:]])
        v = np.concatenate([p[1] for p in parts] + [qkv[2][h, n0:]])
        y = np.concatenate([p[2] for p in parts] + [np.abs(qkv[1][h, n0:])])
        x = np.concatenate([p[3] for p in parts] + [np.abs(qkv[2][h, n0:])])
        keep = np.r_[:n0, len(k) - n1:len(k)]
        q = qkv[0][h, n0:].astype(np.float64)
        o, e, P = OH.attend_rows(q, k[keep], v[keep], d ** -0.5)
        HC.check(out[0, h, n0:].cpu().numpy().astype(np.float64),
                 out_lse[0, h, n0:].cpu().numpy().astype(np.float64), o, e, P, x[keep], v[keep],
                 HC.logit_bound(q, y[keep], d ** -0.5, d), False, h)
