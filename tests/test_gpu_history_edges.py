"""The 4-bit history where its arithmetic meets its limits: rows of zeros, masked
places and empty tiles, values far from one another, and large sizes; against the
fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_state_reuse_b200 as dt
from oracle import history as OH

import history_common as HC
from test_history_checks_rows import tie_row

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

PAGE = dt.PAGE
BALLAST = 1200        # queries of the request that makes a batch's work large, over 20000 tokens


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x).tolist(), dtype=dtype, device="cuda")


class Batch:
    """Requests with given keys and values (fp32 numpy of bf16 values, [kv, Hkv, d]
    each), quantised by the oracle.  `many`: one more request of so much work that
    the rows of the others go to the kernel of many rows, if they are more than 16."""

    def __init__(self, rng, kvs, H, q_lens, many, d, fill=0xff):
        self.H, self.d, self.q_lens, self.many = H, d, list(q_lens), many
        self.Hkv = kvs[0][0].shape[1]
        self.kv = [len(k) for k, _ in kvs]
        need = [-(-n // PAGE) for n in self.kv]
        width = max(max(need), 1, -(-20000 // PAGE) if many else 1)
        n_pages = sum(need) + 2
        R = len(kvs) + many
        self.host = HC.HostPages(n_pages, self.Hkv, d, fill)
        self.host.data[-1] = 0x11
        perm = rng.permutation(n_pages - 1)
        self.table = np.full((R, width), 2 ** 30)
        at = 0
        for r, (K, V) in enumerate(kvs):
            self.table[r, :need[r]] = perm[at:at + need[r]]
            at += need[r]
            for t in range(len(K)):
                for h in range(self.Hkv):
                    page = self.table[r, t // PAGE]
                    self.host.put(page, t % PAGE, h, 0, K[t, h])
                    self.host.put(page, t % PAGE, h, 1, V[t, h])
        all_q = self.q_lens + [BALLAST] * many
        if many:
            self.table[-1] = n_pages - 1
        self.T, self.rows = sum(self.q_lens), sum(all_q)
        self.max_q = max(all_q)
        self.c = dt.KV4Cache(n_pages, self.Hkv, d, R, width, max(self.rows, 1), H=H,
                             data=torch.from_numpy(self.host.data.copy()).cuda(), block_table=ints(self.table))
        self.c.kv_len.copy_(ints(self.kv + [20000] * many))
        self.c.q_off.copy_(ints(np.concatenate([[0], np.cumsum(all_q)])))

    def attend(self, q, causal, scale=0.0, lists=None, room=None, dtype=torch.float32):
        """O and lse (fp64 numpy) of q [T, H, d] (fp32 numpy of bf16 values)."""
        Q = torch.zeros((self.rows, self.H, self.d), dtype=torch.bfloat16, device="cuda")
        Q[:self.T] = HC.up(q)
        out = torch.full(Q.shape, 5.0, dtype=dtype, device="cuda")
        lse = torch.full(Q.shape[:2], 5.0, device="cuda")
        sel = count = None
        if lists is not None:
            R = len(self.table)
            sel, count = np.full((R, self.Hkv, room), 123456), np.zeros((R, self.Hkv), int)
            for r, of_r in enumerate(lists):
                for h, x in enumerate(of_r):
                    sel[r, h, :len(x)], count[r, h] = x, len(x)
            if self.many:
                sel[-1], count[-1] = np.arange(room), room
            sel, count = ints(sel), ints(count)
        self.c.attend(Q, out, lse, max_q=self.max_q, causal=causal, scale=scale, sel=sel, sel_count=count)
        torch.cuda.synchronize()
        return (out[:self.T].float().cpu().numpy().astype(np.float64),
                lse[:self.T].cpu().numpy().astype(np.float64))

    def rows_of(self, r, h, lists=None):
        """(k, v, y, x, positions) of what request r holds (or lists) for key head h."""
        blocks = list(range(-(-self.kv[r] // PAGE))) if lists is None else lists[r][h]
        parts = [self.host.get(self.table[r, b], h) for b in blocks]
        pos = np.concatenate([b * PAGE + np.arange(PAGE) for b in blocks]) if blocks else np.zeros(0)
        return [np.concatenate([p[i] for p in parts]) if parts else np.zeros((0, self.d))
                for i in range(4)] + [pos]

    def check(self, q, got_o, got_l, causal, scale=None, lists=None, bf16=False, rows=None):
        scale = self.d ** -0.5 if scale is None else scale
        G, at = self.H // self.Hkv, 0
        for r, n in enumerate(self.q_lens):
            for h in range(self.Hkv):
                k, v, y, x, pos = self.rows_of(r, h, lists)
                for t in range(n) if rows is None else rows:
                    seen = pos < (self.kv[r] - (n - 1 - t) if causal else self.kv[r])
                    g = slice(h * G, (h + 1) * G)
                    qr = q[at + t, g].astype(np.float64)
                    o, e, P = OH.attend_rows(qr, k[seen], v[seen], scale)
                    HC.check(got_o[at + t, g], got_l[at + t, g], o, e, P, x[seen], v[seen],
                             HC.logit_bound(qr, y[seen], scale, self.d), bf16, (r, h, t))
            at += n


def normal(rng, *shape):
    return HC.bf16_round(rng.standard_normal(shape))


# ---------------------------------------------------------------- rows of zeros
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("many", [False, True])
def test_zero_and_tiny_rows_beside_empty_and_masked_tiles(d, many):
    """Rows of Q that are zero or tiny, in requests without keys, with zero keys,
    and with a last tile that few of them see: the mean of the values that they
    see, and nothing where they see none."""
    rng = np.random.default_rng(d)
    Hkv, H, q = 2, 4, 30
    zero = np.zeros((140, Hkv, d), np.float32)
    kvs = [(zero[:0], zero[:0]), (zero, normal(rng, 140, Hkv, d)), HC.keys_values(rng, 131, Hkv, d),
           (zero[:20], normal(rng, 20, Hkv, d))]             # the last: more rows than keys
    b = Batch(rng, kvs, H, [q] * 4, many, d)
    Q = normal(rng, 4 * q, H, d)
    Q[::3] = 0
    Q[1::3] = HC.bf16_round(Q[1::3] * 2.0 ** -120)
    for causal in (False, True):
        for scale in (0.0, 1e-30):
            o, lse = b.attend(Q, causal, scale)
            assert b.c.status.item() == 0
            b.check(Q, o, lse, causal, scale or None)


@pytest.mark.parametrize("many", [False, True])
def test_zero_rows_and_lists_shorter_than_their_room(many):
    """The work of a list is counted by its room: the tiles behind its end have no
    page, and neither do those whose page numbers are out of range."""
    rng = np.random.default_rng(7)
    d, Hkv, H, q = 96, 1, 2, 40
    b = Batch(rng, [HC.keys_values(rng, 700, Hkv, d)] * 2, H, [q, q], many, d)
    Q = normal(rng, 2 * q, H, d)
    Q[::2] = 0
    lists = [[[3, 0, 10]], [[]]]
    o, lse = b.attend(Q, True, lists=lists, room=300)
    assert b.c.status.item() == 0
    b.check(Q, o, lse, True, lists=lists)
    b.c.block_table[1, 4:8] = -1                       # two whole tiles of the second request
    o, lse = b.attend(Q, False)
    assert b.c.status.item() == 5
    b.check(Q, o, lse, False, lists=[[list(range(11))], [[0, 1, 2, 3, 8, 9, 10]]])


# ---------------------------------------------------------------- probabilities far apart
def one_page_many_times(d, Hkv, pages, first, rest):
    """A cache of two pages, `first` and `rest` ((K, V) of 64 tokens each, for every
    head alike), and a request whose table holds the first and then `pages` times
    the other."""
    host = HC.HostPages(2, 1, d)
    for p, (K, V) in enumerate((first, rest)):
        for t in range(PAGE):
            host.put(p, t, 0, 0, K[t])
            host.put(p, t, 0, 1, V[t])
    data = torch.from_numpy(host.data.repeat(Hkv, 1)).cuda()
    c = dt.KV4Cache(2, Hkv, d, 1, pages + 1, 256, data=data)
    c.block_table.fill_(1)
    c.block_table[0, 0] = 0
    c.kv_len.fill_((pages + 1) * PAGE)
    return c, host


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q", [1, 64])
def test_a_long_tail_far_below_one_key_keeps_its_mass(d, q):
    """One key with a value of zero, and 300000 keys 2^-27 below it: the output is
    the tail's mass.  As many heads as blocks of threads, so that each has all keys
    of its own.  A probability is rounded by half a step of fp16's least numbers
    at most, 2^-25, of which the largest is 2^7 in the kernel of many rows and at
    least 2^5 (times the scale of V) in the other: 2^-30 of it."""
    rng = np.random.default_rng(d)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pages, Hkv = 4700, sms * (4 if q == 1 else 1)
    K, V = np.zeros((2, PAGE, d), np.float32), HC.bf16_round(1 + rng.random((2, PAGE, d)))
    K[:, :, 0] = HC.bf16_round(rng.uniform(-0.5, 0.5, (2, PAGE)))
    Q = np.zeros((q, d), np.float32)
    Q[:, 0] = HC.bf16_round(8 + rng.random(q))
    K[0, 0, 0] = HC.bf16_round([27 * np.log(2) / (8.5 * d ** -0.5)])[0]
    V[0, 0] = 0
    c, host = one_page_many_times(d, Hkv, pages, (K[0], V[0]), (K[1], V[1]))
    c.q_off.copy_(ints([0, q]))
    out, lse = torch.zeros((q, Hkv, d), device="cuda"), torch.zeros((q, Hkv), device="cuda")
    c.attend(HC.up(Q)[:, None].repeat(1, Hkv, 1), out, lse, max_q=q)
    torch.cuda.synchronize()
    assert c.status.item() == 0
    (k0, v0, y0, x0), (k1, v1, y1, x1) = host.get(0, 0), host.get(1, 0)
    qs = Q.astype(np.float64)
    s0, s1 = qs @ k0.T * d ** -0.5, qs @ k1.T * d ** -0.5
    m = s0.max(1, keepdims=True)
    p0, p1 = np.exp(s0 - m), np.exp(s1 - m) * pages
    l = (p0.sum(1) + p1.sum(1))[:, None]
    o = (p0 @ v0 + p1 @ v1) / l
    mass = (p0 @ np.abs(v0) + p1 @ np.abs(v1)) / l
    dS = max(HC.logit_bound(qs, y, d ** -0.5, d) for y in (y0, y1))
    step = 2.0 ** -30 * PAGE * (pages + 1) * max(x0.max(), x1.max())
    tol = step + (HC.EPS + 2 * dS + 2.0 ** -19) * mass
    assert (mass > 2 * step).all()
    e = (m + np.log(l))[:, 0]
    for h in range(0, Hkv, 7):
        err = np.abs(out[:, h].cpu().numpy() - o)
        assert (err <= tol).all(), (h, float((err / tol).max()))
        assert (np.abs(lse[:, h].cpu().numpy() - e) <= dS + 2.0 ** -19 * (1 + np.abs(e))).all()


@pytest.mark.parametrize("many", [False, True])
def test_logits_of_any_size(many):
    """Logits up to 2^30, where fp32 knows them to many units only: the largest key
    takes all, and nothing overflows."""
    rng = np.random.default_rng(3)
    d, H, q, n = 64, 1, 40, 500
    K, V = np.zeros((n, 1, d), np.float32), normal(rng, n, 1, d)
    K[:, 0, 0] = HC.bf16_round(np.exp2(rng.uniform(0, 29, n)) * rng.choice([-1, 1], n))
    K[:, 0, 1:] = K[:, :, :1].reshape(n, 1)             # rows of one value: held exactly
    b = Batch(rng, [(K, V)], H, [q], many, d)
    Q = np.zeros((q, H, d), np.float32)
    Q[..., 0] = 2.0
    o, lse = b.attend(Q, True, scale=1.0)
    assert np.isfinite(o).all() and np.isfinite(lse).all() and b.c.status.item() == 0
    for t in range(q):
        seen = n - (q - 1 - t)
        s = 2.0 * K[:seen, 0, 0].astype(np.float64)
        best = np.flatnonzero(s >= s.max() * (1 - 2.0 ** -20))
        if len(best) == 1 and np.partition(s, -2)[-2] < s.max() * 0.99:
            v = b.rows_of(0, 0)[1][best[0]]
            assert (np.abs(o[t, 0] - v) <= HC.EPS * (np.abs(v) + np.abs(v).max())).all()
            assert abs(lse[t, 0] - s.max()) <= 2.0 ** -19 * s.max()


# ---------------------------------------------------------------- values far apart
def outliers(rng, n, Hkv, d, key, unseen=True):
    """n tokens; before the last 20, two that every row sees and whose logits
    (with rows of Q that are `key` and noise) are hundreds below the others: values
    2^40 and 2^90 times the usual; with `unseen`, among the last, that only the later
    rows of a causal chunk see: the largest values there are, and 2^-40 of the usual."""
    K, V = HC.keys_values(rng, n, Hkv, d)
    K = HC.bf16_round(K * 0.25 + key)
    far = HC.bf16_round(-40.0 * key)
    for at, size in ((n // 3, 2.0 ** 40), (n - 40, 2.0 ** 90)):
        K[at] = far
        V[at] = HC.bf16_round(V[at] * size)
    if not unseen:
        return K, V
    V[n - 17] = HC.bf16_round(V[n - 17] * 2.0 ** -40)
    V[n - 10] = 3e38 * np.sign(V[n - 10])
    V[n - 4] = HC.bf16_round(V[n - 4] * 2.0 ** 30)
    return K, V


def check_outliers(b, Q, o, lse, wide):
    """As Batch.check, P s' rounded once; `wide`: P is rounded to fp16 (2^-11) and then
    with V to bf16 (2^-8 each), together at most (1 + 2^-11)(1 + 2^-8)^2 - 1 < 2^-8
    (2 + 2^-2) of P |v|."""
    scale, G, at = b.d ** -0.5, b.H // b.Hkv, 0
    for r, n in enumerate(b.q_lens):
        for h in range(b.Hkv):
            k, v, y, x, pos = b.rows_of(r, h)
            for t in range(n):
                seen = pos < b.kv[r] - (n - 1 - t)
                g = slice(h * G, (h + 1) * G)
                qr = Q[at + t, g].astype(np.float64)
                oo, e, P = OH.attend_rows(qr, k[seen], v[seen], scale)
                dS = HC.logit_bound(qr, y[seen], scale, b.d)
                HC.check(o[at + t, g], lse[at + t, g], oo, e, P, (np.abs(v) * (2 + 2.0 ** -2) if wide else x)[seen],
                         v[seen], dS, False, (r, h, t))
        at += n


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q", [1, 6, 30])
def test_outlying_and_unseen_values_few_rows(d, q):
    rng = np.random.default_rng(d + q)
    Hkv, H = 2, 2
    key = HC.bf16_round(4.0 * rng.choice([-1, 1], d))
    kvs = [outliers(rng, n, Hkv, d, key, q > 6) for n in (70, 200, 900)]
    b = Batch(rng, kvs, H, [q] * 3, False, d)
    Q = HC.bf16_round(key * 0.25 + normal(rng, 3 * q, H, d))
    o, lse = b.attend(Q, True)
    assert b.c.status.item() == 0
    check_outliers(b, Q, o, lse, False)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("many", [False, True])
def test_unseen_and_uneven_keys(d, many):
    """Keys from 2^-100 to 2^100 of the usual beside ordinary ones in every page, and
    keys of 1e38 that only the last rows of a causal chunk see.  Rows whose logits
    fp32 knows to a unit are within the bounds; nothing overflows in the others
    that see no more than 2^40."""
    rng = np.random.default_rng(d)
    Hkv, H, q = 1, 2, 30
    kvs = []
    for n in (150, 700):
        K, V = HC.keys_values(rng, n, Hkv, d)
        tiny = rng.choice(n - 40, 30, replace=False)
        K[tiny] = HC.bf16_round(K[tiny] * 2.0 ** rng.integers(-100, -3, 30)[:, None, None])
        K[n - 12] = HC.bf16_round(K[n - 12] * 2.0 ** 40)     # seen by 13 rows of 30
        K[n - 5] = 1e38 * np.sign(K[n - 5])
        kvs.append((K, V))
    b = Batch(rng, kvs, H, [q, q], many, d)
    Q = normal(rng, 2 * q, H, d)
    Q[3] = HC.bf16_round(Q[3] * 2.0 ** -60)
    o, lse = b.attend(Q, True)
    assert b.c.status.item() == 0
    at, exact = 0, 0
    for r in range(2):
        k, v, y, x, pos = b.rows_of(r, 0)
        for t in range(q):
            seen = pos < b.kv[r] - (q - 1 - t)
            qr = Q[at + t].astype(np.float64)
            dS = HC.logit_bound(qr, y[seen], d ** -0.5, d)
            if dS < 0.1:
                exact += 1
                oo, e, P = OH.attend_rows(qr, k[seen], v[seen], d ** -0.5)
                HC.check(o[at + t], lse[at + t], oo, e, P, x[seen], v[seen], dS, False, (r, t))
            elif np.abs(k[seen]).max() < 2.0 ** 50:
                assert np.isfinite(o[at + t]).all() and np.isfinite(lse[at + t]).all()
                assert (np.abs(o[at + t]) <= np.abs(v[seen]).max(0) * (1 + HC.EPS)).all()
        at += q
    assert exact >= 36


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q,kvs", [(30, (70, 200, 900)), (100, (130, 2000)), (300, (300, 1100))])
def test_outlying_and_unseen_values_many_rows(d, q, kvs):
    """What not all rows of a causal chunk see is of any size.  (Values that all rows
    see stay within 2^20 of one another here: below 2^-25 of the largest they are
    lost, as the header says.)"""
    rng = np.random.default_rng(d + q)
    Hkv, H = 1, 2
    key = HC.bf16_round(4.0 * rng.choice([-1, 1], d))
    made = []
    for n in kvs:
        K, V = outliers(rng, n, Hkv, d, key)
        for at in (n // 3, n - 40):
            V[at] = normal(rng, Hkv, d)
        if n > 3 * q // 2:
            V[n - q - 5] = HC.bf16_round(V[n - q - 5] * 2.0 ** 12)
        made.append((K, V))
    b = Batch(rng, made, H, [q] * len(kvs), True, d)
    Q = HC.bf16_round(key * 0.25 + normal(rng, q * len(kvs), H, d))
    o, lse = b.attend(Q, True)
    assert b.c.status.item() == 0
    check_outliers(b, Q, o, lse, True)
    # the blocks listed in any order: those that no row sees among the first
    lists = [[rng.permutation(-(-n // PAGE)).tolist()] for n in kvs]
    got = b.attend(Q, True, lists=lists, room=300)         # (work for the kernel of many rows)
    check_outliers(b, Q, *got, True)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("many", [False, True])
def test_the_largest_values_and_keys(d, many):
    """Rows of 3.3e38 of both signs: their 15 steps end within fp32, 8 steps from 0 would
    not.  One such value a row of Q takes all; a key of that size is seen only by
    rows of Q that are nothing to it."""
    rng = np.random.default_rng(d)
    H, q, n = 1, 40, 300
    K, V = normal(rng, n, 1, d) * 0.25, normal(rng, n, 1, d)
    K = HC.bf16_round(K)
    K[:, :, 0] = 0
    K[7] = 0
    K[7, :, 0] = 64.0                                      # takes all of the rows that have channel 0
    V[7] = HC.bf16_round(3.3e38 * np.sign(V[7]))
    K[200] = HC.bf16_round(3.3e38 * np.sign(K[200]))
    K[200, :, 0] = -3.3e38
    b = Batch(rng, [(K, V)], H, [q], many, d)
    v = b.rows_of(0, 0)[1][:n]
    assert np.isfinite(v).all()
    Q = np.zeros((q, H, d), np.float32)
    Q[..., 0] = 8.0
    o, lse = b.attend(Q, False)
    assert b.c.status.item() == 0
    k = b.rows_of(0, 0)[0][:n, 0]
    s = 8.0 * k * d ** -0.5
    assert np.argmax(s) == 7 and np.partition(s, -2)[-2] < s[7] - 30
    assert (np.abs(o[:, 0] - v[7]) <= 3 * HC.EPS * np.abs(v[7]).max()).all()
    assert (np.abs(lse - s[7]) <= 2.0 ** -19 * (1 + s[7])).all()


# ---------------------------------------------------------------- the quantiser
@pytest.mark.parametrize("d", [64, 96, 128])
def test_codes_beside_a_tiny_least_value_are_exact(d):
    """Quotients that are a least value of 2^-30 (2^-14 ... 2^-133) of the others away
    from a tie, on either side, and scales that reach the largest value by as little."""
    rng = np.random.default_rng(d)
    rows = []
    for tiny in (2.0 ** -13, 2.0 ** -14, 2.0 ** -15, 2.0 ** -17, 2.0 ** -30, 2.0 ** -60, 2.0 ** -100, 2.0 ** -133, 0.0):
        for sign in (1, -1):
            for size in (1.0, 2.0 ** 30, 2.0 ** -20, 2.0 ** 122):
                x, _ = tie_row(sign * tiny)
                row = np.resize(x, d) * size
                row[np.arange(d) % len(x) == 0] = sign * tiny
                row[d - 1] = x[-1] * size
                rows.append(row)
                rows.append(-row)
    rows.append(np.where(np.arange(d) % 2 == 0, 15 * 2.0 ** 123, -2.0 ** -120))
    rows += [HC.bf16_round(np.abs(rng.standard_normal(d)) * 2.0 ** rng.integers(-30, 1, d)) for _ in range(60)]
    x = np.stack(rows).astype(np.float32)
    assert (HC.bf16_round(x) == x).all()
    n = len(x)
    pages = -(-n // PAGE)
    want = HC.HostPages(pages, 1, d)
    for t in range(n):
        want.put(t // PAGE, t % PAGE, 0, 0, x[t])
        want.put(t // PAGE, t % PAGE, 0, 1, x[n - 1 - t])
    c = dt.KV4Cache(pages, 1, d, 1, pages, n)
    c.write(HC.up(x[:, None]), HC.up(x[::-1, None]), torch.arange(n, device="cuda"))
    torch.cuda.synchronize()
    got = c.data.cpu().numpy()
    bad = np.argwhere(got != want.data)
    for p, h, i in bad:                              # -0 and 0 are the same least value
        assert i >= PAGE * d and got[p, h, i] % 128 == want.data[p, h, i] % 128 == 0, (p, i)
    assert c.status.item() == 0


# ---------------------------------------------------------------- block summaries
@pytest.mark.parametrize("d", [64, 96, 128])
def test_summaries_of_blocks_whose_sums_pass_fp32(d):
    """Rows of 1e38: the sum of four passes fp32, the block's sum is finite in fp64,
    with its codes, scale and mean; a block with an infinity has none."""
    rng = np.random.default_rng(d)
    n, H = 5 * PAGE + 17, 2
    x = HC.bf16_round(rng.choice([-1e38, 1e38, 3e38], (1, H, n, d)) * rng.uniform(0.5, 1.0, (1, H, n, d)))
    x[0, :, :, 3] = HC.bf16_round(rng.standard_normal((H, n)))
    x[0, 1, 70, 5] = np.inf
    op = dt.BlockSparseAttention(1, H, n, n, d, 2)
    op.select(HC.up(x), HC.up(x))
    torch.cuda.synchronize()
    for h in range(H):
        for size, codes, scale in ((PAGE, op.k_codes, op.k_scale), (dt.QBLOCK, op.q_codes, op.q_scale)):
            for j in range(-(-n // size)):
                rows = x[0, h, j * size:(j + 1) * size].astype(np.float64)
                c, s, mean = OH.summary(rows)
                got = codes[0, h, j].cpu().numpy().astype(int)
                if not np.isfinite(rows).all():
                    assert (got == 0).all() and scale[0, h, j].item() == 0
                    continue
                # (channel 3, of another size, is 0 beside the rest whatever its rounding)
                assert (got == c).all() and scale[0, h, j].item() == s and s > 0, (h, size, j)
                if size == PAGE:
                    got = op.k_mean[0, h, j].cpu().numpy()
                    assert np.isfinite(got).all()
                    near = np.abs(got - mean) <= 2.0 ** -22 * np.abs(rows).mean(0)
                    assert near.all(), (h, j, np.flatnonzero(~near))


# ---------------------------------------------------------------- large sizes
def test_a_slot_map_of_two_to_the_31_places():
    """As many token places as the argument can say: every one is written, and no
    other word."""
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("less than 24 GB free")
    buf = torch.full((T + 2048,), 7, dtype=torch.int64, device="cuda")
    slots = buf[1024:1024 + T]
    table, free = ints([[5, 0, 0]]), ints([3, 1])
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 2, 1, 1)]
    dt.ditango_block_tables(1, 3, T, 8, ints([10]), ints([100]), free, 2, table, out[0], out[1], slots, out[2], out[3])
    torch.cuda.synchronize()
    assert out[0].item() == 110 and out[1].tolist() == [0, 100] and out[2].item() == 1 and out[3].item() == 0
    want = [5 * PAGE + p if p < PAGE else 3 * PAGE + p - PAGE for p in range(10, 110)]
    assert slots[:100].tolist() == want
    assert (buf[:1024] == 7).all() and (buf[1024 + T:] == 7).all()
    for a in range(100, T, 2 ** 28):
        assert (slots[a:min(T, a + 2 ** 28)] == -1).all()


# ---------------------------------------------------------------- states of block attention
@pytest.mark.parametrize("n1", [200, 333])
def test_a_state_over_selected_blocks_merges_with_the_partitions_states(n1):
    """Partition 1's queries over listed blocks of partition 0's keys, written into
    their slot of the state buffer (whose rows are more than the queries where
    n1 < n0), and the partition's own, fresh: the merge joins them."""
    rng = np.random.default_rng(n1)
    B, H, d, n0 = 2, 2, 128, 320
    pa = dt.PartitionedAttention(B, H, n0 + n1, d, [0, n0, n0 + n1])
    qkv = [normal(rng, B, H, n0 + n1, d) for _ in range(3)]
    Q, K, V = (HC.up(x) for x in qkv)
    pa.plan.copy_(torch.tensor([0, 0, 2, 1], dtype=torch.int8))      # (1, 0) reused, (1, 1) fresh
    pa.fresh_list[0] = 3
    pa.counts.copy_(ints([1, 1]))
    slot = dt.ditango_slot_table(pa.geom)[1]
    pa.partial(Q, K, V)
    pa.state_O[slot[0]] = 7.0
    pa.state_lse[slot[0]] = 7.0
    op = dt.BlockSparseAttention(B, H, n1, n0, d, 4)
    lists = [[[sorted(rng.choice(5, 3, replace=False).tolist()) for _ in range(op.n_q)] for _ in range(H)]
             for _ in range(B)]
    O = pa.state_O[slot[0]].view(B, H, pa.Lmax, d)[:, :, :n1]
    lse = pa.state_lse[slot[0]].view(B, H, pa.Lmax)[:, :, :n1]
    op.attend(Q[:, :, n0:], K[:, :, :n0], V[:, :, :n0], O, lse, ints(lists), torch.full_like(op.sel_count, 3))
    out = torch.empty((B, H, n0 + n1, d), device="cuda")
    out_lse = torch.empty((B, H, n0 + n1), device="cuda")
    pa.merge(out, out_lse)
    torch.cuda.synchronize()
    assert pa.status.item() == 0 and op.status.item() == 0
    assert (pa.state_lse[slot[0]][:, n1:] == 7).all() and (pa.state_O[slot[0]][:, n1:] == 7).all()
    for b in range(B):
        for h in range(H):
            for i in range(op.n_q):
                at = np.concatenate([np.arange(j * PAGE, (j + 1) * PAGE) for j in lists[b][h][i]]
                                    + [np.arange(n0, n0 + n1)])
                rows = np.arange(n0 + i * dt.QBLOCK, min(n0 + n1, n0 + (i + 1) * dt.QBLOCK))
                q, k, v = (x[b, h].astype(np.float64) for x in qkv)
                o, e, P = OH.attend_rows(q[rows], k[at], v[at], d ** -0.5)
                HC.check(out[b, h, rows].cpu().numpy().astype(np.float64),
                         out_lse[b, h, rows].cpu().numpy().astype(np.float64), o, e, P, v[at], v[at],
                         HC.logit_bound(q[rows], np.abs(k[at]), d ** -0.5, d), False, (b, h, i))


# ---------------------------------------------------------------- layers, and the free list
def test_layers_share_one_batch_and_the_free_list_goes_on_in_a_graph():
    """Two layers' pages over one object's tables, against objects of their own;
    decode steps as replays of one graph, the free list turned on the device."""
    rng = np.random.default_rng(12)
    R, Hkv, H, d, n_pages, width, steps = 3, 2, 4, 64, 24, 6, 70
    first = dt.KV4Cache(n_pages, Hkv, d, R, width, 64 * R, H=H)
    layers = [first, dt.KV4Cache(n_pages, Hkv, d, R, width, 64 * R, H=H, like=first)]
    own = [dt.KV4Cache(n_pages, Hkv, d, R, width, 64 * R, H=H) for _ in range(2)]
    assert layers[1].workspace is first.workspace and layers[1].kv_len is first.kv_len
    perm = rng.permutation(n_pages)
    free = ints(perm)
    turn = torch.arange(n_pages, device="cuda")
    ctx, new = torch.zeros(R, dtype=torch.int32, device="cuda"), ints([60, 1, 64])
    KV = [[HC.up(normal(rng, 125, Hkv, d)) for _ in range(2)] for _ in range(2)]

    def place(cs):
        cs[0].tables(ctx, new, free)
        if cs is own:
            cs[1].tables(ctx, new, free)

    def go_on(c):
        free.copy_(free[(turn + c.pages_used) % n_pages])
        ctx.copy_(c.kv_len)

    for cs in (layers, own):
        place(cs)
        for c, (K, V) in zip(cs, KV):
            c.write(K, V)
    assert layers[1].n_requests == R
    go_on(first)
    new.fill_(1)
    Q = HC.up(normal(rng, R, H, d))
    K1, V1 = HC.up(normal(rng, R, Hkv, d)), HC.up(normal(rng, R, Hkv, d))
    outs = [[torch.zeros((R, H, d), device="cuda") for _ in range(2)] for _ in range(2)]

    def step():
        for cs, out in zip((layers, own), outs):
            place(cs)
            for c, o in zip(cs, out):
                c.write(K1, V1)
                c.summarize(ctx)
                sel, count = c.select(Q, 2, band=0, sink=1)
                c.attend(Q, o, max_q=1, sel=sel, sel_count=count)
        go_on(first)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = np.array([60, 1, 64])
    used = 3
    for i in range(steps):
        K1.copy_(HC.up(normal(rng, R, Hkv, d)))
        graph.replay()
        used += int((lens % PAGE == 0).sum())
        lens += 1
        torch.cuda.synchronize()
        assert first.kv_len.tolist() == lens.tolist() and first.status.item() == 0
        assert free.tolist() == np.roll(perm, -used).tolist()
        for a, b in zip(*outs):
            assert torch.equal(a, b) and (a != 0).any()
    for a, b in zip(layers, own):
        assert torch.equal(a.block_table, b.block_table) and torch.equal(a.data, b.data)
        assert torch.equal(a.sum_codes, b.sum_codes)


# ---------------------------------------------------------------- bad lists
@pytest.mark.parametrize("many", [False, True])
def test_counts_of_a_list_out_of_range_are_clipped_and_recorded(many):
    rng = np.random.default_rng(5)
    d, H, q = 64, 2, 30
    b = Batch(rng, [HC.keys_values(rng, 300, 1, d)] * 2, H, [q, q], many, d)
    Q = normal(rng, 2 * q, H, d)
    room = 300 if many else 3                           # work for the kernel of many rows
    b.attend(Q, False, lists=[[[0, 1, 2]], [[3]]], room=room)
    assert b.c.status.item() == 0
    for counts, lists in (((9999, 1), [[[2, 0, 4]], [[3]]]), ((3, -2), [[[2, 0, 4]], [[]]])):
        b.c.status.zero_()
        R = len(b.table)
        if counts[0] > room:                            # as many as there are: the others have no tokens
            lists = [[[2, 0, 4] + list(range(5, room + 2))], lists[1]]
        sel = np.broadcast_to(np.arange(room), (R, 1, room)).copy()
        sel[0, 0, :] = [2, 0, 4] + list(range(5, room + 2))
        sel[1, 0, :3] = [3, 1, 0]
        sel, count = ints(sel), ints(np.array([[counts[0]], [counts[1]]] + [[room]] * (R - 2)))
        Qd = torch.zeros((b.rows, H, d), dtype=torch.bfloat16, device="cuda")
        Qd[:b.T] = HC.up(Q)
        out, lse = torch.zeros(Qd.shape, device="cuda"), torch.zeros(Qd.shape[:2], device="cuda")
        b.c.attend(Qd, out, lse, max_q=b.max_q, sel=sel, sel_count=count)
        torch.cuda.synchronize()
        assert b.c.status.item() == 5
        lists = [[[j for j in x if j * PAGE < 300] for x in of] for of in lists]
        b.check(Q, out[:b.T].cpu().numpy().astype(np.float64), lse[:b.T].cpu().numpy().astype(np.float64), False,
                lists=lists)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -30, 2.0 ** -60])
def test_a_list_that_hides_the_new_tokens_from_some_rows(d, size):
    """Old values `size` times the new ones; the listed page of new tokens is seen by
    the later rows only, and comes first or in between.  (P and V in bf16: as
    check_outliers says.)"""
    rng = np.random.default_rng(d)
    H, q, n = 2, 100, 700
    K, V = HC.keys_values(rng, n, 1, d)
    V[:500] = HC.bf16_round(V[:500] * size)
    b = Batch(rng, [(K, V)] * 2, H, [q] * 2, True, d)
    Q = normal(rng, 2 * q, H, d)
    lists = [[[10, 0, 1, 2]], [[3, 1, 10, 0]]]
    o, lse = b.attend(Q, True, lists=lists, room=300)      # work for the kernel of many rows
    assert b.c.status.item() == 0
    at = 0
    for r in range(2):
        k, v, y, x, pos = b.rows_of(r, 0, lists)
        for t in range(q):
            seen = pos < n - (q - 1 - t)
            qr = Q[at + t].astype(np.float64)
            oo, e, P = OH.attend_rows(qr, k[seen], v[seen], d ** -0.5)
            dS = HC.logit_bound(qr, y[seen], d ** -0.5, d)
            HC.check(o[at + t], lse[at + t], oo, e, P, (np.abs(v) * (2 + 2.0 ** -2))[seen], v[seen], dS,
                     False, (r, t))
        at += q


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("key,value", [(2.0 ** 4, 1.0), (2.0 ** 5.9, 1.0), (2.0 ** 6.5, 1.0), (1.0, 2.0 ** 9),
                                       (1.0, 2.0 ** 9.9), (1.0, 2.0 ** 10.5), (2.0 ** -5, 2.0 ** -9)])
def test_sizes_on_either_side_of_far_apart(d, key, value):
    """The last tokens' keys and values `key` and `value` times the others': around
    the sizes at which a causal call is done in the other way."""
    rng = np.random.default_rng(d)
    H, q, n = 2, 60, 400
    K, V = HC.keys_values(rng, n, 1, d)
    K, V = (np.clip(x, -3, 3) for x in (K, V))
    K[:, :, 0] = V[:, :, 0] = 3.0                         # every row's bound is 3 or a little more
    K[n - 20:] = HC.bf16_round(K[n - 20:] * key)
    V[n - 20:] = HC.bf16_round(V[n - 20:] * value)
    b = Batch(rng, [(HC.bf16_round(K), HC.bf16_round(V))], H, [q], True, d)
    Q = HC.bf16_round(normal(rng, q, H, d) / max(key, 1.0))
    o, lse = b.attend(Q, True)
    assert b.c.status.item() == 0
    check_outliers(b, Q, o, lse, True)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
@pytest.mark.parametrize("big,small", [(2.0 ** 85, 1.0), (2.0 ** 40, 2.0 ** -58), (2.0 ** 100, 2.0 ** -20), (2.0 ** 9, 1.0)])
def test_a_later_key_that_takes_all_has_a_small_value(d, G, big, small):
    """Values of `big` with ordinary logits in the first page and in a later one, where
    a key 150 above them has a value of `small`: the outputs are that value (in both
    orders of the pages).  Many requests alike, so that one warp takes both pages."""
    rng = np.random.default_rng(d + G)
    n, R = 9 * PAGE, 1500
    K, V = HC.bf16_round(0.1 * rng.standard_normal((n, 1, d))), normal(rng, n, 1, d)
    V[::7] = HC.bf16_round(V[::7] * big)
    V[5 * PAGE] = HC.bf16_round(normal(rng, 1, d) * small)
    K[5 * PAGE] = 0
    K[5 * PAGE, 0, 0] = 16.0
    K[:, 0, 1] = 0
    b = Batch(rng, [(K, V)], G, [1], False, d)
    table = b.c.block_table.repeat(R, 1)
    table[R // 2:] = table[R // 2:].flip(1)
    c = dt.KV4Cache(b.c.n_pages, 1, d, R, 9, R, H=G, data=b.c.data, block_table=table)
    c.kv_len.fill_(n)
    c.q_off.copy_(torch.arange(R + 1, dtype=torch.int32))
    Q = np.zeros((1, G, d), np.float32)
    Q[..., 0] = HC.bf16_round(150 / 16.0 * d ** 0.5)
    Q[..., 1:] = HC.bf16_round(0.1 * rng.standard_normal((1, G, d - 1)))
    out, lse = torch.zeros((R, G, d), device="cuda"), torch.zeros((R, G), device="cuda")
    c.attend(HC.up(Q).repeat(R, 1, 1), out, lse, max_q=1)
    torch.cuda.synchronize()
    k, v, y, x, pos = b.rows_of(0, 0)
    o, e, P = OH.attend_rows(Q[0].astype(np.float64), k, v, d ** -0.5)
    dS = HC.logit_bound(Q[0].astype(np.float64), y, d ** -0.5, d)
    got, got_l = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all() and c.status.item() == 0
    for r in range(0, R, 37):
        HC.check(got[r], got_l[r], o, e, P, x, v, dS, False, r)
