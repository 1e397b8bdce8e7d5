"""The 4-bit history where its arithmetic meets its limits: rows of zeros, masked
places and empty tiles, values far from one another, and large sizes; against the
fp64 oracle."""
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
BALLAST = 600        # queries of the request that makes a batch's work large, over 20000 tokens


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
