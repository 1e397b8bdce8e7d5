"""What is measured of the operators around a 4-bit key/value history and of
attention over selected key blocks.

A case names one operator and its sizes; `run` makes one pass through it,
either in plain torch (`own` false) or by the package's calls (`own` true).

kinds
  tables   block table, slot map and offsets of a batch, from request lengths
  store    new keys and values written into 4-bit pages, and read back as bf16
  history  attention of new query tokens over the 4-bit pages of their request
  sparse   the same for single tokens over the pages that a cheap score selects
  select   block means of Q and K, and the key blocks each query block selects
  blocks   attention of 128-query blocks over their selected 64-key blocks
"""
import torch

own = False

PAGE = 64      # tokens of a page, and keys of a key block
QBLOCK = 128   # queries of a query block
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's tables: one new token for each of 64 running requests
        dict(name="tables_step", kind="tables", R=64, ctx_lo=1, ctx_hi=16000, new_lo=1, new_hi=1),
        # admission of many ragged prompts, some requests idle, some on top of a context
        dict(name="tables_prompts", kind="tables", R=512, ctx_lo=0, ctx_hi=1200, new_lo=0, new_hi=400),
        # one token each of 64 requests (40 heads of 128, as the 32-partition workloads)
        dict(name="store_step", kind="store", T=64, Hkv=40, d=128),
        # the whole 29-frame latent: 8 x 3600 tokens, 24 heads of 96
        dict(name="store_latent", kind="store", T=28800, Hkv=24, d=96),
        # one query token over the history of the 24-frame video, no shared heads
        dict(name="history_one_token", kind="history", R=1, H=24, Hkv=24, d=96, q_lo=1, q_hi=1,
             kv_lo=86400, kv_hi=86400, causal=False),
        # a decode batch of ragged histories, 5 query heads to a key head
        dict(name="history_ragged_step", kind="history", R=48, H=40, Hkv=8, d=128, q_lo=1, q_hi=1,
             kv_lo=1, kv_hi=16000, causal=True),
        # a latent frame of 45 x 80 tokens over the 7 frames before it
        dict(name="history_frame", kind="history", R=1, H=24, Hkv=24, d=96, q_lo=3600, q_hi=3600,
             kv_lo=25200, kv_hi=25200, causal=False),
        # single tokens of 16 requests over 48 selected pages of their long histories
        dict(name="sparse_step", kind="sparse", R=16, H=40, Hkv=8, d=128, kv_lo=30000, kv_hi=76800,
             k=48, band=1, sink=1),
        # the lists of the 29-frame latent: 225 x 450 blocks for each of 24 heads
        dict(name="select_latent", kind="select", B=1, H=24, Hkv=24, Nq=28800, Nk=28800, d=96, k=75,
             band=4, sink=2),
        # the lists of the 76800-token video: 600 x 1200 blocks for each of 40 heads
        dict(name="select_long", kind="select", B=1, H=40, Hkv=40, Nq=76800, Nk=76800, d=128, k=150,
             band=4, sink=2),
        # a short ragged cross attention with shared key heads, two batch entries
        dict(name="blocks_short", kind="blocks", B=2, H=8, Hkv=4, Nq=1000, Nk=1333, d=64, k=7,
             empty=True, padded=True),
        # the 76800-token video at an eighth of its key blocks
        dict(name="blocks_long", kind="blocks", B=1, H=40, Hkv=40, Nq=76800, Nk=76800, d=128, k=150,
             empty=False, padded=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["tables", "store", "history", "history", "sparse", "select", "blocks", "blocks"])
    d = rng.choice([64, 96, 128])
    if kind == "tables":
        ctx = _log(rng, 1, 4000)
        return dict(kind=kind, R=_log(rng, 1, 512), ctx_lo=rng.randrange(0, ctx), ctx_hi=ctx,
                    new_lo=rng.randrange(0, 2), new_hi=_log(rng, 1, 400))
    if kind == "store":
        return dict(kind=kind, T=_log(rng, 1, 28800), Hkv=rng.choice([1, 2, 3, 8, 24]), d=d)
    if kind == "history":
        Hkv = rng.choice([1, 2, 8])
        if rng.random() < 0.5:        # decode batches
            hi = _log(rng, 1, 16000)
            q = _log(rng, 1, 5)
            return dict(kind=kind, R=_log(rng, 1, 48), H=Hkv * rng.choice([1, 3, 5, 8]), Hkv=Hkv, d=d,
                        q_lo=1, q_hi=q, kv_lo=rng.randrange(0, hi), kv_hi=hi,
                        causal=rng.random() < 0.5)
        hi = _log(rng, 100, 12000)    # chunks
        q = _log(rng, 6, 2000)
        return dict(kind=kind, R=rng.choice([1, 2, 3]), H=Hkv * rng.choice([1, 2, 5]), Hkv=Hkv, d=d,
                    q_lo=max(1, q // 2), q_hi=q, kv_lo=max(1, hi // 3), kv_hi=hi,
                    causal=rng.random() < 0.5)
    if kind == "sparse":
        hi = _log(rng, 64, 76800)
        Hkv = rng.choice([1, 4, 8])
        return dict(kind=kind, R=_log(rng, 1, 16), H=Hkv * rng.choice([1, 3, 5]), Hkv=Hkv, d=d,
                    kv_lo=max(1, hi // 4), kv_hi=hi, k=_log(rng, 1, 48), band=rng.choice([0, 1, 3]),
                    sink=rng.choice([0, 1, 2]))
    Hkv = rng.choice([1, 3, 8])
    H = Hkv * rng.choice([1, 1, 2])
    B = rng.choice([1, 2])
    Nq, Nk = _log(rng, 1, 20000), _log(rng, 1, 20000)
    if kind == "select":
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, k=_log(rng, 1, 150),
                    band=rng.choice([-1, 0, 2, 4]), sink=rng.choice([0, 1, 2]))
    return dict(kind=kind, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, k=_log(rng, 1, 80),
                empty=rng.random() < 0.5, padded=rng.random() < 0.5)


def _spread(n, lo, hi):
    """n lengths between lo and hi, the same for every seed: ragged, the first one hi."""
    return [hi - int((r * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for r in range(n)]


def _lens(case):
    """(history or context lengths, query or new-token lengths) of the requests."""
    R = case["R"]
    if case["kind"] == "tables":
        return (_spread(R, case["ctx_lo"], case["ctx_hi"])[::-1],
                _spread(R, case["new_lo"], case["new_hi"]))
    kv = _spread(R, case["kv_lo"], case["kv_hi"])
    if case["kind"] == "sparse":
        return kv, [1] * R
    return kv, _spread(R, case["q_lo"], case["q_hi"])[::-1]


def _blocks(n):
    return -(-n // PAGE)


def work(case):
    kind = case["kind"]
    if kind == "tables":
        ctx, new = _lens(case)
        pages = sum(_blocks(c + n) for c, n in zip(ctx, new))
        return dict(bytes=12 * len(ctx) + 8 * pages + 8 * sum(new), flops=sum(new))
    if kind == "store":
        n = case["T"] * case["Hkv"]
        d = case["d"]
        # K and V in, codes and their scales out, and back: codes in, K and V out
        return dict(bytes=n * (2 * 4 * d + 2 * (d + 8)) + 8 * case["T"], flops=8 * n * d)
    if kind in ("history", "sparse"):
        kv, q = _lens(case)
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        if kind == "sparse":
            need = [min(n, max(case["k"], 1) * PAGE) for n in kv]
            extra = sum(_blocks(n) for n in kv) * Hkv * (d + 4)
        else:
            need, extra = kv, 0
        pairs = sum(a * b - (b * (b - 1) // 2 if case.get("causal") and a >= b else 0)
                    for a, b in zip(need, q))
        return dict(bytes=sum(need) * Hkv * (d + 8) + sum(q) * H * (4 * d + 4) + extra,
                    flops=4 * d * H * pairs + 2 * (extra // (d + 4)) * d * (H // Hkv))
    B, H, Hkv, Nq, Nk, d = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    nq, nk = -(-Nq // QBLOCK), _blocks(Nk)
    if kind == "select":
        k = min(nk, case["k"])
        return dict(bytes=2 * B * d * (H * Nq + Hkv * Nk) + 4 * B * Hkv * (nk * d + nq * k),
                    flops=B * d * (H * Nq + Hkv * Nk) + 2 * B * H * nq * nk * d)
    k = min(nk, case["k"])
    return dict(bytes=2 * B * d * (2 * H * Nq + 2 * Hkv * Nk) + 4 * B * H * Nq + 4 * B * Hkv * nq * k,
                flops=4 * d * B * H * Nq * min(Nk, k * PAGE))


# ---------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _keys_values(gen, T, Hkv, d):
    """Keys with channels that sit off zero, as projected keys do; values around zero."""
    K = (_randn(gen, T, Hkv, d) + 1.5 * _randn(gen, 1, Hkv, d)).bfloat16()
    V = _randn(gen, T, Hkv, d).bfloat16()
    return K, V


def _pack(x):
    """4-bit codes and (scale, least value) of each row of bf16 x, for the input pages."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) / 15 * (1 + 2.0 ** -8)).bfloat16()
    c = torch.round((f - lo) / s.float().clamp_min(1e-30)).clamp_(0, 15).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([s, lo.bfloat16()], -1).contiguous()


def _history_pages(gen, n_pages, Hkv, d):
    """Pages [n_pages, Hkv, 64 * (d + 8)] of keys and values as a model leaves them."""
    data = torch.empty((n_pages, Hkv, PAGE * (d + 8)), dtype=torch.uint8, device=DEV)
    off = 1.5 * _randn(gen, 1, Hkv, 1, d)
    step = max(1, (1 << 26) // (Hkv * PAGE * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        kc, km = _pack((_randn(gen, n, Hkv, PAGE, d) + off).bfloat16())
        vc, vm = _pack(_randn(gen, n, Hkv, PAGE, d).bfloat16())
        data[p:p + n] = torch.cat([x.reshape(n, Hkv, -1).view(torch.uint8) for x in (kc, vc, km, vm)], -1)
    return data


def _table(gen, counts, n_pages):
    """A block table whose rows hold counts[r] distinct pages in random order, and the other pages."""
    R, width = len(counts), max(max(counts), 1)
    perm = torch.randperm(n_pages, generator=gen, device=DEV).int()
    have = torch.tensor(counts, device=DEV)
    mask = torch.arange(width, device=DEV)[None] < have[:, None]
    table = torch.zeros((R, width), dtype=torch.int32, device=DEV)
    used = int(sum(counts))
    table[mask] = perm[:used]
    return table, perm[used:].contiguous()


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind = case["kind"]
    st = dict(case=case)
    if kind == "tables":
        ctx, new = _lens(case)
        n_pages = sum(_blocks(c + n) for c, n in zip(ctx, new)) + 7
        width = max(_blocks(c + n) for c, n in zip(ctx, new)) + 1
        old, st["free"] = _table(gen, [_blocks(c) for c in ctx], n_pages)
        st["table"] = torch.zeros((case["R"], width), dtype=torch.int32, device=DEV)
        st["table"][:, :min(width, old.shape[1])] = old[:, :width]
        st["ctx"], st["new"] = _ints(ctx), _ints(new)
        st["T"], st["n_pages"] = sum(new), n_pages
        if own:
            import sparse_state_reuse_b200 as dt
            st["cache"] = dt.KV4Cache(n_pages, 1, 64, case["R"], width, max(st["T"], 1),
                                      block_table=st["table"])
        return st
    if kind == "store":
        T, Hkv, d = case["T"], case["Hkv"], case["d"]
        st["K"], st["V"] = _keys_values(gen, T, Hkv, d)
        n_pages = _blocks(T) + 3
        # the tokens take consecutive places of pages that lie anywhere
        pages = torch.randperm(n_pages, generator=gen, device=DEV)
        t = torch.arange(T, device=DEV) + int(seed) % PAGE
        st["slots"] = pages[t // PAGE] * PAGE + t % PAGE
        st["n_pages"] = n_pages
        st["data"] = torch.zeros((n_pages, Hkv, PAGE * (d + 8)), dtype=torch.uint8, device=DEV)
        st["Kr"], st["Vr"] = torch.empty_like(st["K"]), torch.empty_like(st["V"])
        if own:
            import sparse_state_reuse_b200 as dt
            st["cache"] = dt.KV4Cache(n_pages, Hkv, d, 1, 1, T, data=st["data"])
        return st
    if kind in ("history", "sparse"):
        kv, q = _lens(case)
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        counts = [_blocks(n) for n in kv]
        n_pages = sum(counts) + 3
        st["data"] = _history_pages(gen, n_pages, Hkv, d)
        st["table"], _ = _table(gen, counts, n_pages)
        st["kv"], st["q_lens"] = _ints(kv), _ints(q)
        st["q_off"] = _ints([sum(q[:r]) for r in range(len(q) + 1)])
        st["max_q"], st["T"] = max(q), sum(q)
        st["Q"] = (1.5 * _randn(gen, st["T"], H, d)).bfloat16()
        st["out"] = torch.empty_like(st["Q"])
        st["lse"] = torch.empty((st["T"], H), dtype=torch.float32, device=DEV)
        if kind == "sparse":
            # the page summaries are kept beside the pages, as they were written
            lens = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
            pos = torch.arange(st["table"].shape[1], device=DEV)[None] * PAGE
            fill = (st["kv"][:, None] - pos).clamp(0, PAGE)
            lens[st["table"][fill > 0].long()] = fill[fill > 0].long()
            st["sum_codes"], st["sum_scale"] = _page_summaries(st["data"], lens, d)
        if own:
            import sparse_state_reuse_b200 as dt
            c = dt.KV4Cache(n_pages, Hkv, d, case["R"], st["table"].shape[1], st["T"], H=H,
                            data=st["data"], block_table=st["table"])
            c.kv_len.copy_(st["kv"])
            c.q_off.copy_(st["q_off"])
            if kind == "sparse":
                c.sum_codes.copy_(st["sum_codes"])
                c.sum_scale.copy_(st["sum_scale"])
            st["cache"] = c
        return st
    B, H, Hkv, Nq, Nk, d = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    nq, nk = -(-Nq // QBLOCK), _blocks(Nk)
    # neighbouring tokens look alike: a component shared by 64 of them
    near = _randn(gen, B, Hkv, nk, d)
    pick = torch.arange(max(Nq, Nk), device=DEV) // PAGE % nk
    st["Q"] = (_randn(gen, B, H, Nq, d)
               + 0.5 * near.repeat_interleave(H // Hkv, 1)[:, :, pick[:Nq]]).bfloat16()
    st["K"] = (_randn(gen, B, Hkv, Nk, d) + 0.5 * near[:, :, pick[:Nk]]).bfloat16()
    if kind == "select":
        if own:
            import sparse_state_reuse_b200 as dt
            st["op"] = dt.BlockSparseAttention(B, H, Nq, Nk, d, case["k"], case["band"], case["sink"],
                                               Hkv=Hkv)
        return st
    st["V"] = _randn(gen, B, Hkv, Nk, d).bfloat16()
    k = min(nk, case["k"])
    pick = torch.rand((B, Hkv, nq, nk), generator=gen, device=DEV).topk(k, -1).indices.sort(-1).values
    count = torch.full((B, Hkv, nq), k, dtype=torch.int32, device=DEV)
    if case["empty"]:   # query blocks that attend nothing, and shorter lists
        count = torch.where(torch.rand((B, Hkv, nq), generator=gen, device=DEV) < 0.2,
                            torch.randint(0, k + 1, (B, Hkv, nq), generator=gen, device=DEV).int(), count)
    st["sel"] = torch.where(torch.arange(k, device=DEV) < count[..., None], pick, -1).int()
    st["count"] = count
    st["k_len"] = _ints([max(0, Nk - (b + 1) * (Nk // 3)) for b in range(B)]) if case["padded"] else None
    st["out"] = torch.empty_like(st["Q"])
    st["lse"] = torch.empty((B, H, Nq), dtype=torch.float32, device=DEV)
    if own:
        import sparse_state_reuse_b200 as dt
        st["op"] = dt.BlockSparseAttention(B, H, Nq, Nk, d, case["k"], -1, 0, Hkv=Hkv)
    return st


# ---------------------------------------------------------------- plain forms
def _unpack(pages, d):
    """K and V in fp32, [..., 64, d], of pages [..., 64 * (d + 8)]."""
    lead = pages.shape[:-1]
    n = PAGE * d // 2
    meta = pages[..., 2 * n:].contiguous().view(torch.bfloat16).float().view(*lead, 2, PAGE, 2)
    codes = pages[..., :2 * n].view(*lead, 2, PAGE, d // 2)
    x = torch.stack([codes & 15, codes >> 4], -1).view(*lead, 2, PAGE, d).float()
    x = x * meta[..., :1] + meta[..., 1:]
    return x[..., 0, :, :], x[..., 1, :, :]


def _quantize(x):
    """Codes 0..15, bf16 scale and bf16 least value of every row of x: the
    scale is the least bf16 value that reaches the row's largest value in 15 steps."""
    f = x.double()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    want = (hi - lo) / 15
    bits = want.float().view(torch.int32) & -65536
    s = bits.view(torch.float32).double()
    s = torch.where(s < want, (bits + 65536).view(torch.float32).double(), s)
    c = torch.where(s > 0, torch.round((f - lo) / torch.where(s > 0, s, 1.0)), 0.0)
    return c.to(torch.uint8), s.bfloat16(), lo.bfloat16()


def _summary(x, count):
    """8-bit codes, scale and mean of sums x in fp64 over the last dimension."""
    top = x.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, torch.round(x * 127 / torch.where(top > 0, top, 1.0)), 0.0)
    scale = (top[..., 0] / (127.0 * count)).float()
    return codes.to(torch.int8), scale, (x / count[..., None]).float()


def _page_summaries(data, lens, d):
    K, _ = _unpack(data, d)
    inside = torch.arange(PAGE, device=DEV)[None, :] < lens[:, None]
    sums = (K.double() * inside[:, None, :, None]).sum(2)
    codes, scale, _ = _summary(sums, lens.clamp_min(1)[:, None].double())
    return codes, scale


def _block_means(x, block):
    B, H, N, d = x.shape
    n = -(-N // block)
    pad = torch.zeros((B, H, n * block, d), dtype=torch.float64, device=DEV)
    pad[:, :, :N] = x
    count = (N - torch.arange(n, device=DEV) * block).clamp(max=block).double()
    return _summary(pad.view(B, H, n, block, d).sum(3), count)


def _choose(score, forced, eligible, k):
    """Ascending indices of the forced and then best eligible entries, ties to the lower index."""
    score = torch.where(eligible, score, float("-inf"))
    score = torch.where(forced & eligible, float("inf"), score)
    count = torch.minimum(eligible.sum(-1), torch.clamp((forced & eligible).sum(-1), min=k)).int()
    width = max(1, int(count.max()))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :width]
    live = torch.arange(width, device=DEV) < count[..., None]
    n = score.shape[-1]
    best = torch.where(live, best, n).sort(-1).values
    return torch.where(live, best, -1).int(), count


def _scores(qc, qs, kc, ks):
    """scale_k * sum over the group's heads of scale_q * (q . k), sums in head order."""
    dot = qc.float() @ kc.float().transpose(-1, -2)     # [..., G, n_q, n_k]; whole numbers
    part = qs[..., None] * dot
    total = part[..., 0, :, :]
    for g in range(1, part.shape[-3]):
        total = total + part[..., g, :, :]
    return total * ks


def _softmax_attend(S, V):
    m = S.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    P = torch.exp(S - m)
    del S
    total = P.sum(-1, keepdim=True)
    O = (P @ V) / torch.where(total > 0, total, 1.0)
    return O, (torch.log(total) + m)[..., 0]


def _plain_tables(st):
    table, free, ctx, new, T = (st[n] for n in ("table", "free", "ctx", "new", "T"))
    kv = ctx + new
    q_off = torch.zeros(len(ctx) + 1, dtype=torch.int32, device=DEV)
    q_off[1:] = new.cumsum(0)
    have, need = (ctx + PAGE - 1) // PAGE, (kv + PAGE - 1) // PAGE
    start = (need - have).cumsum(0) - (need - have)
    col = torch.arange(table.shape[1], device=DEV)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    take = (start[:, None] + col - have[:, None]).clamp(0, len(free) - 1)
    table.copy_(torch.where(fresh, free[take], table))
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(q_off[1:], t.int(), right=True)
    pos = ctx[req] + t - q_off[req]
    slots = table[req, pos // PAGE].long() * PAGE + pos % PAGE
    return table, kv, q_off, slots, (need - have).sum(0, keepdim=True).int()


def _plain_store(st):
    case, data, slots = st["case"], st["data"], st["slots"]
    T, Hkv, d = case["T"], case["Hkv"], case["d"]
    page, at = slots // PAGE, slots % PAGE
    for which, x in enumerate((st["K"], st["V"])):
        c, s, lo = _quantize(x)
        codes = data[..., which * PAGE * d // 2:(which + 1) * PAGE * d // 2].view(-1, Hkv, PAGE, d // 2)
        codes[page, :, at] = c[..., 0::2] | (c[..., 1::2] << 4)
        at0 = PAGE * d + which * PAGE * 4
        meta = data[..., at0:at0 + PAGE * 4].view(-1, Hkv, PAGE, 4)
        meta[page, :, at] = torch.cat([s, lo], -1).view(torch.uint8)
    K, V = _unpack(data, d)
    st["Kr"].copy_(K[page, :, at])
    st["Vr"].copy_(V[page, :, at])
    return st["Kr"], st["Vr"]


def _plain_history(st, sel, count):
    """Attention of each request's new tokens over its (selected) pages."""
    case = st["case"]
    H, Hkv, d, R = case["H"], case["Hkv"], case["d"], case["R"]
    n = st["max_q"]
    q_at = st["q_off"][:-1, None] + torch.arange(n, device=DEV)
    live = torch.arange(n, device=DEV)[None] < st["q_lens"][:, None]
    Q = st["Q"][q_at.clamp(max=st["T"] - 1)].float()                  # [R, n, H, d]
    Q = Q.view(R, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, d)
    pages = torch.gather(st["table"], 1, sel.clamp_min(0).flatten(1).long()).view(sel.shape).long()
    K, V = _unpack(st["data"][pages, torch.arange(Hkv, device=DEV)[None, :, None]], d)
    pos = (sel[..., None] * PAGE + torch.arange(PAGE, device=DEV)).flatten(2)     # [R, Hkv, keys]
    seen = st["kv"][:, None]
    if case.get("causal"):
        seen = seen - (st["q_lens"][:, None] - 1 - torch.arange(n, device=DEV))
    seen = seen.expand(R, n)[:, None, None, :].expand(R, 1, H // Hkv, n).reshape(R, 1, -1, 1)
    ok = (pos[:, :, None] < seen) & (torch.arange(sel.shape[-1], device=DEV)
                                     < count[..., None]).repeat_interleave(PAGE, -1)[:, :, None]
    K, V = K.flatten(2, 3), V.flatten(2, 3)
    inside = ok.any(2)[..., None]
    K, V = torch.where(inside, K, 0.0), torch.where(inside, V, 0.0)
    S = (Q @ K.transpose(-1, -2)) * d ** -0.5
    O, lse = _softmax_attend(S.masked_fill_(~ok, float("-inf")), V)
    O = O.view(R, Hkv, H // Hkv, n, d).permute(0, 3, 1, 2, 4).reshape(R, n, H, d)
    lse = lse.view(R, Hkv, H // Hkv, n).permute(0, 3, 1, 2).reshape(R, n, H)
    st["out"].copy_(O[live])
    st["lse"].copy_(lse[live])
    return st["out"], st["lse"]


def _plain_sparse(st):
    case = st["case"]
    R, H, Hkv, d = case["R"], case["H"], case["Hkv"], case["d"]
    qc, qs, _ = _summary(st["Q"].double(), torch.ones((1, 1), dtype=torch.float64, device=DEV))
    pages = st["table"].long()
    kc = st["sum_codes"][pages].permute(0, 2, 1, 3)               # [R, Hkv, blocks, d]
    ks = st["sum_scale"][pages].permute(0, 2, 1)
    score = _scores(qc.view(R, Hkv, H // Hkv, 1, d), qs.view(R, Hkv, H // Hkv, 1), kc[:, :, None],
                    ks[:, :, None])[:, :, 0]
    n = (st["kv"][:, None, None] + PAGE - 1) // PAGE
    j = torch.arange(pages.shape[1], device=DEV)
    eligible = (j < n).expand_as(score)
    forced = (j < case["sink"]) | (j >= n - 1 - case["band"])
    sel, count = _choose(score, forced.expand_as(score), eligible, case["k"])
    out, lse = _plain_history(st, sel, count)
    return _padded(sel, _room(case)), count, out, lse


def _room(case):
    """Entries of a list: what the budget, the first blocks and the band can ask for."""
    own_blocks = 1 if case["kind"] == "sparse" else QBLOCK // PAGE
    near = own_blocks + 2 * case["band"] if case["band"] >= 0 else 0
    return max(1, case["k"], case["sink"] + near)


def _padded(sel, width):
    out = torch.full((*sel.shape[:-1], width), -1, dtype=torch.int32, device=DEV)
    out[..., :sel.shape[-1]] = sel
    return out


def _plain_select(st):
    case = st["case"]
    B, H, Hkv, Nk = case["B"], case["H"], case["Hkv"], case["Nk"]
    qc, qs, _ = _block_means(st["Q"], QBLOCK)
    kc, ks, mean = _block_means(st["K"], PAGE)
    nq, nk = qs.shape[-1], ks.shape[-1]
    score = _scores(qc.view(B, Hkv, H // Hkv, nq, -1), qs.view(B, Hkv, H // Hkv, nq), kc[:, :, None],
                    ks[:, :, None])
    j, i = torch.arange(nk, device=DEV), torch.arange(nq, device=DEV)[:, None]
    forced = j.expand(nq, nk) < case["sink"]
    if case["band"] >= 0:
        per = QBLOCK // PAGE
        forced = forced | ((j >= i * per - case["band"]) & (j < (i + 1) * per + case["band"]))
    sel, count = _choose(score, forced.expand_as(score), torch.ones_like(score, dtype=torch.bool),
                         case["k"])
    return mean, _padded(sel, _room(case)), count


def _plain_blocks(st):
    """Head by head, since the gathered keys of all heads would not fit."""
    case, sel, count = st["case"], st["sel"], st["count"]
    B, H, Hkv, Nq, Nk, d = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    nq, nk = sel.shape[2], _blocks(Nk)
    at = torch.arange(PAGE, device=DEV)
    step = max(1, (1 << 30) // (sel.shape[-1] * PAGE * d))
    for b in range(B):
        n_keys = Nk if st["k_len"] is None else st["k_len"][b]
        for h in range(H):
            g = h // (H // Hkv)
            K = torch.zeros((nk * PAGE, d), device=DEV)
            V = torch.zeros((nk * PAGE, d), device=DEV)
            K[:Nk], V[:Nk] = st["K"][b, g], st["V"][b, g]
            Q = torch.zeros((nq * QBLOCK, d), device=DEV)
            Q[:Nq] = st["Q"][b, h]
            K, V, Q = K.view(nk, PAGE, d), V.view(nk, PAGE, d), Q.view(nq, QBLOCK, d)
            for i in range(0, nq, step):
                s = sel[b, g, i:i + step]
                rows = slice(i * QBLOCK, min(Nq, (i + step) * QBLOCK))
                pos = (s[..., None] * PAGE + at).flatten(1)
                ok = ((s >= 0)[..., None] & (s[..., None] * PAGE + at < n_keys)).flatten(1)
                Kg, Vg = K[s.clamp_min(0)].flatten(1, 2), V[s.clamp_min(0)].flatten(1, 2)
                S = (Q[i:i + step] @ Kg.transpose(-1, -2)) * d ** -0.5
                O, lse = _softmax_attend(S.masked_fill_(~ok[:, None], float("-inf")), Vg)
                st["out"][b, h, rows] = O.flatten(0, 1)[:rows.stop - i * QBLOCK].bfloat16()
                st["lse"][b, h, rows] = lse.flatten()[:rows.stop - i * QBLOCK]
    return st["out"], st["lse"]


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        if kind == "tables":
            c = st["cache"]
            c.tables(st["ctx"], st["new"], st["free"])
            return c.block_table, c.kv_len, c.q_off, c.slot_map[:st["T"]], c.pages_used
        if kind == "store":
            st["cache"].write(st["K"], st["V"], st["slots"])
            st["cache"].read(st["slots"], st["Kr"], st["Vr"])
            return st["Kr"], st["Vr"]
        if kind == "history":
            st["cache"].attend(st["Q"], st["out"], st["lse"], max_q=st["max_q"], causal=case["causal"])
            return st["out"], st["lse"]
        if kind == "sparse":
            c = st["cache"]
            sel, count = c.select(st["Q"], case["k"], case["band"], case["sink"])
            c.attend(st["Q"], st["out"], st["lse"], max_q=1, sel=sel, sel_count=count)
            return sel, count, st["out"], st["lse"]
        if kind == "select":
            op = st["op"]
            sel, count = op.select(st["Q"], st["K"])
            return op.k_mean, sel, count
        st["op"].attend(st["Q"], st["K"], st["V"], st["out"], st["lse"], sel=st["sel"],
                        sel_count=st["count"], k_len=st["k_len"])
        return st["out"], st["lse"]
    if kind == "tables":
        return _plain_tables(st)
    if kind == "store":
        return _plain_store(st)
    if kind == "history":
        case = st["case"]
        n = (st["kv"][:, None, None] + PAGE - 1) // PAGE
        j = torch.arange(st["table"].shape[1], device=DEV, dtype=torch.int32)
        return _plain_history(st, j.expand(case["R"], case["Hkv"], -1),
                              n[..., 0].expand(-1, case["Hkv"]))
    if kind == "sparse":
        return _plain_sparse(st)
    if kind == "select":
        return _plain_select(st)
    return _plain_blocks(st)


# ---------------------------------------------------------------- in 64 bits
def _exact_rows(q, k, v):
    """O and log-sum-exp of rows q over keys k, values v, all fp64."""
    if not len(k):
        return torch.zeros_like(q), torch.full((len(q),), float("-inf"), dtype=torch.float64, device=q.device)
    s = q @ k.T / q.shape[1] ** 0.5
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ v, lse


def _exact_history(st, pick):
    case = st["case"]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    G = H // Hkv
    kv, q_off = st["kv"].tolist(), st["q_off"].tolist()
    out = torch.zeros((st["T"], H, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((st["T"], H), dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        rows = range(q_off[r], q_off[r + 1])
        for g in range(Hkv):
            blocks = pick(r, g)
            if not blocks:
                out[rows.start:rows.stop, g * G:(g + 1) * G] = 0
                lse[rows.start:rows.stop, g * G:(g + 1) * G] = float("-inf")
                continue
            pages = st["data"][st["table"][r, blocks].long(), g]
            at = torch.tensor(blocks, device=DEV)[:, None] * PAGE + torch.arange(PAGE, device=DEV)
            keep = (at < kv[r]).flatten()
            half = PAGE * d // 2
            pos = at.flatten()[keep]
            # all pages of this head at once, code by code
            flat = pages[:, :half].reshape(-1, d // 2), pages[:, half:2 * half].reshape(-1, d // 2)
            meta = pages[:, 2 * half:].contiguous().view(torch.bfloat16).double().view(-1, 2, PAGE, 2)
            val = []
            for which in range(2):
                code = torch.empty((len(blocks) * PAGE, d), dtype=torch.float64, device=DEV)
                code[:, 0::2], code[:, 1::2] = flat[which] % 16, flat[which] // 16
                sm = meta[:, which].reshape(-1, 2)
                val.append((code * sm[:, :1] + sm[:, 1:])[keep])
            for h in range(g * G, (g + 1) * G):
                if case.get("causal"):
                    for t in rows:
                        seen = pos < kv[r] - (rows.stop - 1 - t)
                        o, e = _exact_rows(st["Q"][t:t + 1, h].double(), val[0][seen], val[1][seen])
                        out[t, h], lse[t, h] = o[0], e[0]
                else:
                    o, e = _exact_rows(st["Q"][rows.start:rows.stop, h].double(), *val)
                    out[rows.start:rows.stop, h], lse[rows.start:rows.stop, h] = o, e
    return out, lse


def _best(scores, must, k):
    """Python: forced blocks, then the best by (score descending, index ascending), ascending."""
    want = min(len(scores), max(len(must), k))
    rest = sorted((j for j in range(len(scores)) if j not in must), key=lambda j: (-scores[j], j))
    return sorted(list(must) + rest[:want - len(must)])


def _codes64(total, count):
    top = total.abs().amax(-1)
    safe = torch.where(top > 0, top, torch.ones_like(top))
    codes = torch.round(total * 127 / safe[..., None]) * (top > 0)[..., None]
    return codes, (top / (127 * count)).float()


def exact(case, seed):
    kind = case["kind"]
    if kind == "history" and case.get("causal") and sum(_lens(case)[1]) * case["H"] > 20000:
        return None
    if kind == "select" and case["B"] * case["Hkv"] * -(-case["Nq"] // QBLOCK) * _blocks(case["Nk"]) > 4e6:
        return None
    st = prepare(case, seed)
    if kind == "tables":
        ctx, new, free = st["ctx"].tolist(), st["new"].tolist(), st["free"].tolist()
        table = st["table"].tolist()
        used, slots, off = 0, [], [0]
        for r, (c, n) in enumerate(zip(ctx, new)):
            for blk in range(_blocks(c), _blocks(c + n)):
                table[r][blk] = free[used]
                used += 1
            slots += [table[r][p // PAGE] * PAGE + p % PAGE for p in range(c, c + n)]
            off.append(off[-1] + n)
        return (_ints(table), _ints([c + n for c, n in zip(ctx, new)]), _ints(off),
                _ints(slots, torch.int64), _ints([used]))
    if kind == "store":
        found = []
        for x in (st["K"], st["V"]):
            f = x.double()
            lo = f.min(-1, keepdim=True).values
            step = (f.max(-1, keepdim=True).values - lo) / 15
            # the least bf16 value that is not below the step
            near = step.bfloat16()
            up = torch.nextafter(near, torch.full_like(near, float("inf")))
            s = torch.where(near.double() >= step, near, up).double()
            found.append(torch.round((f - lo) / s.clamp_min(1e-300)) * s + lo)
        return tuple(found)
    if kind == "history":
        kv = st["kv"].tolist()
        return _exact_history(st, lambda r, g: list(range(_blocks(kv[r]))))
    if kind == "sparse":
        R, H, Hkv, d = case["R"], case["H"], case["Hkv"], case["d"]
        G = H // Hkv
        kv = st["kv"].tolist()
        qc, qs = _codes64(st["Q"].double(), 1)
        sel = torch.full((R, Hkv, _room(case)), -1, dtype=torch.int32, device=DEV)
        count = torch.zeros((R, Hkv), dtype=torch.int32, device=DEV)
        lists = {}
        for r in range(R):
            n = _blocks(kv[r])
            pages = st["table"][r, :n].long()
            for g in range(Hkv):
                heads = slice(g * G, (g + 1) * G)
                dots = qc[r, heads] @ st["sum_codes"][pages, g].double().T
                part = qs[r, heads, None] * dots.float()
                total = part[0]
                for x in part[1:]:
                    total = total + x
                must = set(range(min(case["sink"], n))) | set(range(max(0, n - 1 - case["band"]), n))
                best = _best((total * st["sum_scale"][pages, g]).tolist(), must, case["k"])
                lists[r, g] = best
                sel[r, g, :len(best)] = _ints(best)
                count[r, g] = len(best)
        out, lse = _exact_history(st, lambda r, g: lists[r, g])
        return sel, count, out, lse
    B, H, Hkv, Nq, Nk, d = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    G, nq, nk = H // Hkv, -(-Nq // QBLOCK), _blocks(Nk)
    if kind == "select":
        sums = lambda x, size: torch.stack([p.double().sum(2) for p in x.split(size, 2)], 2)  # noqa: E731
        size = lambda N, n, blk: _ints([min(blk, N - i * blk) for i in range(n)]).double()  # noqa: E731
        ksum, kn = sums(st["K"], PAGE), size(Nk, nk, PAGE)
        qc, qs = _codes64(sums(st["Q"], QBLOCK), size(Nq, nq, QBLOCK))
        kc, ks = _codes64(ksum, kn)
        sel = torch.full((B, Hkv, nq, _room(case)), -1, dtype=torch.int32)
        count = torch.zeros((B, Hkv, nq), dtype=torch.int32)
        for b in range(B):
            for g in range(Hkv):
                total = None
                for h in range(g * G, (g + 1) * G):
                    part = qs[b, h][:, None] * (qc[b, h] @ kc[b, g].T).float()
                    total = part if total is None else total + part
                rows = (total * ks[b, g]).tolist()
                for i, row in enumerate(rows):
                    must = set(range(min(case["sink"], nk)))
                    if case["band"] >= 0:
                        per = QBLOCK // PAGE
                        must |= set(range(max(0, i * per - case["band"]),
                                          max(0, min(nk, (i + 1) * per + case["band"]))))
                    best = _best(row, must, case["k"])
                    sel[b, g, i, :len(best)] = torch.tensor(best, dtype=torch.int32)
                    count[b, g, i] = len(best)
        return ksum / kn[:, None], sel.to(DEV), count.to(DEV)
    out = torch.zeros((B, H, Nq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, H, Nq), dtype=torch.float64, device=DEV)
    if B * H * nq * case["k"] > 4e6:
        return None
    lists = st["sel"].tolist()
    k_len = [Nk] * B if st["k_len"] is None else st["k_len"].tolist()
    for b in range(B):
        for h in range(H):
            k, v = st["K"][b, h // G].double(), st["V"][b, h // G].double()
            for i in range(nq):
                spans = [(j * PAGE, min(k_len[b], (j + 1) * PAGE)) for j in lists[b][h // G][i] if j >= 0]
                keys = torch.cat([torch.arange(a, max(a, e)) for a, e in spans] or [torch.arange(0)]).to(DEV)
                rows = slice(i * QBLOCK, min(Nq, (i + 1) * QBLOCK))
                out[b, h, rows], lse[b, h, rows] = _exact_rows(st["Q"][b, h, rows].double(), k[keys], v[keys])
    return out, lse
