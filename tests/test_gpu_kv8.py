"""The paged 8-bit cache on the GPU: tables, append and attention against the plain forms.

Whole numbers (tables, slots, codes) and scales are compared exactly: every step of the
append is one fp32 operation that the reference rounds the same way.  Attention is compared
with float64 within the bound that tests/kv8_ref.py counts.
"""
import math
import random

import pytest
import torch

from tests import kv8_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_token_sparse_b200 as ds

D = 128
FORMATS = [torch.int8, torch.float8_e4m3fn]
SCALE = 1.0 / math.sqrt(D)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- tables ---------------------------------------------------------------------

def assign(lens, n_new, free, n_free, table, N, page, state=None):
    """The call's outputs as lists (table, lens_out, n_free_out, cu, slots) and its status."""
    ds.device_status()
    t, f = i32(table), i32(free)
    lo, nf = i32([-7] * len(lens)), i32([-7])
    cu, slots = i32([-7] * (len(lens) + 1)), i32([-7] * N)
    ds.page_assign(i32(lens), i32(n_new), f, i32([n_free]), t, lo, nf, cu, slots, page)
    assert f.tolist() == list(free)
    return t.tolist(), lo.tolist(), nf.item(), cu.tolist(), slots.tolist(), ds.device_status()


def pool(rng, P, lens, W, page):
    """A shuffled pool: table rows of the given lengths (unused entries -1), free list, count."""
    ids = list(range(P))
    rng.shuffle(ids)
    table = []
    for n in lens:
        k = -(-n // page)
        table.append([ids.pop() for _ in range(k)] + [-1] * (W - k))
    return table, ids + [-1] * (P - len(ids)), len(ids)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,len_max,new_max", [(1, 0, 1), (1, 40, 300), (7, 200, 1), (33, 300, 5),
                                               (300, 100, 90), (1025, 50, 20), (3000, 20, 1)])
def test_assign(page, B, len_max, new_max):
    rng = random.Random(B * page + new_max)
    lens = [rng.randint(0, len_max) for _ in range(B)]
    n = [rng.randint(0, new_max) for _ in range(B)]
    lens[-1] = len_max
    W = -(-(len_max + new_max) // page)
    P = sum(-(-x // page) for x in lens) + sum(-(-x // page) + 1 for x in n) + 3
    table, free, nf = pool(rng, P, lens, W, page)
    want = ref.assign(lens, n, free, nf, table, sum(n) + 11, page)  # 11 padded slots
    got = assign(lens, n, free, nf, table, sum(n) + 11, page)
    assert got == want and got[5] == 0


def test_assign_refuses_what_does_not_fit():
    page, W, P = 16, 4, 30
    rng = random.Random(5)
    for lens, n, nf_cut, N in [
            ([16, 0, 40, 3], [20, 33, 0, 1], None, 60),   # all fit
            ([16, 0, 40, 3], [20, 33, 0, 1], 3, 60),      # too few pages for the second
            ([16, 0, 48, 3], [20, 33, 16, 1], 3, 80),     # the third and fourth: one more, none
            ([16, 0, 40, 3], [20, 33, 0, 1], 0, 60),      # no page at all: only the fourth
            ([16, 0, 40, 3], [20, 65, 0, 1], None, 90),   # the second past its table row
            ([16, -1, 40, 3], [20, 5, -3, 1], None, 60),  # negative values
            ([16, 0, 40, 3], [20, 33, 0, 1], None, 40),   # tokens past the buffer
            ([16, 0, 64, 3], [0, 0, 1, 0], None, 5),      # a full row
            ([16, 0, 64, 3], [0, 0, 0, 0], None, 0)]:     # nothing at all
        held = [max(0, x) for x in lens]
        table, free, nf = pool(rng, P, held, W, page)
        nf = nf if nf_cut is None else nf_cut
        want = ref.assign(lens, n, free, nf, table, N, page)
        assert assign(lens, n, free, nf, table, N, page) == want, (lens, n)


def test_assign_flags_bad_pages():
    # a held page and a free page outside the pool
    table, free = [[99, -1, -1], [0, -1, -1]], [1, -5, 2, 3]
    want = ref.assign([3, 16], [2, 30], free, 3, table, 32, 16)
    got = assign([3, 16], [2, 30], free, 3, table, 32, 16)
    assert got == want and got[5] == ds.DEV_BAD_PAGE


def release(lens, done, table, free, n_free, page):
    ds.device_status()
    f, lo, nf = i32(free), i32([-7] * len(lens)), i32([-7])
    ds.page_release(i32(lens), i32(done), i32(table), f, i32([n_free]), lo, nf, page)
    return f.tolist(), lo.tolist(), nf.item(), ds.device_status()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("B,len_max,share", [(1, 0, 1.0), (1, 700, 1.0), (40, 300, 0.0),
                                             (40, 300, 0.3), (1500, 90, 0.8), (900, 900, 1.0)])
def test_release(page, B, len_max, share):
    rng = random.Random(B + len_max)
    lens = [rng.randint(0, len_max) for _ in range(B)]
    done = [rng.choice([1, 7, -1]) if rng.random() < share else 0 for _ in range(B)]
    W = -(-len_max // page) + 2
    table, free, nf = pool(rng, sum(-(-x // page) for x in lens) + 4, lens, W, page)
    want = ref.release(lens, done, table, free, nf, page)
    got = release(lens, done, table, free, nf, page)
    assert got == want and got[3] == 0


def test_release_of_bad_values():
    # lengths outside the table, an id outside the pool, more pages than the pool has room for
    table = [[3, 1], [0, 77], [2, 3]]
    for lens, done, nf in [([-4, 20, 32], [1, 1, 0], 0), ([1000, 20, 32], [1, 0, 0], 1),
                           ([32, 32, 32], [1, 1, 1], 1)]:
        want = ref.release(lens, done, table, [9, 9, 9, 9], nf, 16)
        assert release(lens, done, table, [9, 9, 9, 9], nf, 16) == want, lens


# ---- append ---------------------------------------------------------------------

def cache(seed, P, Hkv, page, dtype, spread=1.0, k_scale=0.02):
    """Random codes and scales [P, Hkv, 2] that differ by about 2^spread from page to page."""
    g = gen(seed)
    shape = (P, Hkv, page, 2, D)
    if dtype == torch.int8:
        KV = torch.randint(-127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8)
    else:
        KV = (torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(dtype)
        k_scale = k_scale / 2
    sc = torch.exp2(torch.randn((P, Hkv, 2), generator=g) * spread) * k_scale
    return KV.cuda(), sc.cuda()


def same_cache(got, want):
    (KV, sc), (KVr, scr) = got, want
    assert torch.equal(KV.cpu().view(torch.uint8), KVr.view(torch.uint8))
    assert torch.equal(sc.cpu(), scr)


def new_rows(seed, N, Hkv, extra=0):
    """K and V rows [N, Hkv, D] as slices of a fused projection's output of more columns."""
    x = torch.randn((N, 2 * Hkv * D + extra), generator=gen(seed))
    x = x * torch.exp2(torch.randn((N, 1), generator=gen(seed + 1)))
    x = x.bfloat16().cuda()
    return x[:, extra:extra + Hkv * D].view(N, Hkv, D), x[:, extra + Hkv * D:].view(N, Hkv, D)


def slots_of(rng, lens, n_new, page, P):
    W = max(-(-(a + b) // page) for a, b in zip(lens, n_new)) + 1
    table, _, _ = pool(rng, P, [a + b for a, b in zip(lens, n_new)], W, page)
    cu, slots = [0], []
    for b, (l, n) in enumerate(zip(lens, n_new)):
        slots += [table[b][p // page] * page + p % page for p in range(l, l + n)]
        cu.append(cu[-1] + n)
    return i32(slots), i32(cu), table


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,lens,n_new,extra", [
    (1, [0], [1], 0),
    (2, [5, 0, 16, 127, 31], [1, 1, 1, 1, 1], 256),
    (3, [0, 7, 128, 50], [300, 0, 1, 78], 8),
    (8, [15, 16, 17], [33, 16, 15], 0),
    (5, [200, 3], [3, 129], 1024),
])
def test_append(dtype, page, Hkv, lens, n_new, extra):
    ds.device_status()
    P = sum(-(-(a + b) // page) for a, b in zip(lens, n_new)) + 3
    slots, cu, _ = slots_of(random.Random(page + Hkv), lens, n_new, page, P)
    K, V = new_rows(Hkv * 10 + page, len(slots), Hkv, extra)
    # old scales below and above what the new rows need, rows behind the new ones of any value
    KV, sc = cache(page, P, Hkv, page, dtype, spread=2.0)
    want = ref.append(K, V, KV, sc, slots, cu, page)
    ds.kv8_append(K, V, KV, sc, slots, cu, max(n_new))
    same_cache((KV, sc), want)
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("most", [1, 1000])
def test_append_of_mixed_runs(dtype, page, most):
    """Single tokens, short runs and prompts side by side: the runs that begin in a block of
    tokens go from none to all of them, whatever max_new says."""
    ds.device_status()
    rng = random.Random(page)
    n = [1] * 40 + [333, 1, 0, 5, 129] + [2] * 30 + [64, 700] + [1] * 9 + [17, 0, 1]
    lens = [rng.randint(0, 200) for _ in n]
    P = sum(-(-(a + b) // page) for a, b in zip(lens, n)) + 3
    slots, cu, _ = slots_of(rng, lens, n, page, P)
    slots[50:53] = -1  # tokens without a place inside a run
    K, V = new_rows(page, len(slots), 2, 64)
    K[100], V[101, 1, 3] = math.nan, math.inf
    KV, sc = cache(page, P, 2, page, dtype, spread=2.0)
    # the rest of the page behind the gap is refused, later pages are stored
    after = 53 + next(k for k in range(page) if slots[53 + k] % page == 0)
    kept = slots.clone()
    kept[53:after] = -1
    want = ref.append(K, V, KV, sc, kept, i32(sorted({*cu.tolist(), 50, after})), page)
    ds.kv8_append(K, V, KV, sc, slots, cu, most)
    same_cache((KV, sc), want)
    stored_odd = after <= 101  # a page of 128 tokens ends behind them
    assert ds.device_status() == ds.DEV_BAD_PAGE | (ds.DEV_NONFINITE if stored_odd else 0)


@pytest.mark.parametrize("dtype", FORMATS)
def test_append_of_odd_values(dtype):
    """Zeros, the smallest and largest bf16 values, infinities and NaN."""
    inf, nan, big = math.inf, math.nan, 3.38e38
    page, Hkv, N = 16, 2, 24
    for vals, flagged in [([0.0, -0.0], 0), ([1e-40, -1e-39], 0), ([big, -big, 1.0], 0),
                          ([inf, -2.0, 3.0], 1), ([nan, 0.5, -inf], 1), ([nan], 1)]:
        ds.device_status()
        x = torch.tensor(vals)[torch.randint(0, len(vals), (2, N, Hkv, D), generator=gen(3))]
        K, V = x.bfloat16().cuda()
        KV, sc = cache(9, 3, Hkv, page, dtype)
        slots = i32([40 + i if i < 8 else i - 8 for i in range(N)])  # off 8 of page 2, page 0
        want = ref.append(K, V, KV, sc, slots, i32([0, N]), page)
        ds.kv8_append(K, V, KV, sc, slots, i32([0, N]), N)
        same_cache((KV, sc), want)
        assert ds.device_status() == (ds.DEV_NONFINITE if flagged else 0)


@pytest.mark.parametrize("dtype", FORMATS)
def test_append_skips_and_flags(dtype):
    page, Hkv, P = 16, 2, 5
    K, V = new_rows(1, 12, Hkv)
    for slots, cu, most, bits in [
            ([-1] * 6 + list(range(32, 38)), [0, 6, 12], 6, 0),          # a refused request
            (list(range(6)) + list(range(32, 38)), [0, 6, 12, 12], 6, 0),  # an empty sequence
            (list(range(12)), [0, 12], 100, 0),                           # a loose bound
            (list(range(80, 92)), [0, 12], 12, ds.DEV_BAD_PAGE),          # a page past the pool
            (list(range(12)), [0, 40], 12, ds.DEV_BAD_LENGTH),            # counts past the buffer
            (list(range(12)), [-3, 12], 12, ds.DEV_BAD_LENGTH)]:
        ds.device_status()
        KV, sc = cache(4, P, Hkv, page, dtype)
        cut = [min(max(c, 0), 12) for c in cu]
        want = (KV.cpu().clone(), sc.cpu().clone()) if bits == ds.DEV_BAD_PAGE else \
            ref.append(K, V, KV, sc, i32(slots), i32(cut), page)
        ds.kv8_append(K, V, KV, sc, i32(slots), i32(cu), most)
        same_cache((KV, sc), want)
        assert ds.device_status() == bits


@pytest.mark.parametrize("Hkv,G,r", [(2, 1, 16), (1, 8, 8), (3, 4, 5), (2, 2, 128)])
def test_append_writes_label_rows(Hkv, G, r):
    ds.device_status()
    Hq, page, lens, n = Hkv * G, 32, [10, 0, 63], [1, 70, 5]
    slots, cu, _ = slots_of(random.Random(r), lens, n, page, 12)
    K, V = new_rows(7, sum(n), Hkv, 128)
    KV, sc = cache(2, 12, Hkv, page, torch.int8)
    T_cap = 69  # the second sequence's last token is past it
    label = torch.full((3, Hq, T_cap, r), 9.0, dtype=torch.bfloat16, device="cuda")
    C = torch.stack([torch.randperm(D, generator=gen(h))[:r] for h in range(Hq)]).int().cuda()
    want = label.clone()
    for b in range(3):
        for h in range(Hq):
            rows = K[cu[b]:cu[b + 1], h // G][:, C[h].long()]
            m = min(n[b], T_cap - lens[b])
            want[b, h, lens[b]:lens[b] + m] = rows[:m]
    kv = ref.append(K, V, KV, sc, slots, cu, page)
    ds.kv8_append(K, V, KV, sc, slots, cu, 70, C=C, label=label, lens=i32(lens))
    assert torch.equal(label, want)
    same_cache((KV, sc), kv)
    assert ds.device_status() == ds.DEV_BAD_LENGTH
    C[0, 0] = 200
    ds.kv8_append(K, V, KV, sc, slots, cu, 70, C=C, label=label, lens=i32([0, 0, 0]))
    assert ds.device_status() & ds.DEV_BAD_CHANNEL


# ---- attention ------------------------------------------------------------------

def setup(seed, lens, Hkv, page, dtype, spread=1.0):
    """A cache of the given lengths; rows behind a sequence's end hold any code (e4m3 NaN too)."""
    P = sum(-(-max(n, 0) // page) for n in lens) + 2
    W = max(-(-max(n, 0) // page) for n in lens) + 1
    table, _, _ = pool(random.Random(seed), P, [max(n, 0) for n in lens], W, page)
    KV, sc = cache(seed, P, Hkv, page, dtype, spread)
    u8 = KV.view(torch.uint8)
    for b, n in enumerate(lens):
        if n > 0 and n % page:
            junk = torch.randint(0, 256, (Hkv, page - n % page, 2, D), generator=gen(b),
                                 dtype=torch.int32).to(torch.uint8).cuda()
            junk[..., ::7] = 0x7f
            u8[table[b][n // page], :, n % page:] = junk
    return KV, sc, i32(table)


def queries(seed, B, Hq):
    return torch.randn((B, Hq, D), generator=gen(seed)).bfloat16().cuda()


def outputs(B, Hq):
    return (torch.full((B, Hq, D), math.nan, device="cuda"),
            torch.full((B, Hq), math.nan, device="cuda"))


def check(Q, KV, sc, table, page, tokens, O, lse, heads=None):
    """O and lse against the reference; tokens(b, h): the tokens of a query head, in any order."""
    B, Hq, _ = Q.shape
    G = Hq // KV.shape[1]
    O, lse = O.cpu().double(), lse.cpu().double()
    KV, sc, table = KV.cpu(), sc.cpu(), table.cpu()
    for b, h in heads or [(b, h) for b in range(B) for h in range(Hq)]:
        ids = tokens(b, h)
        K, V = ref.rows(KV, sc, table, b, h // G, ids, page)
        sv = ref.v_scales(sc, table, b, h // G, ids, page)
        o, l, tol_o, tol_l = ref.attend(Q[b, h], K, V, SCALE, sv)
        if K.shape[0] == 0:
            assert torch.equal(O[b, h], o) and lse[b, h].item() == -math.inf, (b, h)
            continue
        err = (O[b, h] - o).abs()
        assert (err <= tol_o).all(), (b, h, err.max().item(), (err / tol_o).max().item())
        assert abs(lse[b, h].item() - l) <= tol_l, (b, h, lse[b, h].item(), l, tol_l)


def run_dense(Q, KV, sc, table, lens, ws=None):
    O, lse = outputs(*Q.shape[:2])
    ds.kv8_decode(Q, KV, sc, table, lens, O, SCALE, lse=lse, ws=ws)
    return O, lse


DENSE = [
    # lens, Hq, Hkv, page
    ([1], 1, 1, 16),
    ([0, 0], 2, 2, 64),
    ([15, 16, 17], 3, 3, 16),
    ([0, 1, 31, 0, 32, 33, 0], 8, 2, 32),
    ([100, 1, 777], 6, 2, 64),
    ([129, 300], 20, 5, 128),
    ([511, 64, 0, 65], 10, 2, 64),
    ([1000, 17], 8, 1, 16),
    ([333, 334], 24, 2, 32),
    ([640, 5], 16, 1, 128),
    ([90, 200], 34, 2, 64),        # 17 heads a group
    ([150], 64, 1, 16),            # 64 heads a group
    ([20] * 40, 64, 32, 16),       # many short sequences
    ([7] * 200, 4, 2, 16),
    ([6000, 200, 3], 16, 4, 64),
    ([20000], 1, 1, 128),
    ([70001], 3, 1, 32),
    ([33000, 1], 16, 1, 64),
]


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("lens,Hq,Hkv,page", DENSE)
def test_dense(dtype, lens, Hq, Hkv, page):
    ds.device_status()
    seed = sum(lens) + Hq
    KV, sc, table = setup(seed, lens, Hkv, page, dtype)
    Q = queries(seed, len(lens), Hq)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)
    O2, lse2 = run_dense(Q, KV, sc, table, i32(lens))
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    O3 = torch.empty_like(O)
    ds.kv8_decode(Q, KV, sc, table, i32(lens), O3, SCALE)  # without lse
    assert torch.equal(O, O3)
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 13, 16])
def test_dense_group_sizes(dtype, G):
    lens, Hkv, page = [400, 0, 61, 1500], 3, 32
    KV, sc, table = setup(G, lens, Hkv, page, dtype)
    Q = queries(G, 4, G * Hkv)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("B,Hq,Hkv,len_max,page", [
    (129, 8, 2, 70, 16),       # more sequences than a warp plans by itself
    (500, 64, 8, 96, 32),      # lists shorter than a warp's range
    (1600, 4, 1, 90, 64),      # more than one round of a CTA's threads
    (3500, 16, 1, 40, 16),
])
def test_dense_many_sequences(dtype, B, Hq, Hkv, len_max, page):
    ds.device_status()
    rng = random.Random(B)
    lens = [0 if rng.random() < 0.1 else rng.randint(1, len_max) for _ in range(B)]
    KV, sc, table = setup(B, lens, Hkv, page, dtype)
    Q = queries(B, B, Hq)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    empty = i32(lens) == 0
    assert (O[empty] == 0).all() and (lse[empty] == -math.inf).all()
    assert torch.isfinite(O).all() and torch.isfinite(lse[~empty]).all()
    heads = {(0, 0), (B - 1, Hq - 1)} | {(rng.randrange(B), rng.randrange(Hq)) for _ in range(400)}
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse, heads=sorted(heads))
    O2, lse2 = run_dense(Q, KV, sc, table, i32(lens))
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
def test_sparse_bad_lengths(dtype):
    """Lengths outside the table, in the calls over lists."""
    ds.device_status()
    page = 16
    KV, sc, table = setup(45, [64, 64], 2, page, dtype)
    Q = queries(46, 2, 2)
    O, lse = outputs(2, 2)
    idx = lists(47, [table.shape[1] * page - page, 64], 2, 20)
    ds.kv8_sparse_decode(Q, KV, sc, table, i32([10 ** 6, 64]), idx, O, SCALE, lse=lse)
    assert ds.device_status() == ds.DEV_BAD_LENGTH
    check(Q, KV, sc, table, page, lambda b, h: idx[2 * b + h].tolist(), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("spread", [0.0, 6.0, 30.0])
def test_dense_scales_of_any_size(dtype, spread):
    """V scales from page to page up to 2^+-64 apart, K scales that keep the logits ordinary."""
    lens, Hkv, page = [500, 90], 2, 16
    KV, sc, table = setup(11, lens, Hkv, page, dtype, spread=1.0)
    sc[..., 1] = torch.exp2((torch.randn(sc.shape[:2], generator=gen(4)) * spread)
                            .clamp(-64, 64)).cuda()
    Q = queries(12, 2, 8)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
def test_dense_peaked_and_zero_queries(dtype):
    """One token far above the rest, logits of both signs in the hundreds, and q = 0."""
    lens, page = [300, 300, 300], 16
    KV, sc, table = setup(21, lens, 1, page, dtype, spread=0.3)
    Q = queries(22, 3, 4)
    Q[0] *= 16.0
    Q[1] *= 2.0 ** -20
    Q[2] = 0
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("top", [18, 21, 25, 30, 40])
@pytest.mark.parametrize("order", ["up", "down", "mixed", "negative"])
def test_dense_logits_far_from_zero(dtype, top, order):
    """Whole logits of up to 2^top, exact in fp32: the softmax is an even share among the tokens
    that hold the largest, whatever the V scales beside them."""
    n, page = 2000, 16
    KV, sc, table = setup(25, [n, n], 1, page, dtype, spread=1.0)
    sc[..., 0] = 1.0
    sc[..., 1] = torch.exp2((torch.randn(sc.shape[:2], generator=gen(5)) * 30).clamp(-60, 60)).cuda()
    code = torch.randint(-8, 9, (n,), generator=gen(6)).sort().values
    code = {"up": code, "down": code.flip(0), "mixed": code[torch.randperm(n, generator=gen(7))],
            "negative": -code.abs() - 4}[order]
    pages = torch.arange(n) // page
    K = torch.zeros((n, D))
    K[:, 5] = code
    for b in range(2):
        KV[table[b].cpu()[pages].cuda().long(), 0, torch.arange(n).cuda() % page, 0] = \
            K.to(dtype).cuda()
    Q = torch.zeros((2, 4, D), dtype=torch.bfloat16, device="cuda")
    Q[:, :, 5] = 2.0 ** (top - 3)
    Q[:, 1::2, 5] *= -1
    O, lse = outputs(2, 4)
    ds.kv8_decode(Q, KV, sc, table, i32([n, n]), O, 1.0, lse=lse)
    # other tokens are 2^(top-3) below, so what is left to round are the sums (n/4 + 200
    # roundings), the parts of the weights (see ref.attend) and, in lse, the logit itself
    u = 2.0 ** -24
    for b in range(2):
        for h in range(4):
            Kr, V = ref.rows(KV, sc, table, b, 0, range(n), page)
            sv = ref.v_scales(sc, table, b, 0, range(n), page)
            x = Kr @ Q[b, h].cpu().double()
            w = torch.softmax(x, 0)
            tol = (n / 4 + 200) * u * (w @ V.abs()) + \
                2.0 ** -38 * (w * sv).amax() * (V / sv[:, None]).abs().sum(0)
            assert ((O[b, h].cpu().double() - w @ V).abs() <= tol).all(), (b, h)
            want = torch.logsumexp(x, 0).item()
            assert abs(lse[b, h].item() - want) <= 8 * u * abs(want) + 1e-4, (b, h)


@pytest.mark.parametrize("dtype", FORMATS)
def test_dense_zero_scales(dtype):
    """Pages of scale 0 (another program's all-zero pages) count with logit 0 and value 0."""
    lens, page = [100], 16
    KV, sc, table = setup(31, lens, 2, page, dtype)
    sc[table[0, 1:5].long()] = 0.0
    Q = queries(32, 1, 4)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)
    sc.zero_()
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    check(Q, KV, sc, table, page, lambda b, h: range(lens[b]), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
def test_dense_bad_lengths_and_pages(dtype):
    ds.device_status()
    page, W = 16, 4
    KV, sc, table = setup(41, [50, 64, 20], 2, page, dtype)
    table = table[:, :W].contiguous()
    table[2, 2:] = 0
    Q = queries(42, 3, 4)
    O, lse = run_dense(Q, KV, sc, table, i32([-5, 1000, 20]))
    assert ds.device_status() == ds.DEV_BAD_LENGTH
    check(Q, KV, sc, table, page, lambda b, h: range([0, 64, 20][b]), O, lse)
    good = table.clone()
    table[0, 1], table[1, 0] = -1, KV.shape[0]
    O, lse = run_dense(Q, KV, sc, table, i32([50, 64, 20]))
    assert ds.device_status() == ds.DEV_BAD_PAGE
    keep = [[*range(16), *range(32, 50)], range(16, 64), range(20)]
    check(Q, KV, sc, good, page, lambda b, h: keep[b], O, lse)


def lists(seed, lens, H, k, fill=1.0):
    """k distinct tokens a row where the sequence has them, -1 elsewhere, in random order."""
    g, out = gen(seed), torch.full((len(lens), H, k), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            m = min(n, int(k * fill))
            out[b, h, torch.randperm(k, generator=g)[:m]] = \
                torch.randperm(n, generator=g)[:m].int()
    return out.view(-1, k).cuda()


SPARSE = [
    # lens, Hq, Hkv, page, k
    ([1], 1, 1, 16, 1),
    ([5, 0, 40], 4, 2, 16, 3),
    ([100, 17], 6, 2, 32, 16),
    ([300, 20], 8, 1, 64, 17),
    ([4000, 999], 10, 5, 128, 250),
    ([2000, 1, 77], 24, 2, 16, 100),
    ([900], 16, 1, 64, 31),
    ([700, 800], 34, 2, 64, 48),
    ([9000], 2, 1, 32, 9000),
    ([50] * 60, 32, 32, 16, 7),
]


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,page,k", SPARSE)
def test_sparse(dtype, shared, lens, Hq, Hkv, page, k):
    ds.device_status()
    KV, sc, table = setup(k, lens, Hkv, page, dtype)
    B, H = len(lens), Hkv if shared else Hq
    idx = lists(k, lens, H, k, 0.8 if k % 2 else 1.0)
    idx[0] = -1  # a list with nothing in it
    Q = queries(k, B, Hq)
    fn = ds.kv8_group_sparse_decode if shared else ds.kv8_sparse_decode
    O, lse = outputs(B, Hq)
    fn(Q, KV, sc, table, i32(lens), idx, O, SCALE, lse=lse)
    rows = idx.cpu().view(B, H, k)

    def tokens(b, h):
        r = rows[b, h * H // Hq]
        return r[r >= 0].tolist()
    check(Q, KV, sc, table, page, tokens, O, lse)
    O2, lse2 = outputs(B, Hq)
    fn(Q, KV, sc, table, i32(lens), idx, O2, SCALE, lse=lse2, ws=ds.kv8_workspace(Q, KV))
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("shared", [False, True])
def test_sparse_bad_and_repeated_ids(dtype, shared):
    ds.device_status()
    lens, page, k = [60, 33], 16, 20
    KV, sc, table = setup(51, lens, 2, page, dtype)
    Q = queries(52, 2, 4)
    H = 2 if shared else 4
    idx = lists(53, lens, H, k)
    idx[:, 3] = idx[:, 4]         # counts twice
    idx[0, 5], idx[1, 6], idx[2 * H - 1, 7] = 60, -2, 2 ** 31 - 1
    fn = ds.kv8_group_sparse_decode if shared else ds.kv8_sparse_decode
    O, lse = outputs(2, 4)
    fn(Q, KV, sc, table, i32(lens), idx, O, SCALE, lse=lse)
    assert ds.device_status() == ds.DEV_BAD_INDEX
    rows = idx.cpu().view(2, H, k)

    def tokens(b, h):
        r = rows[b, h * H // 4]
        return r[(r >= 0) & (r < lens[b])].tolist()
    check(Q, KV, sc, table, page, tokens, O, lse)
    bad = table.clone()
    bad[0, 1] = KV.shape[0] + 3
    fn(Q, KV, sc, bad, i32(lens), idx, O, SCALE, lse=lse)
    assert ds.device_status() == ds.DEV_BAD_INDEX | ds.DEV_BAD_PAGE
    check(Q, KV, sc, table, page,
          lambda b, h: [t for t in tokens(b, h) if b or t // page != 1], O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
def test_offsets_past_32_bits(dtype):
    """Pages beyond 4 GiB of codes, for the append and the three attention calls."""
    page, Hkv, P, n = 128, 2, 70000, 300
    KV = torch.empty((P, Hkv, page, 2, D), dtype=torch.uint8, device="cuda").view(dtype)
    sc = torch.ones((P, Hkv, 2), device="cuda")
    assert KV.numel() > 2 ** 32
    ids = [P - 1, 3, P - 40]
    table = i32([ids])
    slots = i32([ids[t // page] * page + t % page for t in range(n)])
    K, V = new_rows(61, n, Hkv)
    ds.kv8_append(K, V, KV, sc, slots, i32([0, n]), n)
    small, ssc = KV[ids].contiguous(), sc[ids].contiguous()
    zero = (torch.zeros_like(small.view(torch.uint8)).view(dtype), torch.zeros_like(ssc))
    want = ref.append(K, V, *zero, i32(list(range(n))), i32([0, n]), page)
    KVr = small.cpu().view(torch.uint8).clone()
    KVr[2, :, n % page:] = 0
    same_cache((KVr.view(dtype), ssc), want)
    Q = queries(62, 1, 4)
    O, lse = run_dense(Q, KV, sc, table, i32([n]))
    check(Q, small, ssc, i32([[0, 1, 2]]), page, lambda b, h: range(n), O, lse)
    idx = lists(63, [n], 4, 77)
    ds.kv8_sparse_decode(Q, KV, sc, table, i32([n]), idx, O, SCALE, lse=lse)
    check(Q, small, ssc, i32([[0, 1, 2]]), page, lambda b, h: idx[h].tolist(), O, lse)


@pytest.mark.parametrize("dtype", FORMATS)
def test_codes_in_host_memory(dtype):
    """Codes in page-locked host memory: the same bits as from device memory."""
    lens, page = [200, 45], 32
    KV, sc, table = setup(71, lens, 2, page, dtype)
    host = KV.view(torch.uint8).cpu().pin_memory().view(dtype)
    Q, (K, V) = queries(72, 2, 8), new_rows(73, 3, 2)
    idx = lists(74, lens, 8, 31)
    out = []
    for codes, scales in ((KV, sc), (host, sc.clone())):
        O, lse = run_dense(Q, codes, scales, table, i32(lens))
        O2, lse2 = outputs(2, 8)
        ds.kv8_sparse_decode(Q, codes, scales, table, i32(lens), idx, O2, SCALE, lse=lse2)
        slots = i32([table[1, 1].item() * page + 13 + i for i in range(3)])
        ds.kv8_append(K, V, codes, scales, slots, i32([0, 0, 3]), 3)
        torch.cuda.synchronize()
        out.append((O, lse, O2, lse2, scales, codes.view(torch.uint8).cpu()))
    for a, b in zip(*out):
        assert torch.equal(a, b)


# ---- the calls together -----------------------------------------------------------

class Server:
    """A cache served as a decode loop does: every buffer made once, each step one set of calls."""

    def __init__(self, B, Hq, Hkv, page, W, P, dtype, N):
        self.B, self.Hq, self.Hkv, self.page = B, Hq, Hkv, page
        self.KV = torch.zeros((P, Hkv, page, 2, D), dtype=torch.uint8, device="cuda").view(dtype)
        self.sc = torch.zeros((P, Hkv, 2), device="cuda")
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(P, generator=gen(P)).int().cuda()
        self.n_free, self.n_free2 = i32([P]), i32([0])
        self.lens, self.lens2 = i32([0] * B), i32([0] * B)
        self.cu, self.slots = i32([0] * (B + 1)), i32([0] * N)
        self.n_new, self.done = i32([0] * B), i32([0] * B)
        self.K = torch.zeros((N, Hkv, D), dtype=torch.bfloat16, device="cuda")
        self.V = torch.zeros_like(self.K)
        self.Q = torch.zeros((B, Hq, D), dtype=torch.bfloat16, device="cuda")
        self.O, self.lse = outputs(B, Hq)
        self.ws = ds.kv8_workspace(self.Q, self.KV)

    def step(self, max_new):
        ds.page_assign(self.lens, self.n_new, self.free, self.n_free, self.table, self.lens2,
                       self.n_free2, self.cu, self.slots, self.page)
        ds.kv8_append(self.K, self.V, self.KV, self.sc, self.slots, self.cu, max_new)
        ds.kv8_decode(self.Q, self.KV, self.sc, self.table, self.lens2, self.O, SCALE,
                      lse=self.lse, ws=self.ws)
        ds.page_release(self.lens2, self.done, self.table, self.free, self.n_free2, self.lens,
                        self.n_free, self.page)


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(dtype, captured):
    """Prompts, decode steps, requests that end and others that take their pages; eager, and as
    two captured graphs that share a workspace, replayed on a stream of their own."""
    ds.device_status()
    B, page, N = 5, 16, 200
    s = Server(B, 8, 2, page, 8, 24, dtype, N)
    st = torch.cuda.Stream()
    graphs = {}
    if captured:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            s.step(100), s.step(1)  # nothing new: the first calls outside a capture
            for most in (100, 1):
                graphs[most] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs[most], stream=st):
                    s.step(most)
    past = [[] for _ in range(B)]  # the rows each sequence holds, as bf16
    rng = random.Random(8)
    for it in range(12):
        prompt = it % 4 == 0
        n = [rng.choice([0, 3, 17, 40]) if prompt and not past[b] else int(bool(past[b]))
             for b in range(B)]
        done = [int(bool(past[b]) and rng.random() < 0.25) for b in range(B)]
        K, V = new_rows(100 + it, N, 2)
        Q = queries(it, B, 8)
        torch.cuda.synchronize()
        s.K.copy_(K), s.V.copy_(V), s.Q.copy_(Q)
        s.n_new.copy_(i32(n)), s.done.copy_(i32(done))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graphs[100 if prompt else 1].replay() if captured else s.step(max(1, max(n)))
        st.synchronize()
        at = 0
        for b in range(B):
            past[b] += [(K[i].double().cpu(), V[i].double().cpu()) for i in range(at, at + n[b])]
            at += n[b]
        assert s.lens2.tolist() == [len(p) for p in past]
        check(s.Q, s.KV, s.sc, s.table, page, lambda b, h: range(len(past[b])), s.O, s.lse)
        # the cache holds the rows to half a step, and to one more for each time a scale grew
        for b in range(B):
            for g in range(2):
                rows = ref.rows(s.KV, s.sc, s.table, b, g, range(len(past[b])), page)
                for kv in (0, 1):
                    for t, x in enumerate(past[b]):
                        step = s.sc[s.table[b, t // page], g, kv].item()
                        err = (rows[kv][t] - x[kv][g]).abs()
                        unit = step * (1 if dtype == torch.int8 else 32)  # e4m3 steps at 448
                        assert err.max() <= unit * (0.5 + 0.5 * page), (it, b, t)
        past = [[] if d else p for p, d in zip(past, done)]
        assert s.lens.tolist() == [len(p) for p in past]
        held = sorted(x for b in range(B)
                      for x in s.table[b, :-(-len(past[b]) // page)].tolist())
        assert sorted(held + s.free[:s.n_free.item()].tolist()) == list(range(24))
    assert ds.device_status() == 0


def test_calls_with_selection():
    """Labels from the append, selection by the library's own top-k, attention over the kept."""
    B, Hq, Hkv, page, r, k, T = 2, 8, 2, 64, 16, 50, 400
    s = Server(B, Hq, Hkv, page, 8, 20, torch.int8, B * T)
    K, V = new_rows(5, B * T, Hkv)
    Q = queries(6, B, Hq)
    s.n_new.fill_(T)
    C = torch.stack([torch.randperm(D, generator=gen(h))[:r].sort().values
                     for h in range(Hq)]).int().cuda()
    label = torch.zeros((B, Hq, T, r), dtype=torch.bfloat16, device="cuda")
    ds.page_assign(s.lens, s.n_new, s.free, s.n_free, s.table, s.lens2, s.n_free2, s.cu, s.slots,
                   page)
    ds.kv8_append(K, V, s.KV, s.sc, s.slots, s.cu, T, C=C, label=label, lens=s.lens)
    dense = K.view(B, T, Hkv, D).transpose(1, 2).contiguous()
    label2 = torch.zeros_like(label)
    ds.label_append(dense, C, label2, 0, T)
    assert torch.equal(label, label2)
    idx = torch.empty((B * Hq, k), dtype=torch.int32, device="cuda")
    ds.score_topk(Q, C, label, idx, T)
    O, lse = outputs(B, Hq)
    ds.kv8_sparse_decode(Q, s.KV, s.sc, s.table, s.lens2, idx, O, SCALE, lse=lse, ws=s.ws)
    check(Q, s.KV, s.sc, s.table, page, lambda b, h: idx[b * Hq + h].tolist(), O, lse)
    gidx = torch.empty((B * Hkv, k), dtype=torch.int32, device="cuda")
    scores = torch.empty((B * Hkv, T), dtype=torch.float32, device="cuda")
    ds.group_score_topk(Q, C, label, scores, gidx, T)
    ds.kv8_group_sparse_decode(Q, s.KV, s.sc, s.table, s.lens2, gidx, O, SCALE, lse=lse, ws=s.ws)
    check(Q, s.KV, s.sc, s.table, page, lambda b, h: gidx[b * Hkv + h // 4].tolist(), O, lse)


def test_short_lists_of_tokens_that_do_not_exist():
    """Every sequence empty: no row is read whatever the lists say."""
    ds.device_status()
    KV, sc, table = setup(81, [16, 16], 1, 16, torch.int8)
    Q = queries(82, 2, 2)
    O, lse = outputs(2, 2)
    ds.kv8_sparse_decode(Q, KV, sc, table, i32([0, 0]), i32([[0, 5]] * 4), O, SCALE, lse=lse)
    assert (O == 0).all() and (lse == -math.inf).all()
    assert ds.device_status() == ds.DEV_BAD_INDEX


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("most", [1, 100])
def test_append_after_refused_requests(dtype, most):
    """Sequences in the middle of a page behind requests that got no pages are stored: they begin
    where their counts say, with empty sequences between."""
    ds.device_status()
    page, n = 16, [3, 1, 0, 0, 1, 20, 1]
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    first = [-1, 5, 0, 0, 16 + 15, -1, 64 + 9]  # slots of each sequence's tokens, in a page each
    slots = [-1 if f < 0 else f + i for f, k in zip(first, n) for i in range(k)]
    K, V = new_rows(3, len(slots), 2)
    KV, sc = cache(5, 6, 2, page, dtype, spread=2.0)
    want = ref.append(K, V, KV, sc, i32(slots), i32(cu), page)
    ds.kv8_append(K, V, KV, sc, i32(slots), i32(cu), most)
    same_cache((KV, sc), want)
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
def test_calls_on_two_streams_at_once(dtype):
    """Dense and sparse calls that overlap, each with a workspace of its own."""
    lens, page = [3000, 500], 16
    KV, sc, table = setup(91, lens, 2, page, dtype)
    Q, idx = queries(92, 2, 16), lists(93, lens, 2, 400)
    O, lse = run_dense(Q, KV, sc, table, i32(lens))
    O2, lse2 = outputs(2, 16)
    ds.kv8_group_sparse_decode(Q, KV, sc, table, i32(lens), idx, O2, SCALE, lse=lse2)
    n = i32(lens)
    ws = [ds.kv8_workspace(Q, KV) for _ in range(2)]
    out = [outputs(2, 16) for _ in range(40)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(out):
        with torch.cuda.stream(streams[k % 2]):
            if k % 2 == 0:
                ds.kv8_decode(Q, KV, sc, table, n, o, SCALE, lse=l, ws=ws[0])
            else:
                ds.kv8_group_sparse_decode(Q, KV, sc, table, n, idx, o, SCALE, lse=l, ws=ws[1])
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(out):
        assert torch.equal(o, O2 if k % 2 else O) and torch.equal(l, lse2 if k % 2 else lse)


def test_workspace_is_left_clear():
    """A call leaves the counters of a workspace at zero, whatever it merged."""
    KV, sc, table = setup(95, [2500, 40], 2, 16, torch.int8)
    Q = queries(96, 2, 4)
    ws = ds.kv8_workspace(Q, KV)
    O, lse = run_dense(Q, KV, sc, table, i32([2500, 40]), ws=ws)
    assert (ws[:1024] == 0).all()
    O2, _ = run_dense(Q, KV, sc, table, i32([40, 39]), ws=ws)
    O3, lse3 = run_dense(Q, KV, sc, table, i32([2500, 40]), ws=ws)
    assert torch.equal(O, O3) and torch.equal(lse, lse3) and (ws[:1024] == 0).all()


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("k", [20, 5000])
def test_nothing_listed_whatever_the_query(dtype, shared, k):
    """Infinities and NaN in Q: lists with nothing in them still give 0 and -inf, and heads beside
    them in a group what they give alone.  Over tokens such a head's logits have no softmax: NaN."""
    ds.device_status()
    lens, page, Hq, Hkv = [6000, 0], 16, 8, 2
    KV, sc, table = setup(101, lens, Hkv, page, dtype)
    Q = queries(102, 2, Hq)
    odd = {1: math.nan, 2: math.inf, 5: math.nan, 6: -math.inf}
    for h, v in odd.items():
        Q[0, h, 17] = v
    Q[1] = math.inf
    H = Hkv if shared else Hq
    idx = lists(103, lens, H, k).view(2, H, k)
    idx[0, :H // 2] = -1  # KV head 0
    fn = ds.kv8_group_sparse_decode if shared else ds.kv8_sparse_decode
    O, lse = outputs(2, Hq)
    fn(Q, KV, sc, table, i32(lens), idx.view(-1, k), O, SCALE, lse=lse)
    for o, l in ((O[0, :4], lse[0, :4]), (O[1], lse[1])):
        assert (o == 0).all() and (l == -math.inf).all()
    assert O[0, 5:7].isnan().all() and lse[0, 5:7].isnan().all()
    check(Q, KV, sc, table, page, lambda b, h: idx[0, h * H // Hq].tolist(), O, lse,
          heads=[(0, 4), (0, 7)])
    assert ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("n", [30, 3000])
def test_no_page_left_whatever_the_query(dtype, n):
    """Dense, every page of a sequence bad: 0 and -inf for infinite and NaN queries too."""
    ds.device_status()
    KV, sc, table = setup(105, [n, 40], 2, 16, dtype)
    table[0] = -1
    Q = queries(106, 2, 4)
    Q[0, 0, 3], Q[0, 1, 5], Q[0, 2] = math.inf, -math.inf, math.nan
    O, lse = run_dense(Q, KV, sc, table, i32([n, 40]))
    assert (O[0] == 0).all() and (lse[0] == -math.inf).all()
    check(Q, KV, sc, table, 16, lambda b, h: range(40), O, lse, heads=[(1, h) for h in range(4)])
    assert ds.device_status() == ds.DEV_BAD_PAGE


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("most", [1, 1000])
def test_append_of_slots_out_of_order(dtype, page, most):
    """Slots of a sequence that skip, go back or return inside a page, and two sequences in one
    page: what is no run of its own is refused and flagged, the rest is stored."""
    ds.device_status()
    # (page, first offset, tokens, refused) of each sequence's runs
    seqs = [[(0, 1, 2, 0)],
            [(1, 0, 5, 0), (1, 6, page - 6, 1), (2, 0, 3, 0)],   # skips one slot
            [(3, 0, 8, 0), (3, 2, 4, 1), (4, 0, 2, 0)],          # goes back
            [(5, 3, 1, 0), (5, 3, 1, 1)],                        # the same slot twice
            [(6, 0, 3, 0), (7, 5, 4, 1), (6, 7, 2, 1)],          # away and back
            [(8, 4, 2, 0)], [(8, 9, 2, 1)],                      # two sequences in a page
            [(9, 15, 1, 0), (10, 0, page, 0), (11, 0, 1, 0)],
            [(12, 0, page, 0), (12, 0, 2, 1), (13, 0, 1, 0)]]    # a page twice
    slots, kept, cu, starts = [], [], [0], []
    for runs in seqs:
        for pg, off, n, refused in runs:
            starts.append(len(slots))
            slots += [pg * page + off + i for i in range(n)]
            kept += [-1 if refused else s for s in slots[starts[-1]:]]
        cu.append(len(slots))
    K, V = new_rows(page, len(slots), 3)
    KV, sc = cache(page, 15, 3, page, dtype, spread=2.0)
    want = ref.append(K, V, KV, sc, i32(kept), i32(starts + [len(slots)]), page)
    ds.kv8_append(K, V, KV, sc, i32(slots), i32(cu), most)
    same_cache((KV, sc), want)
    assert ds.device_status() == ds.DEV_BAD_PAGE


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("most", [1, 1000])
def test_append_of_mixed_runs_in_pages_of_32(dtype, most):
    test_append_of_mixed_runs(dtype, 32, most)


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("page", [16, 64])
def test_serving_loop_codes_exactly(dtype, page):
    """Prompts, decode steps, requests that end and others that take their pages: after every
    step the codes and scales are those of the plain append, replayed on the same slots, so a
    page that changes hands is quantised anew."""
    ds.device_status()
    B, N, P = 6, 260, 30
    s = Server(B, 8, 2, page, 160 // page, P, dtype, N)
    KVr, scr = s.KV.cpu(), s.sc.cpu()
    rng, length, reused = random.Random(page), [0] * B, 0
    seen = set()
    for it in range(16):
        prompt = it % 4 == 0
        n = [rng.choice([0, 3, 17, 40]) if prompt and not l else int(l > 0) for l in length]
        done = [int(l + k > 0 and rng.random() < 0.3) for l, k in zip(length, n)]
        K, V = new_rows(200 + it, N, 2)
        s.K.copy_(K), s.V.copy_(V), s.Q.copy_(queries(it, B, 8))
        s.n_new.copy_(i32(n)), s.done.copy_(i32(done))
        s.step(max(1, max(n)))
        length = [l + k for l, k in zip(length, n)]
        assert s.lens2.tolist() == length
        taken = {x // page for x in s.slots.tolist() if x >= 0 and x % page == 0}
        reused += len(taken & seen)
        seen |= taken
        KVr, scr = ref.append(s.K, s.V, KVr, scr, s.slots, s.cu, page)
        same_cache((s.KV, s.sc), (KVr, scr))
        check(s.Q, s.KV, s.sc, s.table, page, lambda b, h: range(length[b]), s.O, s.lse)
        length = [0 if d else l for l, d in zip(length, done)]
        assert s.lens.tolist() == length
    assert reused > 0 and ds.device_status() == 0


@pytest.mark.parametrize("dtype", FORMATS)
def test_group_lists_past_32_bits(dtype):
    """Kept tokens shared by a group, in pages beyond 4 GiB of codes."""
    page, Hkv, P, n, k = 128, 2, 70000, 300, 77
    KV = torch.empty((P, Hkv, page, 2, D), dtype=torch.uint8, device="cuda").view(dtype)
    sc = torch.ones((P, Hkv, 2), device="cuda")
    assert KV.numel() > 2 ** 32
    ids = [P - 1, 3, P - 40]
    small, ssc = cache(64, 3, Hkv, page, dtype)
    KV[ids], sc[ids] = small, ssc
    Q, idx = queries(65, 1, 6), lists(66, [n], Hkv, k)
    O, lse = outputs(1, 6)
    ds.kv8_group_sparse_decode(Q, KV, sc, i32([ids]), i32([n]), idx, O, SCALE, lse=lse)
    check(Q, small, ssc, i32([[0, 1, 2]]), page, lambda b, h: idx[h // 3].tolist(), O, lse)


@pytest.mark.parametrize("shared", [False, True])
def test_selection_for_ragged_sequences(shared):
    """The selections take one length a call.  Over sequences of different lengths they run a
    sequence at a time, each into its rows of one list, and one attention call takes them all.
    One selection at the longest length ranks rows behind a shorter sequence's end too: attention
    leaves these out and flags them."""
    ds.device_status()
    Hq, Hkv, page, r, k, lens = 8, 2, 16, 16, 40, [400, 37, 0, 130, 1]
    B, N = len(lens), sum(lens)
    s = Server(B, Hq, Hkv, page, 26, 40, torch.int8, N)
    K, V = new_rows(7, N, Hkv)
    Q = queries(8, B, Hq)
    s.n_new.copy_(i32(lens))
    C = torch.stack([torch.randperm(D, generator=gen(h))[:r].sort().values
                     for h in range(Hq)]).int().cuda()
    label = torch.randn((B, Hq, max(lens), r), generator=gen(9)).bfloat16().cuda()  # stale rows
    ds.page_assign(s.lens, s.n_new, s.free, s.n_free, s.table, s.lens2, s.n_free2, s.cu, s.slots,
                   page)
    ds.kv8_append(K, V, s.KV, s.sc, s.slots, s.cu, max(lens), C=C, label=label, lens=s.lens)
    H = Hkv if shared else Hq

    def select(b, T, idx):  # sequences b.start .. b.stop - 1
        if shared:
            scores = torch.empty(((b.stop - b.start) * Hkv, T), device="cuda")
            ds.group_score_topk(Q[b], C, label[b], scores, idx, T)
        else:
            ds.score_topk(Q[b], C, label[b], idx, T)

    idx = torch.full((B, H, k), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        if n >= k:
            select(slice(b, b + 1), n, idx[b])
        else:
            idx[b, :, :n] = torch.arange(n, device="cuda")  # all of them
    fn = ds.kv8_group_sparse_decode if shared else ds.kv8_sparse_decode
    O, lse = outputs(B, Hq)
    fn(Q, s.KV, s.sc, s.table, s.lens2, idx.view(-1, k), O, SCALE, lse=lse, ws=s.ws)
    assert ds.device_status() == 0
    check(Q, s.KV, s.sc, s.table, page,
          lambda b, h: [t for t in idx[b, h * H // Hq].tolist() if t >= 0], O, lse)

    select(slice(0, B), max(lens), idx.view(-1, k))
    fn(Q, s.KV, s.sc, s.table, s.lens2, idx.view(-1, k), O, SCALE, lse=lse, ws=s.ws)
    assert ds.device_status() == ds.DEV_BAD_INDEX
    check(Q, s.KV, s.sc, s.table, page,
          lambda b, h: [t for t in idx[b, h * H // Hq].tolist() if t < lens[b]], O, lse)
