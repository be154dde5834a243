"""The weight that cached keys gather, and eviction by it, against plain 64-bit
implementations (cache_ref); what they do not have to touch keeps its bits."""
import math

import numpy as np
import pytest

import cache_ref
import serving_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_19_gb300 as mod
    from exact_attention_19_gb300 import build

    build.build()
    mod.load()
    return mod


@pytest.fixture(autouse=True)
def _status(fa):
    fa.fa_fwd_status(None, clear=True)
    yield
    torch.cuda.synchronize()
    st, word = fa.fa_fwd_status(None, clear=True)
    assert st == 0, f"status word {word:#x}"


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


class Cache:
    """Pages of NaN, of which the sequences' tokens are filled; weights likewise."""

    def __init__(self, seed, lens, Hk, d, page, token_major=False, more_pages=0, w_layers=1):
        rng = np.random.default_rng(seed)
        self.page, self.Hk, self.d = page, Hk, d
        width = max(1, max(-(-max(n, 0) // page) for n in lens))
        self.n_pages = sum(-(-max(n, 0) // page) for n in lens) + 2 + more_pages
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), width), -9, np.int32)  # entries past a sequence's length are not read
        at = 0
        for b, n in enumerate(lens):
            for i in range(-(-max(n, 0) // page)):
                self.table[b, i] = order[at]
                at += 1
        self.free = order[at:]
        shape = (self.n_pages, page, Hk, d) if token_major else (self.n_pages, Hk, page, d)
        self.k, self.v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if token_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.w = torch.full((self.n_pages, w_layers, Hk, page), math.nan, device="cuda")[:, -1]
        for b, n in enumerate(lens):
            self.fill(self.table[b], n, seed + b)

    def fill(self, pages, n, seed):
        if n <= 0:
            return
        g = torch.Generator().manual_seed(seed)
        j = torch.arange(n)
        at, slot = torch.from_numpy(np.asarray(pages)).long()[j // self.page].cuda(), (j % self.page).cuda()
        for c in (self.k, self.v):
            c[at, :, slot] = torch.randn(n, self.Hk, self.d, generator=g).to(torch.bfloat16).cuda()
        self.w[at, :, slot] = torch.randn(n, self.Hk, generator=g).exp().cuda()

    def forget(self, b, first, last):
        """NaN in the weights of tokens [first, last): what stood there must not be read."""
        j = np.arange(max(first, 0), last)
        self.w[torch.from_numpy(self.table[b][j // self.page]).long().cuda(), :, torch.from_numpy(j % self.page).cuda()] = \
            math.nan

    def device_table(self):
        return torch.from_numpy(self.table).cuda()


def check_weights(fa, c, q, lse, lens, new, window=(-1, 0), decay=1.0, scale=None, **kw):
    """One call against the plain form; returns the weights."""
    B, H, T, d = q.shape
    before = c.w.clone()
    got = fa.kv_weights(q, lse, c.k, c.w, c.device_table(), i32(lens), scale=scale,
                        new_lens=None if new is None else i32(new), window=window, decay=decay, **kw)
    assert got is c.w
    torch.cuda.synchronize()
    want, tol, written = cache_ref.key_weights(f64(q), f64(lse), f64(c.k), f64(before), c.table, lens,
                                               [T] * B if new is None else new, *window,
                                               1.0 / math.sqrt(d) if scale is None else scale, decay)
    w = f64(c.w)
    assert torch.equal(bits(c.w.contiguous())[torch.from_numpy(~written).cuda()],
                       bits(before.contiguous())[torch.from_numpy(~written).cuda()])
    assert np.array_equal(np.isnan(w[written]), np.isnan(want[written]))
    err = np.where(written & ~np.isnan(want), np.abs(w - want), 0.0)
    assert np.all(err <= tol), f"off by {err.max():.3e}, over by {(err - tol).max():.3e}"
    return c.w


def lse_of(fa, c, q, lens, new, window=(-1, 0), scale=None):
    return fa.fwd_paged(q, c.k, c.v, c.device_table(), i32(lens), scale=scale,
                        new_lens=None if new is None else i32(new), window=window)[1]


@pytest.mark.parametrize("B,H,Hk,T,d,page,lens,new", [
    (1, 1, 1, 1, 64, 16, [1], None),
    (3, 4, 2, 1, 128, 16, [1, 17, 200], None),
    (3, 12, 12, 1, 64, 32, [130, 31, 257], None),
    (2, 16, 1, 1, 128, 64, [300, 65], None),
    (4, 8, 2, 3, 64, 16, [3, 40, 0, 129], [3, 1, 0, 2]),
    (2, 6, 3, 7, 128, 256, [700, 9], [7, 5]),
    (2, 4, 1, 40, 64, 128, [40, 300], None),
    (1, 8, 2, 300, 128, 64, [300], None),
    (2, 8, 8, 130, 64, 16, [500, 131], [130, 77]),
    (2, 10, 2, 64, 128, 32, [64, 1000], [64, 33]),
    (1, 2, 2, 6, 64, 16, [4], None),  # more new rows than tokens: the first rows' positions are negative
    (2, 5, 5, 17, 128, 16, [-3, 20], [17, 99]),
])
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.0])
def test_weights(fa, B, H, Hk, T, d, page, lens, new, decay):
    c = Cache(B + T, lens, Hk, d, page)
    q = rand(T, B, H, T, d)
    lse = lse_of(fa, c, q, lens, new)
    for b in range(B):
        m = T if new is None else min(new[b], T)
        c.forget(b, 0 if decay == 0 and m else lens[b] - m, max(0, lens[b]))
    check_weights(fa, c, q, lse, lens, new, decay=decay)


@pytest.mark.parametrize("B,H,Hk,T,d,page,lens,new", [
    (1, 48, 1, 1, 64, 16, [200], None),    # the most rows of the warp-level kernel, and one more
    (1, 49, 1, 1, 64, 16, [200], None),
    (2, 24, 2, 4, 128, 32, [300, 70], [4, 3]),
    (2, 14, 2, 7, 128, 32, [300, 70], [7, 3]),
    (1, 130, 1, 1, 128, 64, [520], None),  # more heads than a row block holds
    (4, 8, 8, 1, 128, 64, [2000, 1025, 1, 1999], None),                 # enough units for 32 keys to a warp
    (8, 8, 8, 2, 64, 128, [2048, 2047, 300, 0, 1, 2, 900, 1300], None),  # and for 64
    (5, 8, 4, 100, 64, 32, [1100, 100, 1023, 7, 500], [100, 64, 1, 7, 100]),      # many units: a CTA each
    (3, 16, 1, 130, 128, 16, [700, 131, 300], [130, 100, 129]),         # few: clusters of four
    (3, 4, 2, 140, 64, 64, [2100, 140, 1000], None),                    # of two
    (3, 8, 2, 1300, 64, 64, [4000, 3500, 3777], [1300, 1290, 1281]),    # units given out by what each cluster has to do
    (3, 8, 2, 1300, 128, 64, [4000, 3500, 1300], [1300, 5, 1]),         # too few rows for that
    (1, 8, 1, 1300, 64, 128, [4000], None),                             # the same, clusters of four
    (20, 8, 4, 1024, 64, 64, [1024 + 16 * b for b in range(20)], [1024 - 50 * b for b in range(20)]),  # many row blocks
])
def test_weights_variants(fa, B, H, Hk, T, d, page, lens, new):
    c = Cache(B + T, lens, Hk, d, page)
    q = rand(T, B, H, T, d)
    check_weights(fa, c, q, lse_of(fa, c, q, lens, new), lens, new, decay=0.5)


@pytest.mark.parametrize("T", [1, 60])
def test_weights_captured_as_the_lengths_grow(fa, T):
    """One capture, replayed at other lengths of the same cache, some of them empty, on another stream."""
    B, H, Hk, d, page, width = 3, 8, 2, 64, 16, [900, 400, 64]
    c = Cache(60, width, Hk, d, page)
    q = rand(61, B, H, T, d)
    table, lens, new = c.device_table(), i32([T, T, T]), i32([T, T, T])
    start = c.w.clone()

    def step():
        _, lse = fa.fwd_paged(q, c.k, c.v, table, lens, new_lens=new, window=(300, 0))
        fa.kv_weights(q, lse, c.k, c.w, table, lens, new_lens=new, window=(300, 0), decay=0.5)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, m in (([900, 400, 64], [T, T, T]), ([T, 0, 64], [T, 0, 1]), ([880, -3, 63], [max(1, T - 1), T, 0])):
        c.w.copy_(start)
        lens.copy_(i32(n))
        new.copy_(i32(m))
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            graph.replay()
        torch.cuda.synchronize()
        got = c.w.clone()
        c.w.copy_(start)
        step()
        torch.cuda.synchronize()
        assert torch.equal(bits(got.contiguous()), bits(c.w.contiguous()))


@pytest.mark.parametrize("B,H,Hk,T,d,page,lens", [
    (2, 4, 2, 1, 128, 16, [400, 20]), (2, 8, 2, 5, 64, 64, [300, 7]), (1, 4, 4, 200, 64, 32, [450]),
    (1, 8, 1, 150, 128, 128, [777])])
@pytest.mark.parametrize("window", [(0, 0), (37, 0), (200, 3), (-1, -1), (5, -1), (-1, 2)])
@pytest.mark.parametrize("token_major", [False, True])
def test_weights_windows(fa, B, H, Hk, T, d, page, lens, window, token_major):
    for decay in (1.0, 0.5):
        c = Cache(T, lens, Hk, d, page, token_major, w_layers=3)
        q = rand(T + 1, B, H, T, d)
        check_weights(fa, c, q, lse_of(fa, c, q, lens, None, window), lens, None, window, decay)


def test_weights_of_a_row_sum_to_one(fa):
    """All that the rows of a step give is one for each row, whatever the grouping, also over several steps."""
    B, H, Hk, d, page, lens = 2, 8, 2, 128, 16, [333, 64]
    c = Cache(5, lens, Hk, d, page)
    c.w.zero_()
    steps = 0
    for T in (64, 1, 3):
        q = rand(T, B, H, T, d)
        n = [lens[0] - 10 + steps, lens[1] - 4 + steps] if steps else [lens[0] - 10, lens[1]]
        lse = lse_of(fa, c, q, n, None)
        before = c.w.clone()
        fa.kv_weights(q, lse, c.k, c.w, c.device_table(), i32(n))
        gained = 0.0
        for b in range(B):
            j = np.arange(n[b])
            at = (torch.from_numpy(c.table[b][j // page]).long().cuda(), slice(None), torch.from_numpy(j % page).cuda())
            old = torch.where((torch.arange(n[b], device="cuda") < n[b] - T)[:, None], before[at], torch.zeros(()).cuda())
            gained = (c.w[at].double() - old.double()).sum(0)
            # each p is off by 2^-12 at most beside its row's lse, the sums far less
            assert bool(((gained - H // Hk * T).abs() <= 2.0 ** -11 * (H // Hk * T)).all())
        steps += 1


def test_weights_wide_scores_and_scale(fa):
    """Rows whose largest probability is near one, and a scale of the caller's."""
    B, H, Hk, d, page, lens = 2, 4, 2, 64, 16, [150, 80]
    for T in (1, 50):
        c = Cache(6, lens, Hk, d, page)
        q = rand(7, B, H, T, d, scale=6.0)
        check_weights(fa, c, q, lse_of(fa, c, q, lens, None, scale=0.3), lens, None, scale=0.3)


@pytest.mark.parametrize("T", [1, 2, 70])
def test_weights_of_rows_without_a_key(fa, T):
    """lse = -inf gives nothing, +inf nothing either; padding rows may hold anything, in q and in lse."""
    B, H, Hk, d, page, lens, new = 2, 4, 2, 64, 16, [90, 150], [T, max(1, T - 1)]
    c = Cache(8, lens, Hk, d, page)
    q = rand(9, B, H, T, d)
    lse = lse_of(fa, c, q, lens, new)
    lse[0, 1, 0] = -math.inf
    lse[0, 2, T - 1] = math.inf
    if T > 1:
        q[1, :, T - 1] = math.nan
        lse[1, :, T - 1] = math.nan
    check_weights(fa, c, q, lse, lens, new, decay=0.5)


@pytest.mark.parametrize("T", [1, 40])
def test_nan_keys_reach_their_own_weight_alone(fa, T):
    B, H, Hk, d, page, lens = 1, 4, 2, 128, 32, [100]
    c = Cache(10, lens, Hk, d, page)
    q = rand(11, B, H, T, d)
    lse = lse_of(fa, c, q, lens, None)
    clean = c.w.clone()
    fa.kv_weights(q, lse, c.k, clean, c.device_table(), i32(lens))
    c.k[c.table[0, 1], 1, 5, 3] = math.nan
    fa.kv_weights(q, lse, c.k, c.w, c.device_table(), i32(lens))
    assert bool(torch.isnan(c.w[c.table[0, 1], 1, 5]))
    c.w[c.table[0, 1], 1, 5] = clean[c.table[0, 1], 1, 5]
    assert torch.equal(bits(c.w.contiguous()), bits(clean.contiguous()))


@pytest.mark.parametrize("T", [1, 40])
def test_weights_bad_pages_and_lengths_are_reported(fa, T):
    B, H, Hk, d, page, lens = 2, 2, 1, 64, 16, [40, 64]
    c = Cache(12, lens, Hk, d, page)
    q = rand(13, B, H, T, d)
    lse = lse_of(fa, c, q, lens, None)
    good = c.w.clone()
    fa.kv_weights(q, lse, c.k, good, c.device_table(), i32(lens))
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = c.table.copy()
        table[0, 1] = bad
        w = c.w.clone()
        fa.kv_weights(q, lse, c.k, w, torch.from_numpy(table).cuda(), i32(lens))
        assert fa.fa_fwd_status(None, clear=True) == (12, 2)
        want = good.clone()
        want[c.table[0, 1]] = c.w[c.table[0, 1]]
        assert torch.equal(bits(w), bits(want))
    w = c.w.clone()
    fa.kv_weights(q, lse, c.k, w, c.device_table(), i32([40, 65]))
    assert fa.fa_fwd_status(None, clear=True)[0] == 12


def test_weights_repeat_and_take_another_stream(fa):
    B, H, Hk, d, page, lens = 3, 8, 2, 128, 16, [1000, 3, 517]
    for T in (1, 60):
        c = Cache(14, lens, Hk, d, page)
        q = rand(15, B, H, T, d)
        new = [T, min(T, 3), T]
        lse = lse_of(fa, c, q, lens, new)
        first = None
        for i in range(20):
            w = c.w.clone()
            torch.cuda.synchronize()
            fa.kv_weights(q, lse, c.k, w, c.device_table(), i32(lens), new_lens=i32(new), window=(400, 0), decay=0.9,
                          stream=torch.cuda.Stream() if i % 5 == 4 else None)
            torch.cuda.synchronize()
            first = w if first is None else first
            assert torch.equal(bits(w.contiguous()), bits(first.contiguous()))


def test_weights_beside_a_shared_prefix(fa):
    """The LSE of fwd_prefix: what the own keys get is what is left of each row beside the prefix."""
    B, H, Hk, d, page, lens, n = 2, 4, 2, 64, 16, [30, 55], 100
    c = Cache(16, lens + [n], Hk, d, page)
    pages = torch.from_numpy(c.table[2, :-(-n // page)].copy()).cuda()
    c.table = np.ascontiguousarray(c.table[:2])
    for T in (1, 20):
        q = rand(17, B, H, T, d)
        _, lse = fa.fwd_prefix(q, c.k, c.v, pages, n, c.device_table(), i32(lens))
        check_weights(fa, c, q, lse, lens, None)


def test_caches_past_32_bits(fa):
    """A cache of more than 2^31 elements, weights past 2^31 of their own, eviction among the last pages."""
    n_pages, page, Hk, d = 140000, 256, 1, 64
    if torch.cuda.mem_get_info()[0] < (48 << 30):
        pytest.skip("needs 48 GB")
    c = Cache(18, [700], Hk, d, page)
    small = (c.k, c.v, c.w, c.table[0].copy())
    k, v = (torch.empty(n_pages, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.empty(n_pages * 65 + 1, Hk, page, device="cuda")[::65]
    assert k.numel() > 2 ** 31 and w.stride(0) * (n_pages - 1) > 2 ** 31
    pages = [n_pages - 1, 139000, n_pages - 2]
    w = w[:n_pages]
    for i, p in enumerate(pages):
        k[p], v[p], w[p] = small[0][small[3][i]], small[1][small[3][i]], small[2][small[3][i]]
    q = rand(19, 1, 4, 1, d)
    lse = lse_of(fa, c, q, [700], None)
    fa.kv_weights(q, lse, c.k, c.w, c.device_table(), i32([700]))
    fa.kv_weights(q, lse, k, w, i32([pages]), i32([700]))
    for i, p in enumerate(pages):
        assert torch.equal(bits(w[p]), bits(c.w[small[3][i]]))
    a = fa.kv_evict(c.k, c.v, c.w, c.device_table(), i32([700]), 300, recent=50)
    b = fa.kv_evict(k, v, w, i32([pages]), i32([700]), 300, recent=50)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for i, p in enumerate(pages):
        for x, y in ((k, c.k), (v, c.v), (w, c.w)):
            assert torch.equal(bits(x[p]), bits(y[small[3][i]]))


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def check_evict(fa, c, lens, budget, recent=0, sinks=0, slack=0, fork=False, in_place_lens=False, with_shift=True, **kw):
    B, Hk, most = len(lens), c.Hk, budget + slack
    table_out = None
    if fork:
        room = -(-most // c.page)
        table_out = np.full((B, room), -5, np.int32)
        at = 0
        for b, n in enumerate(lens):
            for i in range(-(-(budget if n > most else max(n, 0)) // c.page)):
                table_out[b, i] = c.free[at]
                at += 1
    arrays = [c.k, c.v, c.w]
    raw = [bits(a.contiguous()).cpu().numpy() for a in arrays]
    want, out, kept_want = cache_ref.evict(raw, f64(c.w), c.table, lens, budget, recent, sinks, slack, table_out)
    seq_lens = i32(lens)
    shift = i32([7 * b for b in range(B)]) if with_shift else None
    got, kept = fa.kv_evict(c.k, c.v, c.w, c.device_table(), seq_lens, budget, recent=recent, sinks=sinks, slack=slack,
                            table_out=None if table_out is None else torch.from_numpy(table_out).cuda(),
                            lens_out=seq_lens if in_place_lens else None, shift=shift, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), out)
    assert np.array_equal(kept.cpu().numpy(), kept_want)
    for a, x in zip(arrays, want):
        assert np.array_equal(bits(a.contiguous()).cpu().numpy(), x)
    if with_shift:
        assert shift.tolist() == [7 * b + max(0, n) - int(o) for b, (n, o) in enumerate(zip(lens, out))]
    if in_place_lens:
        assert got is seq_lens
    else:
        assert seq_lens.tolist() == list(lens)


@pytest.mark.parametrize("Hk,d,page,lens,budget,recent,sinks,slack", [
    (1, 64, 16, [2], 1, 0, 0, 0),
    (2, 128, 16, [40, 17, 5], 16, 4, 2, 0),
    (3, 64, 32, [100, 33, 0, -2], 33, 0, 0, 0),
    (2, 64, 16, [100, 64, 81], 64, 64, 0, 0),   # the last ones alone
    (2, 64, 16, [100, 64, 70], 64, 0, 64, 5),   # the first ones alone
    (1, 128, 64, [1025, 1024, 1023], 1000, 100, 4, 24),
    (2, 128, 128, [3001, 700], 1, 0, 0, 0),
    (2, 64, 256, [5000, 4097, 4096], 4095, 17, 3, 1),
    (5, 128, 16, [2500], 2499, 10, 1, 0),
    (1, 64, 64, [9000], 1500, 1000, 500, 0),
])
@pytest.mark.parametrize("fork", [False, True])
def test_evict(fa, Hk, d, page, lens, budget, recent, sinks, slack, fork):
    c = Cache(budget, lens, Hk, d, page, more_pages=sum(-(-max(n, 0) // page) for n in lens) if fork else 0)
    check_evict(fa, c, lens, budget, recent, sinks, slack, fork)


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("kind", ["ties", "zeros", "nan", "signs", "close"])
def test_evict_ranks(fa, token_major, kind):
    """Equal weights, zeros of both signs, NaN and infinities, negative weights, and weights one step apart."""
    lens = [700, 300, 1500]
    c = Cache(31, lens, 2, 64, 16, token_major, w_layers=2)
    g = torch.Generator().manual_seed(32)
    shape = c.w.shape
    w = torch.randn(shape, generator=g)
    if kind == "ties":
        w = (w * 2).round().abs()
    elif kind == "zeros":
        w = torch.where(w > 1.5, w, torch.where(torch.rand(shape, generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0)))
    elif kind == "nan":
        for v in (math.nan, math.inf, -math.inf):
            w = torch.where(torch.rand(shape, generator=g) < 0.1, torch.tensor(v), w)
    elif kind == "close":
        w = (1.0 + torch.randint(0, 40, shape, generator=g) * 2.0 ** -23)
    c.w.copy_(w)
    check_evict(fa, c, lens, 250, 20, 3, in_place_lens=True)


def test_evict_long_and_many(fa):
    """One long sequence, and more sequences and heads than fit the GPU at once."""
    c = Cache(33, [50001], 1, 64, 256)
    check_evict(fa, c, [50001], 12345, 1000, 16)
    lens = [20 + 3 * b for b in range(90)]
    c = Cache(34, lens, 8, 64, 16)
    check_evict(fa, c, lens, 100, 10, 2, with_shift=False)


@pytest.mark.parametrize("fork", [False, True])
def test_evict_weights_off_the_grid_of_four(fa, fork):
    """Weights whose pages begin on no 16-byte boundary."""
    lens = [300, 77]
    c = Cache(62, lens, 2, 64, 16, more_pages=24)
    flat = torch.full((c.n_pages * 2 * 19 + 1,), math.nan, device="cuda")
    w = flat[1:].view(c.n_pages, 2, 19)[..., :16]
    w.copy_(c.w)
    c.w = w
    check_evict(fa, c, lens, 60, 7, 1, fork=fork)
    q = rand(63, 2, 4, 1, 64)
    n = [60, 60]
    if not fork:
        check_weights(fa, c, q, lse_of(fa, c, q, n, None), n, None, decay=0.5)
    assert bool(torch.isnan(flat[0])) and bool(torch.isnan(flat[1:].view(c.n_pages, 2, 19)[..., 16:]).all())


@pytest.mark.parametrize("fork", [False, True])
def test_evict_ties_over_windows(fa, fork):
    """More weights than a CTA holds at once, nearly all of them equal: the lower slots stay; many CTAs to a head's rows."""
    lens = [50200, 49153]
    c = Cache(64, lens, 1, 128, 256, more_pages=400 if fork else 0)
    c.w.copy_((torch.rand(c.w.shape, generator=torch.Generator().manual_seed(65)) < 0.02).float())
    check_evict(fa, c, lens, 40000, 100, 5, fork=fork)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("fork", [False, True])
def test_evict_long_beside_many_short(fa, fork, ties):
    """Too many heads for several CTAs each, and one with more weights than a CTA holds at once."""
    lens = [50001] + [20 + b for b in range(80)]
    c = Cache(68, lens, 1, 64, 256, more_pages=120 if fork else 0)
    if ties:
        c.w.copy_((torch.rand(c.w.shape, generator=torch.Generator().manual_seed(69)) < 0.02).float())
    check_evict(fa, c, lens, 9000, 100, 5, fork=fork)


@pytest.mark.parametrize("kind,budget,recent,sinks", [
    ("random", 9000, 500, 7), ("random", 1, 0, 0), ("random", 600, 500, 100), ("random", 32000, 0, 300), ("ties", 9000, 31, 40),
    ("digit 0", 16000, 0, 0), ("digit 1", 16000, 0, 0), ("digit 2", 16000, 0, 0), ("digit 2", 15999, 0, 0), ("equal", 20000, 3, 2),
    ("nan", 12000, 100, 0)])
@pytest.mark.parametrize("fork", [False, True])
def test_evict_in_parts(fa, kind, budget, recent, sinks, fork):
    """Few heads of many weights, whose selection several CTAs share: the search ends at every digit, and beside a sequence
    that keeps all its tokens; the other head's weights are random ones."""
    lens, page = [32000, min(budget, 300), 40003], 64
    c = Cache(budget + recent, lens, 2, 64, page, more_pages=3 * (-(-budget // page)) + 20 if fork else 0)
    g = torch.Generator().manual_seed(66)
    j = torch.arange(lens[0])
    w = {"random": torch.randn(lens[0], generator=g).exp(), "ties": torch.randint(0, 9, (lens[0],), generator=g).float(),
         "digit 0": 2.0 ** (j % 4), "digit 1": 1 + (j % 4) * 2.0 ** -12, "digit 2": 1 + (j % 4) * 2.0 ** -22,
         "equal": torch.ones(lens[0]),
         "nan": torch.where(torch.rand(lens[0], generator=g) < 0.5, torch.tensor(math.nan), torch.tensor(-1.0))}[kind]
    pages = torch.from_numpy(c.table[0]).long()[j // page]
    c.w[pages.cuda(), 1, (j % page).cuda()] = w.cuda()
    check_evict(fa, c, lens, budget, recent, sinks, fork=fork)


def test_evict_in_parts_bad_pages_unaligned_and_captured(fa):
    lens, page = [33000, 700], 128
    c = Cache(67, lens, 1, 64, page)
    flat = torch.full((c.n_pages * 131 + 1,), math.nan, device="cuda")
    w = flat[1:].view(c.n_pages, 1, 131)[..., :page]
    w.copy_(c.w)
    c.w = w
    first = [a.clone() for a in (c.k, c.v, c.w)]
    check_evict(fa, c, lens, 600, 50, 3)
    want = [bits(a.contiguous()).clone() for a in (c.k, c.v, c.w)]
    table, n, out = c.device_table(), i32(lens), i32([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv_evict(c.k, c.v, c.w, table, n, 600, recent=50, sinks=3, lens_out=out)
    for _ in range(3):
        for a, f in zip((c.k, c.v, c.w), first):
            a.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a.contiguous()), x) for a, x in zip((c.k, c.v, c.w), want))
        assert out.tolist() == [600, 600]
    fa.fa_fwd_status(None, clear=True)
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        for a, f in zip((c.k, c.v, c.w), first):
            a.copy_(f)
        t = c.table.copy()
        t[0, 3] = bad
        _, kept = fa.kv_evict(c.k, c.v, c.w, torch.from_numpy(t).cuda(), n, 600, recent=50, sinks=3)
        assert fa.fa_fwd_status(None, clear=True) == (12, 2)
        k = kept[0, 0].cpu().numpy()
        assert np.all((k >= 0) & (k < lens[0])) and np.all(np.diff(k) > 0)
        for p in c.table[1]:
            assert all(torch.equal(bits(a[p]), x[p]) for a, x in zip((c.k, c.v, c.w), want) if p >= 0)


def test_evict_repeats_and_takes_buffers(fa):
    lens = [400, 90]
    first = None
    for i in range(4):
        c = Cache(35, lens, 2, 128, 16)
        kw = {}
        if i == 1:
            kw = dict(workspace=torch.full((fa.fa_evict_workspace_bytes(2, 2),), 255, dtype=torch.uint8, device="cuda"),
                      kept=torch.full((2, 2, 100), 77, dtype=torch.int32, device="cuda"))
        if i == 2:
            kw = dict(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        out = fa.kv_evict(c.k, c.v, c.w, c.device_table(), i32(lens), 100, recent=8, **kw)
        torch.cuda.synchronize()
        if i == 1:
            assert out[1] is kw["kept"]
        now = [*out, bits(c.k), bits(c.v), bits(c.w.contiguous())]
        first = now if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_evict_bad_pages_and_lengths_are_reported(fa):
    """No access outside the cache: the tokens of a bad page stay behind, the other sequence is as ever."""
    lens = [60, 64]
    good = Cache(36, lens, 2, 64, 16)
    fa.kv_evict(good.k, good.v, good.w, good.device_table(), i32(lens), 20)
    for bad in (-1, good.n_pages, 2 ** 31 - 1, -2 ** 31):
        c = Cache(36, lens, 2, 64, 16)
        table = c.table.copy()
        table[0, 1] = bad
        out, kept = fa.kv_evict(c.k, c.v, c.w, torch.from_numpy(table).cuda(), i32(lens), 20)
        assert fa.fa_fwd_status(None, clear=True) == (12, 2)
        assert out.tolist() == [20, 20]
        k = kept[0].cpu().numpy()
        assert np.all((k >= 0) & (k < 60)) and np.all(np.diff(k, axis=-1) > 0)
        for p in c.table[1]:
            assert all(torch.equal(bits(a[p]), bits(b[p])) for a, b in ((c.k, good.k), (c.v, good.v), (c.w, good.w)))
    c = Cache(36, lens, 2, 64, 16)
    out, _ = fa.kv_evict(c.k, c.v, c.w, c.device_table(), i32([60, 10 ** 6]), 20)
    assert fa.fa_fwd_status(None, clear=True)[0] == 12 and out.tolist() == [20, 20]
    c = Cache(36, lens, 2, 64, 16, more_pages=8)
    k0 = c.k.clone()
    fa.kv_evict(c.k, c.v, c.w, c.device_table(), i32(lens), 20, table_out=i32([[c.n_pages, -1], [2 ** 31 - 1, -7]]))
    assert fa.fa_fwd_status(None, clear=True)[0] == 12
    assert torch.equal(bits(c.k), bits(k0))


def test_evict_out_of_shared_pages(fa):
    """Two continuations of one cache: its pages are read by both and stay as they are."""
    c = Cache(37, [200], 2, 64, 16, more_pages=10)
    before = [bits(a.contiguous()).clone() for a in (c.k, c.v, c.w)]
    c.table = np.concatenate([c.table, c.table])
    to = c.free[:10].reshape(2, 5)
    out, kept = fa.kv_evict(c.k, c.v, c.w, c.device_table(), i32([200, 150]), 70, recent=10,
                            table_out=torch.from_numpy(to.copy()).cuda())
    assert out.tolist() == [70, 70]
    rest = torch.ones(c.n_pages, dtype=torch.bool)
    rest[torch.from_numpy(to.copy()).long().flatten()] = False
    for a, b in zip((c.k, c.v, c.w), before):
        assert torch.equal(bits(a.contiguous())[rest.cuda()], b[rest.cuda()])
    for b, n in enumerate((200, 150)):
        for h in range(2):
            w = np.concatenate([f64(c.w)[p, h] for p in c.table[b]])[:n]
            stay = cache_ref.kept_slots(w, n, 70, 10, 0)
            assert kept[b, h].tolist() == stay.tolist()
            for a in (c.k, c.v):
                got = torch.cat([a[p, h] for p in to[b]])[:70]
                assert torch.equal(got, torch.cat([a[p, h] for p in c.table[b]])[stay])


def test_refusals(fa):
    c = Cache(38, [40, 30], 2, 64, 16)
    t, lens = c.device_table(), i32([40, 30])
    q = rand(39, 2, 4, 1, 64)
    lse = torch.zeros(2, 4, 1, device="cuda")
    before = [bits(a.contiguous()).clone() for a in (c.k, c.v, c.w)]
    for args, kw, kind in (
            ((q, lse.double(), c.k, c.w, t, lens), {}, TypeError), ((q, lse[:, :3], c.k, c.w, t, lens), {}, ValueError),
            ((q, lse, c.k, c.w[..., :8], t, lens), {}, ValueError), ((q, lse, c.k, c.w.half(), t, lens), {}, TypeError),
            ((q[:, :3], lse[:, :3].contiguous(), c.k, c.w, t, lens), {}, ValueError),
            ((q, lse, c.k, c.w.transpose(0, 1).contiguous().transpose(0, 1).repeat_interleave(2, 2)[..., ::2], t, lens), {},
             ValueError),
            ((q, lse, c.k, c.w, t, lens), dict(decay=-1.0), fa.FaError), ((q, lse, c.k, c.w, t, lens), dict(scale=0.0), fa.FaError),
            ((q, lse, c.k, c.w, t[:1], lens), {}, ValueError), ((q, lse, c.k, c.w, t, lens), dict(window=(-3, 0)), fa.FaError)):
        with pytest.raises(kind):
            fa.kv_weights(*args, **kw)
    for kw, kind in ((dict(budget=0), ValueError), (dict(budget=5, recent=3, sinks=3), ValueError),
                     (dict(budget=20, table_out=t[:, :1].contiguous()), ValueError),
                     (dict(budget=20, table_out=t.long()), TypeError), (dict(budget=20, lens_out=lens[:1]), ValueError),
                     (dict(budget=20, shift=lens.float()), TypeError),
                     (dict(budget=20, kept=torch.empty(2, 2, 19, dtype=torch.int32, device="cuda")), ValueError),
                     (dict(budget=20, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), fa.FaError)):
        with pytest.raises(kind):
            fa.kv_evict(c.k, c.v, c.w, t, lens, **kw)
    torch.cuda.synchronize()
    for a, b in zip((c.k, c.v, c.w), before):
        assert torch.equal(bits(a.contiguous()), b)
    e = q[:, :, :0]
    assert fa.kv_weights(e, lse[:, :, :0], c.k, c.w, t, lens) is c.w


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("d,H,Hk,page", [(64, 4, 4, 16), (128, 8, 2, 32)])
def test_generation_in_a_bounded_cache(fa, d, H, Hk, page, captured):
    """A prompt, then single tokens: normed and turned into the cache at their true positions, attended, weighed and
    evicted every step, against the same in 64 bits that follows the kept lists; every step's list is the heaviest."""
    B, N, budget, recent, slack, eps = 2, 150, 48, 8, 5, 1e-6
    lens0 = [100, 70]
    w, mag = fa.rope_freqs(d)
    wq = (1.0 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(40))).to(torch.bfloat16).cuda()
    q, k, v = rand(41, B, H, N, d), rand(42, B, Hk, N, d), rand(43, B, Hk, N, d)
    c = Cache(44, [128] * B, Hk, d, page)
    for t in (c.k, c.v, c.w):
        t.fill_(math.nan)
    table, lens, shift, new = c.device_table(), i32(lens0), i32([0, 0]), i32(lens0)
    one = [torch.empty(B, h, 1, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk)]

    def step(x, m):
        y = fa.kv_append(*x, c.k, c.v, table, lens, w, new_lens=m, eps=eps, q_weight=wq, k_weight=wq, shift=shift)
        o, lse = fa.fwd_paged(y, c.k, c.v, table, lens, new_lens=m)
        fa.kv_weights(y, lse, c.k, c.w, table, lens, new_lens=m, decay=0.9)
        was = c.w.clone()
        out, kept = fa.kv_evict(c.k, c.v, c.w, table, lens, budget, recent=recent, sinks=2, slack=slack, lens_out=lens,
                                shift=shift)
        return o, was, kept

    def simulate(state, b, h, first, count):
        """Keys and values of head h that sequence b holds, after `count` tokens from `first` came."""
        p = np.arange(first, first + count)
        n = f64(k[b, h, first:first + count])
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps) * f64(wq)
        y, _ = ref.rotate(n, p, f64(w), 1.0, False)
        return np.concatenate([state[0], y]), np.concatenate([state[1], f64(v[b, h, first:first + count])])

    held = {(b, h): (np.zeros((0, d)), np.zeros((0, d))) for b in range(B) for h in range(Hk)}
    vmax = float(v.float().abs().max())
    graph, pos = None, list(lens0)
    for i in range(30):
        if i == 0:
            T = max(lens0)
            o, was, kept = step([q[:, :, :T].contiguous(), k[:, :, :T], v[:, :, :T]], new)
            counts = lens0
        else:
            lens += 1
            for dst, src in zip(one, (q, k, v)):
                for b in range(B):
                    dst[b, :, 0] = src[b, :, pos[b]]
            if not captured or i < 2:
                o, was, kept = step(one, None)
            else:
                if graph is None:
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        result = step(one, None)
                graph.replay()
                o, was, kept = result
            counts = [1] * B
            for b in range(B):
                pos[b] += 1
        torch.cuda.synchronize()
        weights = f64(was)
        for b in range(B):
            for h in range(Hk):
                ks, vs = held[b, h] = simulate(held[b, h], b, h, pos[b] - counts[b], counts[b])
                for g in range(h * (H // Hk), (h + 1) * (H // Hk)):
                    n = f64(q[b, g, pos[b] - 1:pos[b]])
                    n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps) * f64(wq)
                    y, _ = ref.rotate(n, [pos[b] - 1], f64(w), 1.0, False)
                    s = ks @ y[0] / math.sqrt(d)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    # bf16 q, k (their roundings move a score by up to 2^-8 of its terms), P and O
                    terms = (np.abs(ks) @ np.abs(y[0])).max() / math.sqrt(d)
                    err = np.abs(f64(o[b, g, counts[b] - 1]) - p @ vs)
                    assert np.all(err <= (4 * ref.U + 4 * ref.U * terms) * vmax)
                n = len(ks)
                row = kept[b, h].cpu().numpy()
                flat = np.concatenate([weights[pg, h] for pg in c.table[b]])[:n]
                if n > budget + slack:
                    stay = cache_ref.kept_slots(flat, n, budget, recent, 2)
                    assert row.tolist() == stay.tolist() + [-1] * slack
                    held[b, h] = (ks[stay], vs[stay])
                else:
                    assert row[:n].tolist() == list(range(n))
        assert lens.tolist() == [len(held[b, 0][0]) for b in range(B)]
        assert shift.tolist() == [pos[b] - len(held[b, 0][0]) for b in range(B)]
    assert max(lens.tolist()) <= budget + slack


def test_captures_share_no_workspace(fa):
    """Two captured evictions, each with what it allocated in its own capture, replayed at once on two streams."""
    made = []
    for seed in (50, 51):
        c = Cache(seed, [300, 200], 2, 64, 16)
        table, lens, out = c.device_table(), i32([300, 200]), i32([0, 0])
        first = [a.clone() for a in (c.k, c.v, c.w)]
        fa.kv_evict(c.k, c.v, c.w, table, lens, 100, recent=9, lens_out=out)
        torch.cuda.synchronize()
        want = [bits(a.contiguous()).clone() for a in (c.k, c.v, c.w)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.kv_evict(c.k, c.v, c.w, table, lens, 100, recent=9, lens_out=out)
        made.append((c, first, want, graph, torch.cuda.Stream(), (table, lens, out)))
    for _ in range(3):
        for c, first, _, _, _, _ in made:
            for a, f in zip((c.k, c.v, c.w), first):
                a.copy_(f)
        torch.cuda.synchronize()
        for _, _, _, graph, stream, _ in made:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for c, _, want, _, _, _ in made:
            assert all(torch.equal(bits(a.contiguous()), x) for a, x in zip((c.k, c.v, c.w), want))
