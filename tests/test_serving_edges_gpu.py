"""The serving operators at their edges: angles near zero, frequencies and values that are not finite, new lengths
under a window, calls whose input is the call before's output, and prefixes long enough for every way the work of
prefix and own keys is shared out.
"""
import math

import numpy as np
import pytest

import serving_ref as ref

torch = pytest.importorskip("torch")

from test_serving_gpu import Cache, _status, f64, fa, i32, paged_case, rand, run_paged  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("zero", [0, 1])
def test_rope_keeps_the_relative_accuracy_of_sine_and_cosine(fa, zero, interleaved):
    """Pairs one element of which is zero: the results are the other one times a sine or a cosine alone, so an error
    that is small only beside one shows.  Slow pairs at small positions have sines down to 1e-8.

    Roundings, each relative: the reduced angle to fp32 2^-23 (its fixed-point error is below 2^-50 turns), its
    multiplication by 2 pi 2^-23, sine and cosine of it 2^-22.5, mag and the product 2^-23: below 2^-20
    together, then one to bf16."""
    d, mag = 128, 1.375
    w, _ = fa.rope_freqs(d, base=500000.0, scaling="linear", factor=8.0)
    p = np.array([0, 1, -1, 2, 7, 100, -3000, 12345], dtype=np.int32)
    q = rand(101, 1, 2, len(p), d)
    first = q[..., 0::2] if interleaved else q[..., :d // 2]
    second = q[..., 1::2] if interleaved else q[..., d // 2:]
    (second if zero else first).zero_()
    for back in (False, True):
        turn = fa.rope_bwd if back else fa.rope
        y, _ = turn(q, None, w, positions=torch.from_numpy(p).cuda(), interleaved=interleaved, mag=mag)
        want, _ = ref.rotate(f64(q)[0], p, f64(w), mag, interleaved, -1.0 if back else 1.0)
        err = np.abs(f64(y)[0] - want)
        assert np.all(err <= (ref.U + 2.0 ** -20) * np.abs(want)), float((err / np.maximum(np.abs(want), 1e-30)).max())


def test_rope_angle_of_far_positions(fa):
    """The angle is off by at most |p| (2^-65 + |w| 2^-72) turns, beside fp32's roundings: offsets of 64 bits."""
    N, d = 6, 64
    w = torch.tensor([1.0, 0.37, 5e-3, 1e-6, 800.0, 0.0, -2.5, 3e-9], dtype=torch.float64).cuda()
    q = rand(103, 1, 1, N, d)
    for offset in (0, 2 ** 31, 10 ** 12, -10 ** 12, 2 ** 48, -2 ** 48):
        y, _ = fa.rope(q, None, w, offset=offset)
        want, size = ref.rotate(f64(q)[0], offset + np.arange(N), f64(w), 1.0, False)
        turns = (abs(offset) + N) * (2.0 ** -65 + np.abs(f64(w)) * 2.0 ** -72)
        slack = np.zeros(d)
        slack[:8] = slack[8:16] = 2 * math.pi * turns
        assert np.all(np.abs(f64(y)[0] - want) <= ref.U * np.abs(want) + (2.0 ** -20 + slack) * size), offset


def test_frequencies_that_are_not_finite(fa):
    """A frequency of NaN or infinity makes its pairs NaN, in the rotation and in the cache; others stay."""
    d, page, T = 64, 16, 3
    w, _ = fa.rope_freqs(d)
    bad = w.clone()
    bad[3], bad[17], bad[30] = math.nan, math.inf, -math.inf
    q, k = rand(105, 1, 2, T, d), rand(106, 1, 1, T, d)
    hit = torch.zeros(d, dtype=torch.bool, device="cuda")
    for i in (3, 17, 30):
        hit[i] = hit[i + d // 2] = True
    good, _ = fa.rope(q, None, w)
    for turn, want in ((fa.rope, good), (fa.rope_bwd, fa.rope_bwd(q, None, w)[0])):
        y, _ = turn(q, None, bad)
        assert bool(torch.isnan(y[..., hit]).all()) and torch.equal(y[..., ~hit], want[..., ~hit])
    c = Cache(107, 1, 1, d, page, T)
    tq = fa.kv_append(q, k, k, c.k, c.v, c.device_table(), i32([T]), bad)
    at = int(c.table[0, 0])
    assert bool(torch.isnan(tq[..., hit]).all()) and torch.equal(tq[..., ~hit], good[..., ~hit])
    assert bool(torch.isnan(c.k[at, :, :T][..., hit]).all()) and bool(torch.isfinite(c.k[at, :, :T][..., ~hit]).all())
    assert torch.equal(c.v[at, :, :T], k[0])


@pytest.mark.parametrize("B,H,Hk,T,n,at,prefix_len", [
    (1, 2, 1, 1, 3000, 5, 0),        # row blocks of 16, parts joined by several warps to a row
    (1, 32, 1, 1, 384, 200, 0),      # one CTA's query tile: key tiles of the other warpgroup
    (1, 32, 1, 1, 384, 300, 0),
    (2, 40, 1, 1, 6000, 700, 0),     # a query tile in the shares of many CTAs
    (2, 16, 4, 32, 1500, 40, 0),     # 1024 rows, several warps to a row
    (4, 32, 2, 80, 900, 3, 0),       # 10240 rows, four to a warp
    (2, 64, 4, 96, 1300, 700, 0),    # a pair of query tiles
    (40, 8, 2, 2, 30, 1500, 4000),   # the shared prefix's part
    (40, 8, 2, 2, 30, 4000, 4000),   # the own keys' part
])
def test_nan_in_a_value_of_vanishing_weight(fa, B, H, Hk, T, n, at, prefix_len):
    """Keys whose weight is zero in fp32 (a score 300 below the others'), one of their values NaN: 0 * NaN is NaN,
    whichever part of the row holds it, and whoever joins the parts."""
    d, page = 64, 16
    c = Cache(109, B, Hk, d, page, n, prefix_len=prefix_len)
    for b in range(B):
        c.fill(c.table[b], n, b)
    c.fill(c.prefix_pages, prefix_len, 99)
    low = (at // 128) * 128  # its key tile scores low, all others high
    for b in range(B):
        for pages, first, length in ((c.prefix_pages, 0, prefix_len), (c.table[b], prefix_len, n)):
            j = np.arange(length)
            slots = torch.from_numpy(np.asarray(pages)[j // page]).cuda().long()
            tile = (low if at < prefix_len or not prefix_len else prefix_len)
            high = (first + j < tile) | (first + j >= (tile + 128 if at < prefix_len or not prefix_len else 1 << 30))
            x = torch.from_numpy(np.where(high, 20.0, -20.0)).to(torch.bfloat16).cuda()
            c.k[slots, :, torch.from_numpy(j % page).cuda()] = x[:, None, None].expand(-1, Hk, d)
    q = torch.ones(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    good, good_l = run_paged(fa, c, q, [n] * B, None, prefix_len=prefix_len)
    assert bool(torch.isfinite(good).all())
    own = at - prefix_len if prefix_len and at >= prefix_len else at
    hits = range(B) if prefix_len and at < prefix_len else [0]
    pages = c.prefix_pages if prefix_len and at < prefix_len else c.table[0]
    c.v[int(pages[own // page]), :, own % page, 5] = math.nan
    o, lse = run_paged(fa, c, q, [n] * B, None, prefix_len=prefix_len)
    assert torch.equal(lse, good_l)
    sees = torch.ones(T, dtype=torch.bool, device="cuda")
    if not (prefix_len and at < prefix_len):  # tokens before it do not see it
        sees = torch.arange(T, device="cuda") + n - T >= own
    for b in range(B):
        if b in hits:
            assert bool(torch.isnan(o[b][:, sees, 5]).all())
            assert torch.equal(o[b][..., :5], good[b][..., :5]) and torch.equal(o[b][..., 6:], good[b][..., 6:])
        else:
            assert torch.equal(o[b], good[b])


@pytest.mark.parametrize("B,H,Hk,T,n,prefix_len", [
    (4, 8, 2, 1, 700, 0), (2, 8, 2, 20, 400, 0), (2, 16, 1, 40, 500, 0), (6, 8, 2, 1, 90, 1500), (40, 8, 1, 1, 40, 900),
])
def test_an_output_is_the_next_calls_query(fa, B, H, Hk, T, n, prefix_len):
    """Calls one after another without a pause, each reading what the one before wrote into two buffers in turn,
    and lengths that a kernel between them changes: what they give with a wait between them."""
    d, page, rounds = 64, 16, 24
    c = Cache(111, B, Hk, d, page, n, prefix_len=prefix_len)
    for b in range(B):
        c.fill(c.table[b], n, b)
    c.fill(c.prefix_pages, prefix_len, 99)
    table, pages = c.device_table(), torch.from_numpy(c.prefix_pages).cuda()
    ws = torch.empty(fa.fa_paged_workspace_bytes(B, H, Hk, T, d, prefix_len), dtype=torch.uint8, device="cuda")
    q0 = rand(112, B, H, T, d)

    def chain(wait):
        bufs, lses = [q0.clone(), torch.zeros_like(q0)], []
        lens, new = i32([n - rounds - 9 * b % 20 for b in range(B)]), i32([T] * B)
        for i in range(rounds):
            lens.add_(1)
            a, out = bufs[i % 2], bufs[1 - i % 2]
            lse = torch.empty(B, H, T, device="cuda")
            args = dict(new_lens=new, out=out, lse=lse, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            if prefix_len:
                fa.fwd_prefix(a, c.k, c.v, pages, prefix_len, table, lens, **args)
            else:
                fa.fwd_paged(a, c.k, c.v, table, lens, **args)
            if wait:
                torch.cuda.synchronize()
            lses.append(lse)
        return bufs + lses

    want = chain(True)
    for _ in range(6):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def test_windows_and_offsets_past_the_c_types(fa):
    """A window reach past 32 bits is an open one, not its low 32 bits; an offset past 64 bits is refused."""
    B, H, Hk, T, d, n = 2, 4, 2, 2, 64, 100
    c = Cache(141, B, Hk, d, 16, n)
    for b in range(B):
        c.fill(c.table[b], n, b)
    q, lens, table = rand(142, B, H, T, d), i32([n, 60]), c.device_table()
    want = fa.fwd_paged(q, c.k, c.v, table, lens)
    side = torch.cuda.current_stream()
    for left in (2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 63, 2 ** 64 + 1):
        for stream in (None, side):
            got = fa.fwd_paged(q, c.k, c.v, table, lens, window=(left, 0), stream=stream)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), left
    every = fa.fwd_paged(q, c.k, c.v, table, lens, window=(-1, -1))
    got = fa.fwd_paged(q, c.k, c.v, table, lens, window=(2 ** 33, 2 ** 32 + 1))
    assert all(torch.equal(a, b) for a, b in zip(got, every))
    w, _ = fa.rope_freqs(d)
    for bad in (2 ** 63, -2 ** 63 - 1, 2 ** 64 + 5):
        with pytest.raises(ValueError):
            fa.rope(q, None, w, offset=bad)
        with pytest.raises(ValueError):
            fa.kv_append(q, q[:, :Hk], q[:, :Hk], c.k, c.v, table, lens, w, offset=bad)
    with pytest.raises(ValueError):
        fa.fwd_paged(q, c.k, c.v, table, lens, window=(-2 ** 32, 0))


@pytest.mark.parametrize("B,H,Hk,T,d,page,lens,new,window", [
    (3, 4, 2, 5, 64, 16, [300, 40, 77], [5, 1, 0], (20, 0)),
    (3, 4, 4, 3, 128, 32, [129, 7, 64], [1, 3, 2], (0, 0)),
    (3, 4, 2, 20, 64, 16, [500, 90, 31], [20, 3, 0], (64, 0)),        # blocks of 128 rows
    (2, 8, 2, 30, 128, 64, [700, 260], [11, 30], (127, 5)),
    (3, 4, 1, 100, 64, 32, [900, 300, 130], [100, 1, 57], (30, 0)),   # blocks of 256 rows
    (3, 4, 1, 300, 128, 64, [300, 640, 1000], [300, 7, 299], (100, 0)),
    (3, 2, 1, 200, 64, 16, [400, 200, 333], [200, 64, 1], (0, 130)),
    (2, 4, 2, 40, 64, 16, [200, 64], [13, 40], (-1, 3)),
    (2, 4, 2, 40, 64, 16, [200, 20], [13, 40], (16, -1)),
])
def test_new_lens_under_a_window(fa, B, H, Hk, T, d, page, lens, new, window):
    paged_case(fa, 121, B, H, Hk, T, d, page, lens, new, window)


@pytest.mark.parametrize("T", [1, 30, 200])
def test_negative_lengths_are_empty_entries(fa, T):
    """seq_lens and new_lens below zero, as padded entries of a batch may hold."""
    paged_case(fa, 123, 4, 4, 2, T, 64, 16, [-3, 240, 0, -2 ** 31], None, (-1, 0))
    paged_case(fa, 124, 4, 4, 2, T, 64, 16, [-3, 240, 70, 230], [1, -5, -2 ** 31, T], (-1, -1))
    paged_case(fa, 125, 4, 4, 2, T, 64, 16, [-3, 240, 70, 230], [T, 1, -1, T], prefix_len=150)


@pytest.mark.parametrize("H,T,n", [(1, 1, 40), (2, 1, 3000), (32, 1, 300), (32, 1, 5000), (32, 20, 700)])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.bfloat16).min / 64])
def test_keys_of_minus_infinity_weigh_nothing(fa, H, T, n, low):
    """Scores of -inf beside finite ones, and scores near the lowest finite value, in every kernel."""
    d, page = 64, 16
    c = Cache(127, 1, 1, d, page, n)
    c.fill(c.table[0], n, 5)
    q = rand(128, 1, H, T, d).abs().clamp(min=0.01)
    for j in (0, 17, n // 2):  # every row sees them
        c.k[int(c.table[0, j // page]), :, j % page] = low
    o, lse = run_paged(fa, c, q, [n], None)
    want = ref.paged(f64(q), f64(c.k), f64(c.v), c.table, [n], [T], -1, 0, 0.125)
    ref.check_attention(f64(o), f64(lse), want)


def prefix64(q, c, lens, prefix_len, T):
    """fwd_prefix in 64 bits on the GPU: (O, LSE, sum_j p_j |v_j|)."""
    B, H, _, d = q.shape
    Hk, page = c.Hk, c.page
    G = H // Hk

    def keys(cache, pages, n, h):
        j = torch.arange(n, device="cuda")
        at = torch.from_numpy(np.asarray(pages).copy()).cuda().long()[j // page]
        return cache[at, h, j % page].double()

    o, size = (torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for h in range(Hk):
        shared = [keys(x, c.prefix_pages, prefix_len, h) for x in (c.k, c.v)]
        for b in range(B):
            n = lens[b]
            k, v = (torch.cat([s, keys(x, c.table[b], n, h)]) for s, x in zip(shared, (c.k, c.v)))
            s = q[b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
            pos = prefix_len + n - T + torch.arange(T, device="cuda")
            s = s.masked_fill(torch.arange(prefix_len + n, device="cuda") > pos[:, None], -math.inf)
            p = s.softmax(-1)
            o[b, h * G:(h + 1) * G], size[b, h * G:(h + 1) * G] = p @ v, p @ v.abs()
            lse[b, h * G:(h + 1) * G] = s.logsumexp(-1)
    return o.cpu().numpy(), lse.cpu().numpy(), size.cpu().numpy()


@pytest.mark.parametrize("B,H,Hk,T,d,page,prefix_len,most,wide,captured", [
    # rows of the whole batch in one block of 16: prefix and own keys in one launch
    (4, 8, 8, 3, 64, 16, 8000, 700, 0, False),     # the prefix on more CTAs than there are SMs
    (4, 8, 8, 3, 128, 32, 8001, 700, 0, True),
    (3, 4, 2, 2, 128, 16, 5000, 400, 0, False),    # on about half of them
    (5, 6, 2, 1, 128, 64, 900, 130, 100000, False),  # a table for contexts far longer than these
    (2, 16, 16, 8, 128, 128, 32000, 2000, 0, False),
    # a query tile of 128 rows
    (12, 16, 8, 3, 64, 16, 20000, 500, 0, True),
    (12, 16, 8, 3, 128, 64, 20001, 500, 0, False),
    (24, 8, 4, 2, 128, 32, 3000, 300, 60000, True),
    # pairs of query tiles
    (40, 32, 8, 1, 128, 64, 20000, 300, 0, True),
    (100, 16, 4, 1, 64, 16, 12001, 90, 0, False),
    (30, 32, 8, 2, 128, 128, 2500, 200, 30000, False),
    (6, 16, 2, 40, 128, 64, 9000, 400, 0, False),   # own keys on pairs of query tiles too
])
def test_long_prefixes(fa, B, H, Hk, T, d, page, prefix_len, most, wide, captured):
    """Prefixes that fill most SMs, a few of them, or all twice over, with own keys beside and behind them."""
    lens = [T + (most - T) * (7 * b % B) // max(1, B - 1) for b in range(B)]
    c = Cache(131, B, Hk, d, page, max(lens), prefix_len=prefix_len)
    for b in range(B):
        c.fill(c.table[b], lens[b], b)
    c.fill(c.prefix_pages, prefix_len, 99)
    q = rand(132, B, H, T, d)
    want = prefix64(q, c, lens, prefix_len, T)
    if wide:
        table = np.full((B, wide // page), -1, dtype=np.int32)
        table[:, :c.max_pages] = c.table
        c.table = table
    o, lse = run_paged(fa, c, q, lens, None, prefix_len=prefix_len)
    ref.check_attention(f64(o), f64(lse), want, f"{B}x{H}/{Hk} T={T} d={d} behind {prefix_len}")
    if not captured:
        return
    pages, table, device_lens, q_in = torch.from_numpy(c.prefix_pages).cuda(), c.device_table(), i32(lens), q.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fwd_prefix(q_in, c.k, c.v, pages, prefix_len, table, device_lens)
    for _ in range(3):
        graph.replay()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    q_in.copy_(rand(133, B, H, T, d))
    graph.replay()
    again, again_l = fa.fwd_prefix(q_in, c.k, c.v, pages, prefix_len, table, device_lens)
    assert torch.equal(got[0], again) and torch.equal(got[1], again_l)


@pytest.mark.parametrize("H,T,prefix_len", [(2, 3, 0), (4, 40, 0), (4, 150, 0), (2, 3, 300), (8, 20, 300)])
def test_padding_rows_may_hold_anything(fa, H, T, prefix_len):
    """NaN queries in the rows past new_lens and in an empty entry of the batch: O = 0, LSE = -inf there, and nothing
    of it reaches the rows beside them."""
    c, q, o, lse = paged_case(fa, 135, 3, H, 2, T, 64, 16, [T, 2 * T, 0], [T, 1, T], prefix_len=prefix_len)
    q = q.clone()
    q[1, :, 1:] = math.nan
    q[2] = math.inf
    got, got_l = run_paged(fa, c, q, [T, 2 * T, 0], [T, 1, T], prefix_len=prefix_len)
    assert torch.equal(got, o) and torch.equal(got_l, lse)


@pytest.mark.parametrize("B,H,Hk,T,n,prefix_len", [(16, 32, 8, 1, 300, 2000), (40, 8, 2, 2, 100, 3000), (6, 16, 4, 1, 400, 2500),
                                                  (12, 8, 2, 1, 700, 0), (3, 16, 2, 20, 500, 0)])
def test_a_wider_table_changes_nothing(fa, B, H, Hk, T, n, prefix_len):
    """A table as wide as a server's longest context, for sequences far shorter: the same shares of the work, so the
    same bits."""
    d, page = 64, 64
    c = Cache(137, B, Hk, d, page, n, prefix_len=prefix_len)
    lens = [n - 5 * b for b in range(B)]
    for b in range(B):
        c.fill(c.table[b], lens[b], b)
    c.fill(c.prefix_pages, prefix_len, 99)
    q = rand(138, B, H, T, d)
    want = run_paged(fa, c, q, lens, None, prefix_len=prefix_len)
    table = np.full((B, 2000), -1, dtype=np.int32)
    table[:, :c.max_pages] = c.table
    c.table = table
    got = run_paged(fa, c, q, lens, None, prefix_len=prefix_len)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_threads_that_share_a_stream(fa):
    """Host threads whose calls interleave on one stream (prefix, own-key and merge kernels of several calls in any
    order), each with a workspace of its own, give what they give alone."""
    import threading

    d, page = 64, 16
    work = []
    for i, (B, H, Hk, T, n, prefix_len) in enumerate([(6, 8, 2, 1, 90, 1500), (40, 8, 1, 1, 40, 2500), (3, 4, 2, 2, 800, 0),
                                                      (2, 16, 1, 30, 300, 700)]):
        c = Cache(145 + i, B, Hk, d, page, n, prefix_len=prefix_len)
        for b in range(B):
            c.fill(c.table[b], n, b)
        c.fill(c.prefix_pages, prefix_len, 99)
        q = rand(150 + i, B, H, T, d)
        work.append((c, q, [n - b % 7 for b in range(B)], prefix_len))
    want = [run_paged(fa, c, q, lens, None, prefix_len=p) for c, q, lens, p in work]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, failed, go = [[] for _ in work], [], threading.Barrier(len(work))

    def call(i):
        try:
            c, q, lens, p = work[i]
            table, pages, n = c.device_table(), torch.from_numpy(c.prefix_pages).cuda(), i32(lens)
            torch.cuda.synchronize()
            go.wait()
            for _ in range(30):
                if p:
                    got[i].append(fa.fwd_prefix(q, c.k, c.v, pages, p, table, n, stream=side))
                else:
                    got[i].append(fa.fwd_paged(q, c.k, c.v, table, n, stream=side))
            torch.cuda.synchronize()
        except Exception as e:
            failed.append(e)
            go.abort()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i, (o, lse) in enumerate(want):
        assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in got[i])
