"""Rotary positions, the paged cache's append, attention over the paged cache and
shared-prefix attention, against plain 64-bit implementations (serving_ref).

Caches start as NaN everywhere, so a slot that a row must not see shows up in its
output, and a slot that the append must not touch keeps its NaN's bits.
"""
import math

import numpy as np
import pytest

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


def rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------
def packed(seed, B, N, H, Hk, d):
    """Views [B, heads, N, d] of a packed token-major projection."""
    x = rand(seed, B, N, (H + 2 * Hk) * d)
    cut = [x[..., a * d:b * d].unflatten(-1, (b - a, d)).transpose(1, 2)
           for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk))]
    return x, cut


def check_rope(got, x, positions, w, mag, interleaved, sign=1.0, what=""):
    x, got, w = f64(x), f64(got), f64(w)
    for b in range(x.shape[0]):
        p = positions[b] if positions.ndim == 2 else positions
        y, size = ref.rotate(x[b], p, w, mag, interleaved, sign)
        err = np.abs(got[b] - y)
        assert np.all(err <= ref.rope_tol(y, size)), f"{what}: sequence {b} off by {err.max():.3e}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hk,N,d,rot", [
    (1, 1, 1, 1, 64, 64), (2, 3, 1, 33, 64, 16), (1, 4, 4, 65, 64, 48), (3, 12, 12, 7, 64, 64),
    (1, 8, 2, 31, 128, 128), (2, 5, 5, 129, 128, 64), (1, 2, 1, 300, 128, 112), (2, 32, 8, 40, 128, 32),
])
@pytest.mark.parametrize("strided", [False, True])
def test_rope(fa, B, H, Hk, N, d, rot, interleaved, strided):
    if strided:
        _, (q, k, _) = packed(N, B, N, H, Hk, d)
    else:
        q, k = rand(N, B, H, N, d), rand(N + 1, B, Hk, N, d)
    w, mag = fa.rope_freqs(rot)
    assert mag == 1.0
    yq, yk = fa.rope(q, k, w, interleaved=interleaved)
    assert yq.is_contiguous() and yk.is_contiguous()
    for y, x in ((yq, q), (yk, k)):
        check_rope(y, x, np.arange(N), w, 1.0, interleaved)
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("base", 8.0), ("by_parts", 32.0)])
def test_rope_far_positions(fa, scaling, factor):
    """Any 32-bit position, negative ones too, and a large offset: the angle stays exact."""
    N, d = 9, 128
    q = rand(3, 2, 2, N, d)
    w, mag = fa.rope_freqs(d, base=500000.0, scaling=scaling, factor=factor)
    p = np.array([[0, 1, 65535, 100000, 999999, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31],
                  [5, 4, 3, 2, 1, 0, 7, 7, 123456789]], dtype=np.int32)
    y, none = fa.rope(q, None, w, positions=torch.from_numpy(p).cuda(), mag=mag)
    assert none is None
    check_rope(y, q, p, w, mag, False)
    y, _ = fa.rope(q, None, w, positions=torch.from_numpy(p[0]).cuda(), offset=10 ** 12, interleaved=True)
    check_rope(y, q, p[0].astype(np.int64) + 10 ** 12, w, 1.0, True)


def test_rope_frequency_forms(fa):
    """Zero, negative, tiny and above-one-turn frequencies."""
    w = torch.tensor([0.0, -0.25, 1e-300, 2.0 ** -70, 7.0, 1e6, 3.5e9, 1.0], dtype=torch.float64).cuda()
    q = rand(8, 1, 1, 5, 64)
    y, _ = fa.rope(q, None, w, offset=3)
    check_rope(y, q, np.arange(5) + 3, w, 1.0, False)


def test_rope_in_place_and_strided_outputs(fa):
    B, N, H, Hk, d = 2, 37, 4, 2, 64
    w, _ = fa.rope_freqs(32)
    x, (q, k, v) = packed(5, B, N, H, Hk, d)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    oq, ok = fa.rope(q, k, w, q_out=q, k_out=k)
    assert oq is q and ok is k
    check_rope(q, q0, np.arange(N), w, 1.0, False)
    check_rope(k, k0, np.arange(N), w, 1.0, False)
    assert torch.equal(v, v0)  # the packed neighbour is untouched


def test_an_error_left_behind_is_not_this_calls(fa):
    """A runtime call that failed earlier in the process leaves its error to be read: the calls here go by their own
    launches, so nothing is reported, run again or, in place, turned twice."""
    import ctypes

    runtime = ctypes.CDLL("libcudart.so.13")
    q = rand(64, 1, 2, 40, 64)
    w, _ = fa.rope_freqs(64)
    want, _ = fa.rope(q, None, w)
    c = Cache(65, 1, 2, 64, 16, 64)
    table, lens, k = c.device_table(), i32([40]), rand(66, 1, 2, 40, 64)
    fa.kv_append(None, k, k, c.k, c.v, table, lens, w)
    want_o, _ = fa.fwd_paged(want, c.k, c.v, table, lens)
    a, b = q.clone(), q.clone()
    torch.cuda.synchronize()
    try:
        def left():
            runtime.cudaSetDevice(1 << 20)  # no such device
            assert runtime.cudaPeekAtLastError() != 0

        left()
        fa.rope(a, None, w, q_out=a)
        left()
        fa.kv_append(b, k, k, c.k, c.v, table, lens, w, q_out=b)
        o, lse = torch.empty_like(q), torch.empty(1, 2, 40, dtype=torch.float32, device="cuda")
        left()
        fa.fwd_paged(want, c.k, c.v, table, lens, out=o, lse=lse)
    finally:
        runtime.cudaGetLastError()
    assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(o, want_o)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 48)])
def test_rope_backward(fa, d, rot, interleaved):
    """The formula's transpose, and differences: for the linear map R the derivative of <g, R x> along e is
    (<g, R e> - <g, R(-e)>) / 2."""
    B, H, Hk, N, mag = 2, 3, 1, 21, 1.25
    w, _ = fa.rope_freqs(rot)
    gq, gk = rand(1, B, H, N, d), rand(2, B, Hk, N, d)
    dx = torch.zeros(B, N, (H + Hk) * d, device="cuda", dtype=torch.bfloat16)
    oq = dx[..., :H * d].unflatten(-1, (H, d)).transpose(1, 2)
    ok = dx[..., H * d:].unflatten(-1, (Hk, d)).transpose(1, 2)
    dq, dk = fa.rope_bwd(gq, gk, w, offset=50, interleaved=interleaved, mag=mag, q_out=oq, k_out=ok)
    for got, g in ((dq, gq), (dk, gk)):
        check_rope(got, g, np.arange(N) + 50, w, mag, interleaved, -1.0)
    for e in (0, 1, rot // 2, rot - 1, d - 1):
        x = torch.zeros_like(gq)
        x[..., e] = 1.0
        up, _ = fa.rope(x, None, w, offset=50, interleaved=interleaved, mag=mag)
        down, _ = fa.rope(-x, None, w, offset=50, interleaved=interleaved, mag=mag)
        terms = f64(gq) * (f64(up) - f64(down)) / 2
        diff = terms.sum(-1)
        # each of the two terms of R e is rounded to bf16 once, the gradient once
        tol = ref.U * (np.abs(terms).sum(-1) + np.abs(diff)) + 2.0 ** -18 * mag * np.abs(f64(gq)).max()
        assert np.all(np.abs(f64(dq)[..., e] - diff) <= tol)


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------
class Cache:
    """A cache whose pages lie in random order; unused slots hold NaN."""

    def __init__(self, seed, B, Hk, d, page, max_len, token_major=False, prefix_len=0):
        self.page, self.d, self.Hk = page, d, Hk
        rng = np.random.default_rng(seed)
        self.max_pages = max(1, -(-max_len // page))
        n_prefix = -(-prefix_len // page)
        n_pages = B * self.max_pages + n_prefix + 2
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = order[:B * self.max_pages].reshape(B, self.max_pages).copy()
        self.prefix_pages = order[B * self.max_pages:B * self.max_pages + n_prefix].copy()
        shape = (n_pages, page, Hk, d) if token_major else (n_pages, Hk, page, d)
        self.k = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        self.v = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        if token_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.seed = seed

    def fill(self, pages, n, seed):
        """Random K and V for tokens 0..n-1 of a page list."""
        if n <= 0:
            return
        g = torch.Generator().manual_seed(seed)
        for c in (self.k, self.v):
            x = torch.randn(n, self.Hk, self.d, generator=g).to(torch.bfloat16).cuda()
            j = torch.arange(n, device="cuda")
            at = torch.from_numpy(np.asarray(pages)).cuda().long()[j // self.page]
            c[at, :, j % self.page] = x

    def device_table(self):
        return torch.from_numpy(self.table).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("B,H,Hk,T,d,page,rot,lens,new,token_major,interleaved", [
    (1, 1, 1, 1, 64, 16, 64, [1], None, False, False),
    (3, 4, 2, 1, 128, 16, 128, [1, 17, 40], None, False, True),
    (3, 4, 4, 5, 64, 32, 32, [5, 33, 64], None, True, False),
    (4, 8, 1, 7, 128, 64, 64, [7, 3, 0, 70], [7, 2, 0, 1], False, False),
    (2, 2, 2, 100, 64, 128, 64, [100, 130], [100, 63], True, True),
    (2, 6, 3, 300, 128, 256, 0, [300, 512], [300, 299], False, False),
    (2, 0, 2, 4, 64, 16, 16, [4, 9], None, False, False),
    (3, 2, 1, 6, 64, 16, 64, [3, -4, 20], [6, 6, 9], False, False),  # lengths below the new rows, new past T
])
def test_append(fa, B, H, Hk, T, d, page, rot, lens, new, token_major, interleaved):
    c = Cache(B * T, B, Hk, d, page, max(max(lens), 1) + page, token_major)
    _, (q, k, v) = packed(T, B, T, H, Hk, d)
    k0, v0 = c.k.clone(), c.v.clone()
    w, mag = (fa.rope_freqs(rot, scaling="by_parts", factor=4.0) if rot else (None, 1.0))
    q_out = torch.full((B, H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = fa.kv_append(q if H else None, k, v, c.k, c.v, c.device_table(), i32(lens), w, offset=1000,
                       new_lens=None if new is None else i32(new), interleaved=interleaved, mag=mag,
                       q_out=q_out if H else None)
    assert out is (q_out if H else None)
    written = torch.zeros(k0.shape[0], page, dtype=torch.bool)
    for b in range(B):
        m = min(T, new[b]) if new is not None else T
        for t in range(T):
            own = lens[b] - m + t
            if t >= m or own < 0:
                if H:
                    assert torch.all(q_out[b, :, t] == 7.0)
                continue
            at, slot = int(c.table[b, own // page]), own % page
            written[at, slot] = True
            assert torch.equal(c.v[at, :, slot], v[b, :, t])
            pairs = [(c.k[at, :, slot], k[b, :, t])] + ([(q_out[b, :, t], q[b, :, t])] if H else [])
            for got, x in pairs:
                if not rot:
                    assert torch.equal(got, x)
                    continue
                y, size = ref.rotate(f64(x)[:, None], [own + 1000], f64(w), mag, interleaved)
                assert np.all(np.abs(f64(got)[:, None] - y) <= ref.rope_tol(y, size))
    keep = ~written[:, None, :, None].expand(k0.shape).cuda()
    for now, before in ((c.k, k0), (c.v, v0)):
        assert torch.equal(now.contiguous().view(torch.int16)[keep], before.contiguous().view(torch.int16)[keep])


def run_paged(fa, c, q, lens, new, window=(-1, 0), prefix_len=0, **kw):
    args = dict(new_lens=None if new is None else i32(new), **kw)
    if prefix_len:
        return fa.fwd_prefix(q, c.k, c.v, torch.from_numpy(c.prefix_pages).cuda(), prefix_len, c.device_table(),
                             i32(lens), **args)
    return fa.fwd_paged(q, c.k, c.v, c.device_table(), i32(lens), window=window, **args)


def paged_case(fa, seed, B, H, Hk, T, d, page, lens, new=None, window=(-1, 0), token_major=False, prefix_len=0,
               scale=None, q_scale=1.0):
    c = Cache(seed, B, Hk, d, page, max(max(lens), 1), token_major, prefix_len)
    for b in range(B):
        c.fill(c.table[b], lens[b], seed + b)
    c.fill(c.prefix_pages, prefix_len, seed + 99)
    q = (rand(seed + 7, B, H, T, d).float() * q_scale).to(torch.bfloat16)
    # slots wholly below every row's window may hold anything too
    if window[0] >= 0:
        for b in range(B):
            m = T if new is None else min(new[b], T)
            low = max(0, lens[b] - m - window[0])
            for j in range(min(low, lens[b])):
                c.k[int(c.table[b, j // page]), :, j % page] = math.nan
                c.v[int(c.table[b, j // page]), :, j % page] = math.inf
            c.table[b, :low // page] = -1  # their pages may have been given back
    used = np.array([-(-max(0, n) // page) for n in lens])
    c.table[np.arange(c.max_pages)[None, :] >= used[:, None]] = -5
    o, lse = run_paged(fa, c, q, lens, new, window, prefix_len, scale=scale)
    torch.cuda.synchronize()
    table = np.maximum(c.table, 0)
    want = ref.paged(f64(q), f64(c.k), f64(c.v), table, lens, [T] * B if new is None else new, window[0], window[1],
                     1 / math.sqrt(d) if scale is None else scale, c.prefix_pages, prefix_len)
    ref.check_attention(f64(o), f64(lse), want, f"{B}x{H}/{Hk} T={T} d={d} page={page} lens={lens} {window}")
    return c, q, o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hk,T,page,lens,new", [
    (1, 1, 1, 1, 16, [1], None),
    (1, 1, 1, 1, 16, [2000], None),
    (2, 2, 2, 1, 32, [63, 64], None),
    (3, 4, 2, 1, 64, [65, 0, 127], None),
    (4, 8, 1, 1, 128, [128, 129, 1, 500], None),
    (2, 16, 1, 1, 16, [333, 16], None),
    (2, 24, 1, 1, 16, [17, 200], None),              # 24 rows: two row blocks of 16
    (3, 3, 3, 5, 16, [5, 77, 256], None),
    (2, 8, 2, 7, 256, [7, 511], [7, 3]),
    (3, 4, 4, 4, 16, [9, 130, 0], [2, 4, 0]),
    (2, 10, 2, 33, 32, [33, 190], [1, 33]),
    (1, 4, 1, 130, 64, [700], None),                  # 520 rows of one K/V head
    (2, 2, 1, 70, 16, [3, 64], None),                 # shorter than the new rows: some hold no token
    (70, 2, 1, 1, 16, [i * 3 % 50 for i in range(70)], None),
    (150, 1, 1, 1, 16, [i % 7 for i in range(150)], None),
    (60, 24, 1, 1, 32, [i * 5 % 200 for i in range(60)], None),
    (250, 20, 1, 1, 16, [i * 7 % 90 for i in range(250)], None),  # several sequences to a CTA
    (3, 4, 1, 300, 64, [300, 640, 1000], [300, 7, 299]),          # blocks of rows that see part of the keys
    (1, 1, 1, 600, 256, [600], None),
    (300, 2, 1, 1, 16, [i * 11 % 61 for i in range(300)], None),  # more sequences than the merge sums itself
    (1, 2, 1, 1, 256, [20000], None),                             # one row block in the shares of every CTA
    (1, 40, 1, 1, 128, [9000], None),
    (400, 4, 4, 6, 16, [6 + i % 30 for i in range(400)], None),   # 9600 rows to merge
    (2500, 1, 1, 1, 16, [i * 13 % 47 for i in range(2500)], None),
])
def test_paged(fa, B, H, Hk, T, d, page, lens, new):
    paged_case(fa, 1 + B, B, H, Hk, T, d, page, lens, new)


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("B,H,Hk,T,d,page,lens,window", [
    (2, 4, 2, 1, 64, 16, [300, 40], (0, 0)),
    (2, 4, 2, 3, 128, 16, [300, 40], (20, 0)),
    (3, 2, 1, 4, 64, 64, [1000, 64, 5], (63, 0)),
    (2, 2, 2, 6, 64, 32, [100, 6], (10, 2)),
    (2, 2, 2, 9, 128, 16, [100, 5], (-1, -1)),        # every cached key, more rows than keys
    (2, 4, 1, 40, 64, 128, [500, 41], (64, -1)),
    (2, 2, 1, 200, 128, 32, [700, 200], (30, 0)),     # rows of different blocks see different tiles
    (1, 2, 1, 150, 64, 16, [400], (5, 70)),
    (1, 2, 1, 2, 64, 16, [50], (2 ** 31 - 1, 2 ** 31 - 1)),
])
def test_paged_windows(fa, B, H, Hk, T, d, page, lens, window, token_major):
    paged_case(fa, 11, B, H, Hk, T, d, page, lens, None, window, token_major)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hk,T,page,prefix_len,lens,new,token_major", [
    (1, 1, 1, 1, 16, 1, [1], None, False),
    (2, 2, 1, 1, 16, 100, [1, 33], None, False),
    (5, 4, 4, 1, 32, 64, [1, 2, 3, 64, 65], None, True),
    (9, 8, 2, 1, 64, 1000, [i + 1 for i in range(9)], None, False),
    (3, 6, 2, 4, 128, 129, [4, 140, 9], [4, 1, 3], False),
    (4, 2, 1, 3, 16, 77, [3, 0, 2, 50], [3, 0, 3, 2], True),   # an empty entry; a row before its sequence
    (40, 4, 1, 1, 256, 700, [1 + i * 7 % 90 for i in range(40)], None, False),
    (33, 16, 2, 2, 16, 257, [2 + i % 5 for i in range(33)], None, False),
    (3, 40, 2, 3, 16, 90, [3, 30, 70], None, False),           # 60 own rows, 180 prefix rows of a K/V head
    (2, 4, 2, 100, 32, 200, [100, 140], [100, 3], True),       # a chunk behind a prefix
])
def test_prefix(fa, d, B, H, Hk, T, page, prefix_len, lens, new, token_major):
    paged_case(fa, 21 + B, B, H, Hk, T, d, page, lens, new, (-1, 0), token_major, prefix_len)


def test_paged_wide_scores_and_scale(fa):
    """Logits spread over hundreds: the running maximum moves often, most weights vanish."""
    paged_case(fa, 31, 2, 4, 2, 3, 128, 16, [400, 77], scale=1.0, q_scale=4.0)
    paged_case(fa, 32, 2, 4, 2, 1, 64, 16, [400, 77], scale=2.0, q_scale=4.0, prefix_len=150)


def test_paged_infinite_and_lowest_values(fa):
    """Keys of the type's lowest value (finite, scores near -3e38): they weigh nothing beside others."""
    c = Cache(5, 1, 1, 64, 16, 40)
    c.fill(c.table[0], 40, 5)
    q = rand(6, 1, 1, 1, 64).abs()
    c.k[int(c.table[0, 1]), :, 3] = torch.finfo(torch.bfloat16).min / 64
    o, lse = run_paged(fa, c, q, [40], None)
    want = ref.paged(f64(q), f64(c.k), f64(c.v), c.table, [40], [1], -1, 0, 0.125)
    ref.check_attention(f64(o), f64(lse), want)


def test_paged_repeats_bit_for_bit_and_takes_buffers(fa):
    B, H, Hk, T, d = 3, 8, 2, 2, 128
    c = Cache(41, B, Hk, d, 16, 900)
    lens = [900, 3, 411]
    for b in range(B):
        c.fill(c.table[b], lens[b], b)
    q = rand(42, B, H, T, d)
    o1, l1 = run_paged(fa, c, q, lens, None)
    ws = torch.full((fa.fa_paged_workspace_bytes(B, H, Hk, T, d, 0),), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.full_like(o1, math.nan), torch.full_like(l1, math.nan)
    got = run_paged(fa, c, q, lens, None, out=o2, lse=l2, workspace=ws)
    assert got[0] is o2 and got[1] is l2
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    with pytest.raises(fa.FaError) as e:
        run_paged(fa, c, q, lens, None, workspace=ws[:1024])
    assert e.value.status == 11


@pytest.mark.parametrize("T", [1, 40])
def test_bad_pages_and_lengths_are_reported(fa, T):
    """A page index outside the cache, or a length past the table: no access outside, FA_ERR_PAGE."""
    B, H, Hk, d, page = 2, 2, 1, 64, 16
    c = Cache(51, B, Hk, d, page, 64)
    lens = [40, 64]
    for b in range(B):
        c.fill(c.table[b], lens[b], b)
    c.fill(list(range(c.k.shape[0])), c.k.shape[0] * page, 9)
    q = rand(52, B, H, T, d)
    good, _ = run_paged(fa, c, q, lens, None)
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = c.table.copy()
        c.table[0, 1] = bad
        o, lse = run_paged(fa, c, q, lens, None)
        st, word = fa.fa_fwd_status(None, clear=True)
        assert (st, word) == (12, 2)
        assert torch.equal(o[1], good[1]) and bool(torch.isfinite(o).all())
        k0 = c.k.clone()
        fa.kv_append(None, rand(1, B, Hk, 1, d), rand(2, B, Hk, 1, d), c.k, c.v, c.device_table(), i32([17, 0]))
        st, word = fa.fa_fwd_status(None, clear=True)
        assert (st, word) == (12, 2)
        assert torch.equal(c.k, k0)
        c.table = table
    o, _ = run_paged(fa, c, q, [65, 64], None)
    assert fa.fa_fwd_status(None, clear=True)[0] == 12
    assert torch.equal(o[1], good[1])
    fa.kv_append(None, rand(1, B, Hk, 1, d), rand(2, B, Hk, 1, d), c.k, c.v, c.device_table(), i32([65, 0]))
    assert fa.fa_fwd_status(None, clear=True)[0] == 12
    for bad in (-1, c.k.shape[0]):
        c.prefix_pages = np.array([0, bad], dtype=np.int32)
        o, _ = run_paged(fa, c, q, lens, None, prefix_len=20)
        assert fa.fa_fwd_status(None, clear=True)[0] == 12 and bool(torch.isfinite(o).all())


def test_nan_reaches_the_rows_that_see_it_and_no_others(fa):
    """A NaN in a visible key or value makes its sequence's rows NaN, not zero, in every kernel; others stay."""
    for H, T, lens in ((2, 1, [70, 90]), (2, 1, [3000, 2500]), (2, 20, [200, 333]), (4, 70, [500, 450])):
        for what in ("k", "v"):
            c = Cache(57, 2, 1, 64, 16, max(lens))
            for b in range(2):
                c.fill(c.table[b], lens[b], b)
            q = rand(58, 2, H, T, 64)
            good, good_l = run_paged(fa, c, q, lens, None)
            getattr(c, what)[int(c.table[0, 0]), 0, 3, 5] = math.nan  # the first tokens: every row sees them
            o, lse = run_paged(fa, c, q, lens, None)
            hit = torch.isnan(o[0])
            assert bool(hit.all() if what == "k" else hit[..., 5].all())
            if what == "k":
                assert bool(torch.isnan(lse[0]).all())
            else:
                assert torch.equal(lse[0], good_l[0])
            assert torch.equal(o[1], good[1]) and torch.equal(lse[1], good_l[1])


def test_pages_shared_between_sequences(fa):
    """Tables that name the same pages (a forked sequence) read them alike."""
    c = Cache(59, 3, 2, 128, 16, 300)
    c.fill(c.table[0], 300, 1)
    c.table[1] = c.table[0]
    c.table[2, :10] = c.table[0, :10]
    c.fill(c.table[2, 10:], 60, 2)
    q = rand(60, 1, 8, 1, 128).expand(3, -1, -1, -1).contiguous()
    lens = [300, 300, 220]
    o, lse = run_paged(fa, c, q, lens, None)
    want = ref.paged(f64(q), f64(c.k), f64(c.v), c.table, lens, [1] * 3, -1, 0, 1 / math.sqrt(128))
    ref.check_attention(f64(o), f64(lse), want)
    # the parts of a row depend on where its sequence lies in the call, so equal sequences agree to rounding
    assert float((o[0].float() - o[1].float()).abs().max()) <= 4 * ref.U * float(o.float().abs().max())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_keys_and_values_in_one_tensor(fa, T):
    """K and V as views of one allocation, [n_pages, 2, page, Hk, d] and heads outermost: other page, head and
    token strides for the same calls, to the bit."""
    B, H, Hk, d, page, lens = 2, 4, 2, 64, 32, [300, 411]
    q, k, v = rand(71, B, H, T, d), rand(72, B, Hk, T, d), rand(73, B, Hk, T, d)
    w, _ = fa.rope_freqs(d)
    base = Cache(70, B, Hk, d, page, max(lens))
    for b in range(B):
        base.fill(base.table[b], lens[b] - T, 74 + b)
    n = base.k.shape[0]
    one = torch.full((n, 2, page, Hk, d), math.nan, dtype=torch.bfloat16, device="cuda")
    heads = torch.full((2, Hk, n, page, d), math.nan, dtype=torch.bfloat16, device="cuda")
    views = [(base.k, base.v), tuple(one[:, i].transpose(1, 2) for i in range(2)),
             tuple(heads[i].transpose(0, 1) for i in range(2))]
    results = []
    keep = base.k.clone(), base.v.clone()
    for kc, vc in views:
        kc.copy_(keep[0])
        vc.copy_(keep[1])
        turned = fa.kv_append(q, k, v, kc, vc, base.device_table(), i32(lens), w)
        results.append(fa.fwd_paged(turned, kc, vc, base.device_table(), i32(lens)) + (kc.clone(), vc.clone()))
    want = ref.paged(f64(turned), f64(results[0][2]), f64(results[0][3]), base.table, lens, [T] * B, -1, 0, d ** -0.5)
    ref.check_attention(f64(results[0][0]), f64(results[0][1]), want)
    for r in results[1:]:
        assert torch.equal(r[0], results[0][0]) and torch.equal(r[1], results[0][1])
        for a, b in zip(r[2:], results[0][2:]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_long_prompt_at_once(fa):
    """A prompt of 5000 tokens appended and attended in one call, beside a sequence that has one token more."""
    H, Hk, d, page, T, lens, new = 4, 2, 128, 64, 5000, [5000, 700], [5000, 1]
    c = Cache(75, 2, Hk, d, page, max(lens))
    c.fill(c.table[1], lens[1] - 1, 76)
    q, k, v = rand(77, 2, H, T, d), rand(78, 2, Hk, T, d), rand(79, 2, Hk, T, d)
    w, _ = fa.rope_freqs(d, base=500000.0)
    turned = fa.kv_append(q, k, v, c.k, c.v, c.device_table(), i32(lens), w, new_lens=i32(new))
    o, lse = fa.fwd_paged(turned, c.k, c.v, c.device_table(), i32(lens), new_lens=i32(new))
    rows = [0, 1, 127, 128, 255, 256, 2500, 4735, 4998, 4999]  # of the first sequence, and the second's one
    for b, at in ((0, rows), (1, [0])):
        n = lens[b]
        keys, values = ([ref.gather(f64(x), c.table[b], n, hk) for hk in range(Hk)] for x in (c.k, c.v))
        for h in range(H):
            kk, vv = keys[h // (H // Hk)], values[h // (H // Hk)]
            pos = np.array([n - new[b] + t for t in at])
            got_q = f64(turned[b, h])[at]
            want = ref.attend(got_q, kk, vv, np.zeros(len(at), int), pos + 1, d ** -0.5)
            ref.check_attention(f64(o[b, h])[at], f64(lse[b, h])[at], (want[0], want[1], want[2]))
    assert float(o[1, :, 1:].abs().max()) == 0 and bool(torch.isneginf(lse[1, :, 1:]).all())


def test_caches_and_strides_past_32_bits(fa):
    """A cache of more than 2^31 elements whose last pages are used, and a view with row strides as large."""
    n_pages, page, d = 140000, 256, 64
    need = 2 * 2 * n_pages * page * d + (4 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GB")
    k, v = (torch.empty(n_pages, 1, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    c = Cache(63, 2, 1, d, page, 600)
    c.k, c.v = k, v
    c.table = np.array([[n_pages - 1, 139000, n_pages - 7], [0, n_pages - 3, 138001]], dtype=np.int32)
    x = [rand(64 + i, 2, 1, 600, d) for i in range(3)]
    lens = i32([600, 600])
    tq = fa.kv_append(*x, k, v, c.device_table(), lens)
    o, lse = fa.fwd_paged(tq, k, v, c.device_table(), lens)
    want, want_l = fa.fwd(*x, causal=True, n_splits=1)
    err = (o.float() - want.float()).abs()
    assert bool((err <= 4 * ref.U * (want.float().abs() + x[2].float().abs().max())).all())
    assert bool(((lse - want_l).abs() <= 2.0 ** -11 * want_l.abs().clamp(min=1)).all())
    del c, tq, o, lse
    flat = k.view(-1)
    far = torch.as_strided(flat, (2, 3, 2, d), (1024, 64, 2 ** 31 + 64, 1))
    far.copy_(rand(70, 2, 3, 2, d))
    w, _ = fa.rope_freqs(d)
    y, _ = fa.rope(far, None, w, offset=9)
    check_rope(y, far, np.arange(2) + 9, w, 1.0, False)
    out = torch.as_strided(v.view(-1), (2, 3, 2, d), (2 ** 31 + 64, 64, 1024, 1))
    fa.rope(far, None, w, offset=9, q_out=out)
    assert torch.equal(out, y)


def test_many_repeats_agree(fa):
    """Calls with many row blocks per CTA, again and again: the same bits, and no wait that gives up."""
    for B, H, Hk, T, d, n in ((6, 32, 2, 8, 128, 2500), (40, 16, 2, 20, 64, 400), (30, 16, 4, 1, 128, 3000)):
        c = Cache(66, B, Hk, d, 32, n)
        lens = [n - 61 * i % (n - T) for i in range(B)]
        for b in range(B):
            c.fill(c.table[b], lens[b], b)
        q = rand(67, B, H, T, d)
        o, lse = run_paged(fa, c, q, lens, None)
        for _ in range(40):
            a, b = run_paged(fa, c, q, lens, None)
            assert torch.equal(a, o) and torch.equal(b, lse)


def test_another_stream_takes_the_same_path(fa):
    """The calls with an explicit stream (checked in Python) against the usual ones (checked in C++)."""
    B, H, Hk, T, d, page = 2, 4, 2, 3, 64, 16
    w, mag = fa.rope_freqs(d, scaling="by_parts", factor=2.0)
    _, (q, k, v) = packed(68, B, T, H, Hk, d)
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side):
        c = Cache(69, B, Hk, d, page, 40, prefix_len=20)
        c.fill(c.prefix_pages, 20, 5)
        lens = i32([3, 3])
        torch.cuda.synchronize()
        tq = fa.kv_append(q, k, v, c.k, c.v, c.device_table(), lens, w, offset=20, mag=mag, stream=stream)
        torch.cuda.synchronize()
        r = [tq, *fa.rope(q, k, w, mag=mag, stream=stream), *fa.rope_bwd(q, None, w, stream=stream)[:1]]
        torch.cuda.synchronize()
        r += [*run_paged(fa, c, tq, [3, 3], None, stream=stream), *run_paged(fa, c, tq, [3, 3], None, prefix_len=20,
                                                                             stream=stream)]
        torch.cuda.synchronize()
        got.append(r + [c.k[int(c.table[0, 0]), :, :3], c.v[int(c.table[1, 0]), :, :3]])
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,H,Hk,page", [(64, 4, 4, 16), (128, 6, 2, 32)])
def test_generation_matches_the_dense_forward(fa, d, H, Hk, page):
    """A prompt in two chunks, then single tokens, through append and paged attention, against rope and the
    dense causal forward over the whole sequence; then the same with the prompt as a shared prefix."""
    B, N, cuts = 2, 120, [0, 50, 111, 112, 113, 120]
    w, mag = fa.rope_freqs(d, scaling="by_parts", factor=2.0)
    _, (q, k, v) = packed(60, B, N, H, Hk, d)
    rq, rk = fa.rope(q, k, w, mag=mag)
    wide = (lambda x: x.repeat_interleave(H // Hk, dim=1).contiguous())
    want, want_l = fa.fwd(rq, wide(rk), wide(v.contiguous()), causal=True, n_splits=1)
    c = Cache(61, B, Hk, d, page, N)
    table = c.device_table()
    for a, b in zip(cuts, cuts[1:]):
        lens = i32([b] * B)
        tq = fa.kv_append(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], c.k, c.v, table, lens, w, mag=mag)
        assert torch.equal(tq, rq[:, :, a:b])
        o, lse = fa.fwd_paged(tq, c.k, c.v, table, lens)
        # both sides round the same P and O to bf16: two roundings of each
        err = (o.float() - want[:, :, a:b].float()).abs()
        assert bool((err <= 4 * ref.U * (want[:, :, a:b].float().abs() + v.float().abs().max())).all())
        assert bool(((lse - want_l[:, :, a:b]).abs() <= 2.0 ** -11 * want_l[:, :, a:b].abs().clamp(min=1)).all())
    # the first sequence's first 100 tokens as every sequence's prefix
    n = 100
    c = Cache(62, B, Hk, d, page, N - n, prefix_len=n)
    one = torch.from_numpy(c.prefix_pages).cuda()[None]
    fa.kv_append(None, k[:1, :, :n], v[:1, :, :n], c.k, c.v, one, i32([n]), w, mag=mag)
    lens = i32([N - n] * B)
    same = [x[:1, :, n:].expand(B, -1, -1, -1) for x in (q, k, v)]
    tq = fa.kv_append(*same, c.k, c.v, c.device_table(), lens, w, offset=n, mag=mag)
    o, lse = fa.fwd_prefix(tq, c.k, c.v, one[0], n, c.device_table(), lens)
    for b in range(B):
        err = (o[b].float() - want[0, :, n:].float()).abs()
        assert bool((err <= 4 * ref.U * (want[0, :, n:].float().abs() + v.float().abs().max())).all())


def test_training_step_through_rope(fa):
    """rope, fwd, bwd, rope_bwd: the gradient of the packed projection against 64-bit autograd."""
    B, H, N, d = 1, 2, 70, 64
    w, _ = fa.rope_freqs(d)
    x, (q, k, v) = packed(70, B, N, H, H, d)
    g = rand(71, B, H, N, d)
    rq, rk = fa.rope(q, k, w)
    vc = v.contiguous()
    o, lse = fa.fwd(rq, rk, vc, causal=True, n_splits=1)
    dq, dk, dv = fa.bwd(rq, rk, vc, o, lse, g, causal=True)
    dx = torch.empty_like(x)
    oq, ok, ov = (dx[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(3))
    fa.rope_bwd(dq, dk, w, q_out=oq, k_out=ok)
    ov.copy_(dv)
    x64 = x.double().cpu().requires_grad_()
    a = torch.outer(torch.arange(N, dtype=torch.float64), w.cpu())
    turn = torch.polar(torch.ones_like(a), a)
    parts = [x64[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(3)]

    def turned(y):
        z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    s = turned(parts[0]) @ turned(parts[1]).transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    ((s.softmax(-1) @ parts[2]) * g.double().cpu()).sum().backward()
    # bf16 q, k (rotated), P, dS, O and the gradients: about eight roundings of size u, taken of the largest entry
    err = (dx.double().cpu() - x64.grad).abs().max() / x64.grad.abs().max()
    assert err <= 8 * ref.U, float(err)


def test_captured_steps_follow_growing_lengths(fa):
    """One captured decode step (append, attention) replayed token after token, beside eager calls."""
    B, H, Hk, d, page, N = 2, 4, 2, 64, 16, 40
    w, _ = fa.rope_freqs(d)
    _, (q, k, v) = packed(80, B, N, H, Hk, d)
    caches = [Cache(81, B, Hk, d, page, N) for _ in range(2)]
    table = caches[0].device_table()
    lens = i32([1] * B)
    sq, sk, sv = (x[:, :, :1].contiguous() for x in (q, k, v))
    o, lse = torch.empty_like(sq), torch.empty(B, H, 1, device="cuda")

    def step(c):
        tq = fa.kv_append(sq, sk, sv, c.k, c.v, table, lens, w)
        fa.fwd_paged(tq, c.k, c.v, table, lens, out=o, lse=lse)

    step(caches[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0])
    for t in range(N):
        lens.fill_(t + 1)
        for s, x in ((sq, q), (sk, k), (sv, v)):
            s.copy_(x[:, :, t:t + 1])
        o.zero_()
        graph.replay()
        got = o.clone(), lse.clone()
        step(caches[1])
        assert torch.equal(got[0], o) and torch.equal(got[1], lse), t
    assert torch.equal(caches[0].k.view(torch.int16), caches[1].k.view(torch.int16))


def test_captured_rotation_and_prefix_replay(fa):
    """rope, rope_bwd and fwd_prefix replay on new contents; two graphs of one call share no workspace."""
    B, H, Hk, T, d, n = 3, 4, 2, 1, 64, 150
    c = Cache(83, B, Hk, d, 16, 64, prefix_len=n)
    c.fill(c.prefix_pages, n, 1)
    for b in range(B):
        c.fill(c.table[b], 64, 2 + b)
    w, _ = fa.rope_freqs(d)
    pages, table, lens = torch.from_numpy(c.prefix_pages).cuda(), c.device_table(), i32([1, 2, 3])
    q = rand(84, B, H, T, d)

    def step():
        y, _ = fa.rope(q, None, w, offset=7)
        o, lse = fa.fwd_prefix(y, c.k, c.v, pages, n, table, lens)
        g, _ = fa.rope_bwd(o, None, w, offset=7)
        return o, lse, g

    step()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    for i in range(3):
        lens.fill_(5 * i + 1)
        q.copy_(rand(85 + i, B, H, T, d))
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):  # both at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = step()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_capture_behind_copies_and_joined_streams(fa):
    """The calls inside a larger graph: behind a copy and a fill, and behind two streams that join."""
    B, H, Hk, T, d = 2, 4, 2, 1, 64
    c = Cache(87, B, Hk, d, 16, 200)
    for b in range(B):
        c.fill(c.table[b], 200, b)
    table, lens, q = c.device_table(), i32([200, 150]), rand(88, B, H, T, d)
    q_in, lens_in = rand(89, B, H, T, d), i32([31, 180])
    x = torch.zeros(1 << 20, device="cuda")
    fa.fwd_paged(q, c.k, c.v, table, lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.copy_(q_in)
        lens.copy_(lens_in)
        first = fa.fwd_paged(q, c.k, c.v, table, lens)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x.add_(1.0)
            q.copy_(q_in.flip(0))
        x[:7].zero_()
        torch.cuda.current_stream().wait_stream(side)
        second = fa.fwd_paged(q, c.k, c.v, table, lens)
        x.mul_(2.0)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got, qq in ((first, q_in), (second, q_in.flip(0).contiguous())):
        want = fa.fwd_paged(qq, c.k, c.v, table, lens_in)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_streams_at_once(fa):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    B, H, Hk, T, d = 4, 8, 2, 1, 128
    c = Cache(91, B, Hk, d, 16, 3000)
    lens = [3000, 10, 700, 1500]
    for b in range(B):
        c.fill(c.table[b], lens[b], b)
    qs = [rand(92 + i, B, H, T, d) for i in range(2)]
    alone = [run_paged(fa, c, q, lens, None) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(run_paged(fa, c, qs[i], lens, None, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1])


def test_no_tokens_is_a_noop(fa):
    c = Cache(95, 2, 1, 64, 16, 32)
    e = torch.empty(2, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    w, _ = fa.rope_freqs(64)
    assert fa.rope(e, e, w)[0].shape == e.shape
    assert fa.kv_append(e, e, e, c.k, c.v, c.device_table(), i32([3, 3]), w).shape == e.shape
    o, lse = run_paged(fa, c, e, [3, 3], None)
    assert o.shape == e.shape and lse.shape == (2, 1, 0)
