"""The norm of each head with the rotation, its gradients, and the same in the paged
cache's append, against plain 64-bit implementations (norm_ref)."""
import math

import numpy as np
import pytest

import norm_ref
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


def weights(seed, d, kind):
    g = torch.Generator().manual_seed(seed)
    if kind is None:
        return None
    return (1.0 + 0.5 * torch.randn(d, generator=g)).to(kind).cuda()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def weight64(w):
    return 1.0 if w is None else f64(w)


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def packed(seed, B, N, H, Hk, d):
    """Views [B, heads, N, d] of a packed token-major projection."""
    x = rand(seed, B, N, (H + 2 * Hk) * d)
    return x, [x[..., a * d:b * d].unflatten(-1, (b - a, d)).transpose(1, 2)
               for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk))]


def freqs(fa, rot):
    return fa.rope_freqs(rot)[0] if rot else None


def check_norm(got, x, weight, eps, positions, w, mag, interleaved, what=""):
    x, got = f64(x), f64(got)
    for b in range(x.shape[0]):
        p = positions[b] if np.ndim(positions) == 2 else positions
        y, bound = norm_ref.norm_rope(x[b], weight64(weight), eps, p, None if w is None else f64(w), mag, interleaved)
        assert np.all(np.isfinite(got[b]))
        over = np.abs(got[b] - y) - bound
        assert np.all(over <= 0), f"{what}: sequence {b} over its bound by {over.max():.3e}"


def check_bwd(got, gotw, dy, x, weight, eps, positions, w, mag, interleaved, what=""):
    x, dy, got = f64(x), f64(dy), f64(got)
    dw, wbound = 0.0, 0.0
    for b in range(x.shape[0]):
        p = positions[b] if np.ndim(positions) == 2 else positions
        dx, bound, dwb, wb = norm_ref.norm_rope_bwd(dy[b], x[b], weight64(weight), eps, p,
                                                    None if w is None else f64(w), mag, interleaved)
        over = np.abs(got[b] - dx) - bound
        assert np.all(over <= 0), f"{what}: sequence {b} over its bound by {over.max():.3e}"
        dw, wbound = dw + dwb, wbound + wb
    if weight is None:
        assert gotw is None
    else:
        assert gotw.dtype == torch.float32 and gotw.shape == weight.shape
        over = np.abs(f64(gotw) - dw) - wbound
        assert np.all(over <= 0), f"{what}: weight gradient over its bound by {over.max():.3e}"


SHAPES = [  # B, H, Hk, N, d, rot
    (1, 1, 1, 1, 64, 64), (2, 3, 1, 33, 64, 16), (1, 4, 4, 65, 64, 48), (3, 12, 12, 7, 64, 0),
    (1, 8, 2, 31, 128, 128), (2, 5, 5, 129, 128, 64), (1, 2, 1, 300, 128, 112), (2, 32, 8, 40, 128, 0),
]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hk,N,d,rot", SHAPES)
def test_norm_rope(fa, B, H, Hk, N, d, rot, interleaved, kind):
    _, (q, k, _) = packed(N, B, N, H, Hk, d)
    w, wq, wk = freqs(fa, rot), weights(1, d, kind), weights(2, d, kind)
    yq, yk = fa.norm_rope(q, k, w, wq, wk, eps=1e-5, offset=11, interleaved=interleaved, mag=1.25)
    assert yq.is_contiguous() and yk.is_contiguous()
    p = np.arange(N) + 11
    check_norm(yq, q, wq, 1e-5, p, w, 1.25, interleaved, "q")
    check_norm(yk, k, wk, 1e-5, p, w, 1.25, interleaved, "k")


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hk,N,d,rot", SHAPES)
def test_norm_rope_backward(fa, B, H, Hk, N, d, rot, interleaved, kind):
    _, (q, k, _) = packed(N, B, N, H, Hk, d)
    dq, dk = rand(N + 1, B, H, N, d), rand(N + 2, B, Hk, N, d)
    w, wq, wk = freqs(fa, rot), weights(1, d, kind), weights(2, d, kind)
    gq, gk, gwq, gwk = fa.norm_rope_bwd(dq, dk, q, k, w, wq, wk, eps=1e-5, offset=11, interleaved=interleaved, mag=1.25)
    p = np.arange(N) + 11
    check_bwd(gq, gwq, dq, q, wq, 1e-5, p, w, 1.25, interleaved, "q")
    check_bwd(gk, gwk, dk, k, wk, 1e-5, p, w, 1.25, interleaved, "k")


@pytest.mark.parametrize("B,H,Hk,N,d", [(1, 700, 3, 1, 64), (1, 1, 1, 1, 128), (3, 5, 2, 700, 64), (2, 40, 40, 129, 128)])
def test_backward_shares_of_the_heads(fa, B, H, Hk, N, d):
    """CTAs whose heads begin and end within a tile of tokens, and tiles that two sequences share."""
    _, (q, k, _) = packed(N, B, N, H, Hk, d)
    dq, dk = rand(N + 1, B, H, N, d), rand(N + 2, B, Hk, N, d)
    w, wq, wk = freqs(fa, 64), weights(1, d, torch.float32), weights(2, d, torch.float32)
    gq, gk, gwq, gwk = fa.norm_rope_bwd(dq, dk, q, k, w, wq, wk, eps=1e-5, offset=3, mag=1.0)
    p = np.arange(N) + 3
    check_bwd(gq, gwq, dq, q, wq, 1e-5, p, w, 1.0, False, "q")
    check_bwd(gk, gwk, dk, k, wk, 1e-5, p, w, 1.0, False, "k")


def test_many_tokens_and_one_weight(fa):
    """More items than CTAs, a weight for q alone, positions of packed documents; the results repeat bit for bit."""
    B, H, Hk, N, d, rot = 2, 9, 3, 1501, 128, 64
    _, (q, k, _) = packed(3, B, N, H, Hk, d)
    dq, dk = rand(4, B, H, N, d), rand(5, B, Hk, N, d)
    w, wq = freqs(fa, rot), weights(6, d, torch.float32)
    p = ((np.arange(N)[None] + np.array([[0], [77]])) % 400).astype(np.int32)
    pos = torch.from_numpy(p).cuda()
    yq, yk = fa.norm_rope(q, k, w, wq, positions=pos)
    check_norm(yq, q, wq, 1e-6, p, w, 1.0, False, "q")
    check_norm(yk, k, None, 1e-6, p, w, 1.0, False, "k")
    first = fa.norm_rope_bwd(dq, dk, q, k, w, wq, positions=pos)
    check_bwd(first[0], first[2], dq, q, wq, 1e-6, p, w, 1.0, False, "q")
    check_bwd(first[1], first[3], dk, k, None, 1e-6, p, w, 1.0, False, "k")
    ws = torch.full((fa.fa_norm_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")  # NaN as floats
    for kw in ({}, {"workspace": ws}, {"stream": torch.cuda.current_stream()}):
        again = fa.norm_rope_bwd(dq, dk, q, k, w, wq, positions=pos, **kw)
        assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3])) and again[3] is None


def test_queries_alone_and_no_tokens(fa):
    d = 64
    w, wq = freqs(fa, 32), weights(7, d, torch.bfloat16)
    q, dq = rand(8, 2, 3, 5, d), rand(9, 2, 3, 5, d)
    y, none = fa.norm_rope(q, None, w, wq)
    assert none is None
    check_norm(y, q, wq, 1e-6, np.arange(5), w, 1.0, False)
    g, none, gw, nw = fa.norm_rope_bwd(dq, None, q, None, w, wq)
    assert none is None and nw is None
    check_bwd(g, gw, dq, q, wq, 1e-6, np.arange(5), w, 1.0, False)
    e = q[:, :, :0]
    y, _ = fa.norm_rope(e, None, w, wq)
    assert y.shape == e.shape
    g, gk, gw, gwk = fa.norm_rope_bwd(e, e, e, e, w, wq, wq)
    assert g.shape == e.shape and gk.shape == e.shape
    assert torch.equal(gw, torch.zeros_like(gw)) and torch.equal(gwk, torch.zeros_like(gw))


def test_in_place_and_strided_outputs(fa):
    """Outputs over the inputs, the packed neighbour untouched; gradients into a packed one, and over dq or q."""
    B, N, H, Hk, d = 2, 37, 4, 2, 64
    w, wq, wk = freqs(fa, 32), weights(1, d, torch.bfloat16), weights(2, d, torch.bfloat16)
    x, (q, k, v) = packed(5, B, N, H, Hk, d)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    oq, ok = fa.norm_rope(q, k, w, wq, wk, q_out=q, k_out=k)
    assert oq is q and ok is k
    check_norm(q, q0, wq, 1e-6, np.arange(N), w, 1.0, False)
    check_norm(k, k0, wk, 1e-6, np.arange(N), w, 1.0, False)
    assert torch.equal(v, v0)
    dq, dk = rand(6, B, H, N, d), rand(7, B, Hk, N, d)
    want = fa.norm_rope_bwd(dq, dk, q0, k0, w, wq, wk)
    dx = torch.full_like(x, 7.0)
    gq, gk, gv = (dx[..., a * d:b * d].unflatten(-1, (b - a, d)).transpose(1, 2)
                  for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
    got = fa.norm_rope_bwd(dq, dk, q0, k0, w, wq, wk, q_out=gq, k_out=gk)
    assert got[0] is gq and got[1] is gk and all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((gv == 7.0).all())
    dq2, k2 = dq.clone(), k0.contiguous().clone()
    got = fa.norm_rope_bwd(dq2, dk, q0, k2, w, wq, wk, q_out=dq2, k_out=k2)
    assert got[0] is dq2 and got[1] is k2 and all(torch.equal(a, b) for a, b in zip(got, want))
    # a broadcast gradient (stride 0), as of a sum over tokens
    one = rand(8, B, H, 1, d)
    got = fa.norm_rope_bwd(one.expand(B, H, N, d), None, q0, None, w, wq)
    check_bwd(got[0], got[2], one.expand(B, H, N, d), q0, wq, 1e-6, np.arange(N), w, 1.0, False)


def test_sizes_far_from_one(fa):
    """Heads of tiny, huge and zero elements, each by its own norm; eps beside a tiny mean square."""
    d, N = 128, 6
    x = rand(10, 1, 2, N, d)
    size = torch.tensor([2.0 ** 50, 2.0 ** -40, 1.0, 0.0, 2.0 ** 20, 2.0 ** -10]).to(torch.bfloat16).cuda()
    x = x * size[None, None, :, None]
    w, wq = freqs(fa, 64), weights(11, d, torch.float32)
    y, _ = fa.norm_rope(x, None, w, wq, eps=1e-6)
    check_norm(y, x, wq, 1e-6, np.arange(N), w, 1.0, False)
    assert bool((y[:, :, 3] == 0).all())
    dy = rand(12, 1, 2, N, d)
    g, _, gw, _ = fa.norm_rope_bwd(dy, None, x, None, w, wq, eps=1e-6)
    check_bwd(g, gw, dy, x, wq, 1e-6, np.arange(N), w, 1.0, False)


def test_values_that_are_not_finite(fa):
    """NaN and infinity stay in their own head; a broken frequency breaks its pair."""
    d, N = 64, 9
    w = freqs(fa, 64)
    q = rand(13, 1, 3, N, d)
    q[0, 1, 4, 7] = float("nan")
    q[0, 2, 5, 9] = float("inf")
    y, _ = fa.norm_rope(q, None, w)
    bad = torch.isnan(y)
    assert bool(bad[0, 1, 4].all())
    assert bool(bad[0, 2, 5, 9]) and bool(bad[0, 2, 5, 41])  # inf / inf and its partner
    left = bad.clone()
    left[0, 1, 4] = False
    left[0, 2, 5, [9, 41]] = False
    assert not bool(left.any())
    f = w.clone()
    f[3] = float("inf")
    y, _ = fa.norm_rope(rand(14, 1, 1, 2, d), None, f)
    assert torch.isnan(y).any(0).any(0).any(0).nonzero().flatten().tolist() == [3, 35]
    g, _, gw, _ = fa.norm_rope_bwd(rand(15, 1, 1, 2, d), None, rand(14, 1, 1, 2, d), None, f, weights(1, d, torch.float32))
    assert bool(torch.isnan(gw[[3, 35]]).all()) and not bool(torch.isnan(torch.cat([gw[:3], gw[4:35], gw[36:]])).any())


def test_refusals(fa):
    d = 64
    w, q = freqs(fa, 32), rand(16, 1, 2, 4, d)
    k, wq, wf = q[:, :1], weights(1, d, torch.bfloat16), weights(1, d, torch.float32)
    for kw, kind in ((dict(q_weight=wq, k_weight=wf), TypeError), (dict(q_weight=wq.half()), TypeError),
                     (dict(q_weight=wq[:32]), ValueError), (dict(q_weight=wq.cpu()), TypeError),
                     (dict(q_weight=wq.repeat(2)[::2]), ValueError), (dict(eps=-1.0), ValueError),
                     (dict(eps=math.nan), ValueError), (dict(inv_freq=w.float()), TypeError),
                     (dict(positions=i32([0, 1])), ValueError), (dict(q_out=k), ValueError)):
        with pytest.raises(kind):
            fa.norm_rope(q, k, **{"inv_freq": w, **kw})
        with pytest.raises(kind):
            fa.norm_rope_bwd(q, k, q, k, **{"inv_freq": w, **kw})
    with pytest.raises(fa.FaError):
        fa.norm_rope(q, k, w[:4])  # a part of 8 elements
    for args in ((q, None, q, k), (q, k, q, None), (k, k, q, k), (q, q, q, k)):
        with pytest.raises(ValueError):
            fa.norm_rope_bwd(*args, w)
    with pytest.raises(ValueError):
        fa.norm_rope_bwd(q, None, q, None, w, None, wq)
    with pytest.raises(fa.FaError):
        fa.norm_rope_bwd(q, None, q, None, w, wq, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    kc = torch.zeros(4, 1, 16, d, dtype=torch.bfloat16, device="cuda")
    args = (q, k, k, kc, kc.clone(), i32([[0]]), i32([4]), w)
    for kw, kind in ((dict(q_weight=wq), ValueError), (dict(eps=-1.0), ValueError), (dict(shift=i32([0, 1])), ValueError),
                     (dict(shift=i32([0]).long()), TypeError), (dict(eps=1e-6, q_weight=wq, k_weight=wf), TypeError)):
        with pytest.raises(kind):
            fa.kv_append(*args, **kw)
    assert bool((kc == 0).all())


# ---------------------------------------------------------------------------
# the paged cache's append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,H,Hk,T,d,page,rot,lens,new,norm", [
    (3, 4, 2, 1, 64, 16, 64, [5, 17, 40], None, True),
    (2, 6, 6, 5, 64, 32, 16, [5, 37], [5, 2], True),
    (2, 8, 2, 33, 128, 64, 128, [33, 100], [20, 33], True),
    (3, 4, 1, 4, 128, 16, 0, [4, 0, 50], [4, 0, 3], True),
    (2, 4, 2, 3, 128, 32, 128, [40, 3], None, False),
])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shifted", [False, True])
def test_append_norm(fa, B, H, Hk, T, d, page, rot, lens, new, norm, interleaved, shifted):
    _, (q, k, v) = packed(20, B, T, H, Hk, d)
    n_pages = sum(-(-max(n, 1) // page) for n in lens) + 2
    g = torch.Generator().manual_seed(21)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    width = max(-(-n // page) for n in lens)
    table, at = np.full((B, width), -7, np.int32), 0
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = order[at]
            at += 1
    kc, vc = (torch.full((n_pages, Hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w, wq, wk = freqs(fa, rot), weights(1, d, torch.bfloat16), weights(2, d, torch.bfloat16)
    shift = np.array([100000, 0, 7][:B], np.int32)
    q_out = torch.full((B, H, T, d), 9.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(eps=1e-6, q_weight=wq, k_weight=wk) if norm else {}
    got = fa.kv_append(q, k, v, kc, vc, torch.from_numpy(table).cuda(), i32(lens), w,
                       new_lens=None if new is None else i32(new), offset=3, interleaved=interleaved, q_out=q_out,
                       shift=torch.from_numpy(shift).cuda() if shifted else None, **kw)
    assert got is q_out
    seen = torch.zeros(n_pages, page, dtype=torch.bool)
    for b in range(B):
        m = T if new is None else new[b]
        j = np.arange(lens[b] - m, lens[b])
        p = j + 3 + (shift[b] if shifted else 0)
        if m:
            pages, slots = torch.from_numpy(table[b][j // page]).long(), torch.from_numpy(j % page)
            seen[pages, slots] = True
            k_got = kc[pages.cuda(), :, slots.cuda()].transpose(0, 1)[None]
            v_got = vc[pages.cuda(), :, slots.cuda()].transpose(0, 1)
            assert torch.equal(v_got, v[b, :, :m])
            if norm:
                check_norm(q_out[b:b + 1, :, :m], q[b:b + 1, :, :m], wq, 1e-6, p, w, 1.0, interleaved)
                check_norm(k_got, k[b:b + 1, :, :m], wk, 1e-6, p, w, 1.0, interleaved)
            else:
                for y, x in ((q_out[b, :, :m], q[b, :, :m]), (k_got[0], k[b, :, :m])):
                    want, size = ref.rotate(f64(x), p, f64(w), 1.0, interleaved)
                    assert np.all(np.abs(f64(y) - want) <= ref.rope_tol(want, size))
        assert bool((q_out[b, :, m:] == 9.0).all())
    untouched = ~seen.cuda()
    assert bool(torch.isnan(kc.transpose(1, 2)[untouched]).all()) and bool(torch.isnan(vc.transpose(1, 2)[untouched]).all())


def test_append_takes_the_same_path_on_another_stream(fa):
    B, H, Hk, T, d, page = 2, 4, 2, 3, 64, 16
    _, (q, k, v) = packed(22, B, T, H, Hk, d)
    w, wq = freqs(fa, d), weights(1, d, torch.float32)
    got = []
    for stream in (None, torch.cuda.Stream()):
        kc, vc = (torch.zeros(4, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        args = (i32([[2], [0]]), i32([7, 3]), w)
        shift = i32([50, 2 ** 30])
        torch.cuda.synchronize()
        y = fa.kv_append(q, k, v, kc, vc, *args, eps=1e-6, q_weight=wq, shift=shift, stream=stream)
        a = fa.norm_rope(q, k, w, wq, stream=stream)
        torch.cuda.synchronize()
        got.append([y, kc, vc, *a])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # a shift and no norm is an offset of each sequence's own
    kc2 = torch.zeros_like(got[0][1])
    y = fa.kv_append(q, k, v, kc2, torch.zeros_like(kc2), i32([[2], [0]]), i32([7, 3]), w, shift=i32([50, 50]))
    kc3 = torch.zeros_like(kc2)
    z = fa.kv_append(q, k, v, kc3, torch.zeros_like(kc2), i32([[2], [0]]), i32([7, 3]), w, offset=50)
    assert torch.equal(y, z) and torch.equal(kc2, kc3)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_training_step(fa):
    """norm_rope, fwd, bwd, norm_rope_bwd: the gradients of the packed projection and of the weights against 64-bit
    autograd of the whole."""
    B, H, N, d, eps = 1, 2, 70, 64, 1e-6
    w, wq, wk = freqs(fa, d), weights(1, d, torch.float32), weights(2, d, torch.float32)
    x, (q, k, v) = packed(30, B, N, H, H, d)
    g = rand(31, B, H, N, d)
    rq, rk = fa.norm_rope(q, k, w, wq, wk, eps)
    vc = v.contiguous()
    o, lse = fa.fwd(rq, rk, vc, causal=True, n_splits=1)
    dq, dk, dv = fa.bwd(rq, rk, vc, o, lse, g, causal=True)
    gq, gk, gwq, gwk = fa.norm_rope_bwd(dq, dk, q, k, w, wq, wk, eps)

    x64 = x.double().requires_grad_(True)
    w64 = [t.double().requires_grad_(True) for t in (wq, wk)]
    parts = [x64[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(3)]
    a = torch.arange(N, device="cuda").double()[:, None] * w

    def turned(t, weight):
        t = t / (t.square().mean(-1, keepdim=True) + eps).sqrt() * weight
        x0, x1 = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()], -1)

    s = turned(parts[0], w64[0]) @ turned(parts[1], w64[1]).transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -math.inf)
    (s.softmax(-1) @ parts[2] * g.double()).sum().backward()
    want = [x64.grad[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(2)]
    # roundings to bf16 on the way: rq, rk, P, dS, dq or dk and the result, each 2^-8 of the values around it, so a
    # few of them relative to the gradient's own size
    for got, ref64 in zip((gq, gk, gwq, gwk), (*want, w64[0].grad, w64[1].grad)):
        err = (got.double() - ref64).norm() / ref64.norm()
        assert float(err) <= 6 * ref.U, float(err)


def test_captured_calls_replay(fa):
    """Forward, backward and append in a graph, replayed on new inputs; the weights' gradients through a workspace of
    the graph's own."""
    B, H, Hk, N, d, page = 2, 4, 2, 50, 128, 16
    w, wq, wk = freqs(fa, d), weights(1, d, torch.bfloat16), weights(2, d, torch.bfloat16)
    q, k, dq, dk = rand(40, B, H, N, d), rand(41, B, Hk, N, d), rand(42, B, H, N, d), rand(43, B, Hk, N, d)
    kc, vc = (torch.zeros(8, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, lens, shift = i32([[0, 1, 2, 3], [7, 6, 5, 4]]), i32([N, N]), i32([0, 0])

    def step():
        y = fa.norm_rope(q, k, w, wq, wk)
        g = fa.norm_rope_bwd(dq, dk, q, k, w, wq, wk)
        a = fa.kv_append(q, k, k, kc, vc, table, lens, w, eps=1e-6, q_weight=wq, k_weight=wk, shift=shift)
        return [*y, *g, a, kc, vc]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (50, 60):
        for t, s in ((q, seed), (dq, seed + 1), (dk, seed + 2)):
            t.copy_(rand(s, *t.shape))
        shift.copy_(i32([seed, 3]))
        kc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        kc.zero_()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
