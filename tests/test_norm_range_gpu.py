"""The norm of heads whose squares leave fp32's range, up (with eps below 2^-96) and down: forward, backward and in the
append, with norm_ref's bounds.  Heads are scaled by a power of two there, which is exact, so no bound grows.
Only results below 2^-126, which heads of very different elements have, need a term that norm_ref has not: bf16 holds
them as multiples of 2^-133, so their rounding is off by up to 2^-134 however small they are."""
import numpy as np
import pytest

import norm_ref

torch = pytest.importorskip("torch")

from test_norm_gpu import check_bwd, check_norm, f64, freqs, i32, weights  # noqa: E402

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


SUBNORMAL = 2.0 ** -134
EXPONENTS = [-130, -120, -100, -76, -63, -49, -48, -47, -46, 0, 59, 61, 62, 63, 64, 65, 100, 124]


def scaled(seed, e, *shape):
    """bf16 of size 2^e, none of them zero or infinite."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g, dtype=torch.float64).clamp(-3.9, 3.9)
    x = torch.where(x.abs() < 0.125, torch.full_like(x, 0.125), x) * 2.0 ** e
    return x.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -120, 2.0 ** -97, 2.0 ** -96, 1e-6])
def test_heads_of_any_size(fa, d, rot, interleaved, eps):
    """One call over heads of all sizes beside one another, and a backward for each size."""
    H, N = 3, 5
    w, wq = freqs(fa, rot), weights(2, d, torch.float32)
    x = torch.cat([scaled(i, e, 1, H, N, d) for i, e in enumerate(EXPONENTS)])
    # every size beside every other in one warp: the sequences become heads
    x = x.permute(1, 2, 0, 3).reshape(1, H * N, len(EXPONENTS), d).contiguous()
    p = np.arange(len(EXPONENTS))
    y, _ = fa.norm_rope(x, None, w, wq, eps=eps, interleaved=interleaved)
    # with eps well above the squares a head's size is kept, down to results that bf16 holds with fewer bits: left out
    keep = [i for i, e in enumerate(EXPONENTS) if eps == 0.0 or 2.0 ** e * eps ** -0.5 > 2.0 ** -110]
    if eps >= 2.0 ** -96:  # elements below 2^60
        keep = [i for i in keep if EXPONENTS[i] < 59]
    z = y.transpose(1, 2).reshape(len(EXPONENTS), H * N, 1, d)
    xs = x.transpose(1, 2).reshape(len(EXPONENTS), H * N, 1, d)
    for i in keep:
        check_norm(z[i:i + 1], xs[i:i + 1], wq, eps, p[i:i + 1], w, 1.0, interleaved, f"2^{EXPONENTS[i]}")
    assert bool(torch.isfinite(y).all())
    for i in keep:
        # gradients of a size that leaves dx among the numbers that bf16 holds with all bits
        dy = scaled(100 + i, round(0.4 * EXPONENTS[i]), 1, H * N, 1, d)
        dx, _, dw, _ = fa.norm_rope_bwd(dy, None, xs[i:i + 1], None, w, wq, eps=eps, offset=i, interleaved=interleaved)
        check_bwd(dx, dw, dy, xs[i:i + 1], wq, eps, p[i:i + 1], w, 1.0, interleaved, f"2^{EXPONENTS[i]}")


@pytest.mark.parametrize("big,small", [(120, 0), (120, 100), (64, 10), (-60, -100), (-100, -130), (-48, -90)])
def test_sizes_that_differ_within_a_head(fa, big, small):
    d, H, N = 128, 2, 9
    w, wq = freqs(fa, d), weights(3, d, torch.bfloat16)
    x = scaled(5, small, 1, H, N, d)
    x[:, 0, :, 7] = scaled(6, big, 1, N)
    x[:, 1, :, ::5] = scaled(7, big, 1, N, 26)
    y, _ = fa.norm_rope(x, None, w, wq, eps=0.0)
    want, bound = norm_ref.norm_rope(f64(x), f64(wq), 0.0, np.arange(N), f64(w), 1.0, False)
    assert np.all(np.abs(f64(y) - want) <= bound + SUBNORMAL)
    dy = scaled(8, round(0.4 * big), 1, H, N, d)
    dx, _, dw, _ = fa.norm_rope_bwd(dy, None, x, None, w, wq, eps=0.0)
    check_bwd(dx, dw, dy, x, wq, 0.0, np.arange(N), w, 1.0, False)


def test_heads_of_zeros(fa):
    """With eps they stay zeros; without they are NaN, and their neighbours are not."""
    d = 64
    w = freqs(fa, 32)
    x = scaled(9, -100, 1, 2, 4, d)
    x[0, 1, 2] = 0.0
    for eps in (2.0 ** -130, 1e-6):
        y, _ = fa.norm_rope(x, None, w, eps=eps)
        assert bool((y[0, 1, 2] == 0).all()) and bool(torch.isfinite(y).all())
    y, _ = fa.norm_rope(x, None, w, eps=0.0)
    assert torch.isnan(y).any(-1).nonzero().tolist() == [[0, 1, 2]]


def test_append_norms_heads_of_any_size(fa):
    """The same bits as norm_rope."""
    B, H, Hk, T, d, page = 2, 4, 2, 9, 128, 16
    w, wq, wk = freqs(fa, d), weights(1, d, torch.float32), weights(2, d, torch.float32)
    q = torch.cat([scaled(10 + i, EXPONENTS[2 * i], B, H, 1, d) for i in range(T)], 2)
    k = torch.cat([scaled(30 + i, EXPONENTS[2 * i + 1], B, Hk, 1, d) for i in range(T)], 2)
    for eps in (0.0, 1e-6):
        kc, vc = (torch.zeros(B, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        y = fa.kv_append(q, k, k, kc, vc, i32([[1], [0]]), i32([T, T]), w, eps=eps, q_weight=wq, k_weight=wk)
        a, b = fa.norm_rope(q, k, w, wq, wk, eps=eps)
        assert torch.equal(y, a) and torch.equal(kc[[1, 0], :, :T], b)
        assert bool(torch.isfinite(a).all()) and bool(torch.isfinite(b).all())
    with_zeros = k.clone()
    with_zeros[:, :, 4] = 0.0
    y = fa.kv_append(q, with_zeros, k, kc, vc, i32([[1], [0]]), i32([T, T]), w, eps=0.0)
    assert torch.isnan(kc).any(-1).any(1)[[1, 0], :T].nonzero().tolist() == [[0, 4], [1, 4]]
    assert not bool(torch.isnan(y).any())
