"""The norm with the rotation without a GPU: argument checks of the C ABI and of the
Python entry points, and the tests' own 64-bit gradients against differences."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_attention_19_gb300 as fa  # noqa: E402
import norm_ref  # noqa: E402
from exact_attention_19_gb300 import build as fa_build  # noqa: E402

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load()


def call_norm(**kw):
    a = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, inv_freq=FAKE, q_weight=FAKE, k_weight=FAKE, positions=None,
             position_stride=0, offset=0, strides=None, B=1, H=2, Hk=1, N=8, d=64, rot=64, mag=1.0, interleaved=0,
             eps=1e-6, weights_f32=0, stream=None)
    a.update(kw)
    return fa.fa_norm_rope(*a.values())


COMMON = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(inv_freq=None), 1),
    (dict(q=FAKE + 2), 2), (dict(inv_freq=FAKE + 4), 2), (dict(positions=FAKE + 2), 2), (dict(q_weight=FAKE + 8), 2),
    (dict(k_weight=FAKE + 4), 2), (dict(d=96), 4), (dict(B=0), 3), (dict(H=0), 3), (dict(Hk=-1), 3), (dict(N=-1), 3),
    (dict(rot=8), 3), (dict(rot=-16), 3), (dict(rot=80), 3), (dict(interleaved=2), 3), (dict(weights_f32=2), 3),
    (dict(positions=FAKE, position_stride=7), 3), (dict(B=1 << 16, N=1 << 15), 3),
    (dict(mag=math.inf), 9), (dict(eps=-1e-6), 9), (dict(eps=math.nan), 9), (dict(eps=math.inf), 9),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(q_out=None), 1), (dict(k_out=None), 1), (dict(k_out=FAKE + 8), 2),
    (dict(strides=[64] * 11 + [0]), 13), (dict(strides=[4] + [64] * 11), 13),
    (dict(N=0), 0), (dict(N=0, q=None, k=None, q_out=None, k_out=None), 0)])
def test_norm_rope_refusals(kw, code):
    assert call_norm(**kw) == code


def test_norm_rope_optional_arguments_pass_the_checks():
    for kw in (dict(Hk=0, k=None, k_out=None), dict(rot=0, inv_freq=None), dict(q_weight=None, k_weight=None),
               dict(weights_f32=1), dict(eps=0.0), dict(strides=[0] * 6 + [64] * 6)):
        assert call_norm(**kw) not in (1, 2, 3, 4, 9, 13)


def call_bwd(**kw):
    a = dict(dq=FAKE, dk=FAKE, q=FAKE, k=FAKE, dq_out=FAKE, dk_out=FAKE, dq_weight=FAKE, dk_weight=FAKE, inv_freq=FAKE,
             q_weight=FAKE, k_weight=FAKE, positions=None, position_stride=0, offset=0, strides=None, B=1, H=2, Hk=1,
             N=8, d=64, rot=64, mag=1.0, interleaved=0, eps=1e-6, weights_f32=0, workspace=FAKE,
             workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return fa.fa_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dq=None), 1), (dict(dk=None), 1), (dict(dq_out=None), 1), (dict(dk_out=None), 1), (dict(workspace=None), 1),
    (dict(dq=FAKE + 2), 2), (dict(dk_out=FAKE + 8), 2), (dict(dq_weight=FAKE + 4), 2), (dict(workspace=FAKE + 8), 2),
    (dict(Hk=0), 3), (dict(strides=[64] * 17 + [0]), 13), (dict(strides=[64] * 8 + [12] + [64] * 9), 13),
    (dict(N=0, dq_weight=None, dk_weight=None), 0)])
def test_norm_rope_bwd_refusals(kw, code):
    assert call_bwd(**kw) == code


def test_norm_rope_bwd_optional_arguments_pass_the_checks():
    for kw in (dict(Hk=0, k=None, dk=None, dk_out=None, dk_weight=None), dict(rot=0, inv_freq=None),
               dict(dq_weight=None, dk_weight=None, workspace=None, workspace_bytes=0), dict(dq_weight=None),
               dict(strides=[0] * 12 + [64] * 6),
               dict(N=0, dq=None, dk=None, q=None, k=None, dq_out=None, dk_out=None)):
        assert call_bwd(**kw) not in (0, 1, 2, 3, 4, 9, 13)


def test_norm_workspace_size():
    small, large = fa.fa_norm_bwd_workspace_bytes(64), fa.fa_norm_bwd_workspace_bytes(128)
    assert 0 < small and large == 2 * small and small % 16 == 0
    assert fa.fa_norm_bwd_workspace_bytes(96) == 0


def call_append(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, k_cache=FAKE, v_cache=FAKE, inv_freq=FAKE, q_weight=FAKE,
             k_weight=FAKE, block_table=FAKE, seq_lens=FAKE, new_lens=None, shift=FAKE, strides=[64] * 18, B=2, H=2, Hk=1,
             T=1, d=64, rot=64, n_pages=4, page_size=16, max_pages=2, offset=0, mag=1.0, interleaved=0, norm=1, eps=1e-6,
             weights_f32=0, stream=None)
    a.update(kw)
    return fa.fa_kv_append_norm(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(v_cache=None), 1), (dict(inv_freq=None), 1), (dict(block_table=None), 1),
    (dict(shift=FAKE + 2), 2), (dict(q_weight=FAKE + 8), 2), (dict(k_weight=FAKE + 2), 2), (dict(d=32), 4),
    (dict(norm=2), 3), (dict(norm=-1), 3), (dict(weights_f32=3), 3), (dict(rot=72), 3), (dict(page_size=48), 3),
    (dict(eps=-1.0), 9), (dict(eps=math.nan), 9), (dict(mag=math.nan), 9), (dict(strides=[64] * 17 + [12]), 13),
    (dict(T=0), 0)])
def test_append_norm_refusals(kw, code):
    assert call_append(**kw) == code


def test_append_norm_optional_arguments_pass_the_checks():
    for kw in (dict(shift=None), dict(norm=0, eps=math.nan), dict(q_weight=None, k_weight=None),
               dict(H=0, q=None, q_out=None), dict(rot=0, inv_freq=None)):
        assert call_append(**kw) not in (1, 2, 3, 4, 9, 13)


def test_python_entry_points_refuse_host_tensors():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, dtype=torch.float64)
    t = torch.zeros(1, 1, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: fa.norm_rope(x, x, w), lambda: fa.norm_rope_bwd(x, x, x, x, w),
              lambda: fa.kv_append(x, x, x, x, x, t, n, w, eps=1e-6), lambda: fa.kv_append(x, x, x, x, x, t, n, shift=n)):
        with pytest.raises(TypeError):
            f()
    for bad in (2 ** 63, -2 ** 63 - 1):
        for f in (lambda: fa.norm_rope(x, x, w, offset=bad), lambda: fa.norm_rope_bwd(x, x, x, x, w, offset=bad)):
            with pytest.raises(ValueError):
                f()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_reference_gradient_against_differences(rot, interleaved):
    """norm_ref's gradients against central differences of its forward (step h: an error of h^2 and of 2^-52 / h)."""
    rng = np.random.default_rng(rot)
    d, N, eps, mag = 8, 3, 1e-3, 1.5
    x, dy, w = rng.normal(size=(2, N, d)), rng.normal(size=(2, N, d)), rng.normal(size=d)
    freq = rng.normal(size=rot // 2) if rot else None
    p = [5, 0, 9]

    def loss(x, w):
        return float((norm_ref.norm_rope(x, w, eps, p, freq, mag, interleaved)[0] * dy).sum())

    dx, bound, dw, wbound = norm_ref.norm_rope_bwd(dy, x, w, eps, p, freq, mag, interleaved)
    h = 1e-5
    for at in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert math.isclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[at], rel_tol=1e-5, abs_tol=1e-7)
    for i in range(d):
        e = np.zeros_like(w)
        e[i] = h
        assert math.isclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[i], rel_tol=1e-5, abs_tol=1e-7)
    assert np.all(bound > 0) and np.all(wbound > 0)
    # the gradient of a norm has no part along x (eps aside): the weights' part shows it
    n, _ = norm_ref.normed(x, 0.0)
    assert np.allclose((n * n).mean(-1), 1.0)
