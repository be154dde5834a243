"""The cached keys' weights and eviction without a GPU: argument checks of the C ABI and
of the Python entry points, workspace, and pins of the tests' own plain forms."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_ref  # noqa: E402
import exact_attention_19_gb300 as fa  # noqa: E402
from exact_attention_19_gb300 import build as fa_build  # noqa: E402

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load()


def call_weights(**kw):
    a = dict(q=FAKE, lse=FAKE, k_cache=FAKE, weights=FAKE, block_table=FAKE, seq_lens=FAKE, new_lens=None,
             strides=[64] * 5, B=2, H=4, Hk=2, T=1, d=64, n_pages=4, page_size=16, max_pages=2, scale=0.125, left=-1,
             right=0, decay=1.0, stream=None)
    a.update(kw)
    return fa.fa_kv_weights(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(lse=None), 1), (dict(k_cache=None), 1), (dict(weights=None), 1),
    (dict(block_table=None), 1), (dict(seq_lens=None), 1), (dict(strides=None), 1),
    (dict(q=FAKE + 8), 2), (dict(k_cache=FAKE + 2), 2), (dict(lse=FAKE + 2), 2), (dict(weights=FAKE + 1), 2),
    (dict(new_lens=FAKE + 2), 2), (dict(d=256), 4), (dict(B=0), 3), (dict(H=3), 3), (dict(Hk=0), 3), (dict(T=-1), 3),
    (dict(page_size=17), 3), (dict(page_size=512), 3), (dict(n_pages=0), 3), (dict(max_pages=1 << 27), 3),
    (dict(B=1 << 20, T=1 << 12), 3), (dict(left=-2), 3), (dict(right=-2), 3),
    (dict(scale=0.0), 9), (dict(scale=math.nan), 9), (dict(decay=-0.5), 9), (dict(decay=math.nan), 9),
    (dict(decay=math.inf), 9), (dict(strides=[64, 64, 4, 64, 64]), 13), (dict(strides=[64, 64, 64, 0, 64]), 13),
    (dict(strides=[64, 64, 64, 64, -1]), 13),
    (dict(T=0), 0), (dict(T=0, q=None, lse=None), 0)])
def test_weights_refusals(kw, code):
    assert call_weights(**kw) == code


def test_weights_optional_arguments_pass_the_checks():
    for kw in (dict(new_lens=FAKE), dict(decay=0.0), dict(decay=2.0), dict(strides=[64, 64, 64, 1, 1]),
               dict(lse=FAKE + 4, weights=FAKE + 4)):
        assert call_weights(**kw) not in (0, 1, 2, 3, 4, 9, 13)


def call_evict(**kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, weights=FAKE, block_table=FAKE, table_out=None, out_pages=0, seq_lens=FAKE,
             lens_out=FAKE, shift=None, kept=FAKE, strides=[64] * 8, B=2, Hk=2, d=64, n_pages=4, page_size=16, max_pages=2,
             budget=8, recent=2, sinks=1, slack=0, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return fa.fa_kv_evict(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(weights=None), 1), (dict(block_table=None), 1),
    (dict(seq_lens=None), 1), (dict(lens_out=None), 1), (dict(kept=None), 1), (dict(strides=None), 1),
    (dict(workspace=None), 1), (dict(v_cache=FAKE + 2), 2), (dict(weights=FAKE + 2), 2), (dict(table_out=FAKE + 2), 2),
    (dict(shift=FAKE + 1), 2), (dict(kept=FAKE + 3), 2), (dict(workspace=FAKE + 8), 2), (dict(d=32), 4),
    (dict(B=0), 3), (dict(Hk=0), 3), (dict(n_pages=0), 3), (dict(page_size=24), 3), (dict(max_pages=0), 3),
    (dict(budget=0), 3), (dict(budget=-3), 3), (dict(recent=-1), 3), (dict(sinks=-1), 3), (dict(slack=-1), 3),
    (dict(recent=8), 3), (dict(budget=1 << 30, slack=1), 3), (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), 3),
    (dict(table_out=FAKE + 4, out_pages=0), 3), (dict(table_out=FAKE + 4, out_pages=1, budget=16, slack=1), 3),
    (dict(table_out=FAKE, out_pages=1), 3), (dict(table_out=FAKE, out_pages=3), 3),  # block_table with rows of another width
    (dict(strides=[64] * 7 + [0]), 13), (dict(strides=[64] * 5 + [12] + [64] * 2), 13)])
def test_evict_refusals(kw, code):
    assert call_evict(**kw) == code


def test_evict_optional_arguments_pass_the_checks():
    for kw in (dict(), dict(shift=FAKE), dict(table_out=FAKE + 4, out_pages=1, budget=16), dict(recent=7),
               dict(table_out=FAKE, out_pages=2),
               dict(strides=[64] * 6 + [1, 1])):
        assert call_evict(**kw) not in (0, 1, 2, 3, 4, 9, 13)


def test_evict_workspace_size():
    for B, Hk in ((1, 1), (3, 5), (7, 11), (64, 64)):
        n = fa.fa_evict_workspace_bytes(B, Hk)
        assert n >= 16 * B * Hk and n <= 16 * B * Hk + (4 << 20)
    for bad in ((0, 1), (1, 0), (1 << 20, 1 << 12)):
        assert fa.fa_evict_workspace_bytes(*bad) == 0


def test_python_entry_points_refuse():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f = torch.zeros(1, 2, 4)
    t = torch.zeros(1, 1, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fa.kv_weights(x, f, x, f, t, n), lambda: fa.kv_evict(x, x, f, t, n, 4)):
        with pytest.raises(TypeError):
            call()
    for kw in (dict(budget=0), dict(budget=4, recent=3, sinks=2), dict(budget=4, slack=-1), dict(budget=2 ** 31),
               dict(budget=4, recent=-1), dict(budget=2 ** 31 - 1, slack=1), dict(budget=2 ** 32 + 4)):
        with pytest.raises(ValueError):
            fa.kv_evict(x, x, f, t, n, **kw)
    with pytest.raises(ValueError):
        fa.kv_weights(x, f, x, f, t, n, window=(-2 ** 31 - 1, 0))


def test_reference_pins():
    """The tests' own forms: a softmax's columns, what stays of a short list, ties, NaN and zeros of both signs."""
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(1, 2, 3, 4)), rng.normal(size=(1, 1, 16, 4))
    table, s = np.array([[0]]), 0.5
    lse = np.full((1, 2, 3), -np.inf)
    for h in range(2):
        for t in range(3):
            lse[0, h, t] = np.log(np.exp(q[0, h, t] @ k[0, 0, :5 + t].T * s).sum())
    w0 = rng.uniform(size=(1, 1, 16))
    w, tol, written = cache_ref.key_weights(q, lse, k, w0, table, [7], [3], -1, 0, s, 0.5)
    assert np.isclose((w[0, 0, :7]).sum(), 6 + 0.5 * w0[0, 0, :4].sum())  # each row gives 1 in all
    assert np.array_equal(w[0, 0, 7:], w0[0, 0, 7:]) and written[0, 0].sum() == 7 and np.all(tol[0, 0, :7] > 0)
    w, _, _ = cache_ref.key_weights(q, lse, k, w0, table, [7], [0], -1, 0, s, 0.5)
    assert np.array_equal(w, w0)
    x = np.array([5.0, 0.0, 1.0, -0.0, 1.0, np.nan, 0.0, 2.0])
    assert cache_ref.kept_slots(x, 8, 4, 1, 1).tolist() == [0, 2, 5, 7]
    assert cache_ref.kept_slots(x, 8, 6, 1, 1).tolist() == [0, 1, 2, 4, 5, 7]
    assert cache_ref.kept_slots(x, 8, 2, 1, 1).tolist() == [0, 7]
    moved, out, kept = cache_ref.evict([np.arange(16.0)[None, None]], np.pad(x, (0, 8))[None, None], table, [8], 4, 1, 1, 2)
    assert out[0] == 4 and kept[0, 0].tolist() == [0, 2, 5, 7, -1, -1]
    assert moved[0][0, 0].tolist() == [0, 2, 5, 7] + list(range(4, 16))
