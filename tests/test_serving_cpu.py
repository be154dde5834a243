"""Rotary positions, the paged cache and its attention without a GPU: argument
checks of the C ABI and of the Python entry points, frequencies, workspace."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_attention_19_gb300 as fa  # noqa: E402
import serving_ref as ref  # noqa: E402
from exact_attention_19_gb300 import build as fa_build  # noqa: E402

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load()


def call_rope(**kw):
    a = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, inv_freq=FAKE, positions=None, position_stride=0, offset=0,
             strides=None, B=1, H=2, Hk=1, N=8, d=64, rot=64, mag=1.0, interleaved=0, backward=0, stream=None)
    a.update(kw)
    return fa.fa_rope(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(q_out=None), 1), (dict(k_out=None), 1), (dict(inv_freq=None), 1),
    (dict(q=FAKE + 2), 2), (dict(k_out=FAKE + 8), 2), (dict(inv_freq=FAKE + 4), 2), (dict(positions=FAKE + 2), 2),
    (dict(d=96), 4), (dict(B=0), 3), (dict(H=0), 3), (dict(Hk=-1), 3), (dict(N=-1), 3),
    (dict(rot=0), 3), (dict(rot=8), 3), (dict(rot=24), 3), (dict(rot=80), 3), (dict(interleaved=2), 3),
    (dict(backward=-1), 3), (dict(positions=FAKE, position_stride=7), 3), (dict(B=1 << 16, N=1 << 15), 3),
    (dict(mag=math.inf), 9), (dict(mag=math.nan), 9),
    (dict(strides=[64] * 11 + [0]), 13), (dict(strides=[4] + [64] * 11), 13), (dict(strides=[64] * 6 + [-64] * 6), 13),
    (dict(strides=[1 << 40] + [64] * 11), 13),
    (dict(N=0), 0), (dict(N=0, q=None, k=None, q_out=None, k_out=None), 0),
])
def test_rope_refusals(kw, code):
    assert call_rope(**kw) == code


def test_rope_without_keys_passes_the_checks():
    assert call_rope(Hk=0, k=None, k_out=None) not in (1, 2, 3, 4, 9, 13)
    assert call_rope(strides=[0] * 6 + [64] * 6) not in (1, 2, 3, 4, 9, 13)  # broadcast inputs


def call_append(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, k_cache=FAKE, v_cache=FAKE, inv_freq=FAKE, block_table=FAKE,
             seq_lens=FAKE, new_lens=None, strides=[64] * 18, B=2, H=2, Hk=1, T=1, d=64, rot=64, n_pages=4,
             page_size=16, max_pages=2, offset=0, mag=1.0, interleaved=0, stream=None)
    a.update(kw)
    return fa.fa_kv_append(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q_out=None), 1), (dict(k_cache=None), 1),
    (dict(v_cache=None), 1), (dict(inv_freq=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
    (dict(strides=None), 1),
    (dict(k=FAKE + 2), 2), (dict(v_cache=FAKE + 8), 2), (dict(block_table=FAKE + 1), 2), (dict(new_lens=FAKE + 2), 2),
    (dict(d=32), 4), (dict(B=0), 3), (dict(H=-1), 3), (dict(Hk=0), 3), (dict(T=-1), 3), (dict(rot=72), 3),
    (dict(rot=-16), 3), (dict(n_pages=0), 3), (dict(max_pages=0), 3), (dict(page_size=8), 3),
    (dict(page_size=48), 3), (dict(page_size=512), 3), (dict(interleaved=3), 3), (dict(B=1 << 20, T=1 << 12), 3),
    (dict(mag=math.nan), 9), (dict(strides=[64] * 9 + [0] * 9), 13), (dict(strides=[64] * 17 + [12]), 13),
    (dict(T=0), 0), (dict(T=0, q=None, k=None, v=None, q_out=None), 0),
])
def test_append_refusals(kw, code):
    assert call_append(**kw) == code


def test_append_optional_arguments_pass_the_checks():
    for kw in (dict(H=0, q=None, q_out=None), dict(rot=0, inv_freq=None)):
        assert call_append(**kw) not in (1, 2, 3, 4, 9, 13)


def call_paged(prefix=False, **kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, o=FAKE, lse=FAKE)
    if prefix:
        a.update(prefix_pages=FAKE, prefix_len=100)
    a.update(block_table=FAKE, seq_lens=FAKE, new_lens=None, strides=[64] * 6, B=2, H=4, Hk=2, T=1, d=64, n_pages=4,
             page_size=16, max_pages=2, scale=0.125)
    if not prefix:
        a.update(left=-1, right=0)
    a.update(workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return (fa.fa_fwd_prefix if prefix else fa.fa_fwd_paged)(*a.values())


COMMON = [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(k_cache=None), 1), (dict(block_table=None), 1),
    (dict(seq_lens=None), 1), (dict(workspace=None), 1), (dict(strides=None), 1),
    (dict(q=FAKE + 8), 2), (dict(workspace=FAKE + 4), 2), (dict(seq_lens=FAKE + 2), 2), (dict(new_lens=FAKE + 1), 2),
    (dict(d=256), 4), (dict(B=0), 3), (dict(H=3), 3), (dict(Hk=0), 3), (dict(T=-1), 3), (dict(page_size=17), 3),
    (dict(page_size=512), 3), (dict(n_pages=0), 3), (dict(max_pages=1 << 27), 3), (dict(B=1 << 20, T=1 << 12), 3),
    (dict(scale=0.0), 9), (dict(scale=math.nan), 9), (dict(strides=[64] * 5 + [4]), 13), (dict(strides=[0] * 6), 13),
    (dict(T=0), 0), (dict(T=0, q=None, o=None, lse=None, workspace=None), 0),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(left=-2), 3), (dict(right=-2), 3)])
def test_paged_refusals(kw, code):
    assert call_paged(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(prefix_len=0), 3), (dict(prefix_len=-1), 3), (dict(prefix_len=(1 << 30) + 1), 3),
    (dict(prefix_pages=None), 1), (dict(prefix_pages=FAKE + 2), 2)])
def test_prefix_refusals(kw, code):
    assert call_paged(prefix=True, **kw) == code


def test_workspace_size():
    small = fa.fa_paged_workspace_bytes(1, 1, 1, 1, 64, 0)
    assert small > 0 and small % 16 == 0
    assert fa.fa_paged_workspace_bytes(1, 1, 1, 1, 128, 0) > small
    with_prefix = fa.fa_paged_workspace_bytes(8, 4, 2, 3, 64, 10)
    assert with_prefix >= fa.fa_paged_workspace_bytes(8, 4, 2, 3, 64, 0) + 2 * 8 * 4 * 3 * 65 * 4
    for bad in ((0, 1, 1, 1, 64, 0), (1, 3, 2, 1, 64, 0), (1, 1, 1, 0, 64, 0), (1, 1, 1, 1, 96, 0), (1, 1, 1, 1, 64, -1)):
        assert fa.fa_paged_workspace_bytes(*bad) == 0


def test_python_entry_points_refuse_host_tensors_and_shapes():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, dtype=torch.float64)
    t = torch.zeros(1, 1, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: fa.rope(x, x, w), lambda: fa.rope_bwd(x, None, w),
              lambda: fa.kv_append(x, x, x, x, x, t, n, w), lambda: fa.fwd_paged(x, x, x, t, n),
              lambda: fa.fwd_prefix(x, x, x, n, 5, t, n)):
        with pytest.raises(TypeError):
            f()


def test_rope_freqs():
    w, mag = fa.rope_freqs(64, device="cpu")
    assert w.dtype == torch.float64 and w.shape == (32,) and mag == 1.0
    assert np.allclose(w.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    lin, _ = fa.rope_freqs(64, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(lin.numpy(), w.numpy() / 4, rtol=1e-14)
    base, _ = fa.rope_freqs(64, scaling="base", factor=4.0, device="cpu")
    assert base[0] == w[0] and math.isclose(float(base[-1]), float(w[-1]) / 4, rel_tol=1e-12)
    parts, m = fa.rope_freqs(64, scaling="by_parts", factor=4.0, original_len=4096, device="cpu")
    assert m == 0.1 * math.log(4.0) + 1.0
    turns = 4096 * w / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], w[turns >= 32])
    assert torch.allclose(parts[turns <= 1], w[turns <= 1] / 4, rtol=1e-14)
    between = (turns > 1) & (turns < 32)
    assert bool(between.any()) and bool(((parts < w) & (parts > w / 4))[between].all())
    for bad in (dict(rot=0), dict(rot=3), dict(rot=64, factor=0.5), dict(rot=64, scaling="other"),
                dict(rot=64, base=0.0), dict(rot=2, scaling="base", factor=2.0),
                dict(rot=64, scaling="by_parts", fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            fa.rope_freqs(device="cpu", **bad)


def test_reference_pins():
    """The tests' own 64-bit forms: 1 / (2 pi), a quarter turn, a plain softmax, a window."""
    assert math.isclose(float(ref.INV_2PI), 1 / (2 * math.pi), rel_tol=1e-15)
    y, _ = ref.rotate(np.array([[1.0, 0.0, 5.0]]), [1], [math.pi / 2], 2.0, True)
    assert np.allclose(y, [[0.0, 2.0, 5.0]])
    y, _ = ref.rotate(np.array([[1.0, 0.0, 5.0]]), [1], [math.pi / 2], 2.0, True, -1.0)
    assert np.allclose(y, [[0.0, -2.0, 5.0]])
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=(5, 4))
    o, lse, size = ref.attend(q, k, v, [0, 2, 4], [5, 3, 4], 0.5)
    p = np.exp(q[0] @ k.T * 0.5)
    assert np.allclose(o[0], p @ v / p.sum()) and np.isclose(lse[0], np.log(p.sum()))
    assert np.allclose(o[1], v[2]) and np.all(o[2] == 0) and np.isneginf(lse[2])


def test_python_entry_points_refuse_integers_past_the_c_types():
    """An offset, length or window reach that ctypes would cut to its low bits; a reach past 2^31 - 1 is an open side."""
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, dtype=torch.float64)
    t = torch.zeros(1, 1, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for bad in (2 ** 63, -2 ** 63 - 1, 2 ** 64):
        for f in (lambda: fa.rope(x, x, w, offset=bad), lambda: fa.rope_bwd(x, None, w, offset=bad),
                  lambda: fa.kv_append(x, x, x, x, x, t, n, w, offset=bad)):
            with pytest.raises(ValueError):
                f()
    for bad in ((-2 ** 31 - 1, 0), (0, -2 ** 32)):
        with pytest.raises(ValueError):
            fa.fwd_paged(x, x, x, t, n, window=bad)
    for wide in ((2 ** 31, 0), (2 ** 64, 2 ** 40)):  # no refusal of these: the host tensors are what stops the call
        with pytest.raises(TypeError):
            fa.fwd_paged(x, x, x, t, n, window=wide)
    from exact_attention_19_gb300 import serving

    assert [serving._reach("", v) for v in (-1, 0, 7, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5)] == [-1, 0, 7] + [2 ** 31 - 1] * 3
    for bad in (2 ** 31, 2 ** 32 + 8):
        with pytest.raises(ValueError):
            serving._c_int("prefix_len", bad, 32)


@pytest.fixture
def toy_build(tmp_path, monkeypatch):
    """build() on compilers that write a word, into a folder of its own."""
    source = tmp_path / "source"
    source.write_text("x")

    def toy(word):
        return lambda out, *_: ["sh", "-c", f"echo {word} > {out}"]

    monkeypatch.setattr(fa_build, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(fa_build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(fa_build, "torch_lib_path", lambda: str(tmp_path / "torch.so"))
    monkeypatch.setattr(fa_build, "DEPS", [str(source)])
    monkeypatch.setattr(fa_build, "TORCH_DEPS", [str(source)])
    monkeypatch.setattr(fa_build, "command", toy("lib"))
    monkeypatch.setattr(fa_build, "torch_command", toy("torch"))
    return tmp_path


def test_build_puts_both_libraries_in_place(toy_build):
    fa_build.build(strict=True)
    assert sorted(f.name for f in toy_build.iterdir()) == ["lib.so", "source", "torch.so"]
    assert not fa_build.needs_build()


def test_build_of_the_c_library_needs_no_torch(toy_build, monkeypatch, capfd):
    """Without torch, with a torch that does not load, without a host compiler and with one that fails:
    libfa_gb300.so is built, a note or (strict) an error says what is missing."""
    def missing(out):
        raise ImportError("No module named 'torch'")

    def broken(out):
        raise OSError("libtorch.so: cannot open shared object file")

    for torch_command, word in ((missing, "torch"), (broken, "libtorch"), (lambda out: ["/no/such/compiler"], "compiler"),
                                (lambda out: ["sh", "-c", "echo no header >&2; exit 1"], "no header")):
        monkeypatch.setattr(fa_build, "torch_command", torch_command)
        fa_build.build(force=True)
        assert word in capfd.readouterr().err
        assert sorted(f.name for f in toy_build.iterdir()) == ["lib.so", "source"]
        (toy_build / "lib.so").unlink()
        with pytest.raises(RuntimeError, match=word):
            fa_build.build(strict=True)
        assert (toy_build / "lib.so").read_text() == "lib\n"


def test_build_reports_a_failing_c_library(toy_build, monkeypatch):
    monkeypatch.setattr(fa_build, "command", lambda out, *_: ["sh", "-c", "echo bad kernel >&2; exit 2"])
    with pytest.raises(RuntimeError, match="bad kernel"):
        fa_build.build()
    assert not (toy_build / "lib.so").exists() and (toy_build / "torch.so").exists()


def test_the_torch_module_belongs_to_one_torch(monkeypatch):
    """Another torch, ABI or Python has another file, so a module compiled for an earlier one counts as missing."""
    import sysconfig

    fa_build.build()
    here = fa_build.torch_lib_path()
    assert not fa_build.needs_build() and torch.__version__ in here and sysconfig.get_config_var("SOABI") in here
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert fa_build.torch_lib_path() != here and fa_build.needs_build()
    from exact_attention_19_gb300 import serving

    with pytest.raises(ImportError, match="build it"):
        serving._load_native()


def test_needs_build_without_torch(toy_build, monkeypatch):
    def missing():
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(fa_build, "torch_lib_path", missing)
    assert fa_build.needs_build()
    fa_build.build()
    assert not fa_build.needs_build()
