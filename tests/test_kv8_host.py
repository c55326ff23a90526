"""The paged 8-bit cache without a GPU: the 64-bit oracle against first
principles, and the host's refusals (before any device work)."""
import ctypes

import numpy as np
import pytest

from tests import kv8_reference as R


@pytest.fixture(scope="module")
def lib():
    from decoder_only_transformer_02_b200 import build, gpt2
    build.build()
    return gpt2.load_library()


GOOD = dict(format=0, n_layer=2, n_kv_head=3, head_dim=64, page_size=16, num_pages=8, num_slots=4, max_pages=4,
            d_codes=4096, d_scales=4096, d_table=4096, d_lens=4096, d_refs=4096)


def cache(**kw):
    from decoder_only_transformer_02_b200 import gpt2 as G
    v = dict(GOOD, **kw)
    return G._KV8(*[v[n] for n, _ in G._KV8._fields_])


@pytest.mark.parametrize("bad", [
    dict(format=2), dict(format=-1), dict(n_layer=0), dict(n_kv_head=0), dict(n_kv_head=1025), dict(head_dim=96),
    dict(page_size=24), dict(page_size=256), dict(num_pages=0), dict(num_pages=(1 << 24) + 1), dict(num_slots=65537),
    dict(num_slots=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(d_codes=4104), dict(d_refs=4100),
    dict(d_codes=None), dict(d_scales=None), dict(d_table=None), dict(d_lens=None), dict(d_refs=None),
])
def test_bad_caches_are_refused(lib, bad):
    p = ctypes.byref(cache(**bad))
    x = 4096
    assert lib.gpt2_kv8_workspace_bytes(p, 1) == 0
    assert lib.gpt2_kv8_attention_workspace_bytes(p, 3, 1, 1, 1) == 0
    assert lib.gpt2_kv8_resize(p, x, x, 1, x, 1 << 30, None) == -1
    assert lib.gpt2_kv8_fork(p, x, x, 1, x, 1 << 30, None) == -1
    assert lib.gpt2_kv8_compact(p, None, x, 1 << 30, None) == -1
    assert lib.gpt2_kv8_append(p, 0, x, x, 192, x, x, 1, 1, None) == -1
    assert lib.gpt2_kv8_attention(p, 0, x, 192, x, 192, None, 3, x, x, 1, 1, 1, x, 1 << 30, None) == -1


def test_bad_arguments_are_refused(lib):
    p, x, big = ctypes.byref(cache()), 4096, 1 << 30
    assert lib.gpt2_kv8_workspace_bytes(p, 1) > 0
    assert lib.gpt2_kv8_workspace_bytes(p, 4097) == 0 and lib.gpt2_kv8_workspace_bytes(p, -1) == 0
    need = lib.gpt2_kv8_workspace_bytes(p, 5)
    for args in [(None, x, 5, x, big), (x, None, 5, x, big), (x, x, -1, x, big), (x, x, 4097, x, big),
                 (x, x, 5, None, big), (x, x, 5, x, need - 1), (x, x, 5, x + 8, big)]:
        assert lib.gpt2_kv8_resize(p, *args, None) == -1
        assert lib.gpt2_kv8_fork(p, *args, None) == -1
    assert lib.gpt2_kv8_compact(p, None, None, big, None) == -1
    assert lib.gpt2_kv8_compact(p, None, x, 15, None) == -1
    good = dict(layer=0, k=x, v=x, ld=192, slots=x, cu=x, n=1, rows=1)
    for bad in [dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(k=x + 8), dict(v=x + 2), dict(ld=184),
                dict(ld=196), dict(slots=None), dict(cu=None), dict(n=-1), dict(n=4097), dict(rows=-1),
                dict(rows=(1 << 30) + 1)]:
        a = dict(good, **bad)
        assert lib.gpt2_kv8_append(p, *a.values(), None) == -1, bad
    good = dict(layer=0, q=x, ldq=384, out=x, ldo=384, lse=None, heads=6, slots=x, cu=x, n=1, rows=1, max_q=1, work=x, bytes=big)
    for bad in [dict(layer=2), dict(q=None), dict(out=None), dict(q=x + 8), dict(out=x + 8), dict(ldq=376), dict(ldo=376),
                dict(ldq=388), dict(heads=0), dict(heads=5), dict(heads=65 * 3), dict(max_q=0), dict(n=4097),
                dict(rows=-1), dict(work=None), dict(work=x + 4), dict(bytes=0), dict(slots=None), dict(cu=None)]:
        a = dict(good, **bad)
        assert lib.gpt2_kv8_attention(p, *a.values(), None) == -1, bad
    for args in [(0, 1, 1, 1), (5, 1, 1, 1), (195, 1, 1, 1), (3, -1, 1, 1), (3, 4097, 1, 1), (3, 1, -1, 1), (3, 1, 1, 0)]:
        assert lib.gpt2_kv8_attention_workspace_bytes(p, *args) == 0, args


def test_oracle_rounding():
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.05, 0.05, 20001)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.nearest(x, R.E4M3), want)
    assert list(R.nearest(np.array([0.5, 1.5, 2.5, -0.5, -1.5]), R.INT8)) == [0, 2, 2, 0, -2]
    for fmt in (R.INT8, R.E4M3):
        assert R.scale_for(0.0, fmt) == 2.0 ** -126
        assert R.scale_for(R.QMAX[fmt], fmt) == 1.0 and R.scale_for(R.QMAX[fmt] * 1.001, fmt) == 2.0


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_oracle_append_and_attention_against_dense(fmt):
    """Appended in pieces, values stay within a rounding of what came in (half a
    step of the block's last scale for int8, 2^-4 relative or half the smallest
    step for e4m3, and once more for each growth), and attention over them is the
    dense softmax."""
    rng = np.random.default_rng(0)
    c = R.Cache(fmt, 1, 2, 64, 16, 20, 3, 8)
    x = rng.standard_normal((2, 50, 2, 64)).astype(np.float32).astype(np.float64)
    at = 0
    for m in (5, 1, 1, 30, 13):
        c.resize([1], [at + m])
        c.append(0, x[0, at:at + m], x[1, at:at + m], [1], [0, m])
        at += m
    k, v = c.values(0, 1)
    step = c.scales[c.table[1, :4], 0].repeat(16, 0)[:50]  # [50, 2, kvh]
    for side, got in enumerate((k, v)):
        s = step[:, side, :, None]
        tol = 2 * 0.5 * s if fmt == R.INT8 else 2 * np.maximum(2.0 ** -4 * np.abs(x[side]), 2.0 ** -10 * s)
        assert np.all(np.abs(got - x[side]) <= tol)
    q = rng.standard_normal((3, 4, 64))
    out, lse, _, _ = c.attention(0, q, [1], [0, 3])
    for r in range(3):
        for h in range(4):
            z = k[:48 + r, h // 2] @ q[r, h] / 8
            w = np.exp(z)
            np.testing.assert_allclose(out[r, h], w @ v[:48 + r, h // 2] / w.sum(), rtol=1e-10)
            np.testing.assert_allclose(lse[r, h], np.log(w.sum()), rtol=1e-10)


def test_oracle_table_counts_stay_consistent():
    """refs counts the table's entries after any run of calls."""
    rng = np.random.default_rng(1)
    c = R.Cache(R.INT8, 1, 1, 64, 16, 30, 6, 6)
    for _ in range(300):
        try:
            w = rng.integers(0, 3)
            if w == 0:
                s = [int(i) for i in rng.permutation(6)[:3]]
                c.resize(s, [int(rng.integers(0, 97)) for _ in s])
            elif w == 1:
                d = [int(i) for i in np.flatnonzero(c.lens == 0)[:2]]
                c.fork([int(rng.integers(0, 6)) for _ in d], d)
            else:
                live = c.compact()
                assert np.all(c.refs[:live] > 0) and np.all(c.refs[live:] == 0)
        except R.Refused:
            pass
        count = np.zeros(30, int)
        for s in range(6):
            for j in range(c.pages(c.lens[s])):
                count[c.table[s, j]] += 1
                if (j + 1) * 16 > c.lens[s]:
                    assert c.refs[c.table[s, j]] == 1  # an unfinished page is never shared
        np.testing.assert_array_equal(count, c.refs)
