"""The paged 8-bit key/value cache (gpt2_kv8_*) through the C ABI against the
64-bit form in tests/kv8_reference.py.

Codes, scales, tables and counts have to be equal: scales are powers of two, so
x / scale is exact and a code is one rounding.

Attention tolerances.  The output is a bf16 rounding (2^-8 relative) of
sum p_t v_t / sum p_t.  The weights are rounded to half precision or better
before they meet the values (2^-11 each), and a score that is off by ds changes
its weight by about ds; the fp32 dot products over d terms are off by at most
d 2^-24 sum|q||k| / sqrt(d), with the scale and exponent about twice that.  So
|out - ref| <= 2^-8 |ref| + (2^-11 + 2 ds + 2^-14) sum p|v| + T 2^-30 max|v| and
|lse - ref| <= ds + 2^-20 (1 + |ref|).
The last term of the first: a weight so small that its type holds it only to a
fixed step.  In half precision the step is 2^-24; the weights are held as
2^6 p vs / (the largest vs), p relative to the row's maximum, so each is off by
at most 2^-25 2^-6 (largest vs) / vs, and its token's value, of at most
vs qmax, adds 2^-31 (largest vs) qmax <= 2^-30 max|v| over the T tokens seen
(a power-of-two scale times qmax is below twice the block's largest value).
In single precision the same argument gives less (weights below 2^-126 vanish)."""
import numpy as np
import pytest

from tests import kv8_reference as R
from tests.gpu_util import bf16_round, need_gpu, torch

pytestmark = pytest.mark.gpu

FMTS = [R.INT8, R.E4M3]


def _g():
    need_gpu()
    from decoder_only_transformer_02_b200 import gpt2 as G
    return G


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32).reshape(-1), device="cuda")


class Pair:
    """The device's cache and the reference's, taken through the same calls."""

    def __init__(self, fmt, layers=1, kvh=2, d=64, ps=16, num_pages=40, num_slots=8, max_pages=16, seed=0, device="cuda"):
        self.G = _g()
        self.G.check_device_error()
        self.ref = R.Cache(fmt, layers, kvh, d, ps, num_pages, num_slots, max_pages)
        self.dev = self.G.KV8Cache.allocate(fmt, layers, kvh, d, ps, num_pages, num_slots, max_pages, device=device)
        # what no token uses may hold anything: NaN codes (e4m3) and NaN scales
        self.dev.codes.view(torch.uint8).fill_(0x7f)
        self.dev.scales.fill_(float("nan"))
        self.ref.codes[:] = 127 if fmt == R.INT8 else np.nan
        self.ref.scales[:] = np.nan
        self.work = torch.empty(self.dev.workspace_bytes(4096), dtype=torch.uint8, device=device)
        self.rng = np.random.default_rng(seed)

    def resize(self, slots, new, ok=True):
        self._both(lambda: self.ref.resize(slots, new), lambda: self.dev.resize(_i32(slots), _i32(new), self.work), ok)

    def fork(self, src, dst, ok=True):
        self._both(lambda: self.ref.fork(src, dst), lambda: self.dev.fork(_i32(src), _i32(dst), self.work), ok)

    def compact(self):
        live = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = self.ref.compact()
        self.dev.compact(self.work, live=live)
        self.G.check_device_error()
        assert int(live) == want
        self.same()

    def _both(self, ref, dev, ok):
        if ok:
            ref()
            dev()
            self.G.check_device_error()
        else:
            with pytest.raises(R.Refused):
                ref()
            dev()
            with pytest.raises(self.G.GPT2Error) as e:
                self.G.check_device_error()
            assert e.value.name == "ECACHE"
        self.same()

    def same(self):
        """lens, refs, used table entries, and codes and scales of the tokens held."""
        ref, dev = self.ref, self.dev
        np.testing.assert_array_equal(dev.lens.cpu().numpy(), ref.lens)
        np.testing.assert_array_equal(dev.refs.cpu().numpy(), ref.refs)
        table = dev.table.cpu().numpy()
        codes, scales = dev.codes.float().cpu().numpy(), dev.scales.cpu().numpy()
        for s in range(ref.num_slots):
            used = ref.pages(ref.lens[s])
            np.testing.assert_array_equal(table[s, :used], ref.table[s, :used])
            for j in range(used):
                p, m = ref.table[s, j], min(ref.ps, ref.lens[s] - j * ref.ps)
                np.testing.assert_array_equal(scales[p], ref.scales[p])
                np.testing.assert_array_equal(codes[p][..., :m, :], ref.codes[p][..., :m, :])

    def append(self, slots, news, size=1.0, pad=0, mutate=None):
        """news[i] more tokens for slots[i] in every layer, out of one fused buffer."""
        ref, dev = self.ref, self.dev
        self.resize(slots, [int(ref.lens[s] + n) for s, n in zip(slots, news)])
        cu = np.concatenate([[0], np.cumsum(news)]).astype(int)
        w = ref.kvh * ref.d
        for layer in range(ref.layers):
            x = bf16_round(self.rng.standard_normal((cu[-1] + pad, 3 * w)) *
                           size * 2.0 ** self.rng.integers(-2, 3, (cu[-1] + pad, 1)))
            if mutate:
                mutate(x[:, w:])
            buf = torch.from_numpy(x).to(torch.bfloat16).cuda()
            shape = (-1, ref.kvh, ref.d)
            dev.append(layer, buf[:, w:2 * w].unflatten(1, shape[1:]), buf[:, 2 * w:].unflatten(1, shape[1:]), _i32(slots), _i32(cu))
            ref.append(layer, x[:cu[-1], w:2 * w].reshape(shape), x[:cu[-1], 2 * w:].reshape(shape), slots, cu)
        self.G.check_device_error()
        self.same()

    def attention(self, slots, news, group=1, pad=0, size=1.0, layer=0, max_q=None, stream=None):
        ref, dev = self.ref, self.dev
        cu = np.concatenate([[0], np.cumsum(news)]).astype(int)
        rows, heads, d = int(cu[-1]) + pad, ref.kvh * group, ref.d
        q = bf16_round(self.rng.standard_normal((rows, heads + 1, d)) * size)
        dq = torch.from_numpy(q).to(torch.bfloat16).cuda()[:, :heads]  # a row stride of its own
        out = torch.full((rows, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, heads), 7.0, dtype=torch.float32, device="cuda")
        max_q = max_q or max(max(news), 1)
        work = torch.full((dev.attention_workspace_bytes(heads, len(slots), rows, max_q),), 0xff, dtype=torch.uint8, device="cuda")
        dev.attention(layer, dq, out, _i32(slots), _i32(cu), max_q, work, lse=lse)
        self.G.check_device_error()
        want, wl, mag, top = ref.attention(layer, q[:cu[-1], :heads], slots, cu)
        tiny = np.zeros(want.shape)
        for i, s in enumerate(slots):
            v = np.abs(ref.values(layer, s)[1]) if ref.lens[s] else np.zeros((1, ref.kvh, d))
            tiny[cu[i]:cu[i + 1]] = 2.0 ** -30 * len(v) * v.max((0, 2)).repeat(group)[:, None]
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(got[cu[-1]:] == 7.0) and np.all(gl[cu[-1]:] == 7.0)
        ds = 2 * d * 2.0 ** -24 * top
        err = np.abs(got[:cu[-1]] - want)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * ds[..., None] + 2.0 ** -14) * mag + tiny
        over = float(np.max(err - bound)) if err.size else 0.0
        assert over <= 0, over
        over = float(np.max(np.abs(gl[:cu[-1]] - wl) - ds - 2.0 ** -20 * (1 + np.abs(wl)))) if wl.size else 0.0
        assert over <= 0, over
        return out, lse


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps,kvh", [(64, 16, 3), (64, 128, 1), (128, 16, 2), (128, 64, 5), (64, 32, 9)])
def test_append_codes_and_scales(fmt, d, ps, kvh):
    p = Pair(fmt, layers=2, kvh=kvh, d=d, ps=ps, num_pages=30, max_pages=12, seed=d + ps)
    p.append([3, 0], [5, ps + 7])
    p.append([0, 3, 7], [1, ps - 5, 2 * ps], size=3.0, pad=2)  # 3 ends at a page's end
    p.append([3, 7], [1, 1], size=0.01)
    p.append([3, 7, 0, 1], [1, 0, 1, 1], size=50.0)            # scales grow, an entry without rows
    for _ in range(3):
        p.append([0, 1, 3, 7], [1, 1, 1, 1], size=2.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_extreme_values(fmt):
    """Zeros, the largest bf16, subnormals, borders of the range and what is not finite."""
    p = Pair(fmt, kvh=1, ps=16)

    def put(values):
        def mutate(x):
            x[:] = 0
            x.reshape(-1)[:len(values)] = values
        return mutate

    qmax = R.QMAX[fmt]
    border = [bf16_round(np.array([qmax]))[0], -1.0, 0.5, 1.5, 2.5]
    for s, vals in enumerate([[0.0], [2.0 ** 127, 2.0 ** 126], [2.0 ** -133, 2.0 ** -130], border,
                              [0.5, 3.3895313892515355e38]]):
        p.append([s], [3], mutate=put(vals))
        p.append([s], [1], mutate=put([2.0 ** -3]))
    p.append([5], [3], mutate=put([1.0, np.inf]))
    p.append([6], [3], mutate=put([1.0, 2.0]))
    p.append([6], [1], mutate=put([np.nan]))
    p.append([6], [1], mutate=put([1.0]))
    assert np.isnan(p.ref.scales[p.ref.table[6, 0]]).any()


def test_append_refusals_leave_the_cache():
    G = _g()
    p = Pair(R.INT8)
    p.append([0, 1], [20, 5])
    before = p.dev.codes.clone()
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")

    def refused(slots, cu):
        p.dev.append(0, k, k, _i32(slots), _i32(cu))
        with pytest.raises(G.GPT2Error) as e:
            G.check_device_error()
        assert e.value.name == "ECACHE"
        assert torch.equal(before, p.dev.codes)

    refused([8], [0, 2])          # no such slot
    refused([-1], [0, 2])
    refused([2], [0, 2])          # an empty slot
    refused([0, 1], [0, 2, 5])    # more rows than there are
    refused([0, 1], [2, 1, 3])    # offsets that decrease
    refused([0], [-1, 3])
    p.dev.table[1, 0] = 40        # a page id past the pool
    refused([1], [0, 1])
    p.dev.table[1, 0] = -1
    refused([1], [0, 1])
    p.dev.lens[1] = 16 * 16 + 1   # longer than a slot can be
    refused([1], [0, 1])


def test_append_slot_named_twice():
    """The first entry is written, the later one refused."""
    G = _g()
    p = Pair(R.INT8)
    p.append([0], [3])
    k = torch.full((2, 2, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    k[1] = 2.0
    p.dev.append(0, k, k, _i32([0, 0]), _i32([0, 1, 2]))
    with pytest.raises(G.GPT2Error):
        G.check_device_error()
    p.ref.append(0, np.full((1, 2, 64), 1.0), np.full((1, 2, 64), 1.0), [0], [0, 1])
    p.same()


# --------------------------------------------------------------- attention
CASES = [
    # lens, new rows, group, pad
    ([1], [1], 1, 0),
    ([1, 16, 17, 33], [1, 1, 1, 1], 1, 3),
    ([2, 5], [0, 5], 2, 0),
    ([100, 7, 255], [1, 1, 1], 4, 1),
    ([40, 200, 3], [3, 1, 3], 1, 0),
    ([250, 31], [9, 31], 3, 0),
    ([256, 130], [130, 129], 1, 0),
    ([77, 78, 5], [40, 0, 2], 8, 2),
    ([200], [1], 64, 0),
    ([33], [2], 40, 0),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 16), (64, 64), (128, 128)])
@pytest.mark.parametrize("room", [256, 8192])  # tokens a slot may hold: tiles whole, or cut into parts
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(fmt, d, ps, case, room):
    lens, news, group, pad = CASES[case]
    p = Pair(fmt, layers=2, kvh=1 if group > 4 else 3, d=d, ps=ps, num_pages=50, max_pages=room // ps, seed=case)
    slots = [5, 0, 3, 7][:len(lens)]
    p.append([6], [19])               # so that the pages of the others are not 0, 1, ...
    p.append(slots, [max(0, t - n - 9) for t, n in zip(lens, news)])
    p.append([6], [40], size=3.0)
    p.append(slots[::-1], [t - int(p.ref.lens[s]) for s, t in zip(slots, lens)][::-1])
    for layer in (0, 1):
        p.attention(slots, news, group, pad, layer=layer)


PROMPTS = [
    # lens, new rows, group: more than 64 rows per key/value head
    ([65], [65], 1),
    ([128, 129, 300], [128, 129, 300], 1),
    ([700, 1, 40, 513], [257, 1, 40, 130], 1),   # prompts, a single token and a few tokens in one call
    ([1000, 90], [33, 3], 8),                    # rows of one token in two tiles
    ([500, 300], [100, 299], 3),
    ([70], [2], 40),
    ([1100], [600], 1),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_attention_of_prompts(fmt, d, ps, case):
    lens, news, group = PROMPTS[case]
    p = Pair(fmt, layers=2, kvh=2, d=d, ps=ps, num_pages=150, max_pages=1200 // ps + 1, seed=100 + case)
    slots = [5, 0, 3, 7][:len(lens)]
    p.append([6], [19])
    p.append(slots, [t // 2 for t in lens], size=2.0)
    p.append(slots[::-1], [t - t // 2 for t in lens][::-1], size=0.7)
    p.attention(slots, news, group, pad=2, layer=1)
    p.attention(slots, news, group, layer=0, max_q=1200)  # max_q may be more than any sequence has


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_long(fmt, d):
    """One long sequence and short ones: the work of one is split over many blocks."""
    p = Pair(fmt, kvh=2, d=d, ps=64, num_pages=140, max_pages=128)
    p.append([2, 1, 4], [7001, 300, 1])
    p.append([2], [1], size=6.0)
    p.attention([1, 2, 4], [1, 1, 1], group=2)
    p.attention([2, 4], [5, 1], group=1, pad=1)
    p.attention([2], [40], group=2, size=2.0)
    p.attention([2, 1], [70, 300], group=1)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_prompts_and_cut_tiles(fmt, d):
    """Prompts and few rows in one call, both cut over the tokens: joined together."""
    p = Pair(fmt, kvh=2, d=d, ps=64, num_pages=260, max_pages=80)
    p.append([2, 1, 4, 0], [5001, 300, 4100, 2077])
    p.append([2], [60], size=3.0)
    p.attention([2, 1, 4, 0], [60, 1, 150, 9], group=1, pad=1)
    p.attention([4, 0, 2], [33, 7, 1], group=2)
    p.attention([0, 2, 4], [0, 3, 1], group=3, max_q=500)  # few rows where max_q allows a prompt
    p.attention([2], [2], group=1, max_q=500)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("room", [32, 256])
def test_attention_scales_far_apart(fmt, room):
    """Pages whose values differ by many powers of two, scores far apart and
    far from zero, and queries with large and tiny components."""
    p = Pair(fmt, kvh=2, ps=16, num_pages=60, max_pages=room)
    for i, size in enumerate([1e-6, 1.0, 300.0, 1e-3, 5.0]):
        p.append([0, 1], [33, 16], size=size)
    for size in (0.01, 1.0, 0.3):
        p.attention([0, 1], [1, 2], group=2, size=size)
    for i in range(3):
        p.append([2], [40], size=1e-20)
    p.attention([2], [3], size=1e15)
    p.attention([2], [3], size=1e-15)
    for size in (0.01, 1.0):
        p.attention([0, 1], [70, 66], group=1, size=size)


def test_attention_equal_scores_and_zero_values():
    p = Pair(R.E4M3, kvh=1, ps=16)

    def zero(x):
        x[:] = 0
    p.append([0], [70], mutate=zero)
    for rows in (2, 70):
        out, lse = p.attention([0], [rows])
        assert torch.all(out == 0)


def test_attention_nan_block_reaches_its_readers_only():
    """A block with a value that is not finite makes NaN of the rows that see
    its page, and of no other sequence."""
    p = Pair(R.INT8, kvh=2, ps=16)
    p.append([0, 1], [40, 40])

    def bad(x):
        x[0, :64] = np.nan  # keys of head 0
    p.append([0], [1], mutate=bad)
    out = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones_like(out)
    work = torch.empty(p.dev.attention_workspace_bytes(2, 2, 2, 1), dtype=torch.uint8, device="cuda")
    p.dev.attention(0, q, out, _i32([0, 1]), _i32([0, 1, 2]), 1, work)
    p.G.check_device_error()
    assert torch.isnan(out[0, 0]).all() and not torch.isnan(out[0, 1]).any() and not torch.isnan(out[1]).any()
    # in values too, and with many rows: those before the block do not see it
    p.append([2], [100])

    def bad_value(x):
        x[0, 128:192] = np.inf  # values of head 0
    p.append([2], [20], mutate=bad_value)  # positions 100 .. 119, in the pages from 96
    for rows in (40, 90):
        out = torch.zeros(rows, 2, 64, dtype=torch.bfloat16, device="cuda")
        q = torch.ones_like(out)
        work = torch.empty(p.dev.attention_workspace_bytes(2, 1, rows, rows), dtype=torch.uint8, device="cuda")
        p.dev.attention(0, q, out, _i32([2]), _i32([0, rows]), rows, work)
        p.G.check_device_error()
        sees = torch.arange(120 - rows, 120, device="cuda") >= 96
        assert torch.equal(torch.isnan(out[:, 0]).all(-1), sees) and torch.equal(torch.isnan(out[:, 0]).any(-1), sees)
        assert not torch.isnan(out[:, 1]).any()


@pytest.mark.parametrize("room", [16, 256])
def test_attention_refusals(room):
    G = _g()
    p = Pair(R.INT8, max_pages=room)
    p.append([0, 1], [20, 50])
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    work = torch.empty(p.dev.attention_workspace_bytes(2, 4, 4, 4), dtype=torch.uint8, device="cuda")

    def refused(slots, cu, max_q=4, left=slice(None)):
        out.fill_(7.0)
        p.dev.attention(0, q, out, _i32(slots), _i32(cu), max_q, work)
        with pytest.raises(G.GPT2Error) as e:
            G.check_device_error()
        assert e.value.name == "ECACHE"
        assert torch.all(out[left] == 7.0)

    refused([8], [0, 2])
    refused([-3], [0, 2])
    refused([2], [0, 1])                          # an empty slot
    refused([0, 1], [0, 2, 5])                    # more rows than there are
    refused([0, 1], [2, 1, 3])                    # offsets that decrease
    refused([0, 2], [0, 1, 2], left=slice(1, 4))  # the good sequence's row is written
    refused([0], [0, 3], max_q=2)                 # more rows than max_q says
    saved = p.dev.table.clone()
    for page in (-1, 40, 2 ** 31 - 1):
        p.dev.table[1, 2] = page
        p.dev.attention(0, q, out, _i32([1, 0]), _i32([0, 1, 2]), 1, work)
        with pytest.raises(G.GPT2Error) as e:
            G.check_device_error()
        assert e.value.name == "ECACHE"
    p.dev.table.copy_(saved)
    p.attention([0, 1], [1, 1])


# ------------------------------------------------------- resize, fork, compact
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_random_calls(fmt, seed):
    """A long run of random calls; the whole state compared after each."""
    p = Pair(fmt, layers=2, kvh=1, ps=16, num_pages=37, num_slots=9, max_pages=8, seed=seed)
    rng = p.rng
    for step in range(60):
        what = rng.integers(0, 6)
        lens = p.ref.lens
        free = int((p.ref.refs == 0).sum())
        if what <= 1:
            slots = list(rng.permutation(9)[:rng.integers(1, 5)])
            news = [int(rng.integers(0, min(30, 128 - lens[s]) + 1)) for s in slots]
            need = sum(p.ref.pages(lens[s] + n) - p.ref.pages(lens[s]) for s, n in zip(slots, news))
            if need <= free:
                p.append([int(s) for s in slots], news)
        elif what == 2:
            slots = [int(s) for s in rng.permutation(9)[:rng.integers(1, 9)]]
            new = [int(rng.integers(0, lens[s] + 1)) for s in slots]
            if free >= len(slots):
                p.resize(slots, new)
        elif what == 3:
            dst = [int(s) for s in np.flatnonzero(lens == 0)]
            src = [int(rng.choice(np.flatnonzero(lens > 0))) for _ in dst] if lens.any() else []
            dst = dst[:len(src)]
            if free >= len(dst):
                p.fork(src, dst)
        elif what == 4:
            p.compact()
        else:
            have = [int(s) for s in np.flatnonzero(lens > 0)]
            if have:
                p.attention(have, [int(rng.integers(0, min(4, lens[s]) + 1)) for s in have], group=2)
    p.compact()


def test_resize_truncation_copies_a_shared_page():
    p = Pair(R.INT8, ps=16)
    p.append([0], [45])
    p.fork([0, 0], [1, 2])
    p.resize([0, 1], [20, 20])       # both cut into the shared second page: both copy it
    p.append([0, 1, 2], [5, 6, 7])
    p.resize([2, 1, 0], [0, 16, 17])
    p.attention([0, 1], [1, 1])


def test_table_calls_refused_as_a_whole():
    p = Pair(R.INT8, num_pages=6, max_pages=4, num_slots=5)
    p.append([0, 1], [30, 40])       # 2 + 3 pages of 6
    for slots, new in [([0, 5], [31, 1]), ([0, 0], [31, 32]), ([-1], [1]), ([0], [65]), ([0], [-1]),
                       ([2, 3], [16, 16]), ([0, 2], [16, 49])]:
        p.resize(slots, new, ok=False)
    p.resize([0, 2], [16, 32])       # a page given back serves the same call
    p.resize([2], [0])
    for src, dst in [([0], [1]), ([0, 1], [3, 3]), ([0], [5]), ([7], [3]), ([0, 3], [3, 4]), ([3], [3]), ([-1], [3])]:
        p.fork(src, dst, ok=False)
    p.fork([0], [3])                 # length 16: nothing to copy
    p.fork([1], [4])
    p.resize([2], [1])
    p.resize([3], [0])
    p.fork([1], [3], ok=False)       # no free page for the copy
    p.compact()


def test_table_entries_outside_the_pool_are_passed_over():
    """Recorded, and neither read nor counted; the partly kept page is checked before anything changes."""
    G = _g()

    def run(page, call):
        p = Pair(R.INT8)
        p.append([0, 1], [40, 33])
        p.dev.table[0, 1] = page
        before = [t.clone() for t in (p.dev.refs, p.dev.lens, p.dev.table)]
        call(p)
        with pytest.raises(G.GPT2Error) as e:
            G.check_device_error()
        assert e.value.name == "ECACHE"
        return before, (p.dev.refs, p.dev.lens, p.dev.table)

    for page in (-1, 40, 1 << 30):
        old, new = run(page, lambda p: p.dev.resize(_i32([0]), _i32([25]), p.work))
        assert all(torch.equal(a, b) for a, b in zip(old, new))
        old, new = run(page, lambda p: p.dev.resize(_i32([0]), _i32([0]), p.work))
        assert new[1][0] == 0 and new[0].sum() == old[0].sum() - 2
        old, new = run(page, lambda p: p.dev.fork(_i32([0]), _i32([2]), p.work))
        assert new[1][2] == 40 and new[0].sum() == old[0].sum() + 2
        old, new = run(page, lambda p: p.dev.compact(p.work))
        assert torch.equal(old[1], new[1]) and new[2][0, 1] == page and new[0].sum() == old[0].sum()


def test_lengths_whose_pages_pass_32_bits_are_refused():
    """2^23 pages wanted by each of 256 slots: as a whole, changing nothing."""
    G = _g()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    c = G.KV8Cache.allocate(R.INT8, 1, 1, 64, 16, 20, 300, 1)
    big = G.KV8Cache(c.codes, c.scales, torch.empty(300, 1 << 23, dtype=torch.int32, device="cuda"), c.lens, c.refs)
    work = torch.empty(big.workspace_bytes(300), dtype=torch.uint8, device="cuda")
    slots = _i32(range(300))
    for n in (255, 256, 300):
        big.resize(slots[:n], _i32([16 << 23] * n), work)
        with pytest.raises(G.GPT2Error) as e:
            G.check_device_error()
        assert e.value.name == "ECACHE"
        assert torch.all(c.refs == 0) and torch.all(c.lens == 0)


@pytest.mark.parametrize("pages,taken", [(30011, 20003), (70001, 65531), (16384 + 5000, 16383), (100000, 3)])
def test_pools_larger_than_one_scan(pages, taken):
    """Free pages far into the pool, more entries than one block has threads."""
    G = _g()
    n = 2500
    c = G.KV8Cache.allocate(R.INT8, 1, 1, 64, 16, pages, 5000, 4)
    work = torch.empty(c.workspace_bytes(n), dtype=torch.uint8, device="cuda")
    c.refs[:taken] = 1
    slots = torch.randperm(5000)[:n].int().cuda()
    lens = (torch.arange(n, dtype=torch.int32) % 41).cuda()
    c.resize(slots, lens, work)
    G.check_device_error()
    used = (lens + 15) // 16
    first = used.cumsum(0) - used
    for j in range(4):
        want = torch.where(used > j, taken + first + j, -1).int()
        assert torch.equal(c.table[slots.long(), j], want)
    total = int(used.sum())
    assert torch.all(c.refs[taken:taken + total] == 1) and torch.all(c.refs[taken + total:] == 0)
    c.refs[:taken] = 0
    c.codes.view(torch.uint8)[:] = (torch.arange(pages, device="cuda") % 251).to(torch.uint8).view(-1, 1, 1, 1, 1, 1)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = c.table.clone()
    c.compact(work, live=live)
    G.check_device_error()
    assert int(live) == total and torch.all(c.refs[:total] == 1) and torch.all(c.refs[total:] == 0)
    ids = c.table[slots.long()]
    at = ids >= 0
    assert torch.equal(torch.sort(ids[at]).values, torch.arange(total, device="cuda", dtype=torch.int32))
    assert torch.equal(c.codes.view(torch.uint8)[ids[at].long(), 0, 0, 0, 0, 0], (old[slots.long()][at] % 251).to(torch.uint8))


def test_offsets_past_32_bits():
    """A pool of 6 GB: pages whose bytes lie past 2^32 are written, copied and read."""
    G = _g()
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    ref_pages, shift = 40, 12000 - 40
    c = G.KV8Cache.allocate(R.INT8, 8, 16, 128, 16, 12000, 8, 16)  # 512 KB a page
    c.refs[:shift] = 1
    p = Pair(R.INT8, kvh=16, d=128)  # small twin in which the reference is kept
    slots, news = [3, 1], [40, 21]
    p.append(slots, news)
    x = torch.randn(61, 2, 16, 128, device="cuda").bfloat16()
    for cache, layer in ((c, 7), (p.dev, 0)):
        work = torch.empty(cache.workspace_bytes(8), dtype=torch.uint8, device="cuda")
        if cache is c:
            cache.resize(_i32(slots), _i32(news), work)
        cache.append(layer, x[:, 0], x[:, 1], _i32(slots), _i32([0, 40, 61]))
        cache.fork(_i32([3]), _i32([0]), work)
    out = []
    for cache, layer in ((c, 7), (p.dev, 0)):
        o = torch.empty(2, 16, 128, device="cuda", dtype=torch.bfloat16)
        work = torch.empty(cache.attention_workspace_bytes(16, 2, 2, 1), dtype=torch.uint8, device="cuda")
        cache.attention(layer, x[:2, 0], o, _i32([0, 1]), _i32([0, 1, 2]), 1, work)
        out.append(o)
    G.check_device_error()
    assert torch.equal(out[0], out[1])
    assert torch.all(c.table[3, :3] >= shift)


@pytest.mark.parametrize("d", [64, 128])
def test_wait_that_gives_up_is_reported_and_recovers(d):
    """The prompt kernel's waits run out at once (none is left hanging); with
    the limit restored the same call gives the bits it gave before."""
    p = Pair(R.INT8, kvh=2, d=d, ps=32, num_pages=60, max_pages=40)
    p.append([0, 1], [900, 500])
    work = torch.empty(p.dev.attention_workspace_bytes(2, 2, 1000, 700), dtype=torch.uint8, device="cuda")
    q = torch.randn(1000, 2, d, device="cuda").bfloat16()

    def call():
        out = torch.zeros_like(q)
        p.dev.attention(0, q, out, _i32([0, 1]), _i32([0, 700, 1000]), 700, work)
        return out

    want = call()
    p.G.check_device_error()
    try:
        p.G.set_wait_limit_ns(1)
        call()
        with pytest.raises(p.G.GPT2Error) as e:
            p.G.check_device_error()
        assert e.value.name == "ECUDA"
    finally:
        p.G.set_wait_limit_ns(0)
    got = call()
    p.G.check_device_error()
    assert torch.equal(got, want)


# ------------------------------------------------------------- as they are used
def _step(p, slots, seed, work, awork, news, stream=None):
    """One layerless sampling step: room, append, attention."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = p.lens[slots.long()] + news
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), news.cumsum(0).int()])
    rows = int(cu[-1])
    qkv = torch.randn(rows, 4 + 2 * p.n_kv_head, 64, generator=g, device="cuda").bfloat16()
    out = torch.zeros(rows, 4, 64, device="cuda", dtype=torch.bfloat16)
    p.resize(slots, lens, work, stream=stream)
    p.append(0, qkv[:, 4:4 + p.n_kv_head], qkv[:, 4 + p.n_kv_head:], slots, cu, stream=stream)
    p.attention(0, qkv[:, :4], out, slots, cu, int(news.max()), awork, stream=stream)
    return out


@pytest.mark.parametrize("fmt", FMTS)
def test_prompt_forked_and_continued(fmt):
    """A prompt, four continuations of different lengths, one cut back, the
    pool compacted in between: every attention against the reference."""
    p = Pair(fmt, layers=2, kvh=2, ps=16, num_pages=64, num_slots=8, max_pages=16)
    p.append([2], [53])
    p.attention([2], [53], group=2)
    p.fork([2, 2, 2], [0, 4, 5])
    for step in range(4):
        p.append([0, 2, 4, 5], [1, 1, 1, 2])
        p.attention([0, 2, 4, 5], [1, 1, 1, 2], group=2, layer=step % 2)
    p.resize([5, 2], [50, 0])
    p.compact()
    p.append([5, 4], [3, 1])
    p.attention([5, 4, 0], [3, 1, 1], group=2)


def test_graph_capture_side_stream_and_determinism():
    """The same steps eagerly, on another stream, and captured and replayed
    give the same bits; two graphs with workspaces of their own run at once."""
    G = _g()

    def fresh():
        c = G.KV8Cache.allocate(R.E4M3, 1, 2, 64, 16, 400, 8, 64)
        work = torch.empty(c.workspace_bytes(8), dtype=torch.uint8, device="cuda")
        awork = torch.empty(c.attention_workspace_bytes(4, 8, 4096, 4096), dtype=torch.uint8, device="cuda")
        slots = _i32([3, 1, 6])
        _step(c, slots, 1, work, awork, _i32([700, 33, 1]))
        return c, work, awork, slots

    c, work, awork, slots = fresh()
    want = [_step(c, slots, 2 + i, work, awork, _i32([1, 2, 1])) for i in range(3)]
    torch.cuda.synchronize()

    side = torch.cuda.Stream()
    c2, work2, awork2, slots2 = fresh()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = [_step(c2, slots2, 2 + i, work2, awork2, _i32([1, 2, 1]), stream=side) for i in range(3)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(c.codes.view(torch.uint8), c2.codes.view(torch.uint8))

    # captured: a step whose lengths come from device memory
    runs = []
    for k in range(2):
        c3, work3, awork3, slots3 = fresh()
        q = torch.randn(4, 8, 64, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
        out = torch.zeros(4, 4, 64, device="cuda", dtype=torch.bfloat16)
        lens, cu, one = c3.lens[slots3.long()].clone(), _i32([0, 1, 3, 4]), _i32([1, 2, 1])
        torch.cuda.synchronize()

        def body(stream):
            lens.add_(one)
            c3.resize(slots3, lens, work3, stream=stream)
            c3.append(0, q[:, 4:6], q[:, 6:], slots3, cu, stream=stream)
            c3.attention(0, q[:, :4], out, slots3, cu, 2, awork3, stream=stream)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body(torch.cuda.current_stream())
        runs.append((graph, c3, out, lens, q, cu, one, slots3, work3, awork3))
    c4, work4, awork4, slots4 = fresh()
    q, cu = runs[0][4], runs[0][5]
    out4 = torch.zeros(4, 4, 64, device="cuda", dtype=torch.bfloat16)
    lens4 = c4.lens[slots4.long()].clone()
    for _ in range(5):
        lens4 += _i32([1, 2, 1])
        c4.resize(slots4, lens4, work4)
        c4.append(0, q[:, 4:6], q[:, 6:], slots4, cu)
        c4.attention(0, q[:, :4], out4, slots4, cu, 2, awork4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                r[0].replay()
    torch.cuda.synchronize()
    G.check_device_error()
    for r in runs:
        assert torch.equal(r[2], out4)
        assert torch.equal(r[1].codes.view(torch.uint8), c4.codes.view(torch.uint8))


def test_first_call_of_a_process_inside_a_capture():
    """Every call's one-time set-up happens outside the stream, so that a
    program may capture before it has run anything."""
    _g()
    code = """
import torch
from decoder_only_transformer_02_b200 import gpt2 as G
c = G.KV8Cache.allocate(G.GPT2_KV_E4M3, 1, 2, 64, 16, 600, 4, 300)
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
slots, cu, lens = i32([2, 0]), i32([0, 100, 101]), i32([100, 1])
x = torch.randn(101, 6, 64, device="cuda").bfloat16()
out = torch.zeros(101, 2, 64, dtype=torch.bfloat16, device="cuda")
work = torch.empty(c.workspace_bytes(4), dtype=torch.uint8, device="cuda")
awork = torch.empty(c.attention_workspace_bytes(2, 2, 101, 100), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    st = torch.cuda.current_stream()
    c.resize(slots, lens, work, stream=st)
    c.append(0, x[:, 2:4], x[:, 4:], slots, cu, stream=st)
    c.attention(0, x[:, :2], out, slots, cu, 100, awork, stream=st)
    c.compact(work, stream=st)
g.replay()
torch.cuda.synchronize()
G.check_device_error()
assert torch.isfinite(out).all() and out[100].abs().sum() > 0 and c.lens.tolist() == [1, 0, 100, 0]
print("captured")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_attention_calls_at_once_on_one_cache():
    p = Pair(R.E4M3, kvh=2, ps=32, num_pages=200, max_pages=100)
    p.append([0, 1, 2], [3000, 700, 1])
    q = torch.randn(400, 2, 64, device="cuda").bfloat16()
    calls = [([0, 1, 2], [1, 1, 1], 1), ([1, 0], [300, 70], 300)]
    streams = [torch.cuda.Stream() for _ in calls]

    def run(at_once):
        outs = []
        for st, (slots, news, max_q) in zip(streams, calls):
            cu = _i32(np.concatenate([[0], np.cumsum(news)]))
            out = torch.zeros(sum(news), 2, 64, dtype=torch.bfloat16, device="cuda")
            work = torch.empty(p.dev.attention_workspace_bytes(2, len(slots), len(out), max_q), dtype=torch.uint8, device="cuda")
            outs.append((out, _i32(slots), cu, work))
        torch.cuda.synchronize()
        for _ in range(10 if at_once else 1):
            for st, o, (_, _, max_q) in zip(streams, outs, calls):
                p.dev.attention(0, q[:len(o[0])], o[0], o[1], o[2], max_q, o[3], stream=st)
                if not at_once:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        p.G.check_device_error()
        return [o[0] for o in outs]

    assert all(torch.equal(a, b) for a, b in zip(run(False), run(True)))


def test_as_many_sequences_as_a_call_takes():
    """4096 short sequences, and a prompt among them."""
    G = _g()
    n = 4096
    c = G.KV8Cache.allocate(R.E4M3, 1, 1, 64, 16, 5000, n, 300)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1)).int().cuda()
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    lens[1234] = 300
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).int()])
    rows = int(cu[-1])
    qkv = torch.randn(rows, 3, 1, 64, device="cuda").bfloat16()
    work = torch.empty(c.workspace_bytes(n), dtype=torch.uint8, device="cuda")
    c.resize(slots, lens, work)
    c.append(0, qkv[:, 1], qkv[:, 2], slots, cu)
    for max_q in (300, 4096):
        awork = torch.empty(c.attention_workspace_bytes(1, n, rows, max_q), dtype=torch.uint8, device="cuda")
        out = torch.zeros(rows, 1, 64, dtype=torch.bfloat16, device="cuda")
        c.attention(0, qkv[:, 0], out, slots, cu, max_q, awork)
        G.check_device_error()
        # a single token's output is its own value as the cache holds it
        own = torch.ones(rows, dtype=torch.bool, device="cuda")
        own[1234:1534] = False
        v = qkv[own, 2, 0].float()
        assert torch.all((out[own, 0].float() - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -8 * v.abs().amax(-1, keepdim=True))
        assert torch.isfinite(out).all() and (out[1400:1500].float().std() > 0)
    with pytest.raises(G.GPT2Error) as e:
        c.resize(_i32(range(n + 1)), _i32(range(n + 1)), work)
    assert e.value.name == "EINVAL"


def test_empty_calls():
    G = _g()
    p = Pair(R.INT8)
    none, zero = _i32([]), _i32([0])
    q = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    p.dev.resize(none, none, p.work)
    p.dev.fork(none, none, p.work)
    p.dev.compact(p.work)
    p.dev.append(0, q, q, none, zero)
    p.dev.attention(0, q, q, none, zero, 1, p.work)
    p.dev.append(0, q, q, _i32([0]), _i32([0, 0]))
    p.dev.attention(0, q, q, _i32([0]), _i32([0, 0]), 1, p.work)
    G.check_device_error()
    p.resize([0], [0])


def test_host_refusals():
    G = _g()
    c = G.KV8Cache.allocate(R.INT8, 2, 2, 64, 16, 8, 4, 4)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    k, slots, cu = q[:, :2], _i32([0]), _i32([0, 2])
    work = torch.empty(c.attention_workspace_bytes(4, 1, 2, 2) + 64, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: c.append(2, k, k, slots, cu), lambda: c.append(-1, k, k, slots, cu),
        lambda: c.append(0, k.float(), k, slots, cu), lambda: c.append(0, q, q, slots, cu),
        lambda: c.append(0, k, k, slots.long(), cu), lambda: c.append(0, k, k, slots, slots),
        lambda: c.append(0, k.transpose(0, 1), k, slots, cu), lambda: c.append(0, k[:, :, 1:], k, slots, cu),
        lambda: c.append(0, torch.zeros(2, 2, 66, dtype=torch.bfloat16, device="cuda")[:, :, 1:65], k, slots, cu),
        lambda: c.attention(0, q, q, slots, cu, 0, work), lambda: c.attention(0, q, q, slots, cu, 2, work[:8]),
        lambda: c.attention(0, q, q, slots, cu, 2, work[1:]), lambda: c.attention(0, q[:, :3], q[:, :3], slots, cu, 2, work),
        lambda: c.attention(0, q, q.float(), slots, cu, 2, work), lambda: c.attention(0, q, q[:1], slots, cu, 2, work),
        lambda: c.attention(0, q, q, slots, cu, 2, work, lse=torch.zeros(2, 3, device="cuda")),
        lambda: c.resize(slots, _i32([1, 2]), work), lambda: c.resize(slots, slots, work[:16]),
        lambda: c.fork(slots, cu, work), lambda: c.compact(work[:16]), lambda: c.compact(work.cpu()),
        lambda: G.KV8Cache(c.codes, c.scales[:1], c.table, c.lens, c.refs),
        lambda: G.KV8Cache(c.codes.float(), c.scales, c.table, c.lens, c.refs),
        lambda: G.KV8Cache.allocate(R.INT8, 2, 2, 96, 16, 8, 4, 4), lambda: G.KV8Cache.allocate(R.INT8, 2, 2, 64, 24, 8, 4, 4),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(G.GPT2Error) as e:
            call()
        assert e.value.name == "EINVAL", i
    G.check_device_error()
