"""The paged 8-bit cache where a call is refused, a page is shared or bad, or
what a row must not see is extreme; through the C ABI against the 64-bit form
in tests/kv8_reference.py."""
import numpy as np
import pytest

from tests import kv8_reference as R
from tests.gpu_util import bf16_round, need_gpu, torch
from tests.test_gpu_kv8 import FMTS, Pair, _i32
from tests.test_gpu_kv8_generate import Run, _dev

pytestmark = pytest.mark.gpu


def _state(c):
    return [t.clone() for t in (c.codes.view(torch.uint8), c.scales.view(torch.int32), c.table, c.lens, c.refs)]


def _unchanged(c, before):
    return all(torch.equal(a, b) for a, b in zip(before, _state(c)))


def _refused(G, call, name="ECACHE"):
    call()
    with pytest.raises(G.GPT2Error) as e:
        G.check_device_error()
    assert e.value.name == name


# ------------------------------------------------------------ refused prefills
@pytest.mark.parametrize("slots", [[3, 3], [3, 1, 3], [3, 8], [-1, 3]])
def test_refused_prefill_leaves_slots_of_the_same_length(slots):
    """A slot named twice, or one that does not exist, beside slots that hold as
    many tokens as the call brings, their page shared with a fork."""
    r = Run(R.INT8)
    rng = np.random.default_rng(1)
    r.prefill([3, 1], rng.integers(0, 500, (2, 16)))
    r.cache.fork(_dev([3]), _dev([6]), r.work)
    before = _state(r.cache)
    out = torch.empty(len(slots), dtype=torch.int32, device="cuda")
    r.m.kv8_prefill(r.cache, _dev(slots), _dev(rng.integers(0, 500, (len(slots), 16))), out)
    with pytest.raises(r.G.GPT2Error) as e:
        r.m.get_decode_logits(len(slots))
    assert e.value.name == "ECACHE"
    assert _unchanged(r.cache, before)
    r.m.close()


def test_prefill_without_room_has_freed_its_slots():
    """Six pages of four: the freeing went through, and no row is written."""
    r = Run(R.E4M3, num_pages=4, max_T=40)
    rng = np.random.default_rng(2)
    r.prefill([0, 1], rng.integers(0, 500, (2, 17)))
    codes, scales = r.cache.codes.view(torch.uint8).clone(), r.cache.scales.clone()
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    r.m.kv8_prefill(r.cache, _dev([0, 1]), _dev(rng.integers(0, 500, (2, 40))), out)
    with pytest.raises(r.G.GPT2Error) as e:
        r.m.get_decode_logits(2)
    assert e.value.name == "ECACHE"
    assert torch.all(r.cache.lens == 0) and torch.all(r.cache.refs == 0)
    assert torch.equal(codes, r.cache.codes.view(torch.uint8)) and torch.equal(scales, r.cache.scales)
    r.ref.resize([0, 1], [0, 0])
    r.prefill([0, 1], rng.integers(0, 500, (2, 20)))
    r.m.close()


@pytest.mark.parametrize("length", [-1, -5, -2 ** 31, 2 ** 31 - 1, 64, 65])
@pytest.mark.parametrize("prefill", [False, True])
def test_model_calls_refuse_a_bad_stored_length(length, prefill):
    """A length below zero, or one at which there is no next position, in the
    caller's d_lens: refused, nothing written, no position formed from it."""
    if prefill and length == 64:
        return  # a full slot may be replaced
    r = Run(R.INT8)
    rng = np.random.default_rng(3)
    r.prefill([3, 1], rng.integers(0, 500, (2, 16)))
    r.cache.lens[3] = length
    before = _state(r.cache)
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    if prefill:
        r.m.kv8_prefill(r.cache, _dev([1, 3]), _dev(rng.integers(0, 500, (2, 16))), out)
    else:
        r.m.kv8_decode_step(r.cache, _dev([1, 3]), _dev([5, 6]), out)
    with pytest.raises(r.G.GPT2Error) as e:
        r.m.get_decode_logits(2)
    assert e.value.name == "ECACHE"
    assert _unchanged(r.cache, before)
    r.m.close()


# ------------------------------------------------------------ captured and grown
def test_a_captured_step_survives_a_larger_pool():
    """A step captured with a small pool, then calls with a larger one and more
    rows, which need more scratch: the graph still replays what it captured."""
    def fresh():
        r = Run(R.INT8)
        rng = np.random.default_rng(9)
        prompts = _dev(rng.integers(0, 500, (2, 16)))
        slots, out = _dev([3, 1]), torch.empty(2, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        r.m.set_stream(side)
        torch.cuda.synchronize()
        r.m.kv8_prefill(r.cache, slots, prompts, out)
        torch.cuda.synchronize()
        return r, slots, out, side

    eager, slots, out, _ = fresh()
    want = []
    for _ in range(4):
        eager.m.kv8_decode_step(eager.cache, slots, out, out)
        want.append(eager.m.get_decode_logits(2))
    state = _state(eager.cache)
    eager.m.close()

    r, slots, out, side = fresh()
    r.m.kv8_decode_step(r.cache, slots, out, out)  # (eager once)
    np.testing.assert_array_equal(r.m.get_decode_logits(2), want[0])
    big = r.G.KV8Cache.allocate(R.INT8, 2, 2, 64, 16, 400000, 8, 4)
    s4, t4, o4 = _dev([0, 1, 2, 3]), _dev([5, 6, 7, 8]), torch.empty(4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r.m.kv8_decode_step(r.cache, slots, out, out)
        with pytest.raises(r.G.GPT2Error) as e:  # more scratch is not to be had in a capture, which goes on
            r.m.kv8_decode_step(big, s4, t4, o4)
        assert e.value.name == "ESTATE"
    for i in (1, 2, 3):
        r.m.kv8_decode_step(big, s4, t4, o4)
        torch.cuda.synchronize()
        if i == 1:  # whatever was given back would be taken and overwritten here
            rest = [torch.full((1 << 20,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(64)]
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        got = r.m.get_decode_logits(4)[:2]  # (the rows of the last call that the handle knows of: four)
        np.testing.assert_array_equal(got, want[i])
    assert all(torch.equal(a, b) for a, b in zip(state, _state(r.cache)))
    assert r.m.check_guards() == 0
    del rest
    r.m.close()


# -------------------------------------------- append into pages of several slots
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ps,news", [(16, 3), (16, 40), (64, 70), (128, 1)])
def test_append_does_not_write_into_a_shared_page(fmt, ps, news):
    """Rows that reach a page which another slot holds, or a free one, are
    skipped and recorded; the sequence's own pages are written."""
    p = Pair(fmt, kvh=3, ps=ps, num_pages=20)
    p.append([0, 2], [2 * ps, 5])
    p.fork([0], [1])
    before = _state(p.dev)
    x = torch.randn(news + 1, 2, 3, 64, device="cuda").bfloat16()

    def put(slot):
        p.dev.append(0, x[:, 0], x[:, 1], _i32([slot]), _i32([0, min(news, 2 * ps)]))

    for slot in (0, 1):
        _refused(p.G, lambda: put(slot))
        assert _unchanged(p.dev, before)
    p.resize([0], [2 * ps + 1])  # a page of its own behind the shared ones
    m = min(news, 2 * ps)
    before = _state(p.dev)
    if m == 1:
        put(0)
        p.G.check_device_error()
    else:
        _refused(p.G, lambda: put(0))
    own = int(p.dev.table[0, 2])
    keep = torch.arange(20, device="cuda") != own
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(before[:2], _state(p.dev)[:2]))
    k = x[m - 1:m].double().cpu().numpy()
    p.ref.append(0, k[:, 0], k[:, 1], [0], [0, 1])
    p.same()
    p.dev.refs[int(p.dev.table[2, 0])] = 0  # (a count that the caller has lost)
    before = _state(p.dev)
    p.dev.append(0, x[:1, 0], x[:1, 1], _i32([2]), _i32([0, 1]))
    with pytest.raises(p.G.GPT2Error):
        p.G.check_device_error()
    assert _unchanged(p.dev, before)
    p.dev.refs[int(p.dev.table[2, 0])] = 1
    p.append([0, 1, 2], [3, 4, 5])


def _kernels_of(graph):
    """Kernel nodes of a captured graph."""
    from cuda.bindings import runtime as rt

    def ok(r):
        assert r[0] == rt.cudaError_t.cudaSuccess, r[0]
        return r[1:]

    raw = rt.cudaGraph_t(graph.raw_cuda_graph())
    n = ok(rt.cudaGraphGetNodes(raw, 0))[-1]
    nodes = ok(rt.cudaGraphGetNodes(raw, n))[0]
    return sum(ok(rt.cudaGraphNodeGetType(x))[0] == rt.cudaGraphNodeType.cudaGraphNodeTypeKernel for x in nodes[:n])


@pytest.mark.parametrize("max_pages", [4, 256])  # whole tiles, or cut ones that are joined
@pytest.mark.parametrize("prefill", [False, True])
def test_launches_are_counted(max_pages, prefill):
    r = Run(R.INT8)
    cache = r.G.KV8Cache.allocate(R.INT8, 2, 2, 64, 16, 40, 8, max_pages)
    side = torch.cuda.Stream()
    r.m.set_stream(side)
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    slots, tokens, prompt = _dev([2, 5]), _dev([7, 9]), _dev(np.ones((2, 16)))
    torch.cuda.synchronize()

    def call():
        if prefill:
            r.m.kv8_prefill(cache, slots, prompt, out)
        else:
            r.m.kv8_decode_step(cache, slots, tokens, out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=side):
        n = r.m.kernel_launches
        call()
        n = r.m.kernel_launches - n
    assert n == _kernels_of(graph)
    r.m.close()


def test_a_refused_call_does_not_hide_a_wait_that_gave_up():
    """A refusal first, then a prompt whose waits run out: what is incomplete is reported."""
    p = Pair(R.INT8, kvh=2, ps=32, num_pages=60, max_pages=40)
    p.append([0, 1], [900, 500])
    work = torch.empty(p.dev.attention_workspace_bytes(2, 2, 1000, 700), dtype=torch.uint8, device="cuda")
    q = torch.randn(1000, 2, 64, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    for first in (True, False):
        try:
            p.G.set_wait_limit_ns(1)
            if first:
                p.dev.resize(_i32([0, 0]), _i32([1, 1]), p.work)
            p.dev.attention(0, q, out, _i32([0, 1]), _i32([0, 700, 1000]), 700, work)
            if not first:
                p.dev.resize(_i32([0, 0]), _i32([1, 1]), p.work)
            with pytest.raises(p.G.GPT2Error) as e:
                p.G.check_device_error()
            assert e.value.name == "ECUDA"
        finally:
            p.G.set_wait_limit_ns(0)
        p.G.check_device_error()


# ------------------------------------------------------------------- bad pages
def _near(p, slot, q, out, lse, first):
    """The rows of `slot` (its last ones) before position `first` against the
    64-bit form; tolerances as in tests/test_gpu_kv8.py, with the largest value
    taken over the tokens before `first` alone.  Returns which rows those are."""
    rows, heads, d = q.shape
    n = int(p.ref.lens[slot])
    blind = np.arange(n - rows, n) < first
    assert blind.any() and not blind.all()
    m = int(blind.sum())
    want, wl, mag, top = p.ref.attention(0, q.double().cpu().numpy(), [slot], [0, rows])
    ds = 2 * d * 2.0 ** -24 * top[:m]
    v = np.abs(p.ref.values(0, slot)[1][:first]).max((0, 2)).repeat(heads // p.ref.kvh)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -30 * first * v[:, None]
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.abs(got - want)[:m] <= bound[:m] + 2 * ds[..., None] * mag[:m])
    assert np.all(np.abs(gl - wl)[:m] <= ds + 2.0 ** -20 * (1 + np.abs(wl[:m])))
    return torch.from_numpy(blind).cuda()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps", [(64, 16), (64, 128), (128, 16), (128, 64)])
@pytest.mark.parametrize("rows", [5, 200])       # the streaming kernel, the prompt kernel
@pytest.mark.parametrize("room", [512, 8192])    # tiles whole, or cut
def test_a_page_outside_the_pool_reaches_its_readers_only(fmt, d, ps, rows, room):
    """Rows that see a token of it are NaN; those before it are as the
    definition has them, and those of the other sequence, and of none, as with
    a clean table."""
    p = Pair(fmt, kvh=2, d=d, ps=ps, num_pages=90, max_pages=room // ps)
    p.append([6], [3])
    p.append([0, 1], [290, 259])
    p.resize([6], [0])  # page 0 is free, and holds codes that are no number
    p.dev.codes.view(torch.uint8)[0] = 0x7f
    p.dev.scales[0] = float("nan")
    q = torch.randn(2 * rows + 1, 4, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    work = torch.empty(p.dev.attention_workspace_bytes(4, 2, len(q), rows), dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.full_like(q, 7.0), torch.full((len(q), 4), 7.0, device="cuda")
        p.dev.attention(0, q, out, _i32([1, 0]), _i32([0, rows, 2 * rows]), rows, work, lse=lse)
        return out, lse

    want = call()
    p.G.check_device_error()
    assert torch.isfinite(want[0].float()).all()
    kept = int(p.dev.table[1, 256 // ps])
    for page in (-1, 90, 2 ** 31 - 1):
        p.dev.table[1, 256 // ps] = page
        got = call()
        with pytest.raises(p.G.GPT2Error) as e:
            p.G.check_device_error()
        assert e.value.name == "ECACHE"
        blind = _near(p, 1, q[:rows], got[0][:rows], got[1][:rows], 256)
        for g, w in zip(got, want):
            assert torch.isnan(g[:rows][~blind].float()).all()
            assert torch.equal(g[rows:], w[rows:])
    p.dev.table[1, 256 // ps] = kept
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


# ------------------------------------------------ values that a row does not see
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps", [(64, 16), (64, 32), (128, 16), (128, 64)])
@pytest.mark.parametrize("rows", [30, 100])      # the streaming kernel, the prompt kernel
@pytest.mark.parametrize("room", [512, 8192])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 40, 2.0 ** 100])
def test_later_tokens_do_not_reach_earlier_rows(fmt, d, ps, rows, room, size):
    """The last tokens' keys and values are `size` times the others': rows
    before their page are held to the tokens that they see."""
    p = Pair(fmt, kvh=2, d=d, ps=ps, num_pages=90, max_pages=room // ps)
    p.append([0, 1], [256, 200])
    p.append([0, 1], [17, 9], size=size)  # (slot 1: from the middle of a page on)
    q = torch.randn(2 * rows, 4, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(2 * rows, 4, device="cuda")
    work = torch.empty(p.dev.attention_workspace_bytes(4, 2, 2 * rows, rows), dtype=torch.uint8, device="cuda")
    p.dev.attention(0, q, out, _i32([0, 1]), _i32([0, rows, 2 * rows]), rows, work, lse=lse)
    p.G.check_device_error()
    for i, first in ((0, 256), (1, 192)):
        at = slice(i * rows, (i + 1) * rows)
        _near(p, i, q[at], out[at], lse[at], first)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,ps", [(64, 16), (64, 64), (128, 16)])
@pytest.mark.parametrize("rows", [30, 100])
def test_keys_far_apart_within_a_block(fmt, d, ps, rows):
    """Pages of keys 2^30 times the others whose scores lie far below them: the
    scores of the others keep their own precision."""
    p = Pair(fmt, kvh=1, d=d, ps=ps, num_pages=90, max_pages=8192 // ps)

    def large(x):  # (keys and values of one head, in that order)
        x[:, :d] = -np.abs(x[:, :d]) * 2.0 ** 30

    p.append([0], [2 * ps + 5])
    p.append([0], [ps - 5])
    p.append([0], [ps], mutate=large)
    p.append([0], [3 * ps + rows])
    q = (torch.randn(rows, 1, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").abs() + 0.1).bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(rows, 1, device="cuda")
    work = torch.empty(p.dev.attention_workspace_bytes(1, 1, rows, rows), dtype=torch.uint8, device="cuda")
    p.dev.attention(0, q, out, _i32([0]), _i32([0, rows]), rows, work, lse=lse)
    p.G.check_device_error()
    # against the same sequence without the page: its weights are below e^-(2^20)
    k, v = p.ref.values(0, 0)
    keep = np.arange(len(k)) // ps != 3
    z = np.einsum("rd,td->rt", q[:, 0].double().cpu().numpy(), k[:, 0]) / np.sqrt(d)
    mag = np.einsum("rd,td->rt", q[:, 0].double().cpu().numpy(), np.abs(k[:, 0])) / np.sqrt(d)
    seen = np.arange(len(k))[None] <= np.arange(len(k) - rows, len(k))[:, None]
    assert np.all(z[:, ~keep] < -2.0 ** 20)
    z = np.where(seen & keep, z, -np.inf)
    m = z.max(1, keepdims=True)
    e = np.exp(z - m)
    want, wl = e @ v[:, 0] / e.sum(1, keepdims=True), (m + np.log(e.sum(1, keepdims=True)))[:, 0]
    ds = 2 * d * 2.0 ** -24 * np.where(seen & keep, mag, 0).max(1)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * ds[:, None] + 2.0 ** -14) * (e @ np.abs(v[:, 0]) / e.sum(1, keepdims=True)) \
        + 2.0 ** -30 * len(k) * np.abs(v).max()
    assert np.all(np.abs(out[:, 0].double().cpu().numpy() - want) <= bound)
    assert np.all(np.abs(lse[:, 0].double().cpu().numpy() - wl) <= ds + 2.0 ** -20 * (1 + np.abs(wl)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [30, 100])
@pytest.mark.parametrize("side", [0, 1])
def test_far_apart_and_not_a_number_in_one_block(fmt, d, rows, side):
    """Ordinary, large and NaN pages, and one outside the pool, within 128 tokens."""
    p = Pair(fmt, kvh=1, d=d, ps=16, num_pages=90, max_pages=512)
    p.append([0], [208])
    p.append([0], [16], size=2.0 ** 35)
    p.append([0], [16])

    def bad(x):  # (keys, then values)
        x[3, side * d + 5] = np.inf

    p.append([0], [16], mutate=bad)
    p.append([0], [16], size=2.0 ** -30)
    q = torch.randn(rows, 2, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    work = torch.empty(p.dev.attention_workspace_bytes(2, 1, rows, rows), dtype=torch.uint8, device="cuda")
    for first in (240, 224):  # the NaN page; then a page before it outside the pool too
        out, lse = torch.zeros_like(q), torch.zeros(rows, 2, device="cuda")
        p.dev.attention(0, q[-rows:], out, _i32([0]), _i32([0, rows]), rows, work, lse=lse)
        if first == 240:
            p.G.check_device_error()
        else:
            with pytest.raises(p.G.GPT2Error):
                p.G.check_device_error()
        n = 272
        sees = torch.arange(n - rows, n, device="cuda") >= first
        if (~sees).any():
            _near(p, 0, q, out, lse, first)
        assert torch.isnan(out[sees].float()).all()
        p.dev.table[0, 14] = -1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [30, 100])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3.0e38])
def test_a_query_that_is_not_finite_stays_in_its_row(d, rows, value):
    p = Pair(R.E4M3, kvh=1, d=d, ps=16, num_pages=90, max_pages=512)
    p.append([0], [400])
    q = torch.randn(rows, 1, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    work = torch.empty(p.dev.attention_workspace_bytes(1, 1, rows, rows), dtype=torch.uint8, device="cuda")
    want, wl, mag, top = p.ref.attention(0, q.double().cpu().numpy(), [0], [0, rows])
    q[rows // 2, 0, 7] = value
    out, lse = torch.zeros_like(q), torch.zeros(rows, 1, device="cuda")
    p.dev.attention(0, q, out, _i32([0]), _i32([0, rows]), rows, work, lse=lse)
    p.G.check_device_error()
    k = np.arange(rows) != rows // 2
    ds = 2 * d * 2.0 ** -24 * top[k]
    v = np.abs(p.ref.values(0, 0)[1]).max()
    bound = 2.0 ** -8 * np.abs(want[k]) + (2.0 ** -11 + 2 * ds[..., None] + 2.0 ** -14) * mag[k] + 2.0 ** -30 * 400 * v
    assert np.all(np.abs(out.double().cpu().numpy()[k] - want[k]) <= bound)
    assert np.all(np.abs(lse.double().cpu().numpy()[k] - wl[k]) <= ds + 2.0 ** -20 * (1 + np.abs(wl[k])))
    assert value == 3.0e38 or not torch.isfinite(lse[rows // 2]).any()
