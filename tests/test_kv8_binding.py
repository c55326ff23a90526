"""The Python side of the paged 8-bit cache without a GPU: what it refuses and
what it hands on, with CPU tensors and a library that records its calls."""
import contextlib
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def made():
    """(module, cache, model, library) around CPU tensors."""
    from decoder_only_transformer_02_b200 import gpt2 as G
    c, m, lib = G.KV8Cache.__new__(G.KV8Cache), G.GPT2.__new__(G.GPT2), Lib()
    c._torch, c._i32, c._f32, c._bf16 = torch, torch.int32, torch.float32, torch.bfloat16
    c._only_device, c.device, c._lib, c._p = True, torch.device("cpu"), lib, 1
    c.n_kv_head, c.head_dim, c.num_slots = 2, 64, 8
    m._h, m._lib, m.cfg = None, lib, types.SimpleNamespace(padded_vocab=512)
    m._check = lambda r: None
    yield G, c, m, lib
    m._h = None


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_model_calls_check_their_arrays(made):
    G, c, m, lib = made
    good = dict(slots=i32(3), tokens=i32(3), next_out=i32(3))
    m.kv8_decode_step(c, **good)
    m.kv8_decode_step(c, **dict(good, next_out=i32(5)))
    m.kv8_prefill(c, **dict(good, tokens=i32(3, 7)))
    assert [n for n, _ in lib.calls] == ["gpt2_kv8_decode_step"] * 2 + ["gpt2_kv8_prefill"]
    assert lib.calls[2][1][4:6] == (3, 7)
    bad = [dict(slots=i32(2)), dict(slots=i32(4)), dict(slots=None), dict(slots=i32(3).long()), dict(slots=i32(6)[::2]),
           dict(slots=i32(3, 1)), dict(slots=torch.zeros(3, dtype=torch.int32, device="meta")), dict(next_out=i32(2)),
           dict(next_out=None), dict(next_out=i32(3).float()), dict(next_out=i32(6)[::2]),
           dict(next_out=torch.zeros(3, dtype=torch.int32, device="meta"))]
    steps = bad + [dict(tokens=i32(3).long()), dict(tokens=i32(6)[::2]), dict(tokens=i32(3, 1)), dict(tokens=None),
                   dict(tokens=torch.zeros(3, dtype=torch.int32, device="meta"))]
    prefills = bad + [dict(tokens=i32(3, 7).long()), dict(tokens=i32(7, 3).t()), dict(tokens=i32(3)), dict(tokens=None)]
    for call, base, cases in ((m.kv8_decode_step, good, steps), (m.kv8_prefill, dict(good, tokens=i32(3, 7)), prefills)):
        for i, b in enumerate(cases):
            with pytest.raises(G.GPT2Error) as e:
                call(c, **dict(base, **b))
            assert e.value.name == "EINVAL", (call, i)
    assert len(lib.calls) == 3


def test_a_single_row_may_have_any_stride(made):
    """torch leaves the stride of a dimension of one entry open: keys and values
    of one token out of different buffers are of the same shape all the same."""
    G, c, m, lib = made
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros(1, 5, 64, **bf)[:, :2]                             # row stride 320
    v = torch.as_strided(torch.zeros(128, **bf), (1, 2, 64), (1, 64, 1))  # row stride 1
    cu = torch.tensor([0, 1], dtype=torch.int32)
    c.append(0, k, v, i32(1), cu)
    c.append(0, k[:0], v[:0], i32(1), cu)
    q = torch.as_strided(torch.zeros(259, **bf), (1, 4, 64), (257, 64, 1))
    c.attention(0, q, q, i32(1), cu, 1, torch.zeros(64, dtype=torch.uint8))
    assert [a[1][4] for a in lib.calls[:2]] == [128, 128] and lib.calls[2][1][3] == lib.calls[2][1][5] == 256
    with pytest.raises(G.GPT2Error):
        c.append(0, torch.zeros(2, 5, 64, **bf)[:, :2], torch.zeros(2, 2, 64, **bf), i32(1), cu)


def test_calls_run_on_the_caches_device(made):
    """Also the size of the attention's workspace, which goes by its SMs."""
    G, c, m, lib = made
    now = [0]

    @contextlib.contextmanager
    def device(d):
        now[0], was = d.index, now[0]
        yield
        now[0] = was

    class Calls:
        def __getattr__(self, name):
            return lambda *args: now[0] if name.endswith("bytes") else lib.calls.append((name, now[0])) or 0

    c._lib, c._only_device = Calls(), False
    c._torch = types.SimpleNamespace(cuda=types.SimpleNamespace(current_device=lambda: now[0], device=device))
    dev, c.device = c.device, torch.device("cuda", 3)
    assert c.attention_workspace_bytes(2, 1, 1, 1) == 3 and now == [0]
    c._call("x", c._lib.gpt2_kv8_fork)
    assert lib.calls == [("gpt2_kv8_fork", 3)] and now == [0]
    c.device = dev


def test_decode_logits_have_room_for_the_last_calls_rows(made, monkeypatch):
    """A paged step of four rows between two dense ones of two: the library
    writes four rows whatever the caller asks for."""
    import numpy as np
    G, c, m, lib = made
    heap, room = np.full((16, 512), np.nan, np.float32), []

    class Np:
        def __getattr__(self, name):
            return getattr(np, name)

        def empty(self, shape, dtype):
            room.append(shape[0])
            return heap[:shape[0]]

    class Writes(Lib):
        def gpt2_get_decode_logits(self, h, p):
            heap[:4] = np.arange(4)[:, None]
            return 0

    m._lib = Writes()
    monkeypatch.setattr(G, "np", Np())
    m.kv8_decode_step(c, i32(4), i32(4), i32(4))
    got = m.get_decode_logits(2)
    assert room == [4] and got.shape == (2, 512) and np.all(got == [[0], [1]])
    assert m.get_decode_logits(4).shape == (4, 512)
    with pytest.raises(G.GPT2Error):
        m.get_decode_logits(5)


def test_model_calls_refuse_a_cache_on_another_device(made):
    G, c, m, lib = made
    now = [0]
    c._only_device, c.device = False, torch.device("cuda", 3)
    c._torch = types.SimpleNamespace(cuda=types.SimpleNamespace(current_device=lambda: now[0]))
    for call, tokens in ((m.kv8_decode_step, i32(2)), (m.kv8_prefill, i32(2, 3))):
        with pytest.raises(G.GPT2Error, match="current device") as e:
            call(c, i32(2), tokens, i32(2))
        assert e.value.name == "EINVAL"
    assert lib.calls == []
