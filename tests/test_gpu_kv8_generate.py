"""Generation on a paged 8-bit cache (gpt2_kv8_prefill / gpt2_kv8_decode_step).

The reference decodes in 64 bits with the oracle's layers and the 64-bit cache
of tests/kv8_reference.py, which rounds the same keys and values (as bf16, as
the device's projection stores them) to the same codes.  The logits are held to
the bf16 forward's tolerance (as in tests/test_gpu_generate.py): the rounding to
8 bits is in both, a key or value whose bf16 rounding differs moves a code by
one.  The sampled tokens are checked bit-exactly against the oracle's rule on
the device's own logits."""
import numpy as np
import pytest

from tests import kv8_reference as R
from tests.gpu_util import bf16_round, cosine, need_gpu, torch

pytestmark = pytest.mark.gpu

TINY = dict(n_layer=2, n_head=2, n_embd=128, vocab_size=500, padded_vocab=512, block_size=64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Run:
    def __init__(self, fmt, B=4, max_T=24, num_pages=40, num_slots=8, block=64, ps=16):
        need_gpu()
        from decoder_only_transformer_02_b200 import gpt2 as G
        from oracle import gpt2_oracle as O
        self.G, self.O = G, O
        G.check_device_error()
        cfgd = dict(TINY, block_size=block)
        self.cfg = O.Config(**cfgd)
        self.m = G.GPT2(G.GPT2Config(**cfgd, max_B=B, max_T=max_T, precision=G.GPT2_BF16), seed=11)
        flat = O.init_params(self.cfg, 21).astype(np.float32)
        self.m.set_params(flat)
        self.flat = flat.astype(np.float64)
        self.p = O.unflatten(self.flat, self.cfg)
        L, H = self.cfg.n_layer, self.cfg.n_head
        self.cache = G.KV8Cache.allocate(fmt, L, H, 64, ps, num_pages, num_slots, block // ps)
        self.ref = R.Cache(fmt, L, H, 64, ps, num_pages, num_slots, block // ps)
        self.work = torch.empty(self.cache.workspace_bytes(64), dtype=torch.uint8, device="cuda")
        self.seqs = {}

    def same_tables(self):
        np.testing.assert_array_equal(self.cache.lens.cpu().numpy(), self.ref.lens)
        np.testing.assert_array_equal(self.cache.refs.cpu().numpy(), self.ref.refs)

    def check(self, slots, ref, nxt, temperature, top_k, seed):
        logits, got = self.m.get_decode_logits(len(slots)), nxt.cpu().numpy()
        for b, s in enumerate(slots):
            assert np.max(np.abs(logits[b] - ref[b])) < 0.05 * max(1.0, np.max(np.abs(ref[b]))), b
            assert cosine(logits[b], ref[b]) > 0.9999, b
            u = self.O.sample_uniform(seed, s, len(self.seqs[s]))
            assert got[b] == self.O.sample_next(logits[b], self.cfg.vocab_size, temperature, top_k, u)
        self.same_tables()
        return got

    def prefill(self, slots, prompts, temperature=1.0, top_k=1, seed=0):
        nxt = torch.empty(len(slots), dtype=torch.int32, device="cuda")
        self.m.kv8_prefill(self.cache, _dev(slots), _dev(prompts), nxt, temperature, top_k, seed)
        st = self.O.forward(self.flat, self.cfg, prompts)
        B, T = prompts.shape
        self.ref.resize(slots, [0] * B)
        self.ref.resize(slots, [T] * B)
        for layer in range(self.cfg.n_layer):
            q, k, v = np.split(bf16_round(st["cache"]["layers"][layer]["qkv"]), 3, axis=-1)
            self.ref.append(layer, k.reshape(B * T, -1, 64), v.reshape(B * T, -1, 64), slots, np.arange(B + 1) * T)
        for s, pr in zip(slots, prompts):
            self.seqs[s] = list(pr)
        return self.check(slots, st["logits"][:, -1], nxt, temperature, top_k, seed)

    def step(self, slots, tokens, temperature=1.0, top_k=1, seed=0):
        O, p = self.O, self.p
        B, H = len(slots), self.cfg.n_head
        nxt = torch.empty(B, dtype=torch.int32, device="cuda")
        self.m.kv8_decode_step(self.cache, _dev(slots), _dev(tokens), nxt, temperature, top_k, seed)
        self.ref.resize(slots, [len(self.seqs[s]) + 1 for s in slots])
        pos = [len(self.seqs[s]) for s in slots]
        for s, t in zip(slots, tokens):
            self.seqs[s].append(t)
        x = p["wte"][np.asarray(tokens)] + p["wpe"][pos]
        for layer in range(self.cfg.n_layer):
            pre = f"h{layer}."
            qkv = bf16_round(O.linear_forward(O.layernorm_forward(x, p[pre + "ln1.g"], p[pre + "ln1.b"])[0],
                                              p[pre + "attn.w"], p[pre + "attn.b"]))
            q, k, v = (a.reshape(B, H, 64) for a in np.split(qkv, 3, axis=-1))
            self.ref.append(layer, k, v, slots, np.arange(B + 1))
            o = self.ref.attention(layer, q, slots, np.arange(B + 1))[0].reshape(B, -1)
            x = x + O.linear_forward(o, p[pre + "proj.w"], p[pre + "proj.b"])
            a = O.gelu_tanh(O.linear_forward(O.layernorm_forward(x, p[pre + "ln2.g"], p[pre + "ln2.b"])[0],
                                             p[pre + "fc.w"], p[pre + "fc.b"]))
            x = x + O.linear_forward(a, p[pre + "mproj.w"], p[pre + "mproj.b"])
        ref = O.linear_forward(O.layernorm_forward(x, p["lnf.g"], p["lnf.b"])[0], p["wte"])
        return self.check(slots, ref, nxt, temperature, top_k, seed)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_prompts_forked_cut_back_and_continued(fmt):
    r = Run(fmt)
    rng = np.random.default_rng(3)
    nxt = list(r.prefill([5, 2], rng.integers(0, 500, (2, 19)), 0.8, 20, 7))
    for _ in range(4):
        nxt = list(r.step([5, 2], nxt, 0.8, 20, 7))
    # two more samples of slot 5's text, a shorter prompt of its own, all in one step at different positions
    r.cache.fork(_dev([5, 5]), _dev([0, 7]), r.work)
    r.ref.fork([5, 5], [0, 7])
    r.seqs[0], r.seqs[7] = list(r.seqs[5]), list(r.seqs[5])
    n3 = list(r.prefill([3], rng.integers(0, 500, (1, 3)), 0.8, 20, 7))
    toks = [nxt[0], nxt[0], n3[0], nxt[1]]
    for _ in range(15):
        toks = list(r.step([0, 7, 3, 2], toks, 0.8, 20, 7))
    # cut a sample back, move the pages, go on
    r.cache.resize(_dev([7, 2]), _dev([20, 0]), r.work)
    r.ref.resize([7, 2], [20, 0])
    r.seqs[7] = r.seqs[7][:20]
    r.cache.compact(r.work)
    r.ref.compact()
    r.step([7, 0, 3], [1, 2, 3])
    assert r.m.check_guards() == 0
    r.m.close()


def test_prefill_replaces_what_the_slots_held():
    r = Run(R.INT8)
    rng = np.random.default_rng(4)
    r.prefill([1, 2], rng.integers(0, 500, (2, 20)))
    r.cache.fork(_dev([1]), _dev([6]), r.work)
    r.ref.fork([1], [6])
    r.seqs[6] = list(r.seqs[1])
    r.prefill([1], rng.integers(0, 500, (1, 18)))  # slot 6 keeps the shared page
    r.step([6, 1], [4, 5])
    r.m.close()


def test_reaches_block_size_and_is_then_refused():
    r = Run(R.E4M3, block=32, max_T=30)
    rng = np.random.default_rng(5)
    nxt = list(r.prefill([4], rng.integers(0, 500, (1, 30))))
    for _ in range(2):
        nxt = list(r.step([4], nxt))  # the last step fills position 31
    codes = r.cache.codes.view(torch.uint8).clone()
    out = torch.empty(1, dtype=torch.int32, device="cuda")
    r.m.kv8_decode_step(r.cache, _dev([4]), _dev(nxt), out)
    with pytest.raises(r.G.GPT2Error) as e:
        r.m.get_decode_logits(1)
    assert e.value.name == "ECACHE"
    assert torch.equal(codes, r.cache.codes.view(torch.uint8))
    r.same_tables()
    r.m.close()


def test_refused_calls_leave_the_cache():
    r = Run(R.INT8, num_pages=4)
    rng = np.random.default_rng(6)
    r.prefill([0, 1], rng.integers(0, 500, (2, 16)))
    state = [t.clone() for t in (r.cache.codes, r.cache.lens, r.cache.refs, r.cache.table, r.cache.scales)]
    out = torch.empty(4, dtype=torch.int32, device="cuda")

    def refused(call):
        call()
        with pytest.raises(r.G.GPT2Error) as e:
            r.m.get_decode_logits(1)
        assert e.value.name == "ECACHE"
        assert all(torch.equal(a, b) for a, b in zip(state, (r.cache.codes, r.cache.lens, r.cache.refs, r.cache.table,
                                                             r.cache.scales)))

    refused(lambda: r.m.kv8_decode_step(r.cache, _dev([0, 0]), _dev([1, 2]), out))     # a slot twice
    refused(lambda: r.m.kv8_decode_step(r.cache, _dev([0, 8]), _dev([1, 2]), out))     # no such slot
    refused(lambda: r.m.kv8_decode_step(r.cache, _dev([0, 1, 2]), _dev([1, 2, 3]), out))  # three pages of two
    G = r.G
    other = G.KV8Cache.allocate(R.INT8, 3, 2, 64, 16, 4, 4, 4)
    for call in (lambda: r.m.kv8_decode_step(other, _dev([0]), _dev([1]), out),
                 lambda: r.m.kv8_prefill(r.cache, _dev([0]), _dev(np.zeros((1, 65))), out),
                 lambda: r.m.kv8_prefill(r.cache, _dev([0] * 5), _dev(np.zeros((5, 4))), out),
                 lambda: r.m.kv8_decode_step(r.cache, _dev([0]), _dev([1]), out, top_k=65),
                 lambda: r.m.kv8_decode_step(r.cache, None, _dev([1]), out)):
        with pytest.raises(G.GPT2Error) as e:
            call()
        assert e.value.name == "EINVAL"
    r.step([0, 1], [7, 8])
    r.m.close()


def test_dense_and_paged_generation_side_by_side():
    """One handle, its own cache and a paged one: neither disturbs the other."""
    r = Run(R.INT8)
    rng = np.random.default_rng(8)
    pr = rng.integers(0, 500, (2, 10))
    nxt = torch.empty(2, dtype=torch.int32, device="cuda")
    r.m.prefill(_dev(pr), nxt)
    dense = [nxt.cpu().numpy().copy()]
    n2 = list(r.prefill([1, 4], pr))
    for i in range(5):
        r.m.decode_step(_dev(dense[-1]), 10 + i, nxt)
        dense.append(nxt.cpu().numpy().copy())
        n2 = list(r.step([1, 4], n2))
    alone = Run(R.INT8)
    alone.m.prefill(_dev(pr), nxt)
    for i in range(5):
        np.testing.assert_array_equal(nxt.cpu().numpy(), dense[i])
        alone.m.decode_step(_dev(dense[i]), 10 + i, nxt)
    np.testing.assert_array_equal(nxt.cpu().numpy(), dense[5])
    alone.m.close()
    r.m.close()
