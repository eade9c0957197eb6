"""What a call allocates and fills belongs to the stream it runs on.

A call given `stream` while another stream is current: the weights that its
caller did not pass are cleared on the call's stream (a fill on the current
one is in no order with the kernels and may land after them), and its
workspace and outputs come from that stream's pool (a block of the current
stream's pool may still be read or written there, and is handed out again
there as soon as the caller lets go of it, while the call still uses it).

On the CPU the streams are fakes: a stack of raw handles stands for the
current stream, and every allocation notes the handle it is made under."""
import types

import pytest
import torch

import _budget_util as T
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv

HERE, OWN = 16, 80    # handles of the current stream and of the call's


class FakeLibrary:
    """Every size is 64 bytes and every call succeeds; notes the calls' streams."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_size"):
                args[-1]._obj.value = 64
            else:
                self.calls.append((name, args[-1]))    # (append also reads its status word back)
            return 0
        return call


class Fake:
    def __init__(self, mp):
        self.current, self.made, self.shared, self.lib = [HERE], [], [], FakeLibrary()
        fake = self

        class On:
            def __init__(self, stream):
                self.raw = stream.cuda_stream

            def __enter__(self):
                fake.current.append(self.raw)

            def __exit__(self, *exc):
                fake.current.pop()

        def stream_of(raw, device=None):
            return types.SimpleNamespace(cuda_stream=raw)

        mp.setattr(torch.cuda, "current_device", lambda: 0)
        mp.setattr(torch.Tensor, "get_device", lambda t: 0)
        mp.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: self.current[-1], raising=False)
        mp.setattr(torch.cuda, "current_stream", lambda device=None: stream_of(self.current[-1]))
        mp.setattr(torch.cuda, "ExternalStream", stream_of)
        mp.setattr(torch.cuda, "stream", On)
        mp.setattr(torch.Tensor, "record_stream", lambda t, s: self.shared.append((t.data_ptr(), s.cuda_stream)),
                   raising=False)
        mp.setattr(lrkv, "_check", lambda *specs: None)
        mp.setattr(lrkv, "load", lambda path=None: self.lib)
        for name in ("empty", "zeros", "empty_like"):
            mp.setattr(torch, name, self.noting(name, getattr(torch, name)))

    def noting(self, name, make):
        def made(*args, **kw):
            t = make(*args, **kw)
            self.made.append((name, t, self.current[-1]))
            return t
        return made


@pytest.fixture
def fake(monkeypatch):
    return Fake(monkeypatch)


B, H, DH, R, L = 2, 16, 64, 32, 48


def _tensors():
    bf = lambda *s: torch.ones(s, dtype=torch.bfloat16)
    i = lambda *s: torch.ones(s, dtype=torch.int32)
    q, k, z, b = bf(B, H, DH), bf(B, L, DH), bf(B, L, H, R), bf(H, DH, R)
    return types.SimpleNamespace(q=q, k=k, z=z, b=b, lens=i(B), weights=torch.ones(B, L), pos=i(B, L, 2),
                                 table=torch.ones(L, DH), lse=torch.ones(B, H, 4), prompt=bf(B, 4, H, DH),
                                 decode=(q, k, k, z, z, b, b),
                                 append=(bf(B, 8),) + (bf(DH, 8),) * 2 + (bf(H * R, 8),) * 2)


def weighted(t, stream):
    return lrkv.decode_weighted(*t.decode, t.lens, None, decay=0.0, stream=stream)


def prompt(t, stream):
    return lrkv.prefill_weights(t.prompt, t.k, t.z, t.b, t.lse, t.lens, None, decay=0.0, stream=stream)


@pytest.mark.parametrize("call", [weighted, prompt])
@pytest.mark.parametrize("stream, want", [(None, HERE), (HERE, HERE), (OWN, OWN)])
def test_weights_not_given_are_cleared_on_the_call_s_stream(fake, call, stream, want):
    t = _tensors()
    fake.made.clear()
    call(t, stream)
    fills = [(tuple(x.shape), on) for name, x, on in fake.made if name == "zeros"]
    assert fills == [((B, L), want)]
    assert [s for _, s in fake.lib.calls] == [want] and fake.current == [HERE]


CALLS = dict(
    decode_weighted=(weighted, 4), prefill_weights=(prompt, 2),    # calls and the allocations of each
    evict=(lambda t, s: lrkv.evict(t.k, t.k, t.z, t.z, t.weights, t.lens, 8, stream=s), 1),
    rope_rotate=(lambda t, s: lrkv.rope_rotate(t.prompt, t.pos[:, :4].contiguous(), t.table, [16, 16], stream=s), 1),
    decode_rope_axes=(lambda t, s: lrkv.decode_rope_axes(*t.decode, t.table, t.pos, [16, 16], t.lens, stream=s), 3),
    decode=(lambda t, s: lrkv.decode(*t.decode, t.lens, stream=s), 3),
    decode_normed=(lambda t, s: lrkv.decode_normed(*t.decode, t.lse, t.lens, stream=s), 3),
    decode_paged=(lambda t, s: lrkv.decode_paged(*t.decode, t.pos[..., 0], t.lens, stream=s), 3),
    decode_rope=(lambda t, s: lrkv.decode_rope(*t.decode, t.table, t.lens, stream=s), 3),
    decode_step=(lambda t, s: lrkv.decode_step(*t.append, *t.decode, t.lens, stream=s), 3),
    decode_step_paged=(lambda t, s: lrkv.decode_step_paged(*t.append, *t.decode, t.pos[..., 0], t.lens, stream=s), 3),
    prefill=(lambda t, s: lrkv.prefill(t.prompt, *t.decode[1:], t.lens, stream=s), 3),
    prefill_normed=(lambda t, s: lrkv.prefill_normed(t.prompt, *t.decode[1:], t.lse, t.lens, stream=s), 3),
    prefill_paged=(lambda t, s: lrkv.prefill_paged(t.prompt, *t.decode[1:], t.pos[..., 0], t.lens, stream=s), 3),
    append=(lambda t, s: lrkv.append(t.q, *t.append[1:], t.lens, *t.decode[1:5], stream=s), 1),
    append_paged=(lambda t, s: lrkv.append_paged(t.q, *t.append[1:], t.lens, t.pos[..., 0], *t.decode[1:5], H,
                                                 stream=s), 1),
    dense_decode=(lambda t, s: lrkv.dense_decode(t.q, t.z, t.z, t.lens, stream=s), 3),
    mla_decode=(lambda t, s: lrkv.mla_decode(t.q, t.k, t.b, t.b, t.lens, stream=s), 3),
    rope_table=(lambda t, s: lrkv.rope_table(L, DH, device="cpu", stream=s), 1))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream, want", [(None, HERE), (HERE, HERE), (OWN, OWN)])
def test_allocations_belong_to_the_call_s_stream(fake, call, stream, want):
    t = _tensors()
    fake.made.clear()
    run, n = CALLS[call]
    run(t, stream)
    fake.made[:] = [m for m in fake.made if m[1].numel()]
    assert [on for _, _, on in fake.made] == [want] * n
    assert fake.lib.calls[0][1] == want and fake.current == [HERE]
    # ... and are known to the allocator as used on the caller's stream too
    assert fake.shared == ([(x.data_ptr(), HERE) for _, x, _ in fake.made] if want == OWN else [])


# ------------------------------------------------------------------ on the GPU --

@pytest.fixture
def case():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()
    d = T.cuda(inputs.random_decode_case(seed=3, batch=2, heads=16, head_dim=128, rank=64, max_len=600, dtype="bf16",
                                         lens=[600, 41]))
    p = T.cuda(inputs.random_prefill_case(seed=2, batch=2, q_len=20, heads=16, head_dim=128, rank=64, max_len=600,
                                          lens=[600, 41]))
    lse = torch.full((2, 16, 20), 8.0, device="cuda")
    torch.cuda.synchronize()
    return dict(
        weighted=lambda s: lrkv.decode_weighted(*[d[k] for k in T.NAMES], None, decay=0.0, stream=s)[2],
        prompt=lambda s: lrkv.prefill_weights(p["q"], p["k_s"], p["z_k"], p["b_k"], lse, p["seq_lens"], None,
                                              decay=0.0, stream=s)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["weighted", "prompt"])
@pytest.mark.parametrize("raw", [False, True])
def test_weights_are_whole_while_the_current_stream_is_busy(case, call, raw):
    want = case[call](None).clone()
    torch.cuda.synchronize()
    assert float(want.abs().sum()) > 0
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)           # about 0.1 s of the current stream
    got = case[call](s.cuda_stream if raw else s)
    s.synchronize()
    with torch.cuda.stream(s):
        early = got.clone()
    torch.cuda.synchronize()
    assert torch.equal(early, want) and torch.equal(got, want)


@pytest.mark.gpu
def test_a_dropped_workspace_is_not_handed_out_while_the_call_uses_it():
    """Calls queued behind a busy stream of their own, their workspaces dropped at
    once, while blocks of the same size are taken and filled on the current one."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    B, H, dh, r, Lm, budget = 4, 8, 64, 32, 3000, 900
    case = T.cuda(inputs.random_decode_case(seed=5, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                            lens=[3000, 2999, 1500, 900]))
    weights = torch.rand((B, Lm), generator=torch.Generator().manual_seed(1)).cuda()

    def state():
        return [case[k].clone() for k in ("k_s", "v_s", "z_k", "z_v")] + [weights.clone(), case["seq_lens"].clone()]

    want, got = state(), state()
    lrkv.evict(*want, budget, sink=1, recent=3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    size = lrkv.evict_workspace(B, Lm, budget).numel()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    lrkv.evict(*got, budget, sink=1, recent=3, stream=s)
    others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del others
