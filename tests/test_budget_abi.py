"""Refusals of the calls that keep a cache inside a token budget: every bad
argument is turned away on the host, before anything is enqueued (no GPU is
needed; the addresses are fakes that are never dereferenced)."""
import ctypes

import pytest
import torch

from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv

FAKE = 1 << 20
BAD, NO, SPACE = lrkv.LRKV_ERR_INVALID_ARG, lrkv.LRKV_ERR_UNSUPPORTED, lrkv.LRKV_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _lib(request):
    ensure_built()
    mp = pytest.MonkeyPatch()
    mp.setenv("LRKV_SM_COUNT", "152")     # plans without a device
    request.addfinalizer(mp.undo)


def bf(B=2, H=16, dh=64, r=32, L=256, dtype="bf16", scale=0.0):
    return lrkv.make_dims(B, H, dh, r, L, dtype, scale)


def call(name, order, defaults, **kw):
    a = dict(defaults, **kw)
    dims = a.pop("dims")
    return int(getattr(lrkv.load(), name)(None if dims is None else ctypes.byref(dims), *[a[k] for k in order]))


def size(name, *args):
    n = ctypes.c_size_t(0)
    st = int(getattr(lrkv.load(), name)(*args, ctypes.byref(n)))
    return st, n.value


DECODE = ("q page_size num_pages block_table k_s v_s z_k z_v b_k b_v key_scale seq_lens decay weights weights_out "
          "out lse ws ws_bytes stream").split()
DECODE_OK = dict(dims=bf(), q=FAKE, page_size=0, num_pages=0, block_table=None, k_s=FAKE, v_s=FAKE, z_k=FAKE,
                 z_v=FAKE, b_k=FAKE, b_v=FAKE, key_scale=None, seq_lens=FAKE, decay=1.0, weights=FAKE,
                 weights_out=FAKE, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SPACE, {}), (SPACE, dict(ws=None)), (BAD, dict(ws=FAKE + 4)), (BAD, dict(dims=None)),
    (BAD, dict(q=None)), (BAD, dict(q=FAKE + 8)), (BAD, dict(k_s=None)), (BAD, dict(v_s=FAKE + 2)),
    (BAD, dict(z_k=None)), (BAD, dict(z_v=FAKE + 8)), (BAD, dict(b_k=None)), (BAD, dict(b_v=None)),
    (BAD, dict(seq_lens=None)), (BAD, dict(out=None)), (BAD, dict(lse=None)), (BAD, dict(weights_out=None)),
    (BAD, dict(weights=None)), (SPACE, dict(weights=None, decay=0.0)), (BAD, dict(decay=-0.5)),
    (BAD, dict(decay=float("nan"))), (BAD, dict(decay=float("inf"))),
    (BAD, dict(block_table=FAKE, page_size=24, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=8, num_pages=4)),
    (BAD, dict(block_table=FAKE, page_size=512, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=64, num_pages=0)),
    (NO, dict(block_table=FAKE, page_size=64, num_pages=1 << 26)),
    (NO, dict(dims=bf(dtype="f32"))), (NO, dict(dims=bf(r=30))), (NO, dict(dims=bf(dh=96))),
    (BAD, dict(dims=bf(B=0))), (BAD, dict(dims=bf(scale=float("nan")))),
])
def test_decode_weighted(want, kw):
    assert call("lrkv_decode_weighted", DECODE, DECODE_OK, **kw) == want


PROMPT = ("q_len window q page_size num_pages block_table k_s z_k b_k key_scale lse seq_lens decay weights "
          "weights_out ws ws_bytes stream").split()
PROMPT_OK = dict(dims=bf(), q_len=64, window=16, q=FAKE, page_size=0, num_pages=0, block_table=None, k_s=FAKE,
                 z_k=FAKE, b_k=FAKE, key_scale=None, lse=FAKE, seq_lens=FAKE, decay=1.0, weights=FAKE,
                 weights_out=FAKE, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SPACE, {}), (SPACE, dict(ws=None)), (BAD, dict(ws=FAKE + 4)), (BAD, dict(dims=None)),
    (BAD, dict(window=0)), (BAD, dict(window=65)), (NO, dict(q_len=257)), (BAD, dict(q_len=-1)),
    (NO, dict(window=300, q_len=300)), (BAD, dict(q=None)), (BAD, dict(q=FAKE + 8)), (BAD, dict(k_s=None)),
    (BAD, dict(z_k=None)), (BAD, dict(z_k=FAKE + 8)), (BAD, dict(b_k=None)), (BAD, dict(lse=None)),
    (BAD, dict(seq_lens=None)), (BAD, dict(weights_out=None)), (BAD, dict(weights=None)),
    (SPACE, dict(weights=None, decay=0.0)), (BAD, dict(decay=-1.0)), (BAD, dict(decay=float("nan"))),
    (BAD, dict(block_table=FAKE, page_size=8, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=48, num_pages=4)),
    (BAD, dict(block_table=FAKE, page_size=512, num_pages=4)),
    (NO, dict(dims=bf(dtype="f32"))), (NO, dict(dims=bf(dh=96))), (NO, dict(dims=bf(r=28))), (NO, dict(dims=bf(r=72))),
    (NO, dict(dims=bf(H=512))), (BAD, dict(dims=bf(L=0))), (SPACE, dict(dims=bf(r=0), z_k=None, b_k=None)),
])
def test_prefill_weights(want, kw):
    assert call("lrkv_prefill_weights", PROMPT, PROMPT_OK, **kw) == want


EVICT = ("budget sink recent weights order seq_lens page_size num_pages block_table k_s v_s z_k z_v key_scale "
         "positions axes weights_out order_out new_lens kept ws ws_bytes stream").split()
EVICT_OK = dict(dims=bf(), budget=100, sink=2, recent=8, weights=FAKE, order=None, seq_lens=FAKE, page_size=0,
                num_pages=0, block_table=None, k_s=FAKE, v_s=FAKE, z_k=FAKE, z_v=FAKE, key_scale=None,
                positions=None, axes=0, weights_out=FAKE, order_out=None, new_lens=FAKE, kept=None, ws=FAKE,
                ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SPACE, {}), (SPACE, dict(ws=None)), (BAD, dict(ws=FAKE + 4)), (BAD, dict(dims=None)),
    (BAD, dict(budget=0)), (BAD, dict(budget=257)), (SPACE, dict(budget=256)), (BAD, dict(sink=-1)),
    (BAD, dict(recent=-1)), (BAD, dict(sink=50, recent=51)), (BAD, dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)),
    (BAD, dict(weights=None)), (BAD, dict(seq_lens=None)), (BAD, dict(weights_out=None)), (BAD, dict(new_lens=None)),
    (BAD, dict(k_s=None)), (BAD, dict(k_s=FAKE + 8)), (BAD, dict(v_s=FAKE + 2)), (BAD, dict(z_k=None)),
    (BAD, dict(z_v=FAKE + 4)), (SPACE, dict(dims=bf(r=0), z_k=None, z_v=None)),
    (BAD, dict(positions=FAKE)), (BAD, dict(positions=FAKE, axes=5)), (BAD, dict(axes=1)),
    (BAD, dict(block_table=FAKE, page_size=24, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=64, num_pages=0)),
    (BAD, dict(block_table=FAKE, page_size=512, num_pages=4)),
    (NO, dict(dims=bf(dh=60))), (NO, dict(dims=bf(H=3, r=4))), (NO, dict(dims=bf(B=5000))),
    (NO, dict(dims=bf(B=4000, L=1 << 20))), (BAD, dict(dims=bf(dtype=7))), (BAD, dict(dims=bf(H=0))),
])
def test_evict(want, kw):
    assert call("lrkv_evict", EVICT, EVICT_OK, **kw) == want


def sections(*s):
    return (ctypes.c_int * len(s))(*s)


ROTATE = "n x positions axes sections cos_sin max_pos out ws ws_bytes stream".split()
ROTATE_OK = dict(dims=bf(), n=1, x=FAKE, positions=FAKE, axes=2, sections=sections(8, 24), cos_sin=FAKE, max_pos=64,
                 out=FAKE, ws=FAKE, ws_bytes=8, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SPACE, {}), (BAD, dict(ws=FAKE + 4, ws_bytes=16)), (BAD, dict(dims=None)), (BAD, dict(n=0)),
    (BAD, dict(x=None)), (BAD, dict(x=FAKE + 4)), (BAD, dict(out=None)), (BAD, dict(out=FAKE + 8)),
    (BAD, dict(positions=None)), (BAD, dict(cos_sin=None)), (BAD, dict(cos_sin=FAKE + 4)), (BAD, dict(max_pos=0)),
    (BAD, dict(axes=0)), (BAD, dict(axes=5, sections=sections(8, 6, 6, 6, 6))), (BAD, dict(sections=None)),
    (BAD, dict(sections=sections(8, 23))), (BAD, dict(sections=sections(8, 25))),
    (BAD, dict(sections=sections(-1, 33))), (BAD, dict(sections=sections(2 ** 31 - 1, 2 ** 31 - 1))),
    (NO, dict(dims=bf(dh=36), sections=sections(8, 10))), (BAD, dict(dims=bf(dh=1))),
    (NO, dict(dims=bf(dh=2048), sections=sections(0, 1024))), (BAD, dict(dims=bf(dtype=5))),
])
def test_rope_rotate(want, kw):
    assert call("lrkv_rope_rotate", ROTATE, ROTATE_OK, **kw) == want


ROPE = ("q k_s v_s z_k z_v b_k b_v cos_sin max_pos positions axes sections seq_lens decay weights weights_out out lse "
        "ws ws_bytes stream").split()
ROPE_OK = dict(dims=bf(), q=FAKE, k_s=FAKE, v_s=FAKE, z_k=FAKE, z_v=FAKE, b_k=FAKE, b_v=FAKE, cos_sin=FAKE,
               max_pos=64, positions=FAKE, axes=2, sections=sections(8, 24), seq_lens=FAKE, decay=1.0, weights=None,
               weights_out=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SPACE, {}), (SPACE, dict(ws=None)), (BAD, dict(ws=FAKE + 4)), (BAD, dict(dims=None)),
    (BAD, dict(q=None)), (BAD, dict(q=FAKE + 8)), (BAD, dict(k_s=None)), (BAD, dict(z_v=FAKE + 4)),
    (BAD, dict(b_k=FAKE + 8)), (BAD, dict(b_v=None)), (BAD, dict(cos_sin=None)), (BAD, dict(max_pos=0)),
    (BAD, dict(positions=None)), (BAD, dict(axes=3)), (BAD, dict(sections=sections(8, 8))),
    (BAD, dict(seq_lens=None)), (BAD, dict(out=None)), (BAD, dict(weights_out=FAKE)),          # weights need lse
    (BAD, dict(weights_out=FAKE, lse=FAKE)), (SPACE, dict(weights_out=FAKE, lse=FAKE, weights=FAKE)),
    (SPACE, dict(weights_out=FAKE, lse=FAKE, decay=0.0)), (BAD, dict(weights_out=FAKE, lse=FAKE, weights=FAKE, decay=-1.0)),
    (NO, dict(dims=bf(r=28))), (NO, dict(dims=bf(H=12))), (NO, dict(dims=bf(dh=96))), (NO, dict(dims=bf(dtype="f32"))),
])
def test_decode_rope_axes(want, kw):
    if kw.get("axes") == 3:
        kw = dict(kw, sections=sections(8, 8, 8))
    assert call("lrkv_decode_rope_axes", ROPE, ROPE_OK, **kw) == want


def test_workspace_sizes():
    d = ctypes.byref(bf())
    st, n = size("lrkv_decode_weighted_workspace_size", d)
    assert st == 0 and n >= 4 * 2 * 16 * 256 + size("lrkv_decode_workspace_size", d)[1]
    assert size("lrkv_decode_weighted_workspace_size", ctypes.byref(bf(dtype="f32")))[0] == NO
    assert size("lrkv_decode_weighted_workspace_size", None)[0] == BAD
    assert size("lrkv_prefill_weights_workspace_size", d, 16)[0] == 0
    assert size("lrkv_prefill_weights_workspace_size", d, 0)[0] == BAD
    assert size("lrkv_prefill_weights_workspace_size", d, 257)[0] == NO
    assert size("lrkv_evict_workspace_size", 2, 256, 100)[0] == 0
    assert size("lrkv_evict_workspace_size", 2, 256, 0)[0] == BAD
    assert size("lrkv_evict_workspace_size", 2, 256, 257)[0] == BAD
    assert size("lrkv_evict_workspace_size", 5000, 256, 100)[0] == NO
    # row numbers, rounded up to what a CTA takes, stay in 32 bits
    assert size("lrkv_evict_workspace_size", 1, 2 ** 31 - 2 ** 16, 100)[0] == 0
    assert size("lrkv_evict_workspace_size", 1, 2 ** 31 - 2 ** 16 + 1, 100)[0] == NO
    assert size("lrkv_evict_workspace_size", 2, 2 ** 30, 100)[0] == NO
    assert size("lrkv_prefill_weights_workspace_size", ctypes.byref(bf(B=1, r=0, L=2 ** 31 - 1)), 16)[0] == NO
    assert size("lrkv_decode_rope_axes_workspace_size", d)[0] == 0
    assert size("lrkv_decode_rope_axes_workspace_size", ctypes.byref(bf(r=28)))[0] == NO
    # a size that passes 32 bits
    big = bf(B=8, H=256, dh=64, r=8, L=1 << 20)
    st, n = size("lrkv_decode_weighted_workspace_size", ctypes.byref(big))
    assert st == NO or n > 1 << 32


def test_the_binding_checks_tensors():
    """Types, shapes, layout and device are checked before the library is called."""
    f, i = torch.float32, torch.int32
    q = torch.zeros(2, 16, 64, dtype=torch.bfloat16)
    k, z = torch.zeros(2, 40, 64, dtype=torch.bfloat16), torch.zeros(2, 40, 16, 32, dtype=torch.bfloat16)
    b, lens, w = torch.zeros(16, 64, 32, dtype=torch.bfloat16), torch.zeros(2, dtype=i), torch.zeros(2, 40)
    good = (q, k, k, z, z, b, b, lens, w)

    def refused(fn, *args, match, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*args, **kw)

    refused(lrkv.decode_weighted, *good[:7], lens.long(), w, match="seq_lens")
    refused(lrkv.decode_weighted, *good[:8], w[:, :39].contiguous(), match="weights")
    refused(lrkv.decode_weighted, *good[:8], w.double(), match="weights")
    refused(lrkv.decode_weighted, q, torch.zeros(2, 64, 40, dtype=q.dtype).transpose(1, 2), *good[2:],
            match="contiguous")
    refused(lrkv.decode_weighted, q, k.float(), *good[2:], match="k_s")
    refused(lrkv.decode_weighted, *good[:5], b[:8].contiguous(), b, lens, w, match="b_k")
    refused(lrkv.decode_weighted, *good, match="key_scale", key_scale=torch.zeros(2, 16, 41))
    refused(lrkv.decode_weighted, *good, match="CUDA")                 # right in all but the device
    refused(lrkv.prefill_weights, q[:, None], k, z, b, torch.zeros(2, 16, 2), lens, w, match="lse")
    refused(lrkv.prefill_weights, q[:, None], k, z, b, torch.zeros(2, 16, 1), lens, w.to(torch.float16), match="weights")
    refused(lrkv.evict, k, k, z, z, w, lens, 8, match="order", order=torch.zeros(2, 40))
    refused(lrkv.evict, k, k, z, z, w, lens, 8, match="kept", kept=torch.zeros(2, 9, dtype=i))
    refused(lrkv.evict, k, k, z, z, w, lens, 8, match="positions", positions=torch.zeros(2, 39, 3, dtype=i))
    refused(lrkv.evict, k, k, z, z[:, :39].contiguous(), w, lens, 8, match="z_v")
    table = torch.zeros(10, 64)
    refused(lrkv.rope_rotate, q[:, None], torch.zeros(2, 1, 2, dtype=i), table, [8, 8, 16], match="positions")
    refused(lrkv.rope_rotate, q[:, None], torch.zeros(2, 1, 3, dtype=i), table.double(), [8, 8, 16], match="cos_sin")
    refused(lrkv.rope_rotate, q[:, None], torch.zeros(2, 1, 3, dtype=i), table, [8, 8, 16], match="out",
            out=torch.zeros(2, 1, 16, 64, dtype=f))
    refused(lrkv.decode_rope_axes, *good[:7], table, torch.zeros(2, 40, 2, dtype=i), [8, 8, 16], lens, match="positions")
