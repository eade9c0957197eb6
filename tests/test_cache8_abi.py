"""Refusals of the 8-bit cache's and the pages' calls: every bad argument is
turned away on the host, before anything is enqueued (no GPU is needed; the
addresses are fakes that are never dereferenced), and the binding's own checks
of what it is given."""
import ctypes
import struct

import pytest
import torch

from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv
from test_call_streams import HERE, OWN, Fake

FAKE = 1 << 20
OK, BAD, NO, SPACE = lrkv.LRKV_OK, lrkv.LRKV_ERR_INVALID_ARG, lrkv.LRKV_ERR_UNSUPPORTED, lrkv.LRKV_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _lib(request):
    ensure_built()
    mp = pytest.MonkeyPatch()
    mp.setenv("LRKV_SM_COUNT", "152")     # plans without a device
    request.addfinalizer(mp.undo)


def dims(B=2, H=16, dh=64, r=32, L=256, dtype="bf16", scale=0.0):
    return lrkv.make_dims(B, H, dh, r, L, dtype, scale)


def call(name, order, defaults, **kw):
    a = dict(defaults, **kw)
    d, c = a.pop("dims"), a.pop("cache")
    a["cache"] = None if c is None else ctypes.byref(c)
    return int(getattr(lrkv.load(), name)(None if d is None else ctypes.byref(d), *[a[k] for k in order]))


def cache(**kw):
    c = lrkv.lrkv_cache8(*[FAKE] * 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


NO_Z = dict(z_k=None, z_v=None, z_k_scale=None, z_v_scale=None)
SHAPES = [  # of both calls
    (BAD, dict(dims=None)), (BAD, dict(dims=dims(B=0))), (BAD, dict(dims=dims(H=0))), (BAD, dict(dims=dims(dh=0))),
    (BAD, dict(dims=dims(r=-2))), (BAD, dict(dims=dims(L=0))), (BAD, dict(dims=dims(dtype=7))),
    (BAD, dict(dims=dims(scale=float("nan")))), (NO, dict(dims=dims(dh=24))), (NO, dict(dims=dims(dh=272))),
    (NO, dict(dims=dims(r=33))), (NO, dict(dims=dims(r=66))), (NO, dict(dims=dims(H=3, r=2))), (NO, dict(dims=dims(H=272))),
    (NO, dict(dims=dims(B=4097))), (NO, dict(dims=dims(B=4096, L=1 << 20))),
    (BAD, dict(cache=None)), (BAD, dict(cache=cache(k_s=None))), (BAD, dict(cache=cache(v_s_scale=None))),
    (BAD, dict(cache=cache(z_k=None))), (BAD, dict(cache=cache(z_v_scale=None))), (BAD, dict(cache=cache(z_v=FAKE + 8))),
    (BAD, dict(cache=cache(k_s_scale=FAKE + 4))),
    (BAD, dict(block_table=FAKE, page_size=24, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=8, num_pages=4)),
    (BAD, dict(block_table=FAKE, page_size=512, num_pages=4)), (BAD, dict(block_table=FAKE, page_size=64, num_pages=0)),
    (NO, dict(block_table=FAKE, page_size=64, num_pages=1 << 26)), (BAD, dict(ws=FAKE + 8)),
]

DECODE = "q page_size num_pages block_table cache b_k b_v seq_lens out lse ws ws_bytes stream".split()
DECODE_OK = dict(dims=dims(), q=FAKE, page_size=0, num_pages=0, block_table=None, cache=cache(), b_k=FAKE, b_v=FAKE,
                 seq_lens=FAKE, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", SHAPES + [
    (SPACE, {}), (SPACE, dict(ws=None)), (SPACE, dict(lse=None)), (BAD, dict(q=None)), (BAD, dict(q=FAKE + 8)),
    (BAD, dict(b_k=None)), (BAD, dict(b_v=None)), (BAD, dict(b_k=FAKE + 2)), (BAD, dict(b_v=FAKE + 2)),
    (BAD, dict(seq_lens=None)), (BAD, dict(out=None)), (NO, dict(dims=dims(dtype="f32"))),
    (SPACE, dict(dims=dims(r=0), cache=cache(**NO_Z), b_k=None, b_v=None)), (SPACE, dict(dims=dims(dh=256, r=64))),
    (SPACE, dict(block_table=FAKE, page_size=16, num_pages=4)),
])
def test_decode8(want, kw):
    assert call("lrkv_decode8", DECODE, DECODE_OK, **kw) == want


QUANTIZE = ("n_new k_s v_s z_k z_v start_pos new_lens page_size num_pages block_table cache ws ws_bytes stream").split()
QUANTIZE_OK = dict(dims=dims(), n_new=3, k_s=FAKE, v_s=FAKE, z_k=FAKE, z_v=FAKE, start_pos=FAKE, new_lens=None,
                   page_size=0, num_pages=0, block_table=None, cache=cache(), ws=FAKE, ws_bytes=8, stream=None)


@pytest.mark.parametrize("want, kw", SHAPES + [
    (SPACE, {}), (SPACE, dict(dims=dims(dtype="f32"))), (BAD, dict(n_new=0)), (BAD, dict(n_new=-1)),
    (BAD, dict(k_s=None)), (BAD, dict(v_s=FAKE + 2)), (BAD, dict(z_k=None)), (BAD, dict(z_v=FAKE + 8)),
    (BAD, dict(start_pos=None)), (NO, dict(n_new=1 << 30)),
    (SPACE, dict(dims=dims(r=0), cache=cache(**NO_Z), z_k=None, z_v=None)),
])
def test_quantize(want, kw):
    assert call("lrkv_quantize", QUANTIZE, QUANTIZE_OK, **kw) == want


def size(name, *args):
    n = ctypes.c_size_t(0)
    return int(getattr(lrkv.load(), name)(*args, ctypes.byref(n))), n.value


def test_workspace_sizes():
    assert size("lrkv_decode8_workspace_size", ctypes.byref(dims()))[0] == OK
    assert size("lrkv_decode8_workspace_size", ctypes.byref(dims(dtype="f32")))[0] == NO
    assert lrkv.load().lrkv_decode8_workspace_size(ctypes.byref(dims()), None) == BAD
    for d in (16, 48, 128, 256):                     # every shape that the calls take has a plan
        for r in (0, 2, 28, 62, 64):
            for H in (8, 24, 256):
                for B in (1, 4096):
                    assert size("lrkv_decode8_workspace_size", ctypes.byref(dims(B, H, d, r)))[0] == OK, (d, r, H, B)
    small, large = (size("lrkv_pages_workspace_size", 4, 8, n) for n in (10, 100000))
    assert small[0] == large[0] == OK and large[1] > small[1] + 100000 * 12
    for bad in ((0, 8, 10), (4, 0, 10), (4, 8, 0)):
        assert size("lrkv_pages_workspace_size", *bad)[0] == BAD
    for no in ((4097, 8, 10), (4096, 1 << 20, 10), (4, 8, (1 << 30) + 1)):
        assert size("lrkv_pages_workspace_size", *no)[0] == NO
    assert lrkv.load().lrkv_pages_workspace_size(4, 8, 10, None) == BAD


def pool(data=FAKE, rows=1, bytes_=64):
    return struct.pack("Pii", data or 0, rows, bytes_)


PAGES = dict(batch=4, blocks=8, page=32, pages=10, parent=None, keep=None, new_lens=FAKE, table=FAKE, lens=FAKE,
             refs=FAKE, table_out=FAKE, lens_out=FAKE, refs_out=FAKE, missing=None, moved=None, live=None, pools=pool(),
             n_pools=1, ws=FAKE, ws_bytes=0, stream=None)
ORDER = dict(
    fork="batch blocks page pages parent keep table lens refs table_out lens_out refs_out ws ws_bytes stream",
    extend="batch blocks page pages new_lens table lens refs table_out lens_out refs_out missing pools n_pools ws "
           "ws_bytes stream",
    compact="batch blocks page pages table lens refs table_out refs_out moved live pools n_pools ws ws_bytes stream")
GENERAL = [(SPACE, {}), (SPACE, dict(ws=None)), (BAD, dict(ws=FAKE + 4)), (BAD, dict(batch=0)), (BAD, dict(blocks=0)),
           (BAD, dict(pages=0)), (BAD, dict(page=8)), (BAD, dict(page=48)), (BAD, dict(table=None)), (BAD, dict(lens=None)),
           (BAD, dict(refs=None)), (BAD, dict(table_out=None)), (BAD, dict(refs_out=None)), (NO, dict(batch=5000)),
           (NO, dict(blocks=1 << 27, page=32)), (NO, dict(pages=(1 << 30) + 1))]
POOLS = [(BAD, dict(n_pools=-1)), (BAD, dict(n_pools=17)), (BAD, dict(pools=None)), (BAD, dict(pools=pool(0))),
         (BAD, dict(pools=pool(FAKE + 2))), (BAD, dict(pools=pool(rows=0))), (BAD, dict(pools=pool(rows=64))),
         (BAD, dict(pools=pool(rows=3))), (BAD, dict(pools=pool(bytes_=6))), (BAD, dict(pools=pool(bytes_=0)))]


@pytest.mark.parametrize("name, want, kw", [(n, w, k) for n in ORDER for w, k in GENERAL]
                         + [(n, w, k) for n in ("extend", "compact") for w, k in POOLS]
                         + [("fork", BAD, dict(lens_out=None)), ("extend", BAD, dict(lens_out=None)),
                            ("extend", BAD, dict(new_lens=None))])
def test_pages(name, want, kw):
    if "pools" in kw or "n_pools" in kw:
        kw = dict(kw, ws_bytes=1 << 20)     # (a pool is looked at once the workspace is found to do)
    a = dict(PAGES, **kw)
    assert int(getattr(lrkv.load(), f"lrkv_pages_{name}")(*[a[k] for k in ORDER[name].split()])) == want


def test_status_string_and_code():
    assert lrkv.LRKV_ERR_NO_PAGES == 7 and lrkv.status_string(7) == "LRKV_ERR_NO_PAGES"


# ------------------------------------------------- the binding, on a stand-in --

B, H, DH, R, L = 2, 16, 64, 32, 48


@pytest.fixture
def fake(monkeypatch):
    return Fake(monkeypatch)


def tensors():
    e = torch.float8_e4m3fn
    c = lrkv.Cache8(torch.zeros(B, L, DH, dtype=e), torch.zeros(B, L, DH, dtype=e), torch.zeros(B, L, H, R, dtype=e),
                    torch.zeros(B, L, H, R, dtype=e), torch.ones(B, 3), torch.ones(B, 3), torch.ones(B, 3, H),
                    torch.ones(B, 3, H))
    i = lambda *s: torch.ones(s, dtype=torch.int32)
    return c, torch.ones(B, H, DH).bfloat16(), torch.ones(H, DH, R).bfloat16(), i


@pytest.mark.parametrize("stream, want", [(None, HERE), (HERE, HERE), (OWN, OWN)])
@pytest.mark.parametrize("call, made", [
    (lambda c, q, b, i, s: lrkv.decode8(q, c, b, b, i(B), stream=s), 3),
    (lambda c, q, b, i, s: lrkv.pages_fork(i(B, 4), i(B), i(9), 16, stream=s), 1),
    (lambda c, q, b, i, s: lrkv.pages_extend([torch.ones(9, 16, 4)], i(B, 4), i(B), i(9), 16, i(B), stream=s), 1),
    (lambda c, q, b, i, s: lrkv.pages_compact([torch.ones(9, 1, 4)], i(B, 4), i(B), i(9), 16, stream=s), 1),
])
def test_allocations_belong_to_the_call_s_stream(fake, call, made, stream, want):
    c, q, b, i = tensors()
    fake.made.clear()
    call(c, q, b, i, stream)
    got = [(t.data_ptr(), on) for name, t, on in fake.made if name == "empty"]
    assert len(got) == made and all(on == want for _, on in got)
    assert [s for _, s in fake.lib.calls if s is not None][-1] == want and fake.current == [HERE]


def test_the_binding_looks_at_what_it_is_given(monkeypatch):
    """Types, shapes and layouts, checked on the device number of fakes that live on the CPU."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    c, q, b, i = tensors()
    e = torch.float8_e4m3fn
    parts = {n: getattr(c, n) for n in c.NAMES}
    for wrong in (dict(k_s=parts["k_s"].view(torch.uint8)), dict(v_s=torch.zeros(B, L + 1, DH, dtype=e)),
                  dict(z_k=None), dict(z_v=torch.zeros(B, L, H, R + 2, dtype=e)), dict(k_s_scale=torch.ones(B, 4)),
                  dict(z_v_scale=torch.ones(B, 3, H, dtype=torch.float64)),
                  dict(z_k_scale=torch.ones(B, H, 3).transpose(1, 2))):
        with pytest.raises(ValueError):
            lrkv.Cache8(**dict(parts, **wrong))
    with pytest.raises(ValueError):   # another rank, another batch, another width
        lrkv.decode8(q, c, b[..., :16].contiguous(), b[..., :16].contiguous(), i(B))
    with pytest.raises(ValueError):
        lrkv.decode8(torch.ones(3, H, DH).bfloat16(), c, b, b, i(3))
    with pytest.raises(ValueError):
        lrkv.decode8(torch.ones(B, 8, DH).bfloat16(), c, b[:8], b[:8], i(B))
    with pytest.raises(ValueError):
        lrkv.decode8(q, c, b, b, i(B).long())
    row, z = torch.ones(B, 2, DH).bfloat16(), torch.ones(B, 2, H, R).bfloat16()
    with pytest.raises(ValueError):
        lrkv.quantize(row, row.float(), z, z, i(B), c)
    with pytest.raises(ValueError):
        lrkv.quantize(row, row, z, z[:, :1].contiguous(), i(B), c)
    with pytest.raises(ValueError):
        lrkv.quantize(row, row, z, z, i(B), c, new_lens=i(3))
    for pools in ([torch.ones(9)], [torch.ones(8, 16)], [torch.ones(9, 3)], [torch.ones(9, 0, 4)],
                  [torch.ones(16, 9).t()]):
        with pytest.raises(ValueError):
            lrkv.pages_compact(pools, i(B, 4), i(B), i(9), 16)
    with pytest.raises(ValueError):
        lrkv.pages_fork(i(B, 4), i(3), i(9), 16)
    with pytest.raises(ValueError):
        lrkv.pages_fork(i(B, 4), i(B), i(9), 16, parent=i(B).long())
