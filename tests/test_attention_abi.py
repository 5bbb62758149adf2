"""Argument checks of the attention block's entry points (CPU only: every call
here is refused, or has nothing to do, before any CUDA call)."""

import ctypes
import struct

import pytest

FAKE = 0x10000  # never dereferenced
OK, INVALID, ALIGNMENT, SHAPE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def raw():
    return pytest.importorskip("fp8_w8a8_linear_b200").raw


def _kv(k=FAKE, v=FAKE, pages=4, page_size=16, heads=2, D=64, page_stride=2048, token_stride=128, head_stride=64, table=FAKE,
        batch=2, max_pages=2, cu_q=FAKE, kv_lens=FAKE):
    return struct.pack("@PP7qPqqPP", k, v, pages, page_size, heads, D, page_stride, token_stride, head_stride, table, batch,
                       max_pages, cu_q, kv_lens)


def test_struct_layout_matches_the_header():
    class S(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
            (n, ctypes.c_int64) for n in ("num_pages", "page_size", "heads", "head_dim", "page_stride", "token_stride",
                                          "head_stride")] + [
            ("page_table", ctypes.c_void_p), ("batch", ctypes.c_int64), ("max_pages", ctypes.c_int64),
            ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p)]

    assert len(_kv()) == ctypes.sizeof(S)
    s = S.from_buffer_copy(_kv(pages=77, table=5, kv_lens=9, max_pages=3))
    assert (s.num_pages, s.page_table, s.kv_lens, s.max_pages) == (77, 5, 9, 3)


def test_rope_refusals(raw):
    def go(x=FAKE, ldx=256, pos=FAKE, f=FAKE, T=4, H=4, D=64, R=32, y=FAKE, ldy=256):
        return raw.bf16_rope(x, ldx, pos, f, T, H, D, R, 0, 1.0, y, ldy, None)

    assert go(T=0) == OK
    assert go(T=-1) == go(H=0) == go(D=0) == INVALID
    assert go(D=60, R=32) == SHAPE and go(R=24) == SHAPE and go(H=1, D=1024, R=528) == SHAPE
    assert go(R=80) == go(R=-16) == INVALID
    assert go(f=None) == go(x=None) == go(y=None) == go(pos=None) == INVALID
    assert go(ldx=248) == go(ldy=255) == INVALID
    assert go(ldx=260) == go(x=FAKE + 8) == go(y=FAKE + 2) == go(pos=FAKE + 2) == go(f=FAKE + 1) == ALIGNMENT


def test_kv_append_refusals(raw):
    def go(k=FAKE, ldk=128, v=FAKE, ldv=128, q=None, ldq=256, qo=None, ldqo=256, Hq=4, T=3, kv=None, f=FAKE, R=64):
        return raw.bf16_kv_append(k, ldk, v, ldv, q, ldq, qo, ldqo, Hq, T, _kv() if kv is None else kv, f, R, 0, 1.0, None)

    assert go(T=0) == OK and go(kv=_kv(batch=0)) == OK
    assert raw.bf16_kv_append(FAKE, 128, FAKE, 128, None, 0, None, 0, 0, 3, None, FAKE, 64, 0, 1.0, None) == INVALID
    assert go(T=-1) == go(k=None) == go(v=None) == go(f=None) == INVALID
    assert go(q=FAKE) == INVALID                       # no q_out
    assert go(q=FAKE, qo=FAKE, Hq=0) == INVALID and go(q=FAKE, qo=FAKE, ldq=248) == INVALID
    assert go(R=48 + 8) == SHAPE and go(R=128) == INVALID
    assert go(kv=_kv(D=60)) == SHAPE
    for bad in (dict(k=0), dict(v=0), dict(table=0), dict(cu_q=0), dict(kv_lens=0), dict(heads=0), dict(page_size=0),
                dict(pages=-1), dict(batch=-1), dict(max_pages=-2), dict(token_stride=-8)):
        assert go(kv=_kv(**bad)) == INVALID, bad
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(table=FAKE + 1), dict(cu_q=FAKE + 2), dict(page_stride=2050),
                dict(token_stride=132), dict(head_stride=65)):
        assert go(kv=_kv(**bad)) == ALIGNMENT, bad
    assert go(kv=_kv(page_stride=1 << 40)) == SHAPE
    assert go(kv=_kv(max_pages=(1 << 26) + 1)) == SHAPE and go(T=(1 << 30) + 1) == SHAPE
    assert go(ldk=132) == go(v=FAKE + 8) == ALIGNMENT


def test_paged_attention_refusals(raw):
    def go(q=FAKE, ldq=256, T=3, Hq=4, kv=None, max_q=0, scale=0.125, window=0, o=FAKE, ldo=256, lse=None, ws=FAKE, nws=1 << 30):
        return raw.bf16_paged_attention(q, ldq, T, Hq, _kv() if kv is None else kv, max_q, scale, window, o, ldo, lse, ws, nws,
                                        None)

    assert go(T=0) == OK and go(kv=_kv(batch=0)) == OK
    assert go(T=-1) == go(Hq=0) == go(window=-1) == go(q=None) == go(o=None) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert go(scale=scale) == INVALID
    assert go(Hq=5) == SHAPE and go(Hq=2 * 129, ldq=1 << 20, ldo=1 << 20) == SHAPE
    for D in (8, 96, 512):
        assert go(kv=_kv(D=D)) == SHAPE
    assert go(kv=_kv(page_size=12)) == SHAPE
    assert go(ldq=248) == go(ldo=248) == INVALID
    assert go(q=FAKE + 8) == go(ldo=260) == go(lse=FAKE + 2) == go(ws=FAKE + 8) == ALIGNMENT
    assert go(kv=_kv(cu_q=0)) == INVALID and go(kv=_kv(k=FAKE + 4)) == ALIGNMENT
    assert go() == INVALID                                         # o is q
    assert go(o=FAKE + (1 << 20), scale=2.0 ** 127) == INVALID     # times log2 e: past fp32


def test_workspace_bytes_of_a_refused_width(raw):
    assert raw.bf16_paged_attention_workspace_bytes(96) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch

    f = pytest.importorskip("fp8_w8a8_linear_b200")
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        f.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(16))
    with pytest.raises(ValueError):
        f.paged_attention(x, x[None], x[None], torch.zeros((1, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                          torch.zeros(1, dtype=torch.int32))


def test_in_place_takes_one_pitch(raw):
    """y = x with another pitch would write rows that other blocks still read."""
    def rope(T, ldx, ldy, y=FAKE):
        return raw.bf16_rope(FAKE, ldx, FAKE, FAKE, T, 4, 64, 32, 0, 1.0, y, ldy, None)

    def append(T, ldq, ldqo, qo=FAKE):
        return raw.bf16_kv_append(FAKE, 128, FAKE, 128, FAKE, ldq, qo, ldqo, 4, T, _kv(), FAKE, 64, 0, 1.0, None)

    assert rope(4, 256, 320) == rope(4, 512, 256) == append(3, 256, 264) == append(2, 512, 256) == INVALID
