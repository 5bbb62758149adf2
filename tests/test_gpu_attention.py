"""GPU parity of the attention block against the float64 oracle, element by
element within tolerances counted from the roundings (oracle/attention.py):
rotary positions, appending to the paged cache, attention over it, and the
chain of them between the W8A8 linears."""

import numpy as np
import pytest
import torch

from oracle import attention as A
from tests.gpu_util import bf16_to_np_bits, bf16_values, f32, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

NAN_BITS = 0x7FC0


def _normal(rng, shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Batch:
    """A ragged batch on a paged cache: bf16 bits on the host, pages at random places, NaN wherever no key is."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, D, page, seed=0, extra_rows=0, extra_pages=3, k_scale=1.0):
        rng = np.random.default_rng([seed, D, page, Hq])
        self.q_lens, self.kv_lens, self.page, self.Hq, self.Hkv, self.D = list(q_lens), list(kv_lens), page, Hq, Hkv, D
        self.cu_q = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int64)
        per = [-(-m // page) for m in kv_lens]
        self.pages = sum(per) + extra_pages
        order = rng.permutation(self.pages)
        self.table = np.full((len(kv_lens), max(max(per), 1) + 1), -7, np.int64)
        self.T = int(self.cu_q[-1]) + extra_rows
        shape = (self.pages, page, Hkv, D)
        self.k, self.v = _normal(rng, shape, k_scale), _normal(rng, shape)
        used = np.zeros((self.pages, page), bool)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
            for j in range(n):
                used[self.table[b, j], :min(page, kv_lens[b] - j * page)] = True
        self.k[~used], self.v[~used] = NAN_BITS, NAN_BITS
        self.q = _normal(rng, (self.T, Hq, D), 1.5)
        self.seq, self.pos = A.positions(self.cu_q, kv_lens)

    def dev(self):
        return dict(k_cache=to_dev(self.k), v_cache=to_dev(self.v), page_table=_ints(self.table), cu_q=_ints(self.cu_q),
                    kv_lens=_ints(self.kv_lens))

    def ref(self, window=0, scale=None):
        return A.paged_attention(A.bf16_f64(self.q), A.bf16_f64(self.k), A.bf16_f64(self.v), self.table, self.cu_q,
                                 self.kv_lens, self.D ** -0.5 if scale is None else scale, window)

    def check(self, out, ref, lse=None):
        n = int(self.cu_q[-1])
        tol, ltol = A.attention_tolerance(ref, self.D)
        err = np.abs(bf16_values(out)[:n] - ref["out"][:n])
        bad = ~(err <= tol[:n])
        assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(err / tol[:n])), np.argwhere(bad)[:4].tolist())
        if lse is not None:
            l, r = f32(lse)[:n].astype(np.float64), ref["lse"][:n]
            assert np.array_equal(np.isneginf(l), np.isneginf(r))
            fin = np.isfinite(r)
            lerr = np.abs(l[fin] - r[fin])
            assert np.all(lerr <= ltol[:n][fin]), float((lerr / ltol[:n][fin]).max())


def _run(lib, B, window=0, scale=None, max_q=None, want_lse=True, ws=None):
    q = to_dev(B.q)
    out = torch.full((B.T, B.Hq, B.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B.T, B.Hq), 7.0, device="cuda") if want_lse else None
    lib.paged_attention(q, **B.dev(), window=window, scale=scale, max_q=max(B.q_lens) if max_q is None else max_q, out=out,
                        lse=lse, ws=ws)
    n = int(B.cu_q[-1])
    assert bool((out[n:] == 7.0).all()) and (lse is None or bool((lse[n:] == 7.0).all()))
    B.check(out, B.ref(window, scale), lse)
    assert lib.device_status() == 0
    return out


# ------------------------------------------------------------------ rope
@pytest.mark.parametrize("T,H,D,R,interleaved,amplitude", [
    (1, 32, 128, 128, False, 1.0), (7, 5, 64, 16, True, 1.0), (33, 3, 256, 64, False, 1.2), (5, 1, 64, 64, True, 0.7),
    (300, 8, 128, 32, True, 1.0), (9, 2, 24, 16, False, 1.0), (4, 3, 512, 512, False, 1.0), (6, 4, 40, 0, False, 1.0)])
def test_rope(lib, T, H, D, R, interleaved, amplitude):
    rng = np.random.default_rng([T, D, R])
    x = _normal(rng, (T, H, D))
    pos = rng.integers(0, 200000, T)
    pos[0], pos[-1] = 0, (1 << 20) - 1
    if T > 5:
        pos[1], pos[2] = -5, (1 << 31) - 1
    f, _ = lib.rope_frequencies(max(R, 16), scaling="wavelength", factor=8.0)
    f = f[: R // 2].contiguous()
    y, size = A.rope(A.bf16_f64(x), pos, f.numpy(), interleaved, amplitude)
    xd = to_dev(x)
    got = lib.rope(xd, _ints(pos), f.cuda(), interleaved, amplitude)
    err = np.abs(bf16_values(got) - y)
    tol = A.rope_tolerance(y, size, amplitude)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.array_equal(bf16_to_np_bits(got)[..., R:], x[..., R:])
    # in place, and through a slice of wider rows
    wide = torch.full((T, H + 3, D), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:H + 1] = xd
    view = wide[:, 1:H + 1]
    assert lib.rope(view, _ints(pos), f.cuda(), interleaved, amplitude, y=view) is view
    assert torch.equal(view, got)
    assert bool((wide[:, 0] == 3.0).all()) and bool((wide[:, H + 1:] == 3.0).all())


@pytest.mark.parametrize("T,H,D,R,interleaved", [(1183, 3, 64, 64, False), (5003, 2, 128, 64, True), (2500, 1, 256, 256, False), (1190, 1, 2056, 512, True), (1, 1, 4096, 0, False)])
def test_rope_of_many_tokens(lib, T, H, D, R, interleaved):
    """Enough tokens for several to a block, the last block short."""
    test_rope(lib, T, H, D, R, interleaved, 1.0)


def test_rope_empty(lib):
    x = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert lib.rope(x, _ints([]), torch.ones(8, device="cuda")).shape == (0, 4, 64)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page,R,interleaved", [
    ([1], [1], 4, 1, 64, 16, 64, False), ([1] * 70, [1 + 37 * i for i in range(70)], 8, 8, 128, 16, 128, False),
    ([3, 0, 17, 1], [3, 5, 400, 33], 6, 2, 256, 8, 64, True), ([129], [500], 3, 3, 40, 7, 32, False),
    ([1] * 600, [9] * 600, 2, 1, 64, 8, 32, True), ([20, 5], [20, 1000], 0, 4, 64, 64, 0, False)])
def test_kv_append(lib, q_lens, kv_lens, Hq, Hkv, D, page, R, interleaved):
    B = Batch(q_lens, kv_lens, max(Hq, 1), Hkv, D, page, extra_rows=2)
    rng = np.random.default_rng(5)
    k, v = _normal(rng, (B.T, Hkv, D)), _normal(rng, (B.T, Hkv, D))
    f = lib.rope_frequencies(R)[0] if R else None
    c = B.dev()
    before_k, before_v = c["k_cache"].clone(), c["v_cache"].clone()
    q_out = torch.full((B.T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    got = lib.kv_append(to_dev(k), to_dev(v), **c, inv_freq=None if f is None else f.cuda(), q=to_dev(B.q) if Hq else None,
                        q_out=q_out, interleaved=interleaved)
    assert got is q_out
    n = int(B.cu_q[-1])
    page_of, at = B.table[B.seq, B.pos // page], B.pos % page
    fn = f.numpy() if R else np.zeros(0, np.float32)
    for x, new in ((k, c["k_cache"][_ints(page_of).long(), _ints(at).long()]),) + (((B.q, q_out[:n]),) if Hq else ()):
        y, size = A.rope(A.bf16_f64(x[:n]), B.pos, fn, interleaved)
        err, tol = np.abs(bf16_values(new) - y), A.rope_tolerance(y, size)
        assert np.all(err <= tol), float((err / tol).max())
    assert np.array_equal(bf16_to_np_bits(c["v_cache"][_ints(page_of).long(), _ints(at).long()]), v[:n])
    # nothing else was touched
    for new, old in ((c["k_cache"], before_k), (c["v_cache"], before_v)):
        new[_ints(page_of).long(), _ints(at).long()] = 0
        old[_ints(page_of).long(), _ints(at).long()] = 0
        assert torch.equal(new.view(torch.int16), old.view(torch.int16))
    if Hq:
        assert bool((q_out[n:] == 7.0).all())
    assert lib.device_status() == 0


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page,R,interleaved", [
    ([2011, 0, 700, 1, 2402], [2011, 9, 3001, 50, 2500], 6, 2, 64, 16, 64, False), ([1801], [1801], 2, 2, 128, 24, 64, True),
    ([1] * 1300, [5] * 1300, 2, 1, 64, 8, 32, False), ([0, 3, 0, 0, 1, 2] * 217, [0, 3, 4, 0, 9, 30] * 217, 1, 1, 64, 8, 64, True)])
def test_kv_append_of_many_tokens(lib, q_lens, kv_lens, Hq, Hkv, D, page, R, interleaved):
    """Enough tokens for several to a block, sequences starting inside a block's tokens."""
    test_kv_append(lib, q_lens, kv_lens, Hq, Hkv, D, page, R, interleaved)


def test_kv_append_flags_places_that_are_not_there(lib):
    B = Batch([2, 3, 1], [2, 2, 9], 2, 2, 64, 8)
    B.table[2, 1] = B.pages      # the page of the third sequence's token; the second has a token at position -1
    c = B.dev()
    k = to_dev(_normal(np.random.default_rng(1), (6, 2, 64)))
    lib.kv_append(k, k, **c)
    assert lib.device_status() & lib.DEV_BAD_INDEX
    assert torch.equal(c["k_cache"][int(B.table[0, 0]), :2], k[:2])
    assert torch.equal(c["k_cache"][int(B.table[1, 0]), :2], k[3:5])
    for cu, lens in (([0, 2, 1, 6], [2, 2, 9]), ([0, 2, 5, 6], [2, 2, 1 << 20])):
        c["cu_q"], c["kv_lens"] = _ints(cu), _ints(lens)
        lib.kv_append(k, k, **c)
        assert lib.device_status() & lib.DEV_BAD_INDEX


# ------------------------------------------------------------------ attention
EDGES = [0, 1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(8, 2, 16), (4, 4, 8), (16, 1, 64), (6, 2, 24), (5, 1, 256)])
def test_single_tokens(lib, D, Hq, Hkv, page):
    _run(lib, Batch([1] * len(EDGES), EDGES, Hq, Hkv, D, page, extra_rows=1))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page,q_lens", [
    (8, 2, 16, [1, 2, 3, 0, 4, 4, 4]), (4, 4, 8, [16, 16, 1, 9, 13, 0, 16]), (3, 1, 48, [5, 5, 5, 1, 2, 5, 5])])
def test_a_few_tokens(lib, D, Hq, Hkv, page, q_lens):
    _run(lib, Batch(q_lens, [1, 2, 300, 7, 65, 4, 130], Hq, Hkv, D, page))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page,q_lens,kv_lens", [
    (8, 2, 16, [333], [333]), (4, 4, 8, [130, 1, 0, 257], [130, 500, 3, 900]), (16, 1, 64, [65, 20], [1000, 20]),
    (6, 2, 24, [128, 129, 127], [128, 400, 127]), (10, 2, 128, [200, 30], [150, 30]), (7, 1, 32, [77, 1], [78, 200]),
    (40, 1, 16, [9, 1, 4], [300, 40, 4]), (128, 1, 16, [3, 1], [140, 129])])
def test_chunks(lib, D, Hq, Hkv, page, q_lens, kv_lens):
    _run(lib, Batch(q_lens, kv_lens, Hq, Hkv, D, page, extra_rows=3))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 7, 64, 127, 128, 129, 300, 1 << 40])
@pytest.mark.parametrize("q_lens", [[1, 1, 1, 1], [140, 1, 0, 33]])
def test_windows(lib, D, window, q_lens):
    _run(lib, Batch(q_lens, [600, 129, 5, 128], 4, 2, D, 16), window=window)


@pytest.mark.parametrize("max_q", [0, 3, 1000])
def test_max_q_as_a_bound(lib, max_q):
    _run(lib, Batch([1, 3, 2], [300, 70, 2], 4, 2, 128, 16), max_q=max_q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv", [(1, 20000), (3, 9001), (40, 12345), (300, 6000)])
def test_long_axis_is_split_and_joined(lib, D, q_len, kv):
    """Few rows over many keys: the keys are shared out over the device."""
    _run(lib, Batch([q_len], [kv], 4, 1, D, 32))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("batch,window", [(33, 0), (97, 50), (450, 0)])
def test_many_sequences(lib, D, batch, window):
    """More sequences than the lanes that look for a run, some without new tokens, some without keys."""
    rng = np.random.default_rng([batch, D])
    kv = rng.integers(0, 200, batch)
    _run(lib, Batch([1] * batch, kv.tolist(), 4, 2, D, 16), window=window)
    q = rng.integers(0, 30, batch)
    _run(lib, Batch(q.tolist(), (q + kv).tolist(), 4, 2, D, 16), window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,window", [(12, 4, 0), (4, 4, 0), (16, 2, 700), (5, 1, 129)])
def test_long_runs_over_items_of_every_kind(lib, D, Hq, Hkv, window):
    """Runs of many key tiles that pass from items of one row tile to items of two and back, with cuts in both."""
    q_lens, kv_lens = [300, 20, 1, 70, 513, 129], [5000, 3001, 4100, 900, 2600, 5121]
    _run(lib, Batch(q_lens, kv_lens, Hq, Hkv, D, 32, extra_rows=1), window=window)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [3000, 40, 700]), ([200, 9, 70], [1500, 2000, 70])])
def test_two_calls_at_once(lib, q_lens, kv_lens):
    """Two streams, a workspace each; the calls overlap."""
    batches = [Batch(q_lens, kv_lens, 8, 2, 128, 16, seed=i) for i in range(2)]
    args = [(to_dev(B.q), B.dev(), lib.paged_attention_workspace(128)) for B in batches]
    alone = [lib.paged_attention(q, **c, max_q=max(q_lens), ws=ws) for q, c, ws in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    outs = [[], []]
    for _ in range(20):
        for i, (q, c, ws) in enumerate(args):
            with torch.cuda.stream(streams[i]):
                outs[i].append(lib.paged_attention(q, **c, max_q=max(q_lens), ws=ws))
    torch.cuda.synchronize()
    for i, B in enumerate(batches):
        B.check(alone[i], B.ref())
        assert all(torch.equal(alone[i], o) for o in outs[i])
    assert lib.device_status() == 0


def test_peaked_scores_and_scales(lib):
    """Scores to some hundreds: the running maximum moves far and often, forwards and not at all."""
    for seed, ks, scale in ((1, 8.0, None), (2, 1.0, 3.0), (3, 1e-3, 1e-4)):
        for q_lens in ([1, 1], [150, 2]):
            B = Batch(q_lens, [700, 333], 4, 2, 128, 16, seed=seed, k_scale=ks)
            _run(lib, B, scale=scale)
            B.k[:] = np.sort(B.k.view(np.int16), axis=1).view(np.uint16)  # maxima rise (or fall) along a page
            B.k[B.k == NAN_BITS] = 0
            _run(lib, B, scale=scale)


@pytest.mark.parametrize("q_lens", [[1, 2, 1], [100, 60, 3]])
def test_layouts_and_slices(lib, q_lens):
    """Heads before tokens, the halves of one array, queries in a fused q/k/v row, out in wider rows."""
    B = Batch(q_lens, [200, 61, 90], 8, 2, 128, 16)
    c, ref = B.dev(), B.ref()
    plain = lib.paged_attention(to_dev(B.q), **c, max_q=max(q_lens))
    B.check(plain, ref)
    hnd = {n: c[n].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for n in ("k_cache", "v_cache")}
    assert torch.equal(plain, lib.paged_attention(to_dev(B.q), **{**c, **hnd}, max_q=max(q_lens)))
    both = torch.stack([c["k_cache"], c["v_cache"]], 1)
    half = {"k_cache": both[:, 0], "v_cache": both[:, 1]}
    assert torch.equal(plain, lib.paged_attention(to_dev(B.q), **{**c, **half}, max_q=max(q_lens)))
    fused = torch.zeros((B.T, 12, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, :8] = to_dev(B.q)
    wide = torch.full((B.T, 11, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    lib.paged_attention(fused[:, :8], **c, max_q=max(q_lens), out=wide[:, 2:10])
    assert torch.equal(wide[:, 2:10], plain) and bool((wide[:, :2] == 2).all()) and bool((wide[:, 10:] == 2).all())


def test_nan_where_no_token_looks(lib):
    """Before the window of every new token (pages a server may have given away), table entries there too."""
    for q_lens, window in (([1, 1], 100), ([70, 1], 64)):
        B = Batch(q_lens, [900, 400], 4, 2, 64, 16)
        for b, n in enumerate(q_lens):
            first = B.kv_lens[b] - n - window + 1
            for j in range(first):
                B.k[B.table[b, j // 16], j % 16] = NAN_BITS
                B.v[B.table[b, j // 16], j % 16] = NAN_BITS
        _run(lib, B, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,window", [(8, 0), (8, 90), (24, 100), (40, 1), (16, 130)])
def test_small_pages_with_nan_around_the_keys(lib, D, page, window):
    """Chunks whose first and last tiles hold values that must not count, pages in pieces of 8 rows and of 16."""
    q_lens = [130, 1, 70]
    B = Batch(q_lens, [900, 411, 70], 6, 2, D, page)
    for b, n in enumerate(q_lens):
        first = B.kv_lens[b] - n - window + 1 if window else 0
        for j in range(first):
            B.k[B.table[b, j // page], j % page] = NAN_BITS
            B.v[B.table[b, j // page], j % page] = NAN_BITS
    _run(lib, B, window=window)


def test_offsets_past_32_bits(lib):
    """A cache of 2^31 elements and more, the pages in use at its end."""
    page, Hkv, D = 64, 8, 256
    pages = (1 << 31) // (page * Hkv * D) + 40
    big = [torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for q_lens in ([1, 1], [90, 2]):
        B = Batch(q_lens, [500, 200], 16, Hkv, D, page)
        c = B.dev()
        at = pages - B.pages
        for n, t in zip(("k_cache", "v_cache"), big):
            t[at:] = c[n]
            c[n] = t
        c["page_table"] = torch.where(c["page_table"] >= 0, c["page_table"] + at, c["page_table"])
        out = lib.paged_attention(to_dev(B.q), **c, max_q=max(q_lens))
        B.check(out, B.ref())
        k = _normal(np.random.default_rng(8), (B.T, Hkv, D))
        lib.kv_append(to_dev(k), to_dev(k), **c)
        rows = B.table[B.seq, B.pos // page] + at, B.pos % page
        assert np.array_equal(bf16_to_np_bits(c["k_cache"][_ints(rows[0]).long(), _ints(rows[1]).long()]), k)
    assert lib.device_status() == 0


def test_bad_batches_are_flagged_and_the_others_right(lib):
    for q_lens in ([1, 1, 1], [80, 5, 90]):
        B = Batch(q_lens, [150, 60, 170], 4, 2, 128, 16)
        ref = B.ref()
        rows = {b: slice(int(B.cu_q[b]), int(B.cu_q[b + 1])) for b in range(3)}
        tol, _ = A.attention_tolerance(ref, 128)

        def good(c, which, **kw):
            out = torch.full((B.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            lib.paged_attention(to_dev(B.q), **c, out=out, **{"max_q": max(q_lens), **kw})
            assert lib.device_status() & lib.DEV_BAD_INDEX
            got = bf16_values(out)
            for b in which:
                assert np.all(np.abs(got[rows[b]] - ref["out"][rows[b]]) <= tol[rows[b]])
            return out

        c = B.dev()
        c["page_table"][1, 1] = B.pages + 5
        good(c, (0, 2))
        c = B.dev()
        c["kv_lens"][1] = B.table.shape[1] * 16 + 1
        out = good(c, (0, 2))
        assert bool((out[rows[1]] == 7.0).all())
        c["kv_lens"][1] = -1
        out = good(c, (0, 2))
        assert bool((out[rows[1]] == 7.0).all())
        if q_lens[0] > 1:
            out = good(B.dev(), (1,), max_q=6)      # the first and the third have more
            assert bool((out[rows[0]] == 7.0).all()) and bool((out[rows[2]] == 7.0).all())
        c = B.dev()
        c["cu_q"][3] = B.T + 50
        good(c, (0, 1))


def test_same_bits_again_and_on_another_stream(lib):
    ws = lib.paged_attention_workspace(128)
    for q_lens, kv in (([1, 1, 1], [5000, 20, 700]), ([300, 2], [2000, 90])):
        B = Batch(q_lens, kv, 8, 2, 128, 16)
        c, q = B.dev(), to_dev(B.q)
        a = lib.paged_attention(q, **c, max_q=max(q_lens), ws=ws)
        ws.fill_(255)     # NaN patterns: the workspace's contents mean nothing
        assert torch.equal(a, lib.paged_attention(q, **c, max_q=max(q_lens), ws=ws))
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            b = lib.paged_attention(q, **c, max_q=max(q_lens), ws=lib.paged_attention_workspace(128))
        s.synchronize()
        assert torch.equal(a, b)
        B.check(a, B.ref())


def test_captured_graphs_sharing_a_workspace_follow_their_inputs(lib):
    ws = lib.paged_attention_workspace(64)
    state = []
    for q_lens, kv in (([1, 1], [900, 333]), ([150, 3], [400, 64])):
        B = Batch(q_lens, kv, 4, 2, 64, 16)
        c, q = B.dev(), to_dev(B.q)
        f = lib.rope_frequencies(64)[0].cuda()
        k, v = to_dev(_normal(np.random.default_rng(2), (B.T, 2, 64))), to_dev(_normal(np.random.default_rng(3), (B.T, 2, 64)))
        out, qo = torch.empty_like(q), torch.empty_like(q)

        def step(B=B, c=c, q=q, k=k, v=v, out=out, qo=qo, f=f, n=max(q_lens)):
            lib.kv_append(k, v, **c, inv_freq=f, q=q, q_out=qo)
            lib.paged_attention(qo, **c, max_q=n, ws=ws, out=out)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        state.append((g, step, out, q, c))
    for shrink in (0, 17):
        for g, step, out, q, c in state:
            q.normal_()
            c["kv_lens"] -= shrink
        for g, *_ in state + state:
            g.replay()
        got = [s[2].clone() for s in state]
        for (g, step, out, q, c), a in zip(state, got):
            out.zero_()
            step()
            assert torch.equal(a, out)
    assert lib.device_status() == 0


def test_chunk_by_chunk_is_token_by_token(lib):
    """A prompt appended and attended as one chunk, and then again token by token: the same cache bit for bit, and outputs
    within both roundings of each other."""
    T, Hq, Hkv, D, page = 150, 8, 2, 128, 16
    rng = np.random.default_rng(12)
    q, k, v = (to_dev(_normal(rng, (T, h, D))) for h in (Hq, Hkv, Hkv))
    f = lib.rope_frequencies(D)[0].cuda()
    table = _ints(rng.permutation(10)[None])
    outs, caches = [], []
    for step in (T, 1):
        kc, vc = (torch.zeros((10, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out = []
        for t in range(0, T, step):
            batch = (kc, vc, table, _ints([0, step]), _ints([t + step]))
            qr = lib.kv_append(k[t:t + step], v[t:t + step], *batch, inv_freq=f, q=q[t:t + step])
            out.append(lib.paged_attention(qr, *batch, max_q=step))
        outs.append(bf16_values(torch.cat(out)))
        caches.append((kc, vc))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    # each within u (1 + sum p|v| / |o|) of the exact one, u = 2^-8; |v| < 5 here
    assert np.abs(outs[0] - outs[1]).max() <= 2 * 2.0 ** -8 * (np.abs(outs[0]).max() + 5)
    assert lib.device_status() == 0


def test_attention_block_between_w8a8_linears(lib):
    """x -> q, k, v (linear_siblings) -> kv_append -> paged_attention -> o (linear), each step against the oracle on the
    step before's bits."""
    import oracle
    from workloads import activations_bf16, q4_weights

    T, hidden, Hq, Hkv, D, page = 37, 512, 4, 2, 128, 16
    x = activations_bf16(T, hidden, seed=3, outlier_frac=0.01)
    ws = [oracle.repack_qat(*q4_weights(n, kk, seed=9 + i)) for i, (n, kk) in
          enumerate([(Hq * D, hidden), (Hkv * D, hidden), (Hkv * D, hidden), (hidden, Hq * D)])]
    dw = [(to_dev(w.codes), to_dev(w.scales)) for w in ws]
    q, k, v = (y.view(T, -1, D) for y in lib.linear_siblings(to_dev(x), dw[:3]))
    f = lib.rope_frequencies(D)[0]
    B = Batch([30, 7], [30, 95], Hq, Hkv, D, page)
    c = B.dev()
    qr = lib.kv_append(k, v, **c, inv_freq=f.cuda(), q=q)
    y, size = A.rope(bf16_values(q), B.pos, f.numpy())
    assert np.all(np.abs(bf16_values(qr) - y) <= A.rope_tolerance(y, size))
    o = lib.paged_attention(qr, **c, max_q=30)
    B.q, B.k, B.v = bf16_to_np_bits(qr), bf16_to_np_bits(c["k_cache"]), bf16_to_np_bits(c["v_cache"])
    B.check(o, B.ref())
    out = lib.linear(o.view(T, Hq * D), *dw[3])
    a = oracle.quant_act(bf16_to_np_bits(o).reshape(T, Hq * D))
    ref, absum = oracle.rowwise_linear_ref(a.codes, a.scales, ws[3].codes, ws[3].scales, return_abs=True)
    ok, worst = oracle.check_linear(bf16_values(out), ref, absum)
    assert ok, worst
    assert lib.device_status() == 0


def test_binding_refusals(lib):
    B = Batch([1, 1], [20, 5], 4, 2, 64, 16)
    c, q = B.dev(), to_dev(B.q)
    for bad in (dict(cu_q=c["cu_q"][:2]), dict(kv_lens=c["kv_lens"].long()), dict(page_table=c["page_table"][0]),
                dict(v_cache=c["v_cache"].transpose(1, 2)), dict(k_cache=c["k_cache"][..., :32]),
                dict(ws=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(window=-1), dict(scale=0.0),
                dict(lse=torch.empty((2, 3), device="cuda")), dict(out=torch.empty_like(q).half())):
        with pytest.raises((ValueError, TypeError, lib.Fp8Error)):
            lib.paged_attention(q, **{**c, **bad})
    with pytest.raises(ValueError):
        lib.paged_attention(q.transpose(1, 2).contiguous().transpose(1, 2), **c)
    with pytest.raises(ValueError):
        lib.kv_append(q, q, **c)          # four heads, the cache has two
    with pytest.raises(ValueError):
        lib.kv_append(q[:, :2], q[:, :2], **c, q_out=q)
    assert lib.device_status() == 0


# Whole items and cut ones of both kernels: (q_lens, kv_lens, Hq, Hkv). Many short sequences fill every run with whole items,
# one long context is cut over the device.
KINDS = [([1] * 40, [60] * 40, 16, 4), ([1], [20000], 4, 1), ([9] * 40, [60] * 40, 16, 4), ([40], [12345], 4, 1), ([300], [6000], 4, 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["query", "key", "value"])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", KINDS)
def test_a_nan_that_a_token_sees_reaches_its_output(lib, D, what, q_lens, kv_lens, Hq, Hkv):
    """A query row, a key or one element of a value is NaN: it reaches the rows that see it, however the work was cut and
    however little the part with the key weighs in the sum; what does not see it stays as it is (a NaN value may reach its
    column of the sequence's other rows)."""
    last = len(q_lens) - 1
    for scale in (None, 8.0):      # 8: parts' maxima lie hundreds apart
        B = Batch(q_lens, kv_lens, Hq, Hkv, D, 16)
        ref = B.ref(scale=scale)
        j = kv_lens[last] // 3 if q_lens[last] == 1 else kv_lens[last] - q_lens[last] // 2
        page = B.table[last, j // 16], j % 16, 0
        nan, free = np.zeros((2, B.T, Hq, D), bool)
        if what == "query":
            t, h = int(B.cu_q[last + 1]) - 1, Hq // 2
            B.q[t, h, 3] = NAN_BITS
            nan[t, h] = True
        else:
            sees = np.zeros((B.T, Hq, 1), bool)
            sees[:, : Hq // Hkv, 0] = ((B.seq == last) & (B.pos >= j))[:, None]
            if what == "key":
                B.k[page][D - 1] = NAN_BITS
                nan |= sees
            else:
                B.v[page][D - 1] = NAN_BITS
                nan[..., D - 1:] = sees
                free[B.seq == last, : Hq // Hkv, D - 1] = True
        assert nan.any()
        out = lib.paged_attention(to_dev(B.q), **B.dev(), scale=scale, max_q=max(q_lens))
        got = bf16_values(out)
        assert np.isnan(got[nan]).all(), (scale, int((~np.isnan(got[nan])).sum()))
        tol, _ = A.attention_tolerance(ref, D)
        rest = ~(nan | free)
        assert np.all(np.abs(got - ref["out"])[rest] <= tol[rest]), scale
        assert lib.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", KINDS)
def test_lse_of_rows_with_nan_is_not_that_of_rows_without_keys(lib, D, q_lens, kv_lens, Hq, Hkv):
    """lse is NaN for a NaN query row and for a row whose scores pass fp32 (whose o is NaN too); -inf stays for rows that see no key."""
    B = Batch(q_lens + [3], kv_lens + [2], Hq, Hkv, D, 16)     # the first of the three sees nothing
    t = int(B.cu_q[-2]) - 1
    B.q[t, 1, 5] = NAN_BITS
    big = t, 2
    j = B.kv_lens[-2] // 2 if q_lens[-1] == 1 else B.kv_lens[-2] - q_lens[-1] // 2
    B.q[big] = f32_to_bf16_bits(np.full(D, 2.0 ** 70, np.float32))
    ref = B.ref()
    for h in range(Hkv):
        B.k[B.table[len(q_lens) - 1, j // 16], j % 16, h] = f32_to_bf16_bits(np.full(D, 2.0 ** 70, np.float32))
    hit = (B.seq == len(q_lens) - 1) & (B.pos >= j)
    lse = torch.full((B.T, Hq), 7.0, device="cuda")
    out = lib.paged_attention(to_dev(B.q), **B.dev(), max_q=max(B.q_lens), lse=lse)
    got, l = bf16_values(out), f32(lse)
    for row in ((t, 1), big):
        assert np.isnan(got[row]).all() and np.isnan(l[row]), row
    assert np.all(np.isneginf(l[B.T - 3])) and np.all(got[B.T - 3] == 0)
    _, tol = A.attention_tolerance(ref, D)
    rest = ~hit
    rest[B.T - 3] = False
    assert np.all(np.abs(l[rest] - ref["lse"][rest]) <= tol[rest])
    assert lib.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", KINDS)
def test_scores_that_only_their_scale_takes_past_fp32(lib, D, q_lens, kv_lens, Hq, Hkv):
    """q . k is finite (2^120 D, D = 64 and 128) and scale times it is not: NaN in o and lse, as where q . k is not."""
    B = Batch(q_lens, kv_lens, Hq, Hkv, D, 16)
    t, b = B.T - 1, len(q_lens) - 1
    j = kv_lens[b] // 2 if q_lens[b] == 1 else kv_lens[b] - q_lens[b] // 2
    B.q[t, 1] = f32_to_bf16_bits(np.full(D, 2.0 ** 60, np.float32))
    B.k[B.table[b, j // 16], j % 16, 0] = f32_to_bf16_bits(np.full(D, 2.0 ** 60, np.float32))
    lse = torch.full((B.T, Hq), 7.0, device="cuda")
    out = lib.paged_attention(to_dev(B.q), **B.dev(), scale=32.0, max_q=max(q_lens), lse=lse)
    assert np.isnan(bf16_values(out)[t, 1]).all() and np.isnan(f32(lse)[t, 1])
    assert lib.device_status() == 0


def test_part_of_a_batch_by_its_offsets(lib):
    """cu_q, kv_lens and the table sliced to some sequences of a batch, the rows as they are: the rows in front of the first
    offset belong to no sequence, like those behind the last."""
    for q_lens in ([2, 1, 3, 1], [40, 700, 3, 90], [1] * 900):
        kv_lens = [n + 9 for n in q_lens]
        B = Batch(q_lens, kv_lens, 4, 2, 64, 16)
        c, q = B.dev(), to_dev(B.q)
        k = to_dev(_normal(np.random.default_rng(1), (B.T, 2, 64)))
        b0, b1 = 1, len(q_lens) - 1
        r0, r1 = int(B.cu_q[b0]), int(B.cu_q[b1])
        want = {n: c[n].clone() for n in ("k_cache", "v_cache")}
        at = _ints(B.table[B.seq, B.pos // 16]).long()[r0:r1], _ints(B.pos % 16).long()[r0:r1]
        want["k_cache"][at] = want["v_cache"][at] = k[r0:r1]
        part = {**c, "cu_q": c["cu_q"][b0:b1 + 1].contiguous(), "kv_lens": c["kv_lens"][b0:b1].contiguous(),
                "page_table": c["page_table"][b0:b1].contiguous()}
        qo, o = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
        assert lib.kv_append(k, k, **part, q=q, q_out=qo) is qo
        assert lib.device_status() == 0
        for n, w in want.items():
            assert torch.equal(c[n].view(torch.int16), w.view(torch.int16))
        lib.paged_attention(qo, **part, max_q=max(q_lens), out=o)
        assert lib.device_status() == 0
        for y in (qo, o):
            assert bool((y[:r0] == 7.0).all()) and bool((y[r1:] == 7.0).all())
        assert torch.equal(qo[r0:r1], q[r0:r1])
        B.k, B.v = bf16_to_np_bits(c["k_cache"]), bf16_to_np_bits(c["v_cache"])
        ref = B.ref()
        assert np.all(np.abs(bf16_values(o) - ref["out"])[r0:r1] <= A.attention_tolerance(ref, 64)[0][r0:r1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 24, 64])
@pytest.mark.parametrize("q_lens,window", [([1, 1, 1], 100), ([1, 1, 2], 1), ([70, 1, 9], 64), ([40, 200, 3], 500)])
def test_table_entries_before_the_window_are_not_looked_at(lib, D, page, q_lens, window):
    """A server has given the pages away that lie wholly before the first key that any new token sees: their entries are
    negative or past the end, and no flag is set."""
    B = Batch(q_lens, [900, 1400, 33], 4, 2, D, page)
    ref, gone = B.ref(window), 0
    for b, n in enumerate(q_lens):
        first = max(0, B.kv_lens[b] - n - window + 1) // page
        B.table[b, :first] = [-7 if i % 2 else B.pages + 5 for i in range(first)]
        gone += first
    assert gone > 0
    out = lib.paged_attention(to_dev(B.q), **B.dev(), window=window, max_q=max(q_lens))
    B.check(out, ref)
    assert lib.device_status() == 0


def test_offsets_past_2_to_the_32_elements(lib):
    """k and v are the halves of one array of more than 2^32 elements, the pages in use at its end."""
    page, Hkv, D = 64, 8, 256
    pages = (1 << 32) // (2 * page * Hkv * D) + 40
    big = torch.empty((pages, 2, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    for q_lens in ([1, 1], [90, 2]):
        B = Batch(q_lens, [500, 200], 16, Hkv, D, page)
        c, at = B.dev(), pages - B.pages
        assert at * big.stride(0) >= 1 << 32
        for i, n in enumerate(("k_cache", "v_cache")):
            big[at:, i] = c[n]
            c[n] = big[:, i]
        c["page_table"] = torch.where(c["page_table"] >= 0, c["page_table"] + at, c["page_table"])
        B.check(lib.paged_attention(to_dev(B.q), **c, max_q=max(q_lens)), B.ref())
        k = _normal(np.random.default_rng(8), (B.T, Hkv, D))
        lib.kv_append(to_dev(k), to_dev(k), **c)
        rows = _ints(B.table[B.seq, B.pos // page] + at).long(), _ints(B.pos % page).long()
        for n in ("k_cache", "v_cache"):
            assert np.array_equal(bf16_to_np_bits(c[n][rows]), k)
    assert lib.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_and_single_tokens_are_both_within_the_tolerance(lib, D):
    """A prompt appended and attended whole, in uneven chunks, and token by token: the same cache bit for bit, every row of
    every way within its own tolerance of the float64 form."""
    T, Hq, Hkv, page = 150, 8, 2, 16
    rng = np.random.default_rng(12)
    q, k, v = (to_dev(_normal(rng, (T, h, D))) for h in (Hq, Hkv, Hkv))
    f = lib.rope_frequencies(D)[0].cuda()
    table = rng.permutation(10)[None]
    caches = []
    for steps in ([T], [1] * T, [70, 3, 1, 60, 16]):
        kc, vc = (torch.zeros((10, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out, qrs, t = [], [], 0
        for n in steps:
            batch = (kc, vc, _ints(table), _ints([0, n]), _ints([t + n]))
            qrs.append(lib.kv_append(k[t:t + n], v[t:t + n], *batch, inv_freq=f, q=q[t:t + n]))
            out.append(lib.paged_attention(qrs[-1], *batch, max_q=n))
            t += n
        ref = A.paged_attention(bf16_values(torch.cat(qrs)), bf16_values(kc), bf16_values(vc), table, [0, T], [T], D ** -0.5)
        tol, _ = A.attention_tolerance(ref, D)
        err = np.abs(bf16_values(torch.cat(out)) - ref["out"])
        assert np.all(err <= tol), (len(steps), float((err / tol).max()))
        caches.append((torch.cat(qrs), kc, vc))
    for other in caches[1:]:
        assert all(torch.equal(a, b) for a, b in zip(caches[0], other))
    assert lib.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 2, 1], [100, 60, 3]])
def test_one_head_of_keys_expanded_to_several(lib, D, q_lens):
    """The cache's heads are one head, repeated by a stride of 0."""
    B = Batch(q_lens, [200, 61, 90], 8, 1, D, 16)
    c, q = B.dev(), to_dev(B.q)
    wide = {**c, **{n: c[n].expand(-1, -1, 4, -1) for n in ("k_cache", "v_cache")}}
    assert wide["k_cache"].stride(2) == 0
    B.check(lib.paged_attention(q, **wide, max_q=max(q_lens)), B.ref())
    assert lib.device_status() == 0


@pytest.mark.parametrize("q_lens", [[1, 2], [40, 30]])
def test_a_cache_without_pages(lib, q_lens):
    """No page and no key anywhere: every token sees nothing."""
    for D in (64, 128, 256):
        kc = torch.empty((0, 16, 2, D), dtype=torch.bfloat16, device="cuda")
        T = sum(q_lens)
        q, lse = torch.ones((T, 4, D), dtype=torch.bfloat16, device="cuda"), torch.ones((T, 4), device="cuda")
        table = torch.empty((2, 0), dtype=torch.int32, device="cuda")
        out = lib.paged_attention(q, kc, kc.clone(), table, _ints([0, q_lens[0], T]), _ints([0, 0]), max_q=max(q_lens), lse=lse)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        assert lib.device_status() == 0


@pytest.mark.parametrize("T", [5, 3000])
def test_append_from_fused_rows_in_place(lib, T):
    """q, k and v are slices of one row; the queries are turned in place."""
    Hq, Hkv, D, page = 6, 2, 64, 16
    rng = np.random.default_rng(T)
    x = _normal(rng, (T, Hq + 2 * Hkv + 1, D))
    f = lib.rope_frequencies(D)[0]
    n = -(-T // page)
    kc, vc = (torch.zeros((n, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = to_dev(x)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:Hq + 2 * Hkv]
    assert lib.kv_append(k, v, kc, vc, _ints(np.arange(n)[None]), _ints([0, T]), _ints([T]), inv_freq=f.cuda(), q=q, q_out=q) is q
    for got, a, b in ((q, 0, Hq), (kc.view(-1, Hkv, D)[:T], Hq, Hq + Hkv)):
        y, size = A.rope(A.bf16_f64(x[:, a:b]), np.arange(T), f.numpy())
        assert np.all(np.abs(bf16_values(got) - y) <= A.rope_tolerance(y, size))
    assert np.array_equal(bf16_to_np_bits(vc.view(-1, Hkv, D)[:T]), x[:, Hq + Hkv:Hq + 2 * Hkv])
    assert np.array_equal(bf16_to_np_bits(rows)[:, Hq:], x[:, Hq:])
    assert lib.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_thousands_of_sequences(lib, D):
    rng = np.random.default_rng(D)
    kv = rng.integers(0, 60, 4500)
    _run(lib, Batch([1] * 4500, kv.tolist(), 4, 2, D, 8))
    q = rng.integers(0, 4, 4500)
    _run(lib, Batch(q.tolist(), (q + kv).tolist(), 8, 1, D, 8), window=40)
