"""Sequences that outgrow their block table: a token whose position is past the table has no
place. It is not written (and nothing else is, in its stead), reads as zeros, and as a query
gets O = 0 and LSE = -inf; the tokens before it keep their positions. As for positions
below 0."""
import numpy as np
import pytest

from helpers import compare
from oracle import serving as S
from serving_cases import Batch, bits, dev, to_f64

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
GUARD = 4096


@pytest.fixture(scope="module")
def fa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_tiled_attention_forward_gb300 as fa
    from exact_tiled_attention_forward_gb300 import build
    build.build()
    fa.lib()
    return fa


def batch(new, room, lens, h_kv, d, seed, dtype="bf16", pad=0):
    """Sequences whose tables hold `room` positions at most and whose lengths are `lens`."""
    b = Batch(new, [min(int(x), room) for x in lens], h_kv, d, seed=seed, dtype=dtype, pad=pad, extra_pages=0)
    assert b.max_pages * 128 == room
    b.lens = np.array(lens, np.int32)
    return b


def places(b):
    """(row, page, slot) of the new tokens that have a place."""
    return [(t, int(b.table[s, p // 128]), p % 128) for t, s, p in S.new_positions(b.cu, b.lens)
            if 0 <= p < b.max_pages * 128]


# (new, room, lens)
WRITES = [
    ([1], 128, [129]),                                   # a decode step one past the last page
    ([5], 128, [130]),                                   # three tokens fit
    ([1, 1, 1], 256, [256, 257, 3]),
    ([40, 300, 7], 384, [400, 500, TOP]),
    ([3, 2], 128, [TOP, 128 + 5]),
    ([6], 128, [4]),                                     # and two that stand below 0
]


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: f"{c[0]}of{c[2]}")
def test_append_drops_tokens_past_the_table(fa, case, fp8):
    import torch
    new, room, lens = case
    b = batch(new, room, lens, 2, 64, 71, pad=2)
    k, v = b.draw(b.T, 2, 64), b.draw(b.T, 2, 64)
    fill = lambda shape: b.rng.integers(0, 100, size=shape).astype(np.uint8 if fp8 else np.uint16)  # noqa: E731
    cache, exps = [fill(b.cache_shape()) for _ in range(2)], [fill(b.cache_shape()[:3]).astype(np.uint8) for _ in range(2)]
    got, gexp = [dev(x) for x in cache], [dev(x) for x in exps] if fp8 else [None, None]
    fa.fa_cache_append(dev(k), dev(v), *got, dev(b.table), dev(b.cu), dev(b.lens), k_exp=gexp[0], v_exp=gexp[1])
    torch.cuda.synchronize()
    for x, c, e in ((k, cache[0], exps[0]), (v, cache[1], exps[1])):
        rows, byte = S.quantise_rows(to_f64(x)) if fp8 else (x, None)
        for t, page, slot in places(b):
            c[page, :, slot] = rows[t]
            if fp8:
                e[page, :, slot] = byte[t]
    for g, c in zip(got, cache):
        assert np.array_equal(g.view(torch.uint8 if fp8 else torch.int16).cpu().numpy().view(c.dtype), c)
    if fp8:
        for g, e in zip(gexp, exps):
            assert np.array_equal(g.cpu().numpy(), e)


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: f"{c[0]}of{c[2]}")
def test_read_gives_zeros_past_the_table(fa, case, fp8):
    import torch
    new, room, lens = case
    b = batch(new, room, lens, 2, 64, 72, pad=2)
    x = to_f64(b.draw(*b.cache_shape()))
    codes, byte = S.quantise_rows(x)
    val = S.row_values(codes, byte) if fp8 else x
    c = dev(codes) if fp8 else dev(bits(x, "bf16"))
    out = torch.full((2, b.T, 2, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_cache_read(c, c, dev(b.table), dev(b.cu), dev(b.lens), b.T, k=out[0], v=out[1],
                     k_exp=dev(byte) if fp8 else None, v_exp=dev(byte) if fp8 else None)
    want = np.zeros((b.T, 2, 64))
    want[int(b.cu[-1]):] = -7.0
    for t, page, slot in places(b):
        want[t] = val[page, :, slot]
    for g in out:
        assert np.array_equal(g.double().cpu().numpy(), want)


# (new, room, lens, H_q, H_kv, d, window, sinks)
READS = [
    ([1, 1, 1], 256, [257, 256, 40], 8, 2, 128, 0, 0),
    ([4, 3, 2], 128, [130, 128, TOP], 4, 1, 64, 0, 0),          # rows of one unit on both sides of the end
    ([2, 2], 384, [385, 700], 8, 2, 128, 50, 3),
    ([1, 1], 256, [100000, 255], 8, 2, 64, 90, 0),              # a window that begins past the table
    ([40, 30], 256, [270, 256], 8, 2, 128, 0, 0),
    ([300, 20], 384, [500, 384 + 19], 4, 4, 64, 0, 0),          # units on both sides of the end
    ([200, 70], 512, [600, TOP], 8, 2, 128, 100, 4),
    ([150], 4096, [4096 + 60], 4, 1, 128, 0, 0),                # key ranges cut
    ([150] + [1] * 7, 40960, [41000, 3, 40960, 40961, 500, 128, TOP, 77], 8, 2, 128, 0, 0),   # chunks beside single tokens
]


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", READS, ids=lambda c: f"{c[0][:3]}of{c[2][:3]}h{c[3]}kv{c[4]}d{c[5]}w{c[6]}s{c[7]}")
def test_attention_of_tokens_past_the_table(fa, case, dtype, fp8):
    import torch
    new, room, lens, hq, hkv, d, window, sinks = case
    b = batch(new, room, lens, hkv, d, 73, dtype, pad=2)
    q = b.draw(b.T, hq, d, loud=0)
    keys = [to_f64(b.draw(*b.cache_shape(), loud=loud)) for loud in (0.01, 0)]
    kw, cache = {}, []
    for i, name in enumerate(("k_exp", "v_exp")):
        if fp8:
            codes, byte = S.quantise_rows(keys[i])
            keys[i] = S.row_values(codes, byte)
            cache.append(dev(codes))
            kw[name] = dev(byte)
        else:
            cache.append(dev(bits(keys[i], dtype)))
    n, H = b.T * hq * d, hq
    tq = dev(q)
    ob = torch.full((n + 2 * GUARD,), -7.0, dtype=tq.dtype, device="cuda")
    lb = torch.full((b.T * H + 2 * GUARD,), -7.0, device="cuda")
    o, lse = ob[GUARD:GUARD + n].view(tq.shape), lb[GUARD:GUARD + b.T * H].view(b.T, H)
    scale = 1 / np.sqrt(d)
    fa.fa_extend_paged(tq, *cache, dev(b.table), dev(b.cu), dev(b.lens), max(new), window=window, sinks=sinks,
                       scale=scale, out=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    used = int(b.cu[-1])
    for buf in (ob, lb):
        assert bool(torch.all(buf[:GUARD] == -7.0)) and bool(torch.all(buf[-GUARD:] == -7.0))
    assert bool(torch.all(o[used:] == -7.0)) and bool(torch.all(lse[used:] == -7.0))
    got, glse = o[:used].double().cpu().numpy(), lse[:used].double().cpu().numpy()
    ro, ra, rl = np.zeros((used, hq, d)), np.zeros((used, hq, d)), np.full((used, hq), -np.inf)
    for s in range(len(new)):
        L, t0, t1 = int(b.lens[s]), int(b.cu[s]), int(b.cu[s + 1])
        pos = np.arange(L - (t1 - t0), L)
        live = min(L, room)
        see = S.visible(pos, live, window, sinks) & ((pos >= 0) & (pos < room))[:, None]
        kv = [np.concatenate([x[b.table[s, j]] for j in range(-(-live // 128))], axis=1)[:, :live] for x in keys]
        for h in range(hq):
            qh = to_f64(q)[t0:t1, h]
            ro[t0:t1, h], rl[t0:t1, h], p = S.masked_attention(qh, kv[0][h // (hq // hkv)], kv[1][h // (hq // hkv)], see, scale)
            ra[t0:t1, h] = p @ np.abs(kv[1][h // (hq // hkv)])
    assert np.isneginf(rl).any()
    compare(got, glse, ro, rl, ra, elem=dtype)
