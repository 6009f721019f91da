"""What cu_seqlens and seqlens_k may hold: values that point anywhere are clamped, and what
that leaves is defined, as far as cu_seqlens does not decrease; nothing outside the tensors is
reached in any case."""
import numpy as np
import pytest

from helpers import compare
from oracle import serving as S
from serving_cases import dev, to_f64
from test_gpu_extend import GUARD, Problem, fa  # noqa: F401

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
# single tokens, tiles, and both kernels over E4M3 pages
SHAPES = [([1, 2, 1], [300, 129, 40], False, 1), ([40, 1, 30], [300, 129, 64], False, 1),
          ([1, 2, 1], [300, 129, 40], True, 1), ([70] + [1] * 8, [200] + [130] * 8, True, 600)]
IDS = ["few", "tiles", "few-e4m3", "both"]


def _problem(i):
    new, lens, fp8, extra = SHAPES[i]
    return Problem(new, lens, 8, 2, 128, "bf16", fp8, seed=81, pad=2, extra_pages=extra)


def _guarded(shape, dtype):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), -7.0, dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + n].view(shape)


def _run(fa, p, cu, lens):  # noqa: F811
    """O and LSE of a call with these lengths, inside margins that must stay as they were."""
    import torch
    q, a = dev(p.q), p.args()
    a["cu_seqlens"].copy_(torch.tensor(cu, dtype=torch.int32))
    a["seqlens_k"].copy_(torch.tensor(lens, dtype=torch.int32))
    (ob, o), (lb, lse) = _guarded(q.shape, q.dtype), _guarded(q.shape[:2], torch.float32)
    fa.fa_extend_paged(q, **a, out=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    for buf in (ob, lb):
        assert bool(torch.all(buf[:GUARD] == -7.0)) and bool(torch.all(buf[-GUARD:] == -7.0))
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(p, o, lse, cu, lens, max_q):
    """Against the definition, with cu clamped to [0, T] and lengths to 0 and more."""
    T = p.b.T
    cu = np.clip(np.array(cu, np.int64), 0, T)
    touched = np.zeros(T, bool)
    for b, L in enumerate(np.maximum(np.array(lens, np.int64), 0)):
        n = int(cu[b + 1] - cu[b])
        for t in range(min(n, max_q)):
            row, pos = int(cu[b]) + t, int(L) - n + t
            touched[row] = True
            if not 0 <= pos < p.b.max_pages * 128:
                assert (o[row] == 0).all() and np.isneginf(lse[row]).all()
                continue
            keys = [np.concatenate([x[p.b.table[b, j]] for j in range(pos // 128 + 1)], axis=1)[:, :pos + 1] for x in p.values]
            for h in range(p.h_q):
                kv = [k[h // (p.h_q // k.shape[0])] for k in keys]
                ro, rl, pr = S.masked_attention(to_f64(p.q)[row:row + 1, h], *kv, np.ones((1, pos + 1), bool), p.scale)
                compare(o[row:row + 1, h], lse[row:row + 1, h], ro, rl, pr @ np.abs(kv[1]), tol_rel=1.0)
    assert (o[~touched] == -7.0).all() and (lse[~touched] == -7.0).all()


@pytest.mark.parametrize("i", range(4), ids=IDS)
def test_lengths_of_any_value(fa, i):  # noqa: F811
    p = _problem(i)
    B, T, own = len(p.b.new), p.b.T, p.b.cu.tolist()
    mq, L = int(p.b.new.max()), p.b.lens.tolist()
    for cu, lens in ((own, [-1] * B),                              # no keys: O = 0, LSE = -inf
                     (own, [-TOP - 1] * B),
                     (own, [TOP] * B),                             # all past the table
                     (own, [p.b.max_pages * 128 + mq] * B),
                     (own, L[:-1] + [TOP]),                        # one of them
                     ([TOP] * (B + 1), L),                         # every row is padding
                     ([-TOP] * (B + 1), L),
                     ([0] * B + [TOP], [TOP] * B),                 # one sequence has every row
                     ([-5] + [T] * B, [-1] * B),
                     ([-9, 1] + [1] * (B - 1), L),                 # one row in all
                     ([0] + [1] * B, [-TOP] * B)):
        o, lse = _run(fa, p, cu, lens)
        _check(p, o, lse, cu, lens, mq)


@pytest.mark.parametrize("i", range(4), ids=IDS)
def test_decreasing_cu_seqlens_stay_inside(fa, i):  # noqa: F811
    p = _problem(i)
    B, T = len(p.b.new), p.b.T
    for cu, lens in ((list(range(B, -1, -1)), [100] * B), ([T * (b % 2) for b in range(B + 1)], [TOP] * B),
                     ([T * (b % 2) for b in range(B + 1)], [120] * B), ([T, 0] + [T // 2] * (B - 1), [90] * B)):
        o, lse = _run(fa, p, cu, lens)
        end = min(max(cu), T)          # rows past every sequence are nobody's
        assert (o[end:] == -7.0).all() and (lse[end:] == -7.0).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "e4m3"])
def test_cache_calls_stay_inside(fa, fp8):  # noqa: F811
    import torch
    p = Problem([3, 40, 2], [130, 300, 60], 2, 2, 64, "bf16", fp8, seed=82, pad=2)
    b = p.b
    B, T, own = 3, b.T, b.cu.tolist()
    k, v = dev(b.draw(T, 2, 64)), dev(b.draw(T, 2, 64))
    dt = torch.uint8 if fp8 else torch.bfloat16
    for cu, lens, writes in ((own, [-1] * B, False), (own, [TOP] * B, False), ([TOP] * (B + 1), b.lens.tolist(), False),
                             ([-TOP] * (B + 1), b.lens.tolist(), False), (own, b.lens.tolist(), True),
                             ([T, 3, 0, T], [b.max_pages * 128] * B, True), ([5, 1, 9, 2], [TOP, 60, -3], True)):
        cu_t, lens_t = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens))
        bufs = [_guarded(b.cache_shape(), torch.float32 if fp8 else dt) for _ in range(2)]
        if fp8:
            bufs = [(x := torch.full((buf.numel(),), 9, dtype=dt, device="cuda"), x[GUARD:-GUARD].view(c.shape)) for buf, c in bufs]
            ebuf = [torch.full((c.numel() // 64 + 2 * GUARD,), 9, dtype=dt, device="cuda") for _, c in bufs]
            exps = [e[GUARD:-GUARD].view(b.cache_shape()[:3]) for e in ebuf]
        else:
            ebuf, exps = [], [None, None]
        old = [c.clone() for _, c in bufs]
        fa.fa_cache_append(k, v, bufs[0][1], bufs[1][1], dev(b.table), cu_t, lens_t, k_exp=exps[0], v_exp=exps[1])
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        for x in [y for y, _ in bufs] + ebuf:
            assert bool(torch.all(x[:GUARD] == x[0])) and bool(torch.all(x[-GUARD:] == x[0])) and x[0].item() in (9, -7)
        for (_, c), o in zip(bufs, old):
            assert writes or torch.equal(c, o)
        (kb, kr), (vb, vr) = _guarded((T, 2, 64), torch.bfloat16), _guarded((T, 2, 64), torch.bfloat16)
        fa.fa_cache_read(bufs[0][1], bufs[1][1], dev(b.table), cu_t, lens_t, T, k=kr, v=vr, k_exp=exps[0], v_exp=exps[1])
        torch.cuda.synchronize()
        for x in (kb, vb):
            assert bool(torch.all(x[:GUARD] == -7.0)) and bool(torch.all(x[-GUARD:] == -7.0))
        if not writes:       # rows without a place read as zeros, padding stays
            end = min(max(cu[-1], 0), T)
            start = min(max(cu[0], 0), T)
            assert bool(torch.all(kr[start:end] == 0)) and bool(torch.all(vr[start:end] == 0))
            assert bool(torch.all(kr[end:] == -7.0)) and bool(torch.all(vr[end:] == -7.0))


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "e4m3"])
def test_few_rows_over_several_steps_of_the_plan(fa, fp8):  # noqa: F811
    # the plan takes 128 sequences a step, four a lane
    rng = np.random.default_rng(5)
    new = rng.integers(0, 3, 300).tolist()
    lens = [int(n + rng.integers(0, 400)) for n in new]
    Problem(new, lens, 4, 2, 64, fp8=fp8, seed=83).check(fa)


@pytest.mark.parametrize("new", [1, 40], ids=["few", "tiles"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_value_leaves_the_lse(fa, d, new):  # noqa: F811
    p = Problem([new, new], [300, 400], 4, 2, d, "bf16", True, seed=84)
    clean = p.run(fa)
    page = int(p.b.table[1, 1])
    p.exps[1][page, :, 5], p.caches[1][page, :, 5] = 255, 0x7F
    o, lse = p.run(fa)
    assert np.isnan(o[new:]).all() and np.array_equal(o[:new], clean[0][:new])
    assert np.array_equal(lse, clean[1]) and np.isfinite(lse).all()
