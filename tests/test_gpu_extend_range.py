"""fa_extend_paged over E4M3 pages whose rows differ widely in size, single tokens and
tiles, against the FP64 oracle.

Tolerance, element by element, from the roundings alone (no absolute floor): P is rounded
to the 16-bit type (or to FP16, whose unit roundoff is no larger than either's), which
moves O by at most u A with A the same attention of |V|; the FP16 weights of single
tokens are held to 2^-27 of the largest weight beside them, which adds at most 2^-27 r A
with r the ratio of two keys' weights (scores here lie within +-3, so r <= e^6 < 2^9;
keys without weight are apart); sums and exponentials add 2^-16 A; O is rounded once."""
import numpy as np
import pytest

from helpers import U_ACC, U_BF16, U_F16, half_spacing
from oracle import serving as S
from serving_cases import Batch, bits, dev, to_f64

pytestmark = pytest.mark.gpu


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


class Rows:
    """An E4M3 cache written row by row. Queries have 4 in column 0, so that a key's column 0
    is its score times 4 / scale: ``quiet`` keys have none of it."""

    def __init__(self, new, lens, h_q, h_kv, d, dtype, seed, extra_pages=1):
        self.b = b = Batch(new, lens, h_kv, d, seed=seed, dtype=dtype, extra_pages=extra_pages)
        self.scale = 1 / np.sqrt(d)
        q = np.clip(b.rng.normal(size=(b.T, h_q, d)), -3, 3)
        q[..., 0] = 4.0
        self.q = bits(q, dtype)
        shape = b.cache_shape()
        # |q . k| scale <= 3: rows of k of norm 3 / (scale |q|max)
        k = b.rng.normal(size=shape)
        k[..., 0] = 0.0
        qn = np.sqrt((to_f64(self.q) ** 2).sum(-1)).max()
        self.k = k * (2.8 / (self.scale * qn) / np.sqrt((k ** 2).sum(-1, keepdims=True)))
        self.v = b.rng.normal(size=shape)

    def row(self, x, seq, key):
        """Row of `key` of sequence `seq` in x: [H_kv][d]."""
        return x[self.b.table[seq, key // 128], :, key % 128]

    def check(self, fa, window=0, sinks=0, rows=None):
        b = self.b
        (kc, ke), (vc, ve) = S.quantise_rows(to_f64(bits(self.k, b.dtype))), S.quantise_rows(to_f64(bits(self.v, b.dtype)))
        o, lse = fa.fa_extend_paged(dev(self.q), dev(kc), dev(vc), dev(b.table), dev(b.cu), dev(b.lens), int(b.new.max()),
                                    window=window, sinks=sinks, scale=self.scale, k_exp=dev(ke), v_exp=dev(ve))
        assert fa.fa_device_status() == fa.FA_OK
        ks, vs = b.rows(S.row_values(kc, ke)), b.rows(S.row_values(vc, ve))
        ro, rl, ra = S.extend_reference(to_f64(self.q), ks, vs, b.cu, b.lens, self.scale, window, sinks)
        u = (U_F16 if b.dtype == "f16" else U_BF16) + U_ACC + 2.0 ** (9 - 27)
        err = np.abs(o.double().cpu().numpy() - ro) / (half_spacing(np.abs(ro) + u * ra, b.dtype) + u * ra)
        rows = slice(None) if rows is None else rows
        assert np.isfinite(o[rows].float().cpu().numpy()).all()
        assert err[rows].max() <= 1.0, float(err[rows].max())
        assert np.abs(lse.double().cpu().numpy() - rl)[rows].max() <= 1e-3


FORMS = [([1, 1], 8, 2), ([2, 2], 8, 1), ([20, 9], 8, 2)]     # 4 rows a KV head, 16, tiles
FORM_IDS = ["few8", "few16", "tiles"]


def _loud(d):
    return np.where(np.arange(d) % 2 == 0, 1.0, -0.75)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 36, 40, 58])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_a_loud_value_no_token_gives_weight(fa, form, size, d):
    # rows 2^size above the others, with scores of -150: their weight is below 2^-200
    new, hq, hkv = form
    p = Rows(new, [700, 300], hq, hkv, d, "bf16", 61)
    for seq, key in ((0, 3), (0, 200), (0, 640), (1, 5), (1, 131)):
        p.row(p.v, seq, key)[:] = _loud(d) * 2.0 ** size
        p.row(p.k, seq, key)[:, 0] = -150 / (4 * p.scale)
    p.check(fa)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 40, 58])
@pytest.mark.parametrize("form", [([3, 2], 8, 2), ([5, 3], 6, 2), ([20, 9], 8, 2)], ids=["few12", "few15", "tiles"])
def test_a_loud_value_of_a_later_token(fa, form, size, d):
    # the last token's own row: the tokens before it do not see it
    new, hq, hkv = form
    p = Rows(new, [400, 131], hq, hkv, d, "bf16", 62)
    for seq, key in ((0, 399), (1, 130)):
        p.row(p.v, seq, key)[:] = _loud(d) * 2.0 ** size
    p.check(fa)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 40, 58])
@pytest.mark.parametrize("sinks", [0, 2])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_a_loud_value_left_of_the_window(fa, form, sinks, size, d):
    # in tiles that the window enters, and beside the sinks
    new, hq, hkv = form
    p = Rows(new, [700, 300], hq, hkv, d, "bf16", 63)
    for seq, L, n in ((0, 700, new[0]), (1, 300, new[1])):
        for key in (2, 70, L - n - 90):      # the first token's window begins at L - n - 89
            p.row(p.v, seq, key)[:] = _loud(d) * 2.0 ** size
    p.check(fa, window=90, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20, 40, 58])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_a_loud_value_in_one_column(fa, form, size, d):
    # seen with an ordinary weight: the other columns hold the other keys' values, whole
    new, hq, hkv = form
    p = Rows(new, [90, 260], hq, hkv, d, "bf16", 64)
    for seq, key, col in ((0, 7, 3), (0, 60, 4), (1, 133, 0), (1, 4, d - 1)):
        v = p.row(p.v, seq, key)
        v[:] = 0.0
        v[:, col] = 2.0 ** size
    p.check(fa)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_a_small_weight_on_a_loud_value(fa, form, d):
    # weight 2^-45 on 2^58: the product outweighs all the rest
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, d, "bf16", 65)
    for seq, key in ((0, 20), (0, 150), (1, 40)):
        p.row(p.v, seq, key)[:] = _loud(d) * 2.0 ** 58
        p.row(p.k, seq, key)[:, 0] = -45 * np.log(2) / (4 * p.scale)
    p.check(fa)


@pytest.mark.parametrize("dtype,low,high", [("bf16", -100, 56), ("f16", -14, 13)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_values_of_every_size(fa, form, d, dtype, low, high):
    new, hq, hkv = form
    p = Rows(new, [700, 300], hq, hkv, d, dtype, 66)
    p.v *= 2.0 ** p.b.rng.integers(low, high + 1, p.v.shape[:-1])[..., None]
    p.v[p.b.rng.random(p.v.shape[:-1]) < 0.05] = 0.0
    if dtype == "f16":
        p.v = np.clip(p.v, -60000, 60000)
    p.check(fa)


@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_values_that_are_all_tiny(fa, form):
    # every row at 2^-100: the result is not lost below the accumulators' range
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, 128, "bf16", 67)
    p.v *= 2.0 ** -100
    p.check(fa)


# ---- keys and queries of very different sizes, whose scores are ordinary
@pytest.mark.parametrize("size", [60, 104])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_huge_keys_under_tiny_queries(fa, form, d, size):
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, d, "bf16", 68)
    p.k *= 2.0 ** size
    p.q = bits(to_f64(p.q) * 2.0 ** -size, "bf16")
    p.check(fa)


@pytest.mark.parametrize("size", [60, 100])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_tiny_keys_under_huge_queries(fa, form, d, size):
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, d, "bf16", 69)
    p.k *= 2.0 ** -size
    p.q = bits(to_f64(p.q) * 2.0 ** size, "bf16")
    p.check(fa)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_huge_keys_that_a_huge_query_does_not_meet(fa, form, d):
    # products beyond FP32 where no column is shared: those scores are 0
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, d, "bf16", 70)
    q = np.zeros_like(to_f64(p.q))
    q[..., : d // 2] = 2.0 ** 100
    p.q = bits(q, "bf16")
    p.k[..., : d // 2] = 0.0
    p.k[..., d // 2:] = 2.0 ** 104
    p.check(fa)


@pytest.mark.parametrize("byte", [0, 1, 3, 7])
@pytest.mark.parametrize("form", FORMS, ids=FORM_IDS)
def test_the_smallest_exponent_bytes(fa, form, byte):
    # rows of another writer, below what fa_cache_append makes: still code * 2^(byte - 127)
    new, hq, hkv = form
    p = Rows(new, [300, 90], hq, hkv, 128, "bf16", 74)
    rng = np.random.default_rng(byte)
    b = p.b
    codes = [rng.integers(0x30, 0x7E, b.cache_shape()).astype(np.uint8) for _ in range(2)]
    kb, vb = (np.full(b.cache_shape()[:3], byte, np.uint8) for _ in range(2))
    p.q = bits(rng.normal(size=to_f64(p.q).shape) * 2.0 ** (127 - byte - 13), "bf16")
    o, lse = fa.fa_extend_paged(dev(p.q), dev(codes[0]), dev(codes[1]), dev(b.table), dev(b.cu), dev(b.lens), int(b.new.max()),
                                scale=2.0 ** -5, k_exp=dev(kb), v_exp=dev(vb))
    ks, vs = b.rows(S.row_values(codes[0], kb)), b.rows(S.row_values(codes[1], vb))
    ro, rl, ra = S.extend_reference(to_f64(p.q), ks, vs, b.cu, b.lens, 2.0 ** -5)
    # weights differ by any amount here: the 2^-27 of the largest is on the largest value, 448 * 2^byte
    err = np.abs(o.double().cpu().numpy() - ro)
    u = U_BF16 + U_ACC
    floor = 300 * 2.0 ** -27 * 448 * 2.0 ** (byte - 127)
    assert (err <= half_spacing(np.abs(ro) + u * ra + floor) + u * ra + floor + 2.0 ** -133).all(), float(err.max() / np.abs(ro).max())
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-3 + 2.0 ** -20 * np.abs(rl).max()
