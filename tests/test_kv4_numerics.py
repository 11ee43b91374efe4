"""What the operators of the 4-bit paged cache promise about roundings and ranges, on the GPU."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from test_kv4 import DEV, Setup, axes_of, dev, host, pm, rows  # noqa: F401

pytestmark = pytest.mark.gpu

# D, rotated channels, interleaved: pairs half a head apart, neighbours, any other distance
FORMS = [(128, 128, False), (128, 128, True), (128, 96, False), (128, 48, True), (64, 64, False), (64, 64, True),
         (64, 32, False), (128, 0, False)]


def rope_of(pm, D, rot, inter, axes):  # noqa: F811
    inv = [np.float32(500000.0 ** (-2 * i / max(rot, 1))) for i in range(rot // 2)]
    args = dict(inv_freq=inv, axis=axes_of(rot, axes), rot=rot, interleaved=inter, eps=2.0 ** -20)
    rope = pm.Rope.make(D, rot, inv_freq=inv, axes=args["axis"], interleaved=inter, eps=args["eps"])
    rope.n_axes = axes
    return rope, args


@pytest.mark.parametrize("D,rot,inter", FORMS)
@pytest.mark.parametrize("weights", [True, False])
def test_keys_are_the_64_bit_definitions(pm, D, rot, inter, weights):  # noqa: F811
    """Rotated keys are bf16(fp32(y)) of the definition's y, and what the fused write stores are the
    codes of those rows.  The kernel's y is off by some 2^-50; it rounds otherwise than the
    definition's only where that spans a border of fp32 next to one of bf16, 2^-42 a key.  (fp32
    arithmetic moves one key in 20000 to the neighbouring bf16.)"""
    Hq, Hkv, n, page, axes = 4, 4, 4000, 64, 3
    q, k, v = (rows(i, n, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    r = np.random.default_rng(4)
    w = [ref.bf16(1 + 0.3 * r.standard_normal(D)) if weights else None for _ in range(2)]
    wd = [None if x is None else dev(x) for x in w]
    pos = r.integers(0, 200000, (axes, n)).astype(np.int32)
    rope, args = rope_of(pm, D, rot, inter, axes)
    y, _ = ref.norm_rope(k, w[1], pos, **args)
    want = ref.bf16_from_f32(y.astype(np.float32))
    got = host(pm.norm_rope(rope, dev(q), dev(k), dev(pos, torch.int32), *wd)[1])
    assert np.array_equal(got, want), (got != want).sum()
    s = Setup(pm, [n], [n], Hq, Hkv, D, page)
    s.cache.append_qkv(s.batch, rope, dev(q), dev(k), dev(v), dev(pos, torch.int32), *wd)
    ko, vo = s.cache.read(s.batch)
    assert np.array_equal(host(ko), ref.bf16_from_f32(ref.stand_for(*ref.quantise(want))))
    assert np.array_equal(host(vo), ref.bf16_from_f32(ref.stand_for(*ref.quantise(v))))


@pytest.mark.parametrize("D,rot,inter", FORMS)
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("T,Hq,Hkv", [([1], 4, 2), ([40, 1, 300], 7, 1), ([1400, 0, 9], 6, 3)])
def test_every_form_of_the_fused_write_equals_the_two_calls(pm, D, rot, inter, weights, T, Hq, Hkv):  # noqa: F811
    a, b = (Setup(pm, [t + 5 for t in T], T, Hq, Hkv, D, 32) for _ in range(2))
    qkv = dev(rows(21, a.n, Hq + 2 * Hkv, D))
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    rope, _ = rope_of(pm, D, rot, inter, 2)
    pos = dev(np.random.default_rng(22).integers(-50, 70000, (2, a.n)).astype(np.int32), torch.int32)
    w = [dev(ref.bf16(1 + 0.2 * np.random.default_rng(i).standard_normal(D))) if weights else None for i in range(2)]
    qo = a.cache.append_qkv(a.batch, rope, q, k, v, pos, *w)
    q2, k2 = pm.norm_rope(rope, q, k, pos, *w)
    b.cache.append(b.batch, k2, v)
    assert torch.equal(qo, q2) and torch.equal(a.cache.pages(), b.cache.pages())


def test_keys_of_extreme_rows(pm):  # noqa: F811
    """Rows whose squares leave fp32, zeros, infinities and NaN: as the definition has them."""
    D, n = 128, 7
    k = rows(31, n, 1, D)
    k[1] *= np.float32(1e30)
    k[2] = ref.bf16(k[2].astype(np.float64) * 1e-36)
    k[3] = 0
    k[4, 0, 5], k[5, 0, 6] = np.inf, np.nan
    k = host(dev(k))        # what the call sees: bf16
    w = ref.bf16(1 + 0.3 * np.random.default_rng(32).standard_normal(D))
    pos = np.zeros((1, n), np.int32)
    rope, args = rope_of(pm, D, D, False, 1)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.bf16_from_f32(ref.norm_rope(k, w, pos, **args)[0].astype(np.float32))
    got = host(pm.norm_rope(rope, None, dev(k), dev(pos[0], torch.int32), None, dev(w))[1])
    keep = [0, 1, 2, 3, 6]
    assert np.array_equal(got[keep], want[keep])
    assert np.isnan(got[4, 0, 5]) and np.isnan(got[5]).all()


# ---------------------------------------------------------------- the range of logits

def cached(pm, kv_len, T, Hq, Hkv, D, k, v, page=32):  # noqa: F811
    """A batch over sequences that all hold the rows k, v [tokens][Hkv][D]."""
    s = Setup(pm, kv_len, T, Hq, Hkv, D, page)
    for b, n in enumerate(kv_len):
        one = pm.KV4Batch(dev(np.array([n]), torch.int32), dev(s.table[b:b + 1], torch.int32), n_tokens=n)
        s.cache.append(one, dev(k[:n]), dev(v[:n]))
    return s


def mean_of_tokens(v, tokens):
    """What attention gives whose weight lies evenly on some tokens, and what may be off: the values'
    fp16 form (2^-11 of code * s and of the zero point), the weights' (2^-11 each) and bf16."""
    x = ref.stand_for(*ref.quantise(v[tokens])).astype(np.float64)
    return x.mean(0), np.abs(x).mean(0) * (2.0 ** -8 + 2.0 ** -10) + np.abs(v[tokens]).max() * 2.0 ** -10


FAR = [1e4, 1e6, 1e9, 1e20, 1e29]


@pytest.mark.parametrize("T", [20, 140])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("amp", FAR)
def test_attention_where_logits_are_very_large(pm, T, D, amp):  # noqa: F811
    """Three equal tokens, in three tiles, whose logit is far above all others: each row is their mean."""
    r = np.random.default_rng(401)
    n = 600
    k, v = r.standard_normal((n, 1, D)) * 0.05, rows(402, n, 1, D)
    base = ref.bf16(np.sign(r.standard_normal(D)) * (1 + r.random(D)))
    k = ref.bf16(k)
    hot = [3, 200, 300]
    k[hot] = base
    s = cached(pm, [n], [T], 4, 1, D, k, v)
    q = ref.bf16(np.tile(base, (T, 4, 1)) * amp)
    out = host(s.cache.attend(s.batch, dev(q)))
    assert s.cache.read_error() == 0
    want, tol = mean_of_tokens(v, hot)
    assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max()


@pytest.mark.parametrize("T", [40, 140])
@pytest.mark.parametrize("amp", FAR)
def test_attention_where_very_large_logits_grow(pm, T, amp):  # noqa: F811
    """Each token's logit is a twentieth above the one's before, so every row is its own token's value."""
    r = np.random.default_rng(403)
    n, D = 150, 128
    base = ref.bf16(r.standard_normal(D))
    k = ref.bf16(1.05 ** np.arange(n)[:, None, None] * base * 0.05)
    v = rows(404, n, 1, D)
    s = cached(pm, [n], [T], 2, 1, D, k, v)
    q = ref.bf16(np.tile(base, (T, 2, 1)) * amp)
    out = host(s.cache.attend(s.batch, dev(q)))
    assert s.cache.read_error() == 0
    for j in range(T):
        want, tol = mean_of_tokens(v, [n - T + j])
        assert (np.abs(out[j] - want) <= tol).all(), (j, np.abs(out[j] - want).max())


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("vamp", [1e-5, 1.0, 2000.0])
def test_attention_of_few_rows_where_logits_are_very_large(pm, T, D, vamp):  # noqa: F811
    """As above for tiles of 8 and 16 rows, where the weights meet the fp16 range times a value scale:
    one of the three tokens has values 64 times smaller than the others."""
    r = np.random.default_rng(411)
    n = 600
    k, v = ref.bf16(r.standard_normal((n, 1, D)) * 0.05), rows(412, n, 1, D, vamp)
    v[200] /= 64
    base = ref.bf16(np.sign(r.standard_normal(D)) * (1 + r.random(D)))
    hot = [3, 200, 300]
    k[hot] = base
    s = cached(pm, [n], [T], 4, 1, D, k, v)
    want, tol = mean_of_tokens(v, hot)
    for amp in [2.0 ** i for i in range(12, 40)] + [1e20, 1e29]:
        q = ref.bf16(np.tile(base, (T, 4, 1)) * amp)
        out = host(s.cache.attend(s.batch, dev(q)))
        assert (np.abs(out - want) <= tol).all(), (amp, np.abs(out - want).max())
    assert s.cache.read_error() == 0


@pytest.mark.parametrize("T", [1, 4])
def test_attention_of_few_rows_where_very_large_logits_grow(pm, T):  # noqa: F811
    r = np.random.default_rng(413)
    n, D = 150, 128
    base = ref.bf16(r.standard_normal(D))
    k = ref.bf16(1.05 ** np.arange(n)[:, None, None] * base * 0.05)
    v = rows(414, n, 1, D) * (2.0 ** r.integers(-12, 6, (n, 1, 1))).astype(np.float32)
    s = cached(pm, [n], [T], 4, 1, D, k, v)
    for amp in [2.0 ** i for i in range(12, 40, 3)] + [1e20, 1e29]:
        q = ref.bf16(np.tile(base, (T, 4, 1)) * amp)
        out = host(s.cache.attend(s.batch, dev(q)))
        for j in range(T):
            want, tol = mean_of_tokens(v, [n - T + j])
            assert (np.abs(out[j] - want) <= tol).all(), (amp, j, np.abs(out[j] - want).max())
    assert s.cache.read_error() == 0


@pytest.mark.parametrize("T", [1, 4, 20, 140])
@pytest.mark.parametrize("c,d", [(4.0, 0), (10.5, 0), (13.0, 0), (15.25, 0), (4.0, 0.5), (15.25, 0.5), (16.25, 0.5)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_one_strong_token_over_many_weak_ones(pm, T, c, d, sign):  # noqa: F811
    """A first token whose weight is 2^5 to 2^21.3 times that of each of 30000 others, which hold an
    odd channel each way: what the others add up to is kept.  160 units of one row tile or more, so a
    CTA takes whole ones.  Keys and values are exact in 4 bits, so the logits are.  Off may be, in all
    of 30000 weak terms alike: with up to 16 rows per tile the products of weights and scales by 2^-11 of
    themselves or 2^-33 of the largest (2^-11.7 of the smallest here), with more the weights by 2^-30
    of the largest (2^-8.7 of the smallest); values in fp16 not at all, the fp32 sums 2^-12, bf16 2^-8.
    Where the strong token's zero is code * s + z = 15/16 - 15/16 (negative sign), the row kernel's
    product weight * s is rounded to fp16 and its weight * z is not: 2^-11 of weight * 15/16."""
    B, Hq, Hkv, D, n, page = 40, 16, 4, 64, 30000, 128
    k, v = (np.zeros((n, Hkv, D), np.float32) for _ in range(2))
    k[0, :, ::2] = 15 / 8
    k[1:, :, 1::2] = 15 / 8
    v[0, :, 1::2] = sign * 15 / 16
    v[1:, :, ::2] = 15 / 16
    cfg, pages = pm.KV4Config.make(Hq, Hkv, D, page, 1 / 64), -(-n // page)
    cache = pm.KV4Cache(cfg, pages)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(B, 1)          # all of them share the pages
    length = torch.full((B,), n, dtype=torch.int32, device=DEV)
    cache.append(pm.KV4Batch(length[:1], table[:1], n_tokens=n), dev(k), dev(v))
    q = torch.zeros(B * T, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, ::2] = c
    q[:, :, 1::2] = d
    out = host(cache.attend(pm.KV4Batch(length, table, n_tokens=B * T), q)).reshape(B, T, Hq, D)
    strong = np.exp(32 * 15 / 8 * c / 64)
    weak = np.exp(32 * 15 / 8 * d / 64) * (n - T + np.arange(T))[:, None, None]
    even = np.arange(D) % 2 == 0
    want = np.where(even, 15 / 16 * weak, sign * 15 / 16 * strong) / (weak + strong)
    tol = np.abs(want) * (2.0 ** -8 + (2.0 ** -10 if T < 20 else 2.0 ** -8.5))
    if sign < 0 and T < 20:
        tol = tol + even * 2.0 ** -11 * 15 / 16 * strong / (weak + strong)
    assert (np.abs(out - want) <= tol).all(), np.abs(out / want - 1).max()
    assert cache.read_error() == 0


@pytest.mark.parametrize("T", [1, 4, 20, 140])
@pytest.mark.parametrize("kamp", [1.0, 3000.0])
def test_rows_whose_logits_are_all_very_low(pm, T, kamp):  # noqa: F811
    """Equal logits of -1e31 and below are a softmax like any other."""
    r = np.random.default_rng(421)
    n, D = 700, 128
    base = ref.bf16(np.sign(r.standard_normal(D)) * (1 + r.random(D)))
    k, v = np.tile(ref.bf16(base * kamp), (n, 1, 1)), rows(422, n, 1, D)
    s = cached(pm, [n], [T], 4, 1, D, k, v)
    out = host(s.cache.attend(s.batch, dev(np.tile(ref.bf16(base * -5e29), (T, 4, 1)))))
    for j in range(T):
        want, tol = mean_of_tokens(v, np.arange(n - T + j + 1))
        assert (np.abs(out[j] - want) <= tol).all(), (j, np.abs(out[j] - want).max())


@pytest.mark.parametrize("T", [1, 4, 20, 140])
def test_a_scale_that_leaves_no_logit(pm, T):  # noqa: F811
    """Queries and a softmax scale whose product is below fp32: every row is the mean of what it sees."""
    n, D = 300, 128
    k, v = rows(431, n, 1, D), rows(432, n, 1, D)
    s = cached(pm, [n], [T], 4, 1, D, k, v)
    cfg = pm.KV4Config.make(4, 1, D, 32, 1e-12)
    cache = pm.KV4Cache(cfg, s.n_pages, buffer=s.cache.buffer)
    out = host(cache.attend(s.batch, dev(rows(433, T, 4, D, 1e-36))))
    for j in range(T):
        want, tol = mean_of_tokens(v, np.arange(n - T + j + 1))
        assert (np.abs(out[j] - want) <= tol).all(), (j, np.abs(out[j] - want).max())


@pytest.mark.parametrize("D,Hq,Hkv,T,lens", [(128, 4, 1, 30, [20000]), (64, 4, 2, 70, [9000, 300]),
                                             (128, 8, 2, 140, [6000, 200]), (128, 28, 4, 5, [8000, 5000, 6])])
def test_many_rows_over_long_contexts(pm, D, Hq, Hkv, T, lens):  # noqa: F811
    """Tiles of 128 and 256 rows (the last: 16) whose units many CTAs share, against the definition."""
    s = Setup(pm, lens, [min(T, n) for n in lens], Hq, Hkv, D, 64)
    s.fill(441)
    q = rows(442, s.n, Hq, D)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))
    assert s.cache.read_error() == 0
