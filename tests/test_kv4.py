"""The 4-bit paged cache on the GPU against its restatement in float64 (kv4_ref.py)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def rows(seed, n, heads, D, amp=1.0, outliers=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, heads, D))
    if outliers and n:
        x[:, :, r.integers(0, D, 3)] *= 6
    return ref.bf16(x * amp)


def dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(dtype)


def host(t):
    return t.float().cpu().numpy()


class Setup:
    """A batch of sequences with pages in scattered order."""

    def __init__(self, pm, kv_len, T, Hq, Hkv, D, page, seed=0, spare=2, pad=0, uniform=False, max_pages=None, scale=0.0):
        self.pm, self.kv_len, self.T, self.D, self.page = pm, list(kv_len), list(T), D, page
        self.Hq, self.Hkv = Hq, Hkv
        B = len(kv_len)
        per = max(1, max(-(-int(x) // page) for x in kv_len)) if max_pages is None else max_pages
        r = np.random.default_rng(seed + 99)
        self.n_pages = B * per + spare
        self.table = r.permutation(self.n_pages)[:B * per].reshape(B, per).astype(np.int32)
        self.start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
        self.n = int(self.start[-1]) + pad
        self.cfg = pm.KV4Config.make(Hq, Hkv, D, page, scale)
        self.scale = scale or ref.default_scale(D)
        self.cache = pm.KV4Cache(self.cfg, self.n_pages)
        self.batch = self.make_batch(self.kv_len, self.start, uniform)

    def make_batch(self, kv_len, start, uniform=False, max_q=None):
        n = int(start[-1]) if len(start) else 0
        n = max(n, self.n)
        return self.pm.KV4Batch(dev(np.array(kv_len), torch.int32), dev(self.table, torch.int32),
                                None if uniform else dev(np.array(start), torch.int32), n_tokens=n,
                                max_q=max_q or (None if uniform else max(1, max(np.diff(start)))))

    def fill(self, seed=1, amp=1.0):
        """Append every cached token at once, in front of the measured call."""
        start = np.concatenate([[0], np.cumsum(self.kv_len)]).astype(np.int32)
        n = int(start[-1])
        if n == 0:
            return
        b = self.pm.KV4Batch(dev(np.array(self.kv_len), torch.int32), dev(self.table, torch.int32),
                             dev(start, torch.int32), n_tokens=n)
        self.cache.append(b, dev(rows(seed, n, self.Hkv, self.D, amp)), dev(rows(seed + 1, n, self.Hkv, self.D, amp)))

    def raw(self):
        return self.cache.pages().cpu().numpy()

    def check_attention(self, q, out, start=None, kv_len=None):
        want, tol = ref.attention(self.raw(), self.table, self.kv_len if kv_len is None else kv_len,
                                  self.start if start is None else start, q, self.scale, self.page, self.D)
        got = host(out)
        n = int((self.start if start is None else start)[-1])
        assert np.isfinite(got[:n]).all()
        bad = np.abs(got[:n] - want[:n]) > tol[:n]
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got[:n] - want[:n]).max())


@pytest.fixture(scope="module")
def pm():
    import decode_attention_prefill_b200 as m
    return m


# ---------------------------------------------------------------- norm and rotation

def axes_of(rot, n):
    return [i % n for i in range(rot // 2)] if n > 1 else [0] * (rot // 2)


def check_norm_rope(got, x, w, pos, rope_args):
    want, mag = ref.norm_rope(x, w, pos, **rope_args)
    # half a bf16 step of the value; fp32: a dozen roundings of the pair's magnitude and 2^-22
    # of it from the angle
    tol = np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -19 + 1e-37
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


@pytest.mark.parametrize("n,hq,hk,D,rot,axes,inter", [
    (1, 32, 8, 128, 128, 1, False), (1, 1, 1, 64, 64, 1, True), (7, 3, 1, 128, 96, 3, True),
    (33, 4, 4, 64, 48, 2, False), (65, 28, 4, 128, 128, 3, False), (5, 2, 1, 256, 256, 1, False),
    (5, 2, 3, 256, 16, 4, True), (3, 2, 2, 128, 0, 1, False), (700, 5, 2, 128, 112, 1, False),
    (1300, 3, 1, 64, 64, 1, True)])
@pytest.mark.parametrize("weights", [True, False])
def test_norm_rope(pm, n, hq, hk, D, rot, axes, inter, weights):
    q, k = rows(1, n, hq, D), rows(2, n, hk, D)
    r = np.random.default_rng(5)
    wq, wk = (ref.bf16(1 + 0.3 * r.standard_normal(D)) for _ in range(2)) if weights else (None, None)
    pos = r.integers(0, 200000, (axes, n)).astype(np.int32)
    inv = [10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]
    rope = pm.Rope.make(D, rot, inv_freq=inv, axes=axes_of(rot, axes), interleaved=inter, eps=1e-5)
    if rot == 0:
        rope.n_axes = axes
    qo, ko = pm.norm_rope(rope, dev(q), dev(k), dev(pos, torch.int32), None if wq is None else dev(wq),
                          None if wk is None else dev(wk))
    args = dict(inv_freq=inv, axis=axes_of(rot, axes), rot=rot, interleaved=inter, eps=1e-5)
    check_norm_rope(host(qo), q, wq, pos, args)
    check_norm_rope(host(ko), k, wk, pos, args)


def test_norm_rope_far_and_negative_positions(pm):
    D, n = 128, 6
    q, k = rows(3, n, 2, D), rows(4, n, 1, D)
    pos = np.array([[0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31)]], np.int32)
    inv = [500000.0 ** (-i / 64) for i in range(64)]
    # the fp64 product of a 31-bit position and a 24-bit frequency is off by 2^-53 of up to
    # 2^31 rad: 2^-22; times the pair's magnitude that stays inside check_norm_rope's 2^-19
    qo, ko = pm.norm_rope(pm.Rope.make(D, inv_freq=inv), dev(q), dev(k), dev(pos, torch.int32))
    args = dict(inv_freq=inv, axis=[0] * 64, rot=D, interleaved=False, eps=1e-6)
    check_norm_rope(host(qo), q, None, pos, args)
    check_norm_rope(host(ko), k, None, pos, args)


def test_norm_rope_strided_in_place_and_zero_rows(pm):
    n, hq, hk, D = 19, 4, 2, 128
    qkv = dev(rows(6, n, hq + 2 * hk, D))
    before = qkv.clone()
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    w = dev(np.ones(D, np.float32))
    rope = pm.Rope.make(D)
    want = pm.norm_rope(rope, before[:, :hq].contiguous(), before[:, hq:hq + hk].contiguous(), pos, w, w)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    got = pm.norm_rope(rope, q, k, pos, w, w, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])
    # head-major outputs, as the mixed-precision cache takes its keys
    ko = torch.full((hk, n + 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pm.norm_rope(rope, before[:, :hq], before[:, hq:hq + hk], pos, w, w, k_out=ko[:, :n].transpose(0, 1))
    assert torch.equal(ko[:, :n].transpose(0, 1), want[1]) and (ko[:, n:] == 7).all()
    # a row of zeros stays zero; a broadcast row is read
    z = torch.zeros(n, hq, D, dtype=torch.bfloat16, device=DEV)
    one = before[:1, :hk].expand(n, hk, D)
    zq, bk = pm.norm_rope(rope, z, one, pos, w, w)
    assert (zq == 0).all()
    assert torch.equal(bk, pm.norm_rope(rope, z, one.contiguous(), pos, w, w)[1])
    e = torch.empty(0, hq, D, dtype=torch.bfloat16, device=DEV)
    assert pm.norm_rope(rope, e, e[:, :hk], pos[:0])[0].shape == (0, hq, D)


# ---------------------------------------------------------------- write and read back

SHAPES = [  # kv_len, T, Hq, Hkv, D, page
    ([1], [1], 1, 1, 128, 16),
    ([17], [17], 4, 2, 128, 16),
    ([40, 3, 129], [40, 1, 128], 6, 3, 64, 32),
    ([130, 64, 200, 1], [2, 64, 77, 1], 8, 8, 128, 64),
    ([257, 128], [257, 5], 28, 4, 128, 128),
    ([300] * 3, [300] * 3, 2, 1, 64, 16),
]


@pytest.mark.parametrize("kv_len,T,Hq,Hkv,D,page", SHAPES)
@pytest.mark.parametrize("amp", [1.0, 1e-3, 3000.0])
def test_append_is_bit_exact_and_reads_back(pm, kv_len, T, Hq, Hkv, D, page, amp):
    s = Setup(pm, kv_len, T, Hq, Hkv, D, page)
    s.cache.buffer[:-256].fill_(0xA5)   # stale pages
    k, v = rows(11, s.n, Hkv, D, amp), rows(12, s.n, Hkv, D, amp)
    want = ref.Pages(s.n_pages, Hkv, D, page, s.raw())
    s.cache.append(s.batch, dev(k), dev(v))
    kq, vq = ref.quantise(k), ref.quantise(v)
    for b in range(len(T)):
        for j in range(T[b]):
            row, pos = s.start[b] + j, kv_len[b] - T[b] + j
            for side, (c, sc, z) in enumerate((kq, vq)):
                want.put(s.table[b, pos // page], pos % page, side, c[row], sc[row], z[row])
    assert np.array_equal(s.raw(), want.raw)
    ko, vo = s.cache.read(s.batch)
    assert np.array_equal(host(ko), ref.bf16_from_f32(ref.stand_for(*kq)))
    assert np.array_equal(host(vo), ref.bf16_from_f32(ref.stand_for(*vq)))
    over = max(np.abs(k).max(), np.abs(v).max()) > ref.LIMIT   # some outliers at the largest amplitude
    assert s.cache.read_error() == (pm.DEVERR_NONFINITE if over else 0)


def test_append_special_values(pm):
    D = 128
    s = Setup(pm, [8], [8], 1, 1, D, 16)
    k, v = rows(21, 8, 1, D), rows(22, 8, 1, D)
    k[0] = 0
    k[1] = 5.5                        # a group without a range
    k[2, 0, 3], k[3, 0, 40], v[4, 0, 70] = np.nan, np.inf, -np.inf
    v[5, 0, :4] = [3e38, -3e38, 1e-40, 0]
    v[6] = 1e-30
    s.cache.append(s.batch, dev(k), dev(v))
    ko, vo = s.cache.read(s.batch)
    assert np.array_equal(host(ko), ref.bf16_from_f32(ref.stand_for(*ref.quantise(k))))
    assert np.array_equal(host(vo), ref.bf16_from_f32(ref.stand_for(*ref.quantise(v))))
    assert s.cache.read_error() == pm.DEVERR_NONFINITE and s.cache.read_error() == 0


def test_padding_rows_and_rows_without_a_place(pm):
    D, Hkv, Hq = 64, 2, 4
    s = Setup(pm, [20, 5], [4, 6], Hq, Hkv, D, 16, pad=3)   # sequence 1: a row before position 0
    s.cache.buffer[:-256].fill_(0x11)
    k, v = dev(rows(31, s.n, Hkv, D)), dev(rows(32, s.n, Hkv, D))
    k[-3:], v[-3:] = float("nan"), float("inf")
    s.cache.append(s.batch, k, v)
    assert s.cache.read_error() == pm.DEVERR_BATCH
    out = [torch.full((s.n, Hkv, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    s.cache.read(s.batch, *out)
    for got, x in zip(out, (k, v)):
        want = ref.bf16_from_f32(ref.stand_for(*ref.quantise(host(x))))
        want[4] = 0
        want[-3:] = 9
        assert np.array_equal(host(got), want)
    assert s.cache.read_error() == pm.DEVERR_BATCH
    # a page outside the cache: skipped on write, zeros on read, the neighbour unharmed
    s.table[0, 1] = s.n_pages
    bad = s.make_batch(s.kv_len, s.start)
    pages = s.raw()
    s.cache.append(bad, k, v)
    assert s.cache.read_error() & pm.DEVERR_PAGE
    assert np.array_equal(s.raw(), pages)
    ko, _ = s.cache.read(bad)
    assert (ko[:4] == 0).all() and torch.equal(ko[5:10], out[0][5:10])


@pytest.mark.parametrize("kv_len,T,Hq,Hkv,D,page", SHAPES)
@pytest.mark.parametrize("weights", [True, False])
def test_append_qkv_equals_the_two_calls(pm, kv_len, T, Hq, Hkv, D, page, weights):
    a = Setup(pm, kv_len, T, Hq, Hkv, D, page, pad=2)
    b = Setup(pm, kv_len, T, Hq, Hkv, D, page, pad=2)
    qkv = dev(rows(41, a.n, Hq + 2 * Hkv, D))
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    rope = pm.Rope.make(D, rot_dim=D - 16, axes=axes_of(D - 16, 3))
    pos = torch.randint(0, 5000, (3, a.n), dtype=torch.int32, device=DEV)
    w = [dev(ref.bf16(1 + 0.2 * np.random.default_rng(i).standard_normal(D))) if weights else None for i in range(2)]
    qo = torch.full((a.n, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    a.cache.append_qkv(a.batch, rope, q, k, v, pos, *w, q_out=qo)
    q2, k2 = pm.norm_rope(rope, q, k, pos, *w)
    b.cache.append(b.batch, k2, v)
    n = int(a.start[-1])
    assert torch.equal(qo[:n], q2[:n]) and (qo[n:] == 3).all()
    assert np.array_equal(a.raw(), b.raw())
    # q in place in the projection
    a.cache.append_qkv(a.batch, rope, q, k, v, pos, *w, q_out=q)
    assert torch.equal(qkv[:n, :Hq], q2[:n]) and np.array_equal(a.raw(), b.raw())


# ---------------------------------------------------------------- attention

ATT = [  # kv_len, T, Hq, Hkv, D, page
    ([1], [1], 1, 1, 128, 16),
    ([2, 1, 16, 17, 31, 32, 33], [1] * 7, 4, 2, 128, 16),
    ([777], [1], 32, 8, 128, 16),
    ([777, 1500, 64], [1, 1, 1], 28, 4, 128, 32),
    ([513, 40, 1000], [1, 1, 1], 8, 1, 64, 64),
    ([300, 65, 129], [4, 4, 4], 8, 4, 128, 128),
    ([300, 65, 129, 7], [4, 1, 3, 7], 4, 4, 64, 16),
    ([100, 333], [5, 9], 28, 4, 128, 64),
    ([100, 333], [100, 17], 12, 4, 64, 32),
    ([400], [150], 16, 2, 128, 64),
    ([260, 31], [130, 31], 7, 1, 128, 16),
    ([129], [1], 64, 1, 128, 64),
    ([700, 12], [40, 0], 128, 1, 64, 128),
]


@pytest.mark.parametrize("kv_len,T,Hq,Hkv,D,page", ATT)
@pytest.mark.parametrize("amp", [1.0, 0.02])
def test_attention(pm, kv_len, T, Hq, Hkv, D, page, amp):
    s = Setup(pm, kv_len, T, Hq, Hkv, D, page)
    s.cache.buffer[:-256].fill_(0xFF)      # stale pages: NaN scales behind the sequences
    s.fill(51, amp)
    q = rows(53, s.n, Hq, D, 1.0 / amp ** 0.5)
    out = s.cache.attend(s.batch, dev(q))
    s.check_attention(q, out)
    assert torch.equal(out, s.cache.attend(s.batch, dev(q)))   # the same bits again
    assert s.cache.read_error() == 0


def test_attention_uniform_batch_equals_q_start(pm):
    for T in (1, 3, 40):
        s = Setup(pm, [90, 50, 200], [T] * 3, 8, 2, 128, 32)
        s.fill()
        q = dev(rows(61, s.n, 8, 128))
        u = s.make_batch(s.kv_len, s.start, uniform=True)
        assert torch.equal(s.cache.attend(u, q), s.cache.attend(s.batch, q))


@pytest.mark.parametrize("T", [[3, 8, 2], [40, 64, 2]])
def test_attention_rows_that_see_nothing_and_padding(pm, T):
    # sequence 0 is empty, sequence 1 holds fewer tokens than it has rows
    s = Setup(pm, [0, 5, 37], T, 8, 2, 128, 16, pad=4)
    s.fill()
    q = rows(63, s.n, 8, 128)
    q[-4:] = np.nan
    out = torch.full((s.n, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    s.cache.attend(s.batch, dev(q), out=out)
    s.check_attention(q, out)
    assert (out[:T[0]] == 0).all() and (out[T[0]:T[0] + T[1] - 5] == 0).all() and (out[-4:] == 5).all()


@pytest.mark.parametrize("T", [1, 4, 50])
def test_attention_strides_scale_and_no_workspace_content(pm, T):
    s = Setup(pm, [150, 70], [T, T], 8, 2, 128, 32, scale=0.03)
    s.fill()
    q = rows(64, s.n, 8, 128, 3.0)
    big = torch.zeros(s.n, 20, 128, dtype=torch.bfloat16, device=DEV)
    big[:, 3:11] = dev(q)
    hm = torch.zeros(8, s.n, 128, dtype=torch.bfloat16, device=DEV)      # head-major output
    ws = torch.full((pm.kv4_workspace_bytes(s.cfg, s.batch) + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    ws = ws[(-ws.data_ptr()) % 256:]
    s.cache.attend(s.batch, big[:, 3:11], out=hm.transpose(0, 1), workspace=ws)
    s.check_attention(q, hm.transpose(0, 1))
    assert torch.equal(hm.transpose(0, 1), s.cache.attend(s.batch, dev(q)))


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("kamp,vamp,qamp", [(1e-4, 1e-4, 1e4), (2000.0, 3000.0, 1e-3), (1.0, 1e-3, 1e-12),
                                            (1.0, 1.0, 30.0), (1.0, 20000.0, 1.0)])
def test_attention_magnitudes(pm, T, kamp, vamp, qamp):
    """Small and large keys, values and queries; peaked and flat softmax."""
    s = Setup(pm, [400, 90], [T, T], 4, 2, 128, 32)
    for b in range(2):
        n = s.kv_len[b]
        one = pm.KV4Batch(dev(np.array([n]), torch.int32), dev(s.table[b:b + 1], torch.int32), n_tokens=n)
        s.cache.append(one, dev(rows(71 + b, n, 2, 128, kamp)), dev(rows(73 + b, n, 2, 128, vamp)))
    q = rows(75, s.n, 4, 128, qamp)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))


@pytest.mark.parametrize("T", [1, 40])
def test_attention_growing_values_and_logits(pm, T):
    """Each token's values and logit are larger than the one's before: the reference moves often."""
    s = Setup(pm, [600], [T], 4, 1, 128, 64)
    r = np.random.default_rng(81)
    base = ref.bf16(r.standard_normal(128))
    grow = np.linspace(0.01, 6, 600)[:, None, None]
    k = ref.bf16(grow * base)
    v = ref.bf16(np.exp(np.linspace(-8, 8, 600))[:, None, None] * r.standard_normal((600, 1, 128)))
    one = pm.KV4Batch(s.batch.kv_len, s.batch.page_table, n_tokens=600)
    s.cache.append(one, dev(k), dev(v))
    q = np.tile(base, (T, 4, 1)).astype(np.float32)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))


@pytest.mark.parametrize("T", [2, 40])
def test_attention_nonfinite_query_stays_in_its_row(pm, T):
    s = Setup(pm, [90, 64], [T, T], 8, 2, 128, 16)
    s.fill()
    q = rows(91, s.n, 8, 128)
    clean = host(s.cache.attend(s.batch, dev(q)))
    q[1, 3, 7], q[T, 0, 0] = np.nan, np.inf
    got = host(s.cache.attend(s.batch, dev(q)))
    assert np.isnan(got[1, 3]).all() and np.isnan(got[T, 0]).any()
    keep = np.ones(got.shape[:2], bool)
    keep[1, 3] = keep[T, 0] = False
    assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 40])
def test_attention_bad_page_and_bad_lengths(pm, T):
    s = Setup(pm, [100, 100, 100], [T] * 3, 4, 2, 128, 32)
    s.fill()
    q = rows(92, s.n, 4, 128)
    good = s.cache.attend(s.batch, dev(q))
    page, s.table[1, 2] = s.table[1, 2], -5
    bad = s.make_batch(s.kv_len, s.start)
    got = s.cache.attend(bad, dev(q))
    assert s.cache.read_error() & pm.DEVERR_PAGE
    for b in (0, 2):
        assert torch.equal(got[s.start[b]:s.start[b + 1]], good[s.start[b]:s.start[b + 1]])
    s.table[1, 2] = page
    long = s.make_batch([100, 1 << 30, 100], s.start)       # longer than its page table
    got = s.cache.attend(long, dev(q))
    assert s.cache.read_error() & pm.DEVERR_BATCH
    assert torch.equal(got[:T], good[:T]) and torch.equal(got[2 * T:], good[2 * T:])
    out = torch.full_like(good, 2.0)
    wild = s.make_batch(s.kv_len, [0, 1 << 30, -7, 3 * T], max_q=T)
    s.cache.attend(wild, dev(q), out=out)
    assert s.cache.read_error() & pm.DEVERR_BATCH and (out == 2).all()
    s.cache.attend(s.make_batch(s.kv_len, s.start, max_q=T), dev(q), out=out)
    assert s.cache.read_error() == 0 and torch.equal(out, good)


def test_long_context_and_many_sequences(pm):
    """Split over many CTAs; more sequences than a warp, two CTA scans and empty ones between."""
    s = Setup(pm, [9000, 33], [1, 1], 8, 2, 64, 128)
    s.fill()
    q = rows(93, s.n, 8, 64)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))
    r = np.random.default_rng(94)
    lens = r.integers(0, 60, 300)
    T = np.minimum(r.integers(0, 3, 300), lens)
    s = Setup(pm, lens, T, 4, 2, 64, 16)
    s.fill()
    q = rows(95, s.n, 4, 64)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))
    k, _ = s.cache.read(s.batch)
    assert s.cache.read_error() == 0 and torch.isfinite(k).all()


# ---------------------------------------------------------------- together, streams, graphs

def test_decode_loop_equals_one_prefill(pm):
    """Tokens appended step by step, in chunks and as one prompt make the same cache, and each
    step's attention is the row of the whole prompt's attention."""
    D, Hq, Hkv, page, L = 128, 8, 2, 16, 75
    x = dev(rows(101, L, Hq + 2 * Hkv, D))
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    rope = pm.Rope.make(D)
    w = dev(np.ones(D, np.float32))
    one = Setup(pm, [L], [L], Hq, Hkv, D, page)
    pos = torch.arange(L, device=DEV, dtype=torch.int32)
    whole = one.cache.attend(one.batch, one.cache.append_qkv(one.batch, rope, q, k, v, pos, w, w))
    step = Setup(pm, [L], [1], Hq, Hkv, D, page)
    i = 0
    for T in [17, 1, 1, 1, 30, 1, 4, 1, 1, 1, 17]:
        b = pm.KV4Batch(dev(np.array([i + T]), torch.int32), step.batch.page_table, n_tokens=T)
        sl = slice(i, i + T)
        qs = step.cache.append_qkv(b, rope, q[sl], k[sl], v[sl], pos[sl].contiguous(), w, w)
        out = step.cache.attend(b, qs)
        # the same sums in another order and other fp16 operands: half a step of each result and
        # 2^-8 of the row's size for both roundings of weights and keys
        d = (out.float() - whole[sl].float()).abs()
        assert (d <= 2.0 ** -7 * whole[sl].float().abs() + 2.0 ** -7 * whole[sl].float().abs().amax(-1, True)).all()
        i += T
    assert i == L
    a, b = one.cache.read(one.batch), step.cache.read(pm.KV4Batch(step.batch.kv_len, step.batch.page_table, n_tokens=L))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 24])
def test_graph_replay_on_changing_lengths(pm, T):
    D, Hq, Hkv, page = 128, 8, 2, 32
    s = Setup(pm, [200, 200], [T, T], Hq, Hkv, D, page)
    kv_len = dev(np.array([60, 33]), torch.int32)
    batch = pm.KV4Batch(kv_len, s.batch.page_table, n_tokens=2 * T)
    x = torch.empty(2 * T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(2 * T, dtype=torch.int32, device=DEV)
    rope = pm.Rope.make(D)

    def step(cache, out=None):
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
        return cache.attend(batch, cache.append_qkv(batch, rope, q, k, v, pos), out=out)

    other = pm.KV4Cache(s.cfg, s.n_pages)
    graphs, outs = [], []
    x.copy_(dev(rows(0, 2 * T, Hq + 2 * Hkv, D)))
    step(s.cache)
    torch.cuda.synchronize()
    s.cache.reset()
    for _ in range(2):   # two graphs of the same call
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s.cache))
        graphs.append(g)
    for i in range(4):
        x.copy_(dev(rows(110 + i, 2 * T, Hq + 2 * Hkv, D)))
        pos.copy_(torch.arange(2 * T, device=DEV) + 7 * i)
        kv_len.copy_(dev(np.array([60 + T * i, 33 + T * i]), torch.int32))
        graphs[i % 2].replay()
        want = step(other)
        assert torch.equal(outs[i % 2], want), i
        assert torch.equal(s.cache.pages(), other.pages())


def test_two_streams_at_once(pm):
    sets = []
    for i in range(2):
        s = Setup(pm, [1500 + 100 * i] * 4, [1] * 4, 8, 2, 128, 64, seed=i)
        s.fill(120 + i)
        q = dev(rows(121 + i, s.n, 8, 128))
        sets.append((s, q, s.cache.attend(s.batch, q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, (s, q, _) in enumerate(sets):
            got[i].append(s.cache.attend(s.batch, q, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, _, want) in enumerate(sets):
        assert all(torch.equal(g, want) for g in got[i])


# ---------------------------------------------------------------- the mixed-precision cache's own path

def test_projected_prefill_and_steps_equal_the_separate_calls(pm):
    B, Hq, Hkv, L, D, steps = 2, 8, 2, 100, 128, 3
    G = Hq // Hkv
    x = dev(rows(131, B * (L + steps), Hq + 2 * Hkv, D)).view(B, L + steps, Hq + 2 * Hkv, D)
    w = [dev(ref.bf16(1 + 0.2 * np.random.default_rng(i).standard_normal(D))) for i in range(2)]
    rope = pm.Rope.make(D, axes=axes_of(D, 3))
    pos = torch.randint(0, 3000, (B, 3, L + steps), dtype=torch.int32, device=DEV)
    cfg = pm.Config.make(Hq, Hkv)
    a, b = (pm.PNMixCache(cfg, B, 128) for _ in range(2))
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    k_rot = a.prefill_projected(rope, q[:, :L], k[:, :L], v[:, :L], pos[:, :, :L].contiguous(), *w)
    flat = pos.transpose(0, 1).reshape(3, -1).contiguous()
    qr, kr = pm.norm_rope(rope, q.flatten(0, 1), k.flatten(0, 1), flat, *w)
    qr, kr = qr.view(B, L + steps, Hq, D), kr.view(B, L + steps, Hkv, D)
    hm = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
    b.prefill(hm(qr[:, L - 64:L]), hm(kr[:, :L]), hm(v[:, :L]), L)
    assert torch.equal(k_rot, hm(kr[:, :L])) and torch.equal(a.buffer, b.buffer)
    for i in range(L, L + steps):
        got = a.step_projected(rope, q[:, i], k[:, i], v[:, i], pos[:, :, i].t().contiguous(), *w)
        want = torch.empty(B, Hq, D, dtype=torch.float32, device=DEV)
        pm.pnmix_append_decode(cfg, kr[:, i].contiguous(), v[:, i].contiguous(), qr[:, i].contiguous(), b, want)
        assert torch.equal(got, want) and torch.equal(a.buffer, b.buffer)
    assert G * Hkv == Hq


def test_norm_rope_of_one_side(pm):
    n, D = 21, 128
    q, k = dev(rows(141, n, 3, D)), dev(rows(142, n, 2, D))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = pm.Rope.make(D)
    qo, ko = pm.norm_rope(rope, q, k, pos)
    assert torch.equal(pm.norm_rope(rope, q, None, pos)[0], qo) and torch.equal(pm.norm_rope(rope, None, k, pos)[1], ko)
    with pytest.raises(TypeError):
        pm.norm_rope(rope, None, None, pos)


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("Hq,T", [(8, 1), (8, 40), (8, 140)])
def test_a_staging_wait_that_runs_out_sets_the_error_bit(pm, Hq, T):
    """One row tile of 8 rows, one of 128 and two of 128: the call returns, and the next one is right."""
    import ctypes
    from decode_attention_prefill_b200 import kv4
    s = Setup(pm, [400, 300, 500], [T] * 3, Hq, 2, 128, 32)
    s.fill()
    q = dev(rows(151, s.n, Hq, 128))
    want = s.cache.attend(s.batch, q)
    out = torch.empty_like(q)
    ws = torch.empty(pm.kv4_workspace_bytes(s.cfg, s.batch), dtype=torch.uint8, device=DEV)
    shape, B = (s.n, Hq, 128), ctypes.byref
    st = pm._lib.pnmix_debug_kv4_stall(B(s.cfg), s.batch.ref, B(kv4._rows(q, shape, q.device, "q")), B(s.cache.c),
                                       B(kv4._rows(out, shape, q.device, "out")), ws.data_ptr(), ws.numel(), 1, 200,
                                       torch.cuda.current_stream().cuda_stream)
    assert st == pm.OK
    assert s.cache.read_error() & pm.DEVERR_TIMEOUT
    assert torch.equal(s.cache.attend(s.batch, q, workspace=ws), want) and s.cache.read_error() == 0


def test_quantiser_on_many_values(pm):
    """Bit-exact on a million values: offsets far above the range, ranges of a few bf16 steps,
    powers of two (exact half-way codes), tiny numbers and zeros."""
    r = np.random.default_rng(161)
    n, H, D = 2000, 2, 128
    x = r.standard_normal((n, H, D)) * np.exp(r.uniform(-12, 10, (n, H, 1))) + \
        r.choice([0, 1, -1, 30, -300, 20000], (n, H, 1)) * r.uniform(0.5, 2, (n, H, 1))
    x[::7] = r.integers(-40, 40, (len(x[::7]), H, D)) * 0.125
    x[1::11] *= 2.0 ** -30
    x[2::13, :, ::3] = 0
    x = ref.bf16(np.where(np.abs(x) > 61440, 0, x)) + np.float32(0)        # no negative zeros
    s = Setup(pm, [n], [n], 2, H, D, 64)
    s.cache.append(s.batch, dev(x), dev(x[:, :, ::-1]))
    k, v = s.cache.read(s.batch)
    assert np.array_equal(host(k), ref.bf16_from_f32(ref.stand_for(*ref.quantise(x))))
    assert np.array_equal(host(v), ref.bf16_from_f32(ref.stand_for(*ref.quantise(x[:, :, ::-1]))))
    want = ref.Pages(s.n_pages, H, D, 64, s.raw())
    for i in r.integers(0, n, 60):
        for side, y in enumerate((x, x[:, :, ::-1])):
            c, sc, z = ref.quantise(y[i])
            want.put(s.table[0, i // 64], i % 64, side, c, sc, z)
    assert np.array_equal(s.raw(), want.raw)


@pytest.mark.parametrize("D,Hq,Hkv,T,lens", [
    (128, 8, 2, 3, [5, 900, 17, 260]), (128, 8, 2, 9, [1000, 300, 9, 64]), (64, 12, 2, 30, [999, 30, 128, 511]),
    (128, 4, 4, 129, [129, 1290, 500]), (64, 4, 1, 70, [70, 640, 71]), (128, 8, 1, 257, [1500])])
def test_rows_of_both_tile_forms(pm, D, Hq, Hkv, T, lens):
    """8, 16, 128 and 256 rows per tile, tiles that end inside a token, units shared by CTAs."""
    s = Setup(pm, lens, [min(T, n) for n in lens], Hq, Hkv, D, 16)
    s.fill(171)
    q = rows(172, s.n, Hq, D)
    s.check_attention(q, s.cache.attend(s.batch, dev(q)))


def test_offsets_past_32_bits(pm):
    """Pages whose bytes lie more than 4 GiB behind the first."""
    D, Hq, Hkv, page = 128, 8, 8, 128
    cfg = pm.KV4Config.make(Hq, Hkv, D, page)
    n_pages = (5 << 30) // (Hkv * page * 20 * D // 16)
    cache = pm.KV4Cache(cfg, n_pages)
    table = np.array([[n_pages - 1, 3, n_pages - 2], [n_pages - 3, n_pages - 4, 0]], np.int32)
    lens = [300, 260]
    n = sum(lens)
    whole = pm.KV4Batch(dev(np.array(lens), torch.int32), dev(table, torch.int32),
                        dev(np.array([0, lens[0], n]), torch.int32), n_tokens=n)
    k, v = dev(rows(181, n, Hkv, D)), dev(rows(182, n, Hkv, D))
    cache.append(whole, k, v)
    ko, vo = cache.read(whole)
    assert np.array_equal(host(ko), ref.bf16_from_f32(ref.stand_for(*ref.quantise(host(k)))))
    assert np.array_equal(host(vo), ref.bf16_from_f32(ref.stand_for(*ref.quantise(host(v)))))
    small = pm.KV4Cache(cfg, 6)          # the same tokens in a small cache give the same bits
    near = pm.KV4Batch(whole.kv_len, dev(np.arange(6).reshape(2, 3), torch.int32), whole.q_start, n_tokens=n)
    small.append(near, k, v)
    for T in (1, 60):
        q = dev(rows(183, 2 * T, Hq, D))
        a = cache.attend(pm.KV4Batch(whole.kv_len, whole.page_table, n_tokens=2 * T), q)
        b = small.attend(pm.KV4Batch(whole.kv_len, near.page_table, n_tokens=2 * T), q)
        assert torch.equal(a, b)


def test_more_rows_than_max_q_is_an_error(pm):
    s = Setup(pm, [50, 60], [3, 7], 4, 2, 64, 16)
    s.fill()
    q = dev(rows(191, s.n, 4, 64))
    out = torch.full_like(q, 4.0)
    s.cache.attend(s.make_batch(s.kv_len, s.start, max_q=6), q, out=out)
    assert s.cache.read_error() == pm.DEVERR_BATCH and (out == 4).all()


def test_inputs_of_a_named_stream_may_be_dropped(pm):
    """Memory of tensors that another stream still reads is not handed out again."""
    s = Setup(pm, [3000] * 4, [1] * 4, 8, 2, 128, 64)
    s.fill()
    side = torch.cuda.Stream()
    q = rows(193, s.n, 8, 128)
    want = s.cache.attend(s.batch, dev(q))
    torch.cuda.synchronize()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        t = dev(q)
        side.wait_stream(torch.cuda.current_stream())
        out = s.cache.attend(s.batch, t, stream=side)
        del t
        torch.full((s.n, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        side.synchronize()
        assert torch.equal(out, want)


def test_the_same_workspace_in_two_graphs(pm):
    """Two graphs that were captured with one workspace, replayed in turn."""
    sets = []
    a = Setup(pm, [900, 400], [1, 1], 8, 2, 128, 32)
    b = Setup(pm, [300, 800], [30, 30], 8, 2, 128, 32, seed=3)
    need = max(pm.kv4_workspace_bytes(x.cfg, x.batch) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for s in (a, b):
        s.fill(195)
        q = dev(rows(196, s.n, 8, 128))
        want = s.cache.attend(s.batch, q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = s.cache.attend(s.batch, q, workspace=ws)
        sets.append((g, out, want, q))          # a replay reads q where it was captured
    for i in range(6):
        g, out, want, _ = sets[i % 2]
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("B,T", [(40, 1), (12, 20)])
def test_waits_of_one_round(pm, B, T):
    """Nearly every wait gives up at once, with copies in flight: the call returns, and the next
    ones are right."""
    import ctypes
    from decode_attention_prefill_b200 import kv4
    s = Setup(pm, [700 + 13 * i for i in range(B)], [T] * B, 8, 2, 128, 16)
    s.fill()
    q = dev(rows(211, s.n, 8, 128))
    want = s.cache.attend(s.batch, q)
    out = torch.empty_like(q)
    ws = torch.empty(pm.kv4_workspace_bytes(s.cfg, s.batch), dtype=torch.uint8, device=DEV)
    shape, ref_ = (s.n, 8, 128), ctypes.byref
    for seq in (0, B // 2, B - 1):
        st = pm._lib.pnmix_debug_kv4_stall(ref_(s.cfg), s.batch.ref, ref_(kv4._rows(q, shape, q.device, "q")),
                                           ref_(s.cache.c), ref_(kv4._rows(out, shape, q.device, "out")), ws.data_ptr(),
                                           ws.numel(), seq, 1, torch.cuda.current_stream().cuda_stream)
        assert st == pm.OK and s.cache.read_error() & pm.DEVERR_TIMEOUT
        assert torch.equal(s.cache.attend(s.batch, q, workspace=ws), want) and s.cache.read_error() == 0


def test_the_answer_does_not_depend_on_earlier_calls(pm):
    """The split of the work follows from the call: a first call with very many sequences (whose
    launch leaves less room on the GPU) changes no bit of a later one."""
    import os
    import subprocess
    import sys
    code = """
import sys, hashlib, torch
import decode_attention_prefill_b200 as pm
torch.manual_seed(5)
cfg = pm.KV4Config.make(16, 4, 128, 64)
cache = pm.KV4Cache(cfg, 400)
i32 = dict(dtype=torch.int32, device="cuda")
k = torch.randn(4 * 6400, 4, 128, device="cuda").bfloat16()
table = torch.arange(400, **i32).view(4, 100)
full = torch.full((4,), 6400, **i32)
cache.append(pm.KV4Batch(full, table, n_tokens=4 * 6400), k, k)
q = torch.randn(2048, 16, 128, device="cuda").bfloat16()
if sys.argv[1] == "many":
    cache.attend(pm.KV4Batch(torch.full((2048,), 64, **i32), table.view(-1)[:1].repeat(2048).view(2048, 1), n_tokens=2048), q)
out = cache.attend(pm.KV4Batch(full, table, n_tokens=4), q[:4].contiguous())
print(hashlib.sha256(out.cpu().view(torch.int16).numpy().tobytes()).hexdigest())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(pm.__file__)))
    got = [subprocess.run([sys.executable, "-c", code, how], cwd=root, capture_output=True, text=True, timeout=300)
           for how in ("many", "alone")]
    assert all(g.returncode == 0 for g in got), got
    assert got[0].stdout == got[1].stdout


def test_projected_calls_refuse_what_is_not_the_caches(pm):
    cache = pm.PNMixCache(pm.Config.make(8, 2), 2, 128)
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    rope, pos = pm.Rope.make(128), torch.zeros(2, 70, dtype=torch.int32, device=DEV)
    good = bf(2, 70, 8, 128), bf(2, 70, 2, 128), bf(2, 70, 2, 128)
    cache.prefill_projected(rope, *good, pos)
    step, at = (bf(2, 8, 128), bf(2, 2, 128), bf(2, 2, 128)), pos[:, 0].contiguous()
    cache.step_projected(rope, *step, at)
    before = cache.buffer.clone()
    for i, bad in [(0, bf(1, 70, 8, 128)), (0, bf(2, 70, 4, 128)), (1, bf(2, 69, 2, 128)), (2, bf(2, 70, 1, 128)),
                   (2, bf(2, 70, 2, 64)), (0, bf(70, 8, 128))]:
        with pytest.raises(ValueError):
            cache.prefill_projected(rope, *[bad if i == j else t for j, t in enumerate(good)], pos)
    for i, bad in [(0, bf(1, 8, 128)), (1, bf(2, 1, 128)), (2, bf(2, 2, 64)), (0, bf(2, 1, 8, 128))]:
        with pytest.raises(ValueError):
            cache.step_projected(rope, *[bad if i == j else t for j, t in enumerate(step)], at)
    with pytest.raises(TypeError):
        cache.step_projected(rope, step[0].float(), *step[1:], at)
    with pytest.raises(ValueError):
        cache.step_projected(rope, *step, at, out=torch.empty(1, 8, 128, device=DEV))
    with pytest.raises(ValueError):
        cache.step_projected(rope, *step, pos)
    assert torch.equal(cache.buffer, before)


def test_what_a_batch_and_a_cache_were_made_with_stays(pm):
    s = Setup(pm, [40], [2], 8, 2, 128, 16)
    s.fill()
    q = dev(rows(201, 2, 8, 128))
    want = s.cache.attend(s.batch, q)
    for name, value in (("n_tokens", 200), ("kv_len", q), ("page_table", None), ("q_start", None)):
        with pytest.raises(AttributeError):
            setattr(s.batch, name, value)
    s.cfg.n_q_heads, s.cfg.softmax_scale = 16, 9.0      # the caller's, no longer the cache's
    assert torch.equal(s.cache.attend(s.batch, q), want)
    with pytest.raises(pm.PNMixError):
        s.cache.attend(s.batch, q, out=q)
