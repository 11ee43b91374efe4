"""The 4-bit paged cache on the host: refusals before any launch, and the restatement's own
consistency."""
import ctypes

import numpy as np
import pytest
import torch

import decode_attention_prefill_b200 as pm
import kv4_ref as ref
from decode_attention_prefill_b200 import kv4

B = ctypes.byref
P = 1 << 41            # a device address that nothing looks at: every call here is refused

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers; runs only where no kernel "
                                                              "can launch")


def cache(cfg, n_pages=4):
    c = kv4._Cache()
    need = pm.kv4_cache_bytes(cfg, n_pages)
    assert pm._lib.pnmix_kv4_cache_init(B(cfg), n_pages, ctypes.c_void_p(1 << 40), need, B(c)) == pm.OK
    return c


def batch(**kw):
    d = dict(batch=2, n_tokens=6, max_pages=3, max_q=4, q_start=P, kv_len=P, page_table=P)
    d.update(kw)
    return kv4._Batch(*[d[k] for k, _ in kv4._Batch._fields_])


def rows(heads=8, D=128, data=P, ts=None, hs=None):
    return kv4._Rows(data, heads * D if ts is None else ts, D if hs is None else hs)


def test_cache_bytes_and_regions():
    for D in (64, 128):
        for page in (16, 32, 64, 128):
            cfg = pm.KV4Config.make(8, 2, D, page)
            assert pm.kv4_cache_bytes(cfg, 5) == 5 * 2 * page * 20 * D // 16 + 256
            c = cache(cfg, 5)
            assert c.error - c.pages == 5 * 2 * page * 20 * D // 16
    cfg = pm.KV4Config.make(8, 2)
    c, out = kv4._Cache(), ctypes.c_size_t(0)
    need = pm.kv4_cache_bytes(cfg, 4)
    init = pm._lib.pnmix_kv4_cache_init
    assert init(B(cfg), 4, ctypes.c_void_p((1 << 40) + 16), need, B(c)) == pm.ERR_ALIGNMENT
    assert init(B(cfg), 4, ctypes.c_void_p(1 << 40), need - 1, B(c)) == pm.ERR_CAPACITY
    assert init(B(cfg), 0, ctypes.c_void_p(1 << 40), need, B(c)) == pm.ERR_INVALID_ARG
    assert init(B(cfg), 4, None, need, B(c)) == pm.ERR_INVALID_ARG
    assert pm._lib.pnmix_kv4_cache_bytes(B(cfg), -1, B(out)) == pm.ERR_INVALID_ARG


@pytest.mark.parametrize("args,status", [
    (dict(n_q_heads=8, n_kv_heads=3), pm.ERR_INVALID_ARG), (dict(n_q_heads=0, n_kv_heads=1), pm.ERR_INVALID_ARG),
    (dict(n_q_heads=8, n_kv_heads=2, head_dim=96), pm.ERR_UNSUPPORTED),
    (dict(n_q_heads=8, n_kv_heads=2, page_tokens=48), pm.ERR_UNSUPPORTED),
    (dict(n_q_heads=258, n_kv_heads=2), pm.ERR_UNSUPPORTED), (dict(n_q_heads=8192, n_kv_heads=8192), pm.ERR_UNSUPPORTED),
    (dict(n_q_heads=8, n_kv_heads=2, softmax_scale=float("nan")), pm.ERR_INVALID_ARG),
    (dict(n_q_heads=8, n_kv_heads=2, softmax_scale=float("inf")), pm.ERR_INVALID_ARG)])
def test_config_refusals(args, status):
    out = ctypes.c_size_t(0)
    assert pm._lib.pnmix_kv4_cache_bytes(B(pm.KV4Config.make(**args)), 4, B(out)) == status
    assert pm._lib.pnmix_kv4_workspace_bytes(B(pm.KV4Config.make(**args)), B(batch())) == 0


BATCHES = [(dict(batch=0), pm.ERR_INVALID_ARG), (dict(n_tokens=-1), pm.ERR_INVALID_ARG),
           (dict(max_pages=0), pm.ERR_INVALID_ARG), (dict(kv_len=None), pm.ERR_INVALID_ARG),
           (dict(page_table=None), pm.ERR_INVALID_ARG), (dict(max_q=0), pm.ERR_INVALID_ARG),
           (dict(max_q=7), pm.ERR_INVALID_ARG), (dict(batch=2049), pm.ERR_UNSUPPORTED),
           (dict(max_pages=1 << 28), pm.ERR_UNSUPPORTED), (dict(n_tokens=1 << 28, max_q=9), pm.ERR_UNSUPPORTED),
           (dict(q_start=None, n_tokens=7), pm.ERR_INVALID_ARG),
           (dict(q_start=None, max_q=2), pm.ERR_INVALID_ARG),
           (dict(kv_len=P + 2), pm.ERR_ALIGNMENT), (dict(q_start=P + 1), pm.ERR_ALIGNMENT)]


@no_gpu
@pytest.mark.parametrize("change,status", BATCHES)
def test_batch_refusals(change, status):
    cfg = pm.KV4Config.make(8, 2)
    c, b, L = cache(cfg), batch(**change), pm._lib
    k, q = rows(2), rows(8)
    rope = pm.Rope.make(128)
    ws = ctypes.c_void_p(P)
    assert L.pnmix_kv4_append(B(cfg), B(b), B(k), B(k), B(c), None) == status
    assert L.pnmix_kv4_append_qkv(B(cfg), B(rope), B(b), B(q), B(k), B(k), None, None, P, B(q), B(c), None) == status
    assert L.pnmix_kv4_read(B(cfg), B(b), B(c), B(k), B(k), None) == status
    assert L.pnmix_kv4_attention(B(cfg), B(b), B(q), B(c), B(q), ws, 1 << 40, None) == status
    assert L.pnmix_kv4_workspace_bytes(B(cfg), B(b)) == 0


ROWS = [(dict(data=None), pm.ERR_INVALID_ARG), (dict(data=P + 8), pm.ERR_ALIGNMENT), (dict(ts=1028), pm.ERR_ALIGNMENT),
        (dict(hs=132), pm.ERR_ALIGNMENT), (dict(ts=-1024), pm.ERR_INVALID_ARG)]
WRITES = [(dict(ts=0), pm.ERR_INVALID_ARG), (dict(hs=64), pm.ERR_INVALID_ARG), (dict(ts=512), pm.ERR_INVALID_ARG)]


@no_gpu
@pytest.mark.parametrize("change,status", ROWS + WRITES)
def test_row_refusals(change, status):
    cfg = pm.KV4Config.make(8, 8)
    c, b, L = cache(cfg), batch(), pm._lib
    good, bad = rows(), rows(**change)
    rope = pm.Rope.make(128)
    ws = ctypes.c_void_p(P)
    big = 1 << 40
    writes = [L.pnmix_kv4_read(B(cfg), B(b), B(c), B(bad), B(good), None),
              L.pnmix_kv4_read(B(cfg), B(b), B(c), B(good), B(bad), None),
              L.pnmix_kv4_attention(B(cfg), B(b), B(good), B(c), B(bad), ws, big, None),
              L.pnmix_norm_rope(B(rope), 6, 8, 8, B(good), B(good), None, None, P, B(bad), B(good), None),
              L.pnmix_norm_rope(B(rope), 6, 8, 8, B(good), B(good), None, None, P, B(good), B(bad), None),
              L.pnmix_kv4_append_qkv(B(cfg), B(rope), B(b), B(good), B(good), B(good), None, None, P, B(bad), B(c), None)]
    assert writes == [status] * 6
    if (change, status) in WRITES:
        return
    reads = [L.pnmix_kv4_append(B(cfg), B(b), B(bad), B(good), B(c), None),
             L.pnmix_kv4_append(B(cfg), B(b), B(good), B(bad), B(c), None),
             L.pnmix_kv4_attention(B(cfg), B(b), B(bad), B(c), B(good), ws, big, None),
             L.pnmix_norm_rope(B(rope), 6, 8, 8, B(bad), B(good), None, None, P, B(good), B(good), None),
             L.pnmix_norm_rope(B(rope), 6, 8, 8, B(good), B(bad), None, None, P, B(good), B(good), None),
             L.pnmix_kv4_append_qkv(B(cfg), B(rope), B(b), B(good), B(bad), B(good), None, None, P, B(good), B(c), None)]
    assert reads == [status] * 6


@no_gpu
def test_workspace_cache_and_rope_refusals():
    cfg = pm.KV4Config.make(8, 2)
    c, b, L, q, k = cache(cfg), batch(), pm._lib, rows(8), rows(2)
    need = L.pnmix_kv4_workspace_bytes(B(cfg), B(b))
    assert need > 0
    att = lambda ws, n: L.pnmix_kv4_attention(B(cfg), B(b), B(q), B(c), B(q), ws, n, None)  # noqa: E731
    assert att(None, need) == pm.ERR_INVALID_ARG
    assert att(ctypes.c_void_p(P + 16), need) == pm.ERR_ALIGNMENT
    assert att(ctypes.c_void_p(P), need - 1) == pm.ERR_CAPACITY
    assert att(ctypes.c_void_p(P), need) == pm.ERR_INVALID_ARG          # the output is the query tensor
    stall = lambda seq, rounds: L.pnmix_debug_kv4_stall(B(cfg), B(b), B(q), B(c), B(q), ctypes.c_void_p(P), need, seq,  # noqa: E731
                                                        rounds, None)
    assert stall(-1, 5) == stall(2, 5) == stall(0, 0) == pm.ERR_INVALID_ARG
    other = cache(pm.KV4Config.make(8, 4))
    assert L.pnmix_kv4_append(B(cfg), B(b), B(k), B(k), B(other), None) == pm.ERR_INVALID_ARG
    assert L.pnmix_kv4_append(B(cfg), B(b), B(k), B(k), None, None) == pm.ERR_INVALID_ARG
    assert L.pnmix_kv4_cache_reset(None, None) == pm.ERR_INVALID_ARG
    rope = pm.Rope.make(64)      # not the cache's head size
    assert L.pnmix_kv4_append_qkv(B(cfg), B(rope), B(b), B(q), B(k), B(k), None, None, P, B(q), B(c), None) \
        == pm.ERR_INVALID_ARG

    def nr(rope, n=6, hq=8, hk=2, pos=P, w=None):
        return L.pnmix_norm_rope(B(rope), n, hq, hk, B(q), B(k), w, None, pos, B(q), B(k), None)
    good = pm.Rope.make(128)
    assert nr(good, pos=None) == pm.ERR_INVALID_ARG and nr(good, w=P + 2) == pm.ERR_ALIGNMENT
    assert nr(good, n=-1) == pm.ERR_INVALID_ARG and nr(good, hq=0, hk=0) == pm.ERR_INVALID_ARG
    assert nr(good, n=1 << 28) == pm.ERR_UNSUPPORTED
    assert nr(good, n=0, pos=None) == pm.OK              # nothing to do
    for change, status in [(dict(head_dim=96), pm.ERR_UNSUPPORTED), (dict(rot_dim=24), pm.ERR_UNSUPPORTED),
                           (dict(rot_dim=144), pm.ERR_UNSUPPORTED), (dict(n_axes=0), pm.ERR_UNSUPPORTED),
                           (dict(n_axes=5), pm.ERR_UNSUPPORTED), (dict(eps=-1.0), pm.ERR_INVALID_ARG),
                           (dict(eps=float("nan")), pm.ERR_INVALID_ARG)]:
        r = pm.Rope.make(128)
        for name, value in change.items():
            setattr(r, name, value)
        assert nr(r) == status, change
    r = pm.Rope.make(128)
    r.axis[5] = 1
    assert nr(r) == pm.ERR_INVALID_ARG
    r = pm.Rope.make(128)
    r.inv_freq[0] = float("inf")
    assert nr(r) == pm.ERR_INVALID_ARG


def test_python_refusals():
    with pytest.raises(ValueError):
        pm.Rope.make(128, 64, inv_freq=[1.0] * 20)
    with pytest.raises(ValueError):
        pm.Rope.make(128, axes=[0] * 63)
    with pytest.raises(ValueError):
        pm.Rope.make(64, axes=[4] * 32)
    with pytest.raises(TypeError):
        pm.KV4Batch(torch.ones(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32), n_tokens=2)
    with pytest.raises(TypeError):
        pm.norm_rope(pm.Rope.make(64), torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), torch.zeros(1, 1))
    with pytest.raises(pm.PNMixError):
        pm.kv4_cache_bytes(pm.KV4Config.make(8, 3), 4)


def test_python_refuses_other_structures():
    """The calls read what a structure's type promises, so another one is refused by type."""
    from types import SimpleNamespace
    cfg, x = pm.KV4Config.make(8, 2), torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="Rope"):
        pm.norm_rope(cfg, x, x, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(TypeError, match="KV4Config"):
        pm.KV4Cache(pm.Config.make(8, 2), 4)
    c = object.__new__(pm.KV4Cache)
    c.device, c._q, c._kv = torch.device("cuda", 0), (8, 128), (2, 128)
    with pytest.raises(TypeError, match="Rope"):
        c.append_qkv(None, cfg, x, x, x, None)
    with pytest.raises(TypeError, match="KV4Batch"):
        c._on(SimpleNamespace(device=c.device, n_tokens=1, ref=None), None)


# ---------------------------------------------------------------- the restatement itself

def test_layout_is_a_bijection_and_round_trips():
    for D in (64, 128):
        p = ref.Pages(2, 2, D, 32)
        for side in (0, 1):
            seen = {p._code(side, t, ch) for t in range(16) for ch in range(D)}
            lo = 10 * D * side
            assert len(seen) == 16 * D and {b for b, _ in seen} == set(range(lo, lo + 8 * D))
        r = np.random.default_rng(0)
        rows_ = r.standard_normal((32, 2, D)).astype(np.float32)
        c, s, z = ref.quantise(rows_)
        for t in range(32):
            p.put(1, t, t % 2, c[t], s[t], z[t])
        for t in range(32):
            assert np.array_equal(p.get(1, t, t % 2), ref.stand_for(c[t], s[t], z[t]))
        k, v, cs = ref.dequant_all(p.raw, D)
        assert np.array_equal(k[1, :, 4], ref.stand_for(c[4], s[4], z[4]).astype(np.float64).reshape(2, D)) or \
            np.allclose(k[1, :, 4], ref.stand_for(c[4], s[4], z[4]), rtol=2.0 ** -23)
        assert np.allclose(v[1, :, 5], ref.stand_for(c[5], s[5], z[5]), rtol=2.0 ** -23)


def test_quantiser_error_is_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 3, 128)).astype(np.float32) * 100
    c, s, z = ref.quantise(x)
    y = ref.stand_for(c, s, z).reshape(50, 3, 4, 32)
    step = s.astype(np.float32)[..., None]
    # half a step, the fp16 rounding of the zero point (2^-11 of it) and of the scale (15 * 2^-11)
    tol = step / 2 + np.abs(z.astype(np.float32))[..., None] * 2.0 ** -11 + step * 15 * 2.0 ** -11
    assert (np.abs(y - x.reshape(y.shape)) <= tol).all()
    assert ref.quantise(np.full((1, 1, 32), 7.0))[0].max() == 0


def test_bf16_rounding_of_the_restatement():
    x = np.random.default_rng(2).standard_normal(1000) * 10.0 ** np.arange(-30, 30).repeat(17)[:1000]
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    got = ref.bf16(x)
    # torch rounds through fp32: they differ where that is a tie at most
    assert (got != want).sum() <= 2
    f = x.astype(np.float32)
    assert np.array_equal(ref.bf16_from_f32(f), torch.from_numpy(f).to(torch.bfloat16).float().numpy())


# ---------------------------------------------------------------- the reference of a row's softmax

def compiled(tmp_path, body):
    """A C++ function over the arithmetic that the kernels share with the host."""
    import os
    import subprocess
    csrc = os.path.join(os.path.dirname(os.path.abspath(pm.__file__)), "csrc")
    src, so = tmp_path / "t.cpp", tmp_path / "t.so"
    src.write_text('#include "kv4_softmax.cuh"\nusing namespace pnmix::kv4;\n' + body)
    subprocess.run(["g++", "-O1", "-ffp-contract=off", "-std=c++17", "-shared", "-fPIC", "-I", csrc, str(src), "-o",
                    str(so)], check=True)
    return ctypes.CDLL(str(so))


COLUMNS = """
// Rows of n columns in steps of 32, as the many-row kernel takes them: weights, one move where a
// step's sum passes 2^15, the weights again.  Gives for each row the largest sum of a step behind
// its move, and the weights in the end, relative to the last reference.
extern "C" void rows32(const float* x, const float* fac, int rows, int n, float* worst, double* weight) {
  for (int r = 0; r < rows; ++r) {
    RowRef ref = {0.f, kFirstReference};
    worst[r] = 0.f;
    for (int c = 0; c < n; c += 32) {
      const float* at = x + (long)r * n + c;
      for (int turn = 0; turn < 2; ++turn) {
        float sum = 0.f, mx = -INFINITY;
        for (int k = 0; k < 32; ++k) {
          const float p = exp2f(fmaf(at[k] - ref.base, fac[r], -ref.ref));
          weight[(long)r * n + c + k] = p;
          sum += p;
          mx = fmaxf(mx, at[k]);
        }
        if (turn == 1 || !(sum > 32768.f)) {
          worst[r] = fmaxf(worst[r], sum);
          break;
        }
        const RowRef to = move_reference(ref, mx, fac[r]);
        const double f = exp2(move_exponent(ref, to, fac[r]));
        for (int k = 0; k < c; ++k) weight[(long)r * n + k] *= f;
        ref = to;
      }
    }
  }
}
"""


def run_rows(tmp_path, x, fac):
    lib = compiled(tmp_path, COLUMNS)
    x, fac = np.ascontiguousarray(x, np.float32), np.ascontiguousarray(fac, np.float32)
    worst, w = np.zeros(len(x), np.float32), np.zeros(x.shape, np.float64)
    P_ = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    lib.rows32(P_(x), P_(fac), ctypes.c_int(x.shape[0]), ctypes.c_int(x.shape[1]), P_(worst), P_(w))
    return worst, w


@pytest.mark.parametrize("log2", range(-10, 96, 5))
def test_one_move_of_the_reference_is_enough(tmp_path, log2):
    """Logits of any size up to 2^95: behind one move the 32 weights stay in range (a second move
    would change nothing), and the largest weight of the row does not vanish."""
    r = np.random.default_rng(300 + log2)
    rows_, n = 4000, 96
    fac = (1 + r.random(rows_)) * 2.0 ** r.integers(-20, 20, rows_)
    size = 2.0 ** log2 * (1 + r.random(rows_))
    x = r.standard_normal((rows_, n)) * r.choice([1, 1e-3, 1e-7], (rows_, 1)) + r.choice([-1, 0, 1], (rows_, 1))
    x = (x * (size / fac)[:, None]).astype(np.float32)
    worst, w = run_rows(tmp_path, x, fac)
    # 32 weights of at most 2^(2^-5) each where the row moved, else what was in range anyway
    assert np.isfinite(w).all() and (worst <= 32768).all()
    top = np.take_along_axis(w, x.argmax(1)[:, None], 1)[:, 0]
    assert (top >= 2.0 ** -1).all() and (w <= top[:, None] * (1 + 2.0 ** -20)).all()


def test_weights_of_moderate_logits_are_the_softmax(tmp_path):
    r = np.random.default_rng(41)
    x = (r.standard_normal((500, 192)) * r.uniform(0.1, 200, (500, 1))).astype(np.float32)
    fac = r.uniform(0.01, 2, 500).astype(np.float32)
    _, w = run_rows(tmp_path, x, fac)
    z = x.astype(np.float64) * fac[:, None].astype(np.float64)
    want = 2.0 ** (z - z.max(1, keepdims=True))
    want /= want.sum(1, keepdims=True)
    got = w / w.sum(1, keepdims=True)
    # exponents of up to 2^11 are off by 2^-14 of a bit at most, exp2f by a few 2^-24
    assert (np.abs(got - want) <= want * 2.0 ** -12 + 1e-30).all()


@pytest.mark.parametrize("log2", [100, 110, 120])
def test_a_row_whose_logits_are_all_very_low_keeps_its_weights(tmp_path, log2):
    r = np.random.default_rng(500 + log2)
    fac = (1 + r.random(1000)) * 2.0 ** r.integers(40, 60, 1000)
    x = (-(1 + r.random((1000, 96))) * (2.0 ** log2 / fac)[:, None]).astype(np.float32)
    worst, w = run_rows(tmp_path, x, fac)
    assert np.isfinite(w).all() and (worst <= 32768).all()
    assert (np.take_along_axis(w, x.argmax(1)[:, None], 1) >= 0.5).all()


@pytest.mark.parametrize("batch", [None, 3, object(), torch.zeros(1, dtype=torch.int32)])
def test_calls_refuse_what_is_no_batch_by_type(batch):
    c, x = object.__new__(pm.KV4Cache), torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    c.device, c._q, c._kv = torch.device("cuda", 0), (8, 128), (2, 128)
    rope = pm.Rope.make(128)
    for call in (lambda: c.append(batch, x, x), lambda: c.append_qkv(batch, rope, x, x, x, x), lambda: c.read(batch),
                 lambda: c.attend(batch, x)):
        with pytest.raises(TypeError, match="KV4Batch"):
            call()


@no_gpu
def test_outputs_over_other_tensors_are_refused():
    """The same memory for two outputs, or for an output and another tensor's input."""
    cfg = pm.KV4Config.make(8, 8)
    c, b, L, rope = cache(cfg), batch(), pm._lib, pm.Rope.make(128)
    w, x, y, z = (rows(data=P + (i << 30)) for i in range(4))
    assert L.pnmix_kv4_read(B(cfg), B(b), B(c), B(x), B(x), None) == pm.ERR_INVALID_ARG

    def nr(q, k, qo, ko):
        return L.pnmix_norm_rope(B(rope), 6, 8, 8, B(q), B(k), None, None, P, B(qo), B(ko), None)
    assert nr(w, x, y, y) == nr(w, x, x, y) == nr(w, x, y, w) == nr(w, x, x, w) == pm.ERR_INVALID_ARG
    for out in (x, y):
        assert L.pnmix_kv4_append_qkv(B(cfg), B(rope), B(b), B(w), B(x), B(y), None, None, P, B(out), B(c), None) \
            == pm.ERR_INVALID_ARG


@pytest.mark.parametrize("big", [(1 << 32) + 8, 1 << 31, -(1 << 32) + 8])
def test_sizes_past_32_bits_are_refused(big):
    """A C field would keep their low bits: 2^32 + 8 heads were 8."""
    good = dict(n_q_heads=8, n_kv_heads=8, head_dim=128, page_tokens=64)
    for name in good:
        with pytest.raises(ValueError, match=name):
            pm.KV4Config.make(**{**good, name: big})
    with pytest.raises(ValueError, match="n_pages"):
        pm.kv4_cache_bytes(pm.KV4Config.make(**good), big)
    with pytest.raises(ValueError, match="head_dim"):
        pm.Rope.make(big, 64)
    i32 = dict(dtype=torch.int32)
    for kw in (dict(n_tokens=big), dict(n_tokens=8, max_q=big)):
        with pytest.raises(ValueError, match=list(kw)[-1]):
            pm.KV4Batch(torch.ones(2, **i32), torch.zeros(2, 3, **i32), **kw)
