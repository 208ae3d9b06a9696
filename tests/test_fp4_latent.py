"""4-bit (E2M1) latent cache: the oracle's format against closed forms, the
refusals of the entry points (CPU), and on the GPU the quantising append and
the read back bit for bit, attention over selected blocks and over the whole
cache against 64-bit softmax attention of the dequantised rows, and the four
run together as a decoder uses them."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _gpu_helpers import bits_of, f64_of, need_gpu, to_dev_bf16

FAKE = 1 << 20  # an aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from conftest import build_lib
    build_lib()
    import long_context_decode_indexpool_b200 as m
    return m


# ---------------------------------------------------------------------------
# the format (CPU)
# ---------------------------------------------------------------------------
def test_e2m1_closed_forms():
    assert list(oracle.e2m1_value(np.arange(8))) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(oracle.e2m1_value(np.arange(8, 16)), -oracle.e2m1_value(np.arange(8)))
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, code in ties.items():
        assert oracle.e2m1_code(v) == code and oracle.e2m1_code(-v) == code + 8
        up = code if oracle.e2m1_value(code) > v else code + 1
        assert oracle.e2m1_code(np.nextafter(v, 9)) == up
        assert oracle.e2m1_code(np.nextafter(v, 0)) == up - 1
    assert [oracle.e2m1_code(float(v)) for v in oracle.e2m1_value(np.arange(16))] == list(range(16))
    assert oracle.e2m1_code(-0.0) == 8 and oracle.e2m1_code(1e300) == 7
    assert oracle.e2m1_code(float("-inf")) == 15


def test_latent_fp4_invariants():
    rng = np.random.default_rng(51)
    x = rng.standard_normal((64, 512)) * np.exp2(rng.integers(-9, 9, (64, 16))).repeat(32, 1)
    x *= np.exp2(rng.integers(-30, 30, (64, 1)))
    x[5] = 0.0
    x[6, 64:96] = 0.0
    bits = synth.f32_to_bf16_bits_np(x.astype(np.float32))
    x = oracle.bf16_to_f64(bits)
    codes, scales = oracle.latent_fp4(bits)
    v = oracle.dequant_fp4(codes, scales)
    e = scales.astype(np.int64) - 127
    amax = np.abs(x).reshape(64, 16, 32).max(-1)
    E = e.max(-1, keepdims=True)
    E[5] = -50
    assert (amax <= 6 * 2.0 ** e).all()
    assert (amax > 6 * 2.0 ** (e - 1))[(e > E - 15) & (amax > 0)].all()  # the smallest such exponent
    assert (e[amax == 0] == np.broadcast_to(E - 15, e.shape)[amax == 0]).all()
    # within half a step of the group's grid, whose widest step is 2 * 2^e
    assert (np.abs(v - x).reshape(64, 16, 32) <= 2.0 ** e[..., None]).all()
    # values on the grid are stored exactly
    g = rng.choice(oracle.e2m1_value(np.arange(16)), (64, 16, 32))
    g[..., 0] = 6.0
    step = np.exp2(rng.integers(-15, 1, (64, 16, 1)))
    step[:, 0] = 1.0  # the row's largest group
    g = (g * step).reshape(64, 512)
    assert np.array_equal(oracle.dequant_fp4(*oracle.latent_fp4(
        synth.f32_to_bf16_bits_np(g.astype(np.float32)))), g)


def test_latent_fp4_edges():
    nan, inf = float("nan"), float("inf")
    x = np.zeros((6, 512))
    x[0, :4] = [6.0, 0.25, -0.75, -0.1]
    x[0, 32] = 2.0 ** -40               # more than 2^15 below the row: the group's floor
    x[1, 0], x[1, 40] = nan, 3.0
    x[2, 0], x[2, 33] = -inf, 1.0
    x[3, 0] = 2.0 ** 100
    x[4, 0] = 2.0 ** -60
    x[5, :2] = [6.0625, 6.0]            # just above 6 * 2^0: exponent 1
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    v = oracle.dequant_fp4(codes, scales)
    assert list(scales[0, :3]) == [127, 112, 112] and list(v[0, :4]) == [6, 0, -1, 0]
    assert codes[0, 1] == 2 + 8 + (8 << 4) and v[0, 32] == 0
    assert scales[1, 0] == 255 and np.isnan(v[1, :32]).all() and v[1, 40] == 3.0
    assert v[2, 0] == -6 * 2.0 ** 50 and scales[2, 1] == 127 + 35
    assert v[3, 0] == 6 * 2.0 ** 50
    assert v[4, 0] == 2.0 ** -60 and scales[4, 0] == 127 - 62 and (scales[4, 1:] == 127 - 65).all()
    assert scales[5, 0] == 128 and v[5, 0] == 6.0


# ---------------------------------------------------------------------------
# refusals (CPU: every call returns before it launches anything)
# ---------------------------------------------------------------------------
def _status(lib, f, *a, **k):
    with pytest.raises(lib.SpxError) as e:
        f(*a, stream=0, **k)
    return e.value.status


def test_append_refusals(lib):
    f = lib.spx_latent_append_fp4
    ok = dict(B=2, latent=FAKE, n_new=4, n_add=None, codes=FAKE, scales=FAKE, cap_tok=64,
              len_dev=FAKE, max_len=64, stored=None)
    for key, val, status in (("B", 0, 2), ("B", 65536, 2), ("n_new", -1, 2), ("cap_tok", 0, 2),
                             ("max_len", 65, 2), ("max_len", -1, 2), ("n_new", 1 << 31, 2),
                             ("cap_tok", 1 << 31, 2),
                             ("latent", None, 1), ("codes", None, 1), ("scales", None, 1),
                             ("len_dev", None, 1), ("latent", FAKE + 8, 1), ("codes", FAKE + 8, 1),
                             ("scales", FAKE + 4, 1), ("len_dev", FAKE + 4, 1),
                             ("n_add", FAKE + 2, 1), ("stored", FAKE + 8, 1)):
        assert _status(lib, f, **{**ok, key: val}) == status, (key, val)
    f(**{**ok, "n_new": 0}, stream=0)  # nothing to write: no launch
    assert _status(lib, f, **{**ok, "B": 65535, "n_new": 1 << 20}) == 2


def test_read_refusals(lib):
    f = lib.spx_latent_read_fp4
    ok = dict(B=2, codes=FAKE, scales=FAKE, cap_tok=64, pos=FAKE, m=3, n_vis=FAKE, out=FAKE)
    for key, val, status in (("B", 0, 2), ("B", 65536, 2), ("m", -1, 2), ("m", 1 << 31, 2),
                             ("cap_tok", 0, 2), ("codes", None, 1), ("scales", None, 1),
                             ("n_vis", None, 1), ("out", None, 1), ("out", FAKE + 8, 1),
                             ("pos", FAKE + 4, 1), ("n_vis", FAKE + 4, 1), ("codes", FAKE + 4, 1)):
        assert _status(lib, f, **{**ok, key: val}) == status, (key, val)
    f(**{**ok, "m": 0}, stream=0)


def test_attention_refusals(lib):
    d = lib.dims(64, 1.0)
    need = lib.spx_attn_fp4_workspace_size(d, 4, 8192)
    ok = dict(d=d, rows=4, q=FAKE, codes=FAKE, scales=FAKE, seq_stride=8192 * 512, cap_tok=8192,
              idx=FAKE, count=FAKE, n_vis=FAKE, max_len=8192, out=FAKE, lse=FAKE, ws=FAKE,
              ws_bytes=need)
    for key, val, status in (("rows", 0, 2), ("rows", 65536, 2), ("max_len", -1, 2),
                             ("cap_tok", 0, 2), ("cap_tok", 1 << 31, 2), ("seq_stride", -512, 2),
                             ("seq_stride", 8191 * 512, 2), ("seq_stride", 8192 * 512 + 8, 2),
                             ("q", None, 1), ("codes", None, 1), ("scales", None, 1),
                             ("idx", None, 1), ("count", None, 1), ("n_vis", None, 1),
                             ("out", None, 1), ("q", FAKE + 8, 1), ("scales", FAKE + 8, 1),
                             ("lse", FAKE + 2, 1), ("idx", FAKE + 2, 1), ("n_vis", FAKE + 4, 1)):
        assert _status(lib, lib.spx_sparse_mla_attn_fp4, **{**ok, key: val}) == status, (key, val)
    if need:
        assert _status(lib, lib.spx_sparse_mla_attn_fp4, **{**ok, "ws_bytes": need - 1}) == 4
        assert _status(lib, lib.spx_sparse_mla_attn_fp4, **{**ok, "ws": None, "ws_bytes": 0}) == 4
    need = lib.spx_latent_attn_fp4_workspace_size(d, 6, 3, 8192)
    ok = dict(d=d, rows=6, rows_per_seq=3, q=FAKE, codes=FAKE, scales=FAKE, cap_tok=8192,
              n_vis=FAKE, max_len=8192, out=FAKE, lse=None, ws=FAKE, ws_bytes=need)
    for key, val, status in (("rows", 0, 2), ("rows", 7, 2), ("rows", 65536, 2),
                             ("rows_per_seq", 0, 2), ("rows_per_seq", 4, 2), ("max_len", -1, 2),
                             ("cap_tok", 0, 2), ("q", None, 1), ("codes", FAKE + 8, 1),
                             ("n_vis", None, 1), ("out", FAKE + 2, 1)):
        assert _status(lib, lib.spx_latent_attn_fp4, **{**ok, key: val}) == status, (key, val)
    if need:
        assert _status(lib, lib.spx_latent_attn_fp4, **{**ok, "ws_bytes": need - 1}) == 4
        assert _status(lib, lib.spx_latent_attn_fp4, **{**ok, "ws": FAKE + 8}) == 4
    for bad in ((0, 1, 64), (5, 2, 64), (4, 0, 64), (4, 1, -1)):
        with pytest.raises(lib.SpxError) as e:
            lib.spx_latent_attn_fp4_workspace_size(d, *bad)
        assert e.value.status == 2
    bad_d = lib.dims(64, 1.0)
    bad_d.latent = 256
    with pytest.raises(lib.SpxError) as e:
        lib.spx_attn_fp4_workspace_size(bad_d, 4, 64)
    assert e.value.status == 3


# ---------------------------------------------------------------------------
# append and read back (GPU)
# ---------------------------------------------------------------------------
def _wild_rows(rng, n):
    """Rows of every magnitude, with zeros, ties, infinities and NaN among them."""
    x = rng.standard_normal((n, 512)) * np.exp2(rng.integers(-70, 70, (n, 1)).astype(float))
    x *= np.exp2(rng.integers(-20, 1, (n, 16)).astype(float)).repeat(32, 1)
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    for i in range(0, n, 7):  # values on the grid and half-way between
        x[i] = rng.choice(grid, 512) * rng.choice([-1.0, 1.0], 512)
        x[i, ::32] = 6.0
    for i in range(3, n, 29):
        x[i] = rng.choice([0.0, -0.0], 512)
    for i in range(5, n, 31):
        x[i, rng.integers(0, 512, 2)] = np.nan
    for i in range(6, n, 37):
        x[i, rng.integers(0, 512, 2)] = [np.inf, -np.inf]
    return synth.f32_to_bf16_bits_np(np.clip(x, -3e38, 3e38).astype(np.float32)
                                     if not np.isinf(x).any() else x.astype(np.float32))


def _bf16_bits(v):
    return (v.astype(np.float32).view(np.uint32) >> np.uint32(16)).astype(np.uint16)


def _same_values(got_bits, ref_vals):
    """bf16 bits equal to the fp64 values, sign of zero included; NaN where the values are."""
    nan = np.isnan(ref_vals)
    got = oracle.bf16_to_f64(got_bits)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got_bits[~nan], _bf16_bits(ref_vals[~nan]))


@pytest.mark.gpu
@pytest.mark.parametrize("n_new,B", [(1, 5), (37, 3), (130, 1)])
@pytest.mark.parametrize("alias", [False, True])
def test_append_matches_oracle(n_new, B, alias):
    spx = need_gpu()
    rng = np.random.default_rng(100 + n_new)
    cap = n_new + 40
    bits = _wild_rows(rng, B * n_new).reshape(B, n_new, 512)
    lat = to_dev_bf16(bits)
    codes = torch.full((B, cap, 256), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((B, cap, 16), 0x5A, dtype=torch.uint8, device="cuda")
    lens = np.array([0, 7, 40, 39, 1][:B], dtype=np.int64)
    stored = lat if alias else torch.full_like(lat, 9.0)
    spx.spx_latent_append_fp4(B, lat, n_new, None, codes, scales, cap,
                              torch.from_numpy(lens).cuda(), cap, stored)
    gc, gs, gv = codes.cpu().numpy(), scales.cpu().numpy(), bits_of(stored)
    rc, rs = np.full((B, cap, 256), 0xA5, np.uint8), np.full((B, cap, 16), 0x5A, np.uint8)
    for b in range(B):
        c, s = oracle.latent_fp4(bits[b])
        rc[b, lens[b]:lens[b] + n_new], rs[b, lens[b]:lens[b] + n_new] = c, s
        _same_values(gv[b], oracle.dequant_fp4(c, s))
    assert np.array_equal(gs, rs)
    assert np.array_equal(gc, rc)


@pytest.mark.gpu
def test_append_padded_batch_and_bounds():
    spx = need_gpu()
    rng = np.random.default_rng(7)
    B, n_new, cap, max_len = 6, 9, 32, 30
    bits = _wild_rows(rng, B * n_new).reshape(B, n_new, 512)
    n_add = np.array([9, 0, 4, -3, 200, 9], np.int32)
    # the fifth sequence runs past max_len after 5 rows; the last has a length out of range
    lens = np.array([3, 3, 20, 0, 25, -1], np.int64)
    for bad in (-1, 31, 1 << 62):
        lens[5] = bad
        codes = torch.full((B, cap, 256), 1, dtype=torch.uint8, device="cuda")
        scales = torch.full((B, cap, 16), 2, dtype=torch.uint8, device="cuda")
        stored = torch.full((B, n_new, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        spx.spx_latent_append_fp4(B, to_dev_bf16(bits), n_new, torch.from_numpy(n_add).cuda(),
                                  codes, scales, cap, torch.from_numpy(lens).cuda(), max_len,
                                  stored)
        rc, rs = np.full((B, cap, 256), 1, np.uint8), np.full((B, cap, 16), 2, np.uint8)
        got = bits_of(stored)
        for b, k in enumerate([9, 0, 4, 0, 5, 0]):
            c, s = oracle.latent_fp4(bits[b, :k])
            if k:
                rc[b, lens[b]:lens[b] + k], rs[b, lens[b]:lens[b] + k] = c, s
                _same_values(got[b, :k], oracle.dequant_fp4(c, s))
            assert (got[b, k:] == 0x4040).all()  # 3.0: rows not written are left alone
        assert np.array_equal(codes.cpu().numpy(), rc)
        assert np.array_equal(scales.cpu().numpy(), rs)


@pytest.mark.gpu
@pytest.mark.parametrize("ragged", [False, True])
def test_append_and_read_many_rows(ragged):
    """Enough rows for the kernels' form of several rows a warp, a ragged number of them."""
    spx = need_gpu()
    rng = np.random.default_rng(9)
    B, n_new, cap = 7, 6001, 6011
    base = _wild_rows(rng, 997)
    pick = rng.integers(0, 997, (B, n_new))
    rc, rs = oracle.latent_fp4(base)
    vals = _bf16_bits(np.nan_to_num(oracle.dequant_fp4(rc, rs)))
    nan = np.isnan(oracle.dequant_fp4(rc, rs))
    lens = np.array([0, 10, 3, 5, 0, 7, 1], np.int64)
    n_add = np.array([6001, 0, 1, 6000, 4002, 4003, 5999], np.int32)
    k = n_add if ragged else np.full(B, n_new, np.int32)
    codes = torch.full((B, cap, 256), 1, dtype=torch.uint8, device="cuda")
    scales = torch.full((B, cap, 16), 2, dtype=torch.uint8, device="cuda")
    spx.spx_latent_append_fp4(B, to_dev_bf16(base[pick]), n_new,
                              torch.from_numpy(n_add).cuda() if ragged else None, codes, scales,
                              cap, torch.from_numpy(lens).cuda(), cap)
    gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
    for b in range(B):
        at = slice(lens[b], lens[b] + k[b])
        assert np.array_equal(gc[b, at], rc[pick[b, :k[b]]])
        assert np.array_equal(gs[b, at], rs[pick[b, :k[b]]])
        assert (gc[b, :lens[b]] == 1).all() and (gc[b, lens[b] + k[b]:] == 1).all()
    n_vis = torch.from_numpy(lens + k).cuda()
    pos = np.sort(rng.integers(0, cap, (B, n_new)), -1)
    for p in (None, torch.from_numpy(pos).cuda()):
        out = torch.full((B, n_new, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        spx.spx_latent_read_fp4(B, codes, scales, cap, p, n_new, n_vis, out)
        got = bits_of(out)
        for b in range(B):
            want = pos[b] if p is not None else np.arange(n_new)
            row = want - lens[b]
            mine = (row >= 0) & (row < k[b])
            src = pick[b, row[mine]]
            assert np.array_equal(got[b][mine][~nan[src]], vals[src][~nan[src]])
            assert np.isnan(oracle.bf16_to_f64(got[b][mine][nan[src]])).all()
            assert (got[b][want >= lens[b] + k[b]] == 0).all()


def _cache(rng, seqs, cap, lo=-3, hi=3):
    """A quantised cache of random rows (finite), as device arrays and values."""
    x = rng.standard_normal((seqs * cap, 512)) * np.exp2(rng.integers(lo, hi + 1, (seqs * cap, 1)))
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    codes, scales = codes.reshape(seqs, cap, 256), scales.reshape(seqs, cap, 16)
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
            oracle.dequant_fp4(codes, scales))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 33, 257])
def test_read_back(m):
    spx = need_gpu()
    rng = np.random.default_rng(m)
    B, cap = 3, 100
    codes, scales, vals = _cache(rng, B, cap)
    scales[1, 5, 3] = 255  # a NaN group
    scales[0, 6, 0] = 0    # the smallest scale, 2^-127
    vals = oracle.dequant_fp4(codes.cpu().numpy(), scales.cpu().numpy())
    n_vis = np.array([cap, 60, 500], np.int64)
    pos = rng.integers(0, cap, (B, m))
    pos[:, : m // 8] = pos[:, m // 8: 2 * (m // 8)]  # the same rows again
    pos[0, 0] = 6
    if m > 4:
        pos[1, :4] = [-1, 60, 5, 1 << 40]
        pos[2, 0] = cap  # inside n_vis, behind the cache's end
    out = torch.full((B, m, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    spx.spx_latent_read_fp4(B, codes, scales, cap, torch.from_numpy(pos).cuda(), m,
                            torch.from_numpy(n_vis).cuda(), out)
    got = bits_of(out)
    for b in range(B):
        for i in range(m):
            p = pos[b, i]
            _same_values(got[b, i], vals[b, p] if 0 <= p < min(n_vis[b], cap) else np.zeros(512))
    # no positions: the first m rows, zeros behind the sequence's end
    out.fill_(7.0)
    spx.spx_latent_read_fp4(B, codes, scales, cap, None, m, torch.from_numpy(n_vis).cuda(), out)
    got = bits_of(out)
    for b in range(B):
        for i in range(m):
            _same_values(got[b, i], vals[b, i] if i < min(n_vis[b], cap) else np.zeros(512))


# ---------------------------------------------------------------------------
# attention (GPU)
# ---------------------------------------------------------------------------
def _softmax64(q, c, scale):
    """q [H, 512], c [S, 512] -> out, lse, and the bounds' ingredients."""
    if c.shape[0] == 0:
        z = np.zeros((q.shape[0], 512))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0]), np.zeros((q.shape[0], 1))
    s = scale * (q @ c.T)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    w = p / l
    reach = scale * (np.abs(q) @ np.abs(c).T).max(-1)  # largest sum of |terms| of a logit
    top = (w * np.maximum(np.abs(c).max(-1), 2.0 ** -48)).max(-1, keepdims=True)
    return w @ c, (m + np.log(l))[:, 0], w @ np.abs(c), reach, top


def _check(got, got_lse, q, rows, scale, splits_tokens, what):
    """Bounds by arithmetic: a logit is a sum of 512 exact products in fp32, so off by at
    most 512 * 2^-23 * reach (a truncating adder counted), which moves each weight by that
    much relative and the normaliser too; a weight is rounded to fp16 (2^-11); the sums
    over a CTA's tokens run in fp32 in steps of 16 tokens; exp2 and log2 are good to
    2^-20; the output is rounded to bf16 once (2^-8).  Weights below fp16's normal range
    are off by at most 2^-25 in units where the largest w_t 2^E_t is 2^7 or more (E_t a
    row's exponent, or that of a row among its 8 neighbours, up to 4 larger): S of them,
    times values of at most 6 * 2^E_t <= 2^5 max |c_t|, are S * 2^-27 * max_t w_t max |c_t|
    (2^E >= 2^-50 stands in for a row of zeros).  Where several CTAs share a row, each
    one's part is rounded to fp16 once more, normalised by the sum of its w_t 2^E_t: 2^-11
    of a value no larger than the mass, or 2^-25 of that sum (its subnormals), in all
    2^-25 * S * 2^3 * max_t w_t max |c_t| by the same 2^E_t."""
    o, l, mass, reach, top = _softmax64(q, rows, scale)
    dz = 2.0 ** -14 * reach
    n_adds = splits_tokens / 16 + 64
    rel = 2 * dz[:, None] + 2 * 2.0 ** -11 + 2.0 ** -19 + n_adds * 2.0 ** -23
    tol = 2.0 ** -8 * (np.abs(o) + rel * mass) + rel * mass + 1e-38 \
        + rows.shape[0] * (2.0 ** -27 + 2.0 ** -22) * top
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (what, float(np.abs(got - o).max()), int(bad.sum()))
    if got_lse is not None:
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(got_lse), empty), what
        err = np.abs(got_lse[~empty] - l[~empty])
        assert (err <= dz[~empty] + 2.0 ** -19 + 2.0 ** -22 * np.abs(l[~empty])).all(), \
            (what, float(err.max()))


def _sparse_inputs(rng, n_vis, spoil=True):
    rows = len(n_vis)
    idx, cnt = np.full((rows, 512), -1, np.int32), np.zeros(rows, np.int32)
    for r, n in enumerate(n_vis):
        k = min(512, n // 4)
        sel = np.sort(rng.choice(n // 4, k, replace=False)) if k else np.zeros(0, int)
        idx[r, :k] = sel
        if spoil and k > 3:
            idx[r, 1], idx[r, 2] = n // 4 + 5, -3  # ids outside the row: skipped
        cnt[r] = k
    return idx, cnt


def _tokens(idx, cnt, n):
    sel = [int(b) for b in idx[:cnt] if 0 <= b < n // 4]
    return oracle.token_set(np.array(sel, np.int32), n)


def _run_sparse(spx, d, q, codes, scales, seq_stride, cap, idx, cnt, n_vis, max_len, ws=None):
    rows = q.shape[0]
    out = torch.full_like(q, 5.0)
    lse = torch.full((rows, d.heads), 5.0, device="cuda")
    if ws is None:
        ws = spx.workspace(spx.spx_attn_fp4_workspace_size(d, rows, max_len), "cuda")
        ws.fill_(0xFF)  # NaN patterns: a part that is read must have been written
    spx.spx_sparse_mla_attn_fp4(d, rows, q, codes, scales, seq_stride, cap, idx, cnt, n_vis,
                                max_len, out, lse, ws)
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 0
    return f64_of(out), lse.cpu().numpy().astype(np.float64)


SPARSE_LENS = [[1], [3, 4, 0, 5], [2051, 9001, 3, 2052, 0, 4, 700], [64, 65, 128, 257, 255]]


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 48, 64, 80, 128])
@pytest.mark.parametrize("lens", range(len(SPARSE_LENS)))
@pytest.mark.parametrize("shared", [False, True])
def test_sparse_attention(heads, lens, shared):
    spx = need_gpu()
    n_vis = SPARSE_LENS[lens]
    rng = np.random.default_rng(heads + 1000 * lens)
    rows, cap = len(n_vis), max(max(n_vis), 1)
    scale = 0.7
    d = spx.dims(heads, scale)
    codes, scales, vals = _cache(rng, 1 if shared else rows, cap)
    idx, cnt = _sparse_inputs(rng, n_vis)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((rows, heads, 512)) / 20).astype(np.float32))
    got, lse = _run_sparse(spx, d, to_dev_bf16(qb), codes, scales, 0 if shared else cap * 512, cap,
                           torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                           torch.tensor(n_vis, dtype=torch.int64, device="cuda"), cap)
    q = oracle.bf16_to_f64(qb)
    for r, n in enumerate(n_vis):
        c = vals[0 if shared else r][_tokens(idx[r], cnt[r], n)]
        _check(got[r], lse[r], q[r], c, scale, 2051, f"row {r} ({n} tokens)")
        if n == 0:
            assert (got[r] == 0).all()


@pytest.mark.gpu
def test_sparse_attention_odd_selections():
    """Ids in any order, the same block twice (its tokens count twice), counts
    below zero and above the row's blocks."""
    spx = need_gpu()
    rng = np.random.default_rng(31)
    heads, n = 48, 1203
    codes, scales, vals = _cache(rng, 1, n)
    idx = rng.integers(0, n // 4, (4, 512)).astype(np.int32)
    idx[0, :3] = 7
    cnt = np.array([200, 300, -5, 600], np.int32)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((4, heads, 512)) / 20).astype(np.float32))
    got, lse = _run_sparse(spx, spx.dims(heads, 1.0), to_dev_bf16(qb), codes, scales, 0, n,
                           torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                           torch.full((4,), n, dtype=torch.int64, device="cuda"), n)
    q = oracle.bf16_to_f64(qb)
    for r, k in enumerate([200, 300, 0, n // 4]):
        blocks = (4 * idx[r, :k, None] + np.arange(4)).reshape(-1)
        c = vals[0][np.concatenate([blocks, np.arange(n // 4 * 4, n)])]
        _check(got[r], lse[r], q[r], c, 1.0, 2051, f"row {r}")


@pytest.mark.gpu
def test_sparse_attention_many_rows():
    """A causal chunk on a shared cache: more rows than the device has SMs."""
    spx = need_gpu()
    rng = np.random.default_rng(3)
    T, n = 333, 2600
    d = spx.dims(64, 1.0)
    n_vis = list(range(n - T + 1, n + 1))
    codes, scales, vals = _cache(rng, 1, n)
    idx, cnt = _sparse_inputs(rng, n_vis)
    cnt[5], cnt[6], cnt[7] = 0, 9999, -4  # counts outside 0 .. 512 are clamped
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((T, 64, 512)) / 22).astype(np.float32))
    got, lse = _run_sparse(spx, d, to_dev_bf16(qb), codes, scales, 0, n,
                           torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                           torch.tensor(n_vis, dtype=torch.int64, device="cuda"), n)
    q = oracle.bf16_to_f64(qb)
    for r in range(T):
        k = min(max(int(cnt[r]), 0), 512)
        _check(got[r], lse[r], q[r], vals[0][_tokens(idx[r], k, n_vis[r])], 1.0, 2051, f"row {r}")


def _run_latent(spx, d, per, q, codes, scales, n_vis, max_len, ws=None, cap=None):
    rows = q.shape[0]
    out = torch.full_like(q, 5.0)
    lse = torch.full((rows, d.heads), 5.0, device="cuda")
    if ws is None:
        ws = spx.workspace(spx.spx_latent_attn_fp4_workspace_size(d, rows, per, max_len), "cuda")
        ws.fill_(0xFF)
    spx.spx_latent_attn_fp4(d, rows, per, q, codes, scales, cap or codes.shape[1], n_vis, max_len,
                            out, lse, ws)
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 0
    return f64_of(out), lse.cpu().numpy().astype(np.float64)


LATENT_CASES = [  # rows per sequence, lengths of the rows
    (1, [1]), (1, [0, 63, 64, 65]), (1, [1, 2000, 0, 129]), (2, [5, 6, 0, 1]),
    (3, [0, 0, 1, 500, 501, 502]), (4, [130, 7, 0, 129]), (7, [200 + i for i in range(7)]),
    (1, [5000]), (1, [3001, 17, 900]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("case", range(len(LATENT_CASES)))
def test_latent_attention(heads, case):
    spx = need_gpu()
    per, n_vis = LATENT_CASES[case]
    rng = np.random.default_rng(heads + 1000 * case)
    rows, cap = len(n_vis), max(max(n_vis), 1) + 3
    scale = 1.3
    d = spx.dims(heads, scale)
    codes, scales, vals = _cache(rng, rows // per, cap)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((rows, heads, 512)) / 25).astype(np.float32))
    got, lse = _run_latent(spx, d, per, to_dev_bf16(qb), codes, scales,
                           torch.tensor(n_vis, dtype=torch.int64, device="cuda"), cap)
    q = oracle.bf16_to_f64(qb)
    for r, n in enumerate(n_vis):
        _check(got[r], lse[r], q[r], vals[r // per][:n], scale, n, f"row {r} ({n} tokens)")
        if n == 0:
            assert (got[r] == 0).all()


@pytest.mark.gpu
def test_latent_attention_many_short_sequences():
    spx = need_gpu()
    rng = np.random.default_rng(17)
    rows, cap, heads = 613, 70, 16
    n_vis = rng.integers(0, cap + 1, rows)
    codes, scales, vals = _cache(rng, rows, cap)
    d = spx.dims(heads, 1.0)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((rows, heads, 512)) / 25).astype(np.float32))
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), codes, scales,
                           torch.from_numpy(n_vis).cuda(), cap)
    q = oracle.bf16_to_f64(qb)
    for r in range(rows):
        _check(got[r], lse[r], q[r], vals[r][:n_vis[r]], 1.0, cap, f"row {r}")


@pytest.mark.gpu
def test_more_units_than_threads():
    """Many rows of two head groups and of unequal lengths, some of them empty."""
    spx = need_gpu()
    rng = np.random.default_rng(27)
    seqs, per, cap, heads = 300, 3, 200, 80
    n_vis = rng.integers(0, cap + 1, seqs * per)
    n_vis[rng.integers(0, seqs * per, 40)] = 0
    codes, scales, vals = _cache(rng, seqs, cap)
    d = spx.dims(heads, 0.9)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((seqs * per, heads, 512)) / 25)
                                   .astype(np.float32))
    got, lse = _run_latent(spx, d, per, to_dev_bf16(qb), codes, scales,
                           torch.from_numpy(n_vis).cuda(), cap)
    q = oracle.bf16_to_f64(qb)
    for r in range(seqs * per):
        _check(got[r], lse[r], q[r], vals[r // per][:n_vis[r]], 0.9, cap, f"row {r}")


@pytest.mark.gpu
def test_latent_attention_lengths_out_of_range():
    """Lengths are clamped to [0, min(max_len, cap_tok)]."""
    spx = need_gpu()
    rng = np.random.default_rng(18)
    d = spx.dims(32, 1.0)
    codes, scales, vals = _cache(rng, 4, 50)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((4, 32, 512)) / 25).astype(np.float32))
    q = oracle.bf16_to_f64(qb)
    n_vis = torch.tensor([-5, 1 << 40, 49, 45], dtype=torch.int64, device="cuda")
    for max_len, seen in ((1000, [0, 50, 49, 45]), (47, [0, 47, 47, 45]), (0, [0, 0, 0, 0])):
        got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), codes, scales, n_vis, max_len)
        for r in range(4):
            _check(got[r], lse[r], q[r], vals[r][:seen[r]], 1.0, 50, f"row {r}, {max_len}")


@pytest.mark.gpu
def test_attention_of_rows_far_apart():
    """Row exponents 2^100 apart, groups 2^15 apart within a row, one-hot
    softmaxes, zero rows, zero queries and queries of extreme size."""
    spx = need_gpu()
    rng = np.random.default_rng(19)
    heads, n = 32, 150
    x = rng.standard_normal((n, 512)) * np.exp2(rng.integers(-15, 1, (n, 16))).repeat(32, 1)
    x[:20] *= 2.0 ** -48      # rows far below the others
    x[20:23] = 0.0
    x[23:26] *= 2.0 ** 12
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    vals = oracle.dequant_fp4(codes, scales)
    q = rng.standard_normal((3, heads, 512)) / 25
    q[0, 0] = 0.0
    q[0, 1] *= 2.0 ** -60
    q[0, 2] *= np.exp2(rng.integers(-30, 1, 512))
    q[0, 3] *= 40.0            # a sharp softmax
    q[1] *= 2.0 ** -13
    qb = synth.f32_to_bf16_bits_np(q.astype(np.float32))
    q = oracle.bf16_to_f64(qb)
    d = spx.dims(heads, 1.0)
    n_vis = [n, n - 1, 23]
    got, lse = _run_latent(spx, d, 3, to_dev_bf16(qb), torch.from_numpy(codes)[None].cuda(),
                           torch.from_numpy(scales)[None].cuda(),
                           torch.tensor(n_vis, dtype=torch.int64, device="cuda"), n)
    for r in range(3):
        _check(got[r], lse[r], q[r], vals[:n_vis[r]], 1.0, n, f"row {r}")
    # a cache whose rows differ by 2^100 but hardly matter to the logits
    x = rng.standard_normal((60, 512))
    x[:30] *= 2.0 ** 49
    x[30:] *= 2.0 ** -49
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    vals = oracle.dequant_fp4(codes, scales)
    qb = synth.f32_to_bf16_bits_np((q[:1] * 2.0 ** -52).astype(np.float32))
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), torch.from_numpy(codes)[None].cuda(),
                           torch.from_numpy(scales)[None].cuda(),
                           torch.tensor([60], dtype=torch.int64, device="cuda"), 60)
    _check(got[0], lse[0], oracle.bf16_to_f64(qb)[0], vals, 1.0, 60, "2^100")


@pytest.mark.gpu
def test_attention_ignores_what_no_row_sees():
    """Rows behind a sequence's end and blocks that are not selected may hold
    anything: NaN groups, any code, any scale byte."""
    spx = need_gpu()
    rng = np.random.default_rng(20)
    heads, cap, n = 64, 400, 301
    codes, scales, vals = _cache(rng, 2, cap)
    codes[:, n:], scales[:, n:] = 0xFF, 255
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((2, heads, 512)) / 25).astype(np.float32))
    q = oracle.bf16_to_f64(qb)
    d = spx.dims(heads, 1.0)
    n_vis = torch.tensor([n, n - 2], dtype=torch.int64, device="cuda")
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), codes, scales, n_vis, cap)
    for r in range(2):
        _check(got[r], lse[r], q[r], vals[r][:n - 2 * r], 1.0, n, f"row {r}")
    scales[:, 40:48] = 255  # two blocks that no row selects
    idx, cnt = np.full((2, 512), -1, np.int32), np.array([60, 60], np.int32)
    idx[:, :60] = np.delete(np.arange(75), [10, 11])[:60]
    got, lse = _run_sparse(spx, d, to_dev_bf16(qb), codes, scales, cap * 512, cap,
                           torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(), n_vis, cap)
    for r in range(2):
        nn = n - 2 * r
        _check(got[r], lse[r], q[r], vals[r][_tokens(idx[r], 60, nn)], 1.0, n, f"row {r}")


@pytest.mark.gpu
def test_attention_propagates_nan():
    """A visible NaN group makes the rows that see it NaN, and no others."""
    spx = need_gpu()
    rng = np.random.default_rng(21)
    codes, scales, vals = _cache(rng, 2, 130)
    scales[1, 100, 3] = 255
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((2, 64, 512)) / 25).astype(np.float32))
    d = spx.dims(64, 1.0)
    n_vis = torch.tensor([130, 130], dtype=torch.int64, device="cuda")
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), codes, scales, n_vis, 130)
    _check(got[0], lse[0], oracle.bf16_to_f64(qb)[0], vals[0], 1.0, 130, "row 0")
    assert np.isnan(got[1]).all() and np.isnan(lse[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("lens", [(100, 101, 102, 103), (63, 64, 65, 130), (1, 0, 3, 200)])
def test_nan_seen_by_the_later_rows_of_a_sequence_only(heads, lens):
    """Rows of a sequence that see different lengths: a NaN group (or a row of
    them) behind a row's length does not reach its output."""
    spx = need_gpu()
    rng = np.random.default_rng(22)
    n = max(lens)
    codes, scales, vals = _cache(rng, 1, n)
    scales[0, sorted(lens)[-2], 3] = 255  # the row of the most tokens sees both
    scales[0, n - 1] = 255
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((4, heads, 512)) / 25).astype(np.float32))
    d = spx.dims(heads, 1.0)
    got, lse = _run_latent(spx, d, 4, to_dev_bf16(qb), codes, scales,
                           torch.tensor(lens, dtype=torch.int64, device="cuda"), n)
    for r in range(4):
        if lens[r] == n:
            assert np.isnan(got[r]).all() and np.isnan(lse[r]).all()
        else:
            _check(got[r], lse[r], oracle.bf16_to_f64(qb)[r], vals[0][:lens[r]], 1.0, n, f"row {r}")


@pytest.mark.gpu
def test_lse_is_optional_and_calls_repeat_bit_for_bit():
    spx = need_gpu()
    rng = np.random.default_rng(22)
    d = spx.dims(64, 1.0)
    codes, scales, _ = _cache(rng, 2, 1500)
    q = to_dev_bf16(synth.f32_to_bf16_bits_np((rng.standard_normal((2, 64, 512)) / 25)
                                              .astype(np.float32)))
    n_vis = torch.tensor([1500, 777], dtype=torch.int64, device="cuda")
    ws = spx.workspace(spx.spx_latent_attn_fp4_workspace_size(d, 2, 1, 1500), "cuda")
    outs = []
    for i in range(3):
        out = torch.empty_like(q)
        lse = torch.empty(2, 64, device="cuda") if i else None
        spx.spx_latent_attn_fp4(d, 2, 1, q, codes, scales, 1500, n_vis, 1500, out, lse, ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.gpu
def test_streams_and_graphs():
    """Two calls at once on streams of their own, and a captured call replayed
    with new lengths, queries and cache contents."""
    spx = need_gpu()
    rng = np.random.default_rng(23)
    d = spx.dims(16, 1.0)
    cap = 900
    codes, scales, vals = _cache(rng, 2, cap)
    mk = lambda: synth.f32_to_bf16_bits_np(  # noqa: E731
        (rng.standard_normal((2, 16, 512)) / 25).astype(np.float32))
    qb = [mk(), mk()]
    q = [to_dev_bf16(b) for b in qb]
    need = spx.spx_latent_attn_fp4_workspace_size(d, 2, 1, cap)
    ws = [spx.workspace(need, "cuda") for _ in range(2)]
    out = [torch.zeros_like(t) for t in q]
    n_vis = torch.tensor([900, 450], dtype=torch.int64, device="cuda")
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            spx.spx_latent_attn_fp4(d, 2, 1, q[i], codes, scales, cap, n_vis, cap, out[i], None,
                                    ws[i], stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        for r, n in enumerate((900, 450)):
            _check(f64_of(out[i])[r], None, oracle.bf16_to_f64(qb[i])[r], vals[r][:n], 1.0, n,
                   "stream")
    g = torch.cuda.CUDAGraph()
    pos = torch.tensor([[3, 4, 5], [1, 1, 899]], device="cuda")
    back = torch.zeros(2, 3, 512, dtype=torch.bfloat16, device="cuda")
    new = to_dev_bf16(synth.f32_to_bf16_bits_np(rng.standard_normal((2, 1, 512)).astype(np.float32)))
    lens = torch.tensor([898, 440], dtype=torch.int64, device="cuda")
    with torch.cuda.graph(g):
        spx.spx_latent_append_fp4(2, new, 1, None, codes, scales, cap, lens, cap)
        spx.spx_latent_read_fp4(2, codes, scales, cap, pos, 3, n_vis, back)
        spx.spx_latent_attn_fp4(d, 2, 1, q[0], codes, scales, cap, n_vis, cap, out[0], None, ws[0])
    for step in range(3):
        nb = synth.f32_to_bf16_bits_np(rng.standard_normal((2, 1, 512)).astype(np.float32))
        qn = mk()
        new.copy_(to_dev_bf16(nb))
        q[0].copy_(to_dev_bf16(qn))
        nv = [899 - step, 441 + 3 * step]
        n_vis.copy_(torch.tensor(nv))
        lens.copy_(torch.tensor([v - 1 for v in nv]))
        g.replay()
        torch.cuda.synchronize()
        vals = oracle.dequant_fp4(codes.cpu().numpy(), scales.cpu().numpy())
        for r in range(2):
            c, s = oracle.latent_fp4(nb[r])
            assert np.array_equal(vals[r, nv[r] - 1], oracle.dequant_fp4(c, s)[0])
            _check(f64_of(out[0])[r], None, oracle.bf16_to_f64(qn)[r], vals[r][:nv[r]], 1.0, 900,
                   "graph")
            for i in range(3):
                p = int(pos[r, i])
                _same_values(bits_of(back)[r, i], vals[r, p] if p < nv[r] else np.zeros(512))


@pytest.mark.gpu
def test_pinned_host_cache():
    spx = need_gpu()
    rng = np.random.default_rng(24)
    d = spx.dims(16, 1.0)
    codes, scales, vals = _cache(rng, 1, 260)
    hc, hs = codes.cpu().pin_memory(), scales.cpu().pin_memory()
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((1, 16, 512)) / 25).astype(np.float32))
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), hc, hs,
                           torch.tensor([259], dtype=torch.int64, device="cuda"), 260)
    _check(got[0], lse[0], oracle.bf16_to_f64(qb)[0], vals[0][:259], 1.0, 260, "host")


@pytest.mark.gpu
@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """A cache whose codes pass 2^31 bytes: append, read back and attend at its end."""
    spx = need_gpu()
    rng = np.random.default_rng(25)
    cap = 9_000_000  # 2.3 GB of codes
    codes = torch.zeros(1, cap, 256, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, cap, 16), 127, dtype=torch.uint8, device="cuda")
    xb = synth.f32_to_bf16_bits_np(rng.standard_normal((1, 40, 512)).astype(np.float32))
    n = cap - 3
    spx.spx_latent_append_fp4(1, to_dev_bf16(xb), 40, None, codes, scales, cap,
                              torch.tensor([n - 40], device="cuda"), cap)
    c, s = oracle.latent_fp4(xb[0])
    vals = oracle.dequant_fp4(c, s)
    n_vis = torch.tensor([n], dtype=torch.int64, device="cuda")
    pos = torch.arange(n - 41, n + 1, device="cuda")[None].contiguous()
    out = torch.empty(1, 42, 512, dtype=torch.bfloat16, device="cuda")
    spx.spx_latent_read_fp4(1, codes, scales, cap, pos, 42, n_vis, out)
    _same_values(bits_of(out)[0, 1:41], vals)
    assert not out[0, 0].any() and not out[0, 41].any()
    d = spx.dims(16, 1.0)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((1, 16, 512)) / 2).astype(np.float32))
    q = oracle.bf16_to_f64(qb)[0]
    idx = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
    blocks = np.arange((n - 40) // 4 + 1, n // 4)
    idx[0, :blocks.size] = torch.from_numpy(blocks.astype(np.int32)).cuda()
    cnt = torch.tensor([blocks.size], dtype=torch.int32, device="cuda")
    got, lse = _run_sparse(spx, d, to_dev_bf16(qb), codes, scales, 0, cap, idx, cnt, n_vis, cap)
    first = blocks[0] * 4 - (n - 40)
    _check(got[0], lse[0], q, vals[first:], 1.0, 2051, "sparse")
    # every token: n - 40 zero rows (logit 0) beside the 40
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), codes, scales, n_vis, cap)
    z = q @ vals.T
    m = np.maximum(z.max(-1), 0.0)
    w = np.exp(z - m[:, None])
    tot = w.sum(-1) + (n - 40) * np.exp(-m)
    ref = (w @ vals) / tot[:, None]
    dz = 2.0 ** -14 * (np.abs(q) @ np.abs(vals).T).max(-1)
    rel = 2 * dz[:, None] + 2 * 2.0 ** -11 + 2.0 ** -19 + (n / 148 / 16 + 64) * 2.0 ** -23
    mass = (w @ np.abs(vals)) / tot[:, None]
    # (only the 40 rows have values: the zero rows' weights multiply zeros)
    top = (w * np.abs(vals).max(-1)).max(-1, keepdims=True) / tot[:, None]
    tol = 2.0 ** -8 * (np.abs(ref) + rel * mass) + rel * mass + 40 * 2.0 ** -27 * top
    # fp16 subnormals of a part: 2^-25 of its weights' sum in units of 2^E (E = 1 at most here)
    tol = tol + 2.0 ** -25 * 2.0
    assert (np.abs(got[0] - ref) <= tol).all()
    # fp32 sums of up to 61,000 tokens a CTA in steps of a 64-token tile
    assert (np.abs(lse[0] - (m + np.log(tot))) <= dz + 2.0 ** -19 + 2.0 ** -12).all()


# ---------------------------------------------------------------------------
# together, as a decoder runs them (GPU)
# ---------------------------------------------------------------------------
@pytest.mark.gpu
def test_prefill_then_decode_over_the_cache():
    """A prompt of each sequence is written to the indexer's and the 4-bit
    cache; then every step appends a token to both, selects blocks with the
    indexer, attends to the selection and (as a dense layer would) to all of
    the cache, and reads the new row back."""
    spx = need_gpu()
    rng = np.random.default_rng(26)
    B, H, cap, scale = 2, 64, 2600, 1.0
    lens = np.array([2400, 31], np.int64)
    T = int(lens.max())
    d = spx.dims(H, scale)
    wp = spx.pool_weights([0.5, 0.25, 0.125, 0.125])
    keys = rng.integers(-8, 9, (B, cap, 128)).astype(np.float32)
    lat = synth.f32_to_bf16_bits_np(rng.standard_normal((B, cap, 512)).astype(np.float32))
    keyb = synth.f32_to_bf16_bits_np(keys)
    dev = "cuda"
    codes = torch.zeros(B, cap, 256, dtype=torch.uint8, device=dev)
    scales = torch.zeros(B, cap, 16, dtype=torch.uint8, device=dev)
    zero = torch.zeros(B, dtype=torch.int64, device=dev)
    spx.spx_latent_append_fp4(B, to_dev_bf16(lat[:, :T]), T, torch.from_numpy(lens).int().cuda(),
                              codes, scales, cap, zero, cap)
    tail = torch.zeros(B, 3, 128, dtype=torch.bfloat16, device=dev)
    pooled = torch.zeros(B, cap // 4, 128, dtype=torch.bfloat16, device=dev)
    for b in range(B):  # prompts of unequal lengths: one call a sequence
        spx.spx_pool_append(d, 1, to_dev_bf16(keyb[b, :lens[b]]), int(lens[b]), wp, tail[b],
                            pooled[b], cap // 4, zero, cap)
    len_dev = torch.from_numpy(lens.copy()).cuda()
    scores = torch.zeros(B, cap // 4, device=dev)
    idx = torch.zeros(B, 512, dtype=torch.int32, device=dev)
    cnt = torch.zeros(B, dtype=torch.int32, device=dev)
    tws = spx.workspace(spx.spx_topk_workspace_size(d, B, cap), dev)
    for step in range(5):
        at = lens + step
        rows = np.arange(B)
        qi = rng.integers(-4, 5, (B, 32, 128)).astype(np.float32)
        wh = rng.choice([0.25, 0.5, 1.0], (B, 32)).astype(np.float32)
        qb = synth.f32_to_bf16_bits_np((rng.standard_normal((B, H, 512)) / 22).astype(np.float32))
        spx.spx_latent_append_fp4(B, to_dev_bf16(lat[rows, at][:, None]), 1, None, codes, scales,
                                  cap, len_dev, cap)
        spx.spx_pool_append(d, B, to_dev_bf16(keyb[rows, at][:, None]), 1, wp, tail, pooled,
                            cap // 4, len_dev, cap)
        len_dev += 1
        spx.spx_index_score(d, B, to_dev_bf16(synth.f32_to_bf16_bits_np(qi)),
                            torch.from_numpy(wh).cuda(), pooled, cap // 4, len_dev, cap, scores,
                            cap // 4)
        spx.spx_topk_blocks(d, B, scores, cap // 4, len_dev, cap, idx, cnt, tws)
        q = to_dev_bf16(qb)
        got, lse = _run_sparse(spx, d, q, codes, scales, cap * 512, cap, idx, cnt, len_dev, cap)
        all_, all_lse = _run_latent(spx, d, 1, q, codes, scales, len_dev, cap)
        back = torch.zeros(B, 1, 512, dtype=torch.bfloat16, device=dev)
        spx.spx_latent_read_fp4(B, codes, scales, cap, len_dev[:, None] - 1, 1, len_dev, back)
        for b in range(B):
            n = int(at[b]) + 1
            c, s = oracle.latent_fp4(lat[b, :n])
            assert np.array_equal(codes[b, :n].cpu().numpy(), c)
            assert np.array_equal(scales[b, :n].cpu().numpy(), s)
            vals = oracle.dequant_fp4(c, s)
            pool = oracle.pool(keyb[b, :n], [0.5, 0.25, 0.125, 0.125])
            sc = oracle.score(synth.f32_to_bf16_bits_np(qi[b]), wh[b].astype(np.float64), pool)
            sel = oracle.topk(sc)
            assert np.array_equal(idx[b, :int(cnt[b])].cpu().numpy(), sel)
            pos = oracle.token_set(sel, n)
            qv = oracle.bf16_to_f64(qb[b])
            _check(got[b], lse[b], qv, vals[pos], scale, 2051, f"step {step} row {b}")
            _check(all_[b], all_lse[b], qv, vals, scale, n, f"step {step} row {b}, all")
            _same_values(bits_of(back)[b, 0], vals[n - 1])
    assert not codes[1, int(lens[1]) + 5:].any()  # rows behind a sequence stay as they were
