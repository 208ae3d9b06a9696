"""Attention over the 4-bit latent cache where its bounds are met: lengths
without a bound, on the CPU (sizes and refusals) and on the GPU."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _gpu_helpers import LSE_ATOL, assert_attention_close, need_gpu, to_dev_bf16
from test_fp4_latent import _run_latent, _run_sparse, _sparse_inputs, _tokens

FAKE = 1 << 20  # an aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from conftest import build_lib
    build_lib()
    import long_context_decode_indexpool_b200 as m
    return m


# ---------------------------------------------------------------------------
# max_len without a bound
# ---------------------------------------------------------------------------
HUGE = (2 ** 31, 2 ** 40, 2 ** 57, 2 ** 62, 2 ** 63 - 128, 2 ** 63 - 64, 2 ** 63 - 63, 2 ** 63 - 1)


@pytest.mark.parametrize("rows,per", [(1, 1), (4, 2), (63, 1), (64, 1), (65, 1), (128, 64),
                                      (65535, 65535)])
def test_workspace_of_any_length(lib, rows, per):
    for heads in (16, 64, 128):
        d = lib.dims(heads, 1.0)
        sizes = [lib.spx_latent_attn_fp4_workspace_size(d, rows, per, n)
                 for n in (0, 1, 64, 65, 5000, 2 ** 20, 2 ** 31 - 1)]
        assert sizes == sorted(sizes) and 0 < sizes[-1] < 1 << 26
        for n in HUGE:
            assert lib.spx_latent_attn_fp4_workspace_size(d, rows, per, n) == sizes[-1], n
        if per == 1:
            most = lib.spx_attn_fp4_workspace_size(d, rows, 2 ** 31 - 1)
            for n in HUGE:
                assert lib.spx_attn_fp4_workspace_size(d, rows, n) == most, n


@pytest.mark.parametrize("max_len", HUGE)
def test_calls_of_any_length_check_the_workspace(lib, max_len):
    """A call whose rows may be shared by several CTAs wants the workspace for
    that, whatever bound it is given; nothing is launched without it."""
    d = lib.dims(64, 1.0)
    for rows in (1, 63, 64, 65, 100):
        for cap in (8192, 2 ** 31 - 1):
            with pytest.raises(lib.SpxError) as e:
                lib.spx_latent_attn_fp4(d, rows, 1, FAKE, FAKE, FAKE, cap, FAKE, max_len, FAKE,
                                        None, None, 0, stream=0)
            # more than 2^31 - 1 tiles: 64 rows of 2^31 - 1 tokens and up
            assert e.value.status == (3 if cap > 8192 and rows >= 64 else 4), (rows, cap)
        with pytest.raises(lib.SpxError) as e:
            lib.spx_sparse_mla_attn_fp4(d, rows, FAKE, FAKE, FAKE, 0, 8192, FAKE, FAKE, FAKE,
                                        max_len, FAKE, None, None, 0, stream=0)
        assert e.value.status == 4


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 65])
def test_no_bound_is_the_cache_s_own(rows):
    """max_len = INT64_MAX gives bit for bit what max_len = cap_tok gives."""
    spx = need_gpu()
    rng = np.random.default_rng(40 + rows)
    cap, d = 700, spx.dims(64, 1.0)
    codes, scales = oracle.latent_fp4(
        synth.f32_to_bf16_bits_np(rng.standard_normal((cap, 512)).astype(np.float32)))
    codes = torch.from_numpy(codes).cuda().expand(rows, -1, -1).contiguous()
    scales = torch.from_numpy(scales).cuda().expand(rows, -1, -1).contiguous()
    q = to_dev_bf16(synth.f32_to_bf16_bits_np(
        (rng.standard_normal((rows, 64, 512)) / 22).astype(np.float32)))
    n_vis = torch.from_numpy(rng.integers(0, 2 * cap, rows)).cuda()
    got = []
    for max_len in (cap, 2 ** 63 - 64, 2 ** 63 - 1):
        ws = spx.workspace(spx.spx_latent_attn_fp4_workspace_size(d, rows, 1, max_len), "cuda")
        out, lse = torch.empty_like(q), torch.empty(rows, 64, device="cuda")
        spx.spx_latent_attn_fp4(d, rows, 1, q, codes, scales, cap, n_vis, max_len, out, lse, ws)
        torch.cuda.synchronize()
        assert spx.spx_device_error() == 0
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


# ---------------------------------------------------------------------------
# against the oracle's own attention (C++, fp64)
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("heads,n_vis", [(16, [1, 700]), (64, [2049, 130]), (80, [63, 1027])])
def test_against_the_oracle_s_attention(heads, n_vis):
    spx = need_gpu()
    rng = np.random.default_rng(heads)
    d, cap = spx.dims(heads, 0.8), max(n_vis)
    codes, scales = oracle.latent_fp4(
        synth.f32_to_bf16_bits_np(rng.standard_normal((2 * cap, 512)).astype(np.float32)))
    codes, scales = codes.reshape(2, cap, 256), scales.reshape(2, cap, 16)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((2, heads, 512)) / 22).astype(np.float32))
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales)]
    n_dev = torch.tensor(n_vis, dtype=torch.int64, device="cuda")
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), *dev, n_dev, cap)
    idx, cnt = _sparse_inputs(rng, n_vis, spoil=False)
    sp, sp_lse = _run_sparse(spx, d, to_dev_bf16(qb), *dev, cap * 512, cap,
                             torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(), n_dev, cap)
    for r, n in enumerate(n_vis):
        pos = _tokens(idx[r], cnt[r], n)
        for o, l, rows in ((got[r], lse[r], slice(0, n)), (sp[r], sp_lse[r], pos)):
            ref, ref_lse = oracle.attention_fp4(qb[r], codes[r][rows], scales[r][rows], 0.8)
            assert_attention_close(o, ref, f"row {r}")
            assert np.abs(l - ref_lse).max() <= LSE_ATOL


# ---------------------------------------------------------------------------
# the largest queries
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("low,high", [(-50, -50), (-50, -44), (-50, -30)])
def test_largest_queries_over_small_rows(low, high):
    """Queries near bf16's largest value and rows near the format's smallest: logits of
    about 2^80 (finite in fp32), so the softmax picks one token.  Rows alike in size, and
    rows whose 8 neighbours cannot share an exponent."""
    spx = need_gpu()
    rng = np.random.default_rng(65 - low + high)
    n, heads = 150, 16
    x = rng.standard_normal((n, 512)) * np.exp2(rng.choice([low, high], (n, 1)).astype(float))
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    vals = oracle.dequant_fp4(codes, scales)
    qb = synth.f32_to_bf16_bits_np((rng.standard_normal((1, heads, 512)) * 2.0 ** 124)
                                   .astype(np.float32))
    q = oracle.bf16_to_f64(qb)[0]
    z = q @ vals.T
    best = z.argmax(-1)
    top2 = np.sort(z, -1)[:, -2:]
    # the terms' absolute sum times 512 * 2^-23 (a sum of 512 products in fp32) is below
    # the lead of the best token, which is of 2^60 bits and more
    assert (top2[:, 1] - top2[:, 0] > 2.0 ** -14 * (np.abs(q) @ np.abs(vals).T).max(-1)).all()
    d = spx.dims(heads, 1.0)
    got, lse = _run_latent(spx, d, 1, to_dev_bf16(qb), torch.from_numpy(codes)[None].cuda(),
                           torch.from_numpy(scales)[None].cuda(),
                           torch.tensor([n], dtype=torch.int64, device="cuda"), n)
    assert np.array_equal(got[0], vals[best])
    assert (np.abs(lse[0] - top2[:, 1]) <= 2.0 ** -13 * np.abs(q).max() * 512 * np.abs(vals).max()).all()
    assert np.isfinite(lse).all()


# ---------------------------------------------------------------------------
# the read back's two forms
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("more", [-1, 0, 1, 2, 3])
@pytest.mark.parametrize("scattered", [False, True])
def test_read_back_where_its_form_changes(more, scattered):
    """A call of about 128 rows an SM gives what calls of fewer rows give."""
    spx = need_gpu()
    m = 128 * torch.cuda.get_device_properties(0).multi_processor_count + more
    g = torch.Generator(device="cuda").manual_seed(m)
    cap, n = m + 5, m - 7  # the last rows lie behind the sequence's end
    codes = torch.randint(0, 256, (1, cap, 256), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(100, 140, (1, cap, 16), dtype=torch.uint8, device="cuda", generator=g)
    n_vis = torch.tensor([n], device="cuda")
    pos = torch.arange(m, device="cuda")[None]
    if scattered:
        pos = torch.randint(-3, cap + 3, (1, m), device="cuda", generator=g)
    out = torch.full((1, m, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    spx.spx_latent_read_fp4(1, codes, scales, cap, pos if scattered else None, m, n_vis, out)
    ref = torch.full_like(out, 5.0)
    for at in range(0, m, 5000):
        k = min(5000, m - at)
        spx.spx_latent_read_fp4(1, codes, scales, cap, pos[:, at:].contiguous(), k, n_vis,
                                ref[:, at:])
    assert torch.equal(out, ref)
    seen = (pos >= 0) & (pos < n)
    assert (out[~seen] == 0).all() and (out[seen] != 0).any(-1).all()
