"""The 4-bit latent cache's calls in layouts and sizes a caller may choose:
wider strides, pointers on 16-byte boundaries alone, a cache in pinned host
memory, the most rows of a call."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _gpu_helpers import bits_of, need_gpu, to_dev_bf16
from test_fp4_latent import _check, _run_latent, _run_sparse, _sparse_inputs

pytestmark = pytest.mark.gpu


def _rows(rng, seqs, cap):
    x = rng.standard_normal((seqs * cap, 512)) * np.exp2(rng.integers(-3, 4, (seqs * cap, 1)))
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.astype(np.float32)))
    return (torch.from_numpy(codes.reshape(seqs, cap, 256)).cuda(),
            torch.from_numpy(scales.reshape(seqs, cap, 16)).cuda())


def _q(rng, rows, heads):
    return to_dev_bf16(synth.f32_to_bf16_bits_np(
        (rng.standard_normal((rows, heads, 512)) / 22).astype(np.float32)))


def _off16(t):
    """The same values in memory that starts 16 bytes behind a 256-byte boundary."""
    raw = torch.empty(t.numel() * t.element_size() + 512, dtype=torch.uint8, device=t.device)
    at = (-raw.data_ptr()) % 256 + 16
    v = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 256 == 16
    return v


def test_selection_with_a_wider_stride():
    """Sequences further apart than cap_tok: rows between them are not read."""
    spx = need_gpu()
    rng = np.random.default_rng(1)
    n_vis, heads, cap, apart = [700, 513, 2], 64, 700, 737
    d = spx.dims(heads, 1.0)
    codes, scales = _rows(rng, 3, cap)
    wide_c = torch.full((3, apart, 256), 0xFF, dtype=torch.uint8, device="cuda")
    wide_s = torch.full((3, apart, 16), 255, dtype=torch.uint8, device="cuda")  # NaN
    wide_c[:, :cap], wide_s[:, :cap] = codes, scales
    idx, cnt = (torch.from_numpy(a).cuda() for a in _sparse_inputs(rng, n_vis))
    q, n_dev = _q(rng, 3, heads), torch.tensor(n_vis, device="cuda")
    ref = _run_sparse(spx, d, q, codes, scales, cap * 512, cap, idx, cnt, n_dev, cap)
    got = _run_sparse(spx, d, q, wide_c, wide_s, apart * 512, cap, idx, cnt, n_dev, cap)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


@pytest.mark.parametrize("heads,per", [(16, 3), (128, 1)])
def test_pointers_on_16_byte_boundaries(heads, per):
    spx = need_gpu()
    rng = np.random.default_rng(heads)
    seqs, cap, new = 2, 901, 5
    rows = seqs * per
    d = spx.dims(heads, 1.0)
    codes, scales = _rows(rng, seqs, cap)
    lat = to_dev_bf16(synth.f32_to_bf16_bits_np(
        rng.standard_normal((seqs, new, 512)).astype(np.float32)))
    lens = torch.tensor([cap - new, 310], device="cuda")
    n_vis = (lens + new).repeat_interleave(per)
    q = _q(rng, rows, heads)
    idx, cnt = (torch.from_numpy(a).cuda() for a in _sparse_inputs(rng, n_vis.tolist()))
    pos = torch.tensor([[0, cap - 1, 7], [314, 1, 315]], device="cuda")
    need = spx.spx_latent_attn_fp4_workspace_size(d, rows, per, cap)
    res = []
    for f in (lambda t: t.clone(), _off16):
        c, s, x, qq = f(codes), f(scales), f(lat), f(q)
        ws = f(torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda"))
        stored, back = f(torch.zeros_like(lat)), f(torch.zeros(seqs, 3, 512, dtype=torch.bfloat16,
                                                               device="cuda"))
        out, lse = f(torch.zeros_like(q)), f(torch.zeros(rows, heads, device="cuda"))
        spx.spx_latent_append_fp4(seqs, x, new, None, c, s, cap, f(lens), cap, stored)
        spx.spx_latent_read_fp4(seqs, c, s, cap, f(pos), 3, f(lens + new), back)
        spx.spx_latent_attn_fp4(d, rows, per, qq, c, s, cap, f(n_vis), cap, out, lse, ws)
        res.append([c, s, stored, back, out, lse])
        if per == 1:
            out, lse = f(torch.zeros_like(q)), f(torch.zeros(rows, heads, device="cuda"))
            spx.spx_sparse_mla_attn_fp4(d, rows, qq, c, s, cap * 512, cap, f(idx), f(cnt), f(n_vis),
                                        cap, out, lse, ws)
            res[-1] += [out, lse]
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 0
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_append_and_read_in_pinned_host_memory():
    spx = need_gpu()
    rng = np.random.default_rng(3)
    B, cap, new = 2, 70, 33
    lat = to_dev_bf16(synth.f32_to_bf16_bits_np(
        rng.standard_normal((B, new, 512)).astype(np.float32)))
    lens = torch.tensor([0, 37], device="cuda")
    res = []
    for host in (False, True):
        c = torch.zeros(B, cap, 256, dtype=torch.uint8, device="cpu" if host else "cuda", pin_memory=host)
        s = torch.zeros(B, cap, 16, dtype=torch.uint8, device="cpu" if host else "cuda", pin_memory=host)
        out = torch.full((B, cap, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        spx.spx_latent_append_fp4(B, lat, new, None, c, s, cap, lens, cap)
        spx.spx_latent_read_fp4(B, c, s, cap, None, cap, lens + new, out)
        torch.cuda.synchronize()
        res.append((c.cpu(), s.cpu(), out.cpu()))
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("whole", [False, True])
def test_the_most_rows_of_a_call(whole):
    """65,535 rows of queries of zero: each gives the mean of what it sees, which is one
    (a cache of ones), and the logarithm of how many."""
    spx = need_gpu()
    rows, heads, cap = 65535, 16, 193
    d = spx.dims(heads, 1.0)
    codes = torch.full((1, cap, 256), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, cap, 16), 127, dtype=torch.uint8, device="cuda")
    q = torch.zeros(rows, heads, 512, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full((rows, heads), 5.0, device="cuda")
    n_vis = torch.arange(rows, device="cuda") * 7 % (cap + 1)
    if whole:
        need = spx.spx_latent_attn_fp4_workspace_size(d, rows, rows, cap)
        spx.spx_latent_attn_fp4(d, rows, rows, q, codes, scales, cap, n_vis, cap, out, lse,
                                spx.workspace(need, "cuda"))
        seen = n_vis
    else:
        idx = torch.arange(512, dtype=torch.int32, device="cuda").expand(rows, -1).contiguous()
        cnt = (torch.arange(rows, device="cuda") % 50).int()
        need = spx.spx_attn_fp4_workspace_size(d, rows, cap)
        spx.spx_sparse_mla_attn_fp4(d, rows, q, codes, scales, 0, cap, idx, cnt, n_vis, cap, out,
                                    lse, spx.workspace(need, "cuda"))
        seen = 4 * torch.minimum(cnt.long(), n_vis // 4) + n_vis % 4
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 0
    want = torch.where(seen > 0, 1.0, 0.0).bfloat16()[:, None, None]
    assert (out == want).all()
    ref = torch.log(seen.double())
    err = (lse.double() - ref[:, None]).abs()
    # fp32 sums of equal weights, each to 2^-22, and the logarithm: 2^-19 in all
    assert (torch.where(seen[:, None] > 0, err, 0.0) <= 2.0 ** -19 + 2.0 ** -22 * ref.clamp(min=0)[:, None]).all()
    assert torch.isneginf(lse[seen == 0]).all()


def test_whole_cache_needs_no_order_of_lengths():
    """A chunk's rows may see any lengths, in any order, a row none at all between."""
    spx = need_gpu()
    rng = np.random.default_rng(5)
    per, heads, cap = 70, 32, 333
    d = spx.dims(heads, 1.0)
    codes, scales = _rows(rng, 1, cap)
    q = _q(rng, per, heads)
    lens = rng.permutation(np.concatenate([np.zeros(9, int), rng.integers(1, cap + 1, per - 9)]))
    out, lse = _run_latent(spx, d, per, q, codes, scales, torch.from_numpy(lens).cuda(), cap)
    vals = oracle.dequant_fp4(codes[0].cpu().numpy(), scales[0].cpu().numpy())
    qv = oracle.bf16_to_f64(bits_of(q))
    for r, n in enumerate(lens):
        _check(out[r], lse[r], qv[r], vals[:n], 1.0, n, f"row {r} ({n} tokens)")
        if n == 0:
            assert (out[r] == 0).all()
