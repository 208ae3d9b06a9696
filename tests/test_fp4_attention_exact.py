"""Attention over the 4-bit latent cache where the answer is known closely:
queries of zero weigh every token alike, so lse is the logarithm of their
number and the output their mean, with none of the logits' rounding in the
bounds.  A token that is lost, counted twice or masked wrongly shows in both."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _gpu_helpers import need_gpu, to_dev_bf16
from test_fp4_latent import _run_latent, _run_sparse

pytestmark = pytest.mark.gpu


def _quantised(x):
    """Codes and scales of rows [.., 512] whose values the cache holds exactly."""
    codes, scales = oracle.latent_fp4(synth.f32_to_bf16_bits_np(x.reshape(-1, 512).astype(np.float32)))
    assert np.array_equal(oracle.dequant_fp4(codes, scales), x.reshape(-1, 512))
    return (torch.from_numpy(codes.reshape(*x.shape[:-1], 256)).cuda(),
            torch.from_numpy(scales.reshape(*x.shape[:-1], 16)).cuda())


def _check_mean(got, lse, rows, ref_exp, what):
    """rows [n, 512], not negative, which the row's heads weigh alike; 2^ref_exp is at
    least the reference exponent of every token (the largest of its row and of the 7
    beside it).  By arithmetic: a weight (2^(E_t - max + 7), to 2^-22 by ex2) is rounded
    to fp16 (2^-11), and where CTAs share the row, so is each one's part (2^-11, or, the
    part being stored times 2^13, half of fp16's last bit, 2^-25 2^-13 of the weights'
    mean 2^E_t); fp32 sums of at most n / 16 + 64 steps, each off by 2^-23 (a truncating
    adder counted); the joining weights, division and logarithm 2^-19; the output is
    rounded to bf16 once (2^-8).  All of it relative to the mean, which has no
    cancellation."""
    n = rows.shape[0]
    assert (rows >= 0).all()
    o = rows.mean(0)
    adds = n / 16 + 64
    tol = o * (2.0 ** -8 * 1.01 + 2 * 2.0 ** -11 + 2.0 ** -19 + adds * 2.0 ** -23) \
        + 2.0 ** (ref_exp - 38)
    err = np.abs(got - o)
    assert (err <= tol).all(), (what, float((err / np.maximum(o, 1e-30)).max()), int((err > tol).sum()))
    # the normaliser has no roundings to 16 bits
    lse_tol = 2.0 ** -19 + 2.0 ** -22 * np.log(n) + adds * 2.0 ** -23
    assert (np.abs(lse - np.log(n)) <= lse_tol).all(), (what, float(np.abs(lse - np.log(n)).max()))


# ---------------------------------------------------------------------------
# small groups of a row that several CTAs share
# ---------------------------------------------------------------------------
def _small_groups(n, lead):
    """Rows whose group g lies 2^g below group 0: 0.5 or 1 in units of it, by a pattern
    that every tile of 64 tokens repeats (so that the CTAs' parts err alike).  `lead`: of
    8 tokens, the first is 16 times as large in group 0 and zero elsewhere: the 8 then
    share an exponent 4 above the others' own."""
    t, d = np.arange(n) % 64, np.arange(512)
    x = np.where((t[:, None] * 37 + d[None] * 11) % 64 < (d % 32) * 2, 1.0, 0.5)
    x = x * np.exp2(-(d // 32))[None]
    x[:, 0] = 6.0  # the group whose exponent is the row's: 0
    if lead:
        x[::8] = 0.0
        x[::8, 0] = 96.0
    return x


@pytest.mark.parametrize("lead", [False, True])
@pytest.mark.parametrize("n,heads", [(2040, 64), (5000, 16), (40960, 16), (40961, 128)])
def test_small_groups_of_a_shared_row(n, heads, lead):
    """Groups down to 2^15 below a row's largest (2^19 below the exponent it is held
    with) keep their own relative accuracy, whole cache and selection."""
    spx = need_gpu()
    d = spx.dims(heads, 1.0)
    x = _small_groups(n, lead)
    codes, scales = _quantised(x[None])
    q = torch.zeros(1, heads, 512, dtype=torch.bfloat16, device="cuda")
    n_vis = torch.tensor([n], dtype=torch.int64, device="cuda")
    got, lse = _run_latent(spx, d, 1, q, codes, scales, n_vis, n)
    ref_exp = 4 if lead else 0
    _check_mean(got[0], lse[0], x, ref_exp, "whole cache")
    idx = torch.arange(512, dtype=torch.int32, device="cuda")[None]  # the first 512 blocks
    cnt = torch.tensor([512], dtype=torch.int32, device="cuda")
    got, lse = _run_sparse(spx, d, q, codes, scales, 0, n, idx, cnt, n_vis, n)
    k = min(512, n // 4)
    _check_mean(got[0], lse[0], np.concatenate([x[:4 * k], x[n // 4 * 4:]]), ref_exp, "selection")
