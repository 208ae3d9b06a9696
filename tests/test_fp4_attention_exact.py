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
from test_fp4_latent import (LATENT_CASES, SPARSE_LENS, _run_latent, _run_sparse, _sparse_inputs,
                             _tokens)



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


@pytest.mark.gpu
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


# ---------------------------------------------------------------------------
# which tokens count
# ---------------------------------------------------------------------------
def _marked(rng, n, spread):
    """Rows that hold 3 to 6 in the dims t and 211 t + 7 (mod 512) alone, so that the mean
    shows which tokens were counted; with `spread`, times powers of two so far apart that
    8 neighbours do not share an exponent."""
    x = np.zeros((n, 512))
    t = np.arange(n)
    x[t, t % 512] = rng.choice([3.0, 4.0, 6.0], n)
    x[t, (211 * t + 7) % 512] = 6.0
    if spread:
        x *= np.exp2(rng.integers(-spread, spread + 1, (n, 1)).astype(float))
    return x


def _marked_cache(rng, seqs, cap, spread):
    x = np.stack([_marked(rng, cap, spread) for _ in range(seqs)])
    return *_quantised(x), x


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("heads", [16, 48, 64, 80, 128])
@pytest.mark.parametrize("lens", range(len(SPARSE_LENS)))
def test_selection_counts_every_token_once(heads, lens, spread):
    spx = need_gpu()
    n_vis = SPARSE_LENS[lens]
    rng = np.random.default_rng(heads + 1000 * lens)
    rows, cap = len(n_vis), max(n_vis)
    d = spx.dims(heads, 0.7)
    codes, scales, x = _marked_cache(rng, rows, cap, spread)
    idx, cnt = _sparse_inputs(rng, n_vis)
    q = torch.zeros(rows, heads, 512, dtype=torch.bfloat16, device="cuda")
    got, lse = _run_sparse(spx, d, q, codes, scales, cap * 512, cap, torch.from_numpy(idx).cuda(),
                           torch.from_numpy(cnt).cuda(), torch.tensor(n_vis, device="cuda"), cap)
    for r, n in enumerate(n_vis):
        if n == 0:
            assert (got[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        _check_mean(got[r], lse[r], x[r][_tokens(idx[r], cnt[r], n)], spread, f"row {r} ({n})")


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0, 6])
def test_chunk_counts_every_token_once(spread):
    """More rows than SMs on one cache, units that end inside a CTA's part."""
    spx = need_gpu()
    rng = np.random.default_rng(3 + spread)
    T, n, heads = 333, 2600, 64
    d = spx.dims(heads, 1.0)
    n_vis = list(range(n - T + 1, n + 1))
    codes, scales, x = _marked_cache(rng, 1, n, spread)
    idx, cnt = _sparse_inputs(rng, n_vis)
    q = torch.zeros(T, heads, 512, dtype=torch.bfloat16, device="cuda")
    got, lse = _run_sparse(spx, d, q, codes, scales, 0, n, torch.from_numpy(idx).cuda(),
                           torch.from_numpy(cnt).cuda(), torch.tensor(n_vis, device="cuda"), n)
    for r in range(T):
        _check_mean(got[r], lse[r], x[0][_tokens(idx[r], cnt[r], n_vis[r])], spread, f"row {r}")


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("heads", [16, 32, 48, 64, 112, 128])
@pytest.mark.parametrize("case", range(len(LATENT_CASES)))
def test_whole_cache_counts_every_token_once(heads, case, spread):
    spx = need_gpu()
    per, n_vis = LATENT_CASES[case]
    rng = np.random.default_rng(heads + 1000 * case)
    rows, cap = len(n_vis), max(n_vis) + 3
    d = spx.dims(heads, 1.3)
    codes, scales, x = _marked_cache(rng, rows // per, cap, spread)
    q = torch.zeros(rows, heads, 512, dtype=torch.bfloat16, device="cuda")
    got, lse = _run_latent(spx, d, per, q, codes, scales, torch.tensor(n_vis, device="cuda"), cap)
    for r, n in enumerate(n_vis):
        if n == 0:
            assert (got[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        _check_mean(got[r], lse[r], x[r // per][:n], spread, f"row {r} ({n})")


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,per,cap,heads", [(613, 1, 70, 16), (300, 3, 200, 80), (1, 200, 900, 64),
                                                (2, 129, 1300, 16), (31, 1, 600, 64),
                                                (32, 1, 600, 64), (33, 1, 600, 16)])
def test_many_units_count_every_token_once(seqs, per, cap, heads):
    """Many short sequences, and chunks of many rows over one cache, each row with its
    own (causal, or any) length."""
    spx = need_gpu()
    rng = np.random.default_rng(cap)
    if per > 100:  # a causal chunk at the end
        n_vis = np.tile(np.arange(cap - per + 1, cap + 1), seqs)
    else:
        n_vis = rng.integers(0, cap + 1, seqs * per)
    d = spx.dims(heads, 0.9)
    x = _marked(rng, cap, 1)
    codes, scales = _quantised(x[None])
    codes, scales = (t.expand(seqs, -1, -1).contiguous() for t in (codes, scales))
    q = torch.zeros(seqs * per, heads, 512, dtype=torch.bfloat16, device="cuda")
    got, lse = _run_latent(spx, d, per, q, codes, scales, torch.from_numpy(n_vis).cuda(), cap)
    for r, n in enumerate(n_vis):
        if n == 0:
            assert (got[r] == 0).all() and np.isneginf(lse[r]).all()
        else:
            _check_mean(got[r], lse[r], x[:n], 1, f"row {r} ({n})")


@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("n", [2, 64, 129, 700, 2051, 5000])
def test_the_bounds_show_one_wrong_token(n, spread):
    """A count of one token less or more is outside them, and where tokens are of like
    size (a small one among large ones is below the output's own rounding) so is a mean
    over other tokens (mistakes planted in what is checked, on the CPU)."""
    rng = np.random.default_rng(n)
    x = _marked(rng, n + 1, spread)
    for wrong in (np.delete(x[:n], n // 2, 0), x, np.concatenate([x[:n], x[n // 3:n // 3 + 1]])):
        got = np.repeat(wrong.mean(0)[None], 16, 0)
        lse = np.full(16, np.log(wrong.shape[0]))
        _check_mean(got, lse, wrong, spread, "right")
        if spread == 0:
            with pytest.raises(AssertionError):
                _check_mean(got, np.full(16, np.log(n)), x[:n], spread, "mean")
        with pytest.raises(AssertionError):
            _check_mean(np.repeat(x[:n].mean(0)[None], 16, 0), lse, x[:n], spread, "lse")
    wrong = x[:n].copy()
    wrong[n // 2] = x[n]
    if spread == 0:
        with pytest.raises(AssertionError):
            _check_mean(np.repeat(wrong.mean(0)[None], 16, 0), np.full(16, np.log(n)), x[:n], 0, "")
