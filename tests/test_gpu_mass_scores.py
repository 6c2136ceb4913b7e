"""mla_token_mass: how far off the weights of large scores are on average, by
where along the channels a score comes from.

The tensor core cuts the running sum of a score off towards zero at every
accumulation, which on average takes 0.5 ulp of it: kappa = 2^-24 E[1/m] = 4.3e-8 of
it for a mantissa m spread as in nature.  A score that its first channels make
loses that at each of the 36 to 108 accumulations, up to 4.6e-6 of itself; one
that the last channels make, or the only ones that are not 0, next to nothing.
The call gives the mean back.  What is left of the mean comes from the mantissas:
with scores over an octave or more their mean 1/m is within a tenth of E[1/m],
so that at most 0.1 x 4.6e-6 = 4.6e-7 of the score is left.  The 16 rows' kernel gives
nothing back and accumulates 27 times at most: 27 kappa = 1.2e-6 (bf16); its codes'
products are summed in fp32 arithmetic, two accumulations a group.  The log-sum-exp
times log2 e is rounded once, 2^-24 of it at most: 6e-8 of a score of its size.

Where the first 16 channels make the score and the others' queries are 1e-3 as
large, a K-step of the others adds 2^-10 of the sum, and its products with a low
half (2^-12 of the value) 2^-22 of it in 16 addends: 2^-24 each, below the sum's last
place.  Such an accumulation adds nothing and cuts nothing off, yet the mean counts
it: 72 of 108 (the low halves of either side), 36 of 72 where the queries' low halves
have columns of their own (up to 32 rows; those of the keys are left) or there are
none of the keys (bf16), so that up to 36 or 72 kappa too much is given back."""

import math

import pytest
import torch

from tests._helpers import F_BF16, F_I8G8, F_INT4, F_INT4S, F_INT8, FMT_NAME
from tests.test_gpu_mass import SCALE, Mass

pytestmark = pytest.mark.gpu
T, S = 1500, 20.0                                          # tokens, a score's size in nats


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def query(kind, mean, g):
    """A query of 576 channels, of any size, whose score comes from some of them."""
    r, q = torch.randn(576, generator=g), torch.zeros(576)
    if kind == "first step":
        q[:16] = mean[:16]
    elif kind == "latents":
        q[:512] = mean[:512]
    elif kind == "all":
        q[:] = mean
    elif kind == "rope":
        q[512:] = r[512:]
    elif kind == "last step":
        q[560:] = r[560:]
    elif kind == "three channels":
        q[[300, 301, 5]] = mean[[300, 301, 5]]
    elif kind == "first channels, others small":
        q[:] = 1e-3 * r
        q[:16] = mean[:16]
    elif kind == "last channels, others small":
        q[:] = 1e-3 * r
        q[560:] = r[560:]
    else:
        q[:] = r
    return q


def errors(mla, lf, kf, H, n, kind, seed, size=S):
    """(log of the mass over the formula's, score) of every token before the
    queries, which are all the same."""
    t = Mass(mla, [(T, n)], H, lf, kf, seed=seed, counted=[0], decay=0.0)
    x = torch.cat(t.hat[0], -1)[:T]
    q = query(kind, x.mean(0).float(), torch.Generator().manual_seed(seed + 5))
    q *= size / float((x @ q.double() * SCALE).abs().mean())
    t.q_lat[:], t.q_pe[:] = q[:512], q[512:].bfloat16()
    s = x @ torch.cat([t.q_lat[0, 0], t.q_pe[0, 0].float()]).double() * SCALE
    t.lse[:] = float(s.mean())
    got = t.go(mass=torch.zeros(t.num_pages * 64, device="cuda")).double().cpu()
    assert t.err.item() == 0
    at = torch.arange(T)
    want = torch.exp(s - float(t.lse[0, 0])) * n * H
    ok = (want > 1e-25) & (want < 1e25)                    # far from fp32's ends
    return torch.log(got[t.table[0].long()[at // 64] * 64 + at % 64] / want)[ok], s[ok]


KINDS = ["first step", "latents", "all", "rope", "last step", "three channels", "first channels, others small",
         "last channels, others small", "gauss"]
# heads, queries: 16 rows; 32; 48 (a pass of 64); 64; 128; a pass of 128 and one of 16
ROWS = [(16, 1), (32, 1), (16, 3), (64, 1), (64, 2), (16, 9)]


@pytest.mark.parametrize("lf,kf", [(F_BF16, F_BF16), (F_INT8, F_INT8), (F_INT4, F_INT4S), (F_I8G8, F_INT8), (F_BF16, F_INT8), (F_INT8, F_BF16)],
                         ids=lambda f: FMT_NAME[f])
@pytest.mark.parametrize("H,n", ROWS, ids=lambda v: str(v))
def test_mean_error_of_large_scores(mla, lf, kf, H, n):
    few = H * n == 16 and lf in (F_BF16, F_INT8, F_INT4)
    limit = (1.2e-6 if few and F_BF16 in (lf, kf) else 4.6e-7) + 6e-8
    low = 0 if few else (lf != F_BF16) + (H * n > 32)      # low halves among a score's accumulations
    for kind in KINDS:
        e, s = zip(*(errors(mla, lf, kf, H, n, kind, seed) for seed in (1, 2, 3)))
        e, s = torch.cat(e), torch.cat(s)
        left = float((e * s).sum() / (s * s).sum())
        assert abs(left) <= limit + (36 * 4.3e-8 * low if kind == "first channels, others small" else 0.0), (kind, left)


@pytest.mark.parametrize("lf,kf", [(F_BF16, F_BF16), (F_INT8, F_INT8)], ids=lambda f: FMT_NAME[f])
@pytest.mark.parametrize("H,n", ROWS, ids=lambda v: str(v))
def test_every_weight_of_large_scores(mla, lf, kf, H, n):
    """Each weight by itself: the running sums stay below the sum of the products'
    magnitudes, P = sum |q x| scale, and an accumulation cuts off less than 2^-23 of that, on
    either side of the mean; operands of 22 bits, three products."""
    for kind in KINDS:
        for seed in (1, 2):
            t = Mass(mla, [(T, n)], H, lf, kf, seed=seed, counted=[0], decay=0.0)
            x = torch.cat(t.hat[0], -1)[:T]
            q = query(kind, x.mean(0).float(), torch.Generator().manual_seed(seed + 5))
            q *= S / float((x @ q.double() * SCALE).abs().mean())
            q[512:] = q[512:].bfloat16().float()
            P = x.abs() @ q.double().abs() * SCALE
            e, s = errors(mla, lf, kf, H, n, kind, seed)
            full = x @ q.double() * SCALE
            P = P[[i for i in range(T) if 1e-25 < math.exp(float(full[i] - float(t.lse.new_tensor(float(full.mean()))))) * n * H < 1e25]]
            assert P.shape == e.shape
            assert bool((e.abs() <= P * (108 * 2.0 ** -23 + 3 * 2.0 ** -22) + 2.0 ** -21 + 2.0 ** -23 * s.abs() + n * H * 2.0 ** -24).all()), kind


@pytest.mark.parametrize("H,n", ROWS, ids=lambda v: str(v))
@pytest.mark.parametrize("lf,kf", [(F_BF16, F_BF16), (F_INT8, F_INT8), (F_INT4, F_INT4S)], ids=lambda f: FMT_NAME[f])
def test_mean_error_of_small_scores(mla, lf, kf, H, n):
    """Scores of about a nat: 1e-6 of the masses."""
    for kind in ("all", "gauss"):
        e, _ = zip(*(errors(mla, lf, kf, H, n, kind, seed, size=1.0) for seed in (1, 2, 3)))
        assert abs(float(torch.cat(e).mean())) <= 1e-6


@pytest.mark.parametrize("B", [1, 31, 33, 1100], ids=lambda b: "%d sequences" % b)
def test_mean_error_over_a_ragged_batch(mla, B):
    """Which accumulations a row's score goes through depends on its row block, and so
    on where its sequence's rows begin and end: sequences of 16 to 192 rows in passes of
    128, in batches whose sequences are found in one, two and three steps."""
    counts = [1, 12, 4, 5, 9, 2, 8, 3]
    new = [counts[b % 8] for b in range(B)] if B > 1 else [12]
    ctx = 64 if B > 100 else 300
    t = Mass(mla, [(ctx, n) for n in new], 16, F_INT8, F_INT8, seed=3, counted=[0] * B, decay=0.0)
    q = torch.randn(576, generator=torch.Generator().manual_seed(4))
    x = [torch.cat(h, -1)[:ctx] for h in t.hat]
    q *= S / float((torch.cat(x) @ q.double() * SCALE).abs().mean())
    t.q_lat[:], t.q_pe[:] = q[:512], q[512:].bfloat16()
    y = torch.cat([t.q_lat[0, 0], t.q_pe[0, 0].float()]).double()
    s = [a @ y * SCALE for a in x]
    lse = torch.tensor([float(a.mean()) for a in s], dtype=torch.float32)
    for b in range(B):
        t.lse[t.start[b]:t.start[b + 1]] = lse[b]
    got = t.go(mass=torch.zeros(t.num_pages * 64, device="cuda")).double().cpu()
    assert t.err.item() == 0
    at = torch.arange(ctx)
    for n in sorted(set(new)):
        num = den = 0.0
        for b in range(B):
            if new[b] != n:
                continue
            want = torch.exp(s[b] - float(lse[b])) * n * 16
            ok = (want > 1e-25) & (want < 1e25)
            e = torch.log(got[t.table[b].long()[at // 64] * 64 + at % 64] / want)[ok]
            num, den = num + float((e * s[b][ok]).sum()), den + float((s[b][ok] ** 2).sum())
        assert abs(num / den) <= 4.6e-7 + 6e-8, (n, num / den)
