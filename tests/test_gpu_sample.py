"""vc_accept_sample against the oracle: the same tokens for the same random numbers."""
import numpy as np
import pytest
import torch

import lossless_kv_compressed_b200 as vc
from oracle import sample

pytestmark = pytest.mark.gpu


def make(B, k, V, seed, dtype=torch.float32, spread=2.5, noise=0.4):
    g = torch.Generator().manual_seed(seed)
    lg = (torch.randn((B, k + 1, V), generator=g) * spread).to(dtype)
    ql = (lg[:, :k].float() + noise * torch.randn((B, k, V), generator=g)).to(dtype)
    d = torch.distributions.Categorical(logits=ql.float()).sample() if k else torch.zeros((B, 0))
    u = torch.rand((B, k + 1), generator=g, dtype=torch.float64)
    return lg, ql, d.to(torch.int32), u


def check(lg, d, u, ql=None, T=None, n=None):
    cu = lambda t: None if t is None else t.cuda()
    r = vc.accept_sample(lg.cuda(), cu(d), u.cuda(), cu(ql), cu(T), cu(n))
    num = lambda t: None if t is None else t.double().numpy()
    want = sample.accept_sample(num(lg), num(d), num(u), num(ql), num(T),
                                None if n is None else n.numpy())
    for x in ("accept_len", "commit", "n_commit", "err"):
        assert np.array_equal(r[x].cpu().numpy(), want[x]), (x, r[x].cpu(), want[x])
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k,V", [(1, 1, 1000), (3, 4, 8192), (2, 7, 4099), (5, 0, 513),
                                   (2, 3, 128256), (4, 2, 1), (3, 2, 7), (1, 256, 130), (70, 1, 300)])
def test_matches_the_oracle(B, k, V, dtype):
    lg, ql, d, u = make(B, k, V, B + k + V, dtype)
    check(lg, d, u, ql)
    check(lg, d, u)
    T = torch.tensor([(0.7, 1.0, 0.0, 3.0, 0.05)[b % 5] for b in range(B)])
    n = torch.tensor([max(0, k - b % 3) for b in range(B)], dtype=torch.int32)
    check(lg, d, u, ql, T, n)
    check(lg, d, u, None, T, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k,V", [(400, 2, 5003), (297, 1, 40000), (149, 1, 40000)])
def test_sequences_that_one_block_serves(B, k, V, dtype):
    lg, ql, d, u = make(B, k, V, B, dtype)
    check(lg, d, u, ql)
    check(lg, d, u, None, torch.rand(B) * 2)


def test_accepted_drafts_and_the_bonus_token():
    lg, ql, d, u = make(4, 5, 2000, 1, noise=0.0)          # p == q: nothing is refused
    w = check(lg, d, u, lg[:, :5].contiguous())
    assert w["accept_len"].tolist() == [5] * 4
    u[:, :5] = 0.0
    assert check(lg, d, u)["accept_len"].tolist() == [5] * 4


def test_masked_vocabulary_and_one_token_left():
    lg, ql, d, u = make(3, 3, 1500, 2)
    lg[:, :, ::3] = -float("inf")
    check(lg, d, u, ql)
    check(lg, d, u)
    lg[:] = -float("inf")
    lg[:, :, 1499] = -5.0                                  # all of p on the last token
    w = check(lg, d, u, ql)
    assert (w["commit"][:, 0] == 1499).all()
    d[:] = 1499
    check(lg, d, u)


def test_rows_and_arguments_that_are_not_valid():
    lg, ql, d, u = make(8, 3, 700, 3)
    u[:, :3] = 0.0                                         # accept wherever p > 0
    lg[0, 1, 30], lg[0, 1, 12] = float("nan"), float("nan")
    lg[1, 0, 5] = float("inf")
    lg[2, 3] = -float("inf")
    d[3, 1] = -1
    d[4, 0] = 700
    ql[5, 1, 9] = float("nan")
    lg[6, 3, 0] = float("nan")
    d[6, 0] = 700                                          # refused before the bad row is met
    w = check(lg, d, u, ql)
    assert w["err"].tolist() == [1, 1, 1, 1, 1, 1, 1, 0]
    check(lg, d, u)
    check(lg, d, u, ql, torch.zeros(8))
    T = torch.tensor([-1.0, float("nan"), float("inf"), 1e-30, 1e30, 0.0, 1.0, 2.0])
    n = torch.tensor([-1, 4, 3, 0, 1, 2, 3, 3], dtype=torch.int32)
    check(*make(8, 3, 700, 4)[:1], make(8, 3, 700, 4)[2], u, make(8, 3, 700, 4)[1], T, n)


def test_random_numbers_at_the_ends():
    lg, ql, d, u = make(6, 2, 5000, 5)
    u[:3] = 0.0
    u[3:] = 1.0 - 2.0 ** -53
    check(lg, d, u, ql)
    check(lg, d, u)


def test_ties_of_greedy_sequences():
    lg, ql, d, u = make(4, 3, 3000, 6, torch.bfloat16, spread=0.1)
    lg = (lg * 8).round()
    T = torch.zeros(4)
    d[:, 0] = lg[:, 0].float().argmax(-1).to(torch.int32)
    w = check(lg, d, u, ql, T)
    assert (w["accept_len"] >= 1).all()


def test_flat_rows_cross_many_borders():
    """Nearly flat rows of 128K tokens: thousands of borders a percent apart from rounding in
    32 bits; every one of 64 sequences has to give the oracle's token."""
    g = torch.Generator().manual_seed(7)
    lg = torch.randn((16, 2, 128256), generator=g) * 0.05
    ql = (lg[:, :1] + 0.05 * torch.randn((16, 1, 128256), generator=g)).contiguous()
    d = torch.randint(0, 128256, (16, 1), generator=g, dtype=torch.int32)
    for s in range(2):
        u = torch.rand((16, 2), generator=g, dtype=torch.float64)
        check(lg, d, u, ql)
        check(lg, d, u)


def test_captured_twice_and_replayed_on_two_streams():
    a, b = make(3, 4, 9000, 8), make(3, 4, 9000, 9)
    outs, graphs, wants = [], [], []
    for lg, ql, d, u in (a, b):
        t = [x.cuda() for x in (lg, d, u, ql)]
        wants.append(vc.accept_sample(*t)["commit"].clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = vc.accept_sample(*t)
        outs.append((r, t))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (r, _), w in zip(outs, wants):
        assert torch.equal(r["commit"], w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k", [(8200, 3), (16385, 1), (65535, 0), (128, 256)])
def test_more_rows_than_one_plane_of_the_grid(B, k, dtype):
    """Row counts above 32768 and no multiple of it, with and without draft logits: the rows that
    fill up the grid's last plane belong to no sequence."""
    lg, ql, d, u = make(B, k, 7, B, dtype)
    check(lg, d, u)
    if k:
        check(lg, d, u, ql)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,gain", [(1e-18, 60.0), (3e-18, 2000.0), (1e-15, 60.0), (1e-9, 1e4),
                                    (1.0, 1e19), (1.0, 1e20), (0.3, 1e37)])
def test_logits_far_larger_than_the_temperature(T, gain, dtype):
    """Nearly all of p on the largest logit, however large it is against T: it weighs 1."""
    lg, ql, d, u = make(6, 3, 3001, 11, dtype)
    lg = (lg.float() * (gain / 10)).to(dtype)
    ql = (ql.float() * (gain / 10)).to(dtype)
    lg[2:4, :, 5] = lg[2:4].amax(-1)               # a tie: half of p each
    d[1:4] = lg[1:4, :3].float().argmax(-1).to(torch.int32)
    ql[1, torch.arange(3), d[1].long()] = ql[1].amax(-1)
    t = torch.full((6,), T)
    w = check(lg, d, u, None, t)
    assert w["accept_len"][1] == 3 and not w["err"].any()
    check(lg, d, u, ql, t)


@pytest.mark.parametrize("V", [700, 40000])
@pytest.mark.parametrize("shift", [0.0, 1.0])
def test_equal_rows_refused_at_the_last_number(V, shift):
    """p == q to the last bit and u one step below 1: whether u q < p then depends on rounding.
    Where a draft is refused, max(p - q, 0) is 0 everywhere and the token comes from p."""
    B, k = 60, 3
    lg, _, _, u = make(B, k, V, V)
    lg = (lg * 1024).round() / 1024                # adding 1 is exact
    ql = (lg[:, :k] + shift).contiguous()
    d = torch.distributions.Categorical(logits=ql).sample().to(torch.int32)
    u[:, :k] = 1.0 - 2.0 ** -53
    r = vc.accept_sample(lg.cuda(), d.cuda(), u.cuda(), ql.cuda())
    a, commit = r["accept_len"].cpu().numpy(), r["commit"].cpu().numpy()
    assert not r["err"].any() and (a < k).any()
    for b in range(B):
        c = np.cumsum(sample.probabilities(lg[b, a[b]].double().numpy(), 1.0))
        assert commit[b, a[b]] == np.nonzero(c > u[b, k].item() * c[-1])[0][0], b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,gain", [(1e30, 1e30), (1e36, 1e36), (1e38, 2e37), (1e38, 4e37), (3.3e38, 4e37)])
def test_temperatures_up_to_the_largest(T, gain, dtype):
    """log2(e) / T near fp32's smallest numbers, logits as large as T: the weights still count."""
    lg, ql, d, u = make(40, 4, 300, 13, dtype, spread=1.0)
    lg, ql = ((x.float().clamp(-4, 4) * gain).to(dtype) for x in (lg, ql))
    lg[::3, :, ::7] = -float("inf")
    check(lg, d, u, ql, torch.full((40,), T))
    check(lg, d, u * 2.0 ** -5, None, torch.full((40,), T))
