"""GPU tests of the preference loss where its offsets are not in order: read as their
running largest, cut to the rows there are, so that no two sequences share a row."""
import pytest
import torch

import boolean_weight_amd as bw
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def in_order(off, T):
    return off.long().clamp(0, T).cummax(0).values.to(torch.int32)


def run(off, lp, refl, mean):
    pairs, T = len(off) // 2, len(lp)
    loss, dlogp = torch.full((pairs,), -5.0, device=DEV), torch.full((T,), -7.0, device=DEV)
    d = bw.mbok_preference_desc_init(0.3, 0.1, mean=mean, vocab=10)
    bw.mbok_preference(d, off.to(DEV), lp.to(DEV), loss, ref_logp=refl.to(DEV), dlogp=dlogp)
    return loss.cpu(), dlogp.cpu()


def test_decrease_across_a_pair():
    """0 8 | 5 9 10: the second pair begins at 8."""
    say("preference offsets across a pair")
    lp, refl = torch.arange(10.0), torch.zeros(10)
    got = run(torch.tensor([0, 8, 5, 9, 10], dtype=torch.int32), lp, refl, True)
    want = run(torch.tensor([0, 8, 8, 9, 10], dtype=torch.int32), lp, refl, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # rows 0 .. 7 chosen of the first pair, its rejected sequence empty; 8 and 9 alone
    d = got[1]
    assert (d[:8] == d[0]).all() and d[0] < 0 and d[8] < 0 and d[9] == -d[8]


# one wavefront's pass over the offsets, several; either side of the two ways to find a
# pair's start; several passes of the second
@pytest.mark.parametrize("pairs", [1, 2, 31, 33, 700, 1023, 1024, 1025, 2049, 5000])
@pytest.mark.parametrize("kind", ["ordered", "dips", "any"])
def test_offsets_are_read_in_order(pairs, kind):
    say(f"preference offsets pairs={pairs} {kind}")
    T = 3 * pairs + 7
    gen = torch.Generator().manual_seed(pairs)
    lp, refl = torch.randn(T, generator=gen), torch.randn(T, generator=gen)
    off = torch.randint(0, T + 1, (2 * pairs + 1,), generator=gen).sort().values
    if kind == "dips":  # one in five lies up to 40 rows back, some below 0
        dip = torch.rand(2 * pairs + 1, generator=gen) < 0.2
        off = off - dip * torch.randint(0, 41, (2 * pairs + 1,), generator=gen)
    elif kind == "any":  # a few early ones past the end of what follows
        at = torch.randint(0, 2 * pairs + 1, (3,), generator=gen)
        off[at] = torch.tensor([-(1 << 31), T // 2, (1 << 31) - 1])
    off = off.to(torch.int32)
    clean = in_order(off, T)
    got, want = run(off, lp, refl, True), run(clean, lp, refl, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and those against the formula, in float64 (see test_gpu_policy.py)
    diff = torch.cat([torch.zeros(1, dtype=torch.float64),
                      (lp.double() - refl.double()).cumsum(0)])
    o = clean.long()
    size = (o[1:] - o[:-1])
    score = ((diff[o[1:]] - diff[o[:-1]]) / size.clamp_min(1)).view(pairs, 2)
    d = bw.mbok_preference_desc_init(0.3, 0.1)
    beta, s = float(d.beta), float(d.smoothing)
    h = beta * (score[:, 0] - score[:, 1])
    softplus = torch.nn.functional.softplus
    loss = (1 - s) * softplus(-h) + s * softplus(h)
    # the running sums of up to 15007 terms lose 2^-53 of some hundreds each
    assert ((got[0].double() - loss).abs() <= 2.0 ** -23 * loss + 2.0 ** -30).all()
    dh = beta * (s * torch.sigmoid(h) - (1 - s) * torch.sigmoid(-h))
    row = torch.arange(T)
    seq = torch.searchsorted(o[1:].contiguous(), row, right=True)
    inside = (row >= o[0]) & (seq < 2 * pairs)
    seq = seq.clamp_max(2 * pairs - 1)
    want = torch.stack([dh, -dh], 1).view(-1)[seq] / size[seq].clamp_min(1)
    g = got[1].double()
    assert ((g - want).abs() <= 2.0 ** -23 * want.abs() + 2.0 ** -30)[inside].all()
    assert (g[~inside] == -7).all()


def test_many_pairs_captured():
    """The start's kernel and the loss's in a graph, replayed on other offsets."""
    say("preference offsets captured")
    pairs, T = 1500, 4000
    gen = torch.Generator().manual_seed(1)
    lp = torch.randn(T, generator=gen).to(DEV)
    offs = [torch.randint(0, T + 1, (2 * pairs + 1,), generator=gen).sort().values.int().to(DEV)
            for _ in range(4)]
    offs[2][100:200] = 5
    off, d = offs[0].clone(), bw.mbok_preference_desc_init(0.2, vocab=10)
    loss, dlogp = torch.zeros(pairs, device=DEV), torch.zeros(T, device=DEV)

    def step():
        bw.mbok_preference(d, off, lp, loss, dlogp=dlogp)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for o in offs:
        off.copy_(o), dlogp.zero_()
        graph.replay()
        got = loss.clone(), dlogp.clone()
        dlogp.zero_(), loss.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], loss) and torch.equal(got[1], dlogp)
