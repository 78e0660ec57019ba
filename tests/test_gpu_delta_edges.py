"""The delta rule and the norm of queries and keys where calls meet or sizes end: several host threads, two
captured graphs at once, the widest values, very many heads, decays that grow."""
import threading

import pytest
import torch

from _selective_ref import HALF_STEP, REL, close
from test_gpu_delta import BF16, F16, F32, NAMES, check_bwd, cuda, gpu, gpu_bwd, grads, make, plain, plain_bwd, ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F32, BF16])
def test_widest_values(t):
    k = make(1, 70, 1, 1, 128, 1024, t)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    check_bwd(k)


@pytest.mark.parametrize("t", [F32, F16])
def test_very_many_heads(t):
    """More heads than a grid's second dimension holds."""
    k = make(520, 3, 128, 2, 8, 8, t)
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    check_bwd(k)
    c, state = cuda(k), k["h0"].cuda()
    y = torch.stack([ssd().delta_rule_step(*(c[n][:, i].contiguous() for n in NAMES), state) for i in range(3)], 1)
    close(y, ry, "tokens")
    close(state, rfin, "state")


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_growing_states(t):
    """Most steps have the same factor exp(0.02), and its error is the same at each: exp in 32 bits is off by up to 2 units in
    the last place (2^-22), and nothing takes the growing parts out, so over 130 steps the state is off by 130 x 2^-22."""
    k = make(2, 130, 2, 1, 64, 64, t)
    k["g"] = k["g"].abs().clamp(max=0.02)
    dy, df = grads(k)
    y, fin = gpu(cuda(k))
    got = {"y": y, "final": fin, **gpu_bwd(cuda(k), dy.cuda(), df.cuda())}
    ry, rfin = plain(k)
    want = {"y": ry, "final": rfin, **plain_bwd(k, dy, df)}
    for n, w in want.items():
        error = (got[n].double().cpu() - w).norm() / w.norm()
        assert error <= HALF_STEP[got[n].dtype] + REL + 130 * 2.0 ** -22, (n, error.item())


@pytest.mark.parametrize("t", [F32, F16, BF16])
def test_decay_of_plus_infinity(t):
    """No use, but no finite wrong answer either."""
    k = make(1, 70, 1, 1, 64, 64, t)
    k["g"][:] = float("inf")
    y, fin = gpu(cuda(k))
    assert not torch.isfinite(y[:, 1:]).any() and not torch.isfinite(fin).any()


def work(k, dy, df, f):
    """Every call once; a list of results."""
    state = k["h0"].clone()
    one = [k[n][:, 0].contiguous() for n in NAMES]
    qn, kn = ssd().qk_norm(k["q"], k["k"], norm="l2", freqs=f)
    y, fin = ssd().delta_rule(qn, kn, *(k[n] for n in NAMES[2:]), initial_states=k["h0"], return_final_state=True)
    b = ssd().delta_rule_bwd(qn, kn, *(k[n] for n in NAMES[2:]), dy, dfinal=df, initial_states=k["h0"])
    n = ssd().qk_norm_bwd(b["dq"], b["dk"], k["q"], k["k"], norm="l2", freqs=f)
    return [qn, kn, y, fin, *b.values(), *n.values(), ssd().delta_rule_step(*one, state), state]


def sets():
    """Two of one type and other sizes, one of another type, one cut into segments."""
    out = []
    for i, (shape, t) in enumerate([((2, 150, 4, 2, 128, 128), BF16), ((3, 100, 4, 2, 64, 64), BF16), ((2, 90, 2, 2, 40, 24), F32),
                                    ((1, 2000, 1, 1, 128, 64), F16)]):
        k = cuda(make(*shape, t, seed=i))
        dy, df = grads(k)
        out.append((k, dy.cuda(), df.cuda(), torch.ones(shape[4] // 2, device="cuda") / (1 + i)))
    return out


def test_host_threads():
    inputs = sets()
    want = [work(*i) for i in inputs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(inputs))

    def run(i):
        s = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = work(*inputs[i])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_at_once():
    inputs = sets()
    want = [work(*i) for i in inputs]
    torch.cuda.synchronize()
    graphs, results = [], []
    for i in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(work(*i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(results, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))
