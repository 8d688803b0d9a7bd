"""GPU tests of calls made from two threads at once on one stream, and of first calls under
graph capture."""

import threading

import numpy as np
import pytest

import workloads as wlm
from tests.gpu_helpers import bits, host, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsf():
    import newton_schulz_flat_amd as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def at_once(works):
    """Runs the functions in threads that start together; the first failure is raised."""
    gate, failures = threading.Barrier(len(works)), []

    def run(work):
        try:
            gate.wait()
            work()
        except BaseException as e:  # noqa: BLE001 - handed to the test
            failures.append(e)
    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failures:
        raise failures[0]


def test_norms_from_two_threads_on_one_stream(nsf, torch):
    """Lists of two launches each, of one length and of different ones, each thread with its
    own records and the stream's default workspace: the bits of the calls made alone."""
    say("norms from two threads")
    for sizes in ([400000, 400000], [3_000_000, 70000]):
        lists = [nsf.tensor_list([torch.randn(n, device="cuda") * (k + 1)])
                 for k, n in enumerate(sizes)]
        alone = [nsf.clip_state("cuda") for _ in sizes]
        for tl, c in zip(lists, alone):
            nsf.muon_grad_norm(tl, 1.0, c)
        records = [[nsf.clip_state("cuda") for _ in range(200)] for _ in sizes]
        torch.cuda.synchronize()
        at_once([lambda tl=tl, cs=cs: [nsf.muon_grad_norm(tl, 1.0, c) for c in cs]
                 for tl, cs in zip(lists, records)])
        torch.cuda.synchronize()
        for c, cs in zip(alone, records):
            assert all(torch.equal(x.record, c.record) for x in cs)


def test_clipped_steps_from_two_threads_on_one_stream(nsf, torch):
    """Clipped steps of two descriptor sets, each thread with its own buffers and the
    stream's default workspace: the bits of the same calls made one thread after the other."""
    say("clipped steps from two threads")
    table = nsf.group_table([(0.02, 0.01, 0.95, True)], "cuda")
    clip = nsf.clip_state("cuda")
    nsf.clip_coef(clip).fill_(0.5)

    def buffers():
        out = []
        for seed in (61, 62):
            wl = wlm.small_mixed(seed, count=4, max_side=300, param_dtype="bf16")
            out.append((wl.descs, *wlm.make_tensors(wl, "cuda", momentum_std=1e-3)))
        return out

    def steps(descs, params, grads, mom):
        for _ in range(20):
            nsf.muon_step_clipped(params, grads, mom, descs, table, clip)
    want, got = buffers(), buffers()
    for b in want:
        steps(*b)
    torch.cuda.synchronize()
    at_once([lambda b=b: steps(*b) for b in got])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a[1:], b[1:]):
            assert np.array_equal(bits(host(x)), bits(host(y)))


def test_first_clipped_step_is_made_outside_capture(nsf, torch):
    """Under capture a first call with a descriptor set is refused and leaves the capture
    whole; after one call outside it is captured, and every replay is an eager call."""
    say("first clipped step under capture")
    wl = wlm.small_mixed(77, count=3, max_side=200, param_dtype="f32")
    params, grads, mom = wlm.make_tensors(wl, "cuda", momentum_std=1e-3)
    table = nsf.group_table([(0.02, 0.01, 0.95, True)], "cuda")
    clip = nsf.clip_state("cuda")
    cws = torch.empty(nsf.muon_clip_workspace_bytes([grads]), dtype=torch.uint8, device="cuda")
    ws = torch.empty(nsf.muon_workspace_bytes(wl.descs), dtype=torch.uint8, device="cuda")

    def step(p, m):
        nsf.muon_grad_norm([grads], 0.5, clip, workspace=cws)
        nsf.muon_step_clipped(p, grads, m, wl.descs, table, clip, workspace=ws)
    p1, m1, p2, m2 = params.clone(), mom.clone(), params.clone(), mom.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(nsf.MuonError, match="outside graph capture"):
            step(p1, m1)
        grads.mul_(2.0)
    assert torch.equal(p1, params) and torch.equal(m1, mom)
    step(params.clone(), mom.clone())       # the plan
    torch.cuda.synchronize()
    whole = torch.cuda.CUDAGraph()
    with torch.cuda.graph(whole):
        step(p1, m1)
    for rep in range(3):
        graph.replay()                      # the capture that went on after the refusal
        whole.replay()
        torch.cuda.synchronize()
        step(p2, m2)
        torch.cuda.synchronize()
        assert np.array_equal(bits(host(p1)), bits(host(p2))), rep
        assert np.array_equal(bits(host(m1)), bits(host(m2))), rep
