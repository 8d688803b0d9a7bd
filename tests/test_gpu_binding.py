"""GPU tests of calls made from two threads at once on one stream."""

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
