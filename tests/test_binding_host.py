"""Host tests of what the binding does around a call: which workspace it takes,
which device it launches on and which tensors it refuses.  The library and the
GPU are stand-ins here; nothing is computed."""

import contextlib
import ctypes
import threading
import time
import types

import pytest

import newton_schulz_flat_amd as nsf


class Library:
    """Stands in for the library: every call is noted with the device that was current."""

    def __init__(self, gpu, pause=0.0):
        self.gpu, self.pause, self.calls, self.events = gpu, pause, [], []

    def __getattr__(self, name):
        if not name.startswith("muon_"):
            raise AttributeError(name)

        def call(*args):
            self.events.append((name, "begins", threading.get_ident()))
            time.sleep(self.pause)
            self.calls.append((name, self.gpu["device"], args))
            self.events.append((name, "ends", threading.get_ident()))
            return 0
        return call


@pytest.fixture
def gpu(monkeypatch):
    """Two GPUs of which device 0 is current; stream handles are 100 + device."""
    import torch
    state = {"device": 0, "capturing": None}

    @contextlib.contextmanager
    def device(d):
        before = state["device"]
        state["device"] = d if isinstance(d, int) else torch.device(d).index
        try:
            yield
        finally:
            state["device"] = before

    def stream(d=None):
        index = state["device"] if d is None else d if isinstance(d, int) else torch.device(d).index
        return types.SimpleNamespace(cuda_stream=100 + index, device_index=index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                        lambda: state["capturing"] == state["device"])
    monkeypatch.setattr(nsf, "_current_stream", lambda index: 100 + index)
    monkeypatch.setattr(nsf, "_require", lambda t, name, dtypes: None)
    monkeypatch.setattr(nsf, "_require_clip", lambda clip, device: None)
    real_empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real_empty(*a, **kw))
    for name in ("_workspaces", "_clip_workspaces"):
        monkeypatch.setattr(nsf, name, {})
    return state


class Tensor:
    """What the binding asks of a tensor; device memory that is never touched."""

    def __init__(self, numel, dtype, device=0, at=1 << 40, shape=None):
        import torch
        self.n, self.dtype, self.at = numel, dtype, at
        self.device = torch.device("cuda", device)
        self.shape = shape or (numel,)
        self.is_cuda = True

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        import torch
        return torch.empty(0, dtype=self.dtype).element_size()

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


def record(device=0):
    import torch
    return types.SimpleNamespace(record=Tensor(2, torch.float64, device),
                                 device=torch.device("cuda", device))


DESCS = [(0, 8, 16)]


def step_buffers(**devices):
    """Buffers of a step on the matrix of DESCS, on device 0 but for those named."""
    import torch
    at = lambda name: devices.get(name, devices.get("all", 0))
    return dict(params=Tensor(128, torch.float32, at("params")),
                grads=Tensor(128, torch.float32, at("grads")),
                momentum=Tensor(128, torch.float32, at("momentum")),
                u_out=Tensor(128, torch.float32, at("u_out")),
                groups=Tensor(4, torch.int32, at("groups"), shape=(1, 4)),
                model_copy=Tensor(128, torch.bfloat16, at("model_copy")),
                workspace=Tensor(1 << 20, torch.uint8, at("workspace")))


def calls(b, workspace=True):
    """Every entry point that launches a Muon step or a part of it."""
    ws = dict(workspace=b["workspace"]) if workspace else {}
    clip = record(b["grads"].device.index)
    p, g, m = b["params"], b["grads"], b["momentum"]
    every = {
        "muon_step": lambda: nsf.muon_step(p, g, m, DESCS, 0.1, 0.1, 0.9, **ws),
        "muon_step_grouped": lambda: nsf.muon_step_grouped(p, g, m, DESCS, b["groups"],
                                                           model_copy=b["model_copy"], **ws),
        "muon_step_clipped": lambda: nsf.muon_step_clipped(p, g, m, DESCS, b["groups"], clip,
                                                           model_copy=b["model_copy"], **ws),
        "muon_orthogonalize": lambda: nsf.muon_orthogonalize(g, b["u_out"], DESCS, **ws),
    }
    if workspace:
        every.update({
            "muon_step_noalloc": lambda: nsf.muon_step_noalloc(p, g, m, DESCS, 0.1, 0.1, 0.9),
            "muon_momentum": lambda: nsf.muon_momentum(g, m, b["u_out"], DESCS, 0.9),
            "muon_apply": lambda: nsf.muon_apply(p, g, DESCS, 0.1, 0.1),
        })
    return every


# ------------------------------------------------- two threads on one stream

def overlap(events):
    """Whether a call began while another thread's was under way."""
    open_calls = set()
    for _, what, who in events:
        if what == "begins":
            if open_calls:
                return True
            open_calls.add(who)
        else:
            open_calls.discard(who)
    return False


def from_two_threads(call):
    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def default_workspace_calls():
    import torch
    tensors = nsf.tensor_list([torch.ones(1000)])
    every = calls(step_buffers(), workspace=False)
    every["muon_grad_norm"] = lambda: nsf.muon_grad_norm(tensors, 1.0, record())
    return every


@pytest.mark.parametrize("name", ["muon_grad_norm", "muon_step", "muon_step_grouped",
                                  "muon_step_clipped", "muon_orthogonalize"])
def test_calls_that_share_a_default_workspace_do_not_overlap(gpu, monkeypatch, name):
    """A call is several launches that pass results on through the workspace: two threads
    on one stream share the default one, and one call's launches must all be
    enqueued before the other's first."""
    lib = Library(gpu, pause=0.05)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    monkeypatch.setattr(nsf, "muon_workspace_bytes", lambda descs, mode="bf16": 4096)
    monkeypatch.setattr(nsf, "muon_clip_workspace_bytes", lambda tensors: 4096)
    call = default_workspace_calls()[name]
    call()                         # the workspace exists from here on
    lib.events.clear()
    from_two_threads(call)
    assert [n for n, _, _ in lib.calls] == [name] * 3
    assert not overlap(lib.events)


def test_calls_with_their_own_workspaces_may_overlap(gpu, monkeypatch):
    """Nothing waits where the caller names the workspace."""
    lib = Library(gpu, pause=0.2)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    from_two_threads(calls(step_buffers())["muon_step"])
    assert overlap(lib.events)


# ------------------------------------------------------------ another device

EVERY = ["muon_step", "muon_step_grouped", "muon_step_clipped", "muon_orthogonalize",
         "muon_step_noalloc", "muon_momentum", "muon_apply"]


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", EVERY)
def test_steps_launch_on_the_device_of_their_tensors(gpu, monkeypatch, name, index):
    """Kernels go to the current device, plans belong to it: it has to be the tensors' while
    the library runs, and what it was before afterwards."""
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    calls(step_buffers(all=index))[name]()
    (called, current, args), = lib.calls
    stream = getattr(args[-1], "value", args[-1])
    assert (called, current, stream) == (name, index, 100 + index)
    assert gpu["device"] == 0


@pytest.mark.parametrize("name", ["muon_step", "muon_step_clipped", "muon_orthogonalize"])
def test_default_workspace_refused_under_capture_on_another_device(gpu, monkeypatch, name):
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    monkeypatch.setattr(nsf, "muon_workspace_bytes", lambda descs, mode="bf16": 4096)
    gpu["capturing"] = 1
    with pytest.raises(RuntimeError, match="explicit workspace"):
        calls(step_buffers(all=1), workspace=False)[name]()
    assert not lib.calls
    calls(step_buffers(all=1))[name]()      # one of its own is fine
    assert len(lib.calls) == 1


# name -> the buffers that its calls take beside grads
TAKES = {"muon_step": ["params", "momentum", "workspace"],
         "muon_step_grouped": ["params", "momentum", "groups", "model_copy", "workspace"],
         "muon_step_clipped": ["params", "momentum", "groups", "model_copy", "workspace"],
         "muon_orthogonalize": ["u_out", "workspace"],
         "muon_step_noalloc": ["params", "momentum"],
         "muon_momentum": ["momentum", "u_out"],
         "muon_apply": ["params"]}


@pytest.mark.parametrize("name,odd", [(n, k) for n in EVERY for k in TAKES[n]])
def test_steps_refuse_tensors_of_two_devices(gpu, monkeypatch, name, odd):
    """A kernel that reads another device's memory faults."""
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    with pytest.raises(ValueError, match="is on cuda:1"):
        calls(step_buffers(**{odd: 1}))[name]()
    assert not lib.calls


@pytest.mark.parametrize("name", ["muon_step", "muon_step_grouped", "muon_step_clipped",
                                  "muon_orthogonalize"])
def test_steps_refuse_a_workspace_in_host_memory(gpu, monkeypatch, name):
    import torch
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    b = step_buffers()
    b["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        calls(b)[name]()
    b["workspace"] = Tensor(1 << 20, torch.uint8)
    b["workspace"].is_contiguous = lambda: False
    with pytest.raises(ValueError, match="contiguous"):
        calls(b)[name]()
    b["workspace"] = Tensor(1 << 18, torch.float32)     # of any type
    calls(b)[name]()
    assert len(lib.calls) == 1


# ------------------------------------------------------------ short buffers

@pytest.mark.parametrize("name,short", [(n, k) for n in EVERY for k in ("momentum", "u_out")
                                        if k in TAKES[n]])
def test_steps_refuse_a_state_buffer_that_ends_early(gpu, monkeypatch, name, short):
    """The library's own check sees the shorter of the state buffers: a matrix that
    leaves it is out of bounds.  A longer one, or one that ends behind the last matrix, is fine."""
    import os
    if not os.path.exists(nsf.LIB_PATH):
        from newton_schulz_flat_amd import build
        build.build()
    b = step_buffers()
    for k, t in enumerate(b.values()):
        t.at = (k + 1) << 40
    b[short].n = 127
    with pytest.raises(nsf.MuonError, match="OUT_OF_BOUNDS"):
        calls(b)[name]()
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    b["params"].n = b["model_copy"].n = 999
    for own, other in ((200, 128), (128, 200)):
        b[short].n, b["grads"].n = own, other
        calls(b)[name]()
        assert 128 in lib.calls[-1][2]


# ------------------------------------------------------------ kept lists

def moved_by(name, t):
    import torch
    if name == "data":
        t.data = torch.ones(t.numel())
    elif name == "set_":
        t.set_(torch.ones(t.numel()))
    elif name == "resize_":
        t.resize_(10 * t.numel())
    elif name == "storage freed":
        t.untyped_storage().resize_(0)
    elif name == "another part":
        t.data = t.data[8:]


@pytest.mark.parametrize("how", ["data", "set_", "resize_", "storage freed", "another part"])
def test_a_kept_list_refuses_tensors_that_moved(gpu, monkeypatch, how):
    """A list holds addresses; the tensors' memory may have been freed since."""
    import torch
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    monkeypatch.setattr(nsf, "muon_clip_workspace_bytes", lambda tensors: 4096)
    still, t = torch.ones(64), torch.ones(1000)
    kept, out = nsf.tensor_list([still, t]), nsf.tensor_list([torch.ones(64), torch.ones(1000)])
    clip = record()
    clip.device = kept.device

    def every():
        return [lambda: nsf.muon_grad_norm(kept, 1.0, clip), lambda: nsf.muon_clip_grads(kept, clip),
                lambda: nsf.muon_clip_grads(kept, clip, out=out),
                lambda: nsf.muon_clip_grads(out, clip, out=kept)]
    monkeypatch.setattr(nsf, "_current_stream", lambda index: 100)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=100))
    still.mul_(2)                  # new values are fine
    for call in every():
        call()
    assert len(lib.calls) == 4
    moved_by(how, t)
    for call in every():
        with pytest.raises(ValueError, match=r"tensors\[1\] has moved"):
            call()
    assert len(lib.calls) == 4
    nsf.muon_clip_grads([still], clip)          # a list made by the call is of this moment
    assert len(lib.calls) == 5


def test_a_kept_list_keeps_the_memory_it_points_to(gpu):
    """So that no other tensor can come to lie at an address of the list, unnoticed."""
    import torch
    t = torch.full((100000,), 7.0)
    kept = nsf.tensor_list([t])
    t.data = torch.ones(100000)
    others = [torch.zeros(100000) for _ in range(20)]
    assert kept.array[0].data not in [o.data_ptr() for o in others]
    assert ctypes.c_float.from_address(kept.array[0].data).value == 7.0


# ------------------------------------------------------------ descriptors

@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("name", EVERY)
def test_descriptors_from_an_iterator(gpu, monkeypatch, name, workspace):
    """An iterator can be read once; the call has to see every descriptor all the same."""
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    sized = []
    monkeypatch.setattr(nsf, "muon_workspace_bytes",
                        lambda descs, mode="bf16": sized.append(len(list(descs))) or 4096)
    every = calls(step_buffers(), workspace=workspace)
    if name not in every:
        return
    monkeypatch.setitem(globals(), "DESCS", iter([(0, 8, 4), (32, 4, 8), (64, 2, 2)]))
    every[name]()
    (_, _, args), = lib.calls
    at = next(k for k, a in enumerate(args) if isinstance(a, ctypes.Array))
    assert args[at + 1] == len(args[at]) == 3
    assert [d.offset for d in args[at]] == [0, 32, 64]
    assert sized in ([], [3])


# ------------------------------------------------ 8-bit matrices and stacks

def on_gpu(device, *shape, dtype=None):
    """A tensor that says that it is on a GPU."""
    import torch

    class OnGpu(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: torch.device("cuda", self.at))

        def get_device(self):
            return self.at
    t = torch.zeros(*shape, dtype=dtype or torch.float32).as_subclass(OnGpu)
    t.at = device
    return t


MATRIX_TAKES = {"muon_fp8_cast": ["codes", "scales", "codes_t", "scales_t"],
                "muon_fp8_matmul": ["a", "a_scales", "b_scales", "out", "workspace"],
                "muon_orthogonalize_stack": ["out", "workspace"]}


def matrix_call(name, own=True, **devices):
    """A call of one of these entry points with everything on device 0 but for what is named."""
    import torch
    at = lambda what: devices.get(what, devices.get("all", 0))
    e4m3 = torch.float8_e4m3fn
    ws = dict(workspace=on_gpu(at("workspace"), 4096, dtype=torch.uint8)) if own else {}
    if name == "muon_fp8_cast":
        return nsf.muon_fp8_cast(on_gpu(at("x"), 8, 256), on_gpu(at("codes"), 8, 256, dtype=e4m3),
                                 on_gpu(at("scales"), 8, 2), on_gpu(at("codes_t"), 256, 8, dtype=e4m3),
                                 on_gpu(at("scales_t"), 256, 1))
    if name == "muon_fp8_matmul":
        return nsf.muon_fp8_matmul(on_gpu(at("a"), 8, 256, dtype=e4m3), on_gpu(at("a_scales"), 8, 2),
                                   on_gpu(at("b"), 130, 256, dtype=e4m3), on_gpu(at("b_scales"), 2, 2),
                                   on_gpu(at("out"), 8, 130), **ws)
    return nsf.muon_orthogonalize_stack(on_gpu(at("x"), 2, 8, 16), on_gpu(at("out"), 2, 8, 16), **ws)


@pytest.fixture
def matrices(gpu, monkeypatch):
    lib = Library(gpu)
    monkeypatch.setattr(nsf, "load_library", lambda: lib)
    monkeypatch.setattr(nsf, "muon_fp8_workspace_bytes", lambda m, n, k: 4096)
    monkeypatch.setattr(nsf, "muon_stack_workspace_bytes", lambda x: 4096)
    monkeypatch.setattr(nsf, "_call_workspaces", {})
    return lib


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", MATRIX_TAKES)
def test_matrices_launch_on_the_device_of_their_tensors(gpu, matrices, name, index):
    for workspace in (True, False):
        matrices.calls.clear()
        matrix_call(name, workspace, all=index)
        (called, current, args), = matrices.calls
        assert (called, current, getattr(args[-1], "value", args[-1])) == (name, index, 100 + index)
        assert gpu["device"] == 0


@pytest.mark.parametrize("name,odd", [(n, k) for n in MATRIX_TAKES for k in MATRIX_TAKES[n]])
def test_matrices_refuse_tensors_of_two_devices(gpu, matrices, name, odd):
    with pytest.raises(ValueError, match="is on cuda:"):
        matrix_call(name, **{odd: 1})
    assert not matrices.calls


@pytest.mark.parametrize("name", ["muon_fp8_matmul", "muon_orthogonalize_stack"])
def test_matrices_default_workspace(gpu, matrices, name):
    """Refused under capture, one per device and stream otherwise; two threads on one stream
    take turns."""
    gpu["capturing"] = 1
    with pytest.raises(RuntimeError, match="explicit workspace"):
        matrix_call(name, False, all=1)
    assert not matrices.calls
    matrix_call(name, True, all=1)
    matrix_call(name, False)                  # another device captures
    assert len(matrices.calls) == 2 and len(nsf._call_workspaces) == 1
    gpu["capturing"] = None
    matrix_call(name, False, all=1)
    assert len(nsf._call_workspaces) == 2
    matrices.pause = 0.05
    matrices.events.clear()
    from_two_threads(lambda: matrix_call(name, False))
    assert len(matrices.calls) == 5 and not overlap(matrices.events)
