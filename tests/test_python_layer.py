"""The Python layer without a GPU: host tensors that say they are CUDA tensors,
a library that records its calls, and streams that are only handles."""
import contextlib

import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import api


class Pretend(torch.Tensor):
    """A host tensor on "cuda:index"."""
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def record_stream(self, stream):
        World.kept.append((self.data_ptr(), stream.cuda_stream))


def pretend(*shape, dtype=torch.int32, index=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Pretend)
    t.index = index
    return t


class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device_index = handle, index

    def record_event(self):
        World.events.append(self.cuda_stream)
        return len(World.events) - 1

    def wait_event(self, event):
        World.waits.append((self.cuda_stream, event))


class World:
    """What the fake CUDA saw."""
    current = 7           # handle of the current stream
    captured = set()      # handles of the streams under capture
    device = 0            # the current device
    zeroed = []           # (address, handle of the stream that the zeroing is ordered on)
    kept = []
    events, waits = [], []    # the streams that events were recorded on; (stream, event waited for)
    calls = []            # (name, arguments)


class Library:
    need = 4096

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: Library.need
        def call(*a):
            World.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    World.current, World.device, World.zeroed, World.kept, World.calls, World.captured, Library.need = 7, 0, [], [], [], set(), 4096
    World.events, World.waits = [], []

    @contextlib.contextmanager
    def on(stream):
        before, World.current = World.current, stream.cuda_stream
        yield
        World.current = before

    def zeros(n, dtype, device):
        t = pretend(n, dtype=dtype, index=torch.device(device).index)
        World.zeroed.append((t.data_ptr(), World.current))
        return t

    monkeypatch.setattr(api._lib, "load", lambda: Library())
    monkeypatch.setattr(api, "_default_ws", {})
    monkeypatch.setattr(api, "_gpus", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: World.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: World.current in World.captured, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: World.device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: World.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(World.current))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    real = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: real(*a, **kw) if device is None else zeros(*a, device=device, **kw))
    return World


def attend(stream=None, workspace=None, **edit):
    t = dict(q=pretend(2, 4, 64, dtype=torch.bfloat16), cache=pretend(3, 2, 1, 18 * 64, dtype=torch.uint8), seq_lens=pretend(2),
             block_table=pretend(2, 5), k_scale=pretend(1, dtype=torch.float32), v_scale=pretend(1, dtype=torch.float32),
             out=pretend(2, 4, 64, dtype=torch.bfloat16))
    t.update(edit)
    w8.kv4_attention(**t, workspace=workspace, stream=stream)
    return World.calls[-1][1]


def attend_fp8(stream=None, workspace=None):
    e4m3 = lambda *n: pretend(*n, dtype=torch.uint8)  # noqa: E731
    w8.fp8_kv_decode_attention(pretend(2, 4, 128, dtype=torch.bfloat16), e4m3(2, 9, 2, 128), e4m3(2, 9, 2, 128), pretend(2),
                               pretend(1, dtype=torch.float32), pretend(1, dtype=torch.float32),
                               pretend(2, 4, 128, dtype=torch.bfloat16), workspace=workspace, stream=stream)
    return World.calls[-1][1]


def matmul(stream=None, workspace=None):
    one = pretend(1, dtype=torch.float32)
    w8.scaled_mm(pretend(4, 32, dtype=torch.int8), pretend(8, 32, dtype=torch.int8), one, one, pretend(4, 8, dtype=torch.float16),
                 workspace=workspace, stream=stream)
    return World.calls[-1][1]


def quantising_matmul(stream=None, workspace=None):
    w8.quant_scaled_mm(pretend(4, 32, dtype=torch.bfloat16), pretend(8, 32, dtype=torch.int8), pretend(1, dtype=torch.float32),
                       pretend(4, 8, dtype=torch.bfloat16), workspace=workspace, stream=stream)
    return World.calls[-1][1]


def quantise(stream=None, workspace=None):
    w8.scaled_quant(pretend(4, 32, dtype=torch.bfloat16), pretend(4, 32, dtype=torch.int8), pretend(1, dtype=torch.float32),
                    per_token=False, workspace=workspace, stream=stream)
    return World.calls[-1][1]


CALLS = [attend, attend_fp8, matmul, quantising_matmul, quantise]


@pytest.mark.parametrize("call", CALLS)
def test_default_workspaces_go_by_the_stream_that_the_call_runs_on(world, call):
    """Two explicit streams under one current stream: a buffer each, zeroed on
    the stream whose kernel reads it, and again the same one the next time."""
    buffers = {}
    for handle in (21, 22):
        args = call(stream=Stream(handle))
        address, ordered_on = world.zeroed[-1]
        assert address in args and args[-1] == handle and ordered_on == handle
        buffers[handle] = address
    assert len(set(buffers.values())) == 2 and len(world.zeroed) == 2
    for handle in (22, 21):
        assert buffers[handle] in call(stream=Stream(handle))
    world.current = 21
    assert buffers[21] in call()                 # the same stream, as the current one
    world.current = 9
    call()
    assert len(world.zeroed) == 3 and world.zeroed[-1][1] == 9


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("own", [False, True])
def test_a_workspace_grows_on_the_stream_of_the_call(world, call, own):
    if own and call is quantise:
        pytest.skip("takes tensors only")
    ws = w8.Workspace(device="cuda:0") if own else None
    call(stream=Stream(31), workspace=ws)
    old = world.zeroed[-1][0]
    Library.need = 1 << 20
    api._kv4_attention_need.cache_clear()
    args = call(stream=Stream(31), workspace=ws)
    assert world.zeroed[-1][0] in args and world.zeroed[-1][1] == 31
    assert (old, 31) in world.kept               # not given away while the call before may run
    api._kv4_attention_need.cache_clear()


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("explicit", [False, True])
def test_scratch_first_made_in_a_capture_is_the_graphs_own(world, call, explicit):
    """Its zeros come with that graph's replay alone: another graph, or a call
    outside, gets a buffer of its own."""
    world.current = 7 if explicit else 41
    stream = Stream(41) if explicit else None
    world.captured = {41}
    call(stream=stream)
    call(stream=stream)
    assert [on for _, on in world.zeroed] == [41, 41]
    world.captured = set()
    args = call(stream=stream)
    assert len(world.zeroed) == 3 and world.zeroed[2][0] in args
    call(stream=stream)
    assert len(world.zeroed) == 3


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("own", [False, True])
def test_a_captured_buffer_outlives_growth(world, call, own):
    if own and call is quantise:
        pytest.skip("takes tensors only")
    world.current = 51
    ws = w8.Workspace(4096, device="cuda:0") if own else None
    call(workspace=ws)
    keeper = ws if own else next(iter(api._default_ws.values()))
    first = keeper.buf
    world.captured = {51}
    assert first.data_ptr() in call(workspace=ws)            # the graph has its address
    call(workspace=ws)
    Library.need = 1 << 20
    api._kv4_attention_need.cache_clear()
    args = call(workspace=ws)                                # too small: the graph's own, zeroed by it
    assert world.zeroed[-1][0] in args and keeper.buf is first
    world.captured = set()
    args = call(workspace=ws)
    assert keeper.buf is not first and keeper.buf.data_ptr() in args
    assert [b is first for b in keeper._captured] == [True]
    api._kv4_attention_need.cache_clear()


def f32(*n, index=0):
    return pretend(*n, dtype=torch.float32, index=index)


def i8(*n, index=0):
    return pretend(*n, dtype=torch.int8, index=index)


def b16(*n, index=0):
    return pretend(*n, dtype=torch.bfloat16, index=index)


def i64(*n, index=0):
    return pretend(*n, dtype=torch.int64, index=index)


def u8(*n, index=0):
    return pretend(*n, dtype=torch.uint8, index=index)


# every entry point with its tensors as (maker, shape); the last positions of some are workspaces
ENTRIES = {
    "scaled_quant": (lambda x, q, s, w: w8.scaled_quant(x, q, s, per_token=False, workspace=w),
                     [(b16, (4, 32)), (i8, (4, 32)), (f32, (1,)), (u8, (4096,))]),
    "scaled_dequant": (w8.scaled_dequant, [(i8, (4, 32)), (f32, (1,)), (b16, (4, 32))]),
    "scaled_mm": (w8.scaled_mm, [(i8, (4, 32)), (i8, (8, 32)), (f32, (4,)), (f32, (8,)), (b16, (4, 8)), (u8, (4096,))]),
    "quant_scaled_mm": (w8.quant_scaled_mm, [(b16, (4, 32)), (i8, (8, 32)), (f32, (8,)), (b16, (4, 8)), (f32, (4,)), (u8, (4096,))]),
    "expand_shard_scales": (lambda s, b: w8.expand_shard_scales(s, [2, 3], b), [(f32, (2,)), (f32, (5,))]),
    "requant_shards": (lambda q, s, o, t: w8.requant_shards(q, s, [2, 2], o, t), [(i8, (4, 32)), (f32, (2,)), (i8, (4, 32)), (f32, (1,))]),
    "fp8_kv_decode_attention": (lambda q, k, v, n, ks, vs, o, t, w: w8.fp8_kv_decode_attention(q, k, v, n, ks, vs, o, block_table=t, workspace=w),
                                [(b16, (2, 4, 128)), (u8, (9, 16, 2, 128)), (u8, (9, 16, 2, 128)), (pretend, (2,)), (f32, (1,)),
                                 (f32, (1,)), (b16, (2, 4, 128)), (pretend, (2, 5)), (u8, (4096,))]),
    "kv4_cache_write": (w8.kv4_cache_write, [(b16, (3, 2, 64)), (b16, (3, 2, 64)), (u8, (3, 2, 1, 1152)), (i64, (3,)), (f32, (1,)), (f32, (1,))]),
    "kv4_cache_read": (w8.kv4_cache_read, [(u8, (3, 2, 1, 1152)), (i64, (3,)), (f32, (1,)), (f32, (1,)), (b16, (3, 2, 64)), (b16, (3, 2, 64))]),
    "build_block_tables": (lambda c, n, f, k, t, *rest: w8.build_block_tables(c, n, f, k, t, 16, *rest),
                           [(pretend, (2,)), (pretend, (2,)), (pretend, (9,)), (pretend, (1,)), (pretend, (2, 5)), (pretend, (3,)),
                            (pretend, (2,)), (i64, (4,)), (pretend, (4,)), (pretend, (1,)), (pretend, (1,))]),
    "kv4_attention": (lambda q, c, n, t, ks, vs, o, s, w: w8.kv4_attention(q, c, n, t, ks, vs, o, query_start=s, workspace=w),
                      [(b16, (2, 4, 64)), (u8, (3, 2, 1, 1152)), (pretend, (2,)), (pretend, (2, 5)), (f32, (1,)), (f32, (1,)),
                       (b16, (2, 4, 64)), (pretend, (3,)), (u8, (4096,))]),
    "verify_drafts": (w8.verify_drafts, [(f32, (5, 9)), (f32, (3, 9)), (pretend, (3,)), (pretend, (3,)), (f32, (3,)), (f32, (2,)),
                                         (pretend, (2, 4)), (pretend, (2,))]),
}


@pytest.mark.parametrize("entry", ENTRIES)
def test_every_tensor_has_to_be_on_the_current_device(world, entry):
    call, tensors = ENTRIES[entry]
    make = lambda at, index: [m(*n, index=index if i == at or at is None else 0) for i, (m, n) in enumerate(tensors)]  # noqa: E731
    call(*make(None, 0))
    assert len(world.calls) == 1
    for i in range(len(tensors)):
        with pytest.raises(ValueError, match="one device"):
            call(*make(i, 1))
    with pytest.raises(ValueError, match="current device"):
        call(*make(None, 1))
    assert len(world.calls) == 1                              # nothing was launched
    world.device = 1
    call(*make(None, 1))
    assert len(world.calls) == 2


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_has_to_be_of_the_current_device(world, call):
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream(61, index=1))
    assert not world.calls


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("gpus", [1, 2])
def test_no_tensor_of_the_host(world, monkeypatch, entry, gpus):
    monkeypatch.setattr(api, "_gpus", lambda: gpus)
    call, tensors = ENTRIES[entry]
    make = lambda at: [m(*n).as_subclass(torch.Tensor) if i == at else m(*n) for i, (m, n) in enumerate(tensors)]  # noqa: E731
    call(*make(None))
    for i in range(len(tensors)):
        with pytest.raises(ValueError, match="CUDA"):
            call(*make(i))
    assert len(world.calls) == 1


@pytest.mark.parametrize("call", [c for c in CALLS if c is not quantise])
def test_a_workspace_made_on_another_stream_is_waited_for_once(world, call):
    ws = w8.Workspace(4096, device="cuda:0")                 # zeroed on stream 7
    assert world.events == [7]
    for _ in range(2):
        call(stream=Stream(71), workspace=ws)
    world.current = 72
    call(workspace=ws)
    assert world.waits == [(71, 0), (72, 0)]
    assert {handle for _, handle in world.kept} == {71, 72}   # freed only behind what runs there
    world.current = 7
    call(workspace=ws)
    assert len(world.waits) == 2
    world.captured, world.current = {73}, 73
    call(workspace=ws)                                        # no wait for what lies outside the capture
    assert len(world.waits) == 2
