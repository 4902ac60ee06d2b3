"""Where the binding's own allocations go when a call names a stream: with fakes of torch's tensors and streams and of the
library, no GPU.  Scratch has to belong to the stream the kernels run on (the allocator hands a dropped block to the next
allocation of the block's stream only), and a result to that stream with its use on the current one recorded."""
import math

import pytest


class Stream:
    def __init__(self, n):
        self.cuda_stream = n

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    def __hash__(self):
        return self.cuda_stream


class Tensor:
    def __init__(self, shape, dtype, owner=None):
        self.shape, self.dtype, self.owner, self.uses = tuple(shape), dtype, owner, []
        self.is_cuda, self.device = True, "cuda:0"

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return 1

    def record_stream(self, stream):
        self.uses.append(stream)


class Host(Tensor):
    class device:
        type = "cpu"

    def __init__(self, shape, dtype):
        super().__init__(shape, dtype)
        self.is_cuda, self.device = False, Host.device


class Torch:
    """As much of torch as the binding uses; remembers what is allocated."""
    bfloat16, float32, int32, uint8 = "bfloat16", "float32", "int32", "uint8"
    Tensor = Tensor

    def __init__(self):
        self.made = made = []
        now = [Stream(7)]

        class Context:
            def __init__(self, s):
                self.s = s

            def __enter__(self):
                now.append(self.s)

            def __exit__(self, *e):
                now.pop()

        class cuda:
            stream = Context
            current_device = staticmethod(lambda: 0)
            current_stream = staticmethod(lambda device=None: now[-1])
            is_available = staticmethod(lambda: True)

        class _C:
            _cuda_getCurrentRawStream = staticmethod(lambda device: now[-1].cuda_stream)

        self.cuda, self._C = cuda, _C
        self.current = now[0]

        def empty(*shape, dtype, device=None, pin_memory=False):
            shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
            if pin_memory:
                return Host(shape, dtype)
            made.append(Tensor(shape, dtype, now[-1]))
            return made[-1]

        self.empty = empty
        self.empty_like = lambda t: empty(t.shape, dtype=t.dtype)


class Lib:
    """Every size is 4096, every call succeeds; remembers the streams that calls were given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 4096

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


def bf(*shape):
    return Tensor(shape, "bfloat16")


def calls(m):
    B, h, T = 2, 4, 16
    q, kv, f32 = bf(B, h, T, 64), bf(B, 2, T, 64), Tensor((B, h, T), "float32")
    x, w = bf(B, T, 256), bf(256, 256)
    table = {"table": bf(2, h), "bucket_starts": (0, 3)}
    host = Host((B, h, T, 64), "bfloat16")
    params = {n: w if n.startswith("w") else bf(256) for n in m.ENCODER_PARAMS}
    return {
        "sdpa_forward": lambda s: m.sdpa_forward(q, q, q, stream=s),
        "sdpa_forward_lse": lambda s: m.sdpa_forward_lse(q, q, q, stream=s),
        "sdpa_forward_host": lambda s: m.sdpa_forward_host(host, host, host, stream=s),
        "sdpa_backward": lambda s: m.sdpa_backward(q, q, q, q, q, f32, stream=s),
        "positional_encoding_add": lambda s: m.positional_encoding_add(x, stream=s),
        "encoder_layer_forward": lambda s: m.encoder_layer_forward(x, params, h, stream=s),
        "sdpa_decode_forward": lambda s: m.sdpa_decode_forward(bf(B, h, 1, 64), q, q, stream=s),
        "mha_forward": lambda s: m.mha_forward(x, x, w, w, w, w, h, stream=s),
        "mha_forward_add_layernorm": lambda s: m.mha_forward_add_layernorm(x, x, w, w, w, w, bf(256), bf(256), h, stream=s),
        "sdpa_scored_forward": lambda s: m.sdpa_scored_forward(q, kv, kv, stream=s, **table),
        "sdpa_scored_forward_lse": lambda s: m.sdpa_scored_forward_lse(q, kv, kv, stream=s, **table),
        "sdpa_scored_backward": lambda s: m.sdpa_scored_backward(q, kv, kv, q, q, f32, stream=s, **table),
        "sdpa_decode_shared_forward": lambda s: m.sdpa_decode_shared_forward(bf(B, h, 1, 64), bf(2, T, 64), bf(2, T, 64), kv, kv,
                                                                             stream=s, **table),
    }


# scratch tensors of each call: the others are results
SCRATCH = {"sdpa_forward_host": 1, "sdpa_backward": 1, "encoder_layer_forward": 1, "mha_forward": 1,
           "mha_forward_add_layernorm": 1, "sdpa_scored_forward": 1, "sdpa_scored_forward_lse": 1, "sdpa_scored_backward": 1,
           "sdpa_decode_shared_forward": 1}
NAMES = ["sdpa_forward", "sdpa_forward_lse", "sdpa_forward_host", "sdpa_backward", "positional_encoding_add",
         "encoder_layer_forward", "sdpa_decode_forward", "mha_forward", "mha_forward_add_layernorm", "sdpa_scored_forward",
         "sdpa_scored_forward_lse", "sdpa_scored_backward", "sdpa_decode_shared_forward"]


@pytest.fixture
def fakes(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import transformer_scaled_dot_softmax_gb300 as m
    torch, lib = Torch(), Lib()
    monkeypatch.setattr(m, "_torch", lambda: torch)
    monkeypatch.setattr(m, "lib", lib)
    return m, torch, lib


@pytest.mark.parametrize("name", NAMES)
def test_allocations_follow_the_named_stream(fakes, name):
    m, torch, lib = fakes
    side = Stream(9)
    result = calls(m)[name](side)
    results = [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None and t.is_cuda]
    assert lib.streams == [9]
    assert torch.made and all(t.owner == side for t in torch.made), [t.owner.cuda_stream for t in torch.made]
    assert len(torch.made) == len(results) + SCRATCH.get(name, 0)
    for t in torch.made:
        # a result may be read and dropped on the current stream; scratch is dropped as the call returns
        assert t.uses == ([torch.current] if any(t is r for r in results) else [])


@pytest.mark.parametrize("name", NAMES)
def test_allocations_without_a_stream_are_the_current_ones(fakes, name):
    m, torch, lib = fakes
    calls(m)[name](None)
    calls(m)[name](torch.current)
    assert lib.streams == [7, 7]
    assert all(t.owner == torch.current and not t.uses for t in torch.made)
