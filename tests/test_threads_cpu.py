"""Host threads that share a handle: a call's kernels are enqueued one after the other on the stream and share a
workspace, so no two calls on the same workspace may be inside the library at once.  On the CPU, with the library's
entry point replaced by one that looks for that."""
import contextlib
import threading
import time

import pytest

import bit_block_quantized_qm_gb300 as qm
from bit_block_quantized_qm_gb300 import build as qm_build

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    """A CPU tensor that the binding's checks take for a CUDA tensor."""
    is_cuda = True


def on_gpu(*shape, dtype):
    return torch.Tensor._make_subclass(OnGpu, torch.zeros(shape, dtype=dtype))


class Watch:
    """The library, with an entry point that only notes which workspaces are in use at once."""

    def __init__(self, lib, name, struct, place):
        self.lib, self.struct, self.place = lib, struct, place
        self.lock, self.inside, self.met, self.calls = threading.Lock(), [], False, 0
        setattr(self, name, self.enter)

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def enter(self, handle, args, stream):
        ws = self.struct.unpack(args)[self.place]
        with self.lock:
            self.met |= ws in self.inside
            self.inside.append(ws)
            self.calls += 1
        time.sleep(0.02)
        with self.lock:
            self.inside.remove(ws)
        return qm.QM_OK


@pytest.fixture
def patched(monkeypatch):
    qm_build.build()
    lib = qm.load_library()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(qm, "_on_stream", lambda device, handle: contextlib.nullcontext())
    monkeypatch.setattr(qm, "_stream_handle", lambda stream: 7 if stream is None else stream)

    def watch(*args):
        w = Watch(lib, *args)
        monkeypatch.setattr(qm, "load_library", lambda: w)
        return w
    return watch


def run(call, n=4, times=4):
    errors = []

    def work():
        try:
            for _ in range(times):
                call()
        except Exception as e:  # noqa: BLE001 (shown by the assertion)
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_experts_of_two_threads(patched):
    w = patched("qm_experts_q4_0", qm._EXPERTS_ARGS, 4)
    up, down = on_gpu(3, 64, 36, dtype=torch.uint8), on_gpu(3, 64, 36, dtype=torch.uint8)
    experts = qm.Experts(up, up, down)
    x, ids, weights = on_gpu(5, 64, dtype=torch.float32), on_gpu(5, 2, dtype=torch.int32), on_gpu(5, 2, dtype=torch.float32)
    out = on_gpu(5, 64, dtype=torch.float32)
    run(lambda: qm.qm_experts_q4_0(experts, x, ids, weights, out=out))
    assert w.calls == 16 and not w.met
    assert len(experts._workspaces) == 1


def test_attention_of_two_threads(patched):
    w = patched("qm_attn_q4_0", qm._ATTN_ARGS, 5)
    pages = [on_gpu(9, 1, qm.kv_page_bytes(64, 64), dtype=torch.uint8) for _ in range(2)]
    cache = qm.KVCache(*pages, on_gpu(2, 4, dtype=torch.int32), on_gpu(2, dtype=torch.int32), head_dim=64, page_tokens=64)
    q, out = on_gpu(2, 2, 64, dtype=torch.float32), on_gpu(2, 2, 64, dtype=torch.float32)
    weights = on_gpu(2, 1, 256, dtype=torch.float32)
    run(lambda: qm.qm_attn_q4_0(cache, q, out=out, weights=weights))
    assert w.calls == 16 and not w.met
    assert len(cache._workspaces) == 1
