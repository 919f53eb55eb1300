"""What a caller gives beside a call's inputs -- workspace, status word -- is
checked before anything is launched.  On the host: stand-ins for the tensors,
and a launch that only records that it was reached."""
import pytest
import torch

import shared_prefix_attention_b200 as psa
from shared_prefix_attention_b200 import _binding as B

DEV = torch.device("cuda", 0)
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Given:
    """As much of a CUDA tensor as the binding asks for."""

    def __init__(self, *shape, dtype=BF16, device=DEV, dense=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.dense = dense

    is_cuda = property(lambda self: self.device.type == "cuda")

    def stride(self):
        out = [1]
        for n in self.shape[:0:-1]:
            out.insert(0, out[0] * n)
        return tuple(out[:len(self.shape)])

    def is_contiguous(self):
        return self.dense

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


N, HQ, HKV, D = 4, 8, 2, 128


def chunk(**kw):
    _, info = psa.build_chunk_plan([N], [N], HQ, HKV, D)
    plan = psa.ChunkPlan(info, Given(int(info.len), dtype=I32), 256)
    kv = Given(N, HKV, D)
    return psa.chunk(Given(N, HQ, D), kv, kv, plan, 0.1, out=Given(N, HQ, D),
                     lse=Given(N, HQ, dtype=F32), **{"workspace": Given(256, dtype=U8), **kw})


def gradients(**kw):
    q, k = Given(N, HQ, D), Given(N, HKV, D)
    return psa.qk_norm_rope_bwd(q, k, q, k, None, None, dq=q, dk=k,
                                **{"workspace": Given(1 << 20, dtype=U8), **kw})


def forward(**kw):
    q, k = Given(N, HQ, D), Given(N, HKV, D)
    return psa.qk_norm_rope(q, k, None, None, q_out=q, k_out=k, **kw)


def append(**kw):
    k = Given(N, HKV, D)
    return psa.cache_append(None, k, k, k, k, Given(N, dtype=I32), **kw)


def read(**kw):
    k = Given(N, HKV, D)
    return psa.cache_read(k, k, Given(N, dtype=I32), k=k, v=k, **kw)


BAD_STATUS = [Given(1, dtype=I32, device="cpu"), Given(1, dtype=I32, device="cuda:1"),
              Given(1, dtype=torch.int64), Given(1, dtype=torch.float16), Given(0, dtype=I32)]
BAD_WORKSPACE = [Given(1 << 20, dtype=U8, device="cpu"), Given(1 << 20, dtype=U8, device="cuda:1"),
                 Given(1 << 20, dtype=U8, dense=False), Given(1 << 20, dtype=F32)]


@pytest.fixture
def launched(monkeypatch):
    names = []
    monkeypatch.setattr(B, "_launch", lambda name, device, *args: names.append(name))
    return names


@pytest.mark.parametrize("call", [chunk, gradients, forward, append, read])
def test_layer_calls_check_the_status_word(call, launched):
    for bad in BAD_STATUS:
        with pytest.raises(ValueError, match="status"):
            call(status=bad)
    assert not launched
    call()
    call(status=Given(1, dtype=I32))
    call(status=Given(3, 2, dtype=I32))
    assert len(launched) == 3


@pytest.mark.parametrize("call", [chunk, gradients])
def test_layer_calls_check_the_workspace(call, launched):
    for bad in BAD_WORKSPACE:
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    assert not launched
    call()
    assert len(launched) == 1


# ---------------------------------------------------------------- the other attention calls

class Lib:
    """Stands for the loaded library: sizes are 256, calls are recorded."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            if name.endswith("_size") or name.endswith("_splits"):
                return 256
            self.calls.append(name)
            return psa.PSA_OK
        return fn


@pytest.fixture
def library(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_stream", lambda device: None)
    return lib


Q, KV, ROW = Given(N, HQ, D), Given(N, HKV, D), Given(N + 1, dtype=I32)
OUT = dict(out=Q, lse=Given(N, HQ, dtype=F32))
OUT_WS = dict(OUT, workspace=Given(1 << 20, dtype=U8))
GRADS = dict(dq=Q, dk=KV, dv=KV, workspace=Given(1 << 20, dtype=U8))
IDX, MASK = Given(N, dtype=I32), Given(N, N, dtype=U8)
OLDER = {
    "prefill": (lambda **kw: psa.prefill(Q, KV, KV, ROW, 0.1, **kw), OUT_WS),
    "prefill_bwd": (lambda **kw: psa.prefill_bwd(Q, KV, KV, Q, ROW, Q, (ROW, ROW), 0.1, **kw), GRADS),
    "verify": (lambda **kw: psa.verify(Q, KV, KV, KV, KV, ROW, 4, 0.1, 2, 1, **kw),
               dict(OUT_WS, kv_indices=IDX)),
    "verify_noalloc": (lambda **kw: psa.verify_noalloc(Q, KV, KV, KV, KV, ROW, 4, 0.1, 2, 1, **kw),
                       OUT),
    "verify_tree": (lambda **kw: psa.verify_tree(Q, KV, KV, KV, KV, ROW, 4, MASK, 0.1, 2, 1, **kw),
                    dict(OUT_WS, kv_indices=IDX)),
    "verify_extend": (lambda **kw: psa.verify_extend(Q, KV, KV, KV, KV, ROW, 4, ROW, 4, 0.1, nsplit=1,
                                                     **kw),
                      dict(OUT_WS, kv_indices=IDX, draft_mask=MASK, mask_indptr=ROW)),
    "verify_fp8": (lambda **kw: psa.verify_fp8(Q, KV, KV, KV, KV, 1.0, 1.0, ROW, 4, 0.1, 2, 1, **kw),
                   dict(OUT_WS, kv_indices=IDX)),
    "verify_shared": (lambda **kw: psa.verify_shared(Q, KV, KV, KV, KV, 0.1, 2, 1, **kw),
                      dict(OUT_WS, draft_mask=MASK)),
    "sparse_latent": (lambda **kw: psa.sparse_latent(Q, Given(N, D), IDX2, 0.1, **kw), OUT),
}
IDX2 = Given(N, 2, dtype=I32)


@pytest.mark.parametrize("name", OLDER)
def test_attention_calls_check_given_buffers(name, library):
    """Outputs, workspaces, tables, masks and status words on the host or
    strided are refused, one at a time; as they should be, the call goes out."""
    call, good = OLDER[name]
    for key, t in good.items():
        for bad in (Given(*t.shape, dtype=t.dtype, device="cpu"),
                    Given(*t.shape, dtype=t.dtype, dense=False)):
            with pytest.raises(ValueError):
                call(**{**good, key: bad})
    for bad in BAD_STATUS:
        with pytest.raises(ValueError, match="status"):
            call(**good, status=bad)
    assert not library.calls
    call(**good)
    call(**good, status=Given(1, dtype=I32))
    assert len(library.calls) == 2
