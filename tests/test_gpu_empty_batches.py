"""A call over no rows leaves 0 in the error word, whatever an earlier call reported there, on the stream it is given and
inside a capture; a word that is no device memory is left alone (such a call looks at no tensor)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdt():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_absorb_gb300 import build_lib
    build_lib.build()
    import speculative_decoding_tree_absorb_gb300 as k
    return k


def _call(kdt, name, err, stream=None):
    import torch
    bf, i32 = torch.bfloat16, torch.int32

    def z(*s, dt=i32):
        return torch.zeros(*s, dtype=dt, device=err.device)
    q, none = z(0, 9, 4, 576, dt=bf), z(0)
    qn, qp = q[..., :512], q[..., 512:]
    kw = dict(err=err, stream=stream)
    if name == "page_assign":
        kdt.page_assign(z(0, 3), none, z(8), z(1) + 8, none, 8, start=none, T=2, **kw)
    elif name == "verify_attn_paged":
        kdt.verify_attn_paged(qn, qp, z(8, 16, 512, dt=bf), z(8, 16, 64, dt=bf), z(0, 3), none, parent=z(0, 9), **kw)
    elif name == "sample":
        kdt.sample(z(0, 50, dt=bf), z(0, dt=torch.float32), **kw)
    elif name == "tree_sample":
        u = z(0, 9, dt=torch.float32)
        kdt.tree_sample(z(0, 9), z(0, 9), z(0, 9, 50, dt=bf), u, z(0, dt=torch.float32), **kw)
    elif name == "tree_accept":
        kdt.tree_accept(z(0, 9), z(0, 9), z(0, 9), **kw)
    elif name == "build_visibility":
        kdt.build_visibility(z(0, 9), **kw)
    elif name == "verify_attn":
        kdt.verify_attn(qn, qp, z(0, 40, 512, dt=bf), z(0, 40, 64, dt=bf), none, parent=z(0, 9), **kw)
    elif name == "verify_attn_q8":
        u8 = torch.uint8
        kdt.verify_attn_q8(qn, qp, z(0, 40, 512, dt=u8), z(0, 40, 16, dt=u8), z(0, 40, 64, dt=bf), none, parent=z(0, 9), **kw)
    else:
        kdt.vc_up_proj(z(0, 4, 512, dt=torch.float32), z(4, 512, 128, dt=bf), **kw)


NAMES = ["page_assign", "verify_attn_paged", "sample", "tree_sample", "tree_accept", "build_visibility", "verify_attn",
         "verify_attn_q8", "vc_up_proj"]


@pytest.mark.parametrize("name", NAMES)
def test_the_error_word_is_cleared(kdt, name):
    import torch
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    _call(kdt, name, err)
    assert int(err.item()) == 0
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    err.fill_(5)
    torch.cuda.synchronize()
    _call(kdt, name, err, stream=s)
    s.synchronize()
    assert int(err.item()) == 0
    with torch.cuda.graph(graph, stream=s):
        _call(kdt, name, err)
    err.fill_(5)
    graph.replay()
    assert int(err.item()) == 0


def test_a_word_that_is_not_device_memory_is_left_alone(kdt):
    import ctypes
    import torch
    word = torch.full((1,), 7, dtype=torch.int32).pin_memory()
    a = kdt.PageArgs(0, 3, None, 0, None, None, None, 8, 8, None, None, 0, None, word.data_ptr())
    assert kdt.lib().kdt_page_assign(ctypes.byref(a), None) == 0
    torch.cuda.synchronize()
    assert int(word.item()) == 7
