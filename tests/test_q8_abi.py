"""CPU checks of the 8-bit cache's entry points: struct layout, and refusals made on the host
before any launch (no call here touches a GPU: addresses are fakes)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kdt():
    from speculative_decoding_tree_absorb_gb300 import build_lib
    build_lib.build()
    import speculative_decoding_tree_absorb_gb300 as k
    return k


def _layout(struct, ctype, tmp_path):
    fields = [f[0] for f in struct._fields_]
    body = "\n".join(f'printf("{f} %zu\\n", offsetof({ctype}, {f}));' for f in fields)
    prog = tmp_path / "layout.c"
    prog.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kdt.h"\n'
                    f'int main(void) {{ printf("size %zu\\n", sizeof({ctype}));\n{body}\nreturn 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(prog), "-o",
                    str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(struct)
    for f in fields:
        assert int(out[f]) == getattr(struct, f).offset, f


def test_struct_layouts(kdt, tmp_path):
    _layout(kdt.LatentWriteArgs, "kdt_latent_write_args", tmp_path)
    _layout(kdt.VerifyQ8Args, "kdt_verify_q8_args", tmp_path)


def _write(kdt, **kw):
    a = kdt.LatentWriteArgs(2, 9, 512, 64, 1, 0x10000, 576, 0x10400, 576, None, 1e-6, 0x20000, 10000.0, 0x30000, None,
                            0x40000, 0x50000, 0x60000, 100)
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_latent_write_q8(ctypes.byref(a), None)


def test_write_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_latent_write_q8(None, None) == K.KDT_ERR_NULL_ARG
    for kw in (dict(D_c=256), dict(D_r=32), dict(dtype=2), dict(dtype=-1)):
        assert _write(kdt, **kw) == K.KDT_ERR_UNSUPPORTED, kw
    for kw in (dict(B=-1), dict(T=0), dict(B=1 << 20, T=1 << 12), dict(c_row_stride=511), dict(c_row_stride=516),
               dict(k_row_stride=63), dict(kv_row_stride=0), dict(c=0x10008), dict(k=0x10401), dict(c_q8=0x40008),
               dict(c_scale=0x50001), dict(k_pe=0x60002), dict(pos=0x20002), dict(prefix_len=0x30001),
               dict(n_rows=0x30002), dict(gamma=0x70008), dict(gamma=0x70000, eps=float("nan")),
               dict(gamma=0x70000, eps=-1.0), dict(base=0.0), dict(base=float("nan"))):
        assert _write(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in ("c", "k", "prefix_len", "c_q8", "c_scale", "k_pe"):
        assert _write(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _write(kdt, B=0) == K.KDT_OK


def test_read_and_compact_refusals(kdt):
    K, lib = kdt.kdt, kdt.lib()

    def read(c8=0x10000, sc=0x20000, kp=0x30000, L=100, B=2, R=9, start=0x40000, n=None, dt=1, c=0x50000, k=0x60000):
        return lib.kdt_latent_read_q8(c8, sc, kp, L, B, R, start, n, dt, c, k, None)

    for kw in (dict(L=0), dict(B=-1), dict(R=-1), dict(B=1 << 20, R=1 << 12), dict(c8=0x10008), dict(sc=0x20004),
               dict(kp=0x30002), dict(c=0x50004), dict(k=0x60004), dict(start=0x40002), dict(n=0x40001)):
        assert read(**kw) == K.KDT_ERR_BAD_SHAPE, kw
    assert read(dt=3) == K.KDT_ERR_UNSUPPORTED
    for kw in (dict(c8=None), dict(sc=None), dict(kp=None), dict(c=None, k=None)):
        assert read(**kw) == K.KDT_ERR_NULL_ARG, kw
    assert read(B=0) == K.KDT_OK and read(R=0) == K.KDT_OK

    def compact(c8=0x10000, sc=0x20000, kp=0x30000, B=2, T=9, L=100, pre=0x40000, acc=0x50000, n=0x60000):
        return lib.kdt_kv_compact_q8(c8, sc, kp, B, T, L, pre, acc, n, 1, None)

    for kw in (dict(B=-1), dict(T=0), dict(T=4097, L=9999), dict(L=8), dict(c8=0x10008), dict(sc=0x20008),
               dict(kp=0x30008)):
        assert compact(**kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in (dict(c8=None), dict(sc=None), dict(kp=None), dict(pre=None), dict(acc=None), dict(n=None)):
        assert compact(**kw) == K.KDT_ERR_NULL_ARG, kw
    assert compact(B=0) == K.KDT_OK


def _verify(kdt, **kw):
    a = kdt.VerifyQ8Args(2, 9, 8, 512, 64, 0x10000, 576, 0x10400, 576, 0x20000, 0x30000, 0x40000, 100, 0x50000, 46, 0x60000,
                         None, 0.07, 0x70000, 1, 0x80000, None, 0, 0)
    ws = kw.pop("ws", (None, 0))
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_verify_attn_q8(ctypes.byref(a), ws[0], ws[1], None)


def test_verify_q8_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_verify_attn_q8(None, None, 0, None) == K.KDT_ERR_NULL_ARG
    for kw in (dict(D_c=256), dict(D_r=32), dict(out_dtype=2), dict(impl=1), dict(impl=3), dict(impl=5), dict(impl=-1)):
        assert _verify(kdt, **kw) == K.KDT_ERR_UNSUPPORTED, kw
    for kw in (dict(B=-1), dict(B=65536), dict(T=0), dict(T=4097), dict(H=0), dict(H=1025), dict(max_kv_len=8),
               dict(max_kv_len=101), dict(num_splits=-1), dict(q_nope=0x10008), dict(q_pe=0x10402), dict(c_q8=0x20008),
               dict(c_scale=0x30004), dict(k_pe=0x40002), dict(out=0x70008), dict(lse=0x80002), dict(prefix_len=0x50002),
               dict(parent=0x60001), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_nope_row_stride=504),
               dict(q_nope_row_stride=516), dict(q_pe_row_stride=56), dict(q_pe_row_stride=68)):
        assert _verify(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in ("q_nope", "q_pe", "c_q8", "c_scale", "k_pe", "prefix_len", "out", "parent"):
        assert _verify(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _verify(kdt, vis=0x90000) == K.KDT_ERR_NULL_ARG                      # both mask inputs
    assert kdt.verify_attn_q8_workspace_size(2, 32, 8, 69, impl="q8_rows", num_splits=1) == 0
    need = kdt.verify_attn_q8_workspace_size(2, 33, 8, 70, impl="q8_rows", num_splits=1)   # the visibility bits
    assert need > 0
    kw = dict(T=33, max_kv_len=70, impl=4, num_splits=1)
    assert _verify(kdt, **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, ws=(0x100000, need - 1), **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, ws=(0x100010, need), **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, B=0) == K.KDT_OK


def test_verify_q8_plan(kdt):
    p = kdt.verify_attn_q8_plan(2, 9, 8, 46, impl="q8_rows")
    # 72 rows a sequence are two 64-row tiles of one 128-key block each: nothing to cut
    assert p["impl"] == "q8_rows" and p["ctas"] == 4 and p["num_launches"] == 1 and p["workspace_bytes"] == 0
    p = kdt.verify_attn_q8_plan(2, 33, 2, 70, impl="q8_rows")      # more than 32 nodes: a kernel finds the visibility
    assert p["ctas"] == 4 and p["num_launches"] == 2 and 2 * 33 * 2 * 4 <= p["workspace_bytes"] <= 768
    p = kdt.verify_attn_q8_plan(2, 9, 8, 129, impl="q8_rows")
    assert p["ctas"] == 8 and p["num_launches"] == 2 and p["workspace_bytes"] >= 2 * 8 * 64 * 513 * 4
    # the work chooses the kernel: 64 heads of one token, of a tree, of a tree over a short cache
    assert kdt.verify_attn_q8_plan(4, 1, 64, 5000)["impl"] == "q8_rows"
    p = kdt.verify_attn_q8_plan(4, 64, 64, 5000)
    assert p["impl"] == "tcgen05" and p["ctas"] == 4 * p["num_splits"]
    assert kdt.verify_attn_q8_plan(2, 64, 64, 164)["impl"] == "q8_rows"
    p = kdt.verify_attn_q8_plan(2, 9, 8, 46, impl="q8_rows", num_splits=1, bits=True)
    assert p["ctas"] == 1 and p["num_launches"] == 1 and p["workspace_bytes"] == 0
    with pytest.raises(kdt.KdtError):
        kdt.verify_attn_q8_plan(2, 0, 8, 46)


def test_binding_refuses_wrong_tensors(kdt):
    import torch
    c8, sc = torch.zeros(2, 8, 512, dtype=torch.uint8), torch.zeros(2, 8, 16, dtype=torch.uint8)
    kp = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    pre = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros(2, 3, 576)
    bad = [dict(c=kv[..., :511]), dict(k=kv[..., 512:].to(torch.bfloat16)), dict(c_q8=c8[:, ::2]), dict(c_scale=sc[..., :8]),
           dict(k_pe=kp.float()), dict(prefix_len=pre.long()), dict(pos=torch.zeros(2, 3)), dict(gamma=torch.zeros(511)),
           dict(gamma=torch.zeros(512, dtype=torch.bfloat16)), dict(n_rows=torch.zeros(3, dtype=torch.int32)),
           dict(c=kv.transpose(0, 1)[..., :512])]
    for kw in bad:
        args = dict(c=kv[..., :512], k=kv[..., 512:], c_q8=c8, c_scale=sc, k_pe=kp, prefix_len=pre)
        args.update(kw)
        with pytest.raises(ValueError):
            kdt.latent_write_q8(**args)
    with pytest.raises(TypeError):
        kdt.latent_write_q8(kv[..., :512].half(), kv[..., 512:].half(), c8, sc, kp, pre)
    with pytest.raises(ValueError):
        kdt.latent_read_q8(c8, sc, kp, pre, 4, out_c=torch.zeros(2, 5, 512))
    with pytest.raises(ValueError):
        kdt.kv_compact_q8(c8, sc, kp, pre.long(), torch.zeros(2, 3, dtype=torch.int32), pre)


def test_verify_q8_binding_refuses_wrong_tensors(kdt):
    import torch
    c8, sc = torch.zeros(2, 8, 512, dtype=torch.uint8), torch.zeros(2, 8, 16, dtype=torch.uint8)
    kp = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    pre, par = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    for kw in (dict(q_nope=q[..., :511]), dict(q_pe=q[:1, ..., 512:]), dict(parent=par.long()), dict(prefix_len=pre[:1]),
               dict(out=torch.zeros(2, 3, 4, 512), out_dtype=torch.bfloat16), dict(out=torch.zeros(2, 3, 4, 511)),
               dict(lse=torch.zeros(2, 3, 4, dtype=torch.float64)), dict(vis=torch.zeros(2, 3, 2, dtype=torch.int32)),
               dict(k_pe=kp[:, :, :32]), dict(q_nope=q.transpose(1, 2)[..., :512].transpose(1, 2)[:, ::2])):
        args = dict(q_nope=q[..., :512], q_pe=q[..., 512:], c_q8=c8, c_scale=sc, k_pe=kp, prefix_len=pre, parent=par)
        args.update(kw)
        with pytest.raises(ValueError):
            kdt.verify_attn_q8(**args)
    with pytest.raises(TypeError):
        kdt.verify_attn_q8(q[..., :512].float(), q[..., 512:].float(), c8, sc, kp, pre, parent=par)


def test_tree_sample_refusals(kdt):
    K = kdt.kdt

    def call(parent=0x10000, tok=0x20000, logits=0x30000, dt=1, B=2, T=9, V=1000, stride=0, temp=1.0, un=0x40000,
             ub=0x50000, acc=0x60000, n=0x70000, bonus=0x80000, logp=None, err=None):
        return kdt.lib().kdt_tree_sample(parent, tok, logits, dt, B, T, V, stride, temp, un, ub, acc, n, bonus, logp, err,
                                         None)

    for kw in (dict(B=-1), dict(B=65536), dict(T=0), dict(T=4097), dict(V=0), dict(V=524289), dict(stride=999),
               dict(temp=0.0), dict(temp=-1.0), dict(temp=float("nan")), dict(temp=1e-4), dict(temp=1e4),
               dict(logits=0x30001), dict(dt=0, logits=0x30002), dict(un=0x40002), dict(acc=0x60001), dict(logp=0x90002),
               dict(err=0x90001)):
        assert call(**kw) == K.KDT_ERR_BAD_SHAPE, kw
    assert call(dt=2) == K.KDT_ERR_UNSUPPORTED
    for kw in ("parent", "tok", "logits", "un", "ub", "acc", "n", "bonus"):
        assert call(**{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert call(B=0) == K.KDT_OK
    import torch
    par, u = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    lg = torch.zeros(2, 3, 10)
    for kw in (dict(logits=lg[:1]), dict(tok=par.long()), dict(u_node=u.double()), dict(u_bonus=u), dict(logits=lg[..., ::2])):
        args = dict(parent=par, tok=par, logits=lg, u_node=u, u_bonus=u[:, 0].contiguous())
        args.update(kw)
        with pytest.raises(ValueError):
            kdt.tree_sample(**args)


def test_expanded_views_are_refused(kdt):
    """One row shown as many has a row stride of 0 (rows that overlap: one below their width), which the
    library would read as "contiguous": from memory that holds a single row."""
    import torch
    bf = torch.bfloat16
    c8, sc = torch.zeros(2, 8, 512, dtype=torch.uint8), torch.zeros(2, 8, 16, dtype=torch.uint8)
    kp, pre = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    c, k = torch.zeros(2, 3, 512), torch.zeros(2, 3, 64)
    one = torch.zeros(1, 1, 576)
    for kw in (dict(c=one[..., :512].expand(2, 3, 512)), dict(k=one[..., 512:].expand(2, 3, 64)),
               dict(c=torch.zeros(5 * 256 + 512).as_strided((2, 3, 512), (768, 256, 1))),
               dict(k=torch.zeros(400).as_strided((2, 3, 64), (96, 32, 1)))):
        with pytest.raises(ValueError):
            kdt.latent_write_q8(**{**dict(c=c, k=k, c_q8=c8, c_scale=sc, k_pe=kp, prefix_len=pre), **kw})
    with pytest.raises(ValueError):                                  # one sequence: only the row stride tells
        kdt.latent_write_q8(one[..., :512].expand(1, 3, 512), k[:1], c8[:1], sc[:1], kp[:1], pre[:1])
    par, u = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    row = torch.zeros(1, 1, 10)
    for lg, b in ((row.expand(2, 3, 10), 2), (row.expand(1, 3, 10), 1), (row.expand(2, 1, 10), 2)):
        t = lg.shape[1]
        with pytest.raises(ValueError):
            kdt.tree_sample(par[:b, :t].contiguous(), par[:b, :t].contiguous(), lg, u[:b, :t].contiguous(), u[:b, 0].contiguous())
    q, par = torch.zeros(2, 3, 4, 576, dtype=bf), torch.zeros(2, 3, dtype=torch.int32)
    q1 = q[:1, :1, :1]
    for kw in (dict(q_nope=q1[..., :512].expand(2, 3, 4, 512)), dict(q_pe=q1[..., 512:].expand(2, 3, 4, 64))):
        args = {**dict(q_nope=q[..., :512], q_pe=q[..., 512:]), **kw}
        with pytest.raises(ValueError):
            kdt.verify_attn_q8(args["q_nope"], args["q_pe"], c8, sc, kp, pre, parent=par)
        with pytest.raises(ValueError):
            kdt.make_args(args["q_nope"], args["q_pe"], torch.zeros(2, 8, 512, dtype=bf), kp, pre, parent=par)
    # single rows and slices of a combined buffer are taken as they lie
    from speculative_decoding_tree_absorb_gb300.kdt import _row_stride, _row_stride3
    assert _row_stride3(one[..., :512], "c") == 512 and _row_stride3(torch.zeros(2, 3, 576)[..., :512], "c") == 576
    assert _row_stride3(torch.zeros(2, 3, 576)[:, 1:2, :512], "c") == 3 * 576
    assert _row_stride(q[..., :512]) == 576 and _row_stride(q1[..., :512]) == 0


class _FakeLib:
    """Entry points that succeed and compute nothing."""

    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("_size") else (lambda *a: 0)


def test_tensors_made_here_are_kept_for_the_stream_they_are_used_on(kdt, monkeypatch):
    """With ``stream=`` the call's own workspace and outputs belong to the current stream's allocator: each
    is recorded on the stream that uses it, or their memory could be handed out while it still runs."""
    import torch
    from types import SimpleNamespace
    kept = []
    monkeypatch.setattr(kdt.kdt, "lib", _FakeLib)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append((self.data_ptr(), s)))
    side = SimpleNamespace(cuda_stream=0x99)
    B, T, H, V, bf = 2, 3, 4, 10, torch.bfloat16
    made, plain = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(plain(*a, **k)) or made[-1])
    c8, sc = torch.zeros(B, 8, 512, dtype=torch.uint8), torch.zeros(B, 8, 16, dtype=torch.uint8)
    kp, i32 = torch.zeros(B, 8, 64, dtype=bf), torch.zeros(B, T, dtype=torch.int32)
    q, u = torch.zeros(B, T, H, 576, dtype=bf), torch.zeros(B, T)
    pre, o, lse = i32[:, 0].contiguous(), torch.zeros(B, T, H, 512), torch.zeros(B, T, H)
    calls = [
        lambda s: kdt.verify_attn_q8(q[..., :512], q[..., 512:], c8, sc, kp, pre, parent=i32, stream=s),
        lambda s: kdt.verify_attn(q[..., :512], q[..., 512:], torch.zeros(B, 8, 512, dtype=bf), kp, pre, parent=i32, stream=s),
        lambda s: kdt.latent_read_q8(c8, sc, kp, None, 4, stream=s),
        lambda s: kdt.tree_sample(i32, i32, torch.zeros(B, T, V), u, u[:, 0].contiguous(), stream=s),
        lambda s: kdt.build_visibility(i32, stream=s),
        lambda s: kdt.vc_up_proj(o, torch.zeros(H, 512, 128, dtype=bf), stream=s),
        lambda s: kdt.tree_accept(i32, i32, i32, stream=s),
        lambda s: kdt.tree_build(torch.zeros(B, 2, 4, dtype=torch.int32), torch.zeros(B, 2, 4), 5, stream=s),
        lambda s: kdt.merge_attn_states(o, lse, o, lse, stream=s),
    ]
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: torch.empty(t.shape, dtype=t.dtype))
    for k, call in enumerate(calls):
        made.clear(), kept.clear()
        call(side)
        assert made and sorted(kept) == sorted((t.data_ptr(), side) for t in made), k
    mine = dict(out=o, lse=lse, workspace=torch.zeros(8192, dtype=torch.uint8))         # the caller's own: left alone
    kept.clear()
    kdt.verify_attn_q8(q[..., :512], q[..., 512:], c8, sc, kp, pre, parent=i32, stream=side, **mine)
    assert not kept


def test_lengths_near_the_end_of_32_bits_are_refused(kdt):
    """Rounded up to whole blocks they would pass 2^31: no plan with negative counts, for either cache."""
    K = kdt.kdt
    a = kdt.VerifyArgs()
    a.B, a.T, a.H, a.D_c, a.D_r, a.dtype, a.scale = 2, 3, 4, 512, 64, 1, 1.0
    for f in ("q_nope", "q_pe", "c_kv", "k_pe", "prefix_len", "parent", "out"):
        setattr(a, f, 4096)
    for n in (2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 256):
        for impl in ("auto", "q8_rows", "tcgen05"):
            with pytest.raises(kdt.KdtError) as e:
                kdt.verify_attn_q8_plan(2, 3, 4, n, impl=impl)
            assert e.value.status == K.KDT_ERR_BAD_SHAPE
        a.kv_row_stride = a.max_kv_len = n
        for a.impl in range(4):
            with pytest.raises(kdt.KdtError):
                kdt.plan(a)
    assert kdt.verify_attn_q8_plan(2, 3, 4, 2 ** 31 - 257, impl="q8_rows")["ctas"] > 0


def test_error_words_of_another_size_are_refused(kdt):
    import torch
    bf = torch.bfloat16
    c8, sc = torch.zeros(2, 8, 512, dtype=torch.uint8), torch.zeros(2, 8, 16, dtype=torch.uint8)
    kp, par, u = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    q = torch.zeros(2, 3, 4, 576, dtype=bf)
    for err in (torch.zeros(4, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError, match="err"):
            kdt.verify_attn_q8(q[..., :512], q[..., 512:], c8, sc, kp, par[:, 0].contiguous(), parent=par, err=err)
        with pytest.raises(ValueError, match="err"):
            kdt.tree_sample(par, par, torch.zeros(2, 3, 10), u, u[:, 0].contiguous(), err=err)
