"""CPU checks of the paged cache's entry points and of kdt_sample: struct layouts, refusals before any
launch, plans, and what the binding refuses (none of these calls touch a GPU)."""
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


@pytest.mark.parametrize("name,c_name", [("PageArgs", "kdt_page_args"), ("LatentWritePagedArgs", "kdt_latent_write_paged_args"),
                                         ("VerifyPagedArgs", "kdt_verify_paged_args"), ("SampleArgs", "kdt_sample_args")])
def test_struct_layouts(kdt, tmp_path, name, c_name):
    cls = getattr(kdt, name)
    body = "\n".join(f'printf("%zu\\n", offsetof({c_name}, {f[0]}));' for f in cls._fields_)
    (tmp_path / "l.c").write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kdt.h"\n'
                                  f'int main(void) {{ printf("%zu\\n", sizeof({c_name})); {body} return 0; }}')
    exe = str(tmp_path / "l")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(tmp_path / "l.c"), "-o", exe],
                   check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]


def _assign(kdt, **kw):
    a = kdt.PageArgs(3, 5, 0x10000, 0, 0x20000, 0x30000, 0x40000, 100, 64, 0x50000, 0x60000, 7, 0x70000, 0x80000)
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_page_assign(ctypes.byref(a), None)


def test_page_assign_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_page_assign(None, None) == K.KDT_ERR_NULL_ARG
    for kw in (dict(B=-1), dict(B=16385), dict(W=0), dict(T=-1), dict(n_pages=-1), dict(page_size=0), dict(page_size=4),
               dict(page_size=48), dict(page_size=2048), dict(page_size=-64), dict(table_row_stride=4), dict(W=1 << 30),
               dict(T=1 << 30), dict(n_pages=1 << 25), dict(table=0x10002), dict(held=0x20001), dict(free_pages=0x30002),
               dict(n_free=0x40002), dict(new_len=0x50002), dict(start=0x60002), dict(slots=0x70002), dict(err=0x80002)):
        assert _assign(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in ("table", "held", "free_pages", "n_free", "new_len", "start", "slots"):
        assert _assign(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _assign(kdt, B=0) == K.KDT_OK


def _write(kdt, **kw):
    a = kdt.LatentWritePagedArgs(9, 512, 64, 1, 0x10000, 576, 0x10400, 576, 0x20000, 1e-6, 0x30000, 1e4, 0x40000, 0x50000,
                                 0x60000, 640)
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_latent_write_paged(ctypes.byref(a), None)


def test_write_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_latent_write_paged(None, None) == K.KDT_ERR_NULL_ARG
    for kw in (dict(rows=-1), dict(n_slots=-1), dict(c_row_stride=511), dict(c_row_stride=516), dict(k_row_stride=63),
               dict(eps=-1.0), dict(eps=float("nan")), dict(base=0.0), dict(base=float("inf")), dict(c=0x10008), dict(gamma=0x20004),
               dict(k=0x10401), dict(c_kv=0x50008), dict(k_pe=0x60008), dict(pos=0x30002), dict(slots=0x40002)):
        assert _write(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in (dict(D_c=256), dict(D_r=32), dict(dtype=2)):
        assert _write(kdt, **kw) == K.KDT_ERR_UNSUPPORTED, kw
    for kw in ("c", "k", "slots", "c_kv", "k_pe"):
        assert _write(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _write(kdt, rows=0) == K.KDT_OK


def test_compact_refusals(kdt):
    K, lib = kdt.kdt, kdt.lib()

    def call(c=0x10000, k=0x20000, dt=1, Dc=512, Dr=64, n=100, page=64, table=0x30000, W=5, stride=0, B=2, T=9, pre=0x40000,
             acc=0x50000, na=0x60000):
        return lib.kdt_kv_compact_paged(c, k, dt, Dc, Dr, n, page, table, W, stride, B, T, pre, acc, na, 1, None)

    for kw in (dict(B=-1), dict(T=0), dict(T=4097, W=99), dict(Dc=0), dict(Dr=-1), dict(n=0), dict(page=24), dict(W=0),
               dict(stride=4), dict(n=1 << 26), dict(W=1, page=8), dict(Dc=508), dict(Dr=4), dict(Dc=1 << 20), dict(c=0x10008),
               dict(k=0x20008), dict(table=0x30002), dict(pre=0x40001), dict(acc=0x50002), dict(na=0x60002)):
        assert call(**kw) == K.KDT_ERR_BAD_SHAPE, kw
    assert call(dt=3) == K.KDT_ERR_UNSUPPORTED
    for kw in ("c", "k", "table", "pre", "acc", "na"):
        assert call(**{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert call(B=0) == K.KDT_OK


def _verify(kdt, **kw):
    a = kdt.VerifyPagedArgs(2, 9, 8, 512, 64, 0x10000, 576, 0x10400, 576, 0x20000, 0x30000, 100, 64, 0x40000, 2, 0, 0x50000,
                            None, 46, 0x60000, None, 0.07, 0x70000, 1, 0x80000, None, 0)
    ws = kw.pop("ws", (None, 0))
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_verify_attn_paged(ctypes.byref(a), ws[0], ws[1], None)


def test_verify_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_verify_attn_paged(None, None, 0, None) == K.KDT_ERR_NULL_ARG
    for kw in (dict(D_c=256), dict(D_r=32), dict(out_dtype=2)):
        assert _verify(kdt, **kw) == K.KDT_ERR_UNSUPPORTED, kw
    for kw in (dict(B=-1), dict(B=65536), dict(T=0), dict(T=4097), dict(H=0), dict(H=1025), dict(max_kv_len=8),
               dict(max_kv_len=129), dict(num_splits=-1), dict(page_size=4), dict(page_size=65), dict(page_size=2048),
               dict(n_pages=0), dict(n_pages=1 << 25), dict(table_width=0), dict(table_row_stride=1),
               dict(B=8192, T=4096, H=1024, table_width=99, max_kv_len=4100), dict(q_nope=0x10008), dict(q_pe=0x10402),
               dict(c_kv=0x20008), dict(k_pe=0x30008), dict(out=0x70008), dict(lse=0x80002), dict(prefix_len=0x50002),
               dict(n_rows=0x90002), dict(table=0x40002), dict(parent=0x60001), dict(err=0x90001), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q_nope_row_stride=504), dict(q_nope_row_stride=516), dict(q_pe_row_stride=56),
               dict(q_pe_row_stride=68)):
        assert _verify(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    for kw in ("q_nope", "q_pe", "c_kv", "k_pe", "table", "prefix_len", "out", "parent"):
        assert _verify(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _verify(kdt, vis=0x90000) == K.KDT_ERR_NULL_ARG                      # both mask inputs
    need = kdt.verify_attn_paged_workspace_size(2, 33, 8, 70, 64)               # the visibility bits at least
    assert need > 0
    kw = dict(T=33, max_kv_len=70)
    assert _verify(kdt, **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, ws=(0x100000, need - 1), **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, ws=(0x100010, need), **kw) == K.KDT_ERR_WORKSPACE
    assert _verify(kdt, B=0) == K.KDT_OK
    with pytest.raises(kdt.KdtError):
        kdt.verify_attn_paged_plan(2, 0, 8, 46, 64)
    assert kdt.verify_attn_paged_plan(2, 1, 8, 46, 64)["num_launches"] >= 1


def _sample(kdt, **kw):
    a = kdt.SampleArgs(2, 1000, 0x10000, 1, 0, 0x20000, None, 1.0, None, 0, None, 1.0, None, 0.0, 0x30000, 0x40000, 0x50000)
    for k, v in kw.items():
        setattr(a, k, v)
    return kdt.lib().kdt_sample(ctypes.byref(a), None)


def test_sample_refusals(kdt):
    K = kdt.kdt
    assert kdt.lib().kdt_sample(None, None) == K.KDT_ERR_NULL_ARG
    nan = float("nan")
    for kw in (dict(R=-1), dict(V=0), dict(V=524289), dict(row_stride=999), dict(temperature_all=-1.0), dict(temperature_all=nan),
               dict(temperature_all=1e-4), dict(temperature_all=1e4), dict(top_p_all=nan), dict(min_p_all=nan),
               dict(logits=0x10001), dict(dtype=0, logits=0x10002), dict(u=0x20002), dict(temperature=0x60001),
               dict(top_k=0x60002), dict(top_p=0x60002), dict(min_p=0x60002), dict(token=0x30001), dict(logp=0x40002),
               dict(err=0x50002)):
        assert _sample(kdt, **kw) == K.KDT_ERR_BAD_SHAPE, kw
    assert _sample(kdt, dtype=2) == K.KDT_ERR_UNSUPPORTED
    for kw in ("logits", "u", "token"):
        assert _sample(kdt, **{kw: None}) == K.KDT_ERR_NULL_ARG, kw
    assert _sample(kdt, R=0, err=None) == K.KDT_OK


def test_binding_refuses_wrong_tensors(kdt):
    import torch
    i32, bf = torch.int32, torch.bfloat16
    c, k = torch.zeros(6, 16, 512, dtype=bf), torch.zeros(6, 16, 64, dtype=bf)
    table, pre = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    free, one = torch.zeros(6, dtype=i32), torch.zeros(1, dtype=i32)

    def refused(fn, good, bad, error=ValueError):
        for kw in bad:
            with pytest.raises(error):
                fn(**{**good, **kw})

    refused(kdt.page_assign, dict(table=table, held=pre, free_pages=free, n_free=one, new_len=pre, page_size=16, start=pre, T=2),
            [dict(table=table.long()), dict(table=table[:, ::2]), dict(table=table[:1].expand(2, 3)), dict(held=pre[:1]),
             dict(free_pages=free.long()), dict(n_free=pre), dict(new_len=pre.float()), dict(start=None),
             dict(start=torch.zeros(3, dtype=i32)), dict(slots=torch.zeros(2, 3, dtype=i32))])
    kv = torch.zeros(2, 3, 576)
    slots = torch.zeros(2, 3, dtype=i32)
    good = dict(c=kv[..., :512], k=kv[..., 512:], c_kv=c, k_pe=k, slots=slots)
    refused(kdt.latent_write_paged, good,
            [dict(c=kv[..., :511]), dict(k=kv[..., 512:].to(bf)), dict(c_kv=c[:, ::2]), dict(c_kv=c.float()), dict(k_pe=k[:5]),
             dict(slots=slots.long()), dict(slots=None), dict(pos=pre), dict(gamma=torch.zeros(511)),
             dict(c=kv[:1, :, :512].expand(2, 3, 512))])
    refused(kdt.latent_write_paged, {**good, "c": kv[..., :512].half(), "k": kv[..., 512:].half()}, [{}], TypeError)
    refused(kdt.kv_compact_paged, dict(c_kv=c, k_pe=k, table=table, prefix_len=pre, acc_nodes=slots, n_acc=pre),
            [dict(c_kv=c[:, ::2]), dict(k_pe=k.float()), dict(table=table[:1]), dict(prefix_len=pre.long()), dict(acc_nodes=slots.long()),
             dict(n_acc=one)])
    q = torch.zeros(2, 3, 4, 576, dtype=bf)
    good = dict(q_nope=q[..., :512], q_pe=q[..., 512:], c_kv=c, k_pe=k, table=table, prefix_len=pre, parent=slots)
    refused(kdt.verify_attn_paged, good,
            [dict(q_nope=q[..., :511]), dict(q_pe=q[:1, ..., 512:]), dict(table=table[:1]), dict(prefix_len=pre[:1]), dict(n_rows=one),
             dict(parent=slots.long()), dict(vis=torch.zeros(2, 3, 2, dtype=i32)), dict(c_kv=c.float()), dict(k_pe=k[..., :32]),
             dict(out=torch.zeros(2, 3, 4, 512), out_dtype=bf), dict(lse=torch.zeros(2, 3, 4, dtype=torch.float64)),
             dict(q_nope=q[:1, ..., :512].expand(2, 3, 4, 512))])
    refused(kdt.verify_attn_paged, {**good, "q_nope": q[..., :512].float(), "q_pe": q[..., 512:].float()}, [{}], TypeError)
    lg, u = torch.zeros(2, 10), torch.zeros(2)
    refused(kdt.sample, dict(logits=lg, u=u),
            [dict(u=u.double()), dict(u=u[:1]), dict(logits=lg[:, ::2]), dict(logits=lg[:1].expand(2, 10)),
             dict(temperature=u.double()), dict(top_k=u), dict(top_p=u[:1]), dict(min_p=torch.zeros(2, dtype=i32))])
    refused(kdt.sample, dict(logits=lg.half(), u=u), [{}], TypeError)


def test_numbers_that_pass_32_bits(kdt, monkeypatch):
    """ctypes drops what does not fit a C int: sizes that do not are refused, and a top-k that does not keeps all tokens."""
    import torch
    i32, bf, wrap = torch.int32, torch.bfloat16, 2 ** 32
    c, k = torch.zeros(6, 16, 512, dtype=bf), torch.zeros(6, 16, 64, dtype=bf)
    table, pre, par = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32)
    q = torch.zeros(2, 3, 4, 576, dtype=bf)
    qn, qp = q[..., :512], q[..., 512:]
    dense, dk = torch.zeros(2, 40, 512, dtype=bf), torch.zeros(2, 40, 64, dtype=bf)
    for kw in (dict(page_size=wrap + 16), dict(T=wrap + 2), dict(T=2 ** 31)):
        with pytest.raises(ValueError):
            kdt.page_assign(**{**dict(table=table, held=pre, free_pages=torch.zeros(6, dtype=i32), n_free=pre[:1], new_len=pre,
                                      page_size=16, start=pre, T=0), **kw})
    for kw in (dict(max_kv_len=wrap + 40), dict(num_splits=wrap + 1), dict(num_splits=-wrap)):
        with pytest.raises(ValueError):
            kdt.verify_attn_paged(qn, qp, c, k, table, pre, parent=par, **kw)
        with pytest.raises(ValueError):
            kdt.verify_attn(qn, qp, dense, dk, pre, parent=par, **kw)
        with pytest.raises(ValueError):
            kdt.verify_attn_paged_plan(**{**dict(B=2, T=3, H=4, max_kv_len=40, page_size=16), **kw})
        with pytest.raises(ValueError):
            kdt.verify_attn_q8_plan(**{**dict(B=2, T=3, H=4, max_kv_len=40), **kw})
    for kw in (dict(B=wrap + 2), dict(T=wrap + 3), dict(H=wrap + 4), dict(page_size=wrap + 16)):
        with pytest.raises(ValueError):
            kdt.verify_attn_paged_plan(**{**dict(B=2, T=3, H=4, max_kv_len=40, page_size=16), **kw})

    seen = []

    class Lib:
        @staticmethod
        def kdt_sample(a, stream):
            seen.append(a._obj.top_k_all)
            return 0
    monkeypatch.setattr(kdt.kdt, "lib", lambda: Lib)
    monkeypatch.setattr(kdt.kdt, "_stream_ptr", lambda s: None)
    for top_k in (wrap + 1, wrap, 2 ** 31, 2 ** 31 - 1, 10 ** 30, -wrap - 1, -2 ** 31 - 5, 0, None, 7, 7.0):
        kdt.sample(torch.zeros(2, 10), torch.zeros(2), top_k=top_k)
    assert all(v <= 0 or v >= 2 ** 31 - 1 for v in seen[:9]) and seen[9:] == [7, 7]
